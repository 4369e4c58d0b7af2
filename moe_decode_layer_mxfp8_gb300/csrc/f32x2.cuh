// Arithmetic on pairs of f32, one instruction for both.
#pragma once

namespace mono {

__device__ __forceinline__ void fma2(float& x, float& y, float a, float bx, float by) {  // x = x a + bx
  asm("{\n .reg .b64 s, m, b;\n mov.b64 s, {%0, %1};\n mov.b64 m, {%2, %2};\n mov.b64 b, {%3, %4};\n"
      " fma.rn.f32x2 s, s, m, b;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(bx), "f"(by));
}
__device__ __forceinline__ void add2(float& x, float& y, float bx, float by) {
  asm("{\n .reg .b64 s, b;\n mov.b64 s, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 s, s, b;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(bx), "f"(by));
}
__device__ __forceinline__ void sub2(float& x, float& y, float bx, float by) {  // (by an exact product)
  asm("{\n .reg .b64 s, b, m;\n mov.b64 s, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 m, {%4, %4};\n"
      " fma.rn.f32x2 s, b, m, s;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(bx), "f"(by), "f"(-1.0f));
}
__device__ __forceinline__ void mul2(float& x, float& y, float a) {
  asm("{\n .reg .b64 s, m;\n mov.b64 s, {%0, %1};\n mov.b64 m, {%2, %2};\n"
      " mul.rn.f32x2 s, s, m;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a));
}
__device__ __forceinline__ void mul2(float& x, float& y, float ax, float ay) {
  asm("{\n .reg .b64 s, m;\n mov.b64 s, {%0, %1};\n mov.b64 m, {%2, %3};\n"
      " mul.rn.f32x2 s, s, m;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(ax), "f"(ay));
}

}  // namespace mono
