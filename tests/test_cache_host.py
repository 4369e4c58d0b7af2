"""The host side of the cache operators (csrc/cache_ops.cu) on the CPU, compiled against a CUDA runtime
that only keeps books and against launches that record what they are given: no GPU is touched."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from moe_decode_layer_mxfp8_gb300 import build as mb
from moe_decode_layer_mxfp8_gb300 import cache as mc

FAKE = r"""
#include <cstring>
#include "cache_kernels.h"
using namespace mono;
extern "C" {
int shared_error;  // what the attention over shared prefixes says when it is prepared
RotateArgs rotated;
int rotated_sms;
uint8_t *attend_at, *shared_at, *evict_at;
const float* lse_at;
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
  *p = {};
  p->major = 10, p->minor = 3, p->multiProcessorCount = 152;
  return cudaSuccess;
}
size_t rope_positions_given() { return (size_t)rotated.rope_positions; }
int rotation_given() { return rotated.rope.dim; }
}
namespace mono {
size_t attend_workspace_bytes(int rows, int) { return 1000000 + 100 * (size_t)rows; }
size_t evict_workspace_bytes(int) { return 2000000; }
size_t shared_workspace_bytes(int rows, int, int, int) { return 5000000 + 1000 * (size_t)rows; }
cudaError_t attend_prepare() { return cudaSuccess; }
cudaError_t evict_prepare() { return cudaSuccess; }
cudaError_t shared_prepare() { return (cudaError_t)shared_error; }
bool evict_fits(int, int, long long) { return true; }
bool shared_fits(int, int, long long) { return true; }
cudaError_t launch_attend(const Launch&, const AttendArgs& a, uint8_t* ws, int, int) {
  attend_at = ws, lse_at = a.lse;
  return cudaSuccess;
}
cudaError_t launch_attend_shared(const Launch&, const SharedArgs&, uint8_t* ws, int, int) { shared_at = ws; return cudaSuccess; }
cudaError_t launch_evict(const Launch&, const EvictArgs&, uint8_t* ws, int, int) { evict_at = ws; return cudaSuccess; }
cudaError_t launch_rotate(const Launch&, const RotateArgs& a, int, int sms) { rotated = a, rotated_sms = sms; return cudaSuccess; }
cudaError_t launch_verify(const Launch&, const VerifyArgs&, int, int) { return cudaSuccess; }
}
"""
# the runtime's calls, and what the compiler's own start-up code asks for
RUNTIME = r"""
#include <stdlib.h>
#include <string.h>
size_t allocated, zeroed;
int freed;
char* arena;
int cudaMalloc(void** p, size_t n) { allocated = n; *p = arena = malloc(n); return 0; }
int cudaFree(void* p) { ++freed; free(p); return 0; }
int cudaMemset(void* p, int v, size_t n) { zeroed += n; memset(p, v, n); return 0; }
int cudaMemcpy(void* d, const void* s, size_t n, int kind) { (void)kind; memcpy(d, s, n); return 0; }
int cudaDeviceSynchronize(void) { return 0; }
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaSetDevice(int d) { return d; }
int cudaGetLastError(void) { return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int d) { *v = attr * d; return 0; }
void** __cudaRegisterFatBinary(void* f) { static void* h; (void)f; return &h; }
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
char __cudaInitModule(void** h) { (void)h; return 1; }
"""

A = 0x10000  # an address that is never used
SPEC = dict(n_q_heads=16, head_dim=64, kv_dim=128, block_size=64, kv_record_bytes=144)
VIEW = dict(kv_cache=A, kv_stride_block=64 * 144, kv_stride_tok=144, kv_num_blocks=4)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    at = tmp_path_factory.mktemp("host")
    (at / "fake.cu").write_text(FAKE)
    (at / "runtime.c").write_text(RUNTIME)
    jobs = [subprocess.Popen([nvcc, *mb.ARCH, "-std=c++17", "-O0", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-I", mb.CSRC,
                              "-I", os.path.join(mb.ROOT, "include"), "-c", src, "-o", str(at / obj)])
            for src, obj in ((os.path.join(mb.CSRC, "cache_ops.cu"), "ops.o"), (str(at / "fake.cu"), "fake.o"))]
    subprocess.run(["gcc", "-fPIC", "-c", str(at / "runtime.c"), "-o", str(at / "runtime.o")], check=True)
    assert [j.wait() for j in jobs] == [0, 0]
    out = str(at / "host.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", out] + [str(at / o) for o in ("ops.o", "fake.o", "runtime.o")], check=True)
    so = C.CDLL(out)
    so.mono_cache_build.argtypes = [C.POINTER(mc.CacheSpec), C.POINTER(C.c_void_p)]
    so.mono_cache_free.argtypes, so.mono_cache_free.restype = [C.c_void_p], None
    for n in ("attend", "attend_shared", "evict", "append", "rotate"):
        getattr(so, "mono_cache_" + n).argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
    so.rope_positions_given.restype = C.c_size_t
    return so


def value(lib, name, kind=C.c_size_t):
    return kind.in_dll(lib, name).value


class Handle:
    def __init__(self, lib, **kw):
        self.lib, self.h = lib, C.c_void_p()
        spec = mc.CacheSpec(**dict(dict(SPEC, max_rows=8, max_req=4), **kw))
        self.rc = lib.mono_cache_build(C.byref(spec), C.byref(self.h))

    def __enter__(self):
        return self

    def __exit__(self, *_):
        self.lib.mono_cache_free(self.h)

    def call(self, name, args):
        return getattr(self.lib, "mono_cache_" + name)(self.h, C.byref(args), None)


def append_args(**kw):
    rope = kw.pop("rope", {})
    return mc.AppendArgs(**dict(dict(kv=A, positions=A, row_req=A, block_table=A, dtype=1, rows=3, n_req=2,
                                     max_blocks=5, **VIEW), **kw), rope=mc.Rope(**rope))


def test_rotary_positions_without_a_table_are_not_looked_at(lib):
    """Nothing is rotated then: a negative one would have its row left out, unreported."""
    with Handle(lib) as h:
        assert h.call("append", append_args(rope_positions=A)) == 0
        assert lib.rotation_given() == 0 and lib.rope_positions_given() == 0
        rope = dict(table=A, positions=9, dim=32, offset=32)
        assert h.call("append", append_args(rope_positions=A + 64, rope=rope)) == 0
        assert lib.rotation_given() == 32 and lib.rope_positions_given() == A + 64
        assert h.call("append", append_args(rope_positions=A + 2)) == -4  # (a wrong one is still refused)


def test_rotations_are_dealt_out_over_the_devices_sms(lib):
    with Handle(lib) as h:
        rope = dict(table=A, positions=9, dim=32, offset=32)
        rot = mc.RotateArgs(x=A, out=A, positions=A, dtype=1, rows=3, heads=2, rope=mc.Rope(**rope))
        for name, args in (("rotate", rot), ("append", append_args(rope=rope))):
            C.c_int.in_dll(lib, "rotated_sms").value = 0
            assert h.call(name, args) == 0 and value(lib, "rotated_sms", C.c_int) == 152


def attend_args(**kw):
    return mc.AttendArgs(**dict(dict(q=A, o=A, positions=A, row_req=A, block_table=A, max_blocks=5, n_req=2, rows=3, **VIEW), **kw))


def shared_args():
    return mc.SharedArgs(q=A, o=A, positions=A, row_req=A, block_table=A, prefix_table=A, prefix_lengths=A, max_blocks=5,
                         n_req=2, prefix_max_blocks=3, n_prefix=1, rows=3, **VIEW)


def evict_args():
    return mc.EvictArgs(weights=A, lengths=A, new_lengths=A, kept=A, block_table=A, weights_stride=320, kept_stride=8, budget=8,
                        n_req=2, max_blocks=5, **VIEW)


@pytest.mark.parametrize("max_rows,n_q_heads", [(1, 4), (48, 16), (1024, 32)])
def test_operators_that_follow_one_another_share_a_workspace(lib, max_rows, n_q_heads):
    """A handle holds that of the largest, not all of them, and spends no time on its contents."""
    shared = 5000000 + 1000 * max_rows
    before = value(lib, "zeroed")
    with Handle(lib, max_rows=max_rows, n_q_heads=n_q_heads) as h:
        assert h.rc == 0
        all_bytes, lse = value(lib, "allocated"), max_rows * n_q_heads * 4
        assert shared + lse <= all_bytes <= shared + lse + 4096
        assert value(lib, "zeroed") - before <= 4096
        rows = min(3, max_rows)
        for name, args in (("attend", attend_args(rows=rows)), ("attend_shared", shared_args()), ("evict", evict_args())):
            args.rows = rows
            assert h.call(name, args) == 0
        arena = value(lib, "arena", C.c_void_p)
        at = {value(lib, n, C.c_void_p) - arena for n in ("attend_at", "shared_at", "evict_at")}
        # one place, 256-byte aligned in the arena, behind the status word and the attention's own log-sums
        lse_at = value(lib, "lse_at", C.c_void_p) - arena
        assert len(at) == 1 and lse_at >= 4 and min(at) >= lse_at + lse and min(at) % 256 == 0
        assert min(at) + shared <= all_bytes


def test_a_kernel_that_cannot_run_is_its_own_operators_business(lib):
    C.c_int.in_dll(lib, "shared_error").value = 9
    try:
        with Handle(lib) as h:
            assert h.rc == 0
            assert h.call("attend", attend_args()) == 0 and h.call("evict", evict_args()) == 0
            assert h.call("append", append_args()) == 0
            assert h.call("attend_shared", shared_args()) == -7
    finally:
        C.c_int.in_dll(lib, "shared_error").value = 0
    with Handle(lib) as h:
        assert h.call("attend_shared", shared_args()) == 0
