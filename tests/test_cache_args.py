"""The binding's checks of tensors, as the extension makes them and as Python does: the same answers."""
import pytest
import torch

from moe_decode_layer_mxfp8_gb300 import cache as mc

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def tensors():
    big = torch.zeros(20, 64)
    yield from (torch.zeros(6, dtype=I32), torch.zeros(12, dtype=I32)[::2], torch.zeros(1, dtype=I32)[::5],
                torch.zeros(0, dtype=I32), torch.zeros(6, dtype=torch.int64), torch.zeros(6, 1, dtype=I32),
                torch.zeros((), dtype=I32), torch.zeros(5, dtype=I32), torch.zeros(1, dtype=I32).expand(6))
    yield from (big, big[:6, :16], big[:1, 3:19], big.T, big[::2], torch.zeros(6, 16, dtype=BF16), big[:6, ::4],
                torch.zeros(1, 16).expand(6, 16), torch.zeros(16, 6).T, torch.zeros(6, 1), torch.zeros(6, 0),
                torch.zeros(0, 16), torch.zeros(6, 16, dtype=I32), torch.zeros(6, 16, requires_grad=True),
                torch.zeros(6, 16, device="meta"))
    pool = torch.zeros(5, 8, 80, dtype=U8)
    yield from (pool, pool[::2], pool[:, :, :64], pool[..., ::2], pool[:, :4], torch.zeros(5, 80, 8, dtype=U8).transpose(1, 2),
                pool.to(torch.int8), torch.zeros(0, 8, 80, dtype=U8), torch.zeros(1, 8, 96, dtype=U8).expand(5, 8, 96))
    yield from (None, 3, "x", [1, 2])


CHECKS = {  # which check, and its arguments behind the tensor
    "vec": (0, "t", I32, 6, -1),
    "vec of one": (0, "t", I32, 1, -1),
    "vec of none": (0, "t", I32, 0, -1),
    "mat": (1, "t", (F32,), 6, 16, -1),
    "mat of any": (1, "t", mc._FLOATS, None, None, -1),
    "mat elsewhere": (1, "t", (F32,), 6, 16, 0),
    "table": (2, "t", None, -1),
    "table of six": (2, "t", 6, -1),
    "pages": (3, "t", 8, 80, -1),
}


@pytest.mark.parametrize("check", CHECKS)
def test_both_give_the_same(check):
    if mc._args is None:
        pytest.skip("the extension is not there")
    which, *args = CHECKS[check]

    def answer(fn, t):
        try:
            return fn(t, *args)
        except (ValueError, AttributeError) as e:
            return type(e), str(e)

    for t in tensors():
        assert answer((mc._vec, mc._mat, mc._table, mc._pages)[which], t) == answer(mc._IN_PYTHON[which], t), t


def test_what_python_alone_accepts_is_accepted():
    """What the extension does not know goes to the check in Python."""
    if mc._args is None:
        pytest.skip("the extension is not there")
    seen = []
    try:
        mc._args.otherwise(*(lambda *a: seen.append(a) or 7 for _ in range(4)))
        assert mc._vec("not a tensor", "t", I32, 6, -1) == 7 and seen == [("not a tensor", "t", I32, 6, -1)]
    finally:
        mc._args.otherwise(*mc._IN_PYTHON)
    assert mc._vec is mc._args.vec


def test_sizes_that_are_no_numbers():
    if mc._args is None:
        pytest.skip("the extension is not there")
    t = torch.zeros(6, dtype=I32)
    for bad in (lambda: mc._vec(t, "t", I32, 1.5, -1), lambda: mc._vec(t, "t", I32, "6", -1), lambda: mc._vec(t, "t", I32),
                lambda: mc._mat(t, "t", [F32], 6, 1, -1), lambda: mc._pages(t, "t", 8, "80", -1)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(OverflowError):
        mc._vec(t, "t", I32, 2 ** 70, -1)
    assert mc._vec(t, "t", I32, 6, -1) == t.data_ptr()
