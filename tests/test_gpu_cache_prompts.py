"""Prompts on the GPU: so many rows that threads of a rotation take several heads, in every type, and that a
request's rows fill many blocks of the attention over shared prefixes."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro
from tests.test_gpu_cache_append import DTYPES, LAYOUTS, check_append, i32
from tests.test_gpu_cache_shared import _m, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,heads,rows", [("full", 5, 4001), ("full", 64, 1500), ("wide", 16, 1250),
                                               ("wide", 7, 2777), ("wide", 131, 1300), ("tiny", 1, 20003)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rotate_many_rows(layout, heads, rows, inter, dtype):
    """Into another tensor, and in place and back; bit for bit, rounding by rounding."""
    m, spec = _m(), LAYOUTS[layout]
    h, dh = m.Cache(spec, 1, 1), spec["head_dim"]
    rng = np.random.default_rng(heads)
    pos = rng.integers(-1, 300, rows)
    tab = ro.table(300, 48)
    x = torch.from_numpy(rng.standard_normal((rows, heads * dh)).astype(np.float32)).to(DTYPES[dtype])
    xd, td, pd = x.cuda(), torch.from_numpy(tab).cuda(), i32(pos)
    for inverse in (False, True):
        out = torch.full_like(xd, 7.0)
        h.rotate(xd, out, pd, td, rope_offset=8, interleaved=inter, inverse=inverse)
        h.rotate(xd, xd, pd, td, rope_offset=8, interleaved=inter, inverse=inverse)
        want = torch.from_numpy(ro.rotate(x.float().numpy(), tab, pos, dh, 8, inter, inverse,
                                          dtype=np.float32)).to(x.dtype)
        assert torch.equal(xd.cpu(), want)
        x = want.clone()
        want[torch.from_numpy(pos) < 0] = 7.0
        assert torch.equal(out.cpu(), want)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("layout", ["wide", "many", "three", "odd", "full"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_prompts_with_queries(layout, dtype, interleaved):
    spec = LAYOUTS[layout]
    rows = 700 if layout == "full" else 2600
    check_append(spec, [rows + 11, 64, 900], [rows, 1, 800], dtype=dtype, dim=spec["head_dim"] // 2, interleaved=interleaved,
                 shift=77, pads=(0, 5, 500), seed=rows, q="place" if interleaved else "out")


@pytest.mark.parametrize("layout,rows", [("wide", [512, 512]), ("tiny", [1024]), ("three", [300, 7, 500]), ("full", [257, 130]),
                                         ("odd", [100, 333]), ("many", [64, 1, 200])])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_behind_a_prefix(layout, rows, causal):
    """Requests that are admitted behind an instruction: all their own tokens, and some of the prefix's last, are rows."""
    check(LAYOUTS[layout], [700], [0] * len(rows), [max(1, n - 20) for n in rows], rows, seed=sum(rows), causal=causal,
          shuffle=layout != "full")
