"""The sizes beyond which 32-bit indices of the cache operators would overflow are refused."""
import ctypes as C
import os
import re

import pytest

from moe_decode_layer_mxfp8_gb300 import cache as mc


@pytest.mark.parametrize("vocab,code", [(2 ** 31 - 63, -1), (2 ** 31 - 1, -1), (2 ** 31 - 64, -4)])
def test_vocabularies_beyond_the_indices(vocab, code):
    """(The largest one gets as far as the next check: an address that is not aligned.)"""
    from moe_decode_layer_mxfp8_gb300 import build
    build.build()
    a = 0x10000
    args = mc.VerifyArgs(target=a, draft=a, target_stride=2 ** 31, draft_stride=2 ** 31, dtype=0, vocab=vocab,
                         rows=4, n_req=2, row_start=a, draft_tokens=a, u=a + 2, r=a, greedy=None,
                         accepted=a, tokens=a)
    assert mc._lib().mono_verify_drafts(C.byref(args), None) == code


def ranges(length, cs, threads=512):
    """The eviction's share of the slots of each CTA and thread, in 64 bits."""
    per = ((length + cs * threads - 1) // (cs * threads)) | 1
    return length + cs * threads - 1, cs * threads * per, per


@pytest.mark.parametrize("cs", [1, 2, 4, 8, 16])
def test_shares_of_the_longest_caches_fit_32_bits(cs):
    """At the largest length that a call may have, no index that the selection computes passes 2^31; at
    2^31 - 1 one would."""
    text = open(os.path.join(os.path.dirname(mc.__file__), "csrc", "cache_ops.cu")).read()
    less = re.search(r"max_blocks \* s\.block_size > INT32_MAX(?: - (\d+))?", text).group(1)
    assert max(ranges(2 ** 31 - 1 - int(less or 0), cs)) < 2 ** 31 <= max(ranges(2 ** 31 - 1, cs))
