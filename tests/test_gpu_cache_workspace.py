"""Operators of one handle that follow one another in its workspace, on the GPU: each call's results are bit
for bit those of a handle of its own, whichever calls are on their way before and behind it."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro
from tests.test_gpu_cache_shared import FULL, TINY, _m, i32, make_q, make_shared, rows_of

pytestmark = pytest.mark.gpu


def step(spec, seed):
    """The operators on a step of eight requests behind a prefix, as functions of the handles that they use and
    of the tensors that they fill."""
    of, own = [0] * 6 + [-1] * 2, [700, 3, 40, 129, 1, 77, 900, 500]
    ptable, table, cache = make_shared(spec, [1500], of, own, seed)
    pos, req = rows_of([1500], of, own, [3, 1, 3, 2, 1, 3, 2, 3])
    q = make_q(spec, len(pos), seed).cuda()
    p, r, t, c, pt = i32(pos), i32(req), i32(table), torch.from_numpy(cache).cuda(), i32(ptable)
    L, ofd, heads = i32([1500]), i32(of), spec["n_q_heads"]
    lengths = i32([(1500 if g == 0 else 0) + n for g, n in zip(of, own)])
    rng = np.random.default_rng(seed)
    w = torch.from_numpy(rng.random((8, table.shape[1] * spec["block_size"]), np.float32)).cuda()
    dst_table = torch.arange(8 * 40, dtype=torch.int32, device="cuda").view(8, 40)
    kv = torch.from_numpy(rng.standard_normal((len(pos), spec["kv_dim"])).astype(np.float32)).cuda()
    rope = torch.from_numpy(ro.table(4000, 32)).cuda()

    def out():
        return dict(o=torch.zeros_like(q), lse=torch.zeros((len(pos), heads), device="cuda"), o2=torch.zeros_like(q),
                    lse2=torch.zeros((len(pos), heads), device="cuda"), acc=torch.zeros_like(w),
                    kept=torch.zeros((8, 300), dtype=torch.int32, device="cuda"), new=i32([0] * 8), wout=torch.zeros_like(w),
                    moved=torch.zeros((320, *c.shape[1:]), dtype=torch.uint8, device="cuda"), qr=torch.zeros((len(pos), q.shape[1]), device="cuda"),
                    pool=torch.zeros_like(c))

    x = q.float()
    calls = dict(
        attend=lambda h, d: h.attend(q, d["o"], p, r, t, c, lse=d["lse"], weights=d["acc"]),
        shared=lambda h, d: h.attend_shared(q, d["o2"], p, r, t, c, pt, L, prefix_of=ofd, lse=d["lse2"]),
        evict=lambda h, d: h.evict(w, lengths, t, c, d["kept"], d["new"], budget=300, sinks=4, recent=50,
                                   weights_out=d["wout"], dst_table=dst_table, dst_cache=d["moved"]),
        append=lambda h, d: h.append(kv, p, r, t, d["pool"], rope=rope, q=x, q_out=d["qr"]))
    return calls, out, len(pos)


@pytest.mark.parametrize("spec", [FULL, TINY], ids=["full", "tiny"])
def test_calls_of_one_handle_in_any_order(spec):
    m = _m()
    calls, out, rows = step(spec, 31)
    want = out()
    for f in calls.values():
        h = m.Cache(spec, rows, 8)
        f(h, want)
        torch.cuda.synchronize()
        assert h.status() == 0
        h.close()
    rng = np.random.default_rng(7)
    h = m.Cache(spec, rows, 8)
    for _ in range(12):
        got = [out() for _ in range(3)]
        torch.cuda.synchronize()
        for d in got:  # (none waits for another on the host)
            for name in rng.permutation(list(calls)):
                calls[name](h, d)
        torch.cuda.synchronize()
        assert h.status() == 0
        for d in got:
            for name in want:
                assert torch.equal(d[name].view(torch.uint8), want[name].view(torch.uint8)), name
    graph, d = torch.cuda.CUDAGraph(), out()
    with torch.cuda.graph(graph):
        for name in ("shared", "attend", "evict", "shared", "append", "evict"):
            calls[name](h, d)
    for _ in range(5):
        for t in d.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(d[name].view(torch.uint8), want[name].view(torch.uint8)), name
    h.close()


def test_a_handle_takes_the_memory_of_its_largest_operator():
    """The pieces of the shared attention: two places a row and head, and 256 an SM, of head_dim + 8 f32."""
    m = _m()
    torch.cuda.synchronize()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m.Cache(FULL, 1, 1).close()  # (what the first one loads stays)
    for rows in (1, 48, 1024):
        most = 136 * 4 * (2 * rows * 64 + 256 * sms) + 20 * rows * 64 + (4 << 20)
        before = torch.cuda.mem_get_info()[0]
        h = m.Cache(FULL, rows, 8)
        assert before - torch.cuda.mem_get_info()[0] <= most
        h.close()
