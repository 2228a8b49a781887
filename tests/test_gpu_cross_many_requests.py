"""Cross-attention of more requests than one warp schedules (more than 32), few
enough tiles to be cut along their keys: one or a few queries per request over
hundreds to thousands of keys, keyless requests and requests without queries
among them. Bounds as in the tests of few requests."""

import numpy as np
import pytest

from packed_attention_qk_b200 import pqk
from tests.gpu_utils import to_dev, to_dev_bf16, torch_cuda
from tests.test_gpu_cross_attention import _inputs, check

pytestmark = pytest.mark.gpu


def _lens(B, seed, most_q, lo, hi):
    g = np.random.default_rng(seed)
    lens_q = g.integers(1, most_q + 1, B)
    lens_k = np.exp(g.uniform(np.log(lo), np.log(hi), B)).astype(int)
    lens_q[g.random(B) < 0.1] = 0
    lens_k[g.random(B) < 0.1] = 0
    return lens_q.tolist(), lens_k.tolist()


@pytest.mark.parametrize("B", [32, 33, 40, 64, 100, 147])
@pytest.mark.parametrize("H, Hkv, D", [(1, 1, 128), (2, 1, 64), (8, 1, 128)])
def test_few_queries_over_cut_keys(B, H, Hkv, D):
    torch = torch_cuda()
    lens_q, lens_k = _lens(B, B + H, 1 if B > 64 else 3, 600, 6000)
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, H, Hkv, D, seed=B + D, extra_q=3, extra_k=9)
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    d = [to_dev_bf16(t) for t in (q, k, v)] + [to_dev(cu_q), to_dev(cu_k)]
    pqk.varlen_cross_attn_fwd(*d, o=o, lse=lse)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    n = int(cu_q[-1])
    assert (o[n:] == 7.0).all() and (lse[:, n:] == 7.0).all()
    check(q, k, v, cu_q, cu_k, o, lse)
    again, lse2 = pqk.varlen_cross_attn_fwd(*d, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(again[:n], o[:n]) and torch.equal(lse2[:, :n], lse[:, :n])


@pytest.mark.parametrize("lens_q, lens_k", [
    ([1] * 40, [5] * 39 + [30000]),                                   # one long request among short ones
    ([1] * 36 + [300, 20, 0, 129], [700] * 36 + [5000, 0, 800, 640]), # tiles of one and of two query tiles
    ([2] * 73 + [600], [513] * 74),                                   # 148 tiles of pairs of heads: nothing is cut
    ([0] * 50 + [4], [900] * 50 + [9000]),                            # keys without queries
    ([3] * 60, [0] * 59 + [2000])])
def test_uneven_requests(lens_q, lens_k):
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, 2, 2, 64, seed=len(lens_q))
    o, lse = pqk.varlen_cross_attn_fwd(*(to_dev_bf16(t) for t in (q, k, v)), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse)


def test_captured_and_replayed_with_other_lengths():
    """One capture serves other lengths: tiles that are cut, tiles that are not, and keyless requests elsewhere."""
    torch = torch_cuda()
    B, H, D = 48, 2, 128
    sets = []
    for seed, most_q, hi in ((1, 1, 5000), (2, 4, 700), (3, 2, 2000)):
        lens_q, lens_k = _lens(B, seed, most_q, 60, hi)
        sets.append((lens_q, lens_k))
    Tq, Tk = max(sum(a) for a, _ in sets), max(sum(b) for _, b in sets)
    data = []
    for i, (lens_q, lens_k) in enumerate(sets):
        data.append(_inputs(lens_q, lens_k, H, H, D, seed=i, extra_q=Tq - sum(lens_q), extra_k=Tk - sum(lens_k)))
    d = [to_dev_bf16(t) for t in data[0][:3]] + [to_dev(t) for t in data[0][3:]]
    pqk.varlen_cross_attn_fwd(*d)
    torch.cuda.synchronize()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            o, lse = pqk.varlen_cross_attn_fwd(*d, want_lse=True)
    torch.cuda.current_stream().wait_stream(st)
    for x in data + data[:1]:
        for t, h in zip(d, x):
            t.copy_(to_dev_bf16(h) if h.dtype == np.uint16 else to_dev(h))
        graph.replay()
        torch.cuda.synchronize()
        assert pqk.get_device_status() == 0
        check(*x, o, lse)
    del graph


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("at, value", [(20, 10 ** 6), (0, 1), (40, 10 ** 6), (25, -5)])
def test_bad_cu_seqlens_of_many_requests_write_nothing(which, at, value):
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs([2] * 40, [3] * 40, 2, 2, 64, seed=1)
    bad = (cu_q if which == "q" else cu_k).copy()
    bad[at] = value
    o = torch.full((80, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pqk.varlen_cross_attn_fwd(*(to_dev_bf16(t) for t in (q, k, v)), to_dev(bad if which == "q" else cu_q),
                              to_dev(bad if which == "k" else cu_k), o=o)
    assert pqk.get_device_status() == -7
    assert (o == 7.0).all() and pqk.get_device_status() == 0
