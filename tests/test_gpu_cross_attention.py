"""GPU parity of cross-attention (pqk_varlen_cross_attn_fwd) against its
float64 definition.

Bounds: a probability is rounded to bf16 for P V (half a step, 2^-8 relative)
and carries the fp32 error of its score's exponent (below 2^-14 for the scores
here, |s| < 60 in log2 units), so before the output's own rounding
|o - r| <= (2^-8 + 2^-13) * sum p |v|; the output's rounding adds 2^-8 |r|. The
log-sum-exp is fp32: 1e-5 * (1 + |r|).
"""

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _inputs(lens_q, lens_k, H, Hkv, D, seed, extra_q=0, extra_k=0, peak=1.0):
    g = np.random.default_rng(seed)
    b = lambda *s: wl.f32_to_bf16_bits(g.standard_normal(s).astype(np.float32))
    q = wl.f32_to_bf16_bits((peak * g.standard_normal((sum(lens_q) + extra_q, H, D))).astype(np.float32))
    return q, b(sum(lens_k) + extra_k, Hkv, D), b(sum(lens_k) + extra_k, Hkv, D), _cu(lens_q), _cu(lens_k)


def check(q, k, v, cu_q, cu_k, o, lse, scale=None):
    f = wl.bf16_bits_to_f64
    n, m = int(cu_q[-1]), int(cu_k[-1])
    ro, rl, spread = plain64.cross_attention(f(q)[:n], f(k)[:m], f(v)[:m], cu_q, cu_k, scale or q.shape[2] ** -0.5)
    go = bf16_to_f64(o)[:n]
    assert (np.abs(go - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -13) * spread + 1e-30).all(), \
        float(np.abs(go - ro).max())
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64)[:, :n]
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty)
        assert (np.abs(gl[~empty] - rl[~empty]) <= 1e-5 * (1 + np.abs(rl[~empty]))).all()


CASES = [
    ([1], [1]), ([1], [128]), ([2], [129]), ([128], [127]), ([129], [300]), ([256], [1]), ([257], [640]),
    ([200, 312], [77, 120]), ([5, 0, 300, 1], [0, 9, 513, 0]), ([0, 0], [4, 5]), ([40, 700], [0, 0]),
    ([1, 1, 1], [3000, 1025, 5]), ([300], [5000]), ([1], [20000]), ([130, 1, 600], [1, 4097, 700]),
    ([128, 129, 1, 400, 256, 3] * 3, [512, 1, 640, 77, 0, 2000] * 3),
    # many short units one after another: one-tile and two-tile ones, with one key tile each
    ([1, 200, 5, 256, 64, 129] * 40, [3, 128, 100, 20, 1, 64] * 40),
]


@pytest.mark.parametrize("lens_q, lens_k", CASES)
@pytest.mark.parametrize("H, Hkv, D", [(3, 3, 128), (4, 2, 64), (6, 1, 128)])
def test_every_element(lens_q, lens_k, H, Hkv, D):
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, H, Hkv, D, seed=len(lens_q) + sum(lens_q) + H)
    if sum(lens_q) == 0:
        o, lse = pqk.varlen_cross_attn_fwd(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), to_dev(cu_q), to_dev(cu_k))
        assert o.shape == (0, H, D)
        return
    o, lse = pqk.varlen_cross_attn_fwd(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse)


@pytest.mark.parametrize("H, Hkv, D", [(6, 2, 128), (10, 2, 64), (7, 1, 128), (27, 1, 64), (32, 1, 128), (40, 1, 64),
                                       (16, 8, 128)])
@pytest.mark.parametrize("lens_q, lens_k", [
    ([1], [1]), ([1, 2, 3], [2000, 1500, 700]), ([43, 130, 4, 5], [130, 20, 600, 515]), ([300, 0, 9], [700, 4, 0]),
    ([1, 4, 60, 200], [40000, 1, 513, 640])])
def test_query_heads_that_share_key_heads(lens_q, lens_k, H, Hkv, D):
    """Shared key heads put several query heads' rows in one tile: groups that do and do not divide 128, tiles and
    keys that are cut or not, and (one key head for 40) the path that takes each head alone."""
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, H, Hkv, D, seed=H + sum(lens_q))
    o = torch.full((sum(lens_q) + 3, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, sum(lens_q)), 7.0, device="cuda")
    pqk.varlen_cross_attn_fwd(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), to_dev(cu_q), to_dev(cu_k),
                              o=o[:sum(lens_q)], lse=lse)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and (o[sum(lens_q):] == 7.0).all()
    check(q, k, v, cu_q, cu_k, o[:sum(lens_q)], lse)


@pytest.mark.parametrize("n_q", [1, 128, 129, 256])
@pytest.mark.parametrize("n_k", [512, 513, 640, 641, 768, 896, 1025, 1300])
def test_keys_cut_into_parts(n_q, n_k):
    """Parts of two, three and more key tiles, the last one ragged: the softmax groups take turns (up to 128
    queries) or share each tile."""
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs([n_q], [n_k], 2, 2, 128, seed=n_q + n_k)
    o, lse = pqk.varlen_cross_attn_fwd(*(to_dev_bf16(t) for t in (q, k, v)), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_many_tiles_of_few_keys(D):
    """More units than SMs, one to two key tiles each: the path of a long video over a short prompt."""
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs([9000, 2000], [77, 200], 8, 8, D, seed=2)
    o, lse = pqk.varlen_cross_attn_fwd(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse)


@pytest.mark.parametrize("lens_q, lens_k", [([300, 0, 5], [77, 3, 400]), ([2], [6000])])
def test_rows_behind_the_last_request_stay_and_never_leak_in(lens_q, lens_k):
    """cu_seqlens may end before the buffers do. What lies behind (NaN here) reaches no result, nor do other
    requests' rows, and the rows of o and lse behind the last request keep what they held."""
    torch = torch_cuda()
    H, D = 4, 128
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, H, H, D, seed=4, extra_q=150, extra_k=150)
    qd, kd, vd = (to_dev_bf16(t) for t in (q, k, v))
    for t, n in ((qd, cu_q[-1]), (kd, cu_k[-1]), (vd, cu_k[-1])):
        t[int(n):] = float("nan")
    o = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, qd.shape[0]), 7.0, device="cuda")
    pqk.varlen_cross_attn_fwd(qd, kd, vd, to_dev(cu_q), to_dev(cu_k), o=o, lse=lse)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    n = int(cu_q[-1])
    assert (o[n:] == 7.0).all() and (lse[:, n:] == 7.0).all()
    check(q, k, v, cu_q, cu_k, o, lse)
    # a request of NaN and infinity leaves its neighbours alone
    kd[int(cu_k[-2]):int(cu_k[-1])] = float("inf")
    vd[int(cu_k[-2]):int(cu_k[-1])] = float("nan")
    if len(lens_q) > 1:
        o2, _ = pqk.varlen_cross_attn_fwd(qd, kd, vd, to_dev(cu_q), to_dev(cu_k))
        torch.cuda.synchronize()
        first = int(cu_q[-2])
        assert torch.equal(o2[:first], o[:first]) and torch.isnan(o2[first:n]).all()


def test_strides_scale_and_peaked_rows():
    torch = torch_cuda()
    H, Hkv, D = 4, 2, 64
    q, k, v, cu_q, cu_k = _inputs([70, 190], [333, 20], H, Hkv, D, seed=5, peak=6.0)
    Tk = k.shape[0]
    kv = torch.zeros((Tk, 2 * Hkv + 1, D), dtype=torch.bfloat16, device="cuda")     # K and V in one buffer
    kv[:, :Hkv], kv[:, Hkv:2 * Hkv] = to_dev_bf16(k), to_dev_bf16(v)
    qw = torch.zeros((q.shape[0], H + 3, D), dtype=torch.bfloat16, device="cuda")
    qw[:, 1:1 + H] = to_dev_bf16(q)
    ow = torch.full((q.shape[0], H + 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = pqk.varlen_cross_attn_fwd(qw[:, 1:1 + H], kv[:, :Hkv], kv[:, Hkv:2 * Hkv], to_dev(cu_q), to_dev(cu_k),
                                       softmax_scale=0.25, o=ow[:, 2:], want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse, scale=0.25)
    assert (ow[:, :2] == 9.0).all()
    # rows of the output on 16-byte but not on 32-byte boundaries
    flat = torch.full((q.shape[0] * (H * D + 8) + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    odd = flat[8:].view(q.shape[0], H * D + 8)[:, :H * D].unflatten(1, (H, D))
    assert odd.data_ptr() % 32 == 16
    o2, _ = pqk.varlen_cross_attn_fwd(qw[:, 1:1 + H], kv[:, :Hkv], kv[:, Hkv:2 * Hkv], to_dev(cu_q), to_dev(cu_k),
                                      softmax_scale=0.25, o=odd)
    assert torch.equal(o2, o) and (flat[:8] == 9.0).all() and (flat[8:].view(-1, H * D + 8)[:, H * D:] == 9.0).all()


def test_equal_lengths_are_self_attention():
    """With the same cu_seqlens and key heads on both sides the result is the self-attention's."""
    torch = torch_cuda()
    q, k, v, cu, _ = _inputs([300, 513, 2], [300, 513, 2], 24, 24, 128, seed=8)
    d = [to_dev_bf16(t) for t in (q, k, v)]
    a, la = pqk.varlen_attn_fwd(*d, to_dev(cu), want_lse=True)
    b, lb = pqk.varlen_cross_attn_fwd(*d, to_dev(cu), to_dev(cu), want_lse=True)
    torch.cuda.synchronize()
    f = bf16_to_f64
    assert np.abs(f(a) - f(b)).max() <= 2e-2 and (la - lb).abs().max() <= 1e-3


@pytest.mark.parametrize("lens_q, lens_k", [([1, 3], [9000, 2500]), ([3000], [512])])
def test_bitwise_deterministic(lens_q, lens_k):
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, 8, 4, 128, seed=9)
    d = [to_dev_bf16(t) for t in (q, k, v)] + [to_dev(cu_q), to_dev(cu_k)]
    runs = [pqk.varlen_cross_attn_fwd(*d, want_lse=True) for _ in range(4)]
    torch.cuda.synchronize()
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("which, cu", [("q", [0, 50, 40, 60]), ("k", [0, 5, 900, 30]), ("q", [1, 2, 3, 60]),
                                       ("q", [0, 20, 40, 61]), ("k", [0, 10, 20, 31]), ("k", [-1, 10, 20, 30])])
def test_bad_cu_seqlens_write_nothing(which, cu):
    torch = torch_cuda()
    q, k, v, cu_q, cu_k = _inputs([20, 30, 10], [10, 10, 10], 2, 2, 64, seed=1)
    cu = np.array(cu, np.int32)
    o = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pqk.varlen_cross_attn_fwd(*(to_dev_bf16(t) for t in (q, k, v)), to_dev(cu if which == "q" else cu_q),
                              to_dev(cu if which == "k" else cu_k), o=o)
    assert pqk.get_device_status() == -7
    assert (o == 7.0).all() and pqk.get_device_status() == 0


def test_many_requests_and_past_the_sorted_ones():
    """10,000 requests: past the number that the schedule sorts."""
    torch = torch_cuda()
    g = np.random.default_rng(12)
    lens_q, lens_k = g.integers(0, 4, 10000).tolist(), g.integers(0, 6, 10000).tolist()
    q, k, v, cu_q, cu_k = _inputs(lens_q, lens_k, 2, 1, 64, seed=12)
    o, lse = pqk.varlen_cross_attn_fwd(*(to_dev_bf16(t) for t in (q, k, v)), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    check(q, k, v, cu_q, cu_k, o, lse)
