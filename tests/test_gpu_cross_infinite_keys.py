"""Cross-attention with keys whose scores are -inf: they weigh nothing, wherever
they lie among the request's keys, and a row of nothing else is 0 / 0."""

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


def _bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


# the key tiles of 128: first, middle and last ones; all of a part's (parts have at least four tiles, or two for each
# softmax group); the first group's only
GONE = [[(0, 128)], [(0, 256)], [(0, 1)], [(128, 256)], [(0, 512)], [(0, 128), (256, 384)], [(100, 900)],
        [(0, 2000)], [(512, 4096)]]


@pytest.mark.parametrize("gone", GONE)
@pytest.mark.parametrize("n_q, n_k, H, Hkv, D", [(5, 4500, 2, 2, 128), (200, 4500, 2, 1, 64), (1, 2300, 4, 1, 128),
                                                 (300, 300, 3, 3, 64), (2000, 500, 8, 8, 128), (40, 700, 2, 2, 64)])
def test_keys_of_scores_minus_infinity(gone, n_q, n_k, H, Hkv, D):
    torch = torch_cuda()
    g = np.random.default_rng(n_q + n_k + len(gone) + gone[0][1])
    q, k, v = (g.standard_normal(s) for s in ((n_q, H, D), (n_k, Hkv, D), (n_k, Hkv, D)))
    q[:, :, 3] = np.abs(q[:, :, 3]) + 0.25
    for a, b in gone:
        k[a:b, :, 3] = -np.inf
    cu_q, cu_k = np.array([0, n_q], np.int32), np.array([0, n_k], np.int32)
    qb, kb, vb = _bits(q), _bits(k), _bits(v)
    o, lse = pqk.varlen_cross_attn_fwd(to_dev_bf16(qb), to_dev_bf16(kb), to_dev_bf16(vb), to_dev(cu_q), to_dev(cu_k),
                                       want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    got, got_l = bf16_to_f64(o), lse.cpu().numpy().astype(np.float64)
    f = wl.bf16_bits_to_f64
    left = np.ones(n_k, bool)
    for a, b in gone:
        left[a:b] = False
    if not left.any():
        assert np.isnan(got).all() and np.isneginf(got_l).all()
        return
    # the definition over the keys that are left; bounds as in the tests of finite keys
    ref, ref_l, spread = plain64.cross_attention(f(qb), f(kb)[left], f(vb)[left], cu_q, [0, int(left.sum())],
                                                 D ** -0.5)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * spread + 1e-30).all()
    assert (np.abs(got_l - ref_l) <= 1e-5 * (1 + np.abs(ref_l))).all()


def test_nan_among_infinite_keys_is_not_hidden():
    """A part whose rows are NaN beside parts of nothing but -inf."""
    torch = torch_cuda()
    g = np.random.default_rng(2)
    q, k, v = (g.standard_normal((n, 1, 128)) for n in (1, 3000, 3000))
    q[:, :, 3] = 1.0
    k[:, :, 3] = -np.inf
    k[1700, :, 5] = np.nan
    o, lse = pqk.varlen_cross_attn_fwd(*(to_dev_bf16(_bits(t)) for t in (q, k, v)), to_dev(np.array([0, 1], np.int32)),
                                       to_dev(np.array([0, 3000], np.int32)), want_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(o).all() and torch.isnan(lse).all()
