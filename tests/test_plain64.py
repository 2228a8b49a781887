"""Pins of the float64 forms behind the int8 norm, the int8 linear layers and
cross-attention (CPU only): closed forms and the oracle functions that cover
the same ground."""

import numpy as np

from oracle import oracle, plain64
from tests.bruteforce import padded_masked_attention


def test_norm_modulate_is_the_oracles_modulation():
    g = np.random.default_rng(0)
    T, C = 37, 48
    cu = np.array([0, 10, 10, 37], np.int32)
    x, br = g.standard_normal((T, C)), g.standard_normal((T, C))
    gate, shift, scale = (0.3 * g.standard_normal((3, C)).astype(np.float32) for _ in range(3))
    for norm in (0, 1, 2):
        xo, h, _ = oracle.modulate_swiglu(x, shift, scale, gate, cu, branch=br, norm_type=norm, eps=1e-5)
        gx, gh = plain64.norm_modulate(x, branch=br, gate_res=gate, shift=shift, scale=scale, cu_seqlens=cu,
                                       norm_type=norm, eps=1e-5)
        assert np.abs(gx - xo).max() < 1e-12 and np.abs(gh - h).max() < 1e-12


def test_codes_closed_forms():
    h = np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0], [1.0, -1.0, 0.25, 0, 0.125]])
    codes, s = plain64.quantize_rows(h)
    assert s.tolist() == [1.0, 1.0, 1.0 / 127]
    assert codes[0].tolist() == [127, 0, 2, -2, -127]          # ties go to the even code
    assert not codes[1].any()
    assert codes[2].tolist() == [127, -127, 32, 0, 16]         # 31.75 and 15.875
    g = np.random.default_rng(1)
    h = g.standard_normal((50, 33))
    codes, s = plain64.quantize_rows(h)
    assert (np.abs(codes * s[:, None] - h).max(axis=1) <= s / 2 * (1 + 1e-12)).all()
    assert (np.abs(codes).max(axis=1) == 127).all()


def test_linear_closed_forms():
    a = np.array([[1, -2, 3], [127, 127, -128]], np.int8)
    w = np.array([[1, 1, 1], [0, 2, 0]], np.int8)
    y = plain64.linear_i8(a, np.array([0.5, 2.0]), w, np.array([1.0, 0.25]))
    assert y.tolist() == [[1.0, -0.5], [252.0, 127.0]]
    x = np.ones((2, 2))
    out = plain64.gated_residual(y, x, np.array([[1.0, 0.0], [-1.0, 1.0]]), np.array([0, 1, 2]))
    assert out.tolist() == [[2.0, 1.0], [-251.0, 128.0]]
    assert plain64.swiglu(np.array([[0.0, 1.0, 3.0, 2.0]])).tolist() == [[0.0, 2 * 0.7310585786300049]]


def test_cross_attention_against_the_padded_brute_force_and_closed_forms():
    g = np.random.default_rng(2)
    lens = [5, 1, 12]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (g.standard_normal((18, 3, 8)) for _ in range(3))
    o, lse, _ = plain64.cross_attention(q, k, v, cu, cu, 0.3)
    ro, rl = padded_masked_attention(q, k, v, cu, 0.3)         # equal lengths: self-attention
    assert np.abs(o - ro).max() < 1e-12 and np.abs(lse - rl.T).max() < 1e-12
    # zero queries average the request's values; a request without keys gives 0 and -inf
    o, lse, spread = plain64.cross_attention(np.zeros((4, 2, 8)), k[:6, :1], v[:6, :1], [0, 3, 4], [0, 6, 6], 1.0)
    assert np.abs(o[:3] - v[:6, 0].mean(0)).max() < 1e-12 and not o[3].any()
    assert np.abs(lse[:, :3] - np.log(6)).max() < 1e-12 and np.isneginf(lse[:, 3]).all()
    assert np.abs(spread[:3] - np.abs(v[:6, 0]).mean(0)).max() < 1e-12
    # query heads 2 and 3 of four read key head 1 of two
    q = g.standard_normal((3, 4, 8))
    o, _, _ = plain64.cross_attention(q, k[:6, :2], v[:6, :2], [0, 3], [0, 6], 0.5)
    one, _, _ = plain64.cross_attention(q[:, 2:4], k[:6, 1:2], v[:6, 1:2], [0, 3], [0, 6], 0.5)
    assert np.abs(o[:, 2:4] - one).max() < 1e-12
