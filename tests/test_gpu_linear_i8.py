"""GPU parity of the int8 linear layers (pqk_linear_i8_gated_residual,
pqk_linear_i8_swiglu) against their float64 definition.

Bounds: the int32 sums are exact; a product y has 3 fp32 roundings (the sum's
conversion and two scales), the gated residual one more, so before the output's
rounding |g - r| <= 2^-21 (|y gate| + |x|). SwiGLU's exp(-g) has a relative
error of about 2^-22 (1 + |g|) and the quotient two more roundings: 2^-14 for
any |g| whose result is not negligible (1e-30 absolute for the others). The
output is rounded to bf16 by at most half a step, 2^-8 relative.
"""

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8


def _codes(g, rows, cols, full=False):
    return g.integers(-128, 128, (rows, cols)).astype(np.int8) if full else \
        np.clip(np.rint(g.standard_normal((rows, cols)) * 32), -127, 127).astype(np.int8)


def _dev8(torch, codes, pad=0):
    """Device codes with rows on 16-byte boundaries; the bytes between rows hold 99."""
    wide = (codes.shape[1] + 15) // 16 * 16 + pad
    t = torch.full((codes.shape[0], wide), 99, dtype=torch.int8, device="cuda")
    t[:, :codes.shape[1]] = to_dev(codes)
    return t[:, :codes.shape[1]]


def _case(lens, K, N, seed, full=False):
    g = np.random.default_rng(seed)
    T = sum(lens)
    a, w = _codes(g, T, K, full), _codes(g, N, K, full)
    sa = (g.uniform(0.5, 2.0, T) / 32).astype(np.float32)
    sw = (g.uniform(0.5, 2.0, N) / 32 / np.sqrt(K)).astype(np.float32)
    x = wl.f32_to_bf16_bits(g.standard_normal((T, N)).astype(np.float32))
    gate = (0.5 * g.standard_normal((len(lens), N))).astype(np.float32)
    return a, sa, w, sw, x, gate, np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def assert_close(got, ref, terms):
    g = bf16_to_f64(got)
    assert g.shape == ref.shape
    assert (np.abs(g - ref) <= HALF_STEP * np.abs(ref) + 2.0 ** -21 * terms + 1e-38).all(), \
        float(np.max(np.abs(g - ref) / (np.abs(ref) + 1e-30)))


SHAPES = [
    ([1], 8, 8), ([1], 5120, 264), ([1], 64, 2048), ([2, 0, 3], 40, 72), ([7, 9], 256, 640), ([17], 2048, 136),
    ([31, 2], 1000, 384), ([64], 136, 5120), ([65], 4096, 128), ([100, 28], 768, 1032), ([129], 264, 520),
    ([200, 0, 312, 77], 384, 640), ([255], 128, 256), ([256], 1024, 1024), ([1, 130, 300], 200, 264),
    ([5000], 128, 2048), ([1, 2, 3, 4, 1500], 648, 1160),
]


@pytest.mark.parametrize("lens, K, N", SHAPES)
@pytest.mark.parametrize("epi", ["none", "residual", "swiglu"])
def test_every_element(lens, K, N, epi):
    torch = torch_cuda()
    rows = 2 * N if epi == "swiglu" else N
    a, sa, w, sw, x, gate, cu = _case(lens, K, rows, seed=K + N + sum(lens), full=(K + N) % 16 == 8)
    y = plain64.linear_i8(a, sa, w, sw)
    args = (_dev8(torch, a), to_dev(sa), _dev8(torch, w, 32), to_dev(sw))
    if epi == "swiglu":
        out = pqk.linear_i8_swiglu(*args)
        ref = plain64.swiglu(y)
        g = bf16_to_f64(out)
        torch.cuda.synchronize()
        assert pqk.get_device_status() == 0
        assert (np.abs(g - ref) <= (HALF_STEP + 2.0 ** -14) * np.abs(ref) + 1e-30).all()
        return
    if epi == "residual":
        x, gate = x[:, :N], gate[:, :N]
        out = pqk.linear_i8_gated_residual(*args, x=to_dev_bf16(x), gate_res=to_dev(gate), cu_seqlens=to_dev(cu))
        xd = wl.bf16_bits_to_f64(x)
        ref = plain64.gated_residual(y, xd, gate, cu)
        terms = np.abs(ref - xd) + np.abs(xd)
    else:
        out = pqk.linear_i8_gated_residual(*args)
        ref, terms = y, np.abs(y)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    assert_close(out, ref, terms)


@pytest.mark.parametrize("T", [1, 33, 700])
def test_strides_in_place_and_guard_rows(T):
    torch = torch_cuda()
    K, N = 320, 264
    a, sa, w, sw, x, gate, cu = _case([T - T // 2, T // 2], K, N, seed=11)
    wide = torch.full((T + 2, N + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[1:T + 1, 8:8 + N] = to_dev_bf16(x)
    view = wide[1:T + 1, 8:8 + N]
    out = pqk.linear_i8_gated_residual(_dev8(torch, a, 48), to_dev(sa), _dev8(torch, w), to_dev(sw), x=view,
                                       gate_res=to_dev(gate), cu_seqlens=to_dev(cu), out=view)
    torch.cuda.synchronize()
    assert out.data_ptr() == view.data_ptr() and pqk.get_device_status() == 0
    xd = wl.bf16_bits_to_f64(x)
    ref = plain64.gated_residual(plain64.linear_i8(a, sa, w, sw), xd, gate, cu)
    assert_close(view, ref, np.abs(ref - xd) + np.abs(xd))
    wide[1:T + 1, 8:8 + N] = 3.0
    assert (wide == 3.0).all()                                   # nothing around the output was written


@pytest.mark.parametrize("T", [3, 300])
def test_longest_sums_stay_exact(T):
    """All codes -128 at the largest K: the sums reach 2^31 - 2^14."""
    torch = torch_cuda()
    K, N = 131064, 16
    a = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    wide = torch.full((T, K + 8), 1, dtype=torch.int8, device="cuda")
    wide[:, :K] = a
    w = torch.zeros((N, K + 8), dtype=torch.int8, device="cuda")
    w[:, :K] = -128
    w[1, :K] = 127
    one = torch.ones(max(T, N), device="cuda")
    out = pqk.linear_i8_gated_residual(wide[:, :K], one[:T], w[:, :K], one[:N])
    torch.cuda.synchronize()
    ref = torch.full((T, N), float(K * 128 * 128), device="cuda")
    ref[:, 1] = -float(K * 128 * 127)
    assert torch.equal(out, ref.to(torch.bfloat16))


@pytest.mark.parametrize("T", [5, 400])
def test_a_token_whose_scale_is_nan_touches_no_other(T):
    torch = torch_cuda()
    a, sa, w, sw, _, _, _ = _case([T], 256, 512, seed=3)
    clean = pqk.linear_i8_gated_residual(_dev8(torch, a), to_dev(sa), _dev8(torch, w), to_dev(sw))
    sa[2], a[2] = np.nan, 0
    out = pqk.linear_i8_gated_residual(_dev8(torch, a), to_dev(sa), _dev8(torch, w), to_dev(sw))
    act = pqk.linear_i8_swiglu(_dev8(torch, a), to_dev(sa), _dev8(torch, w), to_dev(sw))
    torch.cuda.synchronize()
    assert torch.isnan(out[2]).all() and torch.isnan(act[2]).all()
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(out[keep], clean[keep]) and not torch.isnan(act[keep]).any()


@pytest.mark.parametrize("T", [1, 30, 200, 3000])
def test_bitwise_deterministic_and_the_same_for_a_token_in_any_batch(T):
    """The sums are whole numbers: a token's result does not depend on how many tokens come with it."""
    torch = torch_cuda()
    a, sa, w, sw, x, gate, cu = _case([T], 1024, 768, seed=9)
    a8, w8 = _dev8(torch, a), _dev8(torch, w)
    kw = dict(x=to_dev_bf16(x), gate_res=to_dev(gate), cu_seqlens=to_dev(cu))
    o1 = pqk.linear_i8_gated_residual(a8, to_dev(sa), w8, to_dev(sw), **kw)
    o2 = pqk.linear_i8_gated_residual(a8, to_dev(sa), w8, to_dev(sw), **kw)
    act = pqk.linear_i8_swiglu(a8, to_dev(sa), w8, to_dev(sw))
    assert torch.equal(o1, o2)
    for t in {0, T // 2, T - 1}:
        one = pqk.linear_i8_gated_residual(a8[t:t + 1], to_dev(sa[t:t + 1]), w8, to_dev(sw), x=kw["x"][t:t + 1],
                                           gate_res=kw["gate_res"], cu_seqlens=to_dev(np.array([0, 1], np.int32)))
        assert torch.equal(one[0], o1[t])
        assert torch.equal(pqk.linear_i8_swiglu(a8[t:t + 1], to_dev(sa[t:t + 1]), w8, to_dev(sw))[0], act[t])
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0


def test_empty_call():
    torch = torch_cuda()
    a, sa, w, sw, _, _, _ = _case([4], 64, 32, seed=1)
    assert pqk.linear_i8_swiglu(_dev8(torch, a)[:0], to_dev(sa)[:0], _dev8(torch, w), to_dev(sw)).shape == (0, 16)
