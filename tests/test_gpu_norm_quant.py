"""GPU parity of the int8 norm (pqk_norm_modulate_i8) and row quantisation
(pqk_quantize_i8) against their float64 definition.

Bounds, from the kernel's arithmetic. x' is one fp32 multiply-add; a row's sum
has chains of at most 64 terms and a tree of 13 levels, so its relative error
is below 80 * 2^-24 (half of that in the root); the norm's factor, the weight,
1 + scale and the multiply-add add 7 roundings. With
  size = |n w (1 + scale)| + |shift| + |mean part of n w (1 + scale)|
(what the terms of h add up to without cancellation), |h_gpu - h| is below
128 * 2^-24 * max size over the row. The scale moves by as much over 127 and
two roundings; a code is the integer next to h / scale, so
  |code - h / scale| <= 1/2 + (that bound + |h| * its relative share) / scale.
x' in bf16 is off by at most half a step (2^-8 relative), plus one fp32
rounding.
"""

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


def _bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def _wide(torch, bits, stride):
    """A device bf16 view of `bits` with `stride` elements between rows."""
    t = torch.full((bits.shape[0], stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    t[:, :bits.shape[1]] = to_dev_bf16(bits)
    return t[:, :bits.shape[1]]


def check(x, br, gate, w, shift, scale, cu, norm, eps, x_out, h8, h_scale):
    f = wl.bf16_bits_to_f64
    xd, brd = f(x), None if br is None else f(br)
    wd = None if w is None else f(w)
    xp, h = plain64.norm_modulate(xd, branch=brd, gate_res=gate, weight=wd, shift=shift, scale=scale, cu_seqlens=cu,
                                  norm_type=norm, eps=eps)
    # the terms of h, without cancellation
    sigma = np.ones(len(x)) if norm == 2 else np.sqrt(
        ((xp - (xp.mean(1, keepdims=True) if norm == 1 else 0)) ** 2).mean(1) + eps)
    terms = np.abs(xd) + (0 if brd is None else np.abs(xp - xd)) + (np.abs(xp).mean(1, keepdims=True) if norm == 1 else 0)
    terms = terms / sigma[:, None] * (1 if wd is None else np.abs(wd))
    if scale is not None:
        req = np.searchsorted(np.asarray(cu), np.arange(len(x)), side="right") - 1
        terms = terms * (1 + np.abs(scale[req])) + np.abs(shift[req])
    bound = 128 * 2.0 ** -24 * terms.max(axis=1)
    s = plain64.row_scales(h)
    gs = h_scale.cpu().numpy().astype(np.float64)
    amax = s * 127
    zero = np.abs(h).max(axis=1) == 0
    assert (np.abs(gs - s) <= bound / 127 + 2.0 ** -22 * s).all()
    codes = h8.cpu().numpy().astype(np.float64)
    slack = np.where(zero, 0, (2 * bound + 2.0 ** -21 * amax) / s)
    assert slack.max() < 0.25                                   # the check means something
    assert (np.abs(codes - h / s[:, None]) <= 0.5 + slack[:, None]).all()
    assert (np.abs(codes).max(axis=1) == np.where(zero, 0, 127)).all()
    if x_out is not None:
        g = bf16_to_f64(x_out)
        assert (np.abs(g - xp) <= 2.0 ** -8 * np.abs(xp) + 2.0 ** -23 * (np.abs(xd) + np.abs(xp - xd))).all()


# C covers every way a row is laid over threads, its borders (64, 65, 256, 257, 1,024 and 1,025 chunks of 8) and tails
@pytest.mark.parametrize("C", [8, 24, 256, 512, 520, 1504, 2048, 2056, 4096, 5120, 5632, 8192, 8200, 13824, 16384])
@pytest.mark.parametrize("norm", [pqk.NORM_RMS, pqk.NORM_LAYER, pqk.NORM_NONE])
def test_everything_on(C, norm):
    torch = torch_cuda()
    g = np.random.default_rng(C + norm)
    lens = [3, 0, 7, 1]
    T, B = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, br = _bits(g.standard_normal((T, C)) + 0.5), _bits(g.standard_normal((T, C)))
    w = _bits(g.uniform(0.5, 1.5, C))
    gate, shift, scale = ((0.3 * g.standard_normal((B, C))).astype(np.float32) for _ in range(3))
    x_out = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    xo, h8, s = pqk.norm_modulate_i8(to_dev_bf16(x), branch=to_dev_bf16(br), gate_res=to_dev(gate),
                                     weight=to_dev_bf16(w), shift=to_dev(shift), scale=to_dev(scale),
                                     cu_seqlens=to_dev(cu), norm_type=norm, eps=1e-5, x_out=x_out)
    torch.cuda.synchronize()
    assert xo is x_out and h8.dtype == torch.int8 and h8.stride(0) % 16 == 0
    check(x, br, gate, w, shift, scale, cu, norm, 1e-5, x_out, h8, s)


# many rows: a row is laid over fewer threads than in a call of a few
@pytest.mark.parametrize("C", [256, 264, 520, 776, 1024, 1032, 2048, 2056, 3000, 4096, 5120, 5632, 6152, 7168, 7176, 8200,
                               10248, 13824, 14344, 16384])
def test_many_rows_of_every_layout(C):
    torch = torch_cuda()
    g = np.random.default_rng(C)
    lens = [301, 0, 20, 1, 90]
    T, B = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, br = _bits(g.standard_normal((T, C)) - 0.25), _bits(g.standard_normal((T, C)))
    w = _bits(g.uniform(0.5, 1.5, C))
    gate, shift, scale = ((0.3 * g.standard_normal((B, C))).astype(np.float32) for _ in range(3))
    for norm in (pqk.NORM_RMS, pqk.NORM_LAYER):
        xo = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
        _, h8, s = pqk.norm_modulate_i8(to_dev_bf16(x), branch=to_dev_bf16(br), gate_res=to_dev(gate),
                                        weight=to_dev_bf16(w), shift=to_dev(shift), scale=to_dev(scale),
                                        cu_seqlens=to_dev(cu), norm_type=norm, x_out=xo)
        torch.cuda.synchronize()
        check(x, br, gate, w, shift, scale, cu, norm, 1e-6, xo, h8, s)
    x8, s = pqk.quantize_i8(to_dev_bf16(x))
    torch.cuda.synchronize()
    check(x, None, None, None, None, None, cu, pqk.NORM_NONE, 1.0, None, x8, s)


@pytest.mark.parametrize("branch, gate, weight, mod", [
    (False, False, False, False), (True, False, False, False), (True, True, False, False), (False, False, True, False),
    (False, False, False, True), (True, False, True, True), (True, True, True, False)])
@pytest.mark.parametrize("T, C", [(1, 2048), (2, 136), (53, 1000)])
def test_parts_left_out(branch, gate, weight, mod, T, C):
    torch = torch_cuda()
    g = np.random.default_rng(T + C)
    x = _bits(g.standard_normal((T, C)))
    br = _bits(g.standard_normal((T, C))) if branch else None
    w = _bits(g.uniform(0.5, 1.5, C)) if weight else None
    cu = np.array([0, T], np.int32)
    vec = [(0.3 * g.standard_normal((1, C))).astype(np.float32) for _ in range(3)]
    gt = vec[0] if gate else None
    sh, sc = (vec[1], vec[2]) if mod else (None, None)
    dev = lambda a: None if a is None else to_dev(a)
    bf = lambda a: None if a is None else to_dev_bf16(a)
    xo = torch.empty((T, C), dtype=torch.bfloat16, device="cuda") if branch else None
    _, h8, s = pqk.norm_modulate_i8(bf(x), branch=bf(br), gate_res=dev(gt), weight=bf(w), shift=dev(sh),
                                    scale=dev(sc), cu_seqlens=to_dev(cu) if gate or mod else None, x_out=xo)
    torch.cuda.synchronize()
    check(x, br, gt, w, sh, sc, cu, pqk.NORM_RMS, 1e-6, xo, h8, s)


def test_strides_in_place_and_guard_bytes():
    torch = torch_cuda()
    g = np.random.default_rng(5)
    T, C = 19, 1048
    x, br = _bits(g.standard_normal((T, C))), _bits(g.standard_normal((T, C)))
    xd, brd = _wide(torch, x, C + 24), _wide(torch, br, C + 8)
    h_wide = torch.full((T + 1, 1088), 77, dtype=torch.int8, device="cuda")
    s_wide = torch.full((T + 1,), 5.0, device="cuda")
    _, h8, s = pqk.norm_modulate_i8(xd, branch=brd, x_out=xd, h8=h_wide[:T, :C], h_scale=s_wide[:T])
    torch.cuda.synchronize()
    check(x, br, None, None, None, None, [0, T], 0, 1e-6, xd, h8, s)
    assert (h_wide[:, C:] == 77).all() and (h_wide[T] == 77).all() and s_wide[T] == 5.0
    assert torch.isnan(xd.as_strided((T, 24), (C + 24, 1), C)).all()


def test_vectors_on_16_but_not_32_byte_boundaries():
    torch = torch_cuda()
    g = np.random.default_rng(15)
    lens, C = [70, 400], 1040
    T, cu = sum(lens), np.array([0, 70, 470], np.int32)
    x, br = _bits(g.standard_normal((T, C))), _bits(g.standard_normal((T, C)))
    vec = [(0.3 * g.standard_normal((2, C))).astype(np.float32) for _ in range(3)]
    flat = torch.empty(3 * (2 * C + 4), device="cuda")
    views = []
    for i, v in enumerate(vec):
        t = flat[i * (2 * C + 4) + 4:][:2 * C].view(2, C)
        t.copy_(to_dev(v))
        views.append(t)
    assert any(t.data_ptr() % 32 for t in views)
    xo = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    args = dict(branch=to_dev_bf16(br), cu_seqlens=to_dev(cu), x_out=xo)
    _, h8, s = pqk.norm_modulate_i8(to_dev_bf16(x), gate_res=views[0], shift=views[1], scale=views[2], **args)
    torch.cuda.synchronize()
    check(x, br, vec[0], None, vec[1], vec[2], cu, 0, 1e-6, xo, h8, s)
    again = pqk.norm_modulate_i8(to_dev_bf16(x), gate_res=to_dev(vec[0]), shift=to_dev(vec[1]), scale=to_dev(vec[2]),
                                 **args)
    assert torch.equal(again[1], h8) and torch.equal(again[2], s)


def test_extreme_rows():
    """Zero rows, rows of one value, the smallest and largest bf16 numbers, rows whose halves differ by 2^120, and
    values next to ties: the plain quantisation."""
    torch = torch_cuda()
    C = 264
    g = np.random.default_rng(6)
    rows = [np.zeros(C), np.full(C, -3.0), np.full(C, 1e-40), np.full(C, 3.3e38), g.standard_normal(C) * 1e-38,
            g.standard_normal(C) * 1e-39, np.where(np.arange(C) % 2, 1e20, 1e-20), np.arange(C) - 127.0,
            g.standard_normal(C) * 1e38]
    x = _bits(np.stack(rows))
    xd = wl.bf16_bits_to_f64(x)
    x8, s = pqk.quantize_i8(to_dev_bf16(x))
    torch.cuda.synchronize()
    gs, codes = s.cpu().numpy().astype(np.float64), x8.cpu().numpy().astype(np.float64)
    ref = plain64.row_scales(xd)
    assert (np.abs(gs - ref) <= 2.0 ** -23 * ref + 2.0 ** -149).all()
    assert (np.abs(codes - xd / ref[:, None]) <= 0.5 + 127 * 2.0 ** -22).all()
    assert (codes[0] == 0).all() and gs[0] == 1.0 and (codes[1] == -127).all()


@pytest.mark.parametrize("C", [256, 2048, 5120, 13824])
@pytest.mark.parametrize("norm", [pqk.NORM_RMS, pqk.NORM_LAYER, pqk.NORM_NONE])
def test_rows_that_are_not_finite_are_marked_and_touch_no_other(C, norm):
    torch = torch_cuda()
    g = np.random.default_rng(7)
    x = g.standard_normal((8, C)).astype(np.float32)
    clean = pqk.norm_modulate_i8(to_dev_bf16(_bits(x)), norm_type=norm)
    x[1, 0], x[3, C - 1], x[4, C // 2] = np.nan, np.inf, -np.inf
    x[6] *= 1e30                                                 # squares past fp32's range, when there is a norm
    _, h8, s = pqk.norm_modulate_i8(to_dev_bf16(_bits(x)), norm_type=norm)
    torch.cuda.synchronize()
    bad = [1, 3, 4] + ([6] if norm != pqk.NORM_NONE else [])
    for r in range(8):
        if r in bad:
            assert torch.isnan(s[r]) and not h8[r].any()
        elif r != 6:
            assert torch.equal(h8[r], clean[1][r]) and s[r] == clean[2][r]


def test_many_rows_determinism_and_an_empty_call():
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(60001, 512, generator=g, device="cuda").to(torch.bfloat16)
    a, b = pqk.quantize_i8(x), pqk.quantize_i8(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    amax = x.float().abs().amax(1)
    # the correctly rounded quotient: through fp64, since torch divides a CUDA tensor by a number by multiplying with
    # that number's rounded reciprocal (two roundings); an fp64 quotient of a bf16 number by 127 is never so near a
    # tie between two floats (its distance is a multiple of 2^-25 / 127 relative) that rounding twice could differ
    assert torch.equal(a[1], (amax.double() / 127).float())
    off = (a[0].double() * a[1].double()[:, None] - x.double()).abs().amax(1)
    assert (off <= a[1].double() * (0.5 + 2.0 ** -16)).all()
    e8, es = pqk.quantize_i8(x[:0])
    assert e8.shape == (0, 512) and es.shape == (0,)
    assert pqk.get_device_status() == 0
