"""The codes of pqk_norm_modulate_i8 and pqk_quantize_i8, each one exactly:
127 h / max|h| to the nearest integer, ties to even.

The reference decides by whole numbers: with k the integer part of
127 |h| / a, the code is k or k + 1 as 254 |h| - (2 k + 1) a is negative or
positive, and the even one of them where it is zero. The rows here have h
exactly (bf16 values, sums of two of them that fit fp32, or a norm that scales
a whole row by one factor), so that no tolerance is needed: 254 |h| and
(2 k + 1) a have at most 33 significant bits, exact in float64.

Why the kernel meets it: its quotient is the real one within 2^-45, rounded to
fp32 once. Near a border k + 1/2 of at least 1/2 two floats are 2^-25 to 2^-18
apart, and a bf16 quotient that is not on the border is at least 2^-8 / 510
times the border's power of two away from it, so only ties are rounded to the
border itself."""

import numpy as np
import pytest

from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


def _bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def exact_codes(h):
    """The codes of rows whose values are exact in float64 with few bits."""
    a = np.abs(h).max(axis=1, keepdims=True)
    unit = np.where(a > 0, a, 1.0)
    # a power of two out of each row, so that no product under- or overflows
    scale = 2.0 ** -np.floor(np.log2(unit))
    m, a = np.abs(h) * scale, unit * scale
    k = np.floor(127.0 * m / a)
    over = 254.0 * m - (2.0 * k + 1.0) * a
    code = k + ((over > 0) | ((over == 0) & (k % 2 == 1)))
    return (np.sign(h) * code).astype(np.int64)


def test_reference_on_known_rows():
    h = np.array([[2.0, 1.0, -1.0, 0.0, -2.0], [254.0, 3.0, 5.0, 253.0, 127.0], [1.5, 0.75, -0.75, 1e-30, 1.0]])
    assert exact_codes(h).tolist() == [[127, 64, -64, 0, -127], [127, 2, 2, 126, 64], [127, 64, -64, 0, 85]]


def _rows_of_ties(C, exponent, g):
    """A row for every mantissa of a bf16 maximum: half of it and odd multiples of 1/254 of it where they are bf16
    numbers, among others."""
    top = (128 + np.arange(128)) * 2.0 ** (exponent - 7)
    h = top[:, None] * g.uniform(-1, 1, (128, C))
    at = np.argsort(g.random((128, C)), axis=1)
    n = max(2, C // 3)
    odd = 2 * g.integers(0, 127, (128, n)) + 1
    for r in range(128):
        h[r, at[r, :n]] = top[r] * odd[r] / 254.0
        h[r, at[r, : max(2, C // 8)]] = top[r] / 2 * g.choice([-1, 1], max(2, C // 8))
        h[r, at[r, -1]] = top[r]
    return np.clip(h, -top[:, None], top[:, None])


# C: every way that a row is laid over threads; the exponents reach the smallest and the largest rows
@pytest.mark.parametrize("C", [8, 256, 520, 776, 1032, 2056, 3000, 4096, 5120, 6152, 7168, 8200, 10248, 13824, 16384])
@pytest.mark.parametrize("exponent", [0, -126, -101, 99, 127])
def test_ties_of_every_maximum(C, exponent):
    torch = torch_cuda()
    g = np.random.default_rng([C, exponent + 200])
    x = _bits(_rows_of_ties(C, exponent, g))
    xd = wl.bf16_bits_to_f64(x)
    want = exact_codes(xd)
    assert (np.abs(want) == 64).any(axis=1).mean() >= 0.5       # below 2^-126 only even mantissas have a half
    few, scales = pqk.quantize_i8(to_dev_bf16(x))                     # layouts of few and of many rows
    many, _ = pqk.quantize_i8(to_dev_bf16(np.tile(x, (3, 1))))
    torch.cuda.synchronize()
    assert np.array_equal(few.cpu().numpy(), want)
    assert np.array_equal(many.cpu().numpy(), np.tile(want, (3, 1)))
    assert np.array_equal(scales.cpu().numpy(), np.abs(xd).max(axis=1).astype(np.float32) / np.float32(127))


def test_rows_of_random_values():
    torch = torch_cuda()
    x = _bits(np.random.default_rng(3).standard_normal((600, 13824)))
    c, _ = pqk.quantize_i8(to_dev_bf16(x))
    torch.cuda.synchronize()
    assert np.array_equal(c.cpu().numpy(), exact_codes(wl.bf16_bits_to_f64(x)))


@pytest.mark.parametrize("T", [7, 900])
@pytest.mark.parametrize("C", [256, 2048, 5120, 16384])
def test_ties_of_sums(T, C):
    """x' = x + branch in whole numbers, without a norm: maxima with more bits than bf16 has, multiples of 127 among
    them, where every odd multiple of a 254th of the maximum is a tie."""
    torch = torch_cuda()
    g = np.random.default_rng(T + C)
    a, b = g.integers(-128, 129, (T, C)).astype(np.float64), 128.0 * g.integers(-20, 21, (T, C))
    a[:, 0], b[:, 0] = np.where(np.arange(T) % 3 == 0, 125.0, g.integers(0, 129, T)), 128.0 * 30  # 125 + 3840 = 127 * 31.2
    a[::3, 0] = 97.0                                                  # 3937 = 31 * 127
    a[::3, 1::5], b[::3, 1::5] = 31.0 * g.integers(0, 4, a[::3, 1::5].shape), 0.0
    h = a + b
    x, br = _bits(a), _bits(b)
    assert np.array_equal(wl.bf16_bits_to_f64(x) + wl.bf16_bits_to_f64(br), h)
    _, c, _ = pqk.norm_modulate_i8(to_dev_bf16(x), branch=to_dev_bf16(br), norm_type=pqk.NORM_NONE)
    torch.cuda.synchronize()
    assert np.array_equal(c.cpu().numpy(), exact_codes(h))


@pytest.mark.parametrize("T", [7, 900])
@pytest.mark.parametrize("C", [264, 2048, 5120, 13824])
def test_halves_of_the_maximum_after_a_norm(T, C):
    """RMS norm multiplies a row by one factor, so half the maximum stays half of it to the last bit: 63.5 steps."""
    torch = torch_cuda()
    g = np.random.default_rng(T * C)
    x = g.uniform(-0.4, 0.4, (T, C))
    top = (128 + g.integers(0, 128, T)) / 128.0
    x[:, 3], x[:, 8::11], x[:, 9::11] = top, top[:, None] / 2, -top[:, None] / 2
    x = _bits(x)
    assert (np.abs(wl.bf16_bits_to_f64(x)).max(axis=1) == top).all()
    scale = np.full((1, C), 0.37, np.float32)                         # the same factor for the whole row
    for kw in ({}, {"shift": to_dev(np.zeros((1, C), np.float32)), "scale": to_dev(scale),
                    "cu_seqlens": to_dev(np.array([0, T], np.int32))}):
        _, c, _ = pqk.norm_modulate_i8(to_dev_bf16(x), **kw)
        torch.cuda.synchronize()
        c = c.cpu().numpy()
        assert (c[:, 3] == 127).all() and (c[:, 8::11] == 64).all() and (c[:, 9::11] == -64).all()


@pytest.mark.parametrize("T", [7, 900])
@pytest.mark.parametrize("C", [256, 5120, 16384])
@pytest.mark.parametrize("exponent", [-120, -112, 87, 110])
def test_sums_near_the_ends_of_the_range(T, C, exponent):
    """The same whole numbers times a power of two: maxima on both sides of 2^-100 and 2^100, in one call. Their scale
    is the maximum over 127, rounded once."""
    torch = torch_cuda()
    g = np.random.default_rng([T, C, exponent + 200])
    a, b = g.integers(-128, 129, (T, C)).astype(np.float64), 128.0 * g.integers(-20, 21, (T, C))
    a[:, 0], b[:, 0] = np.where(np.arange(T) % 3 == 0, 97.0, g.integers(0, 129, T)), 128.0 * 30
    a[::3, 1::5], b[::3, 1::5] = 31.0 * g.integers(0, 4, a[::3, 1::5].shape), 0.0
    unit = 2.0 ** (exponent + np.arange(T) % 5)[:, None]
    a, b = a * unit, b * unit
    h = a + b
    x, br = _bits(a), _bits(b)
    assert np.array_equal(wl.bf16_bits_to_f64(x) + wl.bf16_bits_to_f64(br), h)
    xo = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    _, c, s = pqk.norm_modulate_i8(to_dev_bf16(x), branch=to_dev_bf16(br), x_out=xo, norm_type=pqk.NORM_NONE)
    torch.cuda.synchronize()
    assert np.array_equal(c.cpu().numpy(), exact_codes(h))
    assert np.array_equal(s.cpu().numpy(), np.abs(h).max(axis=1).astype(np.float32) / np.float32(127))
    assert np.array_equal(bf16_to_f64(xo), wl.bf16_bits_to_f64(_bits(h)))
