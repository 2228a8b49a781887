"""The moments of pqk_norm_modulate_i8's rows where they are exact or near the
end of fp32's range."""

import numpy as np
import pytest

from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


def _bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


# widths whose rounded reciprocal moves the mean of some constant rows, and powers of two
@pytest.mark.parametrize("C", [88, 264, 776, 2048, 3000, 5120, 6152, 7168, 8200, 13824, 16376])
@pytest.mark.parametrize("repeat", [1, 3])
def test_constant_rows_have_no_variance(C, repeat):
    """LayerNorm of a constant row is 0: scale 1 and codes 0 (its sum, C times a bf16 number, is exact in fp32, as is
    that sum divided by C). A shift then is the whole row."""
    torch = torch_cuda()
    value = np.concatenate([(128 + np.arange(128)) * 2.0 ** e for e in (-7, -40, 10)]) * np.tile([1, -1], 192)
    x = to_dev_bf16(np.tile(_bits(np.repeat(value[:, None], C, axis=1)), (repeat, 1)))
    _, c, s = pqk.norm_modulate_i8(x, norm_type=pqk.NORM_LAYER)
    # a branch of a quarter: 1.25 c has at most 11 bits, the sum of up to 64 of them 17, and sums of whole chunks of 8
    # up to C = 16,384 at most 25 with three zeros at the end, so all of them are exact
    xo, c2, s2 = pqk.norm_modulate_i8(x, branch=(x.float() / 4).to(torch.bfloat16), norm_type=pqk.NORM_LAYER,
                                      x_out=torch.empty_like(x))
    shift = to_dev(np.full((1, C), -2.0, np.float32))
    cu = to_dev(np.array([0, x.shape[0]], np.int32))
    _, c3, s3 = pqk.norm_modulate_i8(x, shift=shift, scale=torch.ones_like(shift), cu_seqlens=cu,
                                     norm_type=pqk.NORM_LAYER)
    torch.cuda.synchronize()
    assert (s == 1.0).all() and not c.any()
    assert (s2 == 1.0).all() and not c2.any()
    assert (s3 == torch.tensor(2.0) / 127).all() and (c3 == -127).all()


@pytest.mark.parametrize("C", [256, 1504, 5120, 16384])
@pytest.mark.parametrize("norm", [pqk.NORM_RMS, pqk.NORM_LAYER])
@pytest.mark.parametrize("T", [3, 320])
def test_mean_squares_up_to_the_end_of_the_range(C, norm, T):
    """A row's mean square may be anywhere in fp32's range, whatever the sum of its C squares is; past it the row is
    marked. Neighbours of either kind are not touched. The bound is that of rows of ordinary size: their rounding
    errors do not depend on the power of two in front."""
    torch = torch_cuda()
    g = np.random.default_rng(C + norm + T)
    x = g.standard_normal((T, C))
    x[:, 0] += 0.5
    plain = x.copy()
    big = np.arange(T) % 3 == 0                                       # mean squares near 2^126.7: sums past the range
    past = np.arange(T) % 3 == 1                                      # and near 2^130
    x[big] *= 2.0 ** 63.35
    x[past] *= 2.0 ** 65
    w = _bits(g.uniform(0.5, 1.5, C))
    bits = _bits(x)
    _, c, s = pqk.norm_modulate_i8(to_dev_bf16(bits), weight=to_dev_bf16(w), norm_type=norm)
    torch.cuda.synchronize()
    c, s = c.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    xd = wl.bf16_bits_to_f64(bits)
    h = xd - (xd.mean(1, keepdims=True) if norm == pqk.NORM_LAYER else 0)
    ms = (h * h).mean(1, keepdims=True)
    top = float(np.finfo(np.float32).max)
    assert (ms[big] < 0.95 * top).all() and (C * ms[big] > 2 * top).all() and (ms[past] > 1.5 * top).all()
    h = h / np.sqrt(ms + 1e-6) * wl.bf16_bits_to_f64(w)
    assert np.isnan(s[past]).all() and not c[past].any()
    keep = ~past
    ref = np.abs(h[keep]).max(axis=1) / 127
    assert (np.abs(s[keep] - ref) <= 128 * 2.0 ** -24 * 2 * ref).all()
    assert (np.abs(c[keep] - h[keep] / ref[:, None]) <= 0.5 + 127 * 256 * 2.0 ** -24).all()
    _, c0, s0 = pqk.norm_modulate_i8(to_dev_bf16(_bits(plain)), weight=to_dev_bf16(w), norm_type=norm)
    rest = ~(big | past)
    assert np.array_equal(c[rest], c0.cpu().numpy()[rest])
    assert np.array_equal(s[rest], s0.cpu().numpy().astype(np.float64)[rest])
