"""The 256-token int8 linear kernel with rows far apart: codes, residual stream
and output rows whose last ones lie past 2^31 elements from the first."""

import pytest

from packed_attention_qk_b200 import pqk
from tests.gpu_utils import torch_cuda

pytestmark = pytest.mark.gpu


def _spread(torch, t, far):
    """t's rows, `far` elements apart."""
    wide = torch.empty((t.shape[0] - 1) * far + t.shape[1], dtype=t.dtype, device="cuda")
    view = wide.as_strided(t.shape, (far, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("epi", ["none", "residual", "swiglu"])
def test_rows_past_32_bits_in_the_256_token_kernel(epi):
    torch = torch_cuda()
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs about 25 GB")
    # 600 tokens and 3,000 or more rows of W: 36 tiles of 256 x 256, where calls of up to 24 take the small tiles
    T, K, N, far = 600, 264, 3000, 3_600_016
    assert (T - 1) * far > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = 2 * N if epi == "swiglu" else N
    a8 = torch.zeros(T, 272, dtype=torch.int8, device="cuda")[:, :K]
    a8.copy_(torch.randint(-127, 128, (T, K), generator=g, device="cuda"))
    w8 = torch.zeros(rows, 272, dtype=torch.int8, device="cuda")[:, :K]
    w8.copy_(torch.randint(-127, 128, (rows, K), generator=g, device="cuda"))
    sa, sw = torch.rand(T, generator=g, device="cuda") * 1e-2, torch.rand(rows, generator=g, device="cuda") * 1e-2
    x = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(2, N, generator=g, device="cuda")
    cu = torch.tensor([0, 333, T], dtype=torch.int32, device="cuda")

    def call(a8, x, out):
        if epi == "swiglu":
            return pqk.linear_i8_swiglu(a8, sa, w8, sw, act=out)
        if epi == "residual":
            return pqk.linear_i8_gated_residual(a8, sa, w8, sw, x=x, gate_res=gate, cu_seqlens=cu, out=out)
        return pqk.linear_i8_gated_residual(a8, sa, w8, sw, out=out)

    want = call(a8, x, None)
    # the same tokens in calls of 40, which take the other kernel: equal bits
    for t0 in (0, 320, 560):
        part = slice(t0, t0 + 40)
        if epi == "swiglu":
            few = pqk.linear_i8_swiglu(a8[part], sa[part], w8, sw)
        elif epi == "residual":
            few = pqk.linear_i8_gated_residual(a8[part], sa[part], w8, sw, x=x[part], gate_res=gate,
                                               cu_seqlens=(cu - t0).clamp(0, 40))
        else:
            few = pqk.linear_i8_gated_residual(a8[part], sa[part], w8, sw)
        assert torch.equal(few, want[part])
    a_far, x_far = _spread(torch, a8, far), _spread(torch, x, far)
    out = _spread(torch, torch.zeros_like(want), far)
    call(a_far, x_far, out)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and torch.equal(out, want)
    if epi == "residual":                                             # in place
        call(a_far, x_far, x_far)
        torch.cuda.synchronize()
        assert torch.equal(x_far, want)
