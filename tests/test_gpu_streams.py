"""Calls on a stream of the caller's choice while the current stream still
works on memory that it has freed. Only row operators are used: whatever
memory their outputs were given, no address depends on what it holds."""

import numpy as np
import pytest

from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_are_not_memory_that_the_current_stream_still_writes(raw):
    torch = torch_cuda()
    bits = wl.f32_to_bf16_bits(np.random.default_rng(1).standard_normal((4096, 1024)).astype(np.float32))
    x = to_dev_bf16(bits)
    want, want_s = pqk.quantize_i8(x)
    a = torch.randn(8192, 8192, device="cuda").to(torch.bfloat16)
    b = a @ a
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):                                           # some 15 ms of work
            torch.matmul(a, a, out=b)
        late = torch.full((4096, 1024), 77, dtype=torch.int8, device="cuda")
        late_s = torch.full((4096,), 5.0, device="cuda")
        del late, late_s                                              # freed here, written when the products are done
        c, s = pqk.quantize_i8(x, stream=side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert torch.equal(c, want) and torch.equal(s, want_s)
        del c, s
    # and what a call returned is not handed to its stream again while the current stream reads it
    c, s = pqk.quantize_i8(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        torch.matmul(a, a, out=b)
    copy = c.clone()
    del c, s
    pqk.quantize_i8(torch.zeros_like(x), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_the_default_streams_handle():
    """Handle 0 is the default stream, also while another stream is the current one."""
    torch = torch_cuda()
    x = torch.randn(300, 264, device="cuda").to(torch.bfloat16)
    want = pqk.quantize_i8(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = pqk.quantize_i8(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = torch.randn(70, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 20, 70], dtype=torch.int32, device="cuda")
    o, _ = pqk.varlen_cross_attn_fwd(q, q, q, cu, cu)
    o0, _ = pqk.varlen_cross_attn_fwd(q, q, q, cu, cu, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(o, o0) and pqk.get_device_status() == 0
