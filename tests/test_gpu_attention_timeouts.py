"""Attention calls of many work units under timeouts about as long as their
waits: a wait that runs out in the middle of a unit's keys ends the block's
work there. Each call either reports the timeout or has computed everything."""

import numpy as np
import pytest

from packed_attention_qk_b200 import pqk
from tests.gpu_utils import torch_cuda

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.mark.parametrize("cross", [True, False])
@pytest.mark.parametrize("ns", [1000, 2000, 4000, 8000])
def test_a_call_reports_its_timeout_or_is_complete(cross, ns):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(ns)
    H, D, lens = 16, 128, [2000, 1, 700, 300, 129] * 4
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens)
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))

    def call(o=None):
        if cross:
            return pqk.varlen_cross_attn_fwd(q, k, v, cu, cu, o=o)[0]
        return pqk.varlen_attn_fwd(q, k, v, cu, o=o)[0]

    want = call()
    assert pqk.get_device_status() == 0
    wide = torch.full((T + 16, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pqk.set_wait_timeout_ns(ns)
    try:
        for _ in range(5):
            wide.fill_(7.0)
            call(wide[8:8 + T])
            status = pqk.get_device_status()
            assert status in (0, TIMEOUT)
            assert status == TIMEOUT or torch.equal(wide[8:8 + T], want)
            assert (wide[:8] == 7.0).all() and (wide[8 + T:] == 7.0).all()
    finally:
        pqk.set_wait_timeout_ns(0)
    assert torch.equal(call(), want) and pqk.get_device_status() == 0
