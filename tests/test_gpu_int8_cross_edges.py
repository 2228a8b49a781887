"""The int8 norm, the int8 linear layers and cross-attention away from the
usual call: waits that run out (bounded, reported, recovered), a first call of
its size under capture, a stream of the caller's choice, offsets past 2^31
elements, and outputs that are inputs."""

import contextlib
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from tests.gpu_utils import bf16_to_f64, torch_cuda

pytestmark = pytest.mark.gpu

TIMEOUT = -6
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@contextlib.contextmanager
def short_timeout(ns):
    pqk.set_wait_timeout_ns(ns)
    try:
        yield
    finally:
        pqk.set_wait_timeout_ns(0)


def _runs_out(call, tries=3):
    """Runs call() under the shortest timeout (1 us) until a wait runs out."""
    with short_timeout(1000):
        for _ in range(tries):
            call()
            st = pqk.get_device_status()
            assert st in (0, TIMEOUT), f"unexpected status {st}"
            if st == TIMEOUT:
                return True
    return False


def _guarded(torch, rows, cols, dtype=None):
    wide = torch.full((rows + 16, cols + 64), 7.0, dtype=dtype or torch.bfloat16, device="cuda")
    return wide, wide[8:8 + rows, :cols]


def _intact(wide, rows, cols):
    return bool((wide[:8] == 7.0).all() and (wide[8 + rows:] == 7.0).all() and (wide[8:8 + rows, cols:] == 7.0).all())


# K so long that the wait for an accumulator, tens of microseconds, outlasts what a poll itself may take
@pytest.mark.parametrize("T, K, N", [(1, 131056, 512), (40, 131056, 512), (200, 131056, 512), (2048, 16384, 2048)])
@pytest.mark.parametrize("epi", ["residual", "swiglu"])
def test_linear_timeout_is_reported_drained_and_recovered(T, K, N, epi):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = 2 * N if epi == "swiglu" else N
    a8 = torch.randint(-127, 128, (T, K), generator=g, device="cuda").to(torch.int8)
    w8 = torch.randint(-127, 128, (rows, K), generator=g, device="cuda").to(torch.int8)
    sa, sw = torch.full((T,), 1e-4, device="cuda"), torch.full((rows,), 1e-2, device="cuda")
    x = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(1, N, generator=g, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def call(out):
        if epi == "swiglu":
            return pqk.linear_i8_swiglu(a8, sa, w8, sw, act=out)
        return pqk.linear_i8_gated_residual(a8, sa, w8, sw, x=x, gate_res=gate, cu_seqlens=cu, out=out)

    wide, out = _guarded(torch, T, N)
    want = call(None)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    assert _runs_out(lambda: call(out))
    assert _intact(wide, T, N)
    again = call(out)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and torch.equal(again, want)


@pytest.mark.parametrize("lens_q, lens_k", [([1000, 1, 129], [4096, 3000, 0]), ([1], [9000]), ([9000], [300])])
@pytest.mark.parametrize("D", [64, 128])
def test_cross_attention_timeout_is_reported_drained_and_recovered(lens_q, lens_k, D):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    H, T = 8, sum(lens_q)
    r = lambda n, h: torch.randn(n, h, D, generator=g, device="cuda").to(torch.bfloat16)
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (lens_q, lens_k)]
    q, k, v = r(T, H), r(sum(lens_k), 4), r(sum(lens_k), 4)
    want, lse = pqk.varlen_cross_attn_fwd(q, k, v, *cu, want_lse=True)
    wide, out = _guarded(torch, T, H * D)
    assert _runs_out(lambda: pqk.varlen_cross_attn_fwd(q, k, v, *cu, o=out.unflatten(1, (H, D))))
    assert _intact(wide, T, H * D)
    o2, lse2 = pqk.varlen_cross_attn_fwd(q, k, v, *cu, want_lse=True)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and torch.equal(o2, want) and torch.equal(lse2, lse)


CAPTURE = r'''
import torch
from packed_attention_qk_b200 import pqk
g = torch.Generator(device="cuda").manual_seed(3)
i8 = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda").to(torch.int8)
bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
cu = lambda *c: torch.tensor(c, dtype=torch.int32, device="cuda")
w, sw = i8(1024, 512), torch.rand(1024, generator=g, device="cuda") * 1e-3
sets = [(i8(T, 512), torch.rand(T, generator=g, device="cuda") * 1e-2) for T in (1, 40, 100, 300, 5000)]
x = bf(300, 2048)
q, k, v = bf(700, 4, 64), bf(5000, 4, 64), bf(5000, 4, 64)
q2, k2, v2 = bf(3, 4, 128), bf(2000, 2, 128), bf(2000, 2, 128)
many = cu(*range(0, 41))

def calls():
    out = [pqk.linear_i8_gated_residual(a, s, w, sw) for a, s in sets]
    out += [pqk.linear_i8_swiglu(a, s, w, sw) for a, s in sets]
    out += list(pqk.quantize_i8(x)) + list(pqk.norm_modulate_i8(x)[1:]) + list(pqk.quantize_i8(x[:5]))
    out += list(pqk.varlen_cross_attn_fwd(q, k, v, cu700, cu5000, want_lse=True))
    out += list(pqk.varlen_cross_attn_fwd(q2, k2, v2, cu3, cu2000, want_lse=True))
    out += list(pqk.varlen_cross_attn_fwd(q, k, v, many, many, want_lse=False))[:1]
    return out

cu700, cu5000, cu3, cu2000 = cu(0, 300, 700), cu(0, 4000, 5000), cu(0, 3), cu(0, 2000)
# one call of each entry point on the device, of one size, as the header asks
pqk.linear_i8_gated_residual(*sets[0], w, sw); pqk.linear_i8_swiglu(*sets[0], w, sw)
pqk.quantize_i8(x); pqk.norm_modulate_i8(x)
pqk.varlen_cross_attn_fwd(q2, k2, v2, cu3, cu2000)
torch.cuda.synchronize()
graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
st.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(st):
    with torch.cuda.graph(graph, stream=st):
        captured = calls()
torch.cuda.current_stream().wait_stream(st)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in captured]
want = calls()
torch.cuda.synchronize()
assert pqk.get_device_status() == 0
written = [t if i < len(want) - 1 else t[:40] for i, t in enumerate(want)]
for i, (a, b) in enumerate(zip(got, written)):
    a = a[:40] if i == len(want) - 1 else a
    assert torch.equal(a, b), i
print("same", len(want))
'''


def test_sizes_first_seen_under_capture():
    """In a process of its own: after one call of each entry point, calls of other sizes (other kernels) are captured
    first and run eagerly later."""
    torch_cuda()
    r = subprocess.run([sys.executable, "-c", CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_a_stream_of_the_callers_choice():
    """Outputs and workspaces that a call allocates are the other stream's until it is through: work on the current
    stream that allocates and overwrites memory meanwhile changes nothing."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(3, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(30000, 16, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cu_q = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, 30000], dtype=torch.int32, device="cuda")
    want, _ = pqk.varlen_cross_attn_fwd(q, k, v, cu_q, cu_k)
    torch.cuda.synchronize()
    for raw in (False, True):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = []
        for _ in range(10):
            o, _ = pqk.varlen_cross_attn_fwd(q, k, v, cu_q, cu_k, stream=side.cuda_stream if raw else side)
            outs.append(o)
            size = pqk.varlen_cross_attn_workspace_size(1, 128)
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")     # lands in freed memory of that size
        c8, s = pqk.quantize_i8(k.view(30000, -1), stream=side)
        torch.cuda.synchronize()
        assert pqk.get_device_status() == 0
        assert all(torch.equal(o, want) for o in outs)
        e8, es = pqk.quantize_i8(k.view(30000, -1))
        assert torch.equal(c8, e8) and torch.equal(s, es)


def test_offsets_past_32_bits():
    """Rows 2^26 elements apart: the last ones lie past 2^31 elements (2^32 bytes) from the first."""
    torch = torch_cuda()
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs about 40 GB")
    far, n = 1 << 26, 40
    g = torch.Generator(device="cuda").manual_seed(5)

    def spread(t):
        """t's rows, far apart."""
        wide = torch.empty((n - 1) * far + t[0].numel(), dtype=t.dtype, device="cuda")
        view = wide.as_strided(t.shape, (far,) + t.stride()[1:])
        view.copy_(t)
        return view

    x, br = (torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    xo, h8, s = torch.empty_like(x), *pqk.norm_modulate_i8(x, branch=br)[1:]
    h_far, x_far = spread(torch.zeros_like(h8)), spread(x)
    pqk.norm_modulate_i8(x_far, branch=br, x_out=x_far, h8=h_far, h_scale=torch.empty_like(s))
    pqk.norm_modulate_i8(x, branch=br, x_out=xo)
    assert torch.equal(h_far, h8) and torch.equal(x_far, xo)
    # a few rows of int8 codes and of output, in both linear kernels (N = 8,192 and 64 tokens or fewer: the small one)
    w8 = torch.randint(-127, 128, (256, 256), generator=g, device="cuda").to(torch.int8)
    sw = torch.rand(256, generator=g, device="cuda")
    y = pqk.linear_i8_gated_residual(h8, s, w8, sw)
    y_far = spread(torch.zeros_like(y))
    pqk.linear_i8_gated_residual(h_far, s, w8, sw, out=y_far)
    assert torch.equal(y_far, y)
    del h_far, x_far, y_far
    q = torch.randn(n, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(n, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    o, _ = pqk.varlen_cross_attn_fwd(q, k, v, cu, cu)
    o_far = spread(torch.zeros_like(q))
    pqk.varlen_cross_attn_fwd(spread(q), spread(k), v, cu, cu, o=o_far)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and torch.equal(o_far, o)


def test_more_than_2_to_the_31_outputs():
    """The 256-token kernel with an output of 2.2e9 elements: its last rows are those of a small call."""
    torch = torch_cuda()
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs about 10 GB")
    g = torch.Generator(device="cuda").manual_seed(6)
    T, N, K = 66000, 33280, 64
    a8 = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    w8 = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = pqk.linear_i8_gated_residual(a8, sa, w8, sw)
    assert y.numel() > 2 ** 31
    tail = pqk.linear_i8_gated_residual(a8[-40:], sa[-40:], w8, sw)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0 and torch.equal(y[-40:], tail)


def test_the_residual_stream_may_replace_the_branch():
    torch = torch_cuda()
    g = np.random.default_rng(7)
    x, br = (torch.from_numpy(g.standard_normal((300, 520)).astype(np.float32)).cuda().to(torch.bfloat16)
             for _ in range(2))
    ref, _ = plain64.norm_modulate(bf16_to_f64(x), branch=bf16_to_f64(br))
    want = pqk.norm_modulate_i8(x, branch=br)
    got = pqk.norm_modulate_i8(x, branch=br, x_out=br)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert (np.abs(bf16_to_f64(br) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-30).all()
