"""The int8 norm, the int8 linear layers and cross-attention together, as a
block uses them: the cross-attention sub-layer and the feed-forward of two
ragged requests in 8-bit integers, checked stage by stage against the float64
definitions (each stage on the previous stage's own output), captured in a CUDA
graph and replayed, on two streams at once, and next to the bf16 layers that
they take the place of."""

import numpy as np
import pytest

from oracle import plain64
from packed_attention_qk_b200 import pqk
from packed_attention_qk_b200 import workloads as wl
from tests.gpu_utils import bf16_to_f64, to_dev, to_dev_bf16, torch_cuda

pytestmark = pytest.mark.gpu

H, D, F = 4, 64, 512
C = H * D


def _bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


class Sublayer:
    """Weights, activations and preallocated outputs of one call."""

    def __init__(self, lens_q, lens_k, seed):
        torch = torch_cuda()
        g = np.random.default_rng(seed)
        self.T, self.S, self.B = sum(lens_q), sum(lens_k), len(lens_q)
        self.cu_q = np.concatenate([[0], np.cumsum(lens_q)]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum(lens_k)]).astype(np.int32)
        self.host = {
            "x": _bits(g.standard_normal((self.T, C))), "branch": _bits(g.standard_normal((self.T, C))),
            "text": _bits(g.standard_normal((self.S, C))),
            **{n: (0.2 * g.standard_normal((self.B, C))).astype(np.float32)
               for n in ("gate", "shift", "scale", "gate_o", "shift_f", "scale_f", "gate_f")}}
        self.w = {n: _bits(g.standard_normal((rows, cols)) / np.sqrt(cols)) for n, rows, cols in (
            ("q", C, C), ("kv", 2 * C, C), ("o", C, C), ("w1", 2 * F, C), ("w2", C, F))}
        self.d = {n: to_dev_bf16(v) if v.dtype == np.uint16 else to_dev(v) for n, v in self.host.items()}
        self.d["cu_q"], self.d["cu_k"] = to_dev(self.cu_q), to_dev(self.cu_k)
        self.w8 = {n: pqk.quantize_i8(to_dev_bf16(v)) for n, v in self.w.items()}
        e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
        T, S = self.T, self.S
        self.o = {"x1": e(T, C), "h8": e(T, C, t=torch.int8), "hs": e(T, t=torch.float32), "q": e(T, C),
                  "t8": e(S, C, t=torch.int8), "ts": e(S, t=torch.float32), "kv": e(S, 2 * C), "att": e(T, H, D),
                  "a8": e(T, C, t=torch.int8), "as": e(T, t=torch.float32), "x2": e(T, C),
                  "f8": e(T, C, t=torch.int8), "fs": e(T, t=torch.float32), "act": e(T, F),
                  "act8": e(T, F, t=torch.int8), "acts": e(T, t=torch.float32), "x3": e(T, C),
                  "ws": e(pqk.varlen_cross_attn_workspace_size(self.B, D), t=torch.uint8)}

    def run(self):
        d, o, w8 = self.d, self.o, self.w8
        pqk.norm_modulate_i8(d["x"], branch=d["branch"], gate_res=d["gate"], shift=d["shift"], scale=d["scale"],
                             cu_seqlens=d["cu_q"], x_out=o["x1"], h8=o["h8"], h_scale=o["hs"])
        pqk.linear_i8_gated_residual(o["h8"], o["hs"], *w8["q"], out=o["q"])
        pqk.quantize_i8(d["text"], x8=o["t8"], scales=o["ts"])
        pqk.linear_i8_gated_residual(o["t8"], o["ts"], *w8["kv"], out=o["kv"])
        kv = o["kv"].view(self.S, 2, H, D)                  # K and V are halves of one buffer's rows
        pqk.varlen_cross_attn_fwd(o["q"].view(self.T, H, D), kv[:, 0], kv[:, 1], d["cu_q"], d["cu_k"], o=o["att"],
                                  workspace=o["ws"])
        pqk.quantize_i8(o["att"].view(self.T, C), x8=o["a8"], scales=o["as"])
        pqk.linear_i8_gated_residual(o["a8"], o["as"], *w8["o"], x=o["x1"], gate_res=d["gate_o"],
                                     cu_seqlens=d["cu_q"], out=o["x2"])
        pqk.norm_modulate_i8(o["x2"], shift=d["shift_f"], scale=d["scale_f"], cu_seqlens=d["cu_q"], h8=o["f8"],
                             h_scale=o["fs"], norm_type=pqk.NORM_LAYER)
        pqk.linear_i8_swiglu(o["f8"], o["fs"], *w8["w1"], act=o["act"])
        pqk.quantize_i8(o["act"], x8=o["act8"], scales=o["acts"])
        pqk.linear_i8_gated_residual(o["act8"], o["acts"], *w8["w2"], x=o["x2"], gate_res=d["gate_f"],
                                     cu_seqlens=d["cu_q"], out=o["x3"])

    def check(self):
        """Each stage's definition on the stage before as the GPU left it."""
        f, o, h = bf16_to_f64, self.o, self.host
        deq = lambda c, s: o[c].cpu().numpy().astype(np.float64) * o[s].cpu().numpy().astype(np.float64)[:, None]
        w = {n: c.cpu().numpy().astype(np.float64) * s.cpu().numpy().astype(np.float64)[:, None]
             for n, (c, s) in self.w8.items()}
        half = 2.0 ** -8

        def near(got, ref, slack, what):
            assert (np.abs(got - ref) <= half * np.abs(ref) + slack).all(), what

        hx = {n: wl.bf16_bits_to_f64(h[n]) for n in ("x", "branch", "text")}
        x1, h1 = plain64.norm_modulate(hx["x"], branch=hx["branch"], gate_res=h["gate"], shift=h["shift"],
                                       scale=h["scale"], cu_seqlens=self.cu_q)
        near(f(o["x1"]), x1, 1e-6, "x1")
        step = plain64.row_scales(h1)[:, None]
        assert (np.abs(deq("h8", "hs") - h1) <= 0.51 * step).all()
        near(f(o["q"]), deq("h8", "hs") @ w["q"].T, 1e-5, "q")
        near(f(o["kv"]), deq("t8", "ts") @ w["kv"].T, 1e-5, "kv")
        kv = f(o["kv"]).reshape(self.S, 2, H, D)
        att, _, spread = plain64.cross_attention(f(o["q"]).reshape(self.T, H, D), kv[:, 0], kv[:, 1], self.cu_q,
                                                 self.cu_k, D ** -0.5)
        near(f(o["att"]), att, (half + 2.0 ** -13) * spread + 1e-30, "attention")
        x2 = plain64.gated_residual(deq("a8", "as") @ w["o"].T, f(o["x1"]), h["gate_o"], self.cu_q)
        near(f(o["x2"]), x2, 1e-5, "x2")
        _, h2 = plain64.norm_modulate(f(o["x2"]), shift=h["shift_f"], scale=h["scale_f"], cu_seqlens=self.cu_q,
                                      norm_type=plain64.NORM_LAYER)
        assert (np.abs(deq("f8", "fs") - h2) <= 0.51 * plain64.row_scales(h2)[:, None]).all()
        near(f(o["act"]), plain64.swiglu(deq("f8", "fs") @ w["w1"].T), 1e-5, "act")
        x3 = plain64.gated_residual(deq("act8", "acts") @ w["w2"].T, f(o["x2"]), h["gate_f"], self.cu_q)
        near(f(o["x3"]), x3, 1e-5, "x3")


CASES = [([200, 312], [77, 120]), ([1, 0, 130], [9, 4, 700]), ([700, 5, 300], [64, 0, 1300])]


@pytest.mark.parametrize("lens_q, lens_k", CASES)
def test_every_stage_against_its_definition(lens_q, lens_k):
    torch = torch_cuda()
    s = Sublayer(lens_q, lens_k, seed=3)
    s.run()
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    s.check()


@pytest.mark.parametrize("lens_q, lens_k", CASES)
def test_captured_sublayer_replays_bitwise_with_new_contents(lens_q, lens_k):
    """One capture serves other activations and other lengths within the same buffers."""
    torch = torch_cuda()
    s = Sublayer(lens_q, lens_k, seed=4)
    s.run()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in s.o.items() if k != "ws"}
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            s.run()
    torch.cuda.current_stream().wait_stream(st)
    for k in s.o:
        s.o[k].zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for k, want in ref.items():
        assert torch.equal(s.o[k], want), k
    # other activations, and the text split differently between the requests
    other = Sublayer(lens_q, lens_k, seed=5)
    cu_k = other.cu_k.copy()
    cu_k[1:-1] = np.sort(np.random.default_rng(1).integers(0, s.S + 1, s.B - 1))
    other.cu_k = s.cu_k = cu_k
    other.d["cu_k"].copy_(to_dev(cu_k))
    for k, v in other.d.items():
        s.d[k].copy_(v)
    other.w8 = s.w8
    other.run()
    g.replay()
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    for k in ref:
        assert torch.equal(s.o[k], other.o[k]), k
    del g


def test_two_graphs_that_share_a_workspace_replay_in_turn():
    torch = torch_cuda()
    subs = [Sublayer([700, 5, 300], [64, 0, 1300], seed=9), Sublayer([3, 0, 130], [9, 4, 2000], seed=10)]
    subs[1].o["ws"] = subs[0].o["ws"]
    refs, graphs = [], []
    for s in subs:
        s.run()
        torch.cuda.synchronize()
        refs.append({k: v.clone() for k, v in s.o.items() if k != "ws"})
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for s in subs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                s.run()
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(st)
    for s in subs:
        for k, v in s.o.items():
            v.zero_()
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    for s, ref in zip(subs, refs):
        for k, want in ref.items():
            assert torch.equal(s.o[k], want), k
    del graphs


def test_two_streams_at_once_each_with_its_own_buffers():
    torch = torch_cuda()
    subs = [Sublayer([700, 5, 300], [64, 0, 1300], seed=6), Sublayer([1, 0, 130], [9, 4, 700], seed=7)]
    refs = []
    for s in subs:
        s.run()
        torch.cuda.synchronize()
        refs.append({k: v.clone() for k, v in s.o.items() if k != "ws"})
    streams = [torch.cuda.Stream() for _ in subs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, st in zip(subs, streams):
            with torch.cuda.stream(st):
                s.run()
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert pqk.get_device_status() == 0
    for s, ref in zip(subs, refs):
        for k, want in ref.items():
            assert torch.equal(s.o[k], want), k


def test_stands_near_the_bf16_layers_it_replaces():
    """The int8 layer is its bf16 counterpart up to the two quantisations: a step of a row's scale is 1/254 of its
    largest element either way, so a product of K terms differs by about sqrt(K) * |a| |w| * that, far below its size
    times 5 %."""
    torch = torch_cuda()
    s = Sublayer([200, 312], [77, 120], seed=8)
    s.run()
    d = s.d
    _, h, _ = pqk.modulate_swiglu(d["x"], d["shift"], d["scale"], d["cu_q"], gate_res=d["gate"], branch=d["branch"])
    q = pqk.linear_gated_residual(h, to_dev_bf16(s.w["q"]))
    torch.cuda.synchronize()
    a, b = bf16_to_f64(s.o["q"]), bf16_to_f64(q)
    assert np.linalg.norm(a - b) <= 0.05 * np.linalg.norm(b)
    assert np.linalg.norm(a - b) > 0                              # they are two computations
