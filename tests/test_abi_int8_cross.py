"""Refusals of the int8 norm, the int8 linear layers and cross-attention: by
the C ABI on the host, before any CUDA call, and by the Python binding's
checks of its tensors (CPU only)."""

import pytest

from packed_attention_qk_b200 import build as pqk_build
from packed_attention_qk_b200 import pqk

ERR_INVALID, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_WORKSPACE = -1, -2, -3, -5
A = 0x10000  # a 16-byte aligned fake device address; never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    pqk_build.build()
    return pqk.lib()


def norm(L, **kw):
    a = dict(x=A, xs=256, br=A + 4096, brs=256, xo=None, xos=0, h8=A, hs=256, sc=A, w=None, shift=A, scale=A, gr=A,
             cu=A, B=2, T=8, C=256, nt=0, eps=1e-6)
    a.update(kw)
    return L.pqk_norm_modulate_i8(a["x"], a["xs"], a["br"], a["brs"], a["xo"], a["xos"], a["h8"], a["hs"], a["sc"],
                                  a["w"], a["shift"], a["scale"], a["gr"], a["cu"], a["B"], a["T"], a["C"], a["nt"],
                                  a["eps"], None)


@pytest.mark.parametrize("kw, want", [
    (dict(C=250, xs=256), ERR_INVALID), (dict(C=16392, xs=16392, brs=16392, hs=16392), ERR_INVALID),
    (dict(C=0), ERR_INVALID), (dict(nt=3), ERR_INVALID), (dict(eps=0.0), ERR_INVALID),
    (dict(eps=float("nan")), ERR_INVALID), (dict(T=-1), ERR_INVALID), (dict(T=2 ** 31 - 1), ERR_INVALID),
    (dict(shift=None), ERR_INVALID), (dict(scale=None), ERR_INVALID),         # both or neither
    (dict(br=None), ERR_INVALID),                                              # a gate without its branch
    (dict(cu=None), ERR_INVALID), (dict(B=0), ERR_INVALID),                    # request vectors without requests
    (dict(xs=248), ERR_INVALID), (dict(brs=128), ERR_INVALID), (dict(hs=128), ERR_INVALID),
    (dict(xo=A + 8192, xos=128), ERR_INVALID), (dict(xo=A, xos=264), ERR_INVALID),   # in place, another stride
    (dict(xo=A + 4096, xos=264), ERR_INVALID),
    (dict(x=None), ERR_INVALID), (dict(h8=None), ERR_INVALID), (dict(sc=None), ERR_INVALID),
    (dict(x=A + 8), ERR_MISALIGNED), (dict(br=A + 8), ERR_MISALIGNED), (dict(xo=A + 8, xos=256), ERR_MISALIGNED),
    (dict(h8=A + 8), ERR_MISALIGNED), (dict(sc=A + 2), ERR_MISALIGNED), (dict(w=A + 2), ERR_MISALIGNED),
    (dict(shift=A + 4), ERR_MISALIGNED), (dict(gr=A + 4), ERR_MISALIGNED), (dict(xs=260), ERR_MISALIGNED),
    (dict(hs=260), ERR_MISALIGNED), (dict(brs=257), ERR_MISALIGNED),
    (dict(T=0, x=None, h8=None, sc=None), 0),
])
def test_norm_modulate_i8_host_errors(L, kw, want):
    assert norm(L, **kw) == want


def test_quantize_i8_host_errors(L):
    f = lambda **k: L.pqk_quantize_i8(k.get("x", A), k.get("xs", 256), k.get("T", 8), k.get("C", 256),
                                      k.get("x8", A), k.get("x8s", 256), k.get("sc", A), None)
    assert f(C=12) == ERR_INVALID
    assert f(x8s=248) == ERR_INVALID
    assert f(sc=None) == ERR_INVALID
    assert f(x=A + 2) == ERR_MISALIGNED
    assert f(x8s=260) == ERR_MISALIGNED
    assert f(T=0, x=None) == 0


def lin(L, **kw):
    a = dict(a8=A, as_=256, asc=A, w8=A, ws=256, wsc=A, x=A, xs=512, gr=A, cu=A, B=2, out=A, os=512, T=300, K=256,
             N=512)
    a.update(kw)
    return L.pqk_linear_i8_gated_residual(a["a8"], a["as_"], a["asc"], a["w8"], a["ws"], a["wsc"], a["x"], a["xs"],
                                          a["gr"], a["cu"], a["B"], a["out"], a["os"], a["T"], a["K"], a["N"], None)


@pytest.mark.parametrize("kw, want", [
    (dict(K=12), ERR_INVALID), (dict(N=4), ERR_INVALID), (dict(K=0), ERR_INVALID), (dict(T=-1), ERR_INVALID),
    (dict(T=2 ** 31), ERR_INVALID), (dict(K=131072, as_=131072, ws=131072), ERR_INVALID),   # int32 sums
    (dict(as_=128), ERR_INVALID), (dict(ws=128), ERR_INVALID), (dict(os=256), ERR_INVALID), (dict(xs=256), ERR_INVALID),
    (dict(gr=None), ERR_INVALID), (dict(x=None), ERR_INVALID), (dict(cu=None), ERR_INVALID), (dict(B=0), ERR_INVALID),
    (dict(a8=None), ERR_INVALID), (dict(asc=None), ERR_INVALID), (dict(wsc=None), ERR_INVALID),
    (dict(os=520), ERR_INVALID),                                                             # in place, another stride
    (dict(a8=A + 8), ERR_MISALIGNED), (dict(w8=A + 8), ERR_MISALIGNED), (dict(wsc=A + 4), ERR_MISALIGNED),
    (dict(asc=A + 2), ERR_MISALIGNED), (dict(out=A + 2), ERR_MISALIGNED), (dict(as_=264), ERR_MISALIGNED),
    (dict(ws=264), ERR_MISALIGNED), (dict(out=A + 4096, os=516), ERR_MISALIGNED),
    (dict(T=2 ** 31 - 300, N=2 ** 30, xs=2 ** 30, os=2 ** 30), ERR_INVALID),                 # output tiles
    (dict(T=0, a8=None), 0),
])
def test_linear_i8_gated_residual_host_errors(L, kw, want):
    assert lin(L, **kw) == want


def test_linear_i8_swiglu_host_errors(L):
    f = lambda **k: L.pqk_linear_i8_swiglu(k.get("a8", A), k.get("as_", 256), k.get("asc", A), k.get("w8", A),
                                           k.get("ws", 256), k.get("wsc", A), k.get("act", A), k.get("acts", 512),
                                           k.get("T", 300), k.get("K", 256), k.get("F", 512), None)
    assert f(K=20) == ERR_INVALID
    assert f(F=4) == ERR_INVALID
    assert f(K=131072, as_=131072, ws=131072) == ERR_INVALID
    assert f(acts=500) == ERR_INVALID
    assert f(wsc=None) == ERR_INVALID
    assert f(act=A + 4) == ERR_MISALIGNED
    assert f(ws=264) == ERR_MISALIGNED
    assert f(T=2 ** 31 - 300, F=2 ** 30, acts=2 ** 30) == ERR_INVALID
    assert f(T=0) == 0


def cross(L, **kw):
    a = dict(q=A, k=A, v=A, o=A, lse=None, qs=1024, ks=512, vs=512, os=1024, cq=A, ck=A, B=2, Tq=300, Tk=77, H=8,
             Hkv=4, D=128, scale=0.1, ws=A, wsb=1 << 30)
    a.update(kw)
    return L.pqk_varlen_cross_attn_fwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["qs"], a["ks"], a["vs"], a["os"],
                                       a["cq"], a["ck"], a["B"], a["Tq"], a["Tk"], a["H"], a["Hkv"], a["D"],
                                       a["scale"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, want", [
    (dict(D=96), ERR_UNSUPPORTED), (dict(B=0), ERR_INVALID), (dict(H=0), ERR_INVALID), (dict(Hkv=0), ERR_INVALID),
    (dict(Hkv=3), ERR_INVALID), (dict(H=4, Hkv=8), ERR_INVALID), (dict(Tq=-1), ERR_INVALID), (dict(Tk=-1), ERR_INVALID),
    (dict(Tq=2 ** 31 - 100), ERR_INVALID), (dict(Tk=2 ** 31 - 100), ERR_INVALID),
    (dict(scale=0.0), ERR_INVALID), (dict(scale=float("inf")), ERR_INVALID), (dict(scale=float("nan")), ERR_INVALID),
    (dict(qs=512), ERR_INVALID), (dict(ks=256), ERR_INVALID), (dict(vs=256), ERR_INVALID), (dict(os=512), ERR_INVALID),
    (dict(q=None), ERR_INVALID), (dict(k=None), ERR_INVALID), (dict(v=None), ERR_INVALID), (dict(o=None), ERR_INVALID),
    (dict(cq=None), ERR_INVALID), (dict(ck=None), ERR_INVALID),
    (dict(q=A + 8), ERR_MISALIGNED), (dict(k=A + 8), ERR_MISALIGNED), (dict(v=A + 8), ERR_MISALIGNED),
    (dict(o=A + 8), ERR_MISALIGNED), (dict(lse=A + 2), ERR_MISALIGNED), (dict(qs=1028), ERR_MISALIGNED),
    (dict(vs=516), ERR_MISALIGNED), (dict(os=1028), ERR_MISALIGNED),
    (dict(ws=None), ERR_WORKSPACE), (dict(wsb=4096), ERR_WORKSPACE), (dict(ws=A + 8), ERR_MISALIGNED),
    (dict(Tq=2 ** 31 - 600, H=4096, Hkv=1, qs=4096 * 128, os=4096 * 128), ERR_INVALID),      # work tiles
    (dict(Tq=0, q=None), 0),
])
def test_varlen_cross_attn_host_errors(L, kw, want):
    assert cross(L, **kw) == want


def test_cross_attn_workspace_size(L):
    f = L.pqk_varlen_cross_attn_workspace_size
    assert f(0, 128) == 0 and f(-1, 128) == 0 and f(2, 96) == 0
    assert 0 < f(1, 64) < f(1, 128) < f(100000, 128)


def test_binding_refuses_wrong_tensors_before_the_library_sees_them():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c8, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        pqk.quantize_i8(x)
    with pytest.raises(ValueError, match="norm_modulate_i8: x is torch.float32, not bfloat16"):
        pqk.norm_modulate_i8(x.float())
    with pytest.raises(ValueError, match="has shape"):
        pqk.quantize_i8(x[0])
    with pytest.raises(ValueError, match="a8 is torch.uint8"):
        pqk.linear_i8_gated_residual(c8.view(torch.uint8), s, c8, s)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        pqk.linear_i8_swiglu(c8, s, c8, s)
    with pytest.raises(ValueError, match="q has shape"):
        pqk.varlen_cross_attn_fwd(x, q, q, None, None)
    with pytest.raises(ValueError, match="x is not a tensor"):
        pqk.quantize_i8(None)
