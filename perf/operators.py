"""The operators of a block's quantised cross-attention sub-layer, as cases to measure.

Three operators, each with its plain form (elementary torch operations in 32 bits) and the library's call:

  norm    x' = x + gate * branch, normalised, modulated and written as int8 with one scale per token
          (``pqk.norm_modulate_i8``), and the quantisation of a tensor's rows alone (``pqk.quantize_i8``)
  linear  the product of int8 tokens and int8 weights with scales for each token and output channel, with the
          gated residual (``pqk.linear_i8_gated_residual``) or SwiGLU (``pqk.linear_i8_swiglu``) behind it
  cross   attention of packed query tokens to another packed sequence, an encoder's states
          (``pqk.varlen_cross_attn_fwd``)

A case is a dict of plain values; ragged lengths are texts such as "200,312".
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6


def _lens(text):
    return [int(v) for v in text.split(",")]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token per request at the pooled conditioning vector of a small block: latency
        {"name": "norm_2_tokens", "op": "norm", "lens": "1,1", "C": 2048, "norm": "rms", "branch": True, "mod": True,
         "weight": False},
        # one joint sequence of 4,096 tokens (text, audio, video) entering its cross-attention sub-layer
        {"name": "norm_4096", "op": "norm", "lens": "4096", "C": 2048, "norm": "layer", "branch": True, "mod": True,
         "weight": False},
        # a 58,048-token clip at hidden 5,120: residual, norm and modulation in front of the first linear layer
        {"name": "norm_58048", "op": "norm", "lens": "58048", "C": 5120, "norm": "rms", "branch": True, "mod": True,
         "weight": False},
        # SwiGLU's output in front of the last linear layer: rows quantised, no norm; an odd token count
        {"name": "quantize_12345", "op": "norm", "lens": "12345", "C": 13824, "norm": "none", "branch": False,
         "mod": False, "weight": False},
        # a pooled token through one projection: latency, the weight's bytes
        {"name": "linear_1_token", "op": "linear", "lens": "1", "K": 5120, "N": 5120, "epi": "none"},
        # two text prompts projected to an encoder's keys
        {"name": "linear_text_389", "op": "linear", "lens": "77,312", "K": 2048, "N": 5120, "epi": "none"},
        # the output projection of 4 requests with its gated residual; ragged lengths
        {"name": "linear_residual_12345", "op": "linear", "lens": "200,312,4096,7737", "K": 5120, "N": 5120,
         "epi": "residual"},
        # the feed-forward's first layer with SwiGLU on a whole 58,048-token clip
        {"name": "linear_swiglu_58048", "op": "linear", "lens": "58048", "K": 5120, "N": 13824, "epi": "swiglu"},
        # two small requests and their prompts: latency
        {"name": "cross_tiny", "op": "cross", "lens_q": "200,312", "lens_k": "77,120", "H": 4, "Hkv": 4, "D": 64},
        # the video tokens of a clip over its text states
        {"name": "cross_video_text", "op": "cross", "lens_q": "55296", "lens_k": "512", "H": 40, "Hkv": 40, "D": 128},
        # audio over video, video over audio, a long clip over a short prompt, and a request without a prompt
        {"name": "cross_ragged", "op": "cross", "lens_q": "2240,12345,29024,512", "lens_k": "12345,2240,77,0",
         "H": 16, "Hkv": 16, "D": 128},
        # one summary token per request over all of its video tokens, key heads shared by pairs
        {"name": "cross_1_query", "op": "cross", "lens_q": "1,1,1", "lens_k": "55296,29024,12345", "H": 16, "Hkv": 8,
         "D": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total):
    """`total` in one to four parts, each at least 1 where it can be."""
    parts = rng.randint(1, 4)
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return ",".join(str(n) for n in lens)


def draw(rng):
    op = rng.choice(["norm", "linear", "cross"])
    if op == "norm":
        C = 8 * _log_int(rng, 8, 2048)
        T = _log_int(rng, 1, min(58000, 55296 * 5120 // C))
        norm = rng.choice(["rms", "rms", "layer", "none"])
        return {"op": op, "lens": _split(rng, T), "C": C, "norm": norm, "branch": rng.random() < 0.6,
                "mod": rng.random() < 0.6, "weight": norm != "none" and rng.random() < 0.5}
    if op == "linear":
        K, N = 8 * _log_int(rng, 8, 1728), 8 * _log_int(rng, 1, 1728)
        epi = rng.choice(["none", "residual", "swiglu"])
        T = _log_int(rng, 1, min(58000, max(1, 58000 * 5120 // K * 13824 // N)))
        return {"op": op, "lens": _split(rng, T), "K": K, "N": N, "epi": epi}
    D = rng.choice([64, 128])
    Hkv = _log_int(rng, 1, 20)
    H = Hkv * rng.choice([1, 1, 2])
    B = rng.randint(1, 4)
    room = 55296 * 512 * 40 // (B * H)
    lens_q, lens_k = [], []
    for _ in range(B):
        nq = _log_int(rng, 1, 56000)
        lens_q.append(nq)
        lens_k.append(0 if rng.random() < 0.05 else _log_int(rng, 1, min(56000, room // nq)))
    return {"op": op, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)), "H": H, "Hkv": Hkv,
            "D": D}


def work(case):
    if case["op"] == "norm":
        lens, C = _lens(case["lens"]), case["C"]
        T, B = sum(lens), len(lens)
        per = 2 + 1 + (4 if case["branch"] else 0)  # x, the codes; branch and x'
        params = (B * C * 4 if case["branch"] else 0) + (2 * B * C * 4 if case["mod"] else 0) + \
            (2 * C if case["weight"] else 0)
        return {"bytes": T * C * per + 4 * T + params, "flops": 8 * T * C}
    if case["op"] == "linear":
        lens, K, N = _lens(case["lens"]), case["K"], case["N"]
        T, rows = sum(lens), (2 * N if case["epi"] == "swiglu" else N)
        extra = T * N * 2 + len(lens) * N * 4 if case["epi"] == "residual" else 0
        return {"bytes": T * K + rows * K + 4 * T + 4 * rows + T * N * 2 + extra, "flops": 2 * T * K * rows}
    q, k = _lens(case["lens_q"]), _lens(case["lens_k"])
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    pairs = sum(a * b for a, b in zip(q, k))
    return {"bytes": 4 * sum(q) * H * D + 4 * sum(q) * H + 4 * sum(k) * Hkv * D, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------- inputs

def _quantised_rows(g, rows, cols, std):
    """Random rows quantised as a model's are: codes and one scale per row."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * std
    scale = v.abs().amax(1).clamp_min(1e-30) / 127
    return torch.round(v / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        lens, C = _lens(case["lens"]), case["C"]
        T, B = sum(lens), len(lens)
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
        s["x"] = normal(T, C)
        if case["branch"]:
            s["branch"], s["gate"] = normal(T, C), normal(B, C, std=0.1, dtype=torch.float32)
        if case["mod"]:
            s["shift"], s["scale"] = (normal(B, C, std=0.1, dtype=torch.float32) for _ in range(2))
        if case["weight"]:
            s["weight"] = (torch.rand(C, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    elif case["op"] == "linear":
        lens, K, N = _lens(case["lens"]), case["K"], case["N"]
        T, B = sum(lens), len(lens)
        rows = 2 * N if case["epi"] == "swiglu" else N
        Kp = (K + 15) // 16 * 16  # rows of codes start on 16-byte boundaries
        for name, n, std in (("a", T, 1.0), ("w", rows, K ** -0.5)):
            codes, scales = _quantised_rows(g, n, K, std)
            wide = torch.zeros(n, Kp, dtype=torch.int8, device="cuda")
            wide[:, :K] = codes
            s[name + "8"], s[name + "_scale"] = wide[:, :K], scales
        if case["epi"] == "residual":
            s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
            s["x"], s["gate"] = normal(T, N), normal(B, N, std=0.1, dtype=torch.float32)
    else:
        q, k, H, Hkv, D = _lens(case["lens_q"]), _lens(case["lens_k"]), case["H"], case["Hkv"], case["D"]
        s["q"], s["k"], s["v"] = normal(sum(q), H, D), normal(sum(k), Hkv, D), normal(sum(k), Hkv, D)
        s["cu_q"] = torch.tensor(_cu(q), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(_cu(k), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def _dequantised(codes, scale):
    """What the codes stand for, in bf16: one pass."""
    return torch.mul(codes, scale[:, None], out=torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device))


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "linear": _plain_linear, "cross": _plain_cross}[s["case"]["op"]](s)


def _run_own(s):
    from packed_attention_qk_b200 import pqk
    case = s["case"]
    if case["op"] == "norm":
        if case["norm"] == "none" and not (case["branch"] or case["mod"]):
            codes, scale = pqk.quantize_i8(s["x"])
            return {"h": _dequantised(codes, scale), "scale": scale}
        x_out = torch.empty_like(s["x"]) if case["branch"] else None
        _, codes, scale = pqk.norm_modulate_i8(
            s["x"], branch=s.get("branch"), gate_res=s.get("gate"), weight=s.get("weight"), shift=s.get("shift"),
            scale=s.get("scale"), cu_seqlens=s["cu"], eps=EPS, x_out=x_out,
            norm_type={"rms": pqk.NORM_RMS, "layer": pqk.NORM_LAYER, "none": pqk.NORM_NONE}[case["norm"]])
        out = {"h": _dequantised(codes, scale), "scale": scale}
        if case["branch"]:
            out["x"] = x_out
        return out
    if case["op"] == "linear":
        if case["epi"] == "swiglu":
            return pqk.linear_i8_swiglu(s["a8"], s["a_scale"], s["w8"], s["w_scale"])
        return pqk.linear_i8_gated_residual(s["a8"], s["a_scale"], s["w8"], s["w_scale"], x=s.get("x"),
                                            gate_res=s.get("gate"), cu_seqlens=s.get("cu"))
    o, lse = pqk.varlen_cross_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], want_lse=True)
    return {"o": o, "lse": lse}


def _request_of(cu, T):
    """The request of each of T tokens."""
    return torch.searchsorted(cu, torch.arange(T, device=cu.device, dtype=cu.dtype), right=True) - 1


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    req = _request_of(s["cu"], x.shape[0])
    out = {}
    if case["branch"]:
        x = x + s["gate"][req] * s["branch"].float()
        out["x"] = x.to(torch.bfloat16)
    if case["norm"] == "layer":
        x = x - x.mean(1, keepdim=True)
    if case["norm"] != "none":
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    if case["weight"]:
        x = x * s["weight"].float()
    if case["mod"]:
        x = x * (1 + s["scale"][req]) + s["shift"][req]
    amax = x.abs().amax(1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 127)
    codes = torch.round(x / scale[:, None]).clamp(-127, 127)
    out["h"], out["scale"] = (codes * scale[:, None]).to(torch.bfloat16), scale
    return out


def _plain_linear(s):
    case = s["case"]
    y = (s["a8"].float() @ s["w8"].float().t()) * s["a_scale"][:, None] * s["w_scale"]
    if case["epi"] == "swiglu":
        gate, up = y[:, :case["N"]], y[:, case["N"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    elif case["epi"] == "residual":
        y = s["x"].float() + s["gate"][_request_of(s["cu"], y.shape[0])] * y
    return y.to(torch.bfloat16)


def _plain_cross(s):
    case = s["case"]
    group = case["H"] // case["Hkv"]
    q, k, v = (t.float().transpose(0, 1) for t in (s["q"], s["k"], s["v"]))  # [heads, tokens, D]
    k, v = k.repeat_interleave(group, 0), v.repeat_interleave(group, 0)
    cq, ck = _cu(_lens(case["lens_q"])), _cu(_lens(case["lens_k"]))
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    for b in range(len(cq) - 1):
        rows, keys = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        if cq[b] == cq[b + 1] or ck[b] == ck[b + 1]:
            continue
        scores = (q[:, rows] @ k[:, keys].transpose(1, 2)) * case["D"] ** -0.5
        top = scores.amax(2, keepdim=True)
        scores = torch.exp(scores - top)
        total = scores.sum(2, keepdim=True)
        o[:, rows] = (scores @ v[:, keys]) / total
        lse[:, rows] = (top + torch.log(total))[..., 0]
    return {"o": o.transpose(0, 1).to(torch.bfloat16).contiguous(), "lse": lse}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "cross": _exact_cross}[case["op"]](case, s)


def _exact_norm(case, s):
    h_all, scales, xs = [], [], []
    cu = _cu(_lens(case["lens"]))
    for b in range(len(cu) - 1):  # request by request, so that its vectors broadcast
        x = s["x"][cu[b]:cu[b + 1]].double()
        if case["branch"]:
            x = torch.addcmul(x, s["branch"][cu[b]:cu[b + 1]].double(), s["gate"][b].double())
            xs.append(x)
        if case["norm"] == "rms":
            h = x * x.square().mean(-1, keepdim=True).add(EPS).rsqrt()
        elif case["norm"] == "layer":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            h = (x - mean) * (var + EPS).rsqrt()
        else:
            h = x
        if case["weight"]:
            h = h * s["weight"].double()
        if case["mod"]:
            h = h + h * s["scale"][b].double() + s["shift"][b].double()
        step = torch.linalg.vector_norm(h, math.inf, -1) / 127
        step[step == 0] = 1.0
        scales.append(step)
        h_all.append((h / step[:, None]).round_().mul_(step[:, None]))
    out = {"h": torch.cat(h_all), "scale": torch.cat(scales)}
    if case["branch"]:
        out["x"] = torch.cat(xs)
    return out


def _exact_linear(case, s):
    a, N = s["a8"].double() * s["a_scale"].double()[:, None], case["N"]
    w = s["w8"].double() * s["w_scale"].double()[:, None]
    if case["epi"] == "swiglu":
        gate = a @ w[:N].t()
        return gate * torch.sigmoid(gate) * (a @ w[N:].t())
    y = a @ w.t()
    if case["epi"] == "residual":
        cu = _cu(_lens(case["lens"]))
        for b in range(len(cu) - 1):
            y[cu[b]:cu[b + 1]] *= s["gate"][b].double()
        y += s["x"].double()
    return y


def _exact_cross(case, s):
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    o, lse = torch.zeros_like(q), torch.full((case["H"], q.shape[0]), -math.inf, device=q.device, dtype=torch.float64)
    cq, ck = _cu(_lens(case["lens_q"])), _cu(_lens(case["lens_k"]))
    for b in range(len(cq) - 1):
        if ck[b + 1] == ck[b]:
            continue
        for h in range(case["H"]):
            kh = h * case["Hkv"] // case["H"]
            u = q[cq[b]:cq[b + 1], h] @ k[ck[b]:ck[b + 1], kh].t() / math.sqrt(case["D"])
            z = torch.logsumexp(u, 1)
            o[cq[b]:cq[b + 1], h] = torch.exp(u - z[:, None]) @ v[ck[b]:ck[b + 1], kh]
            lse[h, cq[b]:cq[b + 1]] = z
    return {"o": o, "lse": lse}
