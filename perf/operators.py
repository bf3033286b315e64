"""Measured cases of the router, the RMS norm and the microscaled (MX) operators.

run() is one pass through an operator: in its plain form (elementary torch
operations in 32 bits, 64 where a decision lies next to a border), or, with
`own` set, through the library's entry points.  Both take what prepare()
makes from a case and a seed.

  gate      router scores -> top-k expert ids and weights
  norm      RMS norm with the residual's addition, output rows in bf16 and
            in 8 or 4 bits with block scales
  quantize  rows to MXFP4 / MXFP8 (32-element blocks, power-of-two scales)
            and the values that they stand for
  gemm      product of MX activation rows with MXFP4 weights, dense or
            grouped over experts

Rows in 8 bits are returned as their float8 values and scales, rows in
4 bits as the bf16 values that they stand for.
"""
import math

import torch

own = False

F4_MAX_EXP, F8_MAX_EXP = 2, 8     # exponent of the largest E2M1 / E4M3 value


def listed():
    return [
        # the router of one decode step of a 30B-class layer
        dict(name="gate-decode", op="gate", T=16, E=128, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, renorm=True, scale=1.0, dtype="f32"),
        # the router of a trillion-class prefill: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="gate-prefill", op="gate", T=8192, E=384, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, dtype="f32"),
        # a single token's norm
        dict(name="norm-token", op="norm", T=1, K=2048, residual=False, y=True, rows="none"),
        # a decode batch entering the MoE block: bf16 tokens for the router, 8-bit rows for the experts
        dict(name="norm-decode", op="norm", T=64, K=7168, residual=True, y=True, rows="mxfp8"),
        # the same of a prefill
        dict(name="norm-prefill", op="norm", T=8192, K=7168, residual=True, y=True, rows="mxfp8"),
        # the SwiGLU output of a ragged 30B-class prefill on its way into the down projection
        dict(name="quantize-acts", op="quantize", T=32763, K=768, dtype="bf16", fmt="mxfp4"),
        # weights of one trillion-class projection at load
        dict(name="quantize-weights", op="quantize", T=4096, K=7168, dtype="f32", fmt="mxfp4"),
        # a shared expert's gate/up on a decode batch
        dict(name="dense-decode", op="gemm", E=1, T=16, k=1, N=4096, K=7168, fmt="mxfp8", swiglu=True,
             skew=0.0),
        # the 30B-class experts on a decode batch
        dict(name="experts-decode", op="gemm", E=128, T=16, k=8, N=1536, K=2048, fmt="mxfp4",
             swiglu=True, skew=1.0),
        # the same on a prefill, experts unevenly loaded
        dict(name="experts-prefill", op="gemm", E=128, T=4096, k=8, N=1536, K=2048, fmt="mxfp4",
             swiglu=True, skew=1.0),
        # a shared expert's gate/up on a prefill
        dict(name="dense-prefill", op="gemm", E=1, T=8192, k=1, N=4096, K=7168, fmt="mxfp4", swiglu=False,
             skew=0.0),
        # one GPU's share (an eighth) of the trillion-class experts on a prefill
        dict(name="share-prefill", op="gemm", E=48, T=8192, k=1, N=4096, K=7168, fmt="mxfp8", swiglu=True,
             skew=1.0),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["gate", "norm", "quantize", "gemm", "gemm"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log(rng, 4, 384 // groups)
        top_groups = rng.randint(1, groups)
        E = groups * per
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(16, top_groups * per)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]))
    if op == "norm":
        rows = rng.choice(["none", "mxfp8", "mxfp4", "nvfp4"])
        return dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 64, 7168, 8 if rows == "none" else 32),
                    residual=rng.random() < 0.7, y=rows == "none" or rng.random() < 0.6, rows=rows)
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 32, 4096, 32), dtype=rng.choice(["bf16", "f32"]),
                    fmt=rng.choice(["mxfp4", "mxfp8"]))
    while True:
        E = rng.choice([1, _log(rng, 2, 160)])
        k = rng.randint(1, min(8, E))
        c = dict(op=op, E=E, T=_log(rng, 1, 8192), k=k, N=_log(rng, 64, 4096, 32), K=_log(rng, 64, 7168, 32),
                 fmt=rng.choice(["mxfp4", "mxfp8"]), swiglu=rng.random() < 0.5,
                 skew=0.0 if E == 1 else rng.choice([0.0, 1.0]))
        if c["T"] * k * c["N"] * c["K"] <= 3e10 and E * c["N"] * c["K"] <= 8e8:
            return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 9973 + 17)


def _tokens(g, T, K):
    """Activations with a hundredth of the channels ten times the others."""
    gain = 1.0 + 9.0 * (torch.rand(K, generator=g, device="cuda") < 0.01).float()
    return (torch.randn(T, K, generator=g, device="cuda") * gain).to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    dev = "cuda"
    c, s = case, {"case": case}
    if c["op"] == "gate":
        logits = torch.randn(c["T"], c["E"], generator=g, device=dev)
        logits += 0.5 * torch.randn(c["E"], generator=g, device=dev)
        s["logits"] = logits.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
        s["bias"] = 0.1 * torch.randn(c["E"], generator=g, device=dev) if c["bias"] else None
        if own:
            from sparse_fp4_expert_amd import moesq as m
            s["gate"] = m.Gate(c["k"], score=m.SCORE_SIGMOID if c["score"] == "sigmoid" else m.SCORE_SOFTMAX,
                               n_group=c["groups"], topk_group=c["top_groups"],
                               group_score=m.GROUP_TOP2 if c["bias"] else m.GROUP_MAX,
                               renormalize=c["renorm"], scale=c["scale"])
    elif c["op"] == "norm":
        s["x"] = _tokens(g, c["T"], c["K"])
        s["weight"] = (1.0 + 0.2 * torch.randn(c["K"], generator=g, device=dev)).to(torch.bfloat16)
        s["residual"] = _tokens(g, c["T"], c["K"]) if c["residual"] else None
    elif c["op"] == "quantize":
        if c["dtype"] == "f32":
            s["x"] = 0.02 * torch.randn(c["T"], c["K"], generator=g, device=dev)
        else:
            s["x"] = _tokens(g, c["T"], c["K"])
    else:
        E, T, k, N, K = c["E"], c["T"], c["k"], c["N"], c["K"]
        s["w"] = [torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev),
                  torch.empty(E, N, K // 32, dtype=torch.uint8, device=dev)]
        for e in range(E):
            dense = 0.02 * torch.randn(N, K, generator=g, device=dev)
            s["w"][0][e], s["w"][1][e] = _mx_rows(dense, "mxfp4")
        s["x"] = list(_mx_rows(_tokens(g, T, K), c["fmt"]))
        if E > 1:
            logits = torch.randn(T, E, generator=g, device=dev)
            logits += c["skew"] * torch.randn(E, generator=g, device=dev)
            ids = logits.topk(k, dim=1).indices.reshape(-1)
            s["perm"] = torch.argsort(ids, stable=True).to(torch.int32)
            load = torch.bincount(ids, minlength=E)
            s["offsets"] = torch.cat([load.new_zeros(1), load.cumsum(0)]).to(torch.int32)
            s["most"] = int(load.max())           # the plan's padded rows per expert
        if own:
            from sparse_fp4_expert_amd import moesq as m
            s["mx_w"] = m.Mx(s["w"][0], s["w"][1], m.ROWS_MXFP4)
            s["mx_x"] = m.Mx(s["x"][0], s["x"][1], _rows_format(m, c["fmt"]))
    return s


# ------------------------------------------------------------------ plain forms

def _f4_codes(q):
    """E2M1 codes of fp32 values, nearest with ties to the even code, saturating."""
    a = q.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
         + (a > 5.0)).to(torch.uint8)
    return c | (((q < 0) & (c > 0)).to(torch.uint8) << 3)


def _f8_codes(q):
    """E4M3 codes of fp32 values, nearest with ties to even, saturating; zero is +0."""
    c = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where((c & 0x7F) == 0, 0, c).to(torch.uint8)


def _mx_rows(x, fmt):
    """Rows [T, K] to MX codes and scale bytes."""
    T, K = x.shape
    b = x.float().view(T, K // 32, 32)
    amax = b.abs().amax(dim=2)
    top = F4_MAX_EXP if fmt == "mxfp4" else F8_MAX_EXP
    e = torch.frexp(amax)[1] - 1 - top                      # floor(log2(amax)) - top
    e = torch.where(amax > 0, e, -127).clamp(-127, 127).to(torch.int32)
    inv = ((127 - e) << 23).view(torch.float32)             # 2^-e
    q = b * inv.unsqueeze(2)
    scale = (e + 127).to(torch.uint8)
    if fmt == "mxfp4":
        c = _f4_codes(q).view(T, K // 2, 2)
        return c[:, :, 0] | (c[:, :, 1] << 4), scale
    return _f8_codes(q).view(T, K), scale


def _pow2(scale):
    """2^(code - 127) in fp32 of E8M0 scale bytes."""
    i = scale.to(torch.int32)
    return torch.where(i > 0, i << 23, 1 << 22).view(torch.float32)


_F4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _f4_values(codes, scale):
    """fp32 values [..., K] of packed E2M1 codes [..., K/2] times [..., K/32] fp32 scales."""
    lut = torch.tensor(_F4, device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], dim=-1)
    v = v.reshape(*scale.shape, 32) * scale.unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _mx_values(codes, scale, fmt):
    if fmt == "mxfp4":
        return _f4_values(codes, _pow2(scale))
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.reshape(*scale.shape, 32) * _pow2(scale).unsqueeze(-1)).reshape(codes.shape)


def _plain_gate(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
    key = l if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        per = key.view(T, G, E // G)
        if c["bias"]:
            best = per.sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        else:
            best = per.amax(dim=2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"ids": ids.reshape(-1).to(torch.int32), "weights": (w * c["scale"]).float().reshape(-1)}


def _nvfp4_values(y):
    """bf16 E2M1 values of NVFP4 rows, their E4M3 block scales and the fp32 scale of each row."""
    T, K = y.shape
    f = y.float()
    amax = f.abs().amax(dim=1)
    g = torch.where(amax > 0, amax / 2688.0, 1.0)
    b = f.view(T, K // 32, 32)
    sc = (b.abs().amax(dim=2) / (6.0 * g)[:, None]).clamp(max=448.0).to(torch.float8_e4m3fn)
    sg = (sc.float() * g[:, None]).unsqueeze(2)
    q = torch.where(sg > 0, b / torch.where(sg > 0, sg, 1.0), 0.0)
    c = _f4_codes(q)
    lut = torch.tensor(_F4, device=y.device, dtype=torch.bfloat16)
    return lut[c.int()], sc, g


def _plain_norm(s):
    c = s["case"]
    x = s["x"]
    out = {}
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(torch.bfloat16)
        out["residual"] = x
    mean = x.double().square().mean(dim=1, keepdim=True)      # long sums, rounded once
    rstd = (1.0 / torch.sqrt(mean + 1e-6)).float()
    y = ((x.float() * rstd) * s["weight"].float()).to(torch.bfloat16)
    if c["y"]:
        out["y"] = y
    if c["rows"] == "mxfp8":
        codes, scale = _mx_rows(y, "mxfp8")
        out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)
    elif c["rows"] == "mxfp4":
        out["values"] = _mx_values(*_mx_rows(y, "mxfp4"), "mxfp4").to(torch.bfloat16)
    elif c["rows"] == "nvfp4":
        v, sc, g = _nvfp4_values(y)
        out["values"], out["scales"], out["row_scale"] = v.view(y.shape), sc, g
    return out


def _plain_quantize(s):
    fmt = s["case"]["fmt"]
    codes, scale = _mx_rows(s["x"], fmt)
    if fmt == "mxfp8":
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scale.view(torch.float8_e8m0fnu)}
    return {"values": _mx_values(codes, scale, fmt).to(torch.bfloat16)}


def _swiglu(y):
    gate, up = y.chunk(2, dim=-1)
    return gate * torch.sigmoid(gate) * up


def _plain_gemm(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    x = _mx_values(*s["x"], c["fmt"])
    w = _mx_values(*s["w"], "mxfp4")
    if E == 1:
        y = x @ w[0].t()
    else:
        rows = s["offsets"][:-1, None].long() + torch.arange(s["most"], device=x.device)
        mine = rows < s["offsets"][1:, None]
        rows = rows.clamp(max=s["perm"].numel() - 1)
        xe = x[s["perm"].long()[rows] // k] * mine.unsqueeze(2)          # [E, most, K]
        ye = torch.bmm(w, xe.transpose(1, 2).contiguous())               # [E, N, most]
        r = torch.arange(s["perm"].numel(), device=x.device)
        e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
        y = ye.transpose(1, 2)[e, r - s["offsets"].long()[e]]
    return (_swiglu(y) if c["swiglu"] else y).to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls

def _rows_format(m, name):
    return {"mxfp4": m.ROWS_MXFP4, "mxfp8": m.ROWS_MXFP8, "nvfp4": m.ROWS_NVFP4}[name]


def _own_rows(m, q, fmt):
    if fmt == "mxfp8":
        return {"codes": q.codes.view(torch.float8_e4m3fn), "scales": q.scales.view(torch.float8_e8m0fnu)}
    return {"values": m.mx_decode(q)}


def _own(s):
    from sparse_fp4_expert_amd import moesq as m
    c = s["case"]
    if c["op"] == "gate":
        ids, w = m.gate_topk(s["logits"], s["gate"], bias=s["bias"])
        return {"ids": ids, "weights": w}
    if c["op"] == "norm":
        fmt = None if c["rows"] == "none" else _rows_format(m, c["rows"])
        y, res, q = m.rmsnorm(s["x"], s["weight"], 1e-6, residual=s["residual"], y=c["y"], rows=fmt)
        out = {}
        if res is not None:
            out["residual"] = res
        if c["y"]:
            out["y"] = y
        if c["rows"] == "nvfp4":
            out["values"] = torch.tensor(_F4, device=q.codes.device, dtype=torch.bfloat16)[
                torch.stack([q.codes & 15, q.codes >> 4], dim=-1).int()].view(c["T"], c["K"])
            out["scales"] = q.scales.view(torch.float8_e4m3fn)
            out["row_scale"] = q.row_scale
        elif fmt is not None:
            out.update(_own_rows(m, q, c["rows"]))
        return out
    if c["op"] == "quantize":
        return _own_rows(m, m.mx_quantize(s["x"], _rows_format(m, c["fmt"])), c["fmt"])
    epi = m.EPI_SWIGLU if c["swiglu"] else m.EPI_NONE
    if c["E"] == 1:
        return m.mx_gemm(s["mx_x"], s["mx_w"], epilogue=epi)
    return m.mx_gemm(s["mx_x"], s["mx_w"], s["offsets"], perm=s["perm"], k=c["k"], epilogue=epi)


_PLAIN = {"gate": _plain_gate, "norm": _plain_norm, "quantize": _plain_quantize, "gemm": _plain_gemm}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "gate":
        bytes_ = c["T"] * c["E"] * (4 if c["dtype"] == "f32" else 2) + 8 * c["T"] * c["k"]
        return {"bytes": bytes_ + (4 * c["E"] if c["bias"] else 0), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "norm":
        per = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0)
        per += {"none": 0, "mxfp8": 33 / 32, "mxfp4": 17 / 32, "nvfp4": 17 / 32}[c["rows"]]
        return {"bytes": c["T"] * c["K"] * per + 2 * c["K"], "flops": 5 * c["T"] * c["K"]}
    if c["op"] == "quantize":
        per = (2 if c["dtype"] == "bf16" else 4) + (33 / 32 if c["fmt"] == "mxfp8" else 2)
        return {"bytes": c["T"] * c["K"] * per, "flops": 2 * c["T"] * c["K"]}
    M = c["T"] * c["k"]
    # experts with rows: all of them, or no more than there are rows
    w = min(c["E"], M) * c["N"] * c["K"] * 17 / 32
    x = c["T"] * c["K"] * (17 / 32 if c["fmt"] == "mxfp4" else 33 / 32)
    y = M * c["N"] * (1 if c["swiglu"] else 2)
    return {"bytes": w + x + y, "flops": 2 * M * c["N"] * c["K"]}


# ------------------------------------------------------------------ 64-bit forms

def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_grid(v, mantissa, low, most):
    """v rounded to `mantissa` fraction bits (exponent at least `low`), ties to even, saturating at `most`."""
    step = _exact_pow2((torch.frexp(v)[1] - 1).clamp(min=low) - mantissa)
    return torch.round(v / step).mul(step).clamp(-most, most)


def _exact_mx(v, fmt):
    """The values and the scales that MX rows of v stand for, in 64 bits."""
    T, K = v.shape
    b = v.view(T, K // 32, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    top = F4_MAX_EXP if fmt == "mxfp4" else F8_MAX_EXP
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - top, -127).clamp(-127, 127)
    scale = _exact_pow2(e)
    q = _exact_grid(b / scale, 1, 0, 6.0) if fmt == "mxfp4" else _exact_grid(b / scale, 3, -6, 448.0)
    return q, scale


def _exact_bf16(v):
    """64-bit values rounded to 8 significant bits, ties to even."""
    return _exact_grid(v, 7, -126, 3.3895313892515355e38)


def _exact_values(codes, scale, fmt):
    """64-bit values from the fields of the codes."""
    if fmt == "mxfp4":
        c = torch.stack([codes % 16, codes // 16], dim=-1).flatten(-2).double()
        sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
        ex, frac = torch.floor(c / 2), c % 2
        v = torch.where(ex == 0, frac * 0.5, (1 + frac * 0.5) * 2.0 ** (ex - 1))
    else:
        c = codes.double()
        sign, c = torch.where(c >= 128, -1.0, 1.0), c % 128
        ex, frac = torch.floor(c / 8), c % 8
        v = torch.where(ex == 0, frac * 2.0 ** -9, (1 + frac / 8) * 2.0 ** (ex - 7))
    return sign * v * (2.0 ** (scale.double() - 127)).repeat_interleave(32, dim=-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gate":
        l = s["logits"].double()
        if c["score"] == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-l))
        else:
            p = torch.exp(l - l.amax(dim=1, keepdim=True))
            p = p / p.sum(dim=1, keepdim=True)
        key = l.clone() if s["bias"] is None else p + s["bias"].double()
        rows, per = torch.arange(c["T"], device=l.device), c["E"] // c["groups"]
        score = []
        for g in range(c["groups"] if c["groups"] > 1 else 0):
            part = key[:, g * per:(g + 1) * per]
            score.append(part.topk(min(2, per), dim=1).values.sum(dim=1) if c["bias"] else part.max(dim=1).values)
        for g in range(len(score)):
            ahead = sum((score[o] > score[g]).int() + ((score[o] == score[g]).int() if o < g else 0)
                        for o in range(len(score)) if o != g)
            key[:, g * per:(g + 1) * per] = torch.where((ahead < c["top_groups"])[:, None],
                                                        key[:, g * per:(g + 1) * per], -math.inf)
        ids = []
        for _ in range(c["k"]):
            best = key.amax(dim=1, keepdim=True)
            ids.append((key == best).int().argmax(dim=1))     # the first of the largest
            key[rows, ids[-1]] = -math.inf
        ids = torch.stack(ids, dim=1)
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        return {"ids": ids.reshape(-1).to(torch.int32), "weights": w.reshape(-1) * c["scale"]}
    if c["op"] == "norm":
        v, out = s["x"].double(), {}
        if s["residual"] is not None:
            v = _exact_bf16(v + s["residual"].double())
            out["residual"] = v
        n = v * (v.pow(2).sum(dim=1, keepdim=True) / c["K"] + 1e-6).rsqrt() * s["weight"].double()
        if c["y"]:
            out["y"] = n
        n = _exact_bf16(n)                # rows are quantised from the bf16 result
        if c["rows"] in ("mxfp8", "mxfp4"):
            q, scale = _exact_mx(n, c["rows"])
            if c["rows"] == "mxfp8":
                out["codes"], out["scales"] = q.reshape(n.shape), scale.squeeze(2)
            else:
                out["values"] = (q * scale).reshape(n.shape)
        elif c["rows"] == "nvfp4":
            # the format takes its decisions on fp32 quotients: each is rounded to fp32 here too
            amax = n.abs().amax(dim=1)
            g = torch.where(amax > 0, (amax / 2688.0).float().double(), 1.0)
            b = n.view(c["T"], -1, 32)
            sc = _exact_grid((b.abs().amax(dim=2) / (6.0 * g).float().double()[:, None]).float().double(),
                             3, -6, 448.0)
            sg = (sc * g[:, None]).float().double().unsqueeze(2)
            q = torch.where(sg > 0, (b / sg.clamp(min=1e-300)).float().double(), 0.0)
            out["values"] = _exact_grid(q, 1, 0, 6.0).view(n.shape)
            out["scales"], out["row_scale"] = sc, g
        return out
    if c["op"] == "quantize":
        q, scale = _exact_mx(s["x"].double(), c["fmt"])
        if c["fmt"] == "mxfp8":
            return {"codes": q.reshape(s["x"].shape), "scales": scale.squeeze(2)}
        return {"values": (q * scale).reshape(s["x"].shape)}
    x = _exact_values(*s["x"], c["fmt"])
    y = torch.empty(c["T"] * c["k"], c["N"], dtype=torch.float64, device=x.device)
    off = [0, c["T"]] if c["E"] == 1 else s["offsets"].tolist()
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        if b > a:
            w = _exact_values(s["w"][0][e], s["w"][1][e], "mxfp4")
            mine = x[a:b] if c["E"] == 1 else x[torch.div(s["perm"][a:b].long(), c["k"], rounding_mode="floor")]
            y[a:b] = mine @ w.t().contiguous()
    if c["swiglu"]:
        h = c["N"] // 2
        y = y[:, :h] / (1.0 + torch.exp(-y[:, :h])) * y[:, h:]
    return y
