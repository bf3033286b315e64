"""Measured cases of the bf16 feed-forward product with its gradients, the
combine's gradient and low-rank adapters.

run() is one pass through an operator: in its plain form (elementary torch
operations in 32 bits), or, with `own` set, through the library's entry
points.  Both take what prepare() makes from a case and a seed.

  gated    both projections of a gated feed-forward block, the activation and
           the product, dense or grouped over experts: h = silu(x Wg') * (x Wu');
           with `save` the two projections are written too, for the backward pass
  ffn-grad the backward pass of such a block and the down projection behind
           it: from the gradient of its result, those of its (routed) rows and
           of both weight matrices of each expert
  combine-grad the gradients of the router-weighted combine: of the experts'
           rows and of the weights
  lora     low-rank adapters of many requests beside a shared projection:
           y = base + s_a (x A_a') B_a' with each row's own adapter a or none
"""
import math

import torch

own = False


def listed():
    return [
        # a single token through a dense block of the 30B class
        dict(name="gated-token", op="gated", E=1, T=1, k=1, N=1536, K=2048, save=False, skew=0.0),
        # the 30B-class experts before their compression, on a decode batch
        dict(name="gated-experts-decode", op="gated", E=128, T=16, k=8, N=1536, K=2048, save=False, skew=1.0),
        # the same in training: uneven loads, projections kept for the backward pass
        dict(name="gated-experts-train", op="gated", E=128, T=4096, k=8, N=1536, K=2048, save=True, skew=1.0),
        # a shared expert of the trillion class on a prefill
        dict(name="gated-dense-prefill", op="gated", E=1, T=8192, k=1, N=4096, K=7168, save=False, skew=0.0),
        # a ragged micro-batch of a dense 30B-class block
        dict(name="grad-dense-small", op="ffn-grad", E=1, T=777, k=1, N=1536, K=2048, skew=0.0),
        # a micro-batch of the trillion-class shared expert
        dict(name="grad-dense", op="ffn-grad", E=1, T=4096, k=1, N=4096, K=7168, skew=0.0),
        # the 30B-class experts, uneven loads
        dict(name="grad-experts", op="ffn-grad", E=128, T=2048, k=8, N=1536, K=2048, skew=1.0),
        # one sequence's end on its way back through the combine
        dict(name="combine-grad-small", op="combine-grad", T=16, k=8, N=2048, dropped=0.0),
        # a trillion-class layer's, some choices without an expert
        dict(name="combine-grad", op="combine-grad", T=4096, k=8, N=7168, dropped=0.02),
        # one request's token beside a 30B-class projection
        dict(name="lora-token", op="lora", T=1, A=8, rank=16, slices=1, N=2048, K=2048, swiglu=False, runs=False),
        # a decode batch of many requests beside the shared expert's gate and up projections
        dict(name="lora-decode", op="lora", T=64, A=32, rank=16, slices=2, N=4096, K=7168, swiglu=True, runs=False),
        # prompts of several requests, one behind the other
        dict(name="lora-prefill", op="lora", T=8192, A=8, rank=64, slices=1, N=4096, K=7168, swiglu=False, runs=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["gated", "gated", "ffn-grad", "ffn-grad", "combine-grad", "lora", "lora"])
    if op == "combine-grad":
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 16), N=_log(rng, 64, 7168, 8),
                     dropped=rng.choice([0.0, 0.1]))
            if c["T"] * c["k"] * c["N"] <= 4096 * 8 * 7168:
                return c
    if op == "lora":
        while True:
            slices = rng.choice([1, 1, 2])
            c = dict(op=op, T=_log(rng, 1, 8192), A=_log(rng, 1, 64), rank=_log(rng, 8, 128, 8), slices=slices,
                     N=_log(rng, 64, 4096, 32), K=_log(rng, 64, 7168, 8), swiglu=slices == 2 and rng.random() < 0.5,
                     runs=rng.random() < 0.5)
            if c["T"] * c["A"] * c["rank"] * slices * (c["K"] + c["N"]) <= 8192 * 8 * 64 * (7168 + 4096):
                return c
    while True:
        E = rng.choice([1, _log(rng, 2, 128)])
        c = dict(op=op, E=E, T=_log(rng, 1, 8192), k=rng.randint(1, min(8, E)), N=_log(rng, 64, 4096, 16),
                 K=_log(rng, 64, 7168, 8), skew=0.0 if E == 1 else rng.choice([0.0, 1.0]))
        if op == "gated":
            c["save"] = rng.random() < 0.5
        if c["T"] * c["k"] * c["N"] * c["K"] <= 5e10 and E * c["N"] * c["K"] <= 4e8:
            return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 9973 + 29)


def _normal(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _tokens(g, T, K):
    """Activations with a hundredth of the channels ten times the others."""
    gain = 1.0 + 9.0 * (torch.rand(K, generator=g, device="cuda") < 0.01).float()
    return (torch.randn(T, K, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _plan(s, g, c):
    """The routing plan of random top-k choices: offsets and permutation."""
    logits = torch.randn(c["T"], c["E"], generator=g, device="cuda")
    logits += c["skew"] * torch.randn(c["E"], generator=g, device="cuda")
    ids = logits.topk(c["k"], dim=1).indices.reshape(-1)
    s["perm"] = torch.argsort(ids, stable=True).to(torch.int32)
    load = torch.bincount(ids, minlength=c["E"])
    s["offsets"] = torch.cat([load.new_zeros(1), load.cumsum(0)]).to(torch.int32)
    s["most"] = int(load.max())               # the plan's padded rows per expert


def prepare(case, seed):
    g = _generator(seed)
    dev = "cuda"
    c, s = case, {"case": case}
    if c["op"] in ("gated", "ffn-grad"):
        E, T, k, N, K = c["E"], c["T"], c["k"], c["N"], c["K"]
        s["x"] = _tokens(g, T, K)
        s["w_up"] = _normal(g, E, N, K, scale=0.02)
        if E > 1:
            _plan(s, g, c)
        if c["op"] == "ffn-grad":
            M, H = T * k, N // 2
            # what the forward pass has kept: both projections and the block's result
            s["z"] = _normal(g, M, N, scale=1.2)
            s["h"] = _swiglu(s["z"].float()).to(torch.bfloat16)
            s["w_down"] = _normal(g, E, K, H, scale=0.03)
            s["dy"] = _normal(g, M, K, scale=1e-3)
    elif c["op"] == "combine-grad":
        T, k, N = c["T"], c["k"], c["N"]
        M = T * k
        s["dout"] = _normal(g, T, N, scale=1e-3)
        s["y"] = _normal(g, M, N)
        w = torch.rand(T, k, generator=g, device=dev)
        s["w"] = (w / w.sum(dim=1, keepdim=True)).reshape(-1)
        # routed rows in random order; the choices with the last places have no expert
        s["rows"] = M - int(c["dropped"] * M)
        place = torch.randperm(M, generator=g, device=dev)
        s["inv_perm"] = torch.where(place < s["rows"], place, -1).to(torch.int32)
    else:
        T, A, r, S, N, K = c["T"], c["A"], c["rank"], c["slices"], c["N"], c["K"]
        s["x"] = _tokens(g, T, K)
        s["a"] = _normal(g, A, S * r, K, scale=K ** -0.5)
        s["b"] = _normal(g, A, N, r, scale=0.05)
        s["scale"] = 0.5 + torch.rand(A, generator=g, device=dev)
        s["base"] = _normal(g, T, N)
        if c["runs"]:                          # requests of many tokens, in any order of adapters
            at = torch.rand(T, generator=g, device=dev) < 16.0 / max(T, 16)
            of = torch.randint(-1, A, (T,), generator=g, device=dev)
            first = torch.cummax(torch.where(at, torch.arange(T, device=dev), 0), dim=0).values
            s["ids"] = of[first].to(torch.int32)
        else:                                  # one token a request, an eighth of them without an adapter
            of = torch.randint(0, A, (T,), generator=g, device=dev)
            none = torch.rand(T, generator=g, device=dev) < 0.125
            s["ids"] = torch.where(none & (T > 1), -1, of).to(torch.int32)
        if own:
            from sparse_fp4_expert_amd import moesq as m
            s["lora"] = m.Lora(s["a"], s["b"], s["scale"], slices=S)
    return s


# ------------------------------------------------------------------ plain forms

def _swiglu(y):
    gate, up = y.chunk(2, dim=-1)
    return gate * torch.sigmoid(gate) * up


class _Rows:
    """Routed rows of all experts padded to the longest: [E, most, ...] and back."""

    def __init__(self, s):
        self.grouped = "offsets" in s
        if self.grouped:
            off, n = s["offsets"].long(), s["perm"].numel()
            rows = off[:-1, None] + torch.arange(s["most"], device=off.device)
            self.mine = (rows < off[1:, None]).unsqueeze(2)
            self.rows = rows.clamp(max=n - 1)
            r = torch.arange(n, device=off.device)
            self.e = torch.searchsorted(off[1:].contiguous(), r, right=True)
            self.at = r - off[self.e]

    def pad(self, v):
        v = v.float()
        return v[self.rows] * self.mine if self.grouped else v.unsqueeze(0)

    def routed(self, v):
        return v[self.e, self.at] if self.grouped else v[0]


def _product(a, b):
    """[E, m, c] by [E, c, n] in fp32."""
    return torch.bmm(a.contiguous(), b.contiguous())


def _routed_tokens(s):
    return s["x"] if "perm" not in s else s["x"][torch.div(s["perm"].long(), s["case"]["k"], rounding_mode="floor")]


def _plain_gated(s):
    rows = _Rows(s)
    z = rows.routed(_product(rows.pad(_routed_tokens(s)), s["w_up"].float().transpose(1, 2)))
    out = {"h": _swiglu(z).to(torch.bfloat16)}
    if s["case"]["save"]:
        out["z"] = z.to(torch.bfloat16)
    return out


def _plain_ffn_grad(s):
    rows = _Rows(s)
    dy = rows.pad(s["dy"])
    gate, up = rows.pad(s["z"]).chunk(2, dim=-1)
    sig = torch.sigmoid(gate)
    dh = _product(dy, s["w_down"].float())
    dz = torch.cat([dh * up * (sig * (1.0 + gate * (1.0 - sig))), dh * gate * sig], dim=-1)
    return {"dx": rows.routed(_product(dz, s["w_up"].float())).to(torch.bfloat16),
            "dw_up": _product(dz.transpose(1, 2), rows.pad(_routed_tokens(s))).to(torch.bfloat16),
            "dw_down": _product(dy.transpose(1, 2), rows.pad(s["h"])).to(torch.bfloat16)}


def _plain_combine_grad(s):
    k = s["case"]["k"]
    there = s["inv_perm"] >= 0
    inv = s["inv_perm"].long()[there]
    d = s["dout"].float().repeat_interleave(k, dim=0)[there]
    dy = torch.empty(s["rows"], d.shape[1], device=d.device)
    dy[inv] = d * s["w"][there].unsqueeze(1)
    dw = torch.zeros_like(s["w"])
    dw[there] = (d * s["y"][inv].float()).sum(dim=1)
    return {"dy": dy.to(torch.bfloat16), "dw": dw}


def _plain_lora(s):
    c = s["case"]
    T, A, r, S, N = c["T"], c["A"], c["rank"], c["slices"], c["N"]
    v = s["x"].float() @ s["a"].float().reshape(A * S * r, -1).t()
    # every adapter's, of which a row keeps its own
    mine = (s["ids"].unsqueeze(1) == torch.arange(A, device=v.device)).float() * s["scale"]
    v = v.view(T, A, S, r) * mine[:, :, None, None]
    b = s["b"].float().view(A, S, N // S, r).permute(1, 0, 3, 2).reshape(S, A * r, N // S)
    d = torch.bmm(v.permute(2, 0, 1, 3).reshape(S, T, A * r).contiguous(), b.contiguous())
    y = s["base"].float() + d.permute(1, 0, 2).reshape(T, N)
    return (_swiglu(y) if c["swiglu"] else y).to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from sparse_fp4_expert_amd import moesq as m
    c = s["case"]
    off, perm, k, E = s.get("offsets"), s.get("perm"), c.get("k"), c.get("E")
    if c["op"] == "gated":
        if c["save"]:
            h, z = m.gemm(s["x"], s["w_up"], off, perm=perm, k=k, epilogue=m.EPI_SWIGLU, save=True)
            return {"h": h, "z": z}
        return {"h": m.gemm(s["x"], s["w_up"], off, perm=perm, k=k, epilogue=m.EPI_SWIGLU)}
    if c["op"] == "ffn-grad":
        dz = m.gemm_dx(s["dy"], s["w_down"], off, z=s["z"])
        return {"dx": m.gemm_dx(dz, s["w_up"], off),
                "dw_up": m.gemm_dw(dz, s["x"], off, E=E, perm=perm, k=k),
                "dw_down": m.gemm_dw(s["dy"], s["h"], off, E=E)}
    if c["op"] == "combine-grad":
        dy, dw = m.unpermute_backward(s["dout"], s["y"], s["inv_perm"], s["w"], c["T"], k)
        return {"dy": dy[:s["rows"]], "dw": dw}
    return m.lora(s["x"], s["lora"], s["ids"], base=s["base"], epilogue=m.EPI_SWIGLU if c["swiglu"] else m.EPI_NONE)


_PLAIN = {"gated": _plain_gated, "ffn-grad": _plain_ffn_grad, "combine-grad": _plain_combine_grad,
          "lora": _plain_lora}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "combine-grad":
        n = c["T"] * c["k"] * c["N"]
        return {"bytes": 2 * c["T"] * c["N"] + 4 * n + 12 * c["T"] * c["k"], "flops": 3 * n}
    if c["op"] == "lora":
        T, R, N, K = c["T"], c["rank"], c["N"], c["K"]
        used = min(c["A"], T)
        return {"bytes": 2 * (T * K + used * R * (c["slices"] * K + N) + T * N + T * N // (2 if c["swiglu"] else 1)),
                "flops": 2 * T * R * (c["slices"] * K + N)}
    M, N, K = c["T"] * c["k"], c["N"], c["K"]
    # experts with rows: all of them, or no more than there are rows
    w = min(c["E"], M) * N * K
    if c["op"] == "gated":
        return {"bytes": 2 * (c["T"] * K + w + M * N // 2 + (M * N if c["save"] else 0)), "flops": 2 * M * N * K}
    # rows: dy, z, h and x in, dx out; weights and their gradients
    return {"bytes": 2 * (2 * M * K + M * N * 3 // 2 + c["T"] * K + 3 * w // 2 + 3 * c["E"] * N * K // 2),
            "flops": 6 * M * N * K}


# ------------------------------------------------------------------ 64-bit forms

def _silu64(v):
    return v / (1.0 + torch.exp(-v))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "combine-grad":
        dy = torch.empty(s["rows"], c["N"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            inv = s["inv_perm"][j::c["k"]].long()
            t = torch.nonzero(inv >= 0).squeeze(1)
            d = s["dout"].double()[t]
            dy[inv[t]] = s["w"].double()[t * c["k"] + j, None] * d
            dw[t * c["k"] + j] = torch.einsum("tn,tn->t", d, s["y"][inv[t]].double())
        return {"dy": dy, "dw": dw}
    if c["op"] == "lora":
        n = c["N"] // c["slices"]
        y = s["base"].double()
        for a in range(c["A"]):
            t = torch.nonzero(s["ids"] == a).squeeze(1)
            for i in range(c["slices"] if len(t) else 0):
                down = s["a"][a, i * c["rank"]:(i + 1) * c["rank"]].double()
                up = s["b"][a, i * n:(i + 1) * n].double()
                part = (s["x"][t].double() @ down.t().contiguous()) @ up.t().contiguous()
                y[t, i * n:(i + 1) * n] += s["scale"][a].double() * part
        if c["swiglu"]:
            y = _silu64(y[:, :n]) * y[:, n:]
        return y
    M, N, K, E, k = c["T"] * c["k"], c["N"], c["K"], c["E"], c["k"]
    H = N // 2
    off = [0, M] if E == 1 else s["offsets"].tolist()
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")      # noqa: E731
    z, dx = (new(M, N), None) if c["op"] == "gated" else (None, new(M, K))
    dw = (None, None) if c["op"] == "gated" else (new(E, N, K), new(E, K, H))
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = s["x"][a:b] if E == 1 else s["x"][s["perm"][a:b].long() // k]
        x, w = x.double(), s["w_up"][e].double()
        if z is not None:
            z[a:b] = x @ w.t().contiguous()
            continue
        dy, gate, up = s["dy"][a:b].double(), s["z"][a:b, :H].double(), s["z"][a:b, H:].double()
        dh = dy @ s["w_down"][e].double()
        # silu'(g) = silu(g) + sigmoid(g) (1 - silu(g))
        act, sig = _silu64(gate), 1.0 / (1.0 + torch.exp(-gate))
        dz = torch.cat([dh * up * (act + sig * (1.0 - act)), dh * act], dim=1)
        dx[a:b] = dz @ w
        dw[0][e] = dz.t().contiguous() @ x
        dw[1][e] = dy.t().contiguous() @ s["h"][a:b].double()
    if z is None:
        return {"dx": dx, "dw_up": dw[0], "dw_down": dw[1]}
    out = {"h": _silu64(z[:, :H]) * z[:, H:]}
    if c["save"]:
        out["z"] = z
    return out
