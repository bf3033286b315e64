"""The bf16 product, its gradients and the combine's against float64.

Tolerances, per result.  Products of two bf16 are exact in fp32.  A matrix
instruction adds 16 or 32 of them to the sum; with a rounding for every four
(each at most 2^-23 of a partial sum, itself at most S = sum |a b|) a sum over
C positions is off by at most acc = (C/4 + 8) 2^-23 S.  A rounding to bf16 adds
2^-8 of the value.
  SwiGLU h = silu(g) u: |silu'| <= 1.1, and its exponential and reciprocal add
(|g| + 2) 2^-22 of h.
  Its gradient of d: s = sigmoid(g) is off by es = s (|g| + 2) 2^-22; silu'(g) = s (1 + g (1 - s))
is then off by (1 + |g| (1 + 2 s)) es and four roundings of at most 2^-24 (1 + |g|) s, silu(g) by
|g| es; d's own error goes through both."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(rng, *shape, scale=1.0):
    """bf16 values over several binades, some zero."""
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-3, 4, shape[-1]))
    v[rng.random(shape) < 0.02] = 0.0
    return torch.from_numpy(scale * v).to(BF).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def acc(a, b):
    """|a| @ |b| times the error of a sum of that many products."""
    return (a.shape[1] / 4 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(b))


def within(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(got - ref)
    assert got.shape == ref.shape and (err <= tol + 1e-38).all(), (what, float((err / (tol + 1e-38)).max()))


def bf16_tol(ref, extra):
    return 2.0 ** -8 * (np.abs(ref) + extra) + extra


def swiglu_bound(z, az):
    n = z.shape[1] // 2
    g, u, ag, au = z[:, :n], z[:, n:], az[:, :n], az[:, n:]
    h = oracle.silu(g) * u
    return h, bf16_tol(h, (np.abs(g) + 2) * 2.0 ** -22 * np.abs(h) + 1.1 * ag * (np.abs(u) + au)
                       + np.abs(oracle.silu(g)) * au)


def swiglu_grad_bound(d, ad, z):
    n = z.shape[1] // 2
    g, u = z[:, :n], z[:, n:]
    s = 1 / (1 + np.exp(-g))
    es = s * (np.abs(g) + 2) * 2.0 ** -22
    ref = oracle.swiglu_grad(d, z)
    e1 = (1 + np.abs(g) * (1 + 2 * s)) * es + 2.0 ** -22 * (1 + np.abs(g)) * s
    da, db = np.abs(s * (1 + g * (1 - s))), np.abs(g * s)
    extra = np.concatenate([np.abs(u) * (np.abs(d) * e1 + ad * (da + e1)),
                            np.abs(d) * (np.abs(g) * es + 2.0 ** -23 * db) + ad * (db + np.abs(g) * es)], axis=1)
    return ref, bf16_tol(ref, extra)


def plan(rng, counts, k, T=None):
    """(offsets, perm, E): T*k routed rows whose experts have `counts` rows."""
    M = int(sum(counts))
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    return off, torch.from_numpy(rng.permutation(M).astype(np.int32)).cuda(), len(counts)


def check(lib, rng, N, K, T=None, counts=None, k=None, swiglu=False, flat=False):
    """The product and both gradients of one layer."""
    E = 1 if counts is None else len(counts)
    M = T if counts is None else int(sum(counts))
    off = perm = None
    if counts is not None:
        off, perm, _ = plan(rng, counts, k)
    kk = k or 1
    x = rand(rng, M // kk if k else M, K)
    w = rand(rng, E, N, K, scale=0.05)
    if not k:
        perm = None
    epi = (lib.EPI_SWIGLU if swiglu else lib.EPI_NONE) | (lib.OUT_FLAT if flat else 0)
    H = N // 2
    out = torch.full((M, H if swiglu else N), 7.0, dtype=BF, device="cuda")
    if swiglu and not flat:
        y, z = lib.gemm(x, w, off, perm=perm, k=kk, epilogue=epi, save=True)
        assert torch.equal(y, lib.gemm(x, w, off, perm=perm, k=kk, epilogue=epi, out=out))
    else:
        y, z = lib.gemm(x, w, off, perm=perm, k=kk, epilogue=epi, out=out), None
    dy = rand(rng, M, N, scale=0.1)
    dx = lib.gemm_dx(dy, w, off)
    # the rows as the result of a gated block with projections zin (K columns): their gradient
    zin = rand(rng, M, 2 * K) if M * K <= 1 << 20 else None
    dz = None if zin is None else lib.gemm_dx(dy, w, off, z=zin)
    if dz is not None:
        own = zin.clone()
        assert torch.equal(lib.gemm_dx(dy, w, off, z=own, out=own), dz)
    dw = lib.gemm_dw(dy, x, off, E=E, perm=perm, k=kk)
    dw32 = lib.gemm_dw(dy, x, off, E=E, perm=perm, k=kk, dtype=torch.float32)
    held = rand(rng, E, N, K).float()
    sums = lib.gemm_dw(dy, x, off, E=E, perm=perm, k=kk, out=held.clone(), accumulate=True)
    assert torch.equal(dw32.to(BF), dw) and torch.equal(held + dw32, sums)
    offs = [0, M] if counts is None else off.cpu().numpy()
    p = np.arange(M) if perm is None else perm.cpu().numpy()
    for e in range(E):
        r = np.arange(offs[e], offs[e + 1])
        if not len(r):
            assert not dw32[e].any()
            continue
        xe, we, dye = f64(x)[p[r] // kk], f64(w[e]), f64(dy)[r]
        ref, tol = xe @ we.T, acc(xe, we.T)
        got = f64(y)[p[r] if flat else r]
        if swiglu:
            if z is not None:
                within(f64(z)[r], ref, bf16_tol(ref, tol), ("z", e))
            h, tol = swiglu_bound(ref, tol)
            within(got, h, tol, ("h", e))
        else:
            within(got, ref, bf16_tol(ref, tol), ("y", e))
        ref, tol = dye @ we, acc(dye, we)
        within(f64(dx)[r], ref, bf16_tol(ref, tol), ("dx", e))
        if dz is not None:
            within(f64(dz)[r], *swiglu_grad_bound(ref, tol, f64(zin)[r]), ("dz", e))
        ref = dye.T @ xe
        within(f64(dw32[e]), ref, acc(dye.T, xe), ("dw", e))


@pytest.mark.parametrize("T,N,K", [(1, 16, 8), (1, 48, 64), (2, 8, 40), (3, 24, 72), (16, 64, 128), (17, 80, 160),
                                   (31, 256, 288), (33, 96, 512), (64, 128, 480), (65, 144, 1024), (128, 264, 256),
                                   (129, 272, 392), (200, 520, 1000), (257, 64, 2056), (1000, 136, 328),
                                   (16, 1536, 2048), (40, 2048, 1032)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_dense(lib, T, N, K, swiglu):
    if swiglu and N % 16:
        N += 8
    print(f"[gemm dense] T={T} N={N} K={K} swiglu={swiglu}", flush=True)
    check(lib, np.random.default_rng(T + N + K), N, K, T=T, swiglu=swiglu)


@pytest.mark.parametrize("counts,k", [([0, 1, 0, 5], 2), ([16, 17, 15, 33], 1), ([130, 0, 2, 64, 300], 8),
                                      ([1] * 40, 4), ([2, 0] * 35, 7), ([260, 3, 128, 256, 129], 4), ([0, 0, 64], 1),
                                      ([5, 0, 0], 5), ([700, 1, 0, 40, 19], 2)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(lib, counts, k, gather):
    print(f"[gemm grouped] {counts[:6]} k={k} gather={gather}", flush=True)
    rng = np.random.default_rng(len(counts))
    check(lib, rng, 96, 328, counts=counts, k=k if gather else None, swiglu=True)
    check(lib, rng, 136, 192, counts=counts, k=k if gather else None, flat=gather)


# Enough tiles for every tile size and for more of them than the chip runs at a time.
@pytest.mark.parametrize("T,N,K", [(250, 4112, 136), (1000, 4128, 264), (2047, 4096, 320), (2300, 2080, 1096),
                                   (4090, 520, 2304)])
def test_dense_tiles(lib, T, N, K):
    print(f"[gemm tiles] T={T} N={N} K={K}", flush=True)
    check(lib, np.random.default_rng(T + K), N, K, T=T, swiglu=K % 16 == 8)


@pytest.mark.parametrize("E,mean,N,K", [(64, 9, 256, 392), (40, 20, 528, 136), (70, 40, 544, 512), (40, 100, 1056, 264),
                                        (33, 250, 1040, 384), (300, 11, 96, 256), (12, 600, 272, 520)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_tiles(lib, E, mean, N, K, swiglu):
    rng = np.random.default_rng(E)
    counts = rng.poisson(mean * rng.gamma(1.0, 1.0, E))
    counts[0] += -counts.sum() % 2
    print(f"[gemm grouped tiles] E={E} M={counts.sum()} N={N} K={K}", flush=True)
    check(lib, rng, N, K, counts=counts, k=2, swiglu=swiglu)


def test_rows_outside_every_expert_stay(lib):
    """Offsets that cover a part of the rows, and offsets outside [0, M]."""
    rng = np.random.default_rng(1)
    M, N, K, E = 90, 64, 72, 3
    x, w, dy = rand(rng, M, K), rand(rng, E, N, K), rand(rng, M, N)
    x[40:] = float("nan")
    dy[40:] = float("nan")
    for offs in ([3, 10, 10, 40], [-5, 12, 12, 40], [40, 3, 3, 40]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        y = torch.full((M, N), 7.0, dtype=BF, device="cuda")
        lib.gemm(x, w, off, out=y)
        dx = torch.full((M, K), 7.0, dtype=BF, device="cuda")
        lib.gemm_dx(dy, w, off, out=dx)
        dw = lib.gemm_dw(dy, x, off, E=E, dtype=torch.float32)
        seen = torch.zeros(M, dtype=torch.bool)
        for e in range(E):
            lo, hi = max(offs[e], 0), offs[e + 1]
            if hi > lo:
                seen[lo:hi] = True
            xe, de, we = f64(x[lo:max(hi, lo)]), f64(dy[lo:max(hi, lo)]), f64(w[e])
            ref = xe @ we.T
            within(y[lo:max(hi, lo)], ref, bf16_tol(ref, acc(xe, we.T)), "y")
            ref = de @ we
            within(dx[lo:max(hi, lo)], ref, bf16_tol(ref, acc(de, we)), "dx")
            within(dw[e], de.T @ xe, (len(xe) / 4 + 8) * 2.0 ** -23 * (np.abs(de.T) @ np.abs(xe)), "dw")
        assert (y[~seen] == 7).all() and (dx[~seen] == 7).all()


def test_choices_without_an_expert(lib):
    """Rows of a plan that routed a part of the choices; entries of perm outside
    [0, T*k) give zero rows and add nothing to the weights' gradient."""
    rng = np.random.default_rng(2)
    T, k, E, N, K = 30, 4, 6, 96, 136
    ids = rng.integers(-1, E, T * k).astype(np.int32)
    x, w = rand(rng, T, K), rand(rng, E, N, K)
    off, perm, inv = lib.route(torch.from_numpy(ids).cuda(), E, k)
    live = int(off[-1])
    perm[live:] = 1 << 30
    bad = [1, live // 2, live - 1]
    perm[bad] = torch.tensor([-1, T * k, -(1 << 31)], dtype=torch.int32, device="cuda")
    y = torch.full((T * k, N), 7.0, dtype=BF, device="cuda")
    lib.gemm(x, w, off, perm=perm, k=k, out=y)
    dy = rand(rng, T * k, N)
    dy[live:] = float("nan")
    dw = lib.gemm_dw(dy, x, off, E=E, perm=perm, k=k, dtype=torch.float32)
    assert (y[live:] == 7).all() and not y[bad].any()
    p = perm.cpu().numpy()
    for e in range(E):
        r = np.array([i for i in range(int(off[e]), int(off[e + 1])) if i not in bad], dtype=np.int64)
        xe, de, we = f64(x)[p[r] // k], f64(dy)[r], f64(w[e])
        ref = xe @ we.T
        within(f64(y)[r], ref, bf16_tol(ref, acc(xe, we.T)), "y")
        within(dw[e], de.T @ xe, (len(r) / 4 + 8) * 2.0 ** -23 * (np.abs(de.T) @ np.abs(xe)), "dw")


def test_other_rows_nan_stays_there(lib):
    """NaN and infinities in one row, one expert or one column reach nothing else."""
    rng = np.random.default_rng(3)
    counts, N, K = [20, 70, 3, 40], 80, 72
    off, _, E = plan(rng, counts, 1)
    M = sum(counts)
    x, w, dy = rand(rng, M, K), rand(rng, E, N, K), rand(rng, M, N)
    clean = [lib.gemm(x, w, off), lib.gemm_dx(dy, w, off), lib.gemm_dw(dy, x, off, E=E)]
    x2, w2, dy2 = x.clone(), w.clone(), dy.clone()
    w2[2] = float("nan")
    x2[25], dy2[25] = float("inf"), float("nan")
    y, dx, dw = lib.gemm(x2, w2, off), lib.gemm_dx(dy2, w2, off), lib.gemm_dw(dy2, x2, off, E=E)
    rows = [r for r in range(M) if r != 25 and not 90 <= r < 93]
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(dx[rows], clean[1][rows])
    assert torch.equal(dw[[0, 2, 3]], clean[2][[0, 2, 3]])
    assert dw[1].isnan().all() and y[90:93].isnan().all() and not torch.isfinite(y[25].float()).any()
    # NaN of the rows and weights behind the last position of a row
    K2 = 8 * 5
    xs, ws = rand(rng, 64, K2), rand(rng, 32, K2)
    xs[1:] = float("nan")
    ws[1:] = float("nan")
    y = lib.gemm(xs, ws)
    assert torch.isfinite(y[0, 0].float()) and y[1:].isnan().all() and y[:, 1:].isnan().all()


def test_gradients_against_differences(lib):
    """The block's gradients are those of its float64 loss, by central differences."""
    rng = np.random.default_rng(4)
    T, H, K = 12, 24, 40
    x, w, wd = rand(rng, T, K, scale=0.3), rand(rng, 2 * H, K, scale=0.2), rand(rng, K, H, scale=0.2)
    dy = rand(rng, T, K, scale=0.3)
    h, z = lib.gemm(x, w, epilogue=lib.EPI_SWIGLU, save=True)
    dz = lib.gemm_dx(dy, wd, z=z)
    grads = dict(x=f64(lib.gemm_dx(dz, w)), w=f64(lib.gemm_dw(dz, x, dtype=torch.float32)[0]),
                 wd=f64(lib.gemm_dw(dy, h, dtype=torch.float32)[0]))
    at = dict(x=f64(x), w=f64(w), wd=f64(wd))

    def loss(v):
        return (oracle.swiglu(v["x"] @ v["w"].T) @ v["wd"].T * f64(dy)).sum()

    for name, grad in grads.items():
        # what bf16 in z, dz, h and the result may move: a few 2^-8 of the gradient's size
        size = np.abs(grad).max()
        for _ in range(25):
            i = tuple(rng.integers(0, n) for n in grad.shape)
            d = 1e-4
            up, dn = ({n: a.copy() for n, a in at.items()} for _ in range(2))
            up[name][i] += d
            dn[name][i] -= d
            num = (loss(up) - loss(dn)) / (2 * d)
            assert abs(num - grad[i]) <= 4 * 2.0 ** -8 * size, (name, i, num, grad[i])


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (1, 8, 2048), (3, 2, 264), (5, 16, 72), (64, 8, 7168), (300, 4, 520)])
@pytest.mark.parametrize("dropped", [False, True])
def test_combine_backward(lib, T, k, N, dropped):
    """dw: a lane adds N/64 products in fp32 (exact products), six more additions
    across the lanes: (N/64 + 8) 2^-24 of sum |products|."""
    rng = np.random.default_rng(T + N)
    M = T * k
    dout, y = rand(rng, T, N), rand(rng, M, N)
    w = torch.from_numpy(rng.random(M).astype(np.float32)).cuda()
    inv = rng.permutation(M).astype(np.int32)
    if dropped:
        inv[rng.random(M) < 0.3] = -1
        inv[rng.random(M) < 0.1] = M
    t = torch.from_numpy(inv).cuda()
    dy, dw = lib.unpermute_backward(dout, y, t, w, T, k)
    ref, refw = oracle.combine_grad(f64(dout), f64(y), inv, w.cpu().numpy(), k)
    for i, r in enumerate(inv):
        if 0 <= r < M:
            within(dy[r], ref[r], bf16_tol(ref[r], 2.0 ** -24 * np.abs(ref[r])), "dy")
            S = np.abs(f64(dout[i // k])) @ np.abs(f64(y[r]))
            assert abs(float(dw[i]) - refw[i]) <= (N / 64 + 8) * 2.0 ** -24 * S
        else:
            assert float(dw[i]) == 0.0
    named = torch.zeros(M, dtype=torch.bool)
    named[[r for r in inv if 0 <= r < M]] = True
    held = y.clone()                                           # in place of y, other rows stay
    gw = torch.empty(M, device="cuda")
    lib.moesq_unpermute_backward(dout, held, t, w, T, k, N, held, gw)
    assert torch.equal(held[named], dy[named]) and torch.equal(held[~named], y[~named]) and torch.equal(gw, dw)
    assert torch.equal(lib.unpermute_backward(dout, None, t, w, T, k, dw=False)[0][named], dy[named])
    assert torch.equal(lib.unpermute_backward(dout, y, t, None, T, k, dy=False)[1], dw)


class Layer:
    """A whole layer in training: router weights, dispatch, gated experts, down
    projection and combine, forward and back."""

    def __init__(self, lib, T=40, E=8, k=3, K=136, N=176, seed=0):
        rng = np.random.default_rng(seed)
        self.lib, self.T, self.E, self.k = lib, T, E, k
        self.x, self.dout = rand(rng, T, K, scale=0.3), rand(rng, T, K, scale=0.1)
        self.wu, self.wd = rand(rng, E, N, K, scale=0.1), rand(rng, E, K, N // 2, scale=0.1)
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1).astype(np.int32)
        self.ids = torch.from_numpy(ids).cuda()
        self.tw = torch.from_numpy(rng.random(T * k).astype(np.float32)).cuda()
        self.ones = torch.ones(T * k, device="cuda")
        self.main = torch.zeros(E, N, K, device="cuda")

    def run(self, stream=None):
        m, s, T, k, E = self.lib, stream, self.T, self.k, self.E
        off, perm, inv = m.route(self.ids, E, k, stream=s)
        h, z = m.gemm(self.x, self.wu, off, perm=perm, k=k, epilogue=m.EPI_SWIGLU, save=True, stream=s)
        y = m.gemm(h, self.wd, off, stream=s)
        out = m.unpermute(y, inv, self.tw, T, k, stream=s)
        dy, dtw = m.unpermute_backward(self.dout, y, inv, self.tw, T, k, stream=s)
        dz = m.gemm_dx(dy, self.wd, off, z=z, stream=s)
        dwd = m.gemm_dw(dy, h, off, E=E, stream=s)
        dwu = m.gemm_dw(dz, self.x, off, E=E, perm=perm, k=k, stream=s)
        m.gemm_dw(dz, self.x, off, E=E, perm=perm, k=k, out=self.main, accumulate=True, stream=s)
        dx = m.unpermute(m.gemm_dx(dz, self.wu, off, stream=s), inv, self.ones, T, k, stream=s)
        return dict(h=h, z=z, y=y, out=out, dtw=dtw, dwd=dwd, dwu=dwu, dx=dx)


def layer_reference(b):
    """Results and gradients in float64, from autograd on the CPU."""
    x, wu, wd, tw = (t.double().cpu().requires_grad_() for t in (b.x, b.wu, b.wd, b.tw))
    out = [torch.zeros(x.shape[1], dtype=torch.float64) for _ in range(b.T)]
    for i, e in enumerate(b.ids.tolist()):
        z = wu[e] @ x[i // b.k]
        g, u = z.chunk(2)
        out[i // b.k] = out[i // b.k] + tw[i] * (wd[e] @ (g * torch.sigmoid(g) * u))
    out = torch.stack(out)
    (out * b.dout.double().cpu()).sum().backward()
    return dict(out=out.detach(), dx=x.grad, dwu=wu.grad, dwd=wd.grad, dtw=tw.grad)


def test_layer(lib):
    """bf16 in z, h, y, dy, dz and the results: each 2^-8 at most, 2^-9 or less
    on average, so 1 % of the tensor's size holds their sum."""
    b = Layer(lib)
    got, ref = b.run(), layer_reference(b)
    for name, r in ref.items():
        d = np.linalg.norm(f64(got[name]) - r.numpy())
        assert d <= 1e-2 * np.linalg.norm(r.numpy()), (name, d / np.linalg.norm(r.numpy()))
    assert torch.equal(b.main.to(BF), got["dwu"])


def test_layer_graph(lib):
    """Captured and replayed with other inputs; every replay is the eager result,
    also while another graph of the same weights lives."""
    b, other = Layer(lib, seed=1), Layer(lib, seed=2)
    b.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = b.run()
        graphs.append((g, got))
    keep = (b.x.clone(), b.dout.clone(), b.ids.clone())
    for rep in range(4):
        for dst, src in zip((b.x, b.dout, b.ids), (other.x, other.dout, other.ids) if rep % 2 else keep):
            dst.copy_(src)
        want = b.run()
        b.main.zero_()
        torch.cuda.synchronize()
        g, got = graphs[rep // 2]
        g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (rep, name)
        assert torch.equal(b.main.to(BF), want["dwu"])


def test_layer_on_a_side_stream(lib):
    """Calls given a stream are ordered behind its work, results allocated there."""
    b = Layer(lib, seed=3)
    want = b.run()
    x = b.x.clone()
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        b.x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s if isinstance(s, torch.cuda.Stream) else torch.cuda.ExternalStream(s)):
            torch.cuda._sleep(2_000_000)
            b.x.copy_(x)
        got = b.run(stream=s)
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_two_layers_at_once(lib):
    blocks = [Layer(lib, seed=s) for s in (4, 5)]
    want = [b.run() for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [b.run(stream=s) for b, s in zip(blocks, streams)]
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            for name in v:
                assert torch.equal(u[name], v[name]), name


def test_adapters_in_training(lib):
    """Low-rank adapters grouped by request: their gradients by the same products
    (rank 8 rows of weights, then rank 8 positions), against float64."""
    rng = np.random.default_rng(6)
    A, r, N, K, T = 5, 8, 72, 136, 60
    ids = torch.from_numpy(rng.integers(-1, A, T).astype(np.int32)).cuda()
    x, dy = rand(rng, T, K, scale=0.3), rand(rng, T, N, scale=0.1)
    a, b = rand(rng, A, r, K, scale=0.2), rand(rng, A, N, r, scale=0.2)
    off, perm, inv = lib.route(ids, A, 1)
    n = int(off[-1])
    dyr = lib.permute(dy, perm[:n].contiguous(), 1)[:n] if n == T else dy[perm[:n].long()].contiguous()
    xr = x[perm[:n].long()].contiguous()
    v = lib.gemm(xr, a, off)
    db = lib.gemm_dw(dyr, v, off, E=A)
    dv = lib.gemm_dx(dyr, b, off)
    da = lib.gemm_dw(dv, xr, off, E=A)
    for e in range(A):
        rows = np.nonzero(ids.cpu().numpy() == e)[0]
        xe, de, ae, be = f64(x)[rows], f64(dy)[rows], f64(a[e]), f64(b[e])
        for got, ref in ((db[e], de.T @ (xe @ ae.T)), (da[e], (de @ be).T @ xe)):
            assert np.linalg.norm(f64(got) - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("counts, k, N, K", [
    (None, 0, 8, 8), (None, 0, 80, 3000), (None, 0, 136, 264), ([5000, 0, 17], 0, 72, 200), ([0, 9, 4000, 64], 4, 104, 328),
    ([2100, 2148], 3, 16, 1000)])
@pytest.mark.parametrize("dtype, add", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
def test_weight_gradient_in_parts(lib, counts, k, N, K, dtype, add):
    """Few matrices of many rows: with a workspace the rows are summed in parts."""
    rng = np.random.default_rng(N + K)
    M = 4163 if counts is None else sum(counts)
    E, off, perm, kk = 1 if counts is None else len(counts), None, None, max(k, 1)
    if counts is not None:
        M = M // kk * kk
        counts = counts[:-1] + [counts[-1] - (sum(counts) - M)]
        off, p, _ = plan(rng, counts, k)
        perm = p if k else None
    x, dy = rand(rng, M // kk, K), rand(rng, M, N, scale=0.1)
    held = rand(rng, E, N, K).to(dtype)
    size = lib.moesq_gemm_dw_workspace_bytes(M, E, N, K)
    assert size % (E * N * K * 4) == 0 and (size > 0 or E > 1)             # (few rows an expert: one part)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")      # (NaN)
    got, one = held.clone(), held.clone()
    lib.moesq_gemm_dw(dy, x, perm, M // kk if k else 0, kk, off, M, E, N, K, got, add, ws)
    lib.moesq_gemm_dw(dy, x, perm, M // kk if k else 0, kk, off, M, E, N, K, one, add)
    assert torch.equal(lib.gemm_dw(dy, x, off, E=E, perm=perm, k=kk, out=held.clone(), accumulate=add), got)
    offs = [0, M] if counts is None else off.cpu().numpy()
    src = np.arange(M) if perm is None else perm.cpu().numpy() // kk
    for e in range(E):
        r = np.arange(offs[e], offs[e + 1])
        d, xe = f64(dy)[r], f64(x)[src[r]]
        ref, tol = d.T @ xe, acc(d.T, xe)
        if add:
            ref = ref + f64(held[e])
            tol = tol + 2.0 ** -23 * (np.abs(ref) + tol)
        if dtype == torch.bfloat16:
            tol = bf16_tol(ref, tol)
        within(f64(got[e]), ref, tol, ("parts", e))
        within(f64(one[e]), ref, tol, ("one", e))


def test_far_rows(lib):
    """The last rows of buffers over 4 GiB are what a call on them alone gives."""
    g = torch.Generator(device="cuda").manual_seed(3)
    tail, K, N = 37, 2080, 96
    M = (1 << 20) + tail
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-tail:] = torch.randn(tail, K, generator=g, device="cuda").to(BF)
    w = torch.randn(N, K, generator=g, device="cuda").to(BF)
    end = x[-tail:].clone()
    y = lib.gemm(x, w)
    xe, we = f64(end), f64(w)
    ref = xe @ we.T
    within(y[-tail:], ref, bf16_tol(ref, acc(xe, we.T)), "y")
    assert not y[:-tail].any()
    # the same rows as dy [M, K] of weights [K, N]: gradients of rows and of weights
    wt = w.t().contiguous()
    d = lib.gemm_dx(x, wt)
    ref = xe @ we.T
    within(d[-tail:], ref, bf16_tol(ref, acc(xe, we.T)), "dx")
    other = torch.zeros(M, 72, dtype=BF, device="cuda")
    other[-tail:] = torch.randn(tail, 72, generator=g, device="cuda").to(BF)
    dw = lib.gemm_dw(x, other, dtype=torch.float32)[0]
    oe = f64(other[-tail:])
    within(dw, xe.T @ oe, (M / 4 + 8) * 2.0 ** -23 * (np.abs(xe.T) @ np.abs(oe)), "dw")


def test_far_weights_and_results(lib):
    """Experts beyond 2^32 bytes of weights, and their gradients."""
    E, N, K = 40, 8192, 8192                                   # 5 GiB
    w = torch.zeros(E, N, K, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    w[-1] = torch.randn(N, K, generator=g, device="cuda").to(BF)
    x = torch.randn(24, K, generator=g, device="cuda").to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 24
    # (one expert and forty take kernels that add in another order: both are held to
    # the products' own bound)
    xe, we = f64(x), f64(w[-1])
    ref = xe @ we.T
    within(lib.gemm(x, w, off), ref, bf16_tol(ref, acc(xe, we.T)), "y")
    ref = xe @ we
    within(lib.gemm_dx(x, w, off), ref, bf16_tol(ref, acc(xe, we)), "dx")
    dw = lib.gemm_dw(x, x, off, E=E, out=w)
    assert torch.equal(dw[-1], lib.gemm_dw(x, x)[0]) and not dw[:-1].any()
