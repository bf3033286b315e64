"""Low-rank adapters against float64.

Tolerance, per result p = base + scale (x a') b': the sums v = x a' are off by
(K/4 + 8) 2^-23 sum |x a| (see the product's tests), enter the second product
within 2^-16 of themselves, and its sum of 2 rank products and the scale add
(rank/2 + 8) 2^-23 of sum |v b|; a rounding to bf16 adds 2^-8 of the result.
SwiGLU as in the product's tests."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(rng, *shape, scale=1.0):
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-2, 3, shape[-1]))
    return torch.from_numpy(scale * v).to(BF).cuda()


class Case:
    def __init__(self, lib, T, A, rank, slices, N, K, seed=0, none=0.2, runs=False):
        rng = np.random.default_rng(seed + T + N + K)
        self.slices, self.N = slices, N
        self.x, self.base = rand(rng, T, K), rand(rng, T, N)
        self.a, self.b = rand(rng, A, slices * rank, K, scale=K ** -0.5), rand(rng, A, N, rank, scale=0.3)
        self.scale = torch.from_numpy(rng.uniform(-2, 2, A).astype(np.float32)).cuda()
        ids = rng.integers(0, A, T)
        if runs:
            ids = ids[np.maximum.accumulate(np.where(rng.random(T) < 0.1, np.arange(T), 0))]
        ids[rng.random(T) < none] = -1
        ids[rng.random(T) < none / 8] = A
        self.ids = torch.from_numpy(ids.astype(np.int32)).cuda()
        self.lora = lib.Lora(self.a, self.b, self.scale, slices=slices)

    def reference(self, base=True):
        """(p, bound before the rounding)."""
        x, a, b, sc, ids = f64(self.x), f64(self.a), f64(self.b), f64(self.scale), self.ids.cpu().numpy()
        K, rank = x.shape[1], b.shape[2]
        p0 = f64(self.base) if base else np.zeros((len(x), self.N))
        p = oracle.lora(x, a, b, sc, ids, p0, self.slices)
        one = oracle.lora(np.abs(x), np.abs(a), np.abs(b), np.abs(sc), ids, np.zeros_like(p0), self.slices)
        off = np.zeros_like(p0)
        for e in np.unique(ids[(ids >= 0) & (ids < len(a))]):
            r = np.nonzero(ids == e)[0]
            v = np.abs(x[r] @ a[e].T)
            off[r] = oracle.lora(v, np.eye(v.shape[1])[None], np.abs(b[e])[None], np.abs(sc[e:e + 1]),
                                 np.zeros(len(r), int), np.zeros((len(r), self.N)), self.slices)
        return p, (K / 4 + 8) * 2.0 ** -23 * one + (2.0 ** -16 + (rank / 2 + 8) * 2.0 ** -23) * off


def check(lib, c):
    p, e = c.reference()
    y = lib.lora(c.x, c.lora, c.ids, base=c.base)
    err = np.abs(f64(y) - p)
    tol = 2.0 ** -8 * (np.abs(p) + e) + e + 2.0 ** -23 * np.abs(p)
    assert (err <= tol).all(), float((err / tol).max())
    none = ~((c.ids >= 0) & (c.ids < len(c.a)))
    assert torch.equal(y[none], c.base[none])
    held = c.base.clone()
    assert lib.lora(c.x, c.lora, c.ids, base=held, out=held) is held and torch.equal(held, y)
    p, e = c.reference(base=False)
    d = lib.lora(c.x, c.lora, c.ids)
    assert (np.abs(f64(d) - p) <= 2.0 ** -8 * (np.abs(p) + e) + e).all() and not d[none].any()
    if c.N % 16 == 0:
        h = c.N // 2
        p, e = c.reference()
        e = e + 2.0 ** -23 * np.abs(p)
        g, u, eg, eu = p[:, :h], p[:, h:], e[:, :h], e[:, h:]
        ref = oracle.silu(g) * u
        extra = (np.abs(g) + 2) * 2.0 ** -22 * np.abs(ref) + 1.1 * eg * (np.abs(u) + eu) + np.abs(oracle.silu(g)) * eu
        got = f64(lib.lora(c.x, c.lora, c.ids, base=c.base, epilogue=lib.EPI_SWIGLU))
        assert (np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + extra) + extra).all()


@pytest.mark.parametrize("T,A,rank,slices,N,K", [
    (1, 1, 8, 1, 8, 8), (1, 4, 16, 1, 2048, 2048), (1, 3, 8, 2, 48, 72), (2, 2, 24, 1, 40, 264), (7, 9, 16, 2, 96, 520),
    (15, 3, 40, 1, 264, 136), (16, 32, 16, 1, 256, 1024), (17, 2, 32, 2, 272, 392), (33, 40, 64, 1, 136, 200),
    (64, 32, 16, 2, 512, 1000), (65, 5, 256, 1, 128, 328), (64, 7, 256, 4, 320, 96), (130, 64, 8, 4, 64, 64),
    (300, 3, 128, 2, 288, 1032), (1000, 4, 48, 1, 80, 456)])
@pytest.mark.parametrize("runs", [False, True])
def test_lora(lib, T, A, rank, slices, N, K, runs):
    print(f"[lora] T={T} A={A} rank={rank} slices={slices} N={N} K={K} runs={runs}", flush=True)
    check(lib, Case(lib, T, A, rank, slices, N, K, runs=runs))


@pytest.mark.parametrize("T,A,rank,slices,N,K", [(2100, 6, 16, 2, 160, 328), (2049, 3, 64, 1, 528, 264),
                                                 (4500, 2, 8, 1, 72, 136), (3000, 40, 136, 1, 64, 104)])
def test_many_rows(lib, T, A, rank, slices, N, K):
    print(f"[lora rows] T={T} A={A} rank={rank} slices={slices} N={N} K={K}", flush=True)
    check(lib, Case(lib, T, A, rank, slices, N, K, none=0.02, runs=True))
    check(lib, Case(lib, T, A, rank, slices, N, K, none=0.02))


def test_no_row_has_an_adapter(lib):
    for ids in (-1, 5, 1 << 30, -(1 << 31)):
        c = Case(lib, 50, 5, 16, 1, 64, 72)
        c.a.fill_(float("nan"))
        c.ids.fill_(ids)
        assert torch.equal(lib.lora(c.x, c.lora, c.ids, base=c.base), c.base)


def test_a_row_is_its_own(lib):
    """Rows do not depend on the other rows' tokens and adapters, NaN included."""
    for T in (40, 700):
        c = Case(lib, T, 6, 16, 2, 96, 136, none=0.0)
        want = lib.lora(c.x, c.lora, c.ids, base=c.base)
        keep = c.ids == 2
        keep[3] = True
        c.ids[3] = 4
        want = lib.lora(c.x, c.lora, c.ids, base=c.base)
        c.x[~keep] = float("inf")
        c.base[~keep] = float("nan")
        for e in (0, 1, 3, 5):
            c.a[e], c.b[e], c.scale[e] = float("nan"), float("inf"), float("nan")
        got = lib.lora(c.x, c.lora, c.ids, base=c.base)
        live = keep & ((c.ids == 2) | (c.ids == 4))
        assert int(live.sum()) > 3 and torch.equal(got[live], want[live])
        # and a changed neighbour's adapter changes nothing
        ids = c.ids.clone()
        ids[~keep] = -1
        assert torch.equal(lib.lora(c.x, c.lora, ids, base=c.base)[live], want[live])


@pytest.mark.parametrize("T, A, rank, runs", [(19, 3, 8, False), (40, 5, 24, False), (70, 4, 72, False), (1500, 3, 40, True),
                                              (1300, 4, 64, False)])
def test_other_adapters_infinite(lib, T, A, rank, runs):
    """Rows of one tile with adapters of which one is not finite: the others' stay as they are."""
    c = Case(lib, T, A, rank, 1, 72, 328, seed=3, runs=runs)
    y = lib.lora(c.x, c.lora, c.ids, base=c.base)
    for e, v in ((1, float("inf")), (2, float("nan"))):
        keep = c.ids != e
        assert keep.any() and not keep.all()
        was = c.a[e].clone(), c.b[e].clone()
        for a, b in ((True, False), (False, True)):
            c.a[e], c.b[e] = was
            if a:
                c.a[e] = v
            if b:
                c.b[e] = v
            got = lib.lora(c.x, c.lora, c.ids, base=c.base)
            assert torch.equal(got[keep], y[keep]) and not got[~keep].isfinite().all()
        c.a[e], c.b[e] = was


def test_beside_projections(lib):
    """The shared expert of a serving step: gate and up with adapters of their
    own, SwiGLU behind them, the down projection with its adapters; MX and bf16
    projections, against float64 of the same weights."""
    rng = np.random.default_rng(5)
    T, K, H, A, r = 48, 256, 160, 6, 16
    x = rand(rng, T, K)
    w1, w2 = rand(rng, 2 * H, K, scale=0.05), rand(rng, K, H, scale=0.05)
    l1 = lib.Lora(rand(rng, A, 2 * r, K, scale=0.05), rand(rng, A, 2 * H, r, scale=0.2),
                  torch.full((A,), 0.5, device="cuda"), slices=2)
    l2 = lib.Lora(rand(rng, A, r, H, scale=0.05), rand(rng, A, K, r, scale=0.2), torch.full((A,), 2.0, device="cuda"))
    ids = torch.from_numpy(rng.integers(-1, A, T).astype(np.int32)).cuda()
    xq, wq = lib.mx_quantize(x, lib.ROWS_MXFP8), lib.mx_quantize(w1)

    def step(mx):
        p = lib.mx_gemm(xq, wq) if mx else lib.gemm(x, w1)
        h = lib.lora(x, l1, ids, base=p, epilogue=lib.EPI_SWIGLU)
        y = lib.gemm(h, w2)
        return lib.lora(h, l2, ids, base=y, out=y)

    for mx in (False, True):
        first = f64(lib.mx_decode(xq)) @ f64(lib.mx_decode(wq)).T if mx else f64(x) @ f64(w1).T
        h = oracle.swiglu(oracle.lora(f64(x), f64(l1.a), f64(l1.b), f64(l1.scale), ids.cpu().numpy(), first, 2))
        ref = oracle.lora(h, f64(l2.a), f64(l2.b), f64(l2.scale), ids.cpu().numpy(), h @ f64(w2).T)
        got = step(mx)
        # three roundings to bf16 on the way, and the projection's own
        assert np.linalg.norm(f64(got) - ref) <= 1e-2 * np.linalg.norm(ref)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = step(mx)
        keep = ids.clone()
        for rep in range(3):
            ids.copy_(keep.roll(rep))
            want = step(mx)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), rep
        ids.copy_(keep)


def test_streams(lib):
    """Two calls at once on two streams, given as an object and as a handle."""
    cs = [Case(lib, T, 4, 16, 1, 264, 520, seed=s) for s, T in enumerate((30, 300))]
    want = [lib.lora(c.x, c.lora, c.ids, base=c.base) for c in cs]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [lib.lora(c.x, c.lora, c.ids, base=c.base, stream=t) for c, t in zip(cs, (s[0], s[1].cuda_stream))]
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_far_rows_and_adapters(lib):
    """Rows and adapters beyond 2^32 bytes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, N = (1 << 20) + 19, 2080, 64
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    x[-19:] = torch.randn(19, K, generator=g, device="cuda").to(BF)
    a, b = torch.randn(3, 16, K, generator=g, device="cuda").to(BF), torch.randn(3, N, 16, generator=g, device="cuda").to(BF)
    ad = lib.Lora(a, b, torch.ones(3, device="cuda"))
    ids = (torch.arange(T, device="cuda") // 1000 % 3).to(torch.int32)
    y = lib.lora(x, ad, ids)
    v = f64(x[-19:])
    ref = oracle.lora(v, f64(a), f64(b), np.ones(3), ids[-19:].cpu().numpy(), np.zeros((19, N)))
    assert np.linalg.norm(f64(y[-19:]) - ref) <= 2.0 ** -8 * np.linalg.norm(ref) and not y[:-19].any()
    del x, y
    A, R, K = 700, 256, 16384                                  # 5.9 GB of a
    a = torch.zeros(A, R, K, dtype=BF, device="cuda")
    a[-1] = torch.randn(R, K, generator=g, device="cuda").to(BF)
    b = torch.zeros(A, 64, R, dtype=BF, device="cuda")
    b[-1] = torch.randn(64, R, generator=g, device="cuda").to(BF)
    x = torch.randn(5, K, generator=g, device="cuda").to(BF)
    one = torch.ones(A, device="cuda")
    ids = torch.tensor([0, A - 1, 3, A - 1, A], dtype=torch.int32, device="cuda")
    y = lib.lora(x, lib.Lora(a, b, one), ids)
    want = lib.lora(x, lib.Lora(a[-1:].clone(), b[-1:].clone(), one[:1]), (ids == A - 1).int() - 1)
    assert torch.equal(y, want) and y[1].any() and not y[[0, 2, 4]].any()


def test_sums_past_the_largest_bf16(lib):
    """A sum between the largest bf16 and the largest fp32 number, of which no bf16 is
    the nearest finite one, and infinite and NaN sums: a row of the second product
    shows them as they are."""
    def up(*e):
        return sum(2.0 ** i for i in e)

    x = torch.zeros(4, 8, dtype=BF)
    x[:, :3] = torch.tensor([2.0 ** 64, 2.0 ** 64, 2.0 ** 64])
    x[1] = -x[1]
    x[2, 3], x[3, 3] = float("inf"), float("nan")
    a = torch.zeros(1, 8, 8, dtype=BF)
    a[0, 0, :3] = torch.tensor([255 * 2.0 ** 56, 2.0 ** 55, 2.0 ** 54])
    a[0, :, 3] = 1                                                 # (every rank is infinite, none 0 * inf)
    b = torch.zeros(1, 8, 8, dtype=BF)
    b[0, :, :] = torch.tensor([2.0 ** -100, -(2.0 ** -120), 1.0, 2.0 ** -126, 2.0 ** -110, 2.0 ** -112, -1.0, 2.0 ** -90])[:, None]
    v = 255 * 2.0 ** 120 + up(119, 118)                            # past the tie between the largest bf16 and infinity
    assert torch.tensor(v).float().isfinite() and torch.tensor(v).to(BF).isinf()
    lora = lib.Lora(a.cuda(), b.cuda(), torch.tensor([2.0 ** -10]).cuda())
    y = f64(lib.lora(x.cuda(), lora, torch.zeros(4, dtype=torch.int32).cuda()))
    p = np.outer([v, -v], f64(b)[0, :, 0]) * 2.0 ** -10
    assert (np.abs(y[:2] - p) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(p)).all()
    assert np.array_equal(y[2], np.sign(f64(b)[0, :, 0]) * np.inf) and np.isnan(y[3]).all()


def test_more_rows_than_one_launch_takes(lib):
    """2^25 + 5 rows of four slices: more than 2^30 threads of the second product.  Small
    integers, so that every sum and result is exact."""
    T, K, rank, slices, N = (1 << 25) + 5, 8, 8, 4, 32
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randint(-1, 2, (T, K), dtype=torch.int8, device="cuda", generator=g).to(BF)
    ids = torch.randint(-1, 2, (T,), dtype=torch.int32, device="cuda", generator=g)
    a = torch.randint(-1, 2, (2, slices * rank, K), device="cuda", generator=g).to(BF)
    b = torch.randint(-1, 2, (2, N, rank), device="cuda", generator=g).to(BF)
    lora = lib.Lora(a, b, torch.tensor([1.0, 2.0]).cuda(), slices=slices)
    y = lib.lora(x, lora, ids)
    for lo in (0, (1 << 23) - 40, (1 << 24) - 100, 3 << 23, T - 77):
        r = slice(lo, min(lo + 200, T))
        want = oracle.lora(f64(x[r]), f64(a), f64(b), np.array([1.0, 2.0]), ids[r].cpu().numpy(),
                           np.zeros((x[r].shape[0], N)), slices)
        assert np.abs(want).max() <= 256 and np.array_equal(f64(y[r]), want)
