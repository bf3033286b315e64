"""MX quantization and decode (bit for bit against the oracle) and the MX
GEMM against the float64 product of the decoded operands.

Tolerance of the GEMM, per result: one rounding to bf16 (2^-8 of the value);
the fp32 accumulation, one aligned addition per 32-element block and K/128
dependent ones, each losing at most 2^-23 of a partial sum, itself at most
S = sum |x w|: (K/32 + 8) 2^-23 S; and with E4M3 elements the matrix unit's
alignment of eight products to the largest of them, whose bits from 2^-13 on
are dropped: 7 * 2^-13 S at most.  SwiGLU h = silu(g) u: |silu'| <= 1.1, and
silu_f32's exponential and reciprocal add (|g| + 2) 2^-22 of h."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

FMT = {"mxfp4": 1, "mxfp8": 2}


def rows_of(rng, rows, K):
    """bf16 values over several binades, with outliers, zeros and a zero block."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 6, (rows, K // 32)).repeat(32, axis=1))
    x[rng.random((rows, K)) < 0.05] = 0.0
    if rows > 2:
        x[1, :32] = 0.0
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 96), (3, 64), (7, 160), (64, 2048), (257, 7168), (5, 8224)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize(lib, fmt, rows, K, dtype):
    rng = np.random.default_rng(rows + K)
    x = rows_of(rng, rows, K)
    if dtype == torch.float32:
        x = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32)) * x.float()
    q = lib.mx_quantize(x.cuda(), FMT[fmt])
    c, s = oracle.mx_quantize(x.double().numpy(), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    assert np.array_equal(q.codes.cpu().numpy(), c)
    v = lib.mx_decode(q)
    assert v.dtype == torch.bfloat16 and tuple(v.shape) == (rows, K)
    assert np.array_equal(v.double().cpu().numpy(), oracle.mx_decode(c, s, fmt))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantize_every_tie_and_saturation(lib, fmt):
    """Every midpoint of the element grid, its fp32 neighbours, and values up
    to the top of the block's binade, at scales from the smallest up."""
    grid = np.arange(0, 129) / 16.0 if fmt == "mxfp4" else np.unique(np.concatenate(
        [np.abs(oracle.E4M3_VALUES[:127]), (oracle.E4M3_VALUES[:126] + oracle.E4M3_VALUES[1:127]) / 2,
         np.arange(440, 512, 1.0)]))
    v = np.unique(np.concatenate([grid, np.nextafter(grid.astype(np.float32), np.float32(-1)),
                                  np.nextafter(grid.astype(np.float32), np.float32(1e9))]).astype(np.float32))
    top = 7.9 if fmt == "mxfp4" else 511.0
    v = v[v <= top]
    v = np.concatenate([v, -v])
    v = np.concatenate([v, np.zeros(-len(v) % 31, np.float32)]).reshape(-1, 31)
    lead = np.full((len(v), 1), 4.0 if fmt == "mxfp4" else 256.0, np.float32)
    for e in (-125, -20, 0, 7, 100):
        x = np.concatenate([lead, v], axis=1) * np.float32(2.0) ** np.float32(e)
        q = lib.mx_quantize(torch.from_numpy(np.ascontiguousarray(x)).cuda(), FMT[fmt])
        c, s = oracle.mx_quantize(x, fmt)
        assert np.array_equal(q.scales.cpu().numpy(), s), e
        assert np.array_equal(q.codes.cpu().numpy(), c), e


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantize_extremes(lib, fmt):
    """Zero, denormal, largest finite, infinite and NaN blocks side by side."""
    f = np.finfo(np.float32)
    x = np.zeros((9, 64), np.float32)
    x[1, 5] = f.smallest_subnormal
    x[2, 5], x[2, 6] = f.tiny, -f.tiny / 2
    x[3, 5], x[3, 6] = f.max, -f.max / 3
    x[4, 5] = np.inf
    x[5, 37] = np.nan
    x[6, 0] = -np.inf
    x[7, 5] = 2.0 ** -125
    x[8, 31], x[8, 32] = -1.0, 3e-39
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(dtype)
        q = lib.mx_quantize(t.cuda(), FMT[fmt])
        c, s = oracle.mx_quantize(t.double().numpy(), fmt)
        assert np.array_equal(q.scales.cpu().numpy(), s) and np.array_equal(q.codes.cpu().numpy(), c)
        want = oracle.bf16_round(np.nan_to_num(oracle.mx_decode(c, s, fmt)))
        got = lib.mx_decode(q).double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.repeat(s == 255, 32, axis=1))
        assert np.array_equal(np.nan_to_num(got), want)


def test_decode_every_code(lib):
    """All codes under all scales whose values bf16 holds."""
    s = np.arange(16, 240, dtype=np.uint8)[:, None]
    c4 = np.tile((np.arange(16, dtype=np.uint8) * 16 + np.arange(16)[::-1].astype(np.uint8)), (len(s), 1))
    q = lib.Mx(torch.from_numpy(c4).cuda(), torch.from_numpy(s).cuda(), FMT["mxfp4"])
    assert np.array_equal(lib.mx_decode(q).double().cpu().numpy(), oracle.mx_decode(c4, s, "mxfp4"))
    c8 = np.tile(np.arange(256, dtype=np.uint8), (len(s), 1))
    c8[:, [127, 255]] = 0                                     # NaN codes
    q = lib.Mx(torch.from_numpy(c8).cuda(), torch.from_numpy(np.repeat(s, 8, axis=1)).cuda(), FMT["mxfp8"])
    want = oracle.bf16_round(oracle.mx_decode(c8, np.repeat(s, 8, axis=1), "mxfp8"))
    assert np.array_equal(lib.mx_decode(q).double().cpu().numpy(), want)


def gemm_bound(xv, wv, fmt, swiglu):
    """(reference, bound) of every result of rows xv with the matrix wv."""
    K = xv.shape[1]
    ref = xv @ wv.T
    S = np.abs(xv) @ np.abs(wv).T
    acc = ((K / 32 + 8) * 2.0 ** -23 + (7 * 2.0 ** -13 if fmt == "mxfp8" else 0.0)) * S
    if not swiglu:
        return ref, 2.0 ** -8 * np.abs(ref) + acc
    n = ref.shape[1] // 2
    g, u, ag, au = ref[:, :n], ref[:, n:], acc[:, :n], acc[:, n:]
    sg = oracle.silu(g)
    h = sg * u
    return h, ((2.0 ** -8 + (np.abs(g) + 2) * 2.0 ** -22) * np.abs(h) + 1.1 * ag * (np.abs(u) + au)
               + np.abs(sg) * au)


def check_gemm(lib, rng, E, N, K, counts, fmt, swiglu=False, k=None, T=None, flat=False, ids=None):
    """Grouped product (or dense, counts None) against the oracle."""
    W = torch.from_numpy(0.02 * rng.standard_normal((E, N, K)).astype(np.float32))
    w = lib.mx_quantize(W.cuda(), FMT["mxfp4"])
    wv = oracle.mx_decode(w.codes.cpu().numpy(), w.scales.cpu().numpy(), "mxfp4")
    epi = lib.EPI_SWIGLU if swiglu else lib.EPI_NONE
    if k is not None:
        x = rows_of(rng, T, K)
        q = lib.mx_quantize(x.cuda(), FMT[fmt])
        off, perm, _ = lib.route(torch.from_numpy(ids.astype(np.int32)).cuda(), E, k)
        y = lib.mx_gemm(q, w, off, perm=perm, k=k, epilogue=epi | (lib.OUT_FLAT if flat else 0))
        off, perm = off.cpu().numpy(), perm.cpu().numpy()
    else:
        M = T if counts is None else int(sum(counts))
        x = rows_of(rng, M, K)
        q = lib.mx_quantize(x.cuda(), FMT[fmt])
        if counts is None:
            y, off = lib.mx_gemm(q, w, epilogue=epi), np.array([0, M])
        else:
            off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
            y = lib.mx_gemm(q, w, torch.from_numpy(off).cuda(), epilogue=epi)
        perm = np.arange(M)
        k = 1
    xv = oracle.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy(), fmt)
    y = y.double().cpu().numpy()
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        if not len(r):
            continue
        ref, tol = gemm_bound(xv[perm[r] // k], wv[e], fmt, swiglu)
        got = y[perm[r] if flat else r]
        err = np.abs(got - ref)
        assert (err <= tol).all(), (e, len(r), float((err / np.maximum(tol, 1e-300)).max()))
    return y


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,N,K", [(1, 16, 32), (1, 32, 64), (2, 48, 96), (16, 64, 128), (17, 80, 160),
                                   (31, 256, 288), (33, 96, 512), (64, 128, 480), (65, 144, 1024),
                                   (128, 256, 256), (129, 272, 384), (200, 512, 2048), (257, 64, 7168)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_dense(lib, fmt, T, N, K, swiglu):
    if swiglu and N % 32:
        N += 16
    print(f"[mx dense] {fmt} T={T} N={N} K={K} swiglu={swiglu}", flush=True)
    check_gemm(lib, np.random.default_rng(T + N + K), 1, N, K, None, fmt, swiglu, T=T)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts", [[0, 1, 0, 5], [16, 17, 15, 33], [130, 0, 1, 64, 300], [0, 0, 0],
                                    [1] * 40, [2, 0] * 35, [260, 3, 128, 256, 127]])
def test_grouped(lib, fmt, counts):
    print(f"[mx grouped] {fmt} {counts[:6]}", flush=True)
    check_gemm(lib, np.random.default_rng(len(counts)), len(counts), 96, 320, counts, fmt,
               swiglu=len(counts) % 2 == 0)
    check_gemm(lib, np.random.default_rng(len(counts)), len(counts), 64, 512, counts, fmt,
               swiglu=len(counts) % 2 == 1)


# Enough tiles to reach every tile size: with 256 CUs, 128 x 64 from 128 tiles
# on, 128 x 128 (FP4) and 256 x 128 (FP8) or 256 x 256 from 256 of their own.
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,N", [(250, 4112), (1000, 4128), (2047, 4096), (4090, 4128)])
@pytest.mark.parametrize("K", [32, 128, 160, 224, 256, 288, 384, 512, 736, 1152])
def test_dense_tiles(lib, fmt, T, N, K):
    swiglu = N % 32 == 0 and K % 256 == 0
    print(f"[mx tiles] {fmt} T={T} N={N} K={K} swiglu={swiglu}", flush=True)
    check_gemm(lib, np.random.default_rng(T + K), 1, N, K, None, fmt, swiglu, T=T)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("E,mean,N,K", [(64, 9, 256, 384), (40, 20, 528, 128), (70, 40, 544, 512), (40, 100, 1056, 256),
                                        (33, 250, 2080, 384), (300, 11, 96, 256),
                                        (50, 90, 800, 96), (35, 210, 2048, 352)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_tiles(lib, fmt, E, mean, N, K, swiglu):
    """Uneven loads about a mean: experts without rows, with one, and with
    several tiles."""
    if swiglu and N % 32:
        N += 16
    rng = np.random.default_rng(E + mean)
    counts = rng.poisson(mean, E) * rng.integers(0, 3, E)
    counts[:3] = 0, 1, 3 * mean
    counts[-1] += max(0, E * mean - counts.sum())       # the mean at least
    print(f"[mx grouped tiles] {fmt} E={E} mean={mean} N={N} K={K} swiglu={swiglu}", flush=True)
    check_gemm(lib, rng, E, N, K, [int(c) for c in counts], fmt, swiglu)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("E,T,k,N,K", [(64, 400, 2, 256, 256), (40, 1300, 3, 1056, 384), (32, 2100, 4, 2112, 512)])
@pytest.mark.parametrize("flat", [False, True])
def test_gather_tiles(lib, fmt, E, T, k, N, K, flat):
    rng = np.random.default_rng(E + T)
    skew = rng.standard_normal(E)
    ids = np.argsort(-(rng.standard_normal((T, E)) + skew), axis=1)[:, :k].reshape(-1)
    print(f"[mx gather tiles] {fmt} E={E} T={T} k={k} flat={flat}", flush=True)
    check_gemm(lib, rng, E, N, K, None, fmt, swiglu=flat, k=k, T=T, flat=flat, ids=ids)


def test_tiles_leave_other_rows(lib):
    """Rows behind the last expert and rows of bad permutation entries, in the
    tiled kernels."""
    rng = np.random.default_rng(11)
    E, T, k, N, K = 64, 700, 2, 512, 256
    ids = rng.integers(0, E, T * k).astype(np.int32)
    ids[1300:] = -1
    w = lib.mx_quantize(torch.randn(E, N, K, device="cuda"))
    for f in FMT.values():
        q = lib.mx_quantize(rows_of(rng, T, K).cuda(), f)
        off, perm, _ = lib.route(torch.from_numpy(ids).cuda(), E, k)
        perm[1300:] = -1
        bad = perm.clone()
        bad[7], bad[900] = T * k, -3
        y = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
        z = y.clone()
        lib.mx_gemm(q, w, off, perm=perm, k=k, out=y)
        lib.mx_gemm(q, w, off, perm=bad, k=k, out=z)
        assert (y[1300:] == 7).all() and (z[1300:] == 7).all() and (z[[7, 900]] == 0).all()
        y[[7, 900]] = 0
        assert torch.equal(y, z)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_unaligned_scales(lib, fmt):
    """Scales that start on any byte give the same results."""
    for T, N, K in ((16, 256, 512), (2048, 4096, 512)):
        x = lib.mx_quantize(torch.randn(T, K, device="cuda").to(torch.bfloat16), FMT[fmt])
        w = lib.mx_quantize(torch.randn(N, K, device="cuda"))
        want = lib.mx_gemm(x, w)

        def moved(q, by):
            s = torch.empty(q.scales.numel() + by, dtype=torch.uint8, device="cuda")
            s = s[by:].view(q.scales.shape).copy_(q.scales)
            return lib.Mx(q.codes, s, q.format)
        for by in (1, 2, 4, 8):
            got = lib.mx_gemm(moved(x, by), moved(w, by)).double()
            assert (got - want.double()).norm() <= 2.0 ** -8 * want.double().norm()
            if by % 4 == 0:
                assert torch.equal(got, want.double())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("E,T,k,N,K", [(8, 1, 2, 64, 256), (8, 64, 2, 128, 256), (128, 16, 8, 160, 256),
                                       (5, 333, 3, 96, 416), (3, 700, 2, 288, 640)])
@pytest.mark.parametrize("flat", [False, True])
def test_gather(lib, fmt, E, T, k, N, K, flat):
    rng = np.random.default_rng(E + T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    print(f"[mx gather] {fmt} E={E} T={T} k={k} flat={flat}", flush=True)
    check_gemm(lib, rng, E, N, K, None, fmt, swiglu=flat, k=k, T=T, flat=flat, ids=ids)


def test_unrouted_ids_and_untouched_rows(lib):
    """Ids of -1 are in no expert's range: their rows of y stay as they were,
    in routed and in flat order; a permutation entry out of range gives a
    zero row."""
    rng = np.random.default_rng(9)
    E, T, k, N, K = 4, 40, 2, 64, 128
    ids = rng.integers(0, E, T * k).astype(np.int32)
    ids[60:] = -1
    w = lib.mx_quantize(torch.randn(E, N, K, device="cuda"))
    q = lib.mx_quantize(rows_of(rng, T, K).cuda())
    off, perm, inv = lib.route(torch.from_numpy(ids).cuda(), E, k)
    perm[60:] = -1                              # rows behind the last expert
    y = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.mx_gemm(q, w, off, perm=perm, k=k, out=y)
    assert (y[60:] == 7).all() and (y[:60] != 7).any(dim=1).all()
    y2 = torch.full_like(y, 7.0)
    lib.mx_gemm(q, w, off, perm=perm, k=k, epilogue=lib.OUT_FLAT, out=y2)
    assert (y2[60:] == 7).all()
    assert torch.equal(y2[perm[:60].long()], y[:60])
    bad = perm.clone()
    bad[3], bad[10] = T * k, -5
    y3 = torch.full_like(y, 7.0)
    lib.mx_gemm(q, w, off, perm=bad, k=k, out=y3)
    keep = torch.ones(60, dtype=torch.bool, device="cuda")
    keep[[3, 10]] = False
    assert (y3[[3, 10]] == 0).all() and torch.equal(y3[:60][keep], y[:60][keep])


def test_bad_offsets_stay_in_bounds(lib):
    """Offsets outside [0, M] are clamped; rows that they leave out stay."""
    E, M, N, K = 3, 50, 32, 64
    w = lib.mx_quantize(torch.randn(E, N, K, device="cuda"))
    q = lib.mx_quantize(torch.randn(M, K, device="cuda").to(torch.bfloat16))
    good = lib.mx_gemm(q, w, torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda"))
    got = lib.mx_gemm(q, w, torch.tensor([-9, 20, 20, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, good)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.mx_gemm(q, w, torch.tensor([30, 20, 10, 0], dtype=torch.int32, device="cuda"), out=y)
    assert (y == 7).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_nan_scale_reaches_its_rows_only(lib, fmt):
    x = torch.randn(40, 256, device="cuda").to(torch.bfloat16)
    w = lib.mx_quantize(torch.randn(96, 256, device="cuda"))
    good = lib.mx_gemm(lib.mx_quantize(x, FMT[fmt]), w)
    x[7, 100] = float("inf")
    x[39, 0] = float("nan")
    y = lib.mx_gemm(lib.mx_quantize(x, FMT[fmt]), w)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[7, 39]] = True
    assert y[bad].isnan().all() and torch.equal(y[~bad], good[~bad])


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,N", [(9, 64), (40, 64), (300, 4096), (1100, 4096), (2050, 4096)])
@pytest.mark.parametrize("K", [32, 96, 160, 352])
def test_what_lies_behind_a_row(lib, fmt, T, N, K):
    """Where K ends inside a stage the kernels read on into the next rows:
    NaN scales and codes there do not reach a result, of tokens or weights."""
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    w = 0.02 * torch.randn(N, K, device="cuda")
    good = lib.mx_gemm(lib.mx_quantize(x, FMT[fmt]), lib.mx_quantize(w))
    assert good.isfinite().all()
    x[1::2], w[1::2] = float("nan"), float("inf")
    xq, wq = lib.mx_quantize(x, FMT[fmt]), lib.mx_quantize(w)
    xq.codes[1::2], wq.codes[1::2] = 0x7f, 0x77
    y = lib.mx_gemm(xq, wq)
    assert torch.equal(y[::2, ::2], good[::2, ::2])
    assert y[1::2].isnan().all() and y[:, 1::2].isnan().all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [16, 1024])
def test_far_weights(lib, fmt, T):
    """Expert matrices beyond 2^31 bytes of codes: the last expert's result is
    the one of the same matrix alone."""
    E, N, K = 300, 2048, 7168
    w = lib.Mx.empty((E, N), K, FMT["mxfp4"])
    one = lib.mx_quantize(0.02 * torch.randn(N, K, device="cuda"))
    w.codes[E - 1], w.scales[E - 1] = one.codes, one.scales
    x = lib.mx_quantize(torch.randn(T, K, device="cuda").to(torch.bfloat16), FMT[fmt])
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = T
    y = lib.mx_gemm(x, w, off)
    one_off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    a = lib.mx_gemm(x, one, one_off).double()
    assert (y.double() - a).norm() <= 2.0 ** -8 * a.norm()


def test_empty(lib):
    w = lib.mx_quantize(torch.randn(2, 32, 64, device="cuda"))
    q = lib.mx_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert tuple(lib.mx_gemm(q, w, off).shape) == (0, 32)
    assert tuple(lib.mx_decode(q).shape) == (0, 64)


@pytest.mark.parametrize("T", [40, 2048])
def test_more_tiles_than_a_launch_has_threads_for(lib, T):
    """Few rows an expert and very many weight rows: the token tiles there may
    be times the weights' workgroups pass the 2^32 threads of a launch (2048
    rows).  All rows are the last expert's; sums of one block are exact."""
    E, N, K = 1024, (1 << 21) - 32, 32
    w = lib.Mx.empty((E, N), K, FMT["mxfp4"])
    one = lib.mx_quantize(0.02 * torch.randn(N, K, device="cuda"))
    w.codes[E - 1], w.scales[E - 1] = one.codes, one.scales
    x = lib.mx_quantize(torch.randn(T, K, device="cuda").to(torch.bfloat16))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = T
    y = lib.mx_gemm(x, w, off)
    alone = lib.mx_gemm(x, one)
    assert torch.equal(y, alone)
    off[E - 1] = T // 2                      # the rows before: another expert's
    w.codes[E - 2], w.scales[E - 2] = one.codes, one.scales
    assert torch.equal(lib.mx_gemm(x, w, off), alone)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [3000, 13000, 60000])
def test_far_weights_tiled(lib, fmt, T):
    """Expert matrices beyond 2^31 bytes of codes in the tiled kernel (more than
    8 rows an expert on average: tiles of 64, 128 and up to 256 rows): the last
    expert's result is the one of the same matrix alone."""
    E, N, K = 300, 2048, 7168
    w = lib.Mx.empty((E, N), K, FMT["mxfp4"])
    one = lib.mx_quantize(0.02 * torch.randn(N, K, device="cuda"))
    w.codes[E - 1], w.scales[E - 1] = one.codes, one.scales
    x = lib.mx_quantize(torch.randn(T, K, device="cuda").to(torch.bfloat16), FMT[fmt])
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = T
    y = lib.mx_gemm(x, w, off)
    a = lib.mx_gemm(x, one, torch.tensor([0, T], dtype=torch.int32, device="cuda")).double()
    assert (y.double() - a).norm() <= 2.0 ** -8 * a.norm()
    # against the formula too: the first rows and the last
    r = torch.cat([torch.arange(5), torch.arange(T - 5, T)]).cuda()
    xv = oracle.mx_decode(x.codes[r].cpu().numpy(), x.scales[r].cpu().numpy(), fmt)
    ref, tol = gemm_bound(xv, oracle.mx_decode(one.codes.cpu().numpy(), one.scales.cpu().numpy(), "mxfp4"), fmt, False)
    assert (np.abs(y[r].double().cpu().numpy() - ref) <= tol).all()
