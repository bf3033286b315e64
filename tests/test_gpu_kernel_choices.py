"""Every kernel of the bf16 product, its gradients and the adapters against float64, on
the calls of kernel_choices.py.

Tolerances are those of the product's tests: a sum over C positions is off by at most
(C/4 + 8) 2^-23 sum |a b|, a rounding to bf16 adds 2^-8 of the value, SwiGLU and
its gradient as there.  Inputs lie between NaN and results between values that have
to stay, so that a read or write beside them shows."""
from __future__ import annotations

import zlib

import pytest
import torch

import test_gpu_lora
from kernel_choices import CHOICES

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PAD = 8192


class Buffer:
    """A tensor in the middle of a longer one of `beside`."""

    def __init__(self, shape, dtype, beside):
        n = 1
        for s in shape:
            n *= s
        self.whole = torch.full((n + 2 * PAD,), beside, dtype=dtype, device="cuda")
        self.t = self.whole[PAD:PAD + n].view(shape)
        self.beside = beside

    def intact(self):
        return bool((self.whole[:PAD] == self.beside).all() and (self.whole[-PAD:] == self.beside).all())


def rand(g, *shape, scale=1.0):
    """bf16 values over several binades, some zero, between NaN."""
    b = Buffer(shape, BF, float("nan"))
    v = torch.randn(*shape, generator=g, device="cuda") * torch.exp2(
        torch.randint(-3, 4, (shape[-1],), generator=g, device="cuda").float())
    v[torch.rand(*shape, generator=g, device="cuda") < 0.02] = 0.0
    b.t.copy_(scale * v)
    return b.t


def result(*shape, dtype=BF):
    return Buffer(shape, dtype, 7.0)


def acc(a, b):
    return (a.shape[1] / 4 + 8) * 2.0 ** -23 * (a.abs() @ b.abs())


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape and bool((err <= tol + 1e-38).all()), (what, float((err / (tol + 1e-38)).max()))


def bf16_tol(ref, extra):
    return 2.0 ** -8 * (ref.abs() + extra) + extra


def swiglu_bound(z, az):
    g, u = z.chunk(2, dim=1)
    ag, au = az.chunk(2, dim=1)
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    return h, bf16_tol(h, (g.abs() + 2) * 2.0 ** -22 * h.abs() + 1.1 * ag * (u.abs() + au) + silu.abs() * au)


def swiglu_grad_bound(d, ad, z):
    g, u = z.chunk(2, dim=1)
    s = 1 / (1 + torch.exp(-g))
    es = s * (g.abs() + 2) * 2.0 ** -22
    ref = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], dim=1)
    e1 = (1 + g.abs() * (1 + 2 * s)) * es + 2.0 ** -22 * (1 + g.abs()) * s
    da, db = (s * (1 + g * (1 - s))).abs(), (g * s).abs()
    extra = torch.cat([u.abs() * (d.abs() * e1 + ad * (da + e1)),
                       d.abs() * (g.abs() * es + 2.0 ** -23 * db) + ad * (db + g.abs() * es)], dim=1)
    return ref, bf16_tol(ref, extra)


def uneven(g, M, E):
    """Offsets of E uneven experts of M rows in all, some empty."""
    load = torch.rand(E, generator=g, device="cuda") ** 2 * (torch.rand(E, generator=g, device="cuda") < 0.9)
    load[E // 2] += 0.1
    ids = torch.multinomial(load, M, replacement=True, generator=g)
    return torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0)]).to(torch.int32)


def experts(off, M):
    offs = [0, M] if off is None else off.tolist()
    return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(offs, offs[1:])) if b > a]


def plans(g, grouped, M, E):
    """(offsets, perm, k) of the ungathered call and, grouped, of a gathered one."""
    if not grouped:
        return [(None, None, 1)]
    off = uneven(g, M, E)
    k = next((k for k in (7, 5, 3) if M % k == 0), 1)
    return [(off, None, 1), (off, torch.randperm(M, generator=g, device="cuda").to(torch.int32), k)]


def check_gemm(lib, g, grouped, M, E, N, K, swiglu):
    for off, perm, k in plans(g, grouped, M, E):
        x, w = rand(g, M // k, K), rand(g, E, N, K, scale=0.05)
        y, z = result(M, N // 2 if swiglu else N), result(M, N) if swiglu else None
        flat = perm is not None and not swiglu
        lib.moesq_gemm(x, perm, M // k if perm is not None else 0, k, off, M, w, E, N, K,
                       (lib.EPI_SWIGLU if swiglu else lib.EPI_NONE) | (lib.OUT_FLAT if flat else 0), y.t, z.t if z else None)
        assert y.intact() and (z is None or z.intact())
        if swiglu and perm is not None:                        # the same in flat order, without z
            f = result(M, N // 2)
            lib.moesq_gemm(x, perm, M // k, k, off, M, w, E, N, K, lib.EPI_SWIGLU | lib.OUT_FLAT, f.t)
            assert f.intact() and torch.equal(f.t[perm.long()], y.t)
        for e, r in experts(off, M):
            src = r if perm is None else perm[r].long() // k
            xe, we = x[src].double(), w[e].double().t().contiguous()
            ref, tol = xe @ we, acc(xe, we)
            got = y.t[perm[r].long()] if flat else y.t[r]
            if swiglu:
                within(z.t[r], ref, bf16_tol(ref, tol), ("z", e))
                within(got, *swiglu_bound(ref, tol), ("h", e))
            else:
                within(got, ref, bf16_tol(ref, tol), ("y", e))


def check_dx(lib, g, grouped, M, E, N, K, with_z):
    off = uneven(g, M, E) if grouped else None
    dy, w = rand(g, M, N, scale=0.1), rand(g, E, N, K)
    z = rand(g, M, 2 * K) if with_z else None
    dx = result(M, 2 * K if with_z else K)
    lib.moesq_gemm_dx(dy, off, M, w, E, N, K, z, dx.t)
    assert dx.intact()
    for e, r in experts(off, M):
        de, we = dy[r].double(), w[e].double()
        ref, tol = de @ we, acc(de, we)
        if with_z:
            within(dx.t[r], *swiglu_grad_bound(ref, tol, z[r].double()), ("dz", e))
        else:
            within(dx.t[r], ref, bf16_tol(ref, tol), ("dx", e))
    if with_z:
        own = z.clone()
        lib.moesq_gemm_dx(dy, off, M, w, E, N, K, own, own)
        assert torch.equal(own, dx.t)


def check_dw(lib, g, gather, grouped, M, E, N, K, ws):
    off, perm, k = plans(g, grouped, M, E)[-1 if gather else 0]
    x, dy = rand(g, M // k, K), rand(g, M, N, scale=0.1)
    held = rand(g, E, N, K).float()
    size = lib.moesq_gemm_dw_workspace_bytes(M, E, N, K) if ws else 0
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    out = {"bf16": result(E, N, K), "fp32": result(E, N, K, dtype=torch.float32), "sum": result(E, N, K, dtype=torch.float32)}
    out["sum"].t.copy_(held)
    for name, o in out.items():
        lib.moesq_gemm_dw(dy, x, perm, M // k if gather else 0, k, off, M, E, N, K, o.t, name == "sum", ws)
        assert o.intact(), name
    full = out["fp32"].t
    assert torch.equal(out["bf16"].t, full.to(BF)) and torch.equal(out["sum"].t, held + full)
    some = dict(experts(off, M))
    for e in range(E):
        if e not in some:
            assert not full[e].any()
            continue
        r = some[e]
        src = r if perm is None else perm[r].long() // k
        de, xe = dy[r].double().t().contiguous(), x[src].double()
        within(full[e], de @ xe, acc(de, xe), ("dw", e))


@pytest.mark.parametrize("call", [call for call, _ in CHOICES if not call.startswith("combine")])
def test_against_float64(lib, call):
    print(f"[kernel choices] {call}", flush=True)
    op, *v = call.split()
    v = [int(n) for n in v]
    g = torch.Generator("cuda").manual_seed(zlib.crc32(call.encode()))
    if op == "gemm":
        check_gemm(lib, g, *v[1:])
    elif op == "dx":
        check_dx(lib, g, *v)
    elif op == "dw":
        check_dw(lib, g, *v[:6], v[7])
    else:
        T, A, rank, slices, N, K, swiglu = v
        for runs in (False, True):
            test_gpu_lora.check(lib, test_gpu_lora.Case(lib, T, A, rank, slices, N, K, runs=runs))


def test_no_rows(lib):
    """Gradients of weights without rows are zeros, or what was there."""
    empty = torch.empty(0, 24, dtype=BF, device="cuda"), torch.empty(0, 40, dtype=BF, device="cuda")
    for E, off in ((1, None), (3, torch.zeros(4, dtype=torch.int32, device="cuda"))):
        out = torch.full((E, 24, 40), 7.0, device="cuda")
        lib.gemm_dw(*empty, off, E=E, out=out, accumulate=True)
        assert (out == 7).all()
        lib.gemm_dw(*empty, off, E=E, out=out)
        assert not out.any()
        assert not lib.gemm_dw(*empty, off, E=E).any()
        assert lib.gemm(empty[1], torch.ones(E, 24, 40, dtype=BF, device="cuda"), off).shape == (0, 24)


def test_more_matrices_than_one_launch_takes(lib):
    """Weights' gradients of more than 2^30 threads (36 GB of results) go out in several launches."""
    E, N, K, M = 986, 32, 555216, 17
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF)
    dy = torch.randint(-2, 3, (M, N), generator=g, device="cuda").to(BF)
    rows = {0: (0, 3), 500: (3, 4), 940: (4, 10), 985: (10, 17)}       # small integers: every sum is exact
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for e, (_, b) in rows.items():
        off[e + 1:] = b
    out = torch.full((E, N, K), 7.0, dtype=BF, device="cuda")
    lib.moesq_gemm_dw(dy, x, None, 0, 1, off, M, E, N, K, out)
    for e in range(E):
        if e in rows:
            r = slice(*rows[e])
            assert torch.equal(out[e].float(), dy[r].float().t().contiguous() @ x[r].float()), e
        else:
            assert not out[e].any(), e
