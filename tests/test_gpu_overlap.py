"""Buffers that touch without sharing a byte, and those that may be the same."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _beside(*shapes):
    """bf16 tensors one behind the other in one buffer."""
    sizes = [a * b for a, b in shapes]
    whole = torch.randn(sum(sizes), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF)
    return [t.view(s) for t, s in zip(whole.split(sizes), shapes)]


def test_neighbours(lib):
    """Results right behind and right before what they are made from."""
    M, N, K = 40, 48, 72
    y, x, w, z, h, dx, dy, dz = _beside((M, N), (M, K), (N, K), (M, N), (M, N // 2), (M, K), (M, N), (M, 2 * K))
    want = lib.gemm(x, w)
    assert torch.equal(lib.gemm(x, w, out=y), want)
    a, b = lib.gemm(x, w, epilogue=lib.EPI_SWIGLU, save=True)
    lib.moesq_gemm(x, None, 0, 1, None, M, w, 1, N, K, lib.EPI_SWIGLU, h, z)
    assert torch.equal(h, a) and torch.equal(z, b)
    want = lib.gemm_dx(dy, w)
    assert torch.equal(lib.gemm_dx(dy, w, out=dx), want)
    want = lib.gemm_dx(dy, w, z=dz)
    assert torch.equal(lib.gemm_dx(dy, w, z=dz, out=dz), want)
    want = lib.gemm_dw(dy, x)
    assert torch.equal(lib.gemm_dw(dy, x, out=w)[None], want)


def test_adapters_on_a_residual(lib):
    """x + its adapter, into x: x, base and y are one buffer."""
    T, N, A, r = 50, 136, 3, 16
    g = torch.Generator("cuda").manual_seed(2)
    rand = lambda *s: (0.1 * torch.randn(*s, generator=g, device="cuda")).to(BF)       # noqa: E731
    x, ad = rand(T, N), lib.Lora(rand(A, r, N), rand(A, N, r), torch.ones(A, device="cuda"))
    ids = torch.randint(-1, A, (T,), generator=g, device="cuda").to(torch.int32)
    want = lib.lora(x.clone(), ad, ids, base=x)
    assert torch.equal(lib.lora(x, ad, ids, base=x, out=x), want)


def test_shared_buffers_are_refused(lib):
    x, w = torch.ones(8, 16, dtype=BF, device="cuda"), torch.ones(16, 16, dtype=BF, device="cuda")
    for call in (lambda: lib.gemm(x, w, out=x), lambda: lib.gemm_dx(x, w, out=x), lambda: lib.gemm_dw(w, w, out=w),
                 lambda: lib.gemm(x, w, out=w[:8])):
        with pytest.raises(lib.MoesqError, match="overlap"):
            call()
    assert (x == 1).all() and (w == 1).all()
