"""The bf16 product and its gradients, the combine's gradient and the adapters
without a GPU: the oracle's gradients against differences and closed forms,
and the refusals of the entry points and of the binding, all before any HIP call."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def m():
    from sparse_fp4_expert_amd import moesq
    return moesq


# ------------------------------------------------------------------ oracle pins

def test_swiglu_grad_is_the_difference_quotient():
    rng = np.random.default_rng(0)
    z, d = rng.standard_normal((5, 12)) * 3, rng.standard_normal((5, 6))
    got = oracle.swiglu_grad(d, z)
    for i in range(5):
        for j in range(12):
            up, dn = z.copy(), z.copy()
            up[i, j] += 1e-6
            dn[i, j] -= 1e-6
            num = ((oracle.swiglu(up) - oracle.swiglu(dn)) * d).sum() / 2e-6
            assert abs(num - got[i, j]) <= 1e-7 * (1 + abs(num))


def test_swiglu_grad_by_hand():
    """g = 0: silu = 0, its derivative 1/2."""
    z = np.array([[0.0, 3.0]])
    assert np.array_equal(oracle.swiglu_grad([[2.0]], z), [[3.0, 0.0]])


def test_combine_grad_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    T, k, N = 4, 3, 5
    y, w, d = rng.standard_normal((T * k, N)), rng.random(T * k), rng.standard_normal((T, N))
    inv = rng.permutation(T * k)
    inv[[1, 7]] = -1

    def loss(y, w):
        return sum(w[i] * (y[r] @ d[i // k]) for i, r in enumerate(inv) if r >= 0)

    dy, dw = oracle.combine_grad(d, y, inv, w, k)
    assert np.isnan(dy).any(axis=1).sum() == 2 and dw[1] == dw[7] == 0
    for i, r in enumerate(inv):
        e = np.zeros(T * k)
        e[i] = 1e-6
        assert abs((loss(y, w + e) - loss(y, w - e)) / 2e-6 - dw[i]) < 1e-8
        if r >= 0:
            e = np.zeros((T * k, N))
            e[r, 2] = 1e-6
            assert abs((loss(y + e, w) - loss(y - e, w)) / 2e-6 - dy[r, 2]) < 1e-8


def test_lora_by_hand():
    """One adapter of rank 1 in each of two slices."""
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0], [0.0, 1.0]]])
    b = np.array([[[1.0], [2.0], [3.0], [4.0]]])
    y = oracle.lora(x, a, b, np.array([10.0]), [0, -1, 0], np.ones((3, 4)), slices=2)
    assert np.array_equal(y, [[11, 21, 61, 81], [1, 1, 1, 1], [51, 101, 181, 241]])


# ------------------------------------------------------------------ refusals

def test_gemm_rejects(m):
    def call(x=0x10, perm=None, T=0, k=1, off=0x10, M=4, w=0x10, E=8, N=64, K=64, epi=0, y=0x10, z=None):
        return m._gemm(x, perm, T, k, off, M, w, E, N, K, epi, y, z, None)

    assert call(epi=2) == m.ERR_ARG and call(epi=m.OUT_FLAT) == m.ERR_ARG
    assert call(z=0x10) == m.ERR_ARG                                    # z without SwiGLU
    assert call(z=0x10, epi=m.EPI_SWIGLU | m.OUT_FLAT, perm=0x10, T=4) == m.ERR_ARG
    assert call(E=0) == m.ERR_SHAPE and call(E=m.MAX_EXPERTS + 1) == m.ERR_SHAPE
    assert call(N=12) == m.ERR_SHAPE and call(N=0) == m.ERR_SHAPE and call(N=-8) == m.ERR_SHAPE
    assert call(K=12) == m.ERR_SHAPE and call(K=0) == m.ERR_SHAPE and call(K=(1 << 20) + 8) == m.ERR_SHAPE
    assert call(N=1 << 16, K=1 << 15) == m.ERR_SHAPE                    # an expert of 4 GiB
    assert call(N=72, epi=m.EPI_SWIGLU) == m.ERR_SHAPE
    assert call(M=-1) == m.ERR_SHAPE and call(M=(1 << 30) + 1) == m.ERR_SHAPE
    assert call(off=None) == m.ERR_NULL                                 # experts without offsets
    assert call(perm=0x10, T=2, k=1) == m.ERR_SHAPE and call(perm=0x10, T=4, k=0) == m.ERR_SHAPE
    assert call(perm=0x10, T=4, off=None, E=1) == m.ERR_NULL
    assert call(perm=0x10, T=1 << 21, M=1 << 21, K=1024) == m.ERR_SHAPE  # gathered tokens of 4 GiB
    for name in ("x", "w", "y"):
        assert call(**{name: None}) == m.ERR_NULL and call(**{name: 0x18}) == m.ERR_ARG
    assert call(epi=m.EPI_SWIGLU, z=0x18) == m.ERR_ARG
    assert call(M=0, x=None, w=None, y=None) == m.OK


def test_gemm_dx_rejects(m):
    def call(dy=0x10, off=0x10, M=4, w=0x10, E=8, N=64, K=64, z=None, dx=0x10):
        return m._gemm_dx(dy, off, M, w, E, N, K, z, dx, None)

    assert call(E=0) == m.ERR_SHAPE and call(N=4) == m.ERR_SHAPE and call(K=4) == m.ERR_SHAPE
    assert call(M=-1) == m.ERR_SHAPE and call(off=None) == m.ERR_NULL
    assert call(dy=None) == m.ERR_NULL and call(w=None) == m.ERR_NULL and call(dx=None) == m.ERR_NULL
    assert call(dy=0x18) == m.ERR_ARG and call(z=0x18) == m.ERR_ARG and call(dx=0x12) == m.ERR_ARG
    assert call(M=0, dy=None, w=None, dx=None) == m.OK


def test_gemm_dw_rejects(m):
    def call(dy=0x10, x=0x10, perm=None, T=0, k=1, off=0x10, M=4, E=8, N=64, K=64, dtype=1, add=0, dw=0x10):
        return m._gemm_dw(dy, x, perm, T, k, off, M, E, N, K, dtype, add, dw, None, 0, None)

    assert call(dtype=2) == m.ERR_ARG and call(dtype=-1) == m.ERR_ARG
    assert call(add=2) == m.ERR_ARG and call(add=1) == m.ERR_ARG          # bf16 is not added to
    assert call(E=0) == m.ERR_SHAPE and call(N=4) == m.ERR_SHAPE and call(K=4) == m.ERR_SHAPE
    assert call(M=-1) == m.ERR_SHAPE and call(off=None) == m.ERR_NULL
    assert call(perm=0x10, T=2) == m.ERR_SHAPE and call(perm=0x10, T=4, off=None, E=1) == m.ERR_NULL
    assert call(dy=None) == m.ERR_NULL and call(x=None) == m.ERR_NULL and call(dw=None) == m.ERR_NULL
    assert call(M=0, dw=None) == m.ERR_NULL                               # zeros are still to be written
    assert call(dy=0x18) == m.ERR_ARG and call(x=0x18) == m.ERR_ARG and call(dw=0x18) == m.ERR_ARG


def test_unpermute_backward_rejects(m):
    def call(dout=0x10, y=0x20, inv=0x10, w=0x10, T=4, k=2, N=16, dy=0x30, dw=0x10):
        return m._unpermute_bw(dout, y, inv, w, T, k, N, dy, dw, None)

    assert call(T=-1) == m.ERR_SHAPE and call(k=0) == m.ERR_SHAPE and call(N=12) == m.ERR_SHAPE
    assert call(N=0) == m.ERR_SHAPE and call(T=1 << 30, k=2) == m.ERR_SHAPE
    assert call(dy=None, dw=None) == m.ERR_NULL and call(dout=None) == m.ERR_NULL and call(inv=None) == m.ERR_NULL
    assert call(w=None) == m.ERR_NULL and call(y=None) == m.ERR_NULL
    assert call(dout=0x18) == m.ERR_ARG and call(y=0x18) == m.ERR_ARG and call(dy=0x18) == m.ERR_ARG
    assert call(dy=0x10) == m.ERR_ARG                                     # over dout
    assert call(T=0, dout=None, y=None, inv=None, w=None, dy=None, dw=None) == m.OK


def test_lora_rejects(m):
    good = dict(a=0x10, b=0x10, scale=0x10, adapters=4, rank=16, slices=1, N=64, K=64)

    def call(x=0x10, ids=0x10, T=4, d=None, base=0x20, epi=0, y=0x30, ws=0x10, n=1 << 30):
        desc = None if d is False else ctypes.byref(m.LoraDesc(*{**good, **(d or {})}.values()))
        assert d is False or (m._lora_ws(T, desc) > 0) == (desc is not None and m._lora(
            None, None, T, desc, None, 0, None, None, 0, None) in (m.ERR_NULL, m.OK) and T > 0)
        return m._lora(x, ids, T, desc, base, epi, y, ws, n, None)

    assert call(d=False) == m.ERR_NULL and m._lora_ws(4, None) == 0
    for bad in (dict(adapters=0), dict(rank=0), dict(rank=12), dict(rank=264), dict(slices=0), dict(slices=5),
                dict(K=0), dict(K=12), dict(K=(1 << 20) + 8), dict(N=0), dict(N=12), dict(N=72, slices=2),
                dict(N=(1 << 20) + 8)):
        assert call(d=bad) == m.ERR_SHAPE, bad
    assert call(T=-1) == m.ERR_SHAPE and call(T=(1 << 26) + 1) == m.ERR_SHAPE
    assert call(epi=2) == m.ERR_ARG and call(epi=m.OUT_FLAT) == m.ERR_ARG
    assert call(epi=1, d=dict(N=72)) == m.ERR_SHAPE and call(epi=1, d=dict(N=96, slices=3)) == m.ERR_SHAPE
    assert call(T=1 << 25, d=dict(rank=256, slices=2)) == m.ERR_SHAPE     # 2^34 sums
    assert call(x=None) == m.ERR_NULL and call(ids=None) == m.ERR_NULL and call(y=None) == m.ERR_NULL
    for name in ("a", "b", "scale"):
        assert call(d={name: None}) == m.ERR_NULL
    assert call(x=0x18) == m.ERR_ARG and call(base=0x28) == m.ERR_ARG and call(y=0x38) == m.ERR_ARG
    assert call(d=dict(a=0x18)) == m.ERR_ARG and call(d=dict(b=0x18)) == m.ERR_ARG and call(ws=0x18) == m.ERR_ARG
    assert call(base=0x30, epi=1) == m.ERR_ARG                            # SwiGLU over its base
    assert call(ws=None) == m.ERR_WORKSPACE and call(n=1) == m.ERR_WORKSPACE
    assert call(T=0, x=None, ids=None, base=None, y=None, ws=None, n=0) == m.OK


def test_binding_rejects_mismatched_sizes(m):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)                       # noqa: E731
    ad = m.Lora(z(3, 16, 24), z(3, 40, 8), z(3, dt=f32), slices=2)
    cases = [
        lambda: m.gemm(z(4, 16), z(8, 24)), lambda: m.gemm(z(4, 16), z(16)), lambda: m.gemm(z(16), z(8, 16)),
        lambda: m.gemm(z(4, 16), z(2, 8, 16), z(2, dt=i32)),
        lambda: m.gemm(z(4, 16), z(2, 8, 16), z(3, dt=i32), perm=z(7, dt=i32), k=2),
        lambda: m.gemm(z(4, 16), z(8, 16), out=z(4, 7)),
        lambda: m.gemm(z(4, 16), z(16, 16), epilogue=m.EPI_SWIGLU, out=z(4, 16)),
        lambda: m.moesq_gemm(z(4, 16), None, 0, 1, None, 4, z(8, 16), 1, 8, 16, 0, z(4, 7)),
        lambda: m.moesq_gemm(z(4, 16), None, 0, 1, None, 4, z(16, 16), 1, 16, 16, 1, z(4, 8), z(4, 8)),
        lambda: m.gemm_dx(z(4, 8), z(16, 8)), lambda: m.gemm_dx(z(4, 8), z(8, 16), z=z(4, 16)),
        lambda: m.gemm_dx(z(4, 8), z(8, 16), out=z(4, 8)), lambda: m.gemm_dx(z(4, 8), z(2, 8, 16), z(2, dt=i32)),
        lambda: m.gemm_dw(z(4, 8), z(3, 16)), lambda: m.gemm_dw(z(4, 8), z(4, 16), out=z(8, 8)),
        lambda: m.gemm_dw(z(4, 8), z(4, 16), out=z()), lambda: m.gemm_dw(z(4, 8), z(4, 16), accumulate=True),
        lambda: m.gemm_dw(z(4, 8), z(2, 16), z(2, dt=i32), perm=z(4, dt=i32), k=3),
        lambda: m.gemm_dw(z(4, 8), z(4, 16), z(3, dt=i32), E=2, out=z(8, 16)),
        lambda: m.unpermute_backward(z(4, 8), z(8, 8), z(8, dt=i32), z(8, dt=f32), 3, 2),
        lambda: m.unpermute_backward(z(4, 8), z(7, 8), z(8, dt=i32), z(8, dt=f32), 4, 2),
        lambda: m.unpermute_backward(z(4, 8), z(8, 8), z(7, dt=i32), z(8, dt=f32), 4, 2),
        lambda: m.unpermute_backward(z(4, 8), z(8, 8), z(8, dt=i32), z(7, dt=f32), 4, 2),
        lambda: m.Lora(z(3, 16, 24), z(3, 40, 16), z(3, dt=f32), slices=2), lambda: m.Lora(z(16, 24), z(40, 8), z(1, dt=f32)),
        lambda: m.Lora(z(2, 8, 24), z(3, 40, 8), z(3, dt=f32)), lambda: m.Lora(z(3, 8, 24), z(3, 40, 8), z(2, dt=f32)),
        lambda: m.Lora(z(3, 0, 24), z(3, 40, 8), z(3, dt=f32), slices=0),
        lambda: m.moesq_lora(z(4, 25), z(4, dt=i32), 4, ad, None, 0, z(4, 40), None),
        lambda: m.moesq_lora(z(4, 24), z(3, dt=i32), 4, ad, None, 0, z(4, 40), None),
        lambda: m.moesq_lora(z(4, 24), z(4, dt=i32), 4, ad, z(4, 20), 0, z(4, 40), None),
        lambda: m.moesq_lora(z(4, 24), z(4, dt=i32), 4, ad, None, 1, z(4, 40), None),
    ]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError) as ei:
            case()
        assert "on the GPU" not in str(ei.value), (i, str(ei.value))
    for case in (lambda: m.gemm(z(4, 16, dt=f32), z(8, 16)), lambda: m.gemm_dw(z(4, 8), z(4, 16), dtype=torch.float16),
                 lambda: m.moesq_lora(z(4, 24), z(4), 4, ad, None, 0, z(4, 40), None)):
        with pytest.raises(TypeError):
            case()
    with pytest.raises(ValueError, match="contiguous"):
        m.gemm(z(16, 4).t(), z(8, 16))
    with pytest.raises(ValueError, match="contiguous"):
        m.gemm_dx(z(4, 16)[:, :8], z(8, 16))
    with pytest.raises(ValueError, match="on the GPU"):
        m.gemm(z(4, 16), z(8, 16))


def test_binding_rejects_counts_beyond_32_bits(m):
    """A wrapped count would leave a part out without an error."""
    z, big = torch.zeros(8, dtype=torch.bfloat16), (1 << 32) + 8
    ad = m.Lora(z.view(1, 1, 8).expand(1, 8, 8), z.view(1, 1, 8), torch.zeros(1))
    for case in (lambda: m.moesq_gemm(z, None, 0, 1, None, big, z, 1, 8, 8, 0, z),
                 lambda: m.moesq_gemm(z, None, 0, 1, None, 1, z, 1, big, 8, 0, z),
                 lambda: m.moesq_gemm(z, z, 1, big, None, big, z, 1, 8, 8, 0, z),
                 lambda: m.moesq_gemm_dx(z, None, big, z, 1, 8, 8, None, z),
                 lambda: m.moesq_gemm_dx(z, None, 1, z, 1, 8, big, None, z),
                 lambda: m.moesq_gemm_dw(z, z, None, 0, 1, None, 1, big, 8, 8, z),
                 lambda: m.moesq_unpermute_backward(z, z, None, None, big, 1, 8, z, None),
                 lambda: m.moesq_unpermute_backward(z, z, None, None, 1, 1, big, z, None),
                 lambda: m.moesq_lora(z, None, big, ad, None, 0, z, None),
                 lambda: m.moesq_lora_workspace_bytes(big, ad)):
        with pytest.raises(ValueError, match="2\\^31"):
            case()


def test_adapters_keep_their_tensors(m):
    a, b, s = torch.zeros(2, 8, 16).bfloat16(), torch.zeros(2, 24, 8).bfloat16(), torch.ones(2)
    ad = m.Lora(a, b, s)
    for name, t in (("a", a), ("b", b), ("scale", s)):
        with pytest.raises(AttributeError):
            setattr(ad, name, t.clone())
    a[0, 0, 0] = 3.0
    assert ad.a is a and float(ad.a[0, 0, 0]) == 3.0
