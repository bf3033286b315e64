"""Router, RMS norm and MX operators without a GPU: the oracle's functions
against closed forms and hand-computed values, and the refusals of the entry
points and of the binding, all before any HIP call."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def m():
    from sparse_fp4_expert_amd import moesq
    return moesq


# ------------------------------------------------------------------ oracle pins

def test_mx_scale_and_codes_by_hand():
    """amax 6.5: floor(log2) = 2, so the FP4 scale is 2^0 and 6.5 saturates at
    6; FP8 takes 2^(2-8) and 6.5 * 64 = 416 is on its grid."""
    x = np.zeros((1, 32))
    x[0, :5] = [6.5, -0.25, 0.75, 2.5, -0.2]
    c, s = oracle.mx_quantize(x, "mxfp4")
    assert s[0, 0] == 127
    v = oracle.mx_decode(c, s, "mxfp4")[0]
    assert list(v[:5]) == [6.0, 0.0, 1.0, 2.0, 0.0]       # ties to the even code
    assert (c[0, 0] >> 4) == 0 and (c[0, 2] & 15) == 0     # zeros are +0
    c, s = oracle.mx_quantize(x, "mxfp8")
    assert s[0, 0] == 127 + 2 - 8
    v = oracle.mx_decode(c, s, "mxfp8")[0]
    assert v[0] == 6.5 and v[1] == -0.25 and v[3] == 2.5
    assert abs(v[4] + 0.2) <= 0.2 * 2.0 ** -4


def test_mx_scale_edges():
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    x = np.zeros((4, 32))
    x[0, 3], x[1, 3], x[2, 3] = tiny, big, np.inf
    for fmt, emax in (("mxfp4", 2), ("mxfp8", 8)):
        c, s = oracle.mx_quantize(x, fmt)
        assert list(s[:, 0]) == [0, 127 + 127 - emax, 255, 0]
        assert not c[3].any() and not c[2].any()
        v = oracle.mx_decode(c, s, fmt)
        assert np.isnan(v[2]).all() and not v[3].any()
        assert v[1, 3] == (6.0 if fmt == "mxfp4" else 448.0) * 2.0 ** (127 - emax)


@pytest.mark.parametrize("fmt,half_step", [("mxfp4", 2.0 ** -2), ("mxfp8", 2.0 ** -4)])
def test_mx_error_bound(fmt, half_step):
    """Values of the block's top binade and below, not saturating, are off by
    at most half a step of their own binade, or of the lowest one."""
    x = np.random.default_rng(0).standard_normal((50, 64)).astype(np.float32).astype(np.float64)
    c, s = oracle.mx_quantize(x, fmt)
    v = oracle.mx_decode(c, s, fmt)
    f = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    top, low = (6.0, 1.0) if fmt == "mxfp4" else (448.0, 2.0 ** -6)
    inside = np.abs(x) <= top * f
    assert (np.abs(v - x) <= half_step * np.maximum(np.abs(x), low * f))[inside].all()
    assert (np.abs(v) == top * f)[~inside].all()


def test_rmsnorm_closed_form():
    s, y = oracle.rmsnorm(np.full((1, 8), 3.0), np.full(8, 2.0), 0.0)
    assert np.allclose(y, 2.0, rtol=0, atol=1e-15) and (s == 3.0).all()
    s, y = oracle.rmsnorm(np.array([[1.0, 0, 0, 0]]), np.ones(4), 0.75, residual=np.array([[0, 1.0, 0, 0]]))
    assert (s == [[1, 1, 0, 0]]).all()
    assert np.allclose(y, [[1 / math.sqrt(1.25)] * 2 + [0, 0]], atol=1e-15)


def test_gate_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = oracle.gate_topk(l, 2)
    assert list(ids) == [2, 1] and np.allclose(w, [4 / 6, 2 / 6])
    ids, w = oracle.gate_topk(l, 3, renormalize=False, scale=2.0)
    assert list(ids) == [2, 1, 0] and np.allclose(w, [1.0, 0.5, 0.25])     # tie 0 / 3 to the lower
    # the bias moves the selection, not the weights
    ids, w = oracle.gate_topk(l, 1, bias=[0, 0, 0, 1.0], renormalize=False)
    assert list(ids) == [3] and np.allclose(w, [1 / 8])
    # groups {0,1}, {2,3}: sums of two 3/8 and 5/8, maxima 2 and 4
    for gs in ("max", "top2"):
        ids, _ = oracle.gate_topk(l, 2, n_group=2, topk_group=1, group_score=gs)
        assert list(ids) == [2, 3]
    # masked experts are never selected
    ids, w = oracle.gate_topk([[0.0, -np.inf, np.nan, 1.0]], 3)
    assert list(ids) == [3, 0, -1] and w[2] == 0 and abs(w.sum() - 1) < 1e-15
    ids, w = oracle.gate_topk([[-np.inf] * 4], 2, score="sigmoid")
    assert list(ids) == [-1, -1] and not w.any()
    ids, w = oracle.gate_topk(np.zeros((3, 4)), 2, n_rows=1)
    assert list(ids) == [0, 1, -1, -1, -1, -1]


# ------------------------------------------------------------------ C refusals

def _gate(m, **kw):
    d = dict(k=2, score=0, n_group=1, topk_group=1, group_score=0, renormalize=1, scale=1.0)
    d.update(kw)
    return m.GateDesc(*(d[f] for f, _ in m.GateDesc._fields_))


def test_gate_rejects(m):
    def call(logits=0x10, dtype=0, T=4, E=8, bias=None, gate=None, ids=0x10, w=0x10, **kw):
        g = ctypes.byref(_gate(m, **kw)) if gate is None else gate
        return m._gate_topk(logits, dtype, T, E, bias, g, None, ids, w, None)

    assert m._gate_topk(0x10, 0, 4, 8, None, None, None, 0x10, 0x10, None) == m.ERR_NULL
    assert call(E=0) == m.ERR_SHAPE and call(E=m.MAX_EXPERTS + 1) == m.ERR_SHAPE
    assert call(k=0) == m.ERR_SHAPE and call(k=9) == m.ERR_SHAPE
    assert call(E=128, k=m.GATE_MAX_TOPK + 1) == m.ERR_SHAPE
    assert call(n_group=3) == m.ERR_SHAPE and call(n_group=0) == m.ERR_SHAPE
    assert call(E=130, n_group=65) == m.ERR_SHAPE
    assert call(n_group=4, topk_group=5) == m.ERR_SHAPE
    assert call(n_group=4, topk_group=0) == m.ERR_SHAPE
    assert call(n_group=4, topk_group=1, k=3) == m.ERR_SHAPE     # two experts a group
    assert call(T=-1) == m.ERR_SHAPE and call(T=1 << 30, k=4) == m.ERR_SHAPE
    assert call(dtype=2) == m.ERR_ARG and call(score=2) == m.ERR_ARG
    assert call(n_group=2, group_score=2) == m.ERR_ARG
    assert call(renormalize=2) == m.ERR_ARG
    assert call(scale=float("nan")) == m.ERR_ARG and call(scale=float("inf")) == m.ERR_ARG
    assert call(logits=None) == m.ERR_NULL and call(ids=None) == m.ERR_NULL
    assert call(w=None) == m.ERR_NULL
    assert call(logits=0x12) == m.ERR_ARG and call(dtype=1, logits=0x11) == m.ERR_ARG
    assert b"aligned" in m._last_error()
    assert call(T=0, logits=None, ids=None, w=None) == m.OK


def test_mx_quantize_rejects(m):
    q = m._mx_quantize
    assert q(0x10, 1, -1, 64, 1, 0x10, 0x10, None) == m.ERR_SHAPE
    assert q(0x10, 1, 4, 48, 1, 0x10, 0x10, None) == m.ERR_SHAPE
    assert q(0x10, 1, 4, 0, 1, 0x10, 0x10, None) == m.ERR_SHAPE
    assert q(0x10, 5, 4, 64, 1, 0x10, 0x10, None) == m.ERR_ARG
    assert q(0x10, 1, 4, 64, m.ROWS_NVFP4, 0x10, 0x10, None) == m.ERR_ARG
    assert q(0x10, 1, 4, 64, m.ROWS_NONE, 0x10, 0x10, None) == m.ERR_ARG
    assert q(None, 1, 4, 64, 1, 0x10, 0x10, None) == m.ERR_NULL
    assert q(0x10, 1, 4, 64, 1, 0x10, None, None) == m.ERR_NULL
    assert q(0x18, 1, 4, 64, 1, 0x10, 0x10, None) == m.ERR_ARG
    assert q(None, 1, 0, 64, 1, None, None, None) == m.OK
    ref = ctypes.byref
    d = m._mx_decode
    assert d(None, 0x10, None) == m.ERR_NULL
    assert d(ref(m.MxDesc(0x10, 0x10, 4, 48, 1)), 0x10, None) == m.ERR_SHAPE
    assert d(ref(m.MxDesc(0x10, 0x10, -1, 64, 1)), 0x10, None) == m.ERR_SHAPE
    assert d(ref(m.MxDesc(0x10, 0x10, 4, 64, 3)), 0x10, None) == m.ERR_ARG
    assert d(ref(m.MxDesc(0x10, None, 4, 64, 1)), 0x10, None) == m.ERR_NULL
    assert d(ref(m.MxDesc(0x18, 0x10, 4, 64, 1)), 0x10, None) == m.ERR_ARG
    assert d(ref(m.MxDesc(None, None, 0, 64, 1)), None, None) == m.OK


def test_rmsnorm_rejects(m):
    def call(x=0x10, res=None, w=0x10, T=4, K=64, eps=1e-6, ro=None, y=0x100, rows=0, c=None, s=None, g=None):
        return m._rmsnorm(x, res, w, T, K, eps, ro, y, rows, c, s, g, None)

    assert call(T=-1) == m.ERR_SHAPE and call(K=12) == m.ERR_SHAPE and call(K=0) == m.ERR_SHAPE
    assert call(K=40, rows=m.ROWS_MXFP8, c=0x10, s=0x10) == m.ERR_SHAPE
    assert call(rows=4) == m.ERR_ARG and call(rows=-1) == m.ERR_ARG
    assert call(eps=-1.0) == m.ERR_ARG and call(eps=float("nan")) == m.ERR_ARG
    assert call(eps=float("inf")) == m.ERR_ARG
    assert call(x=None) == m.ERR_NULL and call(w=None) == m.ERR_NULL
    assert call(res=0x10) == m.ERR_NULL and call(ro=0x10) == m.ERR_NULL
    assert call(y=None) == m.ERR_NULL                       # nothing asked for
    assert call(rows=m.ROWS_MXFP4, c=0x10) == m.ERR_NULL
    assert call(rows=m.ROWS_NVFP4, c=0x10, s=0x10) == m.ERR_NULL
    assert call(res=0x20, ro=0x30, y=0x10) == m.ERR_ARG     # y over x with a residual
    assert call(res=0x20, ro=0x30, y=0x30) == m.ERR_ARG
    assert call(res=0x20, ro=0x30, y=0x20) == m.ERR_ARG
    assert call(x=0x18) == m.ERR_ARG and call(y=0x108) == m.ERR_ARG
    assert call(rows=m.ROWS_MXFP4, c=0x18, s=0x10) == m.ERR_ARG
    assert call(T=0, x=None, w=None, y=None) == m.OK


def test_mx_gemm_rejects(m):
    ref = ctypes.byref
    W = dict(codes=0x1000, scales=0x1000, rows=8 * 64, K=128, format=1)
    X = dict(codes=0x1000, scales=0x1000, rows=4, K=128, format=2)

    def call(x=None, w=None, perm=None, T=0, k=1, off=0x10, M=4, E=8, epi=0, y=0x10):
        d = [None if v is False else ref(m.MxDesc(*{**base, **(v or {})}.values()))
             for v, base in ((x, X), (w, W))]
        return m._mx_gemm(d[0], perm, T, k, off, M, d[1], E, epi, y, None)

    assert call(x=False) == m.ERR_NULL and call(w=False) == m.ERR_NULL
    assert call(x=dict(format=3)) == m.ERR_ARG and call(w=dict(format=2)) == m.ERR_ARG
    assert call(epi=5) == m.ERR_ARG and call(epi=m.OUT_FLAT) == m.ERR_ARG
    assert call(E=0) == m.ERR_SHAPE and call(E=m.MAX_EXPERTS + 1) == m.ERR_SHAPE
    assert call(w=dict(rows=8 * 64 + 1)) == m.ERR_SHAPE and call(w=dict(rows=8 * 24)) == m.ERR_SHAPE
    assert call(w=dict(rows=0)) == m.ERR_SHAPE
    assert call(w=dict(rows=8 * 48), epi=1) == m.ERR_SHAPE        # SwiGLU: N % 32
    assert call(w=dict(K=48), x=dict(K=48)) == m.ERR_SHAPE
    assert call(x=dict(K=64)) == m.ERR_SHAPE
    assert call(M=-1) == m.ERR_SHAPE and call(M=5) == m.ERR_SHAPE
    wide = dict(perm=0x10, T=(1 << 28) - 1, k=5, M=5 * ((1 << 28) - 1))
    assert call(x=dict(rows=wide["T"], K=32, format=1), w=dict(K=32), **wide) == m.ERR_SHAPE
    assert call(perm=0x10, T=2, k=1) == m.ERR_SHAPE               # M != T*k
    assert call(perm=0x10, T=4, k=0) == m.ERR_SHAPE
    assert call(perm=0x10, T=2, k=2) == m.ERR_SHAPE               # x has M rows, not T
    assert call(perm=0x10, T=4, off=None, E=1) == m.ERR_NULL
    assert call(w=dict(rows=8 << 16, K=1 << 17), x=dict(K=1 << 17)) == m.ERR_SHAPE    # an expert of 4 GiB
    assert call(x=dict(rows=1 << 20, K=4096), w=dict(K=4096), M=1 << 20) == m.ERR_SHAPE
    assert call(off=None) == m.ERR_NULL                           # several experts without offsets
    assert call(y=None) == m.ERR_NULL and call(x=dict(scales=None)) == m.ERR_NULL
    assert call(w=dict(codes=0x1008)) == m.ERR_ARG and call(y=0x18) == m.ERR_ARG
    assert call(x=dict(rows=0, codes=None), M=0, y=None) == m.OK


def test_binding_rejects_mismatched_sizes(m):
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)        # noqa: E731
    f32, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    g = m.Gate(2)
    mx = lambda rows, K: m.Mx(z(rows, K // 2), z(rows, K // 32), m.ROWS_MXFP4)      # noqa: E731
    cases = [
        lambda: m.moesq_gate_topk(z(4, 8, dt=f32), 4, 9, None, g, None, z(8, dt=i32), z(8, dt=f32)),
        lambda: m.moesq_gate_topk(z(4, 8, dt=f32), 4, 8, z(7, dt=f32), g, None, z(8, dt=i32), z(8, dt=f32)),
        lambda: m.moesq_gate_topk(z(4, 8, dt=f32), 4, 8, None, g, None, z(7, dt=i32), z(8, dt=f32)),
        lambda: m.moesq_gate_topk(z(4, 8, dt=f32), 4, 8, None, g, z(2, dt=i32), z(8, dt=i32), z(8, dt=f32)),
        lambda: m.gate_topk(z(8, dt=f32), g),
        lambda: m.moesq_mx_quantize(z(2, 64, dt=bf), 2, 96, 1, z(2, 32), z(2, 2)),
        lambda: m.moesq_mx_quantize(z(2, 64, dt=bf), 2, 64, 1, z(2, 64), z(2, 2)),
        lambda: m.moesq_mx_quantize(z(2, 64, dt=bf), 2, 64, 2, z(2, 64), z(2, 3)),
        lambda: m.mx_quantize(z(2, 48, dt=bf)),
        lambda: m.mx_quantize(z(2, 64, dt=bf), m.ROWS_NVFP4),
        lambda: m.Mx(z(2, 32), z(2, 3), m.ROWS_MXFP4),
        lambda: m.Mx(z(2, 32), z(2, 2), m.ROWS_NVFP4),
        lambda: m.Mx(z(2, 24), z(2, 1), m.ROWS_MXFP4),
        lambda: m.moesq_mx_decode(mx(2, 64), z(2, 32, dt=bf)),
        lambda: m.moesq_rmsnorm(z(2, 64, dt=bf), None, z(63, dt=bf), 2, 64, 1e-6, None, z(2, 64, dt=bf)),
        lambda: m.moesq_rmsnorm(z(2, 64, dt=bf), z(1, 64, dt=bf), z(64, dt=bf), 2, 64, 1e-6,
                                z(2, 64, dt=bf), z(2, 64, dt=bf)),
        lambda: m.moesq_rmsnorm(z(2, 64, dt=bf), None, z(64, dt=bf), 2, 64, 1e-6, None, None,
                                m.ROWS_MXFP8, z(2, 32), z(2, 2)),
        lambda: m.rmsnorm(z(64, dt=bf), z(64, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), None, 0, 1, None, 4, mx(32, 96), 1, 0, z(4, 32, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(3, 64), None, 0, 1, None, 4, mx(32, 64), 1, 0, z(4, 32, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), None, 0, 1, None, 4, mx(32, 64), 1, 0, z(4, 16, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), None, 0, 1, None, 4, mx(32, 64), 1, 1, z(4, 32, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), None, 0, 1, z(4, dt=i32), 4, mx(64, 64), 2, 0, z(4, 32, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), z(7, dt=i32), 4, 2, z(3, dt=i32), 8, mx(64, 64), 2, 0,
                                z(8, 32, dt=bf)),
        lambda: m.moesq_mx_gemm(mx(4, 64), None, 0, 1, None, 4, mx(33, 64), 2, 0, z(4, 16, dt=bf)),
        lambda: m.mx_gemm(mx(4, 64), mx(32, 64), out=z(4, 31, dt=bf)),
    ]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError) as ei:
            case()
        assert "on the GPU" not in str(ei.value), (i, str(ei.value))
    with pytest.raises(TypeError):
        m.gate_topk(z(4, 8, dt=torch.float16), g)
    with pytest.raises(TypeError):
        m.mx_quantize(z(2, 64, dt=torch.float64))


def test_binding_rejects_counts_beyond_32_bits(m):
    """A wrapped count would leave rows out without an error."""
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)        # noqa: E731
    bf, big = torch.bfloat16, (1 << 32) + 4
    q = m.Mx.empty((1,), 32, m.ROWS_MXFP4, device="cpu")
    many = m.Mx.__new__(m.Mx)._set(q.codes, q.scales, m.ROWS_MXFP4, (big,), 32)
    for case in (lambda: m.moesq_gate_topk(z(4, dt=bf), big, 1, None, m.Gate(1), None, None, None),
                 lambda: m.moesq_mx_quantize(z(32, dt=bf), big, 32, 1, None, None),
                 lambda: m.moesq_rmsnorm(z(8, dt=bf), None, z(8, dt=bf), big, 8, 1e-6, None, z(8, dt=bf)),
                 lambda: m.moesq_mx_gemm(q, z(4, dt=torch.int32), 1, big, z(2, dt=torch.int32), big, q, 1, 0, None),
                 lambda: many._described()):
        with pytest.raises(ValueError, match="2\\^31"):
            case()


def test_binding_rejects_lengths_beyond_32_bits(m):
    """A wrapped K, E or k would compute a part of every row without an error."""
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)        # noqa: E731
    bf, big = torch.bfloat16, (1 << 32) + 32
    q = m.Mx.empty((1,), 32, m.ROWS_MXFP4, device="cpu")
    long = m.Mx.__new__(m.Mx)._set(q.codes, q.scales, m.ROWS_MXFP4, (1,), big)
    for case in (lambda: m.moesq_gate_topk(z(4, dt=bf), 1, big, None, m.Gate(1), None, None, None),
                 lambda: m.Gate((1 << 32) + 1),
                 lambda: m.moesq_mx_quantize(z(32, dt=bf), 1, big, 1, None, None),
                 lambda: m.moesq_rmsnorm(z(8, dt=bf), None, z(8, dt=bf), 1, big, 1e-6, None, z(8, dt=bf)),
                 lambda: long._described()):
        with pytest.raises(ValueError, match="2\\^31"):
            case()


def test_rows_keep_their_tensors(m):
    """Another tensor in the place of one whose address the descriptor may hold
    would be passed over, and the old one read behind its release."""
    q = m.Mx.empty((4,), 64, m.ROWS_MXFP4, device="cpu")
    codes, scales = q.codes, q.scales
    for name in ("codes", "scales"):
        with pytest.raises(AttributeError):
            setattr(q, name, torch.zeros_like(getattr(q, name)))
    q.codes[1], q.scales[1] = 3, 127                       # their contents may change
    assert q.codes is codes and q.scales is scales and int(codes[1, 0]) == 3
