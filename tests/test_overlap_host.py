"""The bf16 product, its gradients, the combine's gradient and the adapters refuse results that
share bytes with what is still to be read (no GPU: before any HIP call)."""
from __future__ import annotations

import ctypes

import pytest

MB = 1 << 20


@pytest.fixture(scope="module")
def m():
    from sparse_fp4_expert_amd import moesq
    return moesq


def refused(m, status):
    return status == m.ERR_ARG and b"overlap" in m._last_error()


# Buffers of 64 rows, N = 64 and K = 128, two experts: x 16 KB, w 32 KB, y 8 KB (SwiGLU 4), z 8 KB.
# Each case moves one of them to share its first or last 16 bytes with another.

def test_gemm(m):
    def call(x=MB, w=2 * MB, y=3 * MB, z=None, epi=0):
        return m._gemm(x, None, 0, 1, 0x10, 64, w, 2, 64, 128, epi, y, z, None)

    for bad in (dict(y=MB), dict(y=MB + 16384 - 16), dict(y=MB - 8192 + 16), dict(y=2 * MB + 32768 - 16),
                dict(y=2 * MB - 8192 + 16)):
        assert refused(m, call(**bad)), bad
    for bad in (dict(z=MB), dict(z=2 * MB), dict(z=3 * MB), dict(z=3 * MB + 4096 - 16), dict(z=3 * MB - 8192 + 16),
                dict(z=4 * MB, y=MB + 16384 - 16), dict(z=4 * MB, y=MB - 4096 + 16)):
        assert refused(m, call(epi=m.EPI_SWIGLU, **bad)), bad
    # gathered, x has T rows: 32 of 256 bytes here
    gathered = lambda y: m._gemm(MB, 0x10, 32, 2, 0x10, 64, 2 * MB, 2, 64, 128, 0, y, None, None)    # noqa: E731
    assert refused(m, gathered(MB + 8192 - 16)) and refused(m, gathered(MB))


def test_gemm_dx(m):
    def call(dy=MB, w=2 * MB, z=None, dx=3 * MB):
        return m._gemm_dx(dy, 0x10, 64, w, 2, 64, 128, z, dx, None)

    for bad in (dict(dx=MB), dict(dx=MB + 8192 - 16), dict(dx=MB - 16384 + 16), dict(dx=2 * MB + 32768 - 16),
                dict(z=4 * MB, dx=MB - 32768 + 16), dict(z=4 * MB, dx=4 * MB + 16), dict(z=4 * MB, dx=4 * MB - 32768 + 16),
                dict(z=MB, dx=MB)):
        assert refused(m, call(**bad)), bad


def test_gemm_dw(m):
    def call(dy=MB, x=2 * MB, dw=3 * MB, dtype=0, ws=None, n=0):
        return m._gemm_dw(dy, x, None, 0, 1, 0x10, 64, 2, 64, 128, dtype, 0, dw, ws, n, None)

    for bad in (dict(dw=MB), dict(dw=MB + 8192 - 16), dict(dw=MB - 65536 + 16), dict(dw=MB - 32768 + 16, dtype=1),
                dict(dw=2 * MB), dict(dw=2 * MB + 16384 - 16), dict(ws=MB, n=256), dict(ws=2 * MB - 240, n=256),
                dict(ws=3 * MB + 65536 - 16, n=256)):
        assert refused(m, call(**bad)), bad


def test_unpermute_backward(m):
    def call(dout=MB, y=2 * MB, inv=3 * MB, w=4 * MB, dy=5 * MB, dw=6 * MB):
        return m._unpermute_bw(dout, y, inv, w, 32, 2, 64, dy, dw, None)       # 4 KB, 8 KB, 256 bytes

    for bad in (dict(dy=MB), dict(dy=MB - 8192 + 16), dict(dy=MB + 4096 - 16), dict(dy=2 * MB + 16), dict(dy=2 * MB - 16),
                dict(dy=3 * MB), dict(dy=4 * MB - 8192 + 16), dict(dw=MB), dict(dw=2 * MB + 8192 - 4), dict(dw=3 * MB),
                dict(dw=4 * MB + 252), dict(dw=5 * MB + 4)):
        assert refused(m, call(**bad)), bad


def test_lora(m):
    d = ctypes.byref(m.LoraDesc(0x10, 0x10, 0x10, 2, 16, 1, 64, 128))
    ws = m._lora_ws(64, d)

    def call(x=MB, base=2 * MB, y=3 * MB, w=4 * MB, epi=0):
        return m._lora(x, 0x10, 64, d, base, epi, y, w, ws, None)              # 16 KB, 8 KB, 8 KB (SwiGLU 4)

    for bad in (dict(y=2 * MB + 16), dict(y=2 * MB - 8192 + 16), dict(y=2 * MB + 8192 - 16, epi=1),
                dict(y=2 * MB - 4096 + 16, epi=1), dict(w=MB), dict(w=MB - ws + 16), dict(w=2 * MB), dict(w=3 * MB + 8192 - 16)):
        assert refused(m, call(**bad)), bad
