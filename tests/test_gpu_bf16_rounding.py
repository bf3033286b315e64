"""The rounding of results to bf16, on every fp32 number."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_every_number(lib):
    """The gradient of a combine whose dout is 1 is the weight, rounded: nearest, ties to the even
    one, infinite past the largest; NaN stays NaN with its sign."""
    T, N = 1 << 25, 8
    dout = torch.ones(T, N, dtype=torch.bfloat16, device="cuda")
    inv = torch.arange(T, dtype=torch.int32, device="cuda")
    dy = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    for first in range(-(1 << 31), 1 << 31, T):
        bits = torch.arange(first, first + T, device="cuda").to(torch.int32)
        lib.moesq_unpermute_backward(dout, None, inv, bits.view(torch.float32), T, 1, N, dy, None)
        got = dy.view(torch.int16)
        assert bool((got == got[:, :1]).all()), first          # either half of a register
        got = got[:, 0].to(torch.int64) & 0xffff
        u = bits.to(torch.int64) & 0xffffffff
        nan = (u & 0x7fffffff) > 0x7f800000
        want = (u + 0x7fff + ((u >> 16) & 1)) >> 16
        assert bool((nan | (got == want)).all()), first
        assert bool((~nan | (((got & 0x7fff) > 0x7f80) & (got >> 15 == u >> 31))).all()), first
