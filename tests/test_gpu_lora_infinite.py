"""Infinite elements of an adapter's second matrix."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_lora import Case, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T, A, rank, slices", [(1, 1, 8, 1), (40, 5, 24, 1), (70, 4, 72, 2), (1300, 3, 64, 1), (300, 2, 256, 1)])
def test_infinite_elements(lib, T, A, rank, slices):
    """base + scale sum_j v_j b_j with one infinite b_j is infinite, of the sign of scale v_j b_j,
    whether v_j is a bf16 number or lies above or below the nearest one; with v_j = 0 it is
    NaN.  Other columns and other adapters' rows stay as they are."""
    N, K = 96, 136
    c = Case(lib, T, A, rank, slices, N, K, seed=5, none=0.0, runs=T > 1000)
    c.x[::3, 1:] = 0
    c.x[::3, 0] = 1.5
    c.a[:, 3::rank, 0] = -2.0                                  # there v_3 is -3
    y = lib.lora(c.x, c.lora, c.ids, base=c.base)
    n = N // slices
    at = [(s, s * n + i, j, b) for s in range(slices) for i, j, b in ((5, 3, np.inf), (17, rank - 1, -np.inf))]
    for _, col, j, b in at:
        c.b[A - 1, col, j] = b
    got = lib.lora(c.x, c.lora, c.ids, base=c.base)
    its = c.ids == A - 1
    assert its.any()
    x, a, scale = f64(c.x[its]), f64(c.a[A - 1]), float(c.scale[A - 1])
    for s, col, j, b in at:
        v = x @ a[s * rank + j]
        sure = np.abs(v) > (K / 4 + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(a[s * rank + j]))   # its sign is fp32's
        assert sure.sum() > 0.9 * len(v)
        assert np.array_equal(f64(got[its, col])[sure], (np.sign(scale * v) * b)[sure]), (s, col)
    keep = torch.ones(N, dtype=torch.bool)
    keep[[col for _, col, _, _ in at]] = False
    assert torch.equal(got[:, keep], y[:, keep]) and torch.equal(got[~its], y[~its])
    c.x.zero_()
    assert lib.lora(c.x, c.lora, c.ids, base=c.base)[its][:, ~keep].isnan().all()
