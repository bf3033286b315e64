"""moesq_rmsnorm: the residual sum bit for bit, y within its roundings (three
fp32 ones, 2^-24 each, then bf16's 2^-8), the quantized rows bit for bit what
the quantizers make of y."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8), (1, 32), (3, 24), (2, 96), (5, 512), (7, 544), (3, 1024), (2, 1056), (5, 2048), (1, 2056), (17, 4096), (4, 4128), (64, 7168),
          (2, 8192), (3, 8200), (2, 16384), (2, 16416), (3, 20480)]


def inputs(T, K, seed=0):
    g = torch.Generator().manual_seed(seed + T + K)
    x = torch.randn(T, K, generator=g) * (1 + 9 * (torch.rand(K, generator=g) < 0.02).float())
    r = torch.randn(T, K, generator=g)
    w = 1 + 0.2 * torch.randn(K, generator=g)
    return [t.to(torch.bfloat16).cuda() for t in (x, r, w)]


def check_y(y, s, w, eps):
    _, ref = oracle.rmsnorm(s.double().cpu().numpy(), w.double().cpu().numpy(), eps)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(ref) + 2.0 ** -133).all()


def check_rows(lib, q, y, rows):
    if rows == lib.ROWS_NVFP4:
        want = lib.quantize_activations(y)
        assert torch.equal(q.row_scale, want.row_scale)
    else:
        want = lib.mx_quantize(y, rows)
    assert torch.equal(q.scales, want.scales) and torch.equal(q.codes, want.codes)


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("rows", [0, 1, 2, 3])
@pytest.mark.parametrize("residual", [False, True])
def test_shapes(lib, T, K, rows, residual):
    if rows and K % 32:
        pytest.skip("quantized rows need K % 32 == 0")
    x, r, w = inputs(T, K)
    y, s, q = lib.rmsnorm(x, w, 1e-6, residual=r if residual else None, rows=rows)
    if residual:
        assert torch.equal(s, (x.float() + r.float()).to(torch.bfloat16))
    else:
        assert s is None
        s = x
    check_y(y, s, w, 1e-6)
    if rows:
        check_rows(lib, q, y, rows)
        only, s2, q2 = lib.rmsnorm(x, w, 1e-6, residual=r if residual else None, y=False, rows=rows)
        assert only is None and torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)
        assert s2 is None or torch.equal(s2, s)


@pytest.mark.parametrize("K", [64, 3008, 20480])
def test_in_place(lib, K):
    """The residual's buffer, or x's, as residual_out; y over x."""
    x, r, w = inputs(6, K, 1)
    y, s, _ = lib.rmsnorm(x, w, 1e-5, residual=r)
    for target in (0, 1):
        a, b, out = x.clone(), r.clone(), torch.empty_like(x)
        lib.moesq_rmsnorm(a, b, w, 6, K, 1e-5, (a, b)[target], out)
        assert torch.equal(out, y) and torch.equal((a, b)[target], s)
        assert torch.equal((b, a)[target], (r, x)[target])
    y0, _, _ = lib.rmsnorm(x, w, 1e-5)
    a = x.clone()
    lib.moesq_rmsnorm(a, None, w, 6, K, 1e-5, None, a)
    assert torch.equal(a, y0)


def test_extreme_rows(lib):
    """Zero rows (eps alone), tiny, huge and non-finite rows beside ordinary
    ones."""
    K = 256
    x, _, w = inputs(8, K, 2)
    x[0] = 0
    x[1] = x[1] * 2.0 ** -60
    x[2] = x[2] * 2.0 ** 60
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5] = 0
    x[5, 100] = 2.0 ** -120
    for rows in (1, 2):
        y, _, q = lib.rmsnorm(x, w, 1e-6, rows=rows)
        fine = [0, 1, 2, 5, 6, 7]
        check_y(y[fine], x[fine], w, 1e-6)
        assert (y[0] == 0).all()
        assert y[3, 7].isnan() and (y[3, :7] == 0).all() and y[4].isnan().all()
        check_rows(lib, q, y, rows)
    y, _, _ = lib.rmsnorm(x[:3], w, 0.0)
    assert y[0].isnan().all()                     # 0 / sqrt(0)
    check_y(y[1:], x[1:3], w, 0.0)


def test_single_bits_do_not_depend_on_the_batch(lib):
    """A row's results are the same alone and in any batch."""
    x, r, w = inputs(300, 7168, 3)
    y, s, q = lib.rmsnorm(x, w, 1e-6, residual=r, rows=lib.ROWS_MXFP8)
    for t in (0, 150, 299):
        a, b, c = lib.rmsnorm(x[t:t + 1], w, 1e-6, residual=r[t:t + 1], rows=lib.ROWS_MXFP8)
        assert torch.equal(a[0], y[t]) and torch.equal(b[0], s[t])
        assert torch.equal(c.codes[0], q.codes[t]) and torch.equal(c.scales[0], q.scales[t])


def test_no_rows(lib):
    y, s, q = lib.rmsnorm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                          torch.ones(64, dtype=torch.bfloat16, device="cuda"), rows=lib.ROWS_MXFP4)
    assert y.shape == (0, 64) and s is None and q.rows == 0


@pytest.mark.parametrize("K", [64, 256, 7168, 20480])
@pytest.mark.parametrize("residual", [False, True])
def test_nvfp4_rows_with_nan_and_infinity(lib, K, residual):
    """A NaN or an infinity in a weight, a token or through 0 * inf: the rows
    are what the quantizer makes of y, block by block."""
    x, r, w = inputs(9, K, 4)
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    x[3] = 0
    r[3] = 0
    x[4, 32:64], r[4, 32:64] = 0, 0
    for name, at, value in (("finite", 0, 1.0), ("nan", 5, float("nan")), ("inf", 37, float("inf")),
                            ("-inf", 63, -float("inf"))):
        v = w.clone()
        v[at] = value
        for rows in (lib.ROWS_NVFP4, lib.ROWS_MXFP8, lib.ROWS_MXFP4):
            y, s, q = lib.rmsnorm(x, v, 1e-6, residual=r if residual else None, rows=rows)
            if name == "nan":
                assert y[:, 5].isnan().all() and y[0, :5].isfinite().all()
            check_rows(lib, q, y, rows)
            _, _, only = lib.rmsnorm(x, v, 1e-6, residual=r if residual else None, y=False, rows=rows)
            assert torch.equal(only.codes, q.codes) and torch.equal(only.scales, q.scales)


@pytest.mark.parametrize("T,K,rows", [((1 << 26) + 5, 8, 0), ((1 << 26) + 5, 32, 1), ((1 << 25) + 3, 544, 0)])
def test_more_rows_than_a_launch_has_threads_for(lib, T, K, rows):
    """2^26 rows of 64 threads, 2^25 of 128: beyond the 2^32 threads of a launch."""
    tail = 1 << 10
    some, _, w = inputs(tail, K, 5)
    y, _, q = lib.rmsnorm(some, w, rows=rows)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    starts = (0, (1 << 24) - tail // 2, (1 << 25) - tail // 2 if T > 1 << 26 else tail, T - tail)
    for t in starts:
        x[t:t + tail] = some
    yb, _, qb = lib.rmsnorm(x, w, rows=rows)
    for t in starts:
        assert torch.equal(yb[t:t + tail], y)
        if rows:
            assert torch.equal(qb.codes[t:t + tail], q.codes) and torch.equal(qb.scales[t:t + tail], q.scales)


@pytest.mark.parametrize("rows", [2, 3])
def test_rows_on_both_sides_of_two_launches(lib, rows):
    """2^24 rows of 64 threads are one launch, what follows another: the
    residual, its sum and the quantized rows go on there."""
    T, K, tail = (1 << 24) + 77, 32, 1 << 10
    some, res, w = inputs(tail, K, 6)
    want = lib.rmsnorm(some, w, residual=res, rows=rows)
    x, r = (torch.zeros(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    starts = (0, T - tail // 2)                      # the second over the border
    for t in starts:
        n = min(tail, T - t)
        x[t:t + n], r[t:t + n] = some[:n], res[:n]
    y, s, q = lib.rmsnorm(x, w, residual=r, rows=rows)
    for t in starts:
        n = min(tail, T - t)
        parts = [(y, want[0]), (s, want[1]), (q.codes, want[2].codes), (q.scales, want[2].scales)]
        if rows == lib.ROWS_NVFP4:
            parts.append((q.row_scale, want[2].row_scale))
        for u, v in parts:
            assert torch.equal(u[t:t + n], v[:n])
