"""moesq_gate_topk against the float64 oracle: ids exactly, weights within the
one rounding to fp32 (2^-24 of the value, plus the two sides' few 64-bit
roundings)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

W_TOL = 2.0 ** -24 * (1 + 1e-6)


def run(lib, logits, k, bias=None, n_rows=None, dtype=torch.float32, **kw):
    names = dict(score={"softmax": lib.SCORE_SOFTMAX, "sigmoid": lib.SCORE_SIGMOID},
                 group_score={"max": lib.GROUP_MAX, "top2": lib.GROUP_TOP2})
    gate = lib.Gate(k, **{n: names[n][v] if n in names else v for n, v in kw.items()})
    l = torch.as_tensor(np.asarray(logits, np.float32)).to(dtype).cuda()
    b = None if bias is None else torch.as_tensor(np.asarray(bias, np.float32)).cuda()
    n = None if n_rows is None else torch.tensor([n_rows], dtype=torch.int32, device="cuda")
    ids, w = lib.gate_topk(l, gate, bias=b, n_rows=n)
    want_ids, want_w = oracle.gate_topk(l.float().cpu().numpy(), k, bias=bias, n_rows=n_rows, **kw)
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    bad = np.nonzero(ids != want_ids)[0]
    assert not bad.size, (bad[:5], ids[bad[:5]], want_ids[bad[:5]])
    # weights below fp32's normal range round to its fixed step
    assert (np.abs(w - want_w) <= W_TOL * np.abs(want_w) + 2.0 ** -149).all()
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 63, 5), (5, 64, 64), (2, 65, 64), (7, 128, 8),
                                   (33, 129, 1), (4, 200, 13), (65, 384, 8), (9, 511, 6), (6, 1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_sizes(lib, T, E, k, score, biased):
    rng = np.random.default_rng(T * 1000 + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    run(lib, rng.standard_normal((T, E)), k, bias=bias, score=score, renormalize=E % 2 == 0, scale=2.5)


@pytest.mark.parametrize("E,G,kg,k", [(8, 2, 1, 4), (64, 64, 5, 5), (96, 8, 4, 8), (384, 8, 4, 8),
                                      (60, 4, 3, 7), (126, 63, 20, 33), (1024, 64, 7, 9), (30, 5, 5, 30)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(lib, E, G, kg, k, group_score, biased):
    rng = np.random.default_rng(E + G)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if biased else None
    for score in ("softmax", "sigmoid"):
        run(lib, rng.standard_normal((21, E)), k, bias=bias, score=score, n_group=G, topk_group=kg,
            group_score=group_score)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lower_index(lib, dtype):
    """Few distinct scores: whole runs of equal keys, with and without a
    bias, in groups and without."""
    rng = np.random.default_rng(2)
    l = rng.integers(0, 3, (40, 96)) * 0.5
    run(lib, l, 9, dtype=dtype)
    run(lib, l, 9, dtype=dtype, bias=np.zeros(96), score="sigmoid")
    run(lib, l, 9, dtype=dtype, n_group=8, topk_group=3)
    run(lib, l, 9, dtype=dtype, bias=np.zeros(96), n_group=8, topk_group=3, group_score="max")
    run(lib, np.zeros((5, 384)), 8, dtype=dtype, bias=np.zeros(384), score="sigmoid", n_group=8, topk_group=4)


def test_keys_nearer_than_fp32(lib):
    """Biased keys that differ by less than an fp32 rounding of the score:
    sigmoid(l) + b with b = c - fp32(sigmoid(l)), for every expert about c."""
    rng = np.random.default_rng(3)
    l = rng.standard_normal((64, 384)).astype(np.float32)
    l[:] = l[0]
    p = 1.0 / (1.0 + np.exp(-l[0].astype(np.float64)))
    bias = (1.0 - p).astype(np.float32)
    ids, _ = run(lib, l, 16, bias=bias, score="sigmoid")
    assert (ids.reshape(64, 16) == ids[:16]).all()
    p = np.exp(l[0].astype(np.float64) - l[0].max())
    run(lib, l, 16, bias=(0.5 - p / p.sum()).astype(np.float32), score="softmax")
    run(lib, l, 16, bias=bias, score="sigmoid", n_group=8, topk_group=4, group_score="top2")
    run(lib, l, 16, bias=bias, score="sigmoid", n_group=8, topk_group=4, group_score="max")


def test_masked_infinite_and_nan(lib):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((12, 48)).astype(np.float32)
    l[0] = -np.inf                                   # a row with nothing left
    l[1, 3:] = -np.inf                               # fewer experts than slots
    l[2, :] = np.nan
    l[3, ::2] = np.nan
    l[4, 7] = np.inf                                 # the largest finite value
    l[5, 7], l[5, 9] = np.inf, np.finfo(np.float32).max
    l[6] = np.finfo(np.float32).min                  # lowest finite, not masked
    l[7, 5:] = np.finfo(np.float32).min
    l[8, 24:] = -np.inf                              # whole groups masked
    l[9, :] = -np.inf
    l[9, 30] = -200.0                                # one expert, far down
    l[10] = l[10] * 100 - 500                        # scores that vanish in fp32
    for score in ("softmax", "sigmoid"):
        for bias in (None, 0.1 * rng.standard_normal(48)):
            for kw in (dict(), dict(n_group=4, topk_group=2), dict(n_group=4, topk_group=2, group_score="max"),
                       dict(renormalize=False)):
                run(lib, l, 8, bias=bias, score=score, **kw)
    bias = 0.1 * rng.standard_normal(48).astype(np.float32)
    bias[:6] = -np.inf, np.nan, np.inf, np.inf, -np.inf, np.finfo(np.float32).min
    run(lib, l, 8, bias=bias, score="sigmoid")
    run(lib, l, 8, bias=np.full(48, -np.inf), score="softmax")


def test_group_sums_below_fp32_range(lib):
    """TOP2 group scores of finite biases, the sums of which fp32 does not hold."""
    l = np.random.default_rng(5).standard_normal((6, 12)).astype(np.float32)
    bias = np.repeat(np.float32([-3e38, -2e38, -2.5e38]), 4)
    for kept in (1, 2):
        ids, _ = run(lib, l, 3, bias=bias, score="sigmoid", n_group=3, topk_group=kept, group_score="top2")
        assert (ids.reshape(6, 3) // 4 == 1).all()
    bias[5:8] = np.finfo(np.float32).min
    run(lib, l, 6, bias=bias, score="softmax", n_group=3, topk_group=2, group_score="top2")
    run(lib, l, 6, bias=np.full(12, np.finfo(np.float32).max), score="sigmoid", n_group=3, topk_group=2,
        group_score="top2")


@pytest.mark.parametrize("n_rows", [-1, 0, 1, 5, 9, 100])
def test_padded_rows(lib, n_rows):
    rng = np.random.default_rng(5)
    ids, w = run(lib, rng.standard_normal((9, 32)), 4, n_rows=n_rows, score="sigmoid")
    live = max(0, min(9, n_rows)) * 4
    assert (ids[live:] == -1).all() and not w[live:].any() and (ids[:live] >= 0).all()


def test_prefill_size(lib):
    """A trillion-class prefill's rows against torch in 64 bits on the device."""
    g = torch.Generator(device="cuda").manual_seed(6)
    l = torch.randn(8192, 384, generator=g, device="cuda")
    b = 0.1 * torch.randn(384, generator=g, device="cuda")
    ids, w = lib.gate_topk(l, lib.Gate(8, score=lib.SCORE_SIGMOID), bias=b)
    p = torch.sigmoid(l.double())
    want = (p + b.double()).sort(dim=1, descending=True, stable=True).indices[:, :8]
    assert torch.equal(ids.view(-1, 8).long(), want)
    pw = p.gather(1, want)
    pw = pw / pw.sum(dim=1, keepdim=True)
    assert ((w.view(-1, 8).double() - pw).abs() <= W_TOL * pw).all()


def test_no_rows_and_offset_storage(lib):
    ids, w = lib.gate_topk(torch.empty(0, 8, device="cuda"), lib.Gate(2))
    assert ids.numel() == 0 and w.numel() == 0
    # a view that starts on an odd element: bf16 logits on a 2-byte boundary
    base = torch.randn(6 * 33 + 1, device="cuda").to(torch.bfloat16)
    l = base[1:].view(6, 33)
    assert l.data_ptr() % 4 == 2
    ids, _ = lib.gate_topk(l, lib.Gate(3))
    want, _ = oracle.gate_topk(l.float().cpu().numpy(), 3)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(12, 4), (96, 9), (384, 8)])
def test_signed_zeros_are_equal_keys(lib, dtype, E, k):
    """-0.0 and +0.0 are one value: a tie between them goes to the lower
    expert, inside the selection and at its border."""
    rng = np.random.default_rng(7)
    zeros = np.copysign(np.zeros((5, E)), rng.standard_normal((5, E)))
    l = np.concatenate([zeros, zeros, zeros])
    for t in range(5):
        l[5 + t, rng.permutation(E)[:k // 2]] = 1.0 + rng.random(k // 2)      # the border falls among zeros
        l[10 + t] = np.where(rng.random(E) < 0.7, rng.standard_normal(E) * 0.0, -1.0 - rng.random(E))
    l[0, :2] = -0.0, 0.0
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(n_group=4, topk_group=2, group_score="max"),
                   dict(n_group=4, topk_group=3, group_score="top2"), dict(bias=np.zeros(E)),
                   dict(bias=np.copysign(np.zeros(E), rng.standard_normal(E)))):
            run(lib, l, k, dtype=dtype, score=score, **kw)


def test_more_rows_than_a_launch_has_threads_for(lib):
    """2^26 rows and more, a wave each: beyond the 2^32 threads of a launch."""
    T, E, tail = (1 << 26) + 7, 4, 1 << 12
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    some = torch.randn(tail, E, generator=g, device="cuda").to(torch.bfloat16)
    starts = (0, (1 << 25) - tail // 2, T - tail)
    for t in starts:
        l[t:t + tail] = some
    gate = lib.Gate(2)
    want = [v.view(tail, 2) for v in lib.gate_topk(some, gate)]
    n = torch.tensor([T - 3], dtype=torch.int32, device="cuda")
    got = [v.view(T, 2) for v in lib.gate_topk(l, gate, n_rows=n)]
    for u, v in zip(got, want):
        for t in starts[:2]:
            assert torch.equal(u[t:t + tail], v)
        assert torch.equal(u[T - tail:T - 3], v[:-3])
    assert (got[0][T - 3:] == -1).all() and (got[1][T - 3:] == 0).all()
