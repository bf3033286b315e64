"""Router selection: top-k experts and weights from scores.  ORACLE (test
infrastructure only).

  l    = logits, NaN -> -inf, +inf -> the largest finite fp32
  p    = softmax(l) over the experts, or sigmoid(l)
  key  = l without a bias, else p + bias; -inf where l or the bias is -inf (a
         NaN bias counts as -inf)
  groups of E / n_group experts score their largest key ("max"), or the sum of
         their two largest p + bias ("top2"); the topk_group best stay, ties
         to the lower group
  ids  = the k largest remaining keys, descending, ties to the lower expert;
         slots without an unmasked expert hold -1 and weight 0
  w    = p [/ sum of the selected p] * scale

Plain loops over rows, experts and slots in float64.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def gate_topk(logits, k: int, score: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
              group_score: str = "top2", renormalize: bool = True, scale: float = 1.0, n_rows=None):
    L = np.asarray(logits, np.float64)
    T, E = L.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    L = np.minimum(np.where(np.isnan(L), -np.inf, L), FLT_MAX)
    b = None if bias is None else np.asarray(bias, np.float64)
    if b is not None:
        b = np.minimum(np.where(np.isnan(b), -np.inf, b), FLT_MAX)
    per = E // n_group
    for t in range(T if n_rows is None else min(T, max(0, n_rows))):
        l = L[t]
        live = l > -np.inf
        with np.errstate(over="ignore", under="ignore"):
            if score == "sigmoid":
                p = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
            else:
                m = l.max()
                p = np.where(live, np.exp(np.where(live, l, 0.0) - (m if live.any() else 0.0)), 0.0)
                p = p / p.sum() if live.any() else p
        full = p + (0.0 if b is None else b)
        key = np.where(live, l if b is None else full, -np.inf)
        if n_group > 1:
            gs = np.full(n_group, -np.inf)
            for g in range(n_group):
                part = [e for e in range(g * per, (g + 1) * per) if key[e] > -np.inf]
                if part and group_score == "max":
                    gs[g] = max(key[e] for e in part)
                elif part:
                    gs[g] = sum(sorted((full[e] for e in part), reverse=True)[:2])
            kept = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            for g in range(n_group):
                if g not in kept:
                    key[g * per:(g + 1) * per] = -np.inf
        order = sorted((e for e in range(E) if key[e] > -np.inf), key=lambda e: (-key[e], e))[:k]
        for j, e in enumerate(order):
            ids[t, j], w[t, j] = e, p[e]
        if renormalize and w[t].sum() > 0:
            w[t] = w[t] / w[t].sum()
        elif renormalize:
            w[t] = 0.0
    return ids.reshape(-1), (w * scale).reshape(-1)
