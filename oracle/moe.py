"""Router, row layout and combine of a mixture-of-experts layer in 64 bits."""

import numpy as np


def gate(logits, k, renorm=True, w_scale=1.0, loss_coef=0.0, valid=None):
    """dict of topk_idx, topk_w, counts (E + 1), prob_sum, loss, and p (rows that are not routed: zeros)."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    valid = np.ones(T, bool) if valid is None else np.asarray(valid).astype(bool)
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    p = np.zeros((T, E))
    for t in range(T):
        if not valid[t]:
            continue
        ok = np.nonzero(x[t] > -np.inf)[0]  # NaN compares false
        order = ok[np.argsort(-x[t][ok], kind="stable")][:k]
        idx[t, :len(order)] = order
        with np.errstate(invalid="ignore"):
            if len(ok):
                e = np.exp(x[t] - x[t][ok].max())
                p[t] = e / e.sum()
            elif np.isnan(x[t]).any():
                p[t] = np.nan
        if np.isnan(p[t]).any():
            p[t] = np.nan
            w[t] = np.nan
        elif len(order):
            top = p[t, order]
            w[t, :len(order)] = w_scale * top / (top.sum() if renorm else 1.0)
    counts = np.zeros(E + 1, np.int32)
    np.add.at(counts, idx[idx >= 0], 1)
    counts[E] = (idx[:, 0] >= 0).sum()
    prob_sum = p.sum(0)
    C, n = counts[:E].sum(), counts[E]
    a = (counts[:E] * prob_sum).sum()
    loss = loss_coef * E * a / (C * n) if n else a
    return dict(topk_idx=idx, topk_w=w, counts=counts, prob_sum=prob_sum, loss=loss, p=p)


def gate_grad(out, dw, dloss, renorm=True, w_scale=1.0, loss_coef=0.0):
    """(dlogits, sum of the magnitudes its terms have) from gate()'s dict."""
    p, idx, w, counts = out["p"], out["topk_idx"], out["topk_w"], out["counts"]
    T, E = p.shape
    C, n = counts[:E].sum(), counts[E]
    g = dloss * loss_coef * E * counts[:E] / (C * n) if n else np.zeros(E)
    d = np.zeros((T, E))
    mag = np.zeros((T, E))
    for t in range(T):
        if idx[t, 0] < 0:
            continue
        j = idx[t] >= 0
        wd = w[t, j] * dw[t, j]
        base = (p[t] * g).sum() + (0.0 if renorm else wd.sum())
        d[t] = p[t] * (g - base)
        mag[t] = p[t] * (np.abs(g) + (p[t] * np.abs(g)).sum() + np.abs(wd).sum())
        own = w[t, j] * (dw[t, j] - (wd.sum() / w_scale if renorm else 0.0))
        d[t, idx[t, j]] += own
        mag[t, idx[t, j]] += np.abs(wd) + np.abs(w[t, j]) * np.abs(wd).sum() / abs(w_scale)
    return d, mag


def layout(topk_idx, first, G, max_m=0, rows=None):
    """dict of counts, row_token, row_of and (contiguous) m_indices."""
    idx = np.asarray(topk_idx)
    T, k = idx.shape
    rows = G * max_m if max_m else rows
    counts = np.zeros(G, np.int64)
    for e in idx.ravel():
        if e >= 0 and first <= e < first + G:
            counts[e - first] += 1
    start = np.arange(G) * max_m if max_m else np.concatenate(([0], np.cumsum((counts + 127) // 128 * 128)[:-1]))
    row_token = np.full(rows, -1, np.int32)
    m_indices = np.full(rows, -1, np.int32)
    row_of = np.full((T, k), -1, np.int32)
    seen = np.zeros(G, np.int64)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e < 0 or not first <= e < first + G:
                continue
            g = e - first
            r = start[g] + seen[g]
            if (seen[g] < max_m) if max_m else (r < rows):
                row_of[t, j], row_token[r], m_indices[r] = r, t, g
            seen[g] += 1
    held = np.minimum(counts, max_m) if max_m else counts
    return dict(counts=held.astype(np.int32), row_token=row_token, row_of=row_of, m_indices=m_indices)


def combine(rows, row_of, w):
    """(y, sum of the magnitudes of its terms) in fp64; w is used as given."""
    T, k = row_of.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            r = row_of[t, j]
            if 0 <= r < rows.shape[0]:
                y[t] += w[t, j] * rows[r]
                mag[t] += np.abs(w[t, j] * rows[r])
    return y, mag


def combine_grad(dy, rows, row_of, w):
    """(drows with NaN in rows of no choice, dw, sum of |rows| |dy| per choice)."""
    T, k = row_of.shape
    drows = np.full(rows.shape, np.nan)
    dw = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_of[t, j]
            if 0 <= r < rows.shape[0]:
                drows[r] = w[t, j] * dy[t]
                dw[t, j] = rows[r] @ dy[t]
                mag[t, j] = np.abs(rows[r]) @ np.abs(dy[t])
    return drows, dw, mag
