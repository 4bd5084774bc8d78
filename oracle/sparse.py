"""Float64 numpy oracle of block-sparse attention and the passes in front of it:
rotation table, per-head RMS norm with rotation and block means, selection of
key blocks, attention over listed blocks.

Beside each value the functions can return the magnitude that its rounding
errors scale with (sums of absolute terms), from which tests derive tolerances.
"""

from __future__ import annotations

import numpy as np

QBLOCK = 128


def rope_table(pos, dims, base=10000.0):
    """pos [axes][S] whole numbers -> (cos, sin) [S][pairs][2] and the turns [S][pairs]."""
    cols = []
    for p, dim in zip(np.asarray(pos, np.float64), dims):
        j = np.arange(dim // 2)
        cols.append(p[:, None] * base ** (-2.0 * j / dim))
    ang = np.concatenate(cols, axis=1)
    return np.stack([np.cos(ang), np.sin(ang)], axis=-1), ang / (2 * np.pi)


def norm_rope(x, w=None, table=None, halves=False, norm=True, eps=1e-6):
    """x [heads][S][D] -> (y, mag): normalised, rotated rows; mag = |a c| + |b s| of each result."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    y = x
    if norm:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * np.asarray(w, np.float64)
    mag = np.abs(y)
    if table is not None and table.shape[1] > 0:
        t = np.asarray(table, np.float64)
        r = 2 * t.shape[1]
        ia = np.arange(r // 2) if halves else np.arange(0, r, 2)
        ib = ia + (r // 2 if halves else 1)
        a, b, c, s = y[..., ia], y[..., ib], t[..., 0], t[..., 1]
        out, mag = y.copy(), mag.copy()
        out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
        y = out
    assert y.shape[-1] == D
    return y, mag


def block_means(y, block):
    """[heads][S][D] -> [heads][ceil(S/block)][D]."""
    return np.stack([y[:, a:a + block].mean(1) for a in range(0, y.shape[1], block)], axis=1)


def block_select(qm, km, topk, keep_first=0, keep_last=0, margin=np.inf):
    """Lists by brute force: (idx [H][nq][topk] padded with -1, count [H][nq])."""
    qm, km = np.asarray(qm, np.float64), np.asarray(km, np.float64)
    H, nq, D = qm.shape
    nk = km.shape[1]
    idx = np.full((H, nq, topk), -1, np.int32)
    count = np.zeros((H, nq), np.int32)
    for h in range(H):
        kh = km[h // (H // km.shape[0])]
        for i in range(nq):
            with np.errstate(invalid="ignore", over="ignore"):
                s = (qm[h, i] * kh).sum(-1) / np.sqrt(D)
            s = np.where(np.isnan(s), -np.inf, s)
            forced = (np.arange(nk) < keep_first) | (np.arange(nk) >= nk - keep_last)
            order = sorted(range(nk), key=lambda j: (not forced[j], -s[j], j))[:topk]
            if nk and np.isfinite(margin):
                best = s.max()
                order = [j for j in order if forced[j] or s[j] >= best - margin]
            order = sorted(order)
            idx[h, i, :len(order)] = order
            count[h, i] = len(order)
    return idx, count


def block_sparse_attention(q, k, v, idx, count, block):
    """State of every row over its list: (O, L, A, s) with A = sum_j p_j |v_j| / l
    and s = max_j sum_d |q_d k_jd| / sqrt(D), the scales of O's and the logits' errors."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, Sq, D = q.shape
    Sk = k.shape[1]
    O, A = np.zeros((H, Sq, D)), np.zeros((H, Sq, D))
    L, smax = np.full((H, Sq), -np.inf), np.zeros((H, Sq))
    for h in range(H):
        kh, vh = k[h // (H // k.shape[0])], v[h // (H // k.shape[0])]
        for b in range(-(-Sq // QBLOCK)):
            rows = slice(b * QBLOCK, min(Sq, (b + 1) * QBLOCK))
            keys = [np.arange(j * block, min(Sk, (j + 1) * block)) for j in idx[h, b, :count[h, b]]
                    if 0 <= j < -(-Sk // block)]
            if not keys:
                continue
            keys = np.concatenate(keys)
            s = q[h, rows] @ kh[keys].T / np.sqrt(D)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            O[h, rows] = p @ vh[keys] / l
            A[h, rows] = p @ np.abs(vh[keys]) / l
            L[h, rows] = (m + np.log(l))[:, 0]
            smax[h, rows] = (np.abs(q[h, rows]) @ np.abs(kh[keys]).T).max(1) / np.sqrt(D)
    return O, L, A, smax
