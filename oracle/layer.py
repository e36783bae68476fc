"""fp64 definitions of the transformer-layer operators (RMS norm, expert routing, attention), plain numpy loops.

Used only by the tests; shares no code with the GPU path.  Inputs are float arrays (bf16 values already widened).
"""
from __future__ import annotations

import numpy as np

F8_MAX = 448.0


def rms_norm(x, residual, weight, eps: float):
    """(s, y): s = x + residual (residual may be None), y = s / sqrt(mean(s^2) + eps) * weight, by rows."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    return s, s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def f8_scales(y, block: int):
    """Scales of the 8-bit output: max |y| / 448 over each row (block 0) or each block of columns, at least 2^-126."""
    b = block or y.shape[1]
    return np.stack([np.maximum(np.abs(y[:, a:a + b]).max(axis=1) / F8_MAX, 2.0 ** -126)
                     for a in range(0, y.shape[1], b)], axis=1)


def moe_gate(logits, topk: int, score: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
             group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """(ids, gate) of every token, one token after another."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids, gate = np.zeros((T, topk), np.int32), np.zeros((T, topk))
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-x))
        else:
            m = x.max()
            with np.errstate(invalid="ignore"):   # infinity less itself, not taken
                s = np.zeros(E) if m == -np.inf else np.where(x == m, 1.0, np.exp(np.where(x == m, 0.0, x - m)))
            s = s / s.sum() if s.sum() > 0 else s
        c = x if bias is None else s + np.asarray(bias, np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        allowed = np.ones(E, bool)
        if n_group > 1:
            per = E // n_group
            by = c if (bias is not None or group_top == 1) else s
            worth = [sum(sorted(by[g * per:(g + 1) * per], reverse=True)[:group_top]) for g in range(n_group)]
            kept = sorted(range(n_group), key=lambda g: (-worth[g], g))[:topk_group]
            allowed = np.array([e // per in kept for e in range(E)])
        order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-c[e], e))[:topk]
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(topk)
        ids[t], gate[t] = order, w * scale
    return ids, gate


def attention(q, k, v, scale: float, causal: bool):
    """One sequence: q Lq x Hq x D, k and v Lk x Hkv x D.  Returns (out, lse, sum_j p_j |v_j|) with p the softmax."""
    Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[:2]
    out, mag = np.zeros((Lq, Hq, D)), np.zeros((Lq, Hq, D))
    lse = np.full((Lq, Hq), -np.inf)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)].astype(np.float64), v[:, h // (Hq // Hkv)].astype(np.float64)
        z = q[:, h].astype(np.float64) @ kh.T * scale
        for i in range(Lq):
            n = min(max(i + Lk - Lq + 1, 0), Lk) if causal else Lk
            if n == 0:
                continue
            m = z[i, :n].max()
            e = np.exp(z[i, :n] - m)
            lse[i, h] = m + np.log(e.sum())
            p = e / e.sum()
            out[i, h] = p @ vh[:n]
            mag[i, h] = p @ np.abs(vh[:n])
    return out, lse, mag


def packed_attention(q, k, v, cu_q, cu_k, scale: float, causal: bool):
    """Sequences packed one after another (cu_q, cu_k: their offsets)."""
    parts = [attention(q[cu_q[s]:cu_q[s + 1]], k[cu_k[s]:cu_k[s + 1]], v[cu_k[s]:cu_k[s + 1]], scale, causal)
             for s in range(len(cu_q) - 1)]
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(3))


def paged_attention(q, k_cache, v_cache, table, lens, scale: float):
    """One token per sequence over a cache of n_pages x page_size x Hkv x D."""
    n_pages, page = k_cache.shape[:2]
    parts = []
    for b in range(q.shape[0]):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        at = [(int(table[b, j // page]), j % page) for j in range(n)]
        at = [(p, s) for p, s in at if 0 <= p < n_pages]
        pi, si = [p for p, _ in at], [s for _, s in at]
        parts.append(attention(q[b:b + 1], k_cache[pi, si], v_cache[pi, si], scale, False))
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(3))
