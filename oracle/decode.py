"""The 8-bit head and beam search, from their definitions in 64 bits (numpy).

Inputs are float arrays (bf16 values widened exactly) or whole numbers; nothing
here is shared with the product.
"""
from __future__ import annotations

import numpy as np


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float32 values rounded to bf16 (ties to even), as float32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantize(u: np.ndarray, factor=1.0):
    """Codes rint(127 u / max|u|) and scales max|u| factor / 127 of fp64 rows.
    Zero rows: 0 and 0. Rows with a NaN or an infinity: 0 and NaN."""
    u = np.asarray(u, dtype=np.float64)
    bad = ~np.isfinite(u).all(1)
    safe = np.where(bad[:, None], 0.0, u)
    top = np.abs(safe).max(1)
    codes = np.rint(127.0 * safe / np.where(top > 0, top, 1.0)[:, None])
    scales = np.where(bad, np.nan, top * factor / 127.0)
    return codes.astype(np.int8), scales


def rms_norm(x: np.ndarray, gain: np.ndarray, eps: float, residual=None, bf16=False):
    """(codes, scales fp64, h): see quantize; h = x + residual, rounded as the
    inputs' type is."""
    h = np.asarray(x, dtype=np.float32)
    if residual is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            h = h + np.asarray(residual, dtype=np.float32)
            h = bf16_round(h) if bf16 else h
    h64 = h.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        rstd = 1.0 / np.sqrt((h64 * h64).mean(1) + eps)
        codes, scales = quantize(h64 * gain.astype(np.float64), rstd)
    return codes, scales, h


def product(q: np.ndarray, q_scales: np.ndarray, w: np.ndarray, w_scales: np.ndarray) -> np.ndarray:
    """fp32 logits of 8-bit codes: whole-number sums, then two fp32 products.
    (The sums stay below 2^53, so fp64 holds every one of them exactly.)"""
    sums = q.astype(np.float64) @ w.astype(np.float64).T
    return (sums.astype(np.float32) * q_scales.astype(np.float32)[:, None]) * w_scales.astype(np.float32)[None, :]


def beam_select(logits: np.ndarray, scores: np.ndarray, n: int, finished=None, pad_token: int = 0):
    """(scores fp64, parents, tokens, margin) of the n best continuations of
    each group; margin: the smallest gap between two neighbours among the best
    n + 1 scores (inf where there are none), which tells whether rounding could
    exchange them."""
    B, K = scores.shape
    V = logits.shape[1]
    out_s = np.full((B, n), -np.inf)
    out_p = np.full((B, n), -1, dtype=np.int64)
    out_t = np.full((B, n), -1, dtype=np.int64)
    margin = np.full(B, np.inf)
    for b in range(B):
        all_s, all_place = [], []
        for k in range(K):
            s = float(scores[b, k])
            if not s > -np.inf:
                continue
            if finished is not None and finished[b, k]:
                all_s.append(np.array([s]))
                all_place.append(np.array([k * V + pad_token], dtype=np.int64))
                continue
            l = np.asarray(logits[b * K + k], dtype=np.float64)
            ok = np.isfinite(l)
            if not ok.any() or np.isposinf(l).any():
                continue
            m = l[ok].max()
            log_sum = np.log(np.exp(l[ok] - m).sum())
            all_s.append(s + ((l[ok] - m) - log_sum))
            all_place.append(k * V + np.nonzero(ok)[0].astype(np.int64))
        if not all_s:
            continue
        s, place = np.concatenate(all_s), np.concatenate(all_place)
        if len(s) > 4 * n + 64:   # all that can reach the best n, equal ones included
            keep = s >= np.partition(s, len(s) - n - 1)[len(s) - n - 1]
            s, place = s[keep], place[keep]
        order = np.lexsort((place, -s))[: n + 1]
        s, place = s[order], place[order]
        gaps = s[:-1] - s[1:]
        gaps = gaps[gaps > 0]
        if len(gaps):
            margin[b] = gaps.min()
        m = min(n, len(s))
        out_s[b, :m], out_p[b, :m], out_t[b, :m] = s[:m], place[:m] // V, place[:m] % V
    return out_s, out_p, out_t, margin


def beam_reorder(state: np.ndarray, parents: np.ndarray, dim: int) -> np.ndarray:
    """Rows b * beams + i of axis dim from rows b * beams + parents[b, i]."""
    out = state.copy()
    B, K = parents.shape
    src = np.moveaxis(state, dim, 0)
    dst = np.moveaxis(out, dim, 0)
    for b in range(B):
        for i in range(K):
            if 0 <= parents[b, i] < K:
                dst[b * K + i] = src[b * K + parents[b, i]]
    return out
