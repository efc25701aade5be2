"""The operators around shared and bounded decode caches, in fp64 (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Written per sequence
and query token from the definitions, one loop level per sentence of them:

  prefix_attention   entries 0 .. Np-1 shared by all sequences, entry Np + j is
                     row j of the sequence's own cache, plus the raw window;
                     entry e visible to position t iff (e+1) m - 1 < t - W + 1
  attention_weights  sum over heads and query tokens of exp(s - lse) per entry
  evict_select       the entries a cache keeps
  compact            the caches with those entries
"""
from __future__ import annotations

import numpy as np


def _visible(t: int, m: int, W: int) -> int:
    n = 0 if t - W + 1 <= 0 else (t - W + 1) // m
    assert n == 0 or n * m - 1 < t - W + 1
    assert (n + 1) * m - 1 >= t - W + 1
    return n


def prefix_attention(q, kp, vp, kc, vc, k_raw, v_raw, m, W, q_pos, kv_pos0, scale=None):
    """q [B, Lq, Hq, d]; kp, vp [Np, Hkv, d]; kc, vc [B, Nc, Hkv, d]; k_raw, v_raw
    [B, Lkv, Hkv, d]; q_pos [B, Lq]; kv_pos0 [B].  Returns dict(o, lse, a, e, n):
    o, lse, a = sum P |v| (what a relative error of P can move o by), e = the
    largest scale sum |q| |k| over the row's keys (what rounding the products'
    sum is relative to) and n = the number of keys."""
    B, Lq, Hq, d = q.shape
    Np, Hkv = kp.shape[0], kp.shape[1]
    Nc, g = kc.shape[1], Hq // kp.shape[1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, Hq, Lq), -np.inf)
    e, n = np.zeros((B, Hq, Lq)), np.zeros((B, Lq), np.int64)
    for b in range(B):
        for t in range(Lq):
            pos = int(q_pos[b, t])
            nv = _visible(pos, m, W)
            own = min(max(nv - Np, 0), Nc)
            lo = max(0, pos - W + 1) - int(kv_pos0[b])
            hi = pos - int(kv_pos0[b])
            raw = [r for r in range(max(lo, 0), min(hi, k_raw.shape[1] - 1) + 1)] if W else []
            k = np.concatenate([kp[:min(nv, Np)], kc[b, :own], k_raw[b, raw]])
            v = np.concatenate([vp[:min(nv, Np)], vc[b, :own], v_raw[b, raw]])
            n[b, t] = len(k)
            if not len(k):
                continue
            for h in range(Hq):
                s = scale * (k[:, h // g] @ q[b, t, h])
                top = s.max()
                w = np.exp(s - top)
                lse[b, h, t] = top + np.log(w.sum())
                w = w / w.sum()
                o[b, t, h] = w @ v[:, h // g]
                a[b, t, h] = w @ np.abs(v[:, h // g])
                e[b, h, t] = scale * (np.abs(k[:, h // g]) @ np.abs(q[b, t, h])).max()
    return dict(o=o, lse=lse, a=a, e=e, n=n)


def attention_weights(q, kc, lse, m, W, q_pos, idx=None, e0=0, scale=None):
    """q [B, Lq, Hq, d]; kc [B, Nc, Hkv, d] holding entries e0 ..; lse [B, Hq, Lq];
    idx [B, Lq, K] or None.  Returns (acc, tol) [B, Nc]: the weights and
    sum P scale sum |q| |k|, what rounding the scores can move them by."""
    B, Lq, Hq, d = q.shape
    Nc, g = kc.shape[1], Hq // kc.shape[2]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    acc, tol = np.zeros((B, Nc)), np.zeros((B, Nc))
    for b in range(B):
        for t in range(Lq):
            nv = min(max(_visible(int(q_pos[b, t]), m, W) - e0, 0), Nc)
            at = np.arange(nv)
            if idx is not None:
                at = np.array([j for j in idx[b, t] if 0 <= j < nv], np.int64)
            for h in range(Hq):
                s = scale * (kc[b, at, h // g] @ q[b, t, h])
                w = np.exp(s - lse[b, h, t])
                acc[b, at] += w
                tol[b, at] += w * (scale * (np.abs(kc[b, at, h // g]) @ np.abs(q[b, t, h])) + np.abs(lse[b, h, t]))
    return acc, tol


def evict_select(acc, n_keep, n_first=0, n_last=0, n_valid=None):
    """acc [B, Nc] -> keep [B, n_keep] int32."""
    B, Nc = acc.shape
    keep = np.full((B, n_keep), -1, np.int32)
    for b in range(B):
        n = Nc if n_valid is None else min(max(int(n_valid[b]), 0), Nc)
        if n <= n_keep:
            keep[b, :n] = np.arange(n)
            continue
        held = [j for j in range(n) if j < n_first or j >= n - n_last]
        w = np.where(np.isnan(acc[b]), -np.inf, acc[b])
        rest = sorted((j for j in range(n) if n_first <= j < n - n_last), key=lambda j: (-w[j], j))
        keep[b] = np.sort(held + rest[:n_keep - len(held)])
    return keep


def compact(x, keep, out):
    """out [B, No, ...] with row i = x[b, keep[b, i]] where keep[b, i] >= 0."""
    out = out.copy()
    for b in range(keep.shape[0]):
        for i, j in enumerate(keep[b]):
            if j >= 0:
                out[b, i] = x[b, j]
    return out
