"""64-bit reference of attention under any mask, with the error bounds that
dense_common.attend derives (not collected as tests)."""

from __future__ import annotations

import numpy as np
import torch

from dense_common import half_step


def window_mask(p, n_k, window, sinks, causal):
    """Visible [len(p), n_k] to queries at positions p."""
    j, p = np.arange(n_k)[None], np.asarray(p)[:, None]
    near = p - j < window
    if causal:
        return (near | (j < sinks)) & (j <= p)
    return (near & (j - p < window)) | (j < sinks)


def tree_mask(base, parents):
    """Visible [n, base + n] to the n nodes, and their depths."""
    n = len(parents)
    seen, depth = np.zeros((n, base + n), bool), []
    seen[:, :base] = True
    for i, p in enumerate(parents):
        p = p if 0 <= p < i else -1
        depth.append(0 if p < 0 else depth[p] + 1)
        if p >= 0:
            seen[i, base:] = seen[p, base:]
        seen[i, base + i] = True
    return seen, np.array(depth, int)


def attend_masked(q, k, v, dtype, seen, dist=None, cap=0.0, slopes=None, scale=None):
    """q [n_q, hq, d], k, v [n_k, hkv, d] (float64), seen and dist [n_q, n_k]: O,
    lse and the bounds of their errors on the GPU (see dense_common.attend)."""
    n_q, hq, d = q.shape
    n_k, hkv = k.shape[:2]
    g = hq // hkv
    scale = 1 / np.sqrt(d) if scale is None else scale
    o, lse = np.zeros((n_q, hq, d)), np.full((n_q, hq), -np.inf)
    ob, lb = np.zeros((n_q, hq, d)), np.zeros((n_q, hq))
    live = seen.any(1)
    if not live.any():
        return o, lse, ob, lb
    used = seen.any(0)
    # Only what some row sees is read: the rest may hold anything.
    seen, hs = seen[live][:, used], half_step(dtype)
    for h in range(hq):
        kk, vv = k[used, h // g], v[used, h // g]
        z = q[live, h] @ kk.T * scale
        if cap > 0:
            z = cap * np.tanh(z / cap)
        if slopes is not None:
            z = z - float(slopes[h]) * dist[live][:, used]
        zl = np.where(seen, z, -np.inf)
        m = zl.max(1, keepdims=True)
        p = np.exp(zl - m)
        l = p.sum(1, keepdims=True)
        p /= l
        o[live, h] = p @ vv
        lse[live, h] = (m + np.log(l))[:, 0]
        qn = np.linalg.norm(q[live, h], axis=1)
        kn = np.linalg.norm(kk, axis=1).max()
        zmax = np.abs(np.where(seen, zl, 0)).max(1)
        raw = scale * d * 2.0 ** -23 * qn * kn
        ez = raw + 8 * 2.0 ** -24 * (zmax + scale * qn * kn) + cap * 2.0 ** -20
        e = (2 * ez + 2.0 ** -20)[:, None]
        a = p @ np.abs(vv)
        w = hs if dtype != torch.float32 else n_k * 2.0 ** -24
        ob[live, h] = a * (w + e) * 1.01 + hs * (np.abs(o[live, h]) + a * (w + e))
        lb[live, h] = ez + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[live, h])
    return o, lse, ob, lb
