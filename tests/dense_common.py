"""64-bit references of the paged append and the dense attentions (not
collected as tests), with the error bounds the GPU outputs are held to."""

from __future__ import annotations

import numpy as np
import torch


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, d] float64 with its first 2 len(inv_freq) channels rotated."""
    r = 2 * len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out = np.array(x, np.float64)
    if r == 0:
        return out
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = a * c - b * s, a * s + b * c
    return out


def rotation_bound(x, r, interleaved, ref, dtype):
    """Error bound of a rotated row: the angle's fraction of a turn is rounded
    to fp32 (2^-25 turns, 2 pi 2^-25 rad), sine and cosine are good to 2 units
    (2^-23), and two products and a sum round in fp32 (3 * 2^-24), all times
    at most |x| + |y|; then one rounding to dtype."""
    m = np.abs(np.array(x, np.float64))
    if interleaved:
        pair = m[..., 0:r:2] + m[..., 1:r:2]
        m[..., 0:r:2], m[..., 1:r:2] = pair, pair
    else:
        pair = m[..., :r // 2] + m[..., r // 2:r]
        m[..., :r // 2], m[..., r // 2:r] = pair, pair
    fp32 = 2 * np.pi * 2.0 ** -25 + 2.0 ** -23 + 3 * 2.0 ** -24
    bound = m * fp32
    if dtype != torch.float32:
        bound = bound + half_step(dtype) * (np.abs(ref) + bound)
    return bound


def attend(q, k, v, dtype, causal, prefix=0, cap=0.0, slopes=None, scale=None, bend=None):
    """q [n_q, hq, d] at the last n_q positions of k, v [n_k, hkv, d] (float64
    arrays): O, lse, and the bounds of their errors on the GPU.

    Score error (natural units): a dot product of d terms accumulated in fp32,
    each step truncated at worst (2^-23), at most d 2^-23 |q||k|; scaling, cap,
    bias and the log2-domain factor add roundings of the score itself (8 *
    2^-24 |z|) and the cap its tanh (cap 2^-20, or `bend` 2^-20 for a smaller
    `bend`: the largest |z| where tanh is good to 2^-20 relative).  2^x: 2^-22 relative plus the
    rounding of its argument, in all e = the score error twice over (numerator
    and sum) + 2^-20.  Weights of bf16 inputs are rounded to bf16 once before
    they meet the values: half a step of sum p|v|.  O rounds once to dtype.
    fp32 operands taken as two tf32 parts lose 2^-20 of a product: below
    d 2^-23 |q||k| of the scores and inside the e of the weighted values."""
    n_q, hq, d = q.shape
    n_k, hkv = k.shape[:2]
    g = hq // hkv
    scale = 1 / np.sqrt(d) if scale is None else scale
    o, lse = np.zeros((n_q, hq, d)), np.full((n_q, hq), -np.inf)
    ob, lb = np.zeros((n_q, hq, d)), np.zeros((n_q, hq))
    if n_k == 0:
        return o, lse, ob, lb
    pos = n_k - n_q + np.arange(n_q)
    j = np.arange(n_k)
    seen = np.ones((n_q, n_k), bool)
    if causal:
        seen = (j[None] <= pos[:, None]) | (j[None] < prefix)
    dist = np.abs(pos[:, None] - j[None])
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        with np.errstate(all="ignore"):
            z = q[:, h] @ kk.T * scale
            if cap > 0:
                z = cap * np.tanh(z / cap)
            if slopes is not None:
                z = z - float(slopes[h]) * dist
        z = np.where(seen, z, -np.inf)
        live = seen.any(1)
        if not live.any():
            continue
        zl = z[live]
        m = zl.max(1, keepdims=True)
        p = np.exp(zl - m)
        l = p.sum(1, keepdims=True)
        p /= l
        used = seen.any(0)
        vs = np.where(used[:, None], vv, 0)
        o[live, h] = p @ vs
        lse[live, h] = (m + np.log(l))[:, 0]
        qn = np.linalg.norm(q[live, h], axis=1)
        kn = np.linalg.norm(kk[used], axis=1).max()
        zmax = np.abs(np.where(seen[live], zl, 0)).max(1)
        raw = scale * d * 2.0 ** -23 * qn * kn
        ez = raw + 8 * 2.0 ** -24 * (zmax + scale * qn * kn) + (cap if bend is None else bend) * 2.0 ** -20
        e = (2 * ez + 2.0 ** -20)[:, None]
        a = p @ np.abs(vs)
        hs = half_step(dtype)
        w = hs if dtype != torch.float32 else n_k * 2.0 ** -24
        ob[live, h] = a * (w + e) * 1.01 + hs * (np.abs(o[live, h]) + a * (w + e))
        lb[live, h] = ez + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[live, h])
    return o, lse, ob, lb


def check(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref)
    fin = np.isfinite(ref)
    assert (got[~fin] == ref[~fin]).all(), f"{what}: infinities differ"
    err = np.abs(got[fin] - ref[fin])
    bad = ~(err <= np.broadcast_to(bound, ref.shape)[fin])
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst "
                           f"{np.nanmax(err[bad]) if np.isfinite(err[bad]).any() else 'nan'}")


def f64(t):
    return t.detach().cpu().double().numpy()
