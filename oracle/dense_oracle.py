"""Plain fp64 oracle of the dense attention over paged caches and packed
sequences (test infrastructure only; numpy, one sequence at a time).

Beside every result stands how far a kernel may be from it, derived from the
roundings the operations declare (u = 2^-8 is half a bf16 step relative to
the value, f = 2^-24 the same in fp32):
  scores   fp32 sums of 128 products: |dz| <= 128 * 2f * scale * sum |q_i k_i|
  weights  exp2 and the score error: relative (|dz| + 2^-20) each way, and one
           rounding to bf16 before the product with V
  out      u |out| + (u + 2 (|dz| + 2^-20)) sum_s P_s |v_s|
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8
F = 2.0 ** -24
E4M3_MAX = 448.0


def rotate(x, pos, inv_freq, rot_dim, interleaved):
    """x [N, heads, d] fp64, pos [N]: pairs of the leading rot_dim dims turned
    by pos * inv_freq."""
    y = np.array(x, dtype=np.float64)
    if rot_dim == 0:
        return y
    half = rot_dim // 2
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :half]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    i0 = np.arange(half) * (2 if interleaved else 1)
    i1 = i0 + (1 if interleaved else half)
    a, b = x[..., i0], x[..., i1]
    y[..., i0] = a * c - b * s
    y[..., i1] = b * c + a * s
    return y


def token_rows(seq_lens, cu_new):
    """(row, sequence, position) of every new token that a call places."""
    out = []
    for b, n in enumerate(seq_lens):
        lo, hi = (b, b + 1) if cu_new is None else (cu_new[b], cu_new[b + 1])
        if n > 0:
            out += [(r, b, n - hi + r) for r in range(lo, hi)]
    return out


def attend(q, k, v, scale, n_vis):
    """q [n, d], k, v [m, d], row i seeing the first n_vis[i] keys -> out, lse,
    P, out's tolerance, |dz|."""
    n, m = q.shape[0], k.shape[0]
    vis = np.arange(m)[None, :] < np.asarray(n_vis)[:, None]
    z = np.where(vis, scale * (q @ k.T), -np.inf)
    top = np.max(z, axis=1, initial=-np.inf)
    p = np.where(vis, np.exp(z - np.where(np.isfinite(top), top, 0.0)[:, None]), 0.0)
    l = p.sum(1)
    some = l > 0
    p = p / np.where(some, l, 1.0)[:, None]
    lse = np.where(some, np.where(some, top, 0.0) + np.log(np.where(some, l, 1.0)), -np.inf)
    out = p @ v
    dz = np.max(np.where(vis, 256 * F * scale * (np.abs(q) @ np.abs(k).T), 0.0), axis=1, initial=0.0)
    tol = U * np.abs(out) + (U + 2 * (dz + 2.0 ** -20))[:, None] * (p @ np.abs(v))
    return out, lse, p, tol, dz


def dense(q, k, v, cu_q, cu_k, scale=None):
    """Packed q [nq,H,d], k, v [nk,G,d] fp64 -> out, lse, out's tolerance,
    lse's tolerance.  Rows no sequence owns are NaN."""
    nq, H, d = q.shape
    R = H // k.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    out, lse = np.full(q.shape, np.nan), np.full((nq, H), np.nan)
    tol, ltol = np.full(q.shape, np.nan), np.full((nq, H), np.nan)
    for b in range(len(cu_q) - 1):
        i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        n_vis = np.maximum(0, m - n + 1 + np.arange(n))
        for h in range(H):
            o, ls, _, t, dz = attend(q[i, h], k[j, h // R], v[j, h // R], scale, n_vis)
            out[i, h], lse[i, h], tol[i, h] = o, ls, t
            fin = np.where(np.isfinite(ls), np.abs(ls), 0.0)
            ltol[i, h] = dz + 2.0 ** -20 + 4 * F * fin
    return out, lse, tol, ltol


def dense_backward(q, k, v, dout, cu_q, cu_k, scale=None):
    """Gradients of sum(dout * out) -> dq, dk, dv and their tolerances.

    The kernel takes P from the stored lse, rounds P and dZ = P (dP - D) to
    bf16 once each before their products and takes D = dout . out from the
    bf16 out; with r = 2 (|dz| + 2^-20) the relative error of P, so
      |ddZ| <= (u + 2r) |dZ| + P (eD + eP),  eD = sum_i |dout_i| tol_i + 256 f sum |dout out|
      (tol: out's tolerance), eP = 256 f sum |dout v|
    and each gradient gets one more rounding to bf16."""
    nq, H, d = q.shape
    R = H // k.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    res = {n: np.full(x.shape, np.nan) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: np.full(x.shape, np.nan) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    for b in range(len(cu_q) - 1):
        i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        n_vis = np.maximum(0, m - n + 1 + np.arange(n))
        for x in ("dk", "dv"):
            res[x][j] = tol[x][j] = 0.0
        for h in range(H):
            g = h // R
            o, _, p, t, dz = attend(q[i, h], k[j, g], v[j, g], scale, n_vis)
            do = dout[i, h]
            dp = do @ v[j, g].T
            D = (do * o).sum(1, keepdims=True)
            ds = p * (dp - D)
            r = (2 * (dz + 2.0 ** -20))[:, None]
            e_d = (np.abs(do) * (t + 256 * F * np.abs(o))).sum(1, keepdims=True)
            e_ds = (U + 2 * r) * np.abs(ds) + p * (e_d + 256 * F * (np.abs(do) @ np.abs(v[j, g]).T))
            res["dq"][i, h] = scale * ds @ k[j, g]
            tol["dq"][i, h] = scale * e_ds @ np.abs(k[j, g])
            res["dk"][j, g] += scale * ds.T @ q[i, h]
            tol["dk"][j, g] += scale * e_ds.T @ np.abs(q[i, h])
            res["dv"][j, g] += p.T @ do
            tol["dv"][j, g] += ((U + r) * p).T @ np.abs(do)
    for x in res:
        tol[x] += U * np.abs(res[x]) + 2.0 ** -30
    return res, tol
