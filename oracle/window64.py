"""Sliding-window attention with sinks in 64 bits, in NumPy: test
infrastructure only, no code shared with the library.

Beside each value stands the bound on what 16-bit operands and FP32 sums may
move it, from the arithmetic (h = half a step of the element format, eps / 2):

* a score, an FP32 sum of d products, is off by 2^-23 (d + 8) reach_i at most
  (reach_i = scale max_j sum |q_i||k_j|), its exponential by that and by
  2^-22 (4 + 2 reach_i) for the exponent's rounding and ex2: e_i together;
* P_bar is rounded to the element format before P_bar V: h of each P, and in
  fp16 2^-25 absolute where P is below 2^-14 (subnormals).  The shift is at most
  2^4 times 1 / (1 - 2^-11) above the maximum in fp16 (fix_mode 1), or maps it to
  1/2 (fix_mode 2), so that this is at most 2^5 times 2^-25 of the maximum's P;
* O is rounded: h |O|, or in fp16 2^-25 where |O| is below 2^-14 (half a
  subnormal step), and so is each gradient;
* in the backward, P = exp(S - LSE) is off by 2 e_i (LSE carries e_i too) and is
  rounded for dV alone; dP is an FP32 sum like a score; D is taken from the
  rounded O, or as the mean of dP weighted with P: off by what the weights and dP
  are, and 2^-20 of the terms for the sums of up to 8 and the division; dS is
  rounded: h |dS|, or 2^-25 absolute in fp16;
* FP32 accumulation of up to some thousand terms adds less than 2^-18 of the
  terms' size.
"""
from __future__ import annotations

import numpy as np

__all__ = ["visible", "forward", "backward"]


def _f64(x):
    return x.detach().double().cpu().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def visible(N, window, sinks):
    i, j = np.arange(N)[:, None], np.arange(N)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def _row_errors(q, k, scale, vis):
    d = q.shape[-1]
    reach = scale * np.where(vis, np.abs(q) @ np.abs(k).T, 0).max(1, keepdims=True)
    return 2.0 ** -23 * (d + 8) * reach + 2.0 ** -22 * (4 + 2 * reach)


def _forward(q, k, v, scale, vis, h, sub):
    s = np.where(vis, scale * (q @ k.T), -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    o, lse = p @ v, (m + np.log(l))[:, 0]
    err = _row_errors(q, k, scale, vis)
    tol = np.maximum(h * np.abs(o), sub) + (h * (1 + 2 * h) + 2 * err + 2.0 ** -18) * (p @ np.abs(v)) + 32 * sub * (vis @ np.abs(v)) / l
    return p, o, lse, tol, err


def _formats(eps):
    return eps / 2, 2.0 ** -25 if eps < 2.0 ** -8 else 0.0     # fp16 has subnormals in the range of P


def forward(q, k, v, window, sinks, scale, eps):
    """o, lse and their bounds; q [B,H,N,d], k and v [B,Hkv,N,d]; eps of the element format."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, _ = q.shape
    g = H // k.shape[1]
    h, sub = _formats(eps)
    vis = visible(N, window, sinks)
    o, lse, tol, tol_lse = np.zeros_like(q), np.zeros((B, H, N)), np.zeros_like(q), np.zeros((B, H, N))
    for b in range(B):
        for x in range(H):
            _, o[b, x], lse[b, x], tol[b, x], err = _forward(q[b, x], k[b, x // g], v[b, x // g], scale, vis, h, sub)
            tol_lse[b, x] = err[:, 0] + 2.0 ** -23 * np.abs(lse[b, x])
    return o, lse, tol, tol_lse


def backward(q, k, v, do, window, sinks, scale, eps, few=0):
    """(dq, dk, dv) of sum(do * o), and (tol_dq, tol_dk, tol_dv); few: rows of up to
    this many keys take D from their own P and dP."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, H, N, d = q.shape
    g = H // k.shape[1]
    h, sub = _formats(eps)
    vis = visible(N, window, sinks)
    grads = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    tols = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for b in range(B):
        for x in range(H):
            qq, kk, vv, dd = q[b, x], k[b, x // g], v[b, x // g], do[b, x]
            p, o, _, tol_o, err = _forward(qq, kk, vv, scale, vis, h, sub)
            dp, D = dd @ vv.T, (dd * o).sum(1, keepdims=True)
            ds = p * (dp - D)
            size = np.abs(dd) @ np.abs(vv).T
            off_d = (np.abs(dd) * tol_o).sum(1, keepdims=True)
            own = p * (2.0 ** -23 * (d + 8) * size + 2 * err * (np.abs(dp) + np.abs(D)) + 2.0 ** -20 * np.abs(dp))
            off_d = np.where(vis.sum(1, keepdims=True) <= few, own.sum(1, keepdims=True), off_d)
            off = (p * (2.0 ** -23 * (d + 8) * size + off_d
                        + 2 * err * (np.abs(dp) + np.abs(D))))
            off = off + np.maximum(h * (np.abs(ds) + off), sub * vis) + 2.0 ** -18 * np.abs(ds)
            off_p = p * (h + 2 * err + 2.0 ** -18) + sub * vis
            grads[0][b, x] = scale * (ds @ kk)
            grads[1][b, x // g] += scale * (ds.T @ qq)
            grads[2][b, x // g] += p.T @ dd
            tols[0][b, x] = scale * (off @ np.abs(kk))
            tols[1][b, x // g] += scale * (off.T @ np.abs(qq))
            tols[2][b, x // g] += off_p.T @ np.abs(dd)
    return grads, [t + np.maximum(h * (np.abs(w) + t), sub) for t, w in zip(tols, grads)]
