"""Plain 64-bit forms of the serving operators (CPU, numpy), and how far a kernel may be from them.

Bounds.  u = 2^-24 is half a step of fp32.  A score q.k is a sum of d exact products in fp32, so it is off
by at most (d + 2) 2u sum|q_i k_i| (2u: tensor cores may truncate), and so is, relatively, its exponential;
the exponential itself and its argument's rounding add (|argument| + 4) 2u.  Sums over n keys add
(n + 16) 2u.  A weight P that is rounded for the product with V adds half a step of its type, each output
half a step of bf16.
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4, "f16": 2.0 ** -11}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float32).double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def rotate(x, pos, inv_freq, interleaved, scale, norm=None, eps=0.0):
    """x [T, H, d] float64 -> (value, sum of the magnitudes that went into it)."""
    x = x.copy()
    d = x.shape[-1]
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm
    mag = np.abs(x)
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    if r:
        # the angle in extended precision: 131072 radians leave 47 bits of a double's 53 below one
        angle = pos.astype(np.longdouble)[:, None, None] * np.asarray(inv_freq, np.longdouble)
        c, s = np.cos(angle).astype(np.float64) * scale, np.sin(angle).astype(np.float64) * scale
        one, two = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        a, b = x[..., one].copy(), x[..., two].copy()
        x[..., one], x[..., two] = a * c - b * s, b * c + a * s
        m = (np.abs(a) + np.abs(b)) * abs(scale)
        mag[..., one], mag[..., two] = m, m
    assert x.shape[-1] == d
    return x, mag


def rotate_bound(value, mag, dtype, descale=1.0):
    """Sixteen fp32 roundings on the way (squares' sum over 16 + 3 levels, rsqrt, weight, sine and cosine to
    two steps each, two products and their sum), then one to the output's type."""
    b = 32 * U * mag + HALF[dtype] * np.abs(value)
    if dtype == "e4m3":
        b = b + 2.0 ** -10 * descale   # half of the smallest step
    return b


def cache_rows(k, table, r, n):
    """Rows of sequence r's first n tokens in the cache [outer, rows, H, d], as [n, H, d] float64."""
    k = f64(k)
    if table is None:
        return k[r, :n]
    page = k.shape[1]
    t = np.asarray(table)
    j = np.arange(n)
    return k[t[r, j // page], j % page]


def visible(q_len, n, mask):
    """[q_len, n]: mask None (chain) or q_len 64-bit words."""
    base = n - q_len
    vis = np.ones((q_len, n), bool)
    for i in range(q_len):
        word = (1 << (i + 1)) - 1 if mask is None else int(mask[i]) & (2 ** 64 - 1)
        for b in range(q_len):
            vis[i, base + b] = bool(word >> b & 1)
    return vis


def scores(q, k, scale, G):
    """q [Q, Hq, d], k [n, Hkv, d] -> scores and sums of magnitudes [Hq, Q, n]."""
    k = np.repeat(k, G, axis=1)
    with np.errstate(invalid="ignore"):
        return (np.einsum("qhd,nhd->hqn", q, k) * scale,
                np.einsum("qhd,nhd->hqn", np.abs(q), np.abs(k)) * abs(scale))


def attend(q, k, v, scale, vis):
    """-> out [Q, Hq, d], lse [Hq, Q], sum_j p_j |v_j| and the largest sum of magnitudes of a row [Hq, Q]."""
    Q, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros((Q, Hq, d)), np.zeros((Q, Hq, d))
    lse, top = np.full((Hq, Q), -np.inf), np.zeros((Hq, Q))
    for i in range(Q):
        see = vis[i]
        if not see.any():
            continue
        s, m = scores(q[i:i + 1], k[see], scale, G)
        s, m = s[:, 0], m[:, 0]
        big = s.max(-1, keepdims=True)
        p = np.exp(s - big)
        total = p.sum(-1, keepdims=True)
        lse[:, i] = (big + np.log(total))[:, 0]
        p = p / total
        vv = np.repeat(v[see], G, axis=1)
        out[i] = np.einsum("hn,nhd->hd", p, vv)
        mag[i] = np.einsum("hn,nhd->hd", p, np.abs(vv))
        top[:, i] = m.max(-1)
    return out, lse, mag, top


def score_error(top, d):
    return (d + 2) * 2 * U * top


def attend_bounds(out, lse, mag, top, d, n, p_half, dtype="bf16"):
    """p_half: half a step of the type that the weights are rounded to; dtype: of the output."""
    e = 2 * score_error(top, d) + 2 * (2 * top + 4) * 2 * U + (n + 16) * 2 * U + p_half    # [Hq, Q]
    b_out = HALF[dtype] * np.abs(out) * (1 + 2.0 ** -7) + e.T[..., None] * mag * (1 + 2.0 ** -7) + n * 2.0 ** -33 * mag
    b_lse = score_error(top, d) + (2 * top + 4 + n + 16) * 2 * U + np.abs(np.where(np.isfinite(lse), lse, 0)) * 4 * U
    return b_out, b_lse


def key_mass(q, k, scale, vis, lse):
    """-> the weight of each key [Hkv, n] and its bound."""
    Q, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    s, m = scores(q, k, scale, G)
    p = np.where(vis[None] & np.isfinite(lse)[:, :, None], np.exp(np.where(vis[None], s, 0) - np.where(np.isfinite(lse), lse, 0)[:, :, None]), 0.0)
    e = score_error(m, d) + (np.abs(s) + np.abs(np.where(np.isfinite(lse), lse, 0))[:, :, None] + 4) * 4 * U + (Q * G + 16) * 2 * U
    n = k.shape[0]
    return p.reshape(Hkv, G * Q, n).sum(1), (p * np.where(vis[None], e, 0)).reshape(Hkv, G * Q, n).sum(1)


def evict(mass, n, budget, sink, window):
    """Old indexes of the kept keys, ascending, for one (sequence, head)."""
    N = min(n, budget)
    if N == n:
        return np.arange(n)
    w = mass[:n].astype(np.float64)
    w = np.where(np.isnan(w), np.inf, w)
    nan = np.isnan(mass[:n])
    forced = (np.arange(n) < sink) | (np.arange(n) >= n - window)
    order = sorted(range(n), key=lambda j: (not forced[j], not nan[j], -w[j], j))
    return np.sort(np.array(order[:N], dtype=np.int64))
