"""Float64 oracle of latent attention (absorbed and expanded forms) and of
draft verification, written from the definitions. Test infrastructure only:
it shares no code with the CUDA path.

Both attention oracles also return, per output element, how far a kernel may
be off by rounding alone (see ``attention_tolerance``).
"""
from __future__ import annotations

import numpy as np

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128


def _attend(z, zabs, v):
    """Softmax attention of one row: scores z [n], their sums of absolute
    products zabs [n], values v [n, d]. Returns out, lse, sum p|v|, max zabs."""
    if z.shape[0] == 0:
        d = v.shape[1]
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    m = z.max()
    e = np.exp(z - m)
    t = e.sum()
    p = e / t
    return p @ v, m + np.log(t), p @ np.abs(v), zabs.max()


def attention_tolerance(out, mass, zabs, n, width, out_bits, lse):
    """Bounds on |out error| and |lse error| of a kernel that rounds each weight
    p once to bf16 (half a step: 2^-8 of its value), sums in fp32 and rounds the
    output once. `mass` is sum p|v|, `zabs` the largest sum of absolute products
    of a score (already scaled), `width` its number of products.

    A score of `width` exact products summed in fp32 (chopped at worst: one step
    2^-23 an addition) is off by at most ds = width 2^-23 zabs, plus 2^-22 zabs
    for the scale's own rounding and product. A weight is then off by e^ds - 1
    (under 2 ds) and by 2^-21 (the exponential and its argument's rounding), the
    total by as much and by its own summation (n 2^-24, at most 2^-12 for the n
    here); numerator and denominator both carry these."""
    ds = (width + 2) * 2.0 ** -23 * zabs
    dw = 2 * ds + 2.0 ** -21
    dsum = n * 2.0 ** -23
    half_out = 2.0 ** -8 if out_bits == 16 else 2.0 ** -24
    tol = mass * (2.0 ** -8 + 2 * dw + 2 * dsum) * (1 + half_out) + np.abs(out) * half_out + 1e-30
    lse_tol = ds + dw + dsum + 2.0 ** -22 * (1 + np.abs(lse)) if np.isfinite(lse) else 0.0
    return tol, lse_tol


def latent_decode_ref(q, cache, page_table, seqlens, scale, out_bits=16):
    """q [B, Tq, H, 576], cache [N, P, 576] (float64), page_table [B, W],
    seqlens [B]. Returns out [B, Tq, H, 512], lse [B, Tq, H] and their tolerances."""
    B, Tq, H, _ = q.shape
    P = cache.shape[1]
    out, lse = np.zeros((B, Tq, H, LATENT)), np.full((B, Tq, H), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    for b in range(B):
        L = int(seqlens[b])
        rows = cache[page_table[b, :-(-L // P)]].reshape(-1, LATENT + ROPE)[:L]
        for t in range(Tq):
            n = max(0, L - (Tq - 1) + t)
            if n == 0:
                continue
            z = scale * (q[b, t] @ rows[:n].T)
            za = scale * (np.abs(q[b, t]) @ np.abs(rows[:n]).T)
            for h in range(H):
                o, s, mass, zm = _attend(z[h], za[h], rows[:n, :LATENT])
                out[b, t, h], lse[b, t, h] = o, s
                tol[b, t, h], ltol[b, t, h] = attention_tolerance(o, mass, zm, n, LATENT + ROPE, out_bits, s)
    return out, lse, tol, ltol


def latent_prefill_ref(q, k_nope, k_pe, v, cu_q, cu_k, scale, out_bits=16):
    """q [Sq, H, 192], k_nope / v [Sk, H, 128], k_pe [Sk, 64] (float64). Rows of
    no request come back as NaN."""
    Sq, H, _ = q.shape
    out, lse = np.full((Sq, H, VDIM), np.nan), np.full((Sq, H), np.nan)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    for b in range(len(cu_q) - 1):
        n, m = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for h in range(H):
            k = np.concatenate([k_nope[cu_k[b]:cu_k[b + 1], h], k_pe[cu_k[b]:cu_k[b + 1]]], -1)
            vv = v[cu_k[b]:cu_k[b + 1], h]
            for i in range(n):
                see = min(m, max(0, i + 1 + m - n))
                qi = q[cu_q[b] + i, h]
                z = scale * (k[:see] @ qi)
                za = scale * (np.abs(k[:see]) @ np.abs(qi))
                o, s, mass, zm = _attend(z, za, vv[:see])
                at = cu_q[b] + i
                out[at, h], lse[at, h] = o, s
                tol[at, h], ltol[at, h] = attention_tolerance(o, mass, zm, see, NOPE + ROPE, out_bits, s)
    return out, lse, tol, ltol


def verify_draft_ref(target, draft, tokens, num_draft, u):
    """target [B, K+1, V], draft [B, K, V] or None, tokens [B, K], num_draft [B]
    or None, u [B, K+1], all as stored (fp32 / int). Returns tokens [B, K+1] and
    the number emitted [B]."""
    B, K1, V = target.shape
    out, emitted = np.full((B, K1), -1, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in range(B):
        count = K1 - 1 if num_draft is None else min(max(int(num_draft[b]), 0), K1 - 1)
        n = 0
        while n < count:
            x = int(tokens[b, n])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, n, x])
            if not float(u[b, n]) * q < float(target[b, n, x]):
                break
            out[b, n] = x
            n += 1
        w = target[b, n].astype(np.float64)
        if n < count:
            less = np.zeros(V) if draft is None else draft[b, n].astype(np.float64)
            if draft is None and 0 <= int(tokens[b, n]) < V:
                less[int(tokens[b, n])] = np.inf
            r = np.maximum(w - less, 0.0)
            w = r if r.sum() > 0 else w
        c = np.cumsum(w)
        out[b, n] = min(V - 1, int(np.searchsorted(c, float(u[b, -1]) * c[-1], side="right")))
        emitted[b] = n + 1
    return out, emitted
