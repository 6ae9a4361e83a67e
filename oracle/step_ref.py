"""Float64 oracle of a decode step over selected pages: slots of new tokens, cache
writes and page bounds, page selection, attention over selected pages, log
probabilities. Written from the definitions, one request, row or page at a time.
Test infrastructure only: it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .latent_ref import _attend, attention_tolerance

BAD_PAGE, OVERFLOW, BAD_TOKEN, NO_PAGES = 1, 2, 8, 16


def append_slots_ref(seqlens, num_new, free, num_free, P, table, T, slot_max=2 ** 63 - 1):
    """Returns table, slots [T], positions [T], new lengths, cu [B + 1], pages taken, status bits."""
    table = np.array(table, dtype=np.int64)
    B, W = table.shape
    F = len(free) if num_free is None else min(max(int(num_free), 0), len(free))
    status = BAD_PAGE if num_free is not None and int(num_free) > len(free) else 0
    slots, positions = np.full(T, -1, dtype=np.int64), np.zeros(T, dtype=np.int64)
    lens, cu, asked, taken = [], [0], 0, 0
    for b in range(B):
        bad = seqlens[b] < 0 or num_new[b] < 0
        L, n = max(int(seqlens[b]), 0), max(int(num_new[b]), 0)
        row = cu[-1]
        cu.append(row + n)
        before, after = -(-L // P), -(-(L + n) // P)
        bad = bad or L + n > 2 ** 31 - 1 or after > W or row + n > T
        need = 0 if bad else after - before
        asked += need
        ok = not bad and (need == 0 or asked <= F)
        if not ok:
            status |= OVERFLOW if bad else NO_PAGES
        lens.append(L + n if ok else L)
        if ok and need:
            taken = asked
            table[b, before:after] = free[asked - need:asked]
        for i in range(n):
            if row + i >= T:
                break
            positions[row + i] = min(L + i, 2 ** 31 - 1)
            if ok:
                page = int(table[b, (L + i) // P])
                s = page * P + (L + i) % P
                if page < 0 or s > slot_max:
                    status |= BAD_PAGE
                else:
                    slots[row + i] = s
    return table, slots, positions, np.array(lens), np.minimum(np.array(cu), 2 ** 31 - 1), taken, status


def quantise_ref(x, kind):
    """Codes and fp32 scales of one row [D] of float64 values."""
    top = 127 if kind == "int8" else 7
    groups = x.reshape(1 if kind == "int8" else -1, x.size if kind == "int8" else 32)
    codes, scales = [], []
    for g in groups:
        m = np.abs(g).max()                               # (NaN if any is)
        with np.errstate(invalid="ignore"):
            s = np.float32(m / top)
        scales.append(s)
        if not np.isfinite(s) or s == 0:
            codes.append(np.zeros(g.size, dtype=np.int64))
        else:
            codes.append(np.clip(np.rint(g / np.float64(s)), -top, top).astype(np.int64))
    return np.concatenate(codes), np.array(scales, dtype=np.float32)


def outward(x, up):
    """x (float64) to the nearest bf16 value that is not below (up) or not above it."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore"):
        bits = x.astype(np.float32).view(np.uint32).astype(np.int64)
    v = (bits & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)   # towards zero, of the fp32 rounding
    out = v.copy()
    for idx in np.ndindex(x.shape):
        if not np.isfinite(x[idx]):
            out[idx] = x[idx]
            continue
        b = int(bits[idx]) & 0xffff0000
        around = []
        for d in (-0x20000, -0x10000, 0, 0x10000, 0x20000):
            m = (b & 0x7fffffff) + d
            if 0 <= m <= 0x7f800000:
                mag = float(np.array([m], dtype=np.uint32).view(np.float32)[0])
                around += [mag, -mag]
        out[idx] = min(a for a in around if a >= x[idx]) if up else max(a for a in around if a <= x[idx])
    return out


def append_ref(k, v, slots, k_values, bounds, P, kind):
    """k, v [T, Hkv, D] float64; slots [T]; k_values [N * P, Hkv, D] float64: what the
    key cache held before. Returns {slot: per head (codes or values, scales)} of K and V, and the
    bounds [N, Hkv, 2, D] (float64) after the call."""
    rows = ({}, {})
    values = k_values.copy()
    last = {}
    for t, s in enumerate(slots):
        if s < 0 or s >= values.shape[0]:
            continue
        last[s // P] = max(last.get(s // P, -1), s % P)
        for which, x in ((0, k), (1, v)):
            if kind == "bf16":
                rows[which][s] = x[t]
                if which == 0:
                    values[s] = x[t]
                continue
            per_head = [quantise_ref(x[t, h], kind) for h in range(x.shape[1])]
            rows[which][s] = per_head
            if which == 0:
                for h, (c, sc) in enumerate(per_head):
                    with np.errstate(invalid="ignore"):
                        values[s, h] = c * np.repeat(sc.astype(np.float64), c.size // sc.size)
    bounds = None if bounds is None else bounds.copy()
    if bounds is not None:
        for page, off in last.items():
            x = values[page * P:page * P + off + 1]
            bounds[page, :, 0] = outward(x.min(0), False)
            bounds[page, :, 1] = outward(x.max(0), True)
    return rows, bounds


def page_scores_ref(q, lo, hi):
    """q [G, D], lo / hi [n, D] (float64): sum over heads and channels of the larger product."""
    with np.errstate(invalid="ignore"):
        qp, qn = np.maximum(q, 0).sum(0), np.minimum(q, 0).sum(0)
        return hi @ qp + lo @ qn


def select_ref(q, bounds, table, seqlens, P, S, first, last):
    """q [B, Tq, Hq, D], bounds [N, Hkv, 2, D] (float64). Returns selected [B, Tq, Hkv, S]."""
    B, Tq, Hq, _ = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    out = np.full((B, Tq, Hkv, S), -1, dtype=np.int64)
    W = table.shape[1]
    for b in range(B):
        L = min(max(int(seqlens[b]), 0), W * P)
        for t in range(Tq):
            n = -(-max(0, L - (Tq - 1) + t) // P)
            for h in range(Hkv):
                if n <= S:
                    out[b, t, h, :n] = np.arange(n)
                    continue
                ids = table[b, :n]
                good = (ids >= 0) & (ids < bounds.shape[0])
                bd = bounds[np.where(good, ids, 0), h]
                sc = page_scores_ref(q[b, t, h * G:(h + 1) * G], bd[:, 0], bd[:, 1])
                sc = np.where(np.isnan(sc), np.inf, sc)      # a score that is no number ranks above all
                nan_first = np.isnan(page_scores_ref(q[b, t, h * G:(h + 1) * G], bd[:, 0], bd[:, 1])) & good
                keys = [(-1, 0, j) if j < first or j >= n - last else
                        ((3, 0, j) if not good[j] else ((0, 0, j) if nan_first[j] else (1, -sc[j], j))) for j in range(n)]
                out[b, t, h] = sorted(sorted(range(n), key=lambda j: keys[j])[:S])
    return out


def sparse_ref(q, k_values, v_values, table, seqlens, selected, P, scale, out_bits=16):
    """q [B, Tq, Hq, D], k / v_values [N, P, Hkv, D] (float64, dequantised). Returns out, lse and tolerances."""
    B, Tq, Hq, D = q.shape
    N, _, Hkv, _ = k_values.shape
    G, W = Hq // Hkv, table.shape[1]
    out, lse = np.zeros((B, Tq, Hq, D)), np.full((B, Tq, Hq), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    for b in range(B):
        L = min(max(int(seqlens[b]), 0), W * P)
        for t in range(Tq):
            n = L - (Tq - 1) + t
            for h in range(Hkv):
                ks, vs = [], []
                for p in map(int, selected[b, t, h]):
                    if p < 0 or p * P >= n:
                        continue
                    page = int(table[b, p])
                    if not 0 <= page < N:
                        continue
                    m = min(P, n - p * P)
                    ks.append(k_values[page, :m, h])
                    vs.append(v_values[page, :m, h])
                if not ks:
                    continue
                k, v = np.concatenate(ks), np.concatenate(vs)
                for g in range(G):
                    x = q[b, t, h * G + g]
                    o, s, mass, zm = _attend(scale * (k @ x), scale * (np.abs(k) @ np.abs(x)), v)
                    at = (b, t, h * G + g)
                    out[at], lse[at] = o, s
                    tol[at], ltol[at] = attention_tolerance(o, mass, zm, len(k), D, out_bits, s)
    return out, lse, tol, ltol


def logprobs_ref(x, token, K):
    """One row of logits [V] (float64). Returns logprob, rank, entropy, ids [K], their logprobs."""
    V = x.size
    m = x.max()
    if m == -np.inf:
        lp = np.full(V, -np.inf)
        entropy = 0.0
    else:
        lp = (x - m) - np.log(np.exp(x - m).sum())      # (m + ln would lose the logarithm beside a large m)
        p = np.exp(lp)
        entropy = -(p[p > 0] * lp[p > 0]).sum()
    order = np.lexsort((np.arange(V), -x))[:K]
    rank = int((x > x[token]).sum() + (x[:token] == x[token]).sum())
    return lp[token], rank, entropy, order, lp[order]
