"""The paged key/value cache in 64 bits: the allocator's bookkeeping request by request, the copy
slot by slot, and attention over pages as the dense definition ("Self-Attention with Relative
Position Representations" page, section 3.4, eq. 3 and eq. 4, causal) with every key fetched
through the block table. Numpy only; shares nothing with the library.
"""
from __future__ import annotations

import numpy as np


def plan(cached, new, table, free, head, P, max_tokens):
    """Returns (table, kv_len, q_start, slots, head, all_placed)."""
    table = np.array(table, dtype=np.int64)
    M = table.shape[1]
    kv_len, q_start, slots, ok = [], [0], [], True
    at, want = int(head), int(head)
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = int(c), int(n)
        rows = n if 0 <= n <= max_tokens else 0
        fits = c >= 0 and 0 <= n <= max_tokens and -(-(c + n) // P) <= M and c + n < 2 ** 31
        need = -(-(c + n) // P) - -(-c // P) if fits else 0
        want += need
        placed = fits and q_start[-1] + rows <= max_tokens and (need == 0 or (head >= 0 and want <= len(free)))
        if placed:
            for i in range(need):
                table[b, -(-c // P) + i] = free[want - need + i]
            at = max(at, want) if need else at
            slots += [int(table[b, (c + i) // P]) * P + (c + i) % P for i in range(n)]
        else:
            ok = False
            slots += [-1] * rows
        kv_len.append(c + n if placed else c)
        q_start.append(q_start[-1] + rows)
    ok = ok and q_start[-1] <= max_tokens
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return table, np.array(kv_len), np.array(q_start), np.array(slots), at, ok


def append(k, v, slots, k_pages, v_pages):
    P = k_pages.shape[2]
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    for t, s in enumerate(slots):
        if 0 <= s < k_pages.shape[0] * P:
            k_pages[s // P, :, s % P] = k[t]
            v_pages[s // P, :, s % P] = v[t]
    return k_pages, v_pages


def evict(kv_len, table, k_pages, v_pages, mass, budget, limit, sinks, recent, free=None, head=0):
    """Returns (kv_len, k_pages, v_pages, mass, free, head): every request past `limit` keys cut to
    `budget` head by head, key by key; its pages behind the budget put back in front of `head`."""
    k_pages, v_pages, mass = k_pages.copy(), v_pages.copy(), mass.copy()
    free = None if free is None else np.array(free)
    P, cap = mass.shape[2], table.shape[1] * mass.shape[2]
    out, gone = [], []
    for b, n in enumerate(kv_len):
        n = min(max(int(n), 0), cap)
        if n <= limit:
            out.append(int(kv_len[b]))
            continue
        out.append(budget)
        gone += [int(x) for x in table[b, -(-budget // P):-(-n // P)]]
        at = lambda j: (table[b, j // P], j % P)
        for h in range(mass.shape[1]):
            rest = range(sinks, n - recent)
            w = [mass[at(j)[0], h, at(j)[1]] for j in rest]
            w = [np.inf if np.isnan(x) else x for x in w]
            nan = [np.isnan(mass[at(j)[0], h, at(j)[1]]) for j in rest]
            heavy = sorted(range(len(w)), key=lambda i: (not nan[i], -w[i], i))[:budget - sinks - recent]
            kept = list(range(sinks)) + sorted(sinks + i for i in heavy) + list(range(n - recent, n))
            assert len(kept) == budget
            for x in (k_pages, v_pages, mass):
                rows = [x[at(j)[0], h, at(j)[1]].copy() for j in kept]
                for r, row in enumerate(rows):
                    x[at(r)[0], h, at(r)[1]] = row
    if free is not None:
        head -= len(gone)
        free[head:head + len(gone)] = gone
    return np.array(out), k_pages, v_pages, mass, free, head


def attend(q, k_pages, v_pages, table, q_start, kv_len, aK, aV, clip_k, window, sinks, scale):
    """q [T, H, d], pages [N, Hkv, P, d], tables [Hkv|1, 2k+1, d] or None, all float64.

    Returns (z [T, H, d], mass [T, H, d], size [T, H]): the output; sum_j p_j (|v_j| + |aV_j|),
    the mass that a relative error of the weights acts on; and max_j scale * sum_c |q_c| (|k_jc| +
    |aK_c|), the size of the sums behind a score. Rows from q_start[-1] on stay NaN."""
    T, H, d = q.shape
    N, Hkv, P, _ = k_pages.shape
    g = H // Hkv
    cap = table.shape[1] * P
    z = np.full((T, H, d), np.nan)
    mass, size = np.zeros((T, H, d)), np.zeros((T, H))
    for b in range(len(kv_len)):
        n = int(q_start[b + 1] - q_start[b])
        kv = min(max(int(kv_len[b]), 0), cap)
        for i in range(n):
            t = int(q_start[b]) + i
            pos = kv - n + i
            j = np.arange(pos + 1) if pos >= 0 else np.zeros(0, dtype=np.int64)
            if window > 0:
                j = j[(j > pos - window) | (j < sinks)]
            if len(j) == 0:
                z[t] = 0.0
                continue
            page = table[b, j // P]
            good = (page >= 0) & (page < N)
            row = np.clip(j - pos, -clip_k, clip_k) + clip_k
            for h in range(H):
                hk = h // g
                K = np.where(good[:, None], k_pages[np.where(good, page, 0), hk, j % P], 0.0)
                V = np.where(good[:, None], v_pages[np.where(good, page, 0), hk, j % P], 0.0)
                A = np.abs(K)
                if aK is not None:
                    rel = aK[hk if aK.shape[0] > 1 else 0][row]
                    K, A = K + rel, A + np.abs(rel)
                W = np.abs(V)
                if aV is not None:
                    rel = aV[hk if aV.shape[0] > 1 else 0][row]
                    V, W = V + rel, W + np.abs(rel)
                e = scale * (K @ q[t, h])
                p = np.exp(e - e.max())
                p /= p.sum()
                z[t, h] = p @ V
                mass[t, h] = p @ W
                size[t, h] = abs(scale) * (A @ np.abs(q[t, h])).max()
    return z, mass, size


def _rows(q_start, kv_len, cap, window, sinks):
    """(request, query row, position, keys that it sees) of every new token."""
    for b in range(len(kv_len)):
        n = int(q_start[b + 1] - q_start[b])
        kv = min(max(int(kv_len[b]), 0), cap)
        for i in range(n):
            pos = kv - n + i
            j = np.arange(pos + 1) if pos >= 0 else np.zeros(0, dtype=np.int64)
            if window > 0:
                j = j[(j > pos - window) | (j < sinks)]
            yield b, int(q_start[b]) + i, pos, j


def _scores(q, k_pages, table, b, t, h, pos, j, aK, clip_k, scale):
    N, Hkv, P, _ = k_pages.shape
    hk = h // (q.shape[1] // Hkv)
    page = table[b, j // P]
    good = (page >= 0) & (page < N)
    K = np.where(good[:, None], k_pages[np.where(good, page, 0), hk, j % P], 0.0)
    A = np.abs(K)
    if aK is not None:
        rel = aK[hk if aK.shape[0] > 1 else 0][np.clip(j - pos, -clip_k, clip_k) + clip_k]
        K, A = K + rel, A + np.abs(rel)
    return scale * (K @ q[t, h]), abs(scale) * (A @ np.abs(q[t, h]))


def log_sum(q, k_pages, table, q_start, kv_len, aK, clip_k, window, sinks, scale):
    """lse [T, H] (-inf without keys) and the size of the sums behind a row's scores, [T, H]."""
    T, H, _ = q.shape
    lse, size = np.full((T, H), -np.inf), np.zeros((T, H))
    for b, t, pos, j in _rows(q_start, kv_len, table.shape[1] * k_pages.shape[2], window, sinks):
        for h in range(H if len(j) else 0):
            e, a = _scores(q, k_pages, table, b, t, h, pos, j, aK, clip_k, scale)
            lse[t, h] = e.max() + np.log(np.exp(e - e.max()).sum())
            size[t, h] = a.max()
    return lse, size


def weights(q, k_pages, table, q_start, kv_len, aK, clip_k, window, sinks, scale, lse, mass, accumulate):
    """Returns (mass, bound): the masses after the new tokens, and how far fp32 arithmetic may be from
    them (keys of a page that requests share get the sums of all of them). A weight's exponent is the difference of two numbers of at most `size` (a sum of 2 (d + 6)
    rounded terms) and |lse|, its exponential is within 2 x 2^-22, and a key's sum has as many terms
    as rows see it."""
    u = 2.0 ** -24
    Hkv, P, d = k_pages.shape[1], k_pages.shape[2], q.shape[2]
    g = q.shape[1] // Hkv
    mass = mass.copy()
    bound = np.zeros_like(mass)
    got, err, new = {}, {}, {}
    for b, t, pos, j in _rows(q_start, kv_len, table.shape[1] * P, window, sinks):
        first_new = min(max(int(kv_len[b]), 0), table.shape[1] * P) - int(q_start[b + 1] - q_start[b])
        for h in range(q.shape[1]):
            if not len(j):
                continue
            e, a = _scores(q, k_pages, table, b, t, h, pos, j, aK, clip_k, scale)
            w = np.exp(e - lse[t, h])
            delta = 4.0 * (d + 6) * u * a + 8.0 * u * (a + abs(lse[t, h])) + 2.0 ** -21
            for x, p, s in zip(j, w, w * delta):
                at = (b, int(x), h // g)
                got[at] = got.get(at, 0.0) + p
                err[at] = err.get(at, 0.0) + s
                new[at] = x >= first_new
    rows = int(max(np.diff(q_start), default=0)) * g
    for (b, j, h), s in got.items():
        page = table[b, j // P]
        if not 0 <= page < mass.shape[0]:
            continue
        old = mass[page, h, j % P] if accumulate and not new[b, j, h] else 0.0
        mass[page, h, j % P] = old + s
        bound[page, h, j % P] += err[b, j, h] + 2.0 * rows * u * s + 2.0 * u * abs(old + s) + 1e-36
    return mass, bound


def tolerance(z, mass, size, keys, d, half_step, weight_step):
    """How far a kernel may be from z, element by element.

    half_step: relative rounding of the output's type; weight_step: of the weights' type (2^-24
    where they stay fp32). The scores come from fp32 sums of d products and two more terms, each
    within (d + 2) 2^-24 of `size`, and two rounded additions of the (at most `size` large)
    exponents: a weight is off by a factor of 1 + 2 x that (it and the row's sum), with
    2 x 2^-22 for the exponential and its sum. Sums over `keys` terms in fp32 add keys x 2^-24
    of the mass for the output and for the row sum. A sum of all terms is bounded by twice `size`
    because edge terms and products come in separate sums."""
    u = 2.0 ** -24
    delta = 2.0 * (d + 6) * u * size[..., None] * 2.0
    factor = weight_step + 2.0 * delta + 2.0 * 2.0 ** -22 + 2.0 * keys * u
    return half_step * np.abs(z) + (1.0 + half_step) * factor * mass + 1e-30
