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
