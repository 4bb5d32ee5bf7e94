"""Attention over a paged cache in 64 bits, straight from its definitions, and the bounds that its float32
arithmetic keeps to."""
import math

import torch


def page_tables(tables, cached, new, page, free, taken, T):
    """Token by token: (tables, kv, offsets, slots, positions, taken) as lists; a token without a page has slot -1."""
    tables = [list(r) for r in tables]
    kv, offsets, slots, positions = [], [0], [], []
    for row, c, n in zip(tables, cached, new):
        c, n = max(c, 0), max(n, 0)
        held = min(-(-c // page), len(row))
        need = min(-(-(c + n) // page), len(row))
        have = held
        while have < need and taken < len(free):
            row[have] = free[taken]
            taken += 1
            have += 1
        kv.append(min(c + n, have * page))
        for pos in range(c, c + n):
            slots.append(row[pos // page] * page + pos % page if pos // page < have else -1)
            positions.append(pos)
        offsets.append(min(offsets[-1] + n, T))
    slots, positions = slots[:T], positions[:T]
    return (tables, kv, offsets, slots + [-1] * (T - len(slots)), positions + [0] * (T - len(positions)), taken)


# Weights as an operand: two bf16 pieces (16 bits) of the kernel for few rows, one of the tiles' kernel, float32 else.
FEW, TILES, PLAIN = 2.0 ** -16, 2.0 ** -8, 0.0


def attention(q, kc, vc, tables, kv_lens, offsets, scale, weights):
    """(out, lse, tol, lse_tol) in 64 bits, row by row; rows of no request are NaN in out (and tol).

    A score is a sum of D products in float32, which the tensor cores may truncate: it is off by at most
    (D + 4) 2^-23 of its absolute sum, scaled; `ds` is the largest over a row's keys.  A weight is then off by
    twice that (its own score and the maximum), 2^-21 of the exponential, and `weights` of its rounding; sums over
    n keys by (n + 64) 2^-23 of their absolute sums.  The result is rounded to bf16 once: half a step is 2^-8."""
    T, Hq, D = q.shape
    Hk, page = kc.shape[1], kc.shape[2]
    G = Hq // Hk
    q, kc, vc = (t.detach().double().cpu() for t in (q, kc, vc))
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol, lse_tol = out.clone(), lse.clone()
    for b, n in enumerate(kv_lens):
        t0, t1 = offsets[b], offsets[b + 1]
        mine = [tables[b][i] for i in range(-(-n // page))]
        for h in range(Hq):
            k = kc[mine, h // G].reshape(-1, D)[:n]
            v = vc[mine, h // G].reshape(-1, D)[:n]
            for t in range(t0, t1):
                sees = n - (t1 - t) + 1
                if sees <= 0:
                    out[t, h], lse[t, h], tol[t, h], lse_tol[t, h] = 0.0, -math.inf, 0.0, 0.0
                    continue
                s = scale * (k[:sees] @ q[t, h])
                lse[t, h] = torch.logsumexp(s, 0)
                if lse[t, h] == -math.inf:
                    out[t, h], tol[t, h], lse_tol[t, h] = 0.0, 0.0, 0.0
                    continue
                p = torch.softmax(s, 0)
                out[t, h] = p @ v[:sees]
                size = k[:sees].abs() @ q[t, h].abs()
                ds = (D + 4) * 2.0 ** -23 * abs(scale) * size[size < math.inf].max()   # a score of -inf is exact
                tol[t, h] = (2.0 ** -8 * out[t, h].abs() +
                             1.01 * (weights + 4 * ds + 2.0 ** -20 + (sees + 64) * 2.0 ** -23) * (p @ v[:sees].abs()) + 1e-30)
                lse_tol[t, h] = 2.0 ** -22 * lse[t, h].abs() + 2 * ds + 2.0 ** -20 + (sees + 64) * 2.0 ** -23
    return out, lse, tol, lse_tol
