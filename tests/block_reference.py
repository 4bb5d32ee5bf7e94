"""The operators around the expert layer in 64 bits, straight from their definitions (numpy),
and the bounds that their float32 arithmetic keeps to."""
import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


# ---------------------------------------------------------------------------- moe_lora_linear
def linear(x, w, bias=None, A=None, B=None, slots=None, ranks=(), scalings=(), f32=False):
    """(y, tol): the projection with adapters in 64 bits and how far a result summed in float32
    may be from it.  Summing n products costs at most n roundings of 2^-23 of their absolute sum
    (the tensor cores may truncate instead of rounding, hence not 2^-24); the shrunk row is
    rounded to bf16 (8 significant bits: 2^-8) or to 24 bits; the result is rounded once to its type."""
    x, w = f64(x), f64(w)
    K = x.shape[1]
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T          # the absolute sum behind the accumulation bound
    rounded = np.zeros_like(y)             # what rounding the shrunk row can move
    for s, (r, f) in enumerate(zip(ranks, scalings)):
        rows = np.nonzero(slots == s)[0]
        if r == 0 or f == 0.0 or rows.size == 0:
            continue
        a, b = f64(A[s, :r]), f64(B[s, :, :r])
        u = f * (x[rows] @ a.T)
        umag = abs(f) * (np.abs(x[rows]) @ np.abs(a).T)
        y[rows] += u @ b.T
        mag[rows] += np.abs(u) @ np.abs(b).T
        unit = 2.0 ** -24 if f32 else 2.0 ** -8
        rounded[rows] += (1.01 * unit * np.abs(u) + K * 2.0 ** -23 * umag) @ np.abs(b).T
    if bias is not None:
        y += f64(bias)
        mag += np.abs(f64(bias))
    steps = K + sum(ranks) + 16
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(y) + 1.01 * steps * 2.0 ** -23 * mag + 1.01 * rounded + 1e-30
    return y, tol


# -------------------------------------------------------------------- moe_lora_select_experts
def select(z, k, sigmoid, bias=None, n_group=1, topk_group=1, top2=False, renormalize=True, factor=1.0):
    """(ids, weights, keys) token by token; ties to the lower id."""
    z = f64(z)
    T, E = z.shape
    b = np.zeros(E) if bias is None else f64(bias)
    ids = np.zeros((T, k), np.int64)
    wts = np.zeros((T, k))
    keys = np.full((T, E), -np.inf)
    for t in range(T):
        out = np.isnan(z[t]) | (z[t] == -np.inf)
        zt = np.where(out, -np.inf, np.minimum(z[t], np.finfo(np.float32).max))
        if sigmoid:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-zt))
        elif out.all():
            s = np.zeros(E)
        else:
            e = np.where(out, 0.0, np.exp(zt - zt.max()))
            s = e / e.sum()
        key = np.where(out, -np.inf, s + b)
        if n_group > 1:
            best = -np.sort(-key.reshape(n_group, -1), axis=1)
            g = best[:, 0] + best[:, 1] if top2 else best[:, 0]
            stay = np.argsort(-g, kind="stable")[:topk_group]
            keep = np.repeat(np.isin(np.arange(n_group), stay), E // n_group)
            key = np.where(keep, key, -np.inf)
        keys[t] = key
        ids[t] = np.argsort(-key, kind="stable")[:k]
        w = np.where(key[ids[t]] > -np.inf, s[ids[t]], 0.0)
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        wts[t] = w * factor
    return ids, wts, keys


# ---------------------------------------------------------------------- moe_lora_qk_norm_rope
def norm_rope(x, weight, table, positions, eps, interleaved):
    """(y, tol) of one set of heads [T, H, D].  Float32 costs: the mean of D squares at most D / 2
    roundings of 2^-23 relative (half of it after the root), and a dozen for the rest, of the two
    products that a rotated value is the sum of; then one rounding to bf16."""
    x, wt, table = f64(x), f64(weight), f64(table)
    D, R = x.shape[2], table.shape[1]
    n = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps) * wt
    y, mag = n.copy(), np.abs(n)
    pos = positions.cpu().numpy()
    for t in range(x.shape[0]):
        if not 0 <= pos[t] < table.shape[0]:
            continue
        c, s = table[pos[t], :R // 2], table[pos[t], R // 2:]
        a = slice(0, R, 2) if interleaved else slice(0, R // 2)
        b = slice(1, R, 2) if interleaved else slice(R // 2, R)
        y[t, :, a] = n[t, :, a] * c - n[t, :, b] * s
        y[t, :, b] = n[t, :, b] * c + n[t, :, a] * s
        both = np.abs(n[t, :, a]) + np.abs(n[t, :, b])
        mag[t, :, a] = mag[t, :, b] = both
    return y, 2.0 ** -8 * np.abs(y) + (D / 2 + 12) * 2.0 ** -23 * mag * 1.5 + 1e-30
