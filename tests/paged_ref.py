"""Plain 64-bit implementations of the paged operators on the CPU, with error bounds.

Caches are built here from contiguous rows: `paged` scatters them over pages in random
order and fills every other row of the pool with NaN, so that anything read that should
not be shows up."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # a rounding, relative (half a step)


def t64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def paged(rows_per_b, first, total, H, d, rows, cols, dtype, seed, spare=2):
    """rows_per_b[b] = (K, V) float tensors [H, n_b, d] holding rows first[b] .. first[b] + n_b - 1.
    Returns (Kp, Vp, table) on the CPU; pages wholly outside have table entry -1."""
    rng = np.random.default_rng(seed)
    B = len(rows_per_b)
    held = [[c for c in range(cols) if c * rows < first[b] + rows_per_b[b][0].shape[1] and (c + 1) * rows > first[b]]
            for b in range(B)]
    n = sum(map(len, held)) + spare
    order = rng.permutation(n)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    Kp = torch.full((n, H, rows, d), float("nan"), dtype=dtype)
    Vp = torch.full((n, H, rows, d), float("nan"), dtype=dtype)
    i = 0
    for b in range(B):
        for c in held[b]:
            table[b, c] = int(order[i])
            i += 1
        for x in range(rows_per_b[b][0].shape[1]):
            p, r = int(table[b, (first[b] + x) // rows]), (first[b] + x) % rows
            Kp[p, :, r], Vp[p, :, r] = rows_per_b[b][0][:, x].to(dtype), rows_per_b[b][1][:, x].to(dtype)
    return Kp, Vp, table


def row_at(pool, table, rows, b, x):
    return pool[int(table[b, x // rows]), :, x % rows]


def chain(parents, t):
    """t and its ancestors up to the root; None where the chain does not end at -1."""
    out = []
    while t >= 0:
        out.append(t)
        p = int(parents[t])
        t = p if p < t else -2
    return out if t == -1 else None


def window(p, w, g, mode):
    lo = max(0, p - w + 1)
    return lo // g, (lo // g * g if mode else lo)


def softmax_row(q, K, V, tau, dtype):
    """(o, lse, bound of |o's error|, bound of |lse's error|) of one row over keys K, V [n, d] (64 bits).

    Scores are fp32 sums of d exact products (relative error (d + 4) 2^-24 of the sum of their
    magnitudes, the scaling included), the exponential is good to 2^-21 relative, weights and their
    sum carry n 2^-24, and bf16 rounds the weights (half a step) before V and the result after."""
    s = (K @ q) * tau
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    ds = (len(q) + 4) * 2.0 ** -24 * tau * (np.abs(K) @ np.abs(q)).max() + 2.0 ** -21 * max(1.0, np.abs(s - m).max())
    o = p @ V / l
    spread = p @ np.abs(V) / l
    rel = 2 * ds + len(s) * 2.0 ** -24 * 2 + 2.0 ** -20
    if dtype == torch.bfloat16:
        rel += HALF[dtype]
    lse = m + np.log(l)
    return o, lse, rel * spread + HALF[dtype] * (np.abs(o) + rel * spread), ds + len(s) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * abs(lse)


def tree(Q, Kp, Vp, table, Kcp, Vcp, ctable, lens, parents, g, w, rows, crows, mode=0, scale=None):
    """Reference of cca_tree_fwd: (O, LSE, bound of O, bound of LSE) in 64 bits."""
    dtype = Q.dtype
    B, Hq, T, d = Q.shape
    Hkv = Kp.shape[1]
    tau = d ** -0.5 if scale is None else scale
    q, k, v, kc, vc = t64(Q), t64(Kp), t64(Vp), t64(Kcp), t64(Vcp)
    table, ctable = table.cpu().numpy(), ctable.cpu().numpy()
    O, dO = np.zeros(q.shape), np.zeros(q.shape)
    L, dL = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        up = list(range(-1, T - 1)) if parents is None else parents[b].tolist()
        for t in range(T):
            ch = chain(up, t)
            if ch is None:
                continue
            p = n + len(ch) - 1
            cores, start = window(p, w, g, mode)
            raw = list(range(start, n)) + [n + x for x in ch]
            K = np.stack([row_at(kc, ctable, crows, b, j) for j in range(cores)] + [row_at(k, table, rows, b, x) for x in raw], 1)
            V = np.stack([row_at(vc, ctable, crows, b, j) for j in range(cores)] + [row_at(v, table, rows, b, x) for x in raw], 1)
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                O[b, h, t], L[b, h, t], dO[b, h, t], dL[b, h, t] = softmax_row(q[b, h, t], K[kv], V[kv], tau, dtype)
    return O, L, dO, dL


def close(got, want, bound, what=""):
    got = t64(got)
    assert got.shape == want.shape, what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what + ": infinities"
    err = np.abs(np.where(inf, 0, got - np.where(inf, 0, want)))
    assert not np.isnan(err).any(), what + ": NaN"
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(err / np.maximum(bound, 1e-300)).max():.3g} of its bound"


def rotate(X, pos, inv_freq, layout, factor=1.0, sign=1.0):
    """(y, bound of |y's error|) of rotating X [B, H, N, d] by pos [B, N] * inv_freq, in 64 bits.
    Sines and cosines are fp32 values good to 2^-22, and each product and sum rounds."""
    x = t64(X)
    f = np.asarray(inv_freq, dtype=np.float64)
    r = len(f)
    ia = np.arange(r) if layout == "half" else np.arange(0, 2 * r, 2)
    ib = ia + r if layout == "half" else ia + 1
    a = np.asarray(pos, dtype=np.float64)[:, None, :, None] * f
    c, s = factor * np.cos(a), sign * factor * np.sin(a)
    y, bound = x.copy(), np.zeros_like(x)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    size = abs(factor) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    # p * f in 64 bits is itself off by 2^-52 of its size
    bound[..., ia] = bound[..., ib] = (2.0 ** -22 + 4 * 2.0 ** -24 + 2.0 ** -51 * np.abs(a)) * size
    bound[..., ia] += HALF[X.dtype] * np.abs(y[..., ia])
    bound[..., ib] += HALF[X.dtype] * np.abs(y[..., ib])
    return y, bound


def pool_groups(Q, Kp, Vp, table, lens, accepted, path, g, rows, mode=0, scale=None):
    """Yields (b, j, core K [Hkv, d], core V, bound K, bound V) of the groups cca_pool_pages pools."""
    B, Hq, T, d = Q.shape
    Hkv = Kp.shape[1]
    r = Hq // Hkv
    tau = d ** -0.5 if scale is None else scale
    q, k, v, tab = t64(Q), t64(Kp), t64(Vp), table.cpu().numpy()
    for b in range(B):
        n, got = int(lens[b]), int(accepted[b])
        for j in range(n // g, (n + got) // g):
            i = (j + 1) * g - 1 - n
            node = i if path is None else int(path[b, i])
            K = np.stack([row_at(k, tab, rows, b, x) for x in range(j * g, j * g + g)], 1)   # [Hkv, g, d]
            V = np.stack([row_at(v, tab, rows, b, x) for x in range(j * g, j * g + g)], 1)
            qs = q[b, :, node].reshape(Hkv, r, d)
            z = np.einsum("hrd,hgd->hrg", qs, K) * tau
            size = np.einsum("hrd,hgd->hrg", np.abs(qs), np.abs(K)).max() * tau
            if mode == 0:
                z = z.mean(1)
                a = np.exp(z - z.max(-1, keepdims=True))
                a /= a.sum(-1, keepdims=True)
            elif mode == 1:
                a = np.full((Hkv, g), 1.0 / g)
            elif mode == 3:
                a = np.exp(z - z.max(-1, keepdims=True))
                a = (a / a.sum(-1, keepdims=True)).mean(1)
            if mode == 2:
                yield b, j, K.max(1), V.max(1), 0 * K[:, 0], 0 * V[:, 0]
                continue
            spread = (z.max() - z.min()) if mode != 1 else 0.0
            rel = 2 * (d + r + 4) * 2.0 ** -24 * size * (mode != 1) + 2.0 ** -20 * max(1.0, spread) + (2 * g + 8) * 2.0 ** -24
            out = []
            for x in (K, V):
                y, mag = np.einsum("hg,hgd->hd", a, x), np.einsum("hg,hgd->hd", a, np.abs(x))
                out.append((y, rel * mag + HALF[Q.dtype] * (np.abs(y) + rel * mag)))
            yield b, j, out[0][0], out[1][0], out[0][1], out[1][1]
