"""Plain 64-bit implementations of the norms with rotation and of the packed operators on the CPU, with
error bounds.  Half a step of a rounding is HALF; fp32 sums of n terms are off by n 2^-24 of the sum of
their magnitudes, exponentials by 2^-20 relative."""
import numpy as np
import torch

from paged_ref import HALF, t64

U = 2.0 ** -24
EX = 2.0 ** -20


def sequences(cu):
    return [(int(a), int(b)) for a, b in zip(cu, cu[1:]) if b > a]


def visible(n, g, w, mode):
    """[n, n // g + n]: whether row i sees core j / token m of its sequence."""
    i = np.arange(n)[:, None]
    lo = np.maximum(0, i - w + 1)
    start = lo // g * g if mode else lo
    j, m = np.arange(n // g)[None], np.arange(n)[None]
    return np.concatenate([(j + 1) * g <= lo, (m >= start) & (m <= i)], 1)


def pool(Q, K, V, cu, g, mode=0, scale=None):
    """(Kc, Vc, bound of each): rows of no group are zero."""
    Hq, T, d = Q.shape
    Hkv, r = K.shape[0], Q.shape[0] // K.shape[0]
    tau = d ** -0.5 if scale is None else scale
    q, k, v = t64(Q), t64(K), t64(V)
    out = [np.zeros((Hkv, T // g, d)) for _ in range(4)]
    for a, b in sequences(cu):
        for j in range((b - a) // g):
            rows = slice(a + j * g, a + j * g + g)
            al, ra = group_weights(q[:, a + j * g + g - 1].reshape(Hkv, r, d), k[:, rows], tau, mode)
            for x, y, e in ((k, out[0], out[2]), (v, out[1], out[3])):
                c = a // g + j
                y[:, c] = np.einsum("hg,hgd->hd", al, x[:, rows])
                mag = np.einsum("hg,hgd->hd", al, np.abs(x[:, rows]))
                e[:, c] = ra * mag + HALF[Q.dtype] * (np.abs(y[:, c]) + ra * mag)
    return out


def group_weights(ql, kg, tau, mode):
    """(a [Hkv, g], relative error of a): ql [Hkv, r, d] the group-last queries, kg [Hkv, g, d]."""
    Hkv, r, d = ql.shape
    g = kg.shape[1]
    if mode == 1:
        return np.full((Hkv, g), 1.0 / g), (2 * g + 8) * U + EX
    z = np.einsum("hd,hgd->hg", ql.mean(1), kg) * tau
    al = np.exp(z - z.max(-1, keepdims=True))
    al /= al.sum(-1, keepdims=True)
    size = np.einsum("hrd,hgd->hg", np.abs(ql), np.abs(kg)).max() / r * tau
    return al, 2 * (d + r + 4) * U * size + EX * max(1.0, z.max() - z.min()) + (2 * g + 8) * U


def attention(Q, K, V, Kc, Vc, cu, g, w, mode=0, scale=None):
    """(O, LSE, bound of O, bound of LSE); NaN for rows of no sequence."""
    Hq, T, d = Q.shape
    r = Hq // K.shape[0]
    tau = d ** -0.5 if scale is None else scale
    q, k, v = t64(Q), t64(K), t64(V)
    O, L, dO, dL = np.full(q.shape, np.nan), np.full((Hq, T), np.nan), np.full(q.shape, np.nan), np.full((Hq, T), np.nan)
    for a, b in sequences(cu):
        n, see = b - a, visible(b - a, g, w, mode)
        for h in range(Hq):
            kk, vv = keys(k, v, Kc, Vc, h // r, a, n, g)
            used = see.any(0)
            kk, vv, m = kk[used], vv[used], see[:, used]
            with np.errstate(all="ignore"):
                s = np.where(m, q[h, a:b] @ kk.T * tau, -np.inf)
                top = s.max(1, keepdims=True)
                p = np.exp(s - top)
                l = p.sum(1, keepdims=True)
                for i in range(n):       # each row by its own keys: what is masked is not looked at
                    O[h, a + i] = p[i, m[i]] @ vv[m[i]] / l[i]
                spread = np.where(m, p, 0) @ np.nan_to_num(np.abs(vv)) / l
                size = np.where(m, np.abs(q[h, a:b]) @ np.nan_to_num(np.abs(kk)).T, 0).max(1, keepdims=True) * tau
                fall = np.maximum(1.0, np.where(m, np.abs(s - top), 0).max(1, keepdims=True))
            ds = (d + 4) * U * size + 2.0 ** -21 * fall
            rel = 2 * ds + m.sum(1, keepdims=True) * 2 * U + EX + (HALF[Q.dtype] if Q.dtype == torch.bfloat16 else 0.0)
            dO[h, a:b] = rel * spread + HALF[Q.dtype] * (np.abs(O[h, a:b]) + rel * spread)
            L[h, a:b] = (top + np.log(l))[:, 0]
            dL[h, a:b] = (ds + m.sum(1, keepdims=True) * U + EX + 2.0 ** -22 * np.abs(top + np.log(l)))[:, 0]
    return O, L, dO, dL


def keys(k, v, Kc, Vc, kv, a, n, g):
    """A sequence's cores, then its tokens, of one KV head."""
    if Kc is None:
        z = np.zeros((n // g, k.shape[2]))
        return np.concatenate([z, k[kv, a:a + n]]), np.concatenate([z, v[kv, a:a + n]])
    c = slice(a // g, a // g + n // g)
    return np.concatenate([t64(Kc)[kv, c], k[kv, a:a + n]]), np.concatenate([t64(Vc)[kv, c], v[kv, a:a + n]])


def few_keys(see, G):
    """The rows whose tile of 128 sees no core and at most 128 tokens from the first one that its first row sees:
    for these the bf16 kernels form D from P and dP, and not from the rounded O."""
    n = len(see)
    few = np.zeros(n, bool)
    for i0 in range(0, n, 128):
        i1 = min(i0 + 128, n) - 1
        few[i0:i1 + 1] = not see[i1, :G].any() and i1 - see[i0, G:].argmax() < 128
    return few


def backward(Q, K, V, Kc, Vc, O, LSE, dO, cu, g, w, mode=0, pool_mode=0, scale=None):
    """((dQ, dK, dV), (their bounds)) of the formulas at the given Kc, Vc, O and LSE; NaN for rows of no sequence."""
    Hq, T, d = Q.shape
    Hkv = K.shape[0]
    r = Hq // Hkv
    tau = d ** -0.5 if scale is None else scale
    bf = HALF[torch.bfloat16] if Q.dtype == torch.bfloat16 else 0.0   # P and dS before their products
    q, k, v, o, lse, go = t64(Q), t64(K), t64(V), t64(O), t64(LSE), t64(dO)
    out = [np.full(x.shape, np.nan) for x in (q, k, v)]
    err = [np.full(x.shape, np.nan) for x in (q, k, v)]
    for a, b in sequences(cu):
        n, G = b - a, (b - a) // g
        see = visible(n, g, w, mode)
        few = few_keys(see, G)
        dk, dv, ek, ev = (np.zeros((Hkv, G + n, d)) for _ in range(4))
        dq, eq = np.zeros((Hq, n, d)), np.zeros((Hq, n, d))
        for h in range(Hq):
            kk, vv = keys(k, v, Kc, Vc, h // r, a, n, g)
            qs, gs = q[h, a:b], go[h, a:b]
            s = qs @ kk.T * tau
            p = np.where(see, np.exp(np.where(see, s, 0) - lse[h, a:b, None]), 0)
            D = (gs * o[h, a:b]).sum(1, keepdims=True)
            dp = gs @ vv.T
            if bf:
                D = np.where(few[:, None], np.where(see, p * dp, 0).sum(1, keepdims=True), D)
            ds = p * (dp - D)
            ds_abs = (d + 4) * U * tau * (np.abs(qs) @ np.abs(kk).T) + 2 * U * np.abs(lse[h, a:b, None]) + U * np.abs(s) * 4
            relp = ds_abs + EX * np.maximum(1.0, np.abs(s - lse[h, a:b, None]))
            edp = (d + 2) * U * (np.abs(gs) @ np.abs(vv).T) + (d + 2) * U * (np.abs(gs) * np.abs(o[h, a:b])).sum(1, keepdims=True)
            eds = np.where(see, np.abs(ds) * (relp + bf + 4 * U) + p * (1 + relp) * (1 + bf) * edp, 0)
            ep = p * (relp + bf)
            rows, cols = see.sum(1, keepdims=True), see.sum(0)[:, None] * r
            dq[h] = tau * ds @ kk
            eq[h] = tau * (eds @ np.abs(kk) + (rows + 4) * U * (np.abs(ds) @ np.abs(kk)))
            dk[h // r] += tau * ds.T @ qs
            ek[h // r] += tau * (eds.T @ np.abs(qs) + (cols + 4) * U * (np.abs(ds).T @ np.abs(qs)))
            dv[h // r] += p.T @ gs
            ev[h // r] += ep.T @ np.abs(gs) + (cols + 4) * U * (p.T @ np.abs(gs))
        seen = max(0, n - w) // g
        for j in range(seen):
            rows = slice(a + j * g, a + j * g + g)
            ql = q[:, a + j * g + g - 1].reshape(Hkv, r, d)
            al, ra = group_weights(ql, k[:, rows], tau, pool_mode)
            kc, vc, ekc, evc = dk[:, j], dv[:, j], ek[:, j], ev[:, j]
            da = np.einsum("hd,hgd->hg", kc, k[:, rows]) + np.einsum("hd,hgd->hg", vc, v[:, rows])
            mag = np.einsum("hd,hgd->hg", np.abs(kc), np.abs(k[:, rows])) + np.einsum("hd,hgd->hg", np.abs(vc), np.abs(v[:, rows]))
            eda = (2 * d + 4) * U * mag + np.einsum("hd,hgd->hg", ekc, np.abs(k[:, rows])) + np.einsum("hd,hgd->hg", evc, np.abs(v[:, rows]))
            m = (al * da).sum(1, keepdims=True)
            em = (al * (eda + (ra + (g + 2) * U) * np.abs(da))).sum(1, keepdims=True)
            ds = al * (da - m) * (pool_mode == 0)
            eds = (np.abs(ds) * (ra + 4 * U) + al * (1 + ra) * (eda + em)) * (pool_mode == 0)
            c, qsum = tau / r, ql.sum(1)
            t = slice(G + j * g, G + j * g + g)
            for x, e, y, ey in ((dk, ek, kc, ekc), (dv, ev, vc, evc)):
                x[:, t] += al[..., None] * y[:, None]
                e[:, t] += al[..., None] * ((1 + ra) * ey[:, None] + (ra + 4 * U) * np.abs(y[:, None]))
            dk[:, t] += c * ds[..., None] * qsum[:, None]
            ek[:, t] += c * (eds[..., None] + (r + 4) * U * np.abs(ds[..., None])) * np.abs(qsum[:, None])
            dq[:, j * g + g - 1] += np.repeat(c * np.einsum("hg,hgd->hd", ds, k[:, rows]), r, 0)
            eq[:, j * g + g - 1] += np.repeat(c * np.einsum("hg,hgd->hd", eds + (g + 4) * U * np.abs(ds), np.abs(k[:, rows])), r, 0)
        for x, e, y, z in ((out[0], err[0], dq, eq), (out[1], err[1], dk[:, G:], ek[:, G:]), (out[2], err[2], dv[:, G:], ev[:, G:])):
            x[:, a:b] = y
            e[:, a:b] = z + HALF[Q.dtype] * (np.abs(y) + z)
    return out, err


# ---------------------------------------------------------------- norms with rotation

def turn(x, pos, freq, layout, factor, sign=1.0):
    """(rotated x, magnitude behind every element, angle sizes) of x [B, H, N, d]."""
    f = np.asarray(freq, dtype=np.float64)
    r = len(f)
    ia = np.arange(r) if layout == "half" else np.arange(0, 2 * r, 2)
    ib = ia + r if layout == "half" else ia + 1
    ang = np.asarray(pos, dtype=np.float64)[:, None, :, None] * f
    c, s = factor * np.cos(ang), sign * factor * np.sin(ang)
    y, mag, far = x.copy(), np.abs(x), np.zeros_like(x)
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    mag[..., ia] = mag[..., ib] = abs(factor) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    far[..., ia] = far[..., ib] = np.abs(ang) + 0 * x[..., ia]
    return y, mag, far


def weight(w, H, offset, d):
    if w is None:
        return np.ones((1, H, 1, d))
    return np.broadcast_to(t64(w) + offset, (H, d))[None, :, None]


def norm_rope(X, w, pos, freq, layout="half", factor=1.0, eps=1e-6, offset=0.0):
    """(y, bound): sums of squares and the inverse root are good to (d + 8) 2^-24, sines and cosines to 2^-22."""
    x, d = t64(X), X.shape[-1]
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight(w, X.shape[1], offset, d)
    y, mag, far = turn(n, pos, freq, layout, factor)
    bound = ((d + 16) * U + 2.0 ** -22 + 2.0 ** -51 * far) * mag
    return y, bound + HALF[X.dtype] * (np.abs(y) + bound)


def norm_rope_backward(X, dY, w, pos, freq, layout="half", factor=1.0, eps=1e-6, offset=0.0):
    """((dx, dw [H, d]), (bounds)): dw in fp32 before its own rounding and before heads are added up."""
    x, dy, d = t64(X), t64(dY), X.shape[-1]
    W = weight(w, X.shape[1], offset, d)
    rinv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn, mag, far = turn(dy, pos, freq, layout, factor, -1.0)
    edn = (8 * U + 2.0 ** -22 + 2.0 ** -51 * far) * mag
    rel = (d + 16) * U
    t, et = dn * W, (edn + 2 * U * np.abs(dn)) * np.abs(W)
    c = (t * x).mean(-1, keepdims=True) * rinv ** 2
    ec = ((et + (d + 4) * U * np.abs(t)) * np.abs(x)).mean(-1, keepdims=True) * rinv ** 2 + 2 * rel * np.abs(c)
    dx = rinv * (t - x * c)
    ex = rinv * (et + np.abs(x) * ec + (rel + 8 * U) * (np.abs(t) + np.abs(x * c)))
    n = X.shape[0] * X.shape[2]
    dw = (dn * x * rinv).sum((0, 2))
    ew = ((edn + (rel + (n + 8) * U) * np.abs(dn)) * np.abs(x) * rinv).sum((0, 2))
    return (dx, dw), (ex + HALF[X.dtype] * (np.abs(dx) + ex), ew)
