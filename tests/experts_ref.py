"""Plain 64-bit forms of the expert-layer operators (include/sparse_ffn_experts.h) in numpy,
for the GPU tests. They share nothing with the library."""
import numpy as np


def route(l, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """Token by token, slot by slot: idx [T, k] and weights [T, k] in 64 bits."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    per = E // groups
    idx = np.full((T, k), -1, np.int64)
    wts = np.zeros((T, k))
    for t in range(T):
        on = l[t] > -np.inf  # not NaN, not minus infinity
        s = np.zeros(E)
        if on.any():
            with np.errstate(over="ignore", invalid="ignore"):
                if score == "softmax":
                    m = l[t][on].max()
                    s[on] = np.where(l[t][on] == m, 1.0, np.exp(l[t][on] - m))
                    s /= s.sum()
                else:
                    s[on] = 1.0 / (1.0 + np.exp(-l[t][on]))
        c = l[t].copy() if bias is None else s + np.asarray(bias, np.float64)
        ok = on & ~np.isnan(c) & (c > -np.inf)
        if groups > 1:
            worth = []
            for g in range(groups):
                mem = [e for e in range(g * per, (g + 1) * per) if ok[e]]
                v = s if bias is None and group_top == 2 else c
                best = sorted((v[e] for e in mem), reverse=True)[:group_top]
                worth.append(sum(best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            ok &= np.isin(np.arange(E) // per, kept)
        order = sorted((e for e in range(E) if ok[e]), key=lambda e: (-c[e], e))[:k]
        idx[t, :len(order)] = order
        w = s[order]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        wts[t, :len(order)] = w * scale
    return idx, wts


def quantize(x):
    """Rows of numbers -> (q, s): s = max|x| times the 32-bit float 1 / 127, rounded to
    32 bits, q the whole numbers nearest to x / s."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(axis=1)
    with np.errstate(all="ignore"):
        s = (a.astype(np.float32) * (np.float32(1) / np.float32(127))).astype(np.float64)
        s[a < 2.0 ** -100] = 0.0
        bad = ~np.isfinite(a)
        s[bad] = np.nan
        q = np.where((s > 0)[:, None], np.rint(x / s[:, None]), 0.0)
    return q, s


def matmul(q, s, w, ws, bias=None):
    """(y, magnitude): y in 64 bits and |product| + |bias| for the error bound."""
    p = (np.asarray(q, np.float64) @ np.asarray(w, np.float64).T) * np.asarray(s, np.float64)[:, None]
    p = p * np.asarray(ws, np.float64)
    b = 0.0 if bias is None else np.asarray(bias, np.float64)
    return p + b, np.abs(p) + np.abs(b)


def experts(x, idx, weights, wa, sa, wd, sd, b_act=None):
    """(y, magnitude): y in 64 bits and the sum of |weight * product| for the error bound."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    E = wa.shape[0]
    q, s = quantize(x)
    y, mag = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for e, w in zip(idx[t], weights[t]):
            if e < 0 or e >= E:
                continue
            a = (wa[e].astype(np.float64) @ q[t]) * (s[t] * sa[e].astype(np.float64))
            g, u = (a[:, 0], a[:, 1]) if wa.ndim == 4 else (a, 1.0)
            if b_act is not None:
                g = g + b_act[e].astype(np.float64)
            h = np.where(g < 0, 0.0, g) * u
            with np.errstate(over="ignore"):
                h = h.astype(np.float32).astype(np.float64)
            hq, hs = quantize(h[None])
            p = (wd[e].astype(np.float64) @ hq[0]) * hs[0] * sd[e].astype(np.float64)
            y[t] += float(w) * p
            mag[t] += abs(float(w)) * np.abs(p)
    return y, mag
