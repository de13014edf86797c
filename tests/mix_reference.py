"""Plain numpy statements, in 64 bits, of the distance bias, the norm and
rotation of queries and keys, routing, and the experts' per-degree linears, with
their gradients.  Written from the definitions in include/eqtp.h; no code is
shared with the HIP side.  Also the error bounds the GPU tests use (u: half a
step of fp32, relative)."""
import numpy as np

from block_reference import U16, U32, degrees

u = U32


# ---- distance bias ----------------------------------------------------------

def buckets(vec, bounds, r_cut=0.0):
    """(bucket, live, nan) of each edge."""
    r2 = (np.asarray(vec, dtype=np.float64) ** 2).sum(1)
    b = np.asarray(bounds, dtype=np.float64)
    b2 = np.where(b < 0, -1.0, b * b)
    with np.errstate(invalid="ignore"):
        bucket = (r2[:, None] >= b2[None, :]).sum(1)
        far = r2 >= float(r_cut) ** 2 if r_cut else np.zeros(len(r2), bool)
    return bucket, ~far & ~np.isnan(r2), np.isnan(r2)


def distance_bias(vec, bounds, table, r_cut=0.0):
    bucket, live, bad = buckets(vec, bounds, r_cut)
    out = np.where(live[:, None], np.asarray(table)[bucket], -np.inf)
    out[bad] = np.nan
    return out


def distance_bias_backward(vec, bounds, g, B, r_cut=0.0):
    """(grad_table, bound): a lane adds at most all of a bucket's edges one after the other, the rest is in 64 bits."""
    bucket, live, _ = buckets(vec, bounds, r_cut)
    out, size, n = np.zeros((B, g.shape[1])), np.zeros((B, g.shape[1])), np.zeros(B)
    g = np.where(live[:, None], np.asarray(g, dtype=np.float64), 0.0)
    for b in range(B):
        rows = g[live & (bucket == b)]
        out[b], size[b], n[b] = rows.sum(0), np.abs(rows).sum(0), len(rows)
    return out, u * (n[:, None] + 3) * size


# ---- queries and keys -------------------------------------------------------

def head_norm(x, heads, lmax, weight=None, pos=None, freq=None, eps=1e-5):
    """dict of the forward's parts, rows reshaped to [N, heads, w, K]."""
    x = np.asarray(x, dtype=np.float64)
    N, C, K = x.shape
    w = C // heads
    x = x.reshape(N, heads, w, K)
    r = np.empty((N, heads, lmax + 1))
    for l in range(lmax + 1):
        r[..., l] = 1.0 / np.sqrt((x[..., l * l:(l + 1) ** 2] ** 2).mean(axis=(2, 3)) + eps)
    deg = degrees(lmax)
    wt = np.ones((lmax + 1, w)) if weight is None else np.asarray(weight, dtype=np.float64)
    wt = wt.T[:, deg]  # [w, K]
    rr = r[..., deg][:, :, None, :]
    y = x * rr * wt
    c, s = np.ones((N, w)), np.zeros((N, w))
    half = w // 2
    R = 0
    if freq is not None:
        f = np.asarray(freq, dtype=np.float64)
        R = f.shape[1]
        th = np.asarray(pos, dtype=np.float64) @ f
        c[:, :R], s[:, :R] = np.cos(th), np.sin(th)
        c[:, half:half + R], s[:, half:half + R] = np.cos(th), np.sin(th)
    c, s = c[:, None, :, None], s[:, None, :, None]
    other = lambda t: np.concatenate((-t[:, :, half:half + R], np.zeros_like(t[:, :, R:half]), t[:, :, :R],  # noqa: E731
                                      np.zeros_like(t[:, :, half + R:])), 2) if R else np.zeros_like(t)
    return dict(x=x, r=rr, wt=wt, y=y, c=c, s=s, other=other, out=y * c + other(y) * s, R=R, half=half, deg=deg,
                freq=None if freq is None else f)


def head_norm_bounds(p, shape, half_step):
    """Of the output.  A sum of squares takes at most 22 additions (12 of a thread's own, 4 of its slots, 6 over the
    lanes): 22 u of it, 11 u of its root, with the mean, eps and the hardware's root 16 u of r, two products 18 u of y;
    cosine and sine are off by 6 u (the fraction of a turn 1.6 u, the functions 2 steps), the sum of two products by 2 u."""
    size = np.abs(p["y"]) + np.abs(p["other"](p["y"]))
    return (28 * u * size + half_step * np.abs(p["out"])).reshape(shape)


def head_norm_backward(x, g, heads, lmax, weight=None, pos=None, freq=None, eps=1e-5, half_step=u):
    """(gx, gweight, gpos), and their bounds."""
    p = head_norm(x, heads, lmax, weight, pos, freq, eps)
    N, H, w, K = p["x"].shape
    g = np.asarray(g, dtype=np.float64).reshape(p["x"].shape)
    t = g * p["c"] - p["other"](g) * p["s"]          # turned back
    G = np.abs(g) + np.abs(p["other"](g))
    a, xhat = t * p["wt"], p["x"] * p["r"]
    A, X = G * np.abs(p["wt"]), np.abs(p["x"])
    mean, size = np.empty((N, H, lmax + 1)), np.empty((N, H, lmax + 1))
    for l in range(lmax + 1):
        m = slice(l * l, (l + 1) ** 2)
        mean[..., l] = (a[..., m] * xhat[..., m]).mean(axis=(2, 3))
        size[..., l] = (A[..., m] * X[..., m]).mean(axis=(2, 3))
    mean, size = (v[..., p["deg"]][:, :, None, :] for v in (mean, size))
    gx = p["r"] * (a - xhat * mean)
    # a is off by 9 u, r by 16; the mean of a x by 33 (8 of a, 22 + 3 of the sum), beside three more r's and products
    bx = p["r"] * (30 * u * A + X * p["r"] ** 2 * 90 * u * size) + half_step * np.abs(gx)
    gw, bw = np.empty((lmax + 1, w)), np.empty((lmax + 1, w))
    for l in range(lmax + 1):
        m = slice(l * l, (l + 1) ** 2)
        gw[l] = (t[..., m] * xhat[..., m]).sum(axis=(0, 1, 3))
        # a thread adds its own rows in fp32 (all of them at most), the rest is in 64 bits
        bw[l] = u * (30 + N * H) * (G[..., m] * np.abs(xhat[..., m])).sum(axis=(0, 1, 3))
    gpos = bpos = None
    if freq is not None:
        R, half, f = p["R"], p["half"], p["freq"]
        y = p["y"]
        cross = (y[:, :, :R] * t[:, :, half:half + R] - y[:, :, half:half + R] * t[:, :, :R]).sum(axis=(1, 3))
        sz = (np.abs(y[:, :, :R]) * G[:, :, half:half + R] + np.abs(y[:, :, half:half + R]) * G[:, :, :R]).sum(axis=(1, 3))
        gpos, bpos = cross @ f.T, u * (18 + 8 + 4 + H * 6 + w + 8) * (sz @ np.abs(f).T)
    shape = np.asarray(x).shape
    return (gx.reshape(shape), gw, gpos), (bx.reshape(shape), bw, bpos)


# ---- routing ----------------------------------------------------------------

def _shares(t, sigmoid):
    """s / sum of s, from logarithms: also where every s is 0 in 64 bits."""
    ls = np.minimum(t, 0.0) - np.log1p(np.exp(-np.abs(t))) if sigmoid else t
    w = np.exp(ls - ls.max())
    return w / w.sum()


def route(t, k, sigmoid=False, bias=None, groups=1, top_groups=None, renormalise=True, scale=1.0):
    """(idx, weight, s) node by node."""
    t = np.asarray(t, dtype=np.float64)
    N, X = t.shape
    top_groups = groups if top_groups is None else top_groups
    idx, weight, S = np.full((N, k), -1), np.zeros((N, k)), np.zeros((N, X))
    for n in range(N):
        if np.isnan(t[n]).any():
            weight[n], S[n] = np.nan, np.nan
            continue
        if sigmoid:
            with np.errstate(over="ignore"):
                s = np.where(t[n] >= 0, 1.0 / (1.0 + np.exp(-np.abs(t[n]))), np.exp(-np.abs(t[n])) / (1.0 + np.exp(-np.abs(t[n]))))
        else:
            top = t[n].max()
            e = np.exp(t[n] - top) if np.isfinite(top) else np.zeros(X)
            s = e / e.sum() if e.sum() > 0 else e
        S[n] = s
        v = t[n].copy() if bias is None and groups == 1 else s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        v[(t[n] == -np.inf) | np.isnan(v)] = -np.inf
        if groups > 1:
            best = []
            for g in range(groups):
                two = sorted((x for x in v[g * (X // groups):(g + 1) * (X // groups)]), reverse=True)[:2]
                two = [x for x in two if x > -np.inf]
                best.append(sum(two) if two else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    v[g * (X // groups):(g + 1) * (X // groups)] = -np.inf
        for j, x in enumerate(sorted(range(X), key=lambda x: (-v[x], x))[:k]):
            if v[x] > -np.inf:
                idx[n, j] = x
        live = idx[n] >= 0
        taken = np.where(live, s[idx[n]], 0.0)
        if renormalise and live.any():
            taken[live] = _shares(t[n][idx[n][live]], sigmoid)
        weight[n] = taken * scale
    return idx, weight, S


def route_bound(t, k):
    """Relative, of a weight: exponentials of differences of logits (each rounded: u of its size), 2 steps of the
    function, a quotient and two products, a sum of k or all terms with errors like these."""
    t = np.where(np.isfinite(t), t, 0.0)
    return u * (16 + k + 8 + 4 * np.abs(t).max(1) + 2 * np.ptp(t, axis=1))


def route_backward(t, idx, g, sigmoid=False, renormalise=True, scale=1.0):
    """(grad_logits, size): size is what a relative error of the weights is of."""
    t = np.asarray(t, dtype=np.float64)
    out, size = np.zeros_like(t), np.zeros_like(t)
    for n in range(len(t)):
        live = idx[n] >= 0
        at = idx[n][live]
        if len(at) == 0:
            continue
        gg = g[n][live] * scale
        top = t[n].max() if np.isfinite(t[n].max()) else 0.0
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-t[n])) if sigmoid else np.exp(t[n] - top) / np.exp(t[n] - top).sum()
            rest = 1.0 / (1.0 + np.exp(t[n][at]))  # 1 - s, without its cancellation
        if renormalise:
            p = _shares(t[n][at], sigmoid)
            v = p * (gg - (gg * p).sum())
            z = p * (np.abs(gg) + (np.abs(gg) * p).sum())
            out[n, at] = v * rest if sigmoid else v
            size[n, at] = z * rest if sigmoid else z
        elif sigmoid:
            out[n, at] = gg * s[at] * rest
            size[n, at] = np.abs(out[n, at])
        else:
            dot, adot = (gg * s[at]).sum(), (np.abs(gg) * s[at]).sum()
            full, afull = np.zeros(t.shape[1]), np.zeros(t.shape[1])
            full[at], afull[at] = gg, np.abs(gg)
            out[n], size[n] = s * (full - dot), s * (afull + adot)
    return out, size


# ---- experts ----------------------------------------------------------------

def expert(h, W, idx, lmax, weight=None):
    """(out, sum of |terms|)."""
    h, W = np.asarray(h, dtype=np.float64), np.asarray(W, dtype=np.float64)
    N, C, K = h.shape
    out, size = np.zeros_like(h), np.zeros_like(h)
    deg = degrees(lmax)
    for n in range(N):
        for j, e in enumerate(idx[n]):
            if 0 <= e < len(W):
                w = 1.0 if weight is None else float(weight[n, j])
                for m in range(K):
                    out[n, :, m] += w * (W[e, deg[m]] @ h[n, :, m])
                    size[n, :, m] += abs(w) * (np.abs(W[e, deg[m]]) @ np.abs(h[n, :, m]))
    return out, size


def expert_bound(out, size, C, k, half_step):
    """C products added in fp32, the gate's product and k additions; the matrix cores' sums may cut instead of round."""
    return 2 * u * (C + k + 4) * size + half_step * np.abs(out)


def expert_backward(h, W, idx, g, lmax, weight=None, bf16=False):
    """(gh, gW, gweight) and their bounds."""
    h, W, g = (np.asarray(t, dtype=np.float64) for t in (h, W, g))
    N, C, K = h.shape
    k = idx.shape[1]
    gh, gsize = expert(g, W.transpose(0, 1, 3, 2), idx, lmax, weight)
    bh = expert_bound(gh, gsize, C, k, U16 if bf16 else u)
    deg = degrees(lmax)
    gW, sW, nW = np.zeros_like(W), np.zeros_like(W), np.zeros(len(W))
    gw, sw = np.zeros((N, k)), np.zeros((N, k))
    for n in range(N):
        for j, e in enumerate(idx[n]):
            if not 0 <= e < len(W):
                continue
            w = 1.0 if weight is None else float(weight[n, j])
            nW[e] += 1
            for m in range(K):
                gW[e, deg[m]] += w * np.outer(g[n, :, m], h[n, :, m])
                sW[e, deg[m]] += np.abs(w * np.outer(g[n, :, m], h[n, :, m]))
                gw[n, j] += g[n, :, m] @ W[e, deg[m]] @ h[n, :, m]
                sw[n, j] += np.abs(g[n, :, m]) @ np.abs(W[e, deg[m]]) @ np.abs(h[n, :, m])
    terms = nW[:, None, None, None] * (2 * lmax + 1)
    bW = (2 * u * (terms + 4) + (U16 * U16 if bf16 and weight is not None else 0.0)) * sW
    # C products in fp32, then K C / 16 terms a lane (16 K at most), 16 lanes' and 8 waves' sums
    return (gh, gW, gw), (bh, bW, 2 * u * (C + 16 * K + 16) * sw)
