"""Plain numpy statements, in 64 bits, of the transformer-block operators:
layer norm by degree, the counter-based dropout mask, attention over a graph,
and their gradients.  Written from the definitions in include/eqtp.h; no code
is shared with the HIP side.  Also the error bounds the GPU tests use."""
import math

import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative


def degrees(lmax):
    return np.concatenate([[l] * (2 * l + 1) for l in range(lmax + 1)])


# ---- layer norm -------------------------------------------------------------

def norm(x, lmax, weight=None, bias=None, eps=1e-5):
    """(out, zhat, r [N, lmax+1], mean [N]) of x [N, C, K]."""
    x = np.asarray(x, dtype=np.float64)
    N, C, K = x.shape
    out, zhat, r = np.empty_like(x), np.empty_like(x), np.empty((N, lmax + 1))
    mean = x[:, :, 0].mean(axis=1)
    for l in range(lmax + 1):
        t = x[:, :, l * l:(l + 1) ** 2]
        if l == 0:
            t = t - mean[:, None, None]
        r[:, l] = 1.0 / np.sqrt((t * t).mean(axis=(1, 2)) + eps)
        zhat[:, :, l * l:(l + 1) ** 2] = t * r[:, l][:, None, None]
        w = np.ones(C) if weight is None else np.asarray(weight, dtype=np.float64)[l]
        o = zhat[:, :, l * l:(l + 1) ** 2] * w[None, :, None]
        if l == 0 and bias is not None:
            o = o + np.asarray(bias, dtype=np.float64)[None, :, None]
        out[:, :, l * l:(l + 1) ** 2] = o
    return out, zhat, r, mean


def norm_backward(x, lmax, g, weight=None, eps=1e-5):
    """(gx, gweight, gbias)."""
    g = np.asarray(g, dtype=np.float64)
    _, zhat, r, _ = norm(x, lmax, weight, None, eps)
    N, C, K = g.shape
    gx, gw = np.empty_like(g), np.empty((lmax + 1, C))
    for l in range(lmax + 1):
        s = slice(l * l, (l + 1) ** 2)
        w = np.ones(C) if weight is None else np.asarray(weight, dtype=np.float64)[l]
        a, zh = g[:, :, s] * w[None, :, None], zhat[:, :, s]
        t = a - zh * (a * zh).mean(axis=(1, 2), keepdims=True)
        if l == 0:
            t = t - a.mean(axis=(1, 2), keepdims=True)
        gx[:, :, s] = t * r[:, l][:, None, None]
        gw[l] = (g[:, :, s] * zh).sum(axis=(0, 2))
    return gx, gw, g[:, :, 0].sum(axis=0)


# Longest chain of additions behind a row's statistic: at most 64 terms in a
# row of a lane, then a tree over at most 1024 lanes; the squares, products,
# root and quotients around it add a few roundings.
CHAIN = 64 + 10 + 8


def norm_bound(x, lmax, weight, bias, eps, out_bf16):
    """Elementwise bound of |kernel - exact| for the forward pass: the mean is off by at most CHAIN u mean|x|,
    the mean square (of centred values) by CHAIN u relative and twice the mean's error, r by half of that."""
    x = np.asarray(x, dtype=np.float64)
    out, zhat, r, mean = norm(x, lmax, weight, bias, eps)
    w = np.ones((lmax + 1, x.shape[1])) if weight is None else np.abs(np.asarray(weight, dtype=np.float64))
    wk = w.T[:, degrees(lmax)][None]
    rk = r[:, degrees(lmax)][:, None, :]
    dmean = CHAIN * U32 * np.abs(x[:, :, 0]).mean(axis=1)[:, None, None] * (degrees(lmax) == 0)[None, None, :]
    # relative error of r: half of the mean square's; the mean's error enters it squared and by a vanishing sum
    drel = CHAIN * U32 + (dmean * rk) ** 2 + CHAIN * U32 * dmean * rk
    e = wk * (rk * dmean + np.abs(zhat) * drel + 4 * U32 * (np.abs(zhat) + rk * dmean)) + 2 * U32 * np.abs(out)
    return e + (U16 * (np.abs(out) + e) if out_bf16 else 0.0) + 1e-37


def norm_backward_bounds(x, lmax, g, weight, eps, x_bf16, extra=None):
    """Bounds for (gx (+ extra), gweight, gbias).  Each factor carries at most CHAIN u; three factors meet in the
    correction term.  The sums over nodes run over chains of at most N K / 64 + 512 terms."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(g, dtype=np.float64)
    _, zhat, r, _ = norm(x, lmax, weight, None, eps)
    N, C, K = x.shape
    dz = _zhat_error(x, lmax, zhat, r)
    gx = np.empty_like(g)
    gw = np.empty((lmax + 1, C))
    total, _, _ = norm_backward(x, lmax, g, weight, eps)
    chain = N * K / 64.0 + 512
    for l in range(lmax + 1):
        s = slice(l * l, (l + 1) ** 2)
        w = np.ones(C) if weight is None else np.abs(np.asarray(weight, dtype=np.float64)[l])
        a, zh = np.abs(g[:, :, s]) * w[None, :, None], np.abs(zhat[:, :, s])
        rl = r[:, l][:, None, None]
        mean_azh = (a * zh).mean(axis=(1, 2), keepdims=True)
        t = 3 * CHAIN * U32 * (a + zh * mean_azh) + dz[:, :, s] * mean_azh + zh * (a * dz[:, :, s]).mean(axis=(1, 2), keepdims=True)
        if l == 0:
            t = t + 3 * CHAIN * U32 * a.mean(axis=(1, 2), keepdims=True)
        gx[:, :, s] = t * rl
        gw[l] = (chain * U32 * np.abs(g[:, :, s]) * zh + np.abs(g[:, :, s]) * dz[:, :, s]).sum(axis=(0, 2))
    if extra is not None:
        total = total + np.asarray(extra, dtype=np.float64)
        gx = gx + 2 * U32 * np.abs(np.asarray(extra, dtype=np.float64))
    gx = gx + 2 * U32 * np.abs(total)
    if x_bf16:
        gx = gx + U16 * (np.abs(total) + gx)
    return gx + 1e-37, gw + 1e-37, chain * U32 * np.abs(g[:, :, 0]).sum(axis=0) + 1e-37


def _zhat_error(x, lmax, zhat, r):
    rk = r[:, degrees(lmax)][:, None, :]
    dmean = CHAIN * U32 * np.abs(x[:, :, 0]).mean(axis=1)[:, None, None] * (degrees(lmax) == 0)[None, None, :]
    drel = CHAIN * U32 + (dmean * rk) ** 2 + CHAIN * U32 * dmean * rk
    return rk * dmean + np.abs(zhat) * drel + 4 * U32 * (np.abs(zhat) + rk * dmean)


# ---- dropout ----------------------------------------------------------------

def philox(counter, key):
    """Ten rounds of Philox 4x32 on one counter (four words) under one key (two words)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(seed, offset, N, C, p):
    """bool [N, C]: channel number j = n C + c is kept if word j % 4 of block j / 4 is at least floor(p 2^32)."""
    if p == 0.0:
        return np.ones((N, C), dtype=bool)
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    words = []
    for b in range((N * C + 3) // 4):
        words += philox((b & 0xFFFFFFFF, b >> 32, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    return np.array(words[:N * C], dtype=np.uint64).reshape(N, C) >= np.uint64(int(p * 2.0 ** 32))


def dropout(x, keep, p, residual=None):
    x = np.asarray(x, dtype=np.float64)
    scale = np.float64(np.float32(1.0 / (1.0 - p)))  # the factor as the library holds it
    out = np.where(keep[:, :, None], x * scale, 0.0)
    return out if residual is None else out + np.asarray(residual, dtype=np.float64)


# ---- attention --------------------------------------------------------------

def attention(q, k, v, src, row_ptr, heads, scale, bias=None):
    """(out [N, C, K], w [E, heads], lse [N, heads], s [E, heads]); q [N, C, K], k, v [M, Ck, K]."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    N = q.shape[0]
    D = q.shape[1] * q.shape[2] // heads
    G = k.shape[1] * k.shape[2] // D
    qh, kh, vh = q.reshape(N, heads, D), k.reshape(-1, G, D), v.reshape(-1, G, D)
    E = len(src)
    out, w = np.zeros((N, heads, D)), np.zeros((E, heads))
    lse, logits = np.full((N, heads), -np.inf), np.full((E, heads), -np.inf)
    for n in range(N):
        for h in range(heads):
            e = np.arange(row_ptr[n], row_ptr[n + 1])
            if bias is not None:
                e = e[np.asarray(bias)[e, h] != -np.inf]
            if len(e) == 0:
                continue
            s = scale * (kh[src[e], h * G // heads] @ qh[n, h]) + (np.asarray(bias, dtype=np.float64)[e, h] if bias is not None else 0.0)
            top = s.max()
            p = np.exp(s - top)
            logits[e, h], w[e, h] = s, p / p.sum()
            lse[n, h] = top + math.log(p.sum())
            out[n, h] = w[e, h] @ vh[src[e], h * G // heads]
    return out.reshape(q.shape), w, lse, logits


def attention_backward(q, k, v, src, row_ptr, heads, scale, g, bias=None):
    """(gq, gk, gv, gbias)."""
    out, w, _, _ = attention(q, k, v, src, row_ptr, heads, scale, bias)
    q, k, v, g = (np.asarray(t, dtype=np.float64) for t in (q, k, v, g))
    N = q.shape[0]
    D = q.shape[1] * q.shape[2] // heads
    G = k.shape[1] * k.shape[2] // D
    qh, gh, oh, kh, vh = (t.reshape(t.shape[0], -1, D) for t in (q, g, out, k, v))
    gq, gk, gv, u = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(vh), np.zeros_like(w)
    for n in range(N):
        for h in range(heads):
            t = gh[n, h] @ oh[n, h]
            for e in range(row_ptr[n], row_ptr[n + 1]):
                if w[e, h] == 0.0:
                    continue
                m, j = src[e], h * G // heads
                u[e, h] = w[e, h] * (gh[n, h] @ vh[m, j] - t)
                gq[n, h] += scale * u[e, h] * kh[m, j]
                gk[m, j] += scale * u[e, h] * qh[n, h]
                gv[m, j] += w[e, h] * gh[n, h]
    return gq.reshape(q.shape), gk.reshape(k.shape), gv.reshape(v.shape), u


def attention_bounds(q, k, v, src, row_ptr, heads, scale, g, bias, half_step):
    """Elementwise bounds of |kernel - exact| for (out, lse, gq, gk, gv, gbias), from above, by running absolute
    values through the same formulas.  half_step: of the outputs' type.

    A dot product of D terms is off by at most (D / 16 + 16) u of the sum of its terms' sizes (a lane adds at most
    D / 16 of them; trees follow), a logit by that times scale and one rounding of |s| and of the bias; exp turns an absolute error of
    its argument into a relative one and adds its own 4 u (and 2 u |argument|: the hardware's exponential is of
    base 2, and its argument is rounded).  Sums over a row or a source of n edges are off by at most (n + 16) u."""
    q, k, v, g = (np.asarray(t, dtype=np.float64) for t in (q, k, v, g))
    out, w, lse, s = attention(q, k, v, src, row_ptr, heads, scale, bias)
    N = q.shape[0]
    D = q.shape[1] * q.shape[2] // heads
    G = k.shape[1] * k.shape[2] // D
    u = U32
    qh, gh, oh, kh, vh = (np.abs(t.reshape(t.shape[0], -1, D)) for t in (q, g, out, k, v))
    sg, so, sv = (t.reshape(t.shape[0], -1, D) for t in (g, out, v))
    bo, bl = np.zeros_like(oh), np.zeros_like(lse)
    bq, bk, bv, bb = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(vh), np.zeros_like(w)
    cd = (D / 16 + 16) * u
    sources = np.bincount(src, minlength=k.shape[0]) * (heads // G)
    for n in range(N):
        for h in range(heads):
            e = np.arange(row_ptr[n], row_ptr[n + 1])
            e = e[w[e, h] > 0] if len(e) else e
            live = np.arange(row_ptr[n], row_ptr[n + 1])
            if len(e) == 0:
                continue
            j, m = h * G // heads, src[e]
            cn = (len(live) + 16) * u
            size = abs(scale) * (kh[m, j] @ qh[n, h])
            ds = cd * size + 2 * u * np.abs(s[e, h]) + (u * np.abs(np.asarray(bias, dtype=np.float64)[e, h]) if bias is not None else 0.0)
            top = s[e, h].max()
            dw = ds + 4 * u + 2 * u * np.abs(s[e, h] - top)       # relative, of the unnormalised weight
            dsum = (w[e, h] * dw).sum() + cn
            rel = dw + dsum + 4 * u + ds.max()
            bl[n, h] = dsum + 4 * u + 4 * u * abs(lse[n, h]) + 2 * u * abs(top)
            # backward: w again from lse
            relb = ds + bl[n, h] + 4 * u + 2 * u * np.abs(s[e, h] - lse[n, h])
            terms = w[e, h][:, None] * vh[m, j]
            bo[n, h] = (terms * (rel + cn + 2 * u)[:, None]).sum(axis=0)
            bo[n, h] += half_step * (oh[n, h] + bo[n, h])
            dv = vh[m, j] @ gh[n, h]
            a = np.abs(sv[m, j] @ sg[n, h])
            t = abs(sg[n, h] @ so[n, h])
            dt = (w[e, h] * (cd * dv + (relb + cn) * a)).sum()
            along = np.abs(sv[m, j] @ sg[n, h] - sg[n, h] @ so[n, h])
            eu = w[e, h] * (cd * dv + dt + 2 * u * along + relb * along)
            bb[e, h] = eu + u * w[e, h] * along
            # sum u k as sum w a k - t sum w k: both sums round
            bq[n, h] = abs(scale) * (eu[:, None] * kh[m, j] + (w[e, h] * (a + t) * (cn + 4 * u))[:, None] * kh[m, j]).sum(axis=0)
            for i, ei in enumerate(e):
                cs = (sources[src[ei]] + 16) * u
                bk[src[ei], j] += abs(scale) * (eu[i] + w[ei, h] * along[i] * (cs + 4 * u)) * qh[n, h]
                bv[src[ei], j] += w[ei, h] * (relb[i] + cs + 4 * u) * gh[n, h]
    want = attention_backward(q, k, v, src, row_ptr, heads, scale, g, bias)
    res = [bo.reshape(q.shape), bl]
    for b, t in zip((bq, bk, bv), want):
        b = b.reshape(t.shape)
        res.append(b + half_step * (np.abs(t) + b))
    res.append(bb)
    return [b + 1e-37 for b in res]
