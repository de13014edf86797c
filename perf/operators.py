"""Cases of the transformer operators around the convolution: layer norm,
counter-based dropout (alone, and fused with the residual sum and the norm)
and attention over the graph, forward and backward.

Features are [N, C, K] with K = (lmax+1)^2 components per channel, as
everywhere in this package; K = 1 (lmax 0) is the ordinary layout of rows of
width C.  ``run`` evaluates a case in elementary torch operations (``own``
false) or through the package's entry points (``own`` true); ``exact`` gives
the same values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # the smallest call: one norm of a small molecule's features (64 atoms, 8 channels, lmax 2)
        dict(name="norm_tiny", op="norm", N=64, C=8, lmax=2, x="f32", out="f32", train=False),
        # a training step's norm on a batch of 1000 atoms, 32 channels, lmax 3
        dict(name="norm_typical_train", op="norm", N=1000, C=32, lmax=3, x="f32", out="f32", train=True),
        # inference on a 10k-atom cell: fp32 features normalised into the bf16 operand of the channel linear
        dict(name="norm_mid_to_bf16", op="norm", N=10007, C=64, lmax=3, x="f32", out="bf16", train=False),
        # the 64-wide hidden layer of the radial network, one row for each edge of the 10k-atom cell, trained
        dict(name="norm_edges_train", op="norm", N=266116, C=64, lmax=0, x="bf16", out="bf16", train=True),
        # dropout with its residual sum on a batch of 1000 atoms (latency)
        dict(name="drop_typical", op="drop", N=1000, C=32, lmax=3, x="f32", p=0.1, residual=True, train=False),
        # dropout on the radial network's hidden layer, values and gradients
        dict(name="drop_edges_train", op="drop", N=266116, C=64, lmax=0, x="bf16", p=0.2, residual=False, train=True),
        # an odd width and degree: 33 channels at lmax 4, fused residual, dropout and norm, trained
        dict(name="addnorm_odd_train", op="addnorm", N=5003, C=33, lmax=4, x="f32", out="f32", p=0.1, train=True),
        # the residual stream of a 100k-atom cell, 32 channels, lmax 3, trained
        dict(name="addnorm_large_train", op="addnorm", N=100000, C=32, lmax=3, x="f32", out="f32", p=0.1, train=True),
        # attention over a small molecule's graph (latency)
        dict(name="attn_tiny", op="attn", N=64, M=64, E=1094, C=8, lmax=2, heads=2, kv_heads=2, x="f32", bias=True,
             pool=False, train=False),
        # a training step over the 10k-atom cell's neighbour graph
        dict(name="attn_mid_train", op="attn", N=10000, M=10000, E=266116, C=64, lmax=3, heads=4, kv_heads=4, x="f32",
             bias=True, pool=False, train=True),
        # inference over the 100k-atom cell's graph: bf16 features, two heads to each key and value head
        dict(name="attn_large_bf16", op="attn", N=100000, M=100000, E=5239100, C=32, lmax=3, heads=4, kv_heads=2,
             x="bf16", bias=True, pool=False, train=False),
        # readout: 7 graphs, one query each, over the invariant features of all their atoms
        dict(name="attn_readout", op="attn", N=7, M=50000, E=50000, C=128, lmax=0, heads=8, kv_heads=8, x="f32",
             bias=False, pool=True, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "drop", "addnorm", "attn", "attn"])
    x = rng.choice(["f32", "bf16"])
    train = rng.random() < 0.5
    if op != "attn":
        lmax = rng.choice([0, 0, 1, 2, 3, 4, 5, 6])
        K = (lmax + 1) ** 2
        C = _log(rng, 8, 4096) if lmax == 0 else _log(rng, 4, 128)
        N = _log(rng, 16, max(16, min(300000, 40_000_000 // (C * K))))
        c = dict(op=op, N=N, C=C, lmax=lmax, x=x, train=train)
        if op != "drop":
            c["out"] = rng.choice([x, "bf16", "f32"])
        if op != "norm":
            c["p"] = rng.choice([0.05, 0.1, 0.2, 0.5])
        if op == "drop":
            c["residual"] = rng.random() < 0.5
        return c
    lmax = rng.choice([0, 1, 2, 3, 3, 4])
    K = (lmax + 1) ** 2
    kv_heads = rng.choice([1, 2, 4])
    heads = kv_heads * rng.choice([1, 1, 2])
    width = _log(rng, 1, max(1, min(32, 512 // K, 128 // heads)))  # channels of a head
    C = heads * width
    pool = rng.random() < 0.25
    most = min(3_000_000, 800_000_000 // (C * K))
    if pool:
        N, E = _log(rng, 1, 64), _log(rng, 300, min(most, 200000))
        M = E
    else:
        N = _log(rng, 32, 50000)
        M = N if rng.random() < 0.7 else _log(rng, 32, 50000)
        E = min(most, int(N * rng.uniform(1.5, 60)))
    return dict(op="attn", N=N, M=M, E=E, C=C, lmax=lmax, heads=heads, kv_heads=kv_heads, x=x,
                bias=rng.random() < 0.7, pool=pool, train=train)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    N, C, lmax = case["N"], case["C"], case["lmax"]
    K = (lmax + 1) ** 2
    dt = DTYPES[case["x"]]
    st = {"case": case}
    if case["op"] != "attn":
        degree = _degrees(lmax, dev)
        shift = (degree == 0).float() * 0.5  # scalars are not centred, and higher degrees are smaller
        spread = 1.0 / (1.0 + degree.float())
        st["x"] = (normal(N, C, K) * spread + shift).to(dt)
        # the counter-based generator's state: seed and offset
        st["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device=dev)
        if case["op"] == "addnorm" or case.get("residual"):
            st["residual"] = (normal(N, C, K) * spread + shift).to(dt)
        if case["op"] != "drop":
            st["weight"] = 1.0 + 0.2 * normal(lmax + 1, C)
            st["bias"] = 0.2 * normal(C)
        if case["train"]:
            st["grad_out"] = normal(N, C, K).to(DTYPES[case.get("out", case["x"])])
            if case["op"] == "addnorm":
                st["grad_total"] = normal(N, C, K).to(dt)
        return st
    M, E, H = case["M"], case["E"], case["heads"]
    Ckv = C // H * case["kv_heads"]
    st["q"] = normal(N, C, K).to(dt)
    st["k"] = normal(M, Ckv, K).to(dt)
    st["v"] = normal(M, Ckv, K).to(dt)
    # the graph: edges sorted by row; a fiftieth of the rows has none; sources unrelated to rows, or, in a
    # readout, each item in one row
    dst = torch.sort(torch.randint(0, N - N // 50, (E,), generator=g, device=dev))[0]
    src = torch.arange(E, device=dev) if case["pool"] else torch.randint(0, M, (E,), generator=g, device=dev)
    ptr = lambda keys, n: torch.searchsorted(keys, torch.arange(n + 1, device=dev)).to(torch.int32)  # noqa: E731
    st["row_ptr"], st["src"] = ptr(dst, N), src.to(torch.int32)
    st["bias"] = None
    if case["bias"]:
        # distance terms; edges beyond the cut-off are masked, in some rows all of them
        cut = (torch.rand(E, generator=g, device=dev) < 0.05) | (dst % 97 == 5)
        st["bias"] = (0.5 * normal(E, H)).masked_fill(cut[:, None], -math.inf)
    if case["train"]:
        # the same edges grouped by source: a program keeps this for as long as it keeps the graph
        key, perm = torch.sort(src, stable=True)
        st["src_ptr"], st["perm"], st["dst_s"] = ptr(key, M), perm.to(torch.int32), dst[perm].to(torch.int32)
        st["grad_out"] = normal(N, C, K).to(dt)
    return st


def _degrees(lmax, dev):
    """Degree l of each of the (lmax+1)^2 components."""
    return torch.arange((lmax + 1) ** 2, device=dev).double().add(0.5).sqrt().long()


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "drop": _own_drop, "addnorm": _own_addnorm, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "drop": _plain_drop, "addnorm": _plain_addnorm, "attn": _plain_attn}[op](state)


def _code(name):
    import spherical_harmonic_cg_amd as eq

    return eq.EQTP_BF16 if name == "bf16" else eq.EQTP_F32


def _own_norm(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    if not c["train"]:
        return eq.eqtp_layer_norm(st["x"], c["lmax"], st["weight"], st["bias"], eps=EPS, out_dtype=_code(c["out"]))
    stats = torch.empty((c["N"], c["lmax"] + 2), dtype=torch.float32, device="cuda")
    out = eq.eqtp_layer_norm(st["x"], c["lmax"], st["weight"], st["bias"], eps=EPS, out_dtype=_code(c["out"]),
                             stats=stats)
    gx, _, gw, gb = eq.eqtp_layer_norm_backward(st["x"], stats, st["grad_out"], c["lmax"], st["weight"])
    return out, gx, gw, gb


def _own_drop(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    out = eq.eqtp_dropout(st["x"], st["rng"], c["p"], c["lmax"], residual=st.get("residual"))
    if not c["train"]:
        return out
    return out, eq.eqtp_dropout(st["grad_out"], st["rng"], c["p"], c["lmax"])


def _own_addnorm(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    stats = torch.empty((c["N"], c["lmax"] + 2), dtype=torch.float32, device="cuda") if c["train"] else None
    out, total = eq.eqtp_dropout_add_norm(st["x"], st["residual"], st["rng"], c["p"], c["lmax"], st["weight"],
                                          st["bias"], eps=EPS, out_dtype=_code(c["out"]), stats=stats)
    if not c["train"]:
        return out, total
    gr, gx, gw, gb = eq.eqtp_layer_norm_backward(total, stats, st["grad_out"], c["lmax"], st["weight"],
                                                 grad_total=st["grad_total"], rng=st["rng"], p=c["p"])
    return out, total, gr, gx, gw, gb


def _own_attn(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    if not c["train"]:
        return eq.eqtp_attention(st["q"], st["k"], st["v"], st["src"], st["row_ptr"], c["lmax"], c["heads"],
                                 bias=st["bias"])
    lse = torch.empty((c["N"], c["heads"]), dtype=torch.float32, device="cuda")
    out = eq.eqtp_attention(st["q"], st["k"], st["v"], st["src"], st["row_ptr"], c["lmax"], c["heads"],
                            bias=st["bias"], lse=lse)
    gq, gk, gv, gb = eq.eqtp_attention_backward(st["q"], st["k"], st["v"], st["src"], st["row_ptr"], out, lse,
                                                st["grad_out"], st["src_ptr"], st["dst_s"], st["perm"], c["lmax"],
                                                c["heads"], bias=st["bias"])
    return (out, gq, gk, gv, gb) if c["bias"] else (out, gq, gk, gv)


def _keep(rng, rows, C, p):
    """Kept channels [rows, C, 1]: word j % 4 of the ten-round Philox 4x32 block j / 4 (j = row * C + channel)
    under key = seed and counter = (block, offset) is at least p 2^32 (Salmon, Moraes, Dror and Shaw, "Parallel
    random numbers: as easy as 1, 2, 3", 2011)."""
    low = 0xFFFFFFFF
    block = torch.arange((rows * C + 3) // 4, device=rng.device)
    a, b = block & low, block >> 32
    c, d = (rng[1] & low).expand_as(a), (rng[1] >> 32 & low).expand_as(a)
    k0, k1 = rng[0] & low, rng[0] >> 32 & low
    for _ in range(10):
        u, w = a * 0xD2511F53, c * 0xCD9E8D57  # 64-bit products, modulo 2^64
        a, b, c, d = (w >> 32 & low) ^ b ^ k0, w & low, (u >> 32 & low) ^ d ^ k1, u & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack((a, b, c, d), 1).reshape(-1)[: rows * C]
    return (words >= math.floor(p * 2.0 ** 32)).reshape(rows, C, 1)


def _per_degree(v, lmax):
    """Sums over the components of each degree: [..., K] -> [..., lmax+1]."""
    onehot = (_degrees(lmax, v.device)[:, None] == torch.arange(lmax + 1, device=v.device)).to(v.dtype)
    return v @ onehot


def _norm_parts(z, lmax):
    """Centred scalars beside the higher degrees, and 1 / sqrt(mean square + eps) per degree spread over components."""
    C, degree = z.shape[1], _degrees(lmax, z.device)
    scalar = (degree == 0).float()
    zc = z - z.mean(1, keepdim=True) * scalar
    count = C * (2 * torch.arange(lmax + 1, device=z.device) + 1)
    r = torch.rsqrt(_per_degree((zc * zc).sum(1), lmax) / count + EPS)  # [N, lmax+1]
    return zc, r[:, degree][:, None, :], scalar, degree, count


def _plain_norm_forward(z, weight, bias, lmax):
    zc, r, scalar, degree, _ = _norm_parts(z, lmax)
    return zc * r * weight.t()[:, degree] + bias[:, None] * scalar


def _plain_norm_backward(z, weight, g, lmax):
    zc, r, scalar, degree, count = _norm_parts(z, lmax)
    zhat = zc * r
    a = g * weight.t()[:, degree]
    along = (_per_degree((a * zhat).sum(1), lmax) / count)[:, degree][:, None, :]
    gz = r * (a - a.mean(1, keepdim=True) * scalar - zhat * along)
    return gz, _per_degree((g * zhat).sum(0), lmax).t().contiguous(), g[:, :, 0].sum(0)


def _plain_norm(st):
    c = st["case"]
    z = st["x"].float()
    out = _plain_norm_forward(z, st["weight"], st["bias"], c["lmax"]).to(DTYPES[c["out"]])
    if not c["train"]:
        return out
    gz, gw, gb = _plain_norm_backward(z, st["weight"], st["grad_out"].float(), c["lmax"])
    return out, gz.to(st["x"].dtype), gw, gb


def _plain_drop(st):
    c = st["case"]
    keep = _keep(st["rng"], c["N"], c["C"], c["p"])
    scale = 1.0 / (1.0 - c["p"])
    out = torch.where(keep, st["x"].float() * scale, 0.0)
    if "residual" in st:
        out = out + st["residual"].float()
    out = out.to(st["x"].dtype)
    if not c["train"]:
        return out
    return out, torch.where(keep, st["grad_out"].float() * scale, 0.0).to(out.dtype)


def _plain_addnorm(st):
    c = st["case"]
    dt = st["x"].dtype
    keep = _keep(st["rng"], c["N"], c["C"], c["p"])
    scale = 1.0 / (1.0 - c["p"])
    total = (st["residual"].float() + torch.where(keep, st["x"].float() * scale, 0.0)).to(dt)
    z = total.float()  # the norm is that of the sum as it is written
    out = _plain_norm_forward(z, st["weight"], st["bias"], c["lmax"]).to(DTYPES[c["out"]])
    if not c["train"]:
        return out, total
    gz, gw, gb = _plain_norm_backward(z, st["weight"], st["grad_out"].float(), c["lmax"])
    gz = gz + st["grad_total"].float()
    return out, total, gz.to(dt), torch.where(keep, gz * scale, 0.0).to(dt), gw, gb


def _sum_rows(values, at, n, count):
    """Sums of values [E, ...] into rows `at` of n; few long rows as differences of a running sum, in 64 bits."""
    if count > 64 * n:
        at, order = torch.sort(at, stable=True)
        ends = torch.searchsorted(at, torch.arange(n, device=at.device), right=True)
        upto = values.flatten(1)[order].t().double().cumsum(1)
        upto = torch.cat((torch.zeros_like(upto[:, :1]), upto), 1)[:, ends]
        return torch.diff(upto, dim=1, prepend=torch.zeros_like(upto[:, :1])).t().float().reshape((n,) + values.shape[1:])
    return torch.zeros((n,) + values.shape[1:], device=values.device).index_add_(0, at, values)


def _max_rows(values, at, n, count):
    """The largest of values [E, H] in each of n rows, or -inf."""
    if count > 64 * n:
        member = at == torch.arange(n, device=at.device)[:, None]
        return torch.where(member[:, :, None], values, -math.inf).amax(1)
    return torch.full((n, values.shape[1]), -math.inf, device=values.device).scatter_reduce_(
        0, at[:, None].expand_as(values), values, "amax")


def _plain_attn(st):
    c = st["case"]
    N, M, E, H, G = c["N"], c["M"], c["E"], c["heads"], c["kv_heads"]
    dt = st["q"].dtype
    D = c["C"] // H * (c["lmax"] + 1) ** 2
    scale = 1.0 / math.sqrt(D)
    q = st["q"].float().reshape(N, G, H // G, D)
    k, v = (st[n].float().reshape(M, G, 1, D) for n in "kv")
    src = st["src"].long()
    dst = torch.searchsorted(st["row_ptr"], torch.arange(E, dtype=torch.int32, device=src.device), right=True) - 1
    kg, vg = k[src], v[src]
    s = (q[dst] * kg).sum(-1).reshape(E, H) * scale
    if st["bias"] is not None:
        s = s + st["bias"]
    top = _max_rows(s, dst, N, E)
    w = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0)[dst])
    total = _sum_rows(w, dst, N, E)
    p = (w / torch.where(total > 0, total, 1.0)[dst]).reshape(E, G, H // G, 1)  # rows without edges: no terms
    o = _sum_rows(p * vg, dst, N, E)
    out = o.reshape(st["q"].shape).to(dt)
    if not c["train"]:
        return out
    go = st["grad_out"].float().reshape(N, G, H // G, D)
    gg = go[dst]
    along = (go * o).sum(-1, keepdim=True)
    ds = p * ((gg * vg).sum(-1, keepdim=True) - along[dst])
    gq = _sum_rows(ds * kg, dst, N, E) * scale
    gk = _sum_rows((ds * q[dst]).sum(2), src, M, E) * scale
    gv = _sum_rows((p * gg).sum(2), src, M, E)
    grads = (gq.reshape(st["q"].shape).to(dt), gk.reshape(st["k"].shape).to(dt), gv.reshape(st["v"].shape).to(dt))
    return (out,) + grads + ((ds.reshape(E, H),) if st["bias"] is not None else ())


# ---------------------------------------------------------------- 64 bits

def _mask64(rng, count, p):
    """The keep mask from a second statement of the generator (numpy, unsigned 64-bit words)."""
    seed, offset = (int(t) for t in rng.cpu())
    j = np.arange((count + 3) // 4, dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [j & low, j >> half, np.full_like(j, offset & 0xFFFFFFFF), np.full_like(j, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        h0, h1 = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(h1 >> half) ^ x[1] ^ np.uint64(key[0]), h1 & low, (h0 >> half) ^ x[3] ^ np.uint64(key[1]), h0 & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(x, axis=1).ravel()[:count]
    return torch.from_numpy(words >= np.uint64(int(p * 2 ** 32))).to(rng.device)


def _norm64(z, weight, bias, lmax):
    parts = []
    for l in range(lmax + 1):
        t = z[:, :, l * l:(l + 1) * (l + 1)]
        if l == 0:
            t = t - t.mean(dim=1, keepdim=True)
        t = t / (t.pow(2).mean(dim=(1, 2), keepdim=True) + EPS).sqrt() * weight[l][None, :, None]
        parts.append(t + bias[None, :, None] if l == 0 else t)
    return torch.cat(parts, dim=2)


def exact(case, seed):
    st = prepare(case, seed)
    wide = {n: t.double() for n, t in st.items() if torch.is_tensor(t) and t.is_floating_point()}
    with torch.enable_grad():
        if case["op"] == "attn":
            return _exact_attn(case, st, wide)
        return _exact_rows(case, st, wide)


def _exact_rows(case, st, wide):
    x, lmax, train = wide["x"], case["lmax"], case["train"]
    if case["op"] != "norm":
        keep = _mask64(st["rng"], case["N"] * case["C"], case["p"]).reshape(case["N"], case["C"], 1)
        factor = keep.double() / (1.0 - case["p"])
    if case["op"] == "drop":
        out = x * factor + (wide["residual"] if "residual" in wide else 0.0)
        return (out, wide["grad_out"] * factor) if train else out
    total = x
    if case["op"] == "addnorm":
        total = (wide["residual"] + x * factor).to(st["x"].dtype).double()
    leaves = [total.detach().requires_grad_(), wide["weight"].requires_grad_(), wide["bias"].requires_grad_()]
    out = _norm64(*leaves, lmax)
    if not train:
        return out.detach() if case["op"] == "norm" else (out.detach(), total)
    gz, gw, gb = torch.autograd.grad(out, leaves, wide["grad_out"])
    if case["op"] == "norm":
        return out.detach(), gz, gw, gb
    gz = gz + wide["grad_total"]
    return out.detach(), total, gz, gz * factor, gw, gb


def _exact_attn(case, st, wide):
    N, E, H, R = case["N"], case["E"], case["heads"], case["heads"] // case["kv_heads"]
    D = case["C"] // H * (case["lmax"] + 1) ** 2
    dev = st["q"].device
    src = st["src"].long()
    length = (st["row_ptr"][1:] - st["row_ptr"][:-1]).long()
    dst = torch.repeat_interleave(torch.arange(N, device=dev), length)
    leaves = [wide[n] for n in ("q", "k", "v")] + ([wide["bias"]] if case["bias"] else [])
    leaves = [t.requires_grad_(case["train"]) for t in leaves]
    q = leaves[0].reshape(N, H, D)
    k, v = (t.reshape(case["M"], H // R, D) for t in leaves[1:3])
    heads = []
    for h in range(H):
        s = (q[:, h][dst] * k[:, h // R][src]).sum(-1) / math.sqrt(D)
        if case["bias"]:
            s = s + leaves[3][:, h]
        live = s > -math.inf
        at, to, s = src[live], dst[live], s[live]
        e = torch.exp(s - s.detach().max()) if s.numel() else s
        z = torch.zeros(N, dtype=torch.float64, device=dev).index_add(0, to, e)
        heads.append(torch.zeros(N, D, dtype=torch.float64, device=dev)
                     .index_add(0, to, (e / z[to])[:, None] * v[:, h // R][at]))
    out = torch.stack(heads, 1).reshape(wide["q"].shape)
    if not case["train"]:
        return out
    grads = torch.autograd.grad(out, leaves, wide["grad_out"])
    return (out.detach(),) + tuple(grads)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    N, C, K = case["N"], case["C"], (case["lmax"] + 1) ** 2
    es = 2 if case["x"] == "bf16" else 4
    size, train = N * C * K, case["train"]
    if case["op"] == "attn":
        M, E, H = case["M"], case["E"], case["heads"]
        kv = M * (C // H) * case["kv_heads"] * K
        edges = 4 * E + 4 * (N + 1) + (4 * E * H if case["bias"] else 0)
        nbytes = es * (2 * size + 2 * kv) + edges
        flops = 4 * E * C * K
        if train:  # grad_out in; three gradients (and the bias's) out; the edges by source
            nbytes += es * (2 * size + 2 * kv) + 8 * E + 4 * (M + 1) + (4 * E * H if case["bias"] else 0)
            flops += 8 * E * C * K
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "drop":
        return {"bytes": size * es * (2 + bool(case["residual"]) + (2 if train else 0)),
                "flops": size * (1 + bool(case["residual"]) + bool(train))}
    eo = 2 if case["out"] == "bf16" else 4
    nbytes, flops = size * (es + eo), 8 * size
    if train:
        nbytes, flops = nbytes + size * (es + eo), flops + 14 * size
    if case["op"] == "addnorm":
        nbytes, flops = nbytes + 2 * size * es + (2 * size * es if train else 0), flops + 2 * size
    return {"bytes": nbytes, "flops": flops}
