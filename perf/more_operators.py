"""Cases of what stands before and behind the attention over the graph: the
learned bias by distance buckets that it adds to its logits, the norm of
queries and keys by head and degree with the rotation by position, and the
mixture of per-degree channel linears: the router and the experts' products,
forward and backward.

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
        # distance bias of the 1000-atom batch's 20 neighbours each, before one inference step (latency)
        dict(name="bias_typical", op="bias", E=20000, H=4, B=16, r_cut=4.0, train=False),
        # a training step over the 10k-atom cell's neighbour graph, an odd number of buckets
        dict(name="bias_mid_train", op="bias", E=266116, H=4, B=33, r_cut=4.0, train=True),
        # a training step over the 100k-atom cell's graph
        dict(name="bias_large_train", op="bias", E=5239100, H=8, B=64, r_cut=5.0, train=True),
        # queries and keys of a small molecule (latency)
        dict(name="qk_tiny", op="qk", N=64, M=64, C=8, lmax=2, heads=2, kv_heads=2, x="f32", axes=3, R=2, forces=False,
             train=False),
        # a training step on the 10k-atom cell, positions in space, gradients of the positions for forces
        dict(name="qk_mid_train", op="qk", N=10000, M=10000, C=64, lmax=3, heads=4, kv_heads=4, x="f32", axes=3, R=8,
             forces=True, train=True),
        # rows of invariants along a long chain (angles of far positions), four heads to each key head, trained
        dict(name="qk_chain_train_bf16", op="qk", N=100003, M=100003, C=128, lmax=0, heads=8, kv_heads=2, x="bf16",
             axes=1, R=8, forces=False, train=True),
        # inference on the 100k-atom cell: bf16 features, two heads to each key and value head
        dict(name="qk_large_bf16", op="qk", N=100000, M=100000, C=32, lmax=3, heads=4, kv_heads=2, x="bf16", axes=3,
             R=4, forces=False, train=False),
        # routing of a batch of 1000 atoms to 8 experts, two each (latency)
        dict(name="route_typical", op="route", N=1000, X=8, k=2, score="softmax", balance=False, groups=1, top_groups=1,
             renormalise=True, x="f32", train=False),
        # a training step's routing of 100k atoms: 64 experts in 8 groups, the best 4 groups, 6 experts each
        dict(name="route_large_train", op="route", N=100000, X=64, k=6, score="sigmoid", balance=True, groups=8,
             top_groups=4, renormalise=True, x="f32", train=True),
        # one node through two of eight experts (latency)
        dict(name="expert_single", op="expert", N=1, C=64, lmax=3, X=8, k=2, x="f32", gates=True, train=False),
        # the linear whose weights go by the atom's element: ten elements in the 10k-atom cell, trained
        dict(name="expert_elements_train", op="expert", N=10007, C=64, lmax=3, X=10, k=1, x="f32", gates=False,
             train=True),
        # a mixture of eight experts, two for each atom, on the 100k-atom cell's bf16 features, trained
        dict(name="expert_large_train_bf16", op="expert", N=100000, C=32, lmax=3, X=8, k=2, x="bf16", gates=True,
             train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["bias", "qk", "qk", "route", "expert", "expert"])
    train = rng.random() < 0.5
    if op == "bias":
        H = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        return dict(op=op, E=_log(rng, 100, 40_000_000 // max(8, H)), H=H, B=_log(rng, 2, 256),
                    r_cut=rng.choice([0.0, 3.5, 5.0]), train=train)
    x = rng.choice(["f32", "bf16"])
    if op == "qk":
        lmax = rng.choice([0, 0, 1, 2, 3, 3, 4, 6])
        K = (lmax + 1) ** 2
        kv_heads = rng.choice([1, 2, 4])
        heads = kv_heads * rng.choice([1, 1, 2, 8])
        width = _log(rng, 2, min(128, 1024 // K, 512 // heads))  # channels of a head
        axes = rng.choice([0, 1, 3]) if width % 2 == 0 else 0
        R = rng.choice([width // 2, max(1, width // 4)]) if axes else 0
        N = _log(rng, 1, max(1, min(100000, 50_000_000 // (heads * width * K))))
        M = N if rng.random() < 0.7 else _log(rng, 1, N)
        return dict(op=op, N=N, M=M, C=heads * width, lmax=lmax, heads=heads, kv_heads=kv_heads, x=x, axes=axes, R=R,
                    forces=bool(axes) and rng.random() < 0.4, train=train)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        X = groups * _log(rng, 2, 256 // groups if groups > 1 else 160)
        top_groups = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 8]), X // groups * top_groups)
        return dict(op=op, N=_log(rng, 1, 6_400_000 // X), X=X, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    balance=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                    renormalise=rng.random() < 0.7, x=x, train=train)
    C = rng.choice([8, 16, 32, 64, 64, 128])
    lmax = rng.choice([0, 1, 2, 3, 3, 4, 6])
    X = _log(rng, 2, 64)
    k = min(X, rng.choice([1, 1, 2, 2, 4]))
    N = _log(rng, 1, max(1, min(100000, 150_000_000 // (C * (lmax + 1) ** 2 * X))))
    return dict(op=op, N=N, C=C, lmax=lmax, X=X, k=k, x=x, gates=k > 1 or rng.random() < 0.4, train=train)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    uniform = lambda *shape: torch.rand(*shape, generator=g, device=dev)  # noqa: E731
    return {"case": case, **{"bias": _prepare_bias, "qk": _prepare_qk, "route": _prepare_route,
                             "expert": _prepare_expert}[case["op"]](case, normal, uniform, dev)}


def _prepare_bias(c, normal, uniform, dev):
    E, H, B = c["E"], c["H"], c["B"]
    # neighbours are uniform in the ball; the list is made with a skin, so some lie beyond the cut-off
    reach = (c["r_cut"] or 5.0) * 1.05
    away = normal(E, 3)
    vec = away / away.norm(dim=1, keepdim=True) * (reach * uniform(E, 1) ** (1.0 / 3.0))
    st = {"vec": vec, "bounds": torch.linspace(0.6, reach * 0.95, B - 1, device=dev), "table": 0.5 * normal(B, H)}
    if c["train"]:
        st["grad_bias"] = 0.1 * normal(E, H)
    return st


def _prepare_qk(c, normal, uniform, dev):
    N, M, H, lmax, R = c["N"], c["M"], c["heads"], c["lmax"], c["R"]
    K, d, dt = (lmax + 1) ** 2, c["C"] // H, DTYPES[c["x"]]
    Ck = d * c["kv_heads"]
    spread = 3.0 / (1.0 + _degrees(lmax, dev).float())  # higher degrees are smaller
    st = {"q": (normal(N, c["C"], K) * spread).to(dt), "k": (normal(M, Ck, K) * spread).to(dt),
          "wq": 1.0 + 0.2 * normal(lmax + 1, d), "wk": 1.0 + 0.2 * normal(lmax + 1, d),
          "pq": None, "pk": None, "freq": None}
    if c["axes"] == 3:  # atoms in a periodic cell, frequencies from its reciprocal lattice
        box = 10.0 * max(N, 64) ** (1.0 / 3.0) / 4.64
        st["pq"], st["pk"] = box * uniform(N, 3), box * uniform(M, 3)
        st["freq"] = (2.0 * math.pi / box) * torch.round(3.0 * normal(3, R))
    elif c["axes"] == 1:  # places along a chain
        st["pq"] = torch.arange(N, device=dev, dtype=torch.float32)[:, None]
        st["pk"] = torch.arange(M, device=dev, dtype=torch.float32)[:, None]
        st["freq"] = 10000.0 ** (-torch.arange(R, device=dev, dtype=torch.float32) / R)[None, :]
    if c["train"]:
        st["gq"], st["gk"] = normal(N, c["C"], K).to(dt), normal(M, Ck, K).to(dt)
    return st


def _prepare_route(c, normal, uniform, dev):
    st = {"logits": (1.5 * normal(c["N"], c["X"])).to(DTYPES[c["x"]]), "bias": None}
    if c["balance"]:
        st["bias"] = 0.1 * normal(c["X"])
    if c["train"]:
        st["grad_weight"] = normal(c["N"], c["k"])
    return st


def _prepare_expert(c, normal, uniform, dev):
    N, C, lmax, X, k = c["N"], c["C"], c["lmax"], c["X"], c["k"]
    K, dt = (lmax + 1) ** 2, DTYPES[c["x"]]
    # some experts (elements) are met more often than others; a node's experts differ
    liking = normal(1, X) + normal(N, X)
    idx = torch.topk(liking, k, dim=1)[1]
    st = {"h": normal(N, C, K).to(dt), "W": (normal(X, lmax + 1, C, C) / math.sqrt(C)).to(dt),
          "idx": idx.to(torch.int32).contiguous(), "weight": None, "plan": None}
    if c["gates"]:
        st["weight"] = torch.softmax(normal(N, k), 1)
    else:  # elements do not change: a program groups the atoms once
        key, perm = torch.sort(idx.reshape(-1), stable=True)
        ptr = torch.searchsorted(key, torch.arange(X + 1, device=dev)).to(torch.int32)
        st["plan"] = (perm.to(torch.int32), perm.to(torch.int32), ptr)
    if c["train"]:
        st["grad_out"] = normal(N, C, K).to(dt)
    return st


def _degrees(lmax, dev):
    """Degree l of each of the (lmax+1)^2 components."""
    return torch.arange((lmax + 1) ** 2, device=dev).double().add(0.5).sqrt().long()


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"bias": _own_bias, "qk": _own_qk, "route": _own_route, "expert": _own_expert}[op](state)
    return {"bias": _plain_bias, "qk": _plain_qk, "route": _plain_route, "expert": _plain_expert}[op](state)


def _own_bias(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    out = eq.eqtp_distance_bias(st["vec"], st["bounds"], st["table"], r_cut=c["r_cut"])
    if not c["train"]:
        return out
    return out, eq.eqtp_distance_bias_backward(st["vec"], st["bounds"], st["grad_bias"], r_cut=c["r_cut"])


def _own_qk(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    how = dict(weight_q=st["wq"], weight_k=st["wk"], pos_q=st["pq"], pos_k=st["pk"], freq=st["freq"], eps=EPS)
    out = eq.eqtp_qk_norm(st["q"], st["k"], c["lmax"], c["heads"], **how)
    if not c["train"]:
        return out
    grads = eq.eqtp_qk_norm_backward(st["q"], st["k"], st["gq"], st["gk"], c["lmax"], c["heads"],
                                     need_pos=c["forces"], **how)
    return out + (grads if c["forces"] else grads[:4])


def _own_route(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    how = dict(score=eq.EQTP_SCORE_SIGMOID if c["score"] == "sigmoid" else eq.EQTP_SCORE_SOFTMAX,
               renormalise=c["renormalise"], scale=1.5)
    idx, weight = eq.eqtp_route(st["logits"], c["k"], bias=st["bias"], groups=c["groups"], top_groups=c["top_groups"],
                                **how)
    if not c["train"]:
        return idx, weight
    return idx, weight, eq.eqtp_route_backward(st["logits"], idx, st["grad_weight"], **how)


def _own_expert(st):
    import spherical_harmonic_cg_amd as eq

    c = st["case"]
    plan = st["plan"] or eq.eqtp_expert_plan(st["idx"], c["X"])
    code = eq.EQTP_BF16 if c["x"] == "bf16" else eq.EQTP_F32
    out = eq.eqtp_expert_linear(st["h"], st["W"], st["idx"], c["lmax"], weight=st["weight"], plan=plan, out_dtype=code)
    if not c["train"]:
        return out
    gh, gW, gw = eq.eqtp_expert_linear_backward(st["h"], st["W"], st["idx"], st["grad_out"], c["lmax"],
                                                weight=st["weight"], plan=plan)
    return (out, gh, gW, gw) if c["gates"] else (out, gh, gW)


def _plain_bias(st):
    c = st["case"]
    r2 = st["vec"].double().square().sum(1)  # 64 bits: lengths next to a bound
    bucket = torch.searchsorted(st["bounds"].double().square(), r2, right=True)
    out = st["table"][bucket]
    far = (r2 >= c["r_cut"] ** 2)[:, None] if c["r_cut"] else None
    if far is not None:
        out = out.masked_fill(far, -math.inf)
    if not c["train"]:
        return out
    g = st["grad_bias"] if far is None else st["grad_bias"].masked_fill(far, 0.0)
    # long sums, in 64 bits: differences of a running sum over the edges in the order of their buckets
    bucket, order = torch.sort(bucket)
    ends = torch.searchsorted(bucket, torch.arange(c["B"], device=g.device), right=True)
    upto = torch.nn.functional.pad(g[order].t().double().cumsum(1), (1, 0))[:, ends]
    return out, torch.diff(upto, dim=1, prepend=torch.zeros_like(upto[:, :1])).t().float().contiguous()


def _per_degree(v, lmax):
    """Sums over the components of each degree: [..., K] -> [..., lmax+1]."""
    onehot = (_degrees(lmax, v.device)[:, None] == torch.arange(lmax + 1, device=v.device)).to(v.dtype)
    return v @ onehot


def _turns(pos, freq):
    """cos and sin [rows, 1, R, 1]; angles in 64 bits."""
    angle = (pos.double() @ freq.double())[:, None, :, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(y, cos, sin):
    half, R = y.shape[2] // 2, cos.shape[2]
    a, b = y[:, :, :R], y[:, :, half:half + R]
    return torch.cat((a * cos - b * sin, y[:, :, R:half], a * sin + b * cos, y[:, :, half + R:]), 2)


def _plain_head_norm(x, w, pos, freq, heads, lmax, g=None, forces=False):
    rows, C, K = x.shape
    d, degree = C // heads, _degrees(lmax, x.device)
    z = x.float().reshape(rows, heads, d, K)
    count = d * (2 * torch.arange(lmax + 1, device=x.device) + 1)
    r = torch.rsqrt(_per_degree((z * z).sum(2), lmax) / count + EPS)[..., degree][:, :, None, :]
    zhat, wide = z * r, w.t()[:, degree]
    y = zhat * wide
    if pos is not None:
        cos, sin = _turns(pos, freq)
        y = _turn(y, cos, sin)
    out = y.reshape(x.shape).to(x.dtype)
    if g is None:
        return out, None, None, None
    u = g.float().reshape(z.shape)
    gpos = None
    if forces:
        half, R = d // 2, cos.shape[2]
        gt = (y[:, :, :R] * u[:, :, half:half + R] - y[:, :, half:half + R] * u[:, :, :R]).sum((1, 3))
        gpos = gt @ freq.t()
    if pos is not None:
        u = _turn(u, cos, -sin)
    a = u * wide
    along = (_per_degree((a * zhat).sum(2), lmax) / count)[..., degree][:, :, None, :]
    gx = (r * (a - zhat * along)).reshape(x.shape).to(x.dtype)
    gw = _per_degree((u * zhat).sum((0, 1)), lmax).t().contiguous()
    return out, gx, gw, gpos


def _plain_qk(st):
    c = st["case"]
    q, gq, gwq, gpq = _plain_head_norm(st["q"], st["wq"], st["pq"], st["freq"], c["heads"], c["lmax"], st.get("gq"),
                                       c["forces"])
    k, gk, gwk, gpk = _plain_head_norm(st["k"], st["wk"], st["pk"], st["freq"], c["kv_heads"], c["lmax"], st.get("gk"),
                                       c["forces"])
    if not c["train"]:
        return q, k
    return (q, k, gq, gk, gwq, gwk) + ((gpq, gpk) if c["forces"] else ())


def _plain_route(st):
    c = st["case"]
    N, X, G, k = c["N"], c["X"], c["groups"], c["k"]
    wide = st["logits"].double()  # the choice in 64 bits: scores next to each other
    s = torch.softmax(wide, 1) if c["score"] == "softmax" else torch.sigmoid(wide)
    # without a bias the logits' order is the scores'
    v = wide if st["bias"] is None and G == 1 else s if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        member = torch.sort(v.reshape(N, G, X // G), dim=2, descending=True)[0][:, :, :2].sum(2)
        best = torch.sort(member, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        open_ = torch.zeros(N, G, dtype=torch.bool, device=v.device).scatter_(1, best, True)
        v = v.masked_fill(~open_[:, :, None].expand(N, G, X // G).reshape(N, X), -math.inf)
    idx = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :k]
    s = s.float()
    taken = s.gather(1, idx)
    part = taken / taken.sum(1, keepdim=True) if c["renormalise"] else taken
    weight = part * 1.5
    if not c["train"]:
        return idx.to(torch.int32), weight
    g = st["grad_weight"] * 1.5
    if c["renormalise"]:
        g = part * (g - (g * part).sum(1, keepdim=True))
        g = g * (1.0 - taken) if c["score"] == "sigmoid" else g
        grad = torch.zeros_like(s).scatter_(1, idx, g)
    elif c["score"] == "sigmoid":
        grad = torch.zeros_like(s).scatter_(1, idx, g * taken * (1.0 - taken))
    else:
        grad = s * (torch.zeros_like(s).scatter_(1, idx, g) - (g * taken).sum(1, keepdim=True))
    return idx.to(torch.int32), weight, grad.to(st["logits"].dtype)


def _plain_expert(st):
    c = st["case"]
    N, C, X, k, lmax = c["N"], c["C"], c["X"], c["k"], c["lmax"]
    K = (lmax + 1) ** 2
    dt, idx = st["h"].dtype, st["idx"].long()
    weight = st["weight"] if c["gates"] else torch.ones(N, k, device=idx.device)
    gate = torch.zeros(N, X, device=idx.device).scatter_add_(1, idx, weight)
    degree = _degrees(lmax, idx.device)
    W = st["W"].float()[:, degree]  # [X, K, C', C]
    h = st["h"].float().permute(2, 0, 1).contiguous()  # [K, N, C]
    each = torch.bmm(h, W.permute(1, 3, 0, 2).reshape(K, C, X * C).contiguous()).reshape(K, N, X, C)  # all experts
    out = (each * gate[None, :, :, None]).sum(2).permute(1, 2, 0).to(dt).contiguous()
    if not c["train"]:
        return out
    g = st["grad_out"].float().permute(2, 0, 1).contiguous()
    gw = (each * g[:, :, None, :]).sum((0, 3)).gather(1, idx) if c["gates"] else None
    del each
    back = torch.bmm(g, W.permute(1, 2, 0, 3).reshape(K, C, X * C).contiguous()).reshape(K, N, X, C)
    gh = (back * gate[None, :, :, None]).sum(2).permute(1, 2, 0).to(dt).contiguous()
    del back
    weighted = (gate[None, :, :, None] * g[:, :, None, :]).reshape(K, N, X * C).transpose(1, 2).contiguous()
    gW = torch.bmm(weighted, h).reshape(K, X, C, C)
    gW = torch.zeros(lmax + 1, X, C, C, device=h.device).index_add_(0, degree, gW).transpose(0, 1).contiguous()
    return (out, gh, gW, gw) if c["gates"] else (out, gh, gW)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"bias": _exact_bias, "qk": _exact_qk, "route": _exact_route, "expert": _exact_expert}[case["op"]](case, st)


def _exact_bias(c, st):
    bound2 = st["bounds"].double() ** 2
    outs, total = [], torch.zeros(c["B"], c["H"], dtype=torch.float64, device=bound2.device)
    for vec, g in zip(st["vec"].split(1 << 19), st.get("grad_bias", st["vec"]).split(1 << 19)):
        x, y, z = vec.double().unbind(1)
        r2 = x * x + y * y + z * z
        b = (r2[:, None] >= bound2).sum(1)
        near = torch.ones_like(r2, dtype=torch.bool) if not c["r_cut"] else r2 < c["r_cut"] * c["r_cut"]
        outs.append(torch.where(near[:, None], st["table"].double()[b], -math.inf))
        if c["train"]:
            member = ((b[:, None] == torch.arange(c["B"], device=b.device)) & near[:, None]).double()
            total += member.t() @ g.double()
    out = torch.cat(outs)
    return (out, total) if c["train"] else out


def _exact_qk(c, st):
    K, lmax, d = (c["lmax"] + 1) ** 2, c["lmax"], c["C"] // c["heads"]
    freq = None if st["freq"] is None else st["freq"].double()

    def one(x, w, pos, heads):
        z = x.reshape(x.shape[0], heads, d, K)
        parts = []
        for l in range(lmax + 1):
            t = z[..., l * l:(l + 1) * (l + 1)]
            parts.append(t / (t.pow(2).mean((2, 3), keepdim=True) + EPS).sqrt() * w[l][:, None])
        y = torch.cat(parts, 3)
        if pos is not None:
            R, half = c["R"], d // 2
            turn = torch.exp(1j * sum(pos[:, a, None] * freq[a] for a in range(c["axes"])))[:, None, :, None]
            pair = torch.complex(y[:, :, :R], y[:, :, half:half + R]) * turn
            y = torch.cat((pair.real, y[:, :, R:half], pair.imag, y[:, :, half + R:]), 2)
        return y.reshape(x.shape)

    names = ["q", "k", "wq", "wk"] + (["pq", "pk"] if c["forces"] else [])
    with torch.enable_grad():
        leaf = {n: st[n].double().requires_grad_(c["train"]) for n in ("q", "k", "wq", "wk")}
        for n in ("pq", "pk"):
            leaf[n] = None if st[n] is None else st[n].double().requires_grad_(c["train"] and c["forces"])
        q = one(leaf["q"], leaf["wq"], leaf["pq"], c["heads"])
        k = one(leaf["k"], leaf["wk"], leaf["pk"], c["kv_heads"])
        if not c["train"]:
            return q, k
        grads = torch.autograd.grad((q, k), [leaf[n] for n in names], (st["gq"].double(), st["gk"].double()))
    return (q.detach(), k.detach()) + tuple(grads)


def _exact_route(c, st):
    """The choice by counting, for each expert, those before it; gradients by torch's own differentiation."""
    N, X, G, k = c["N"], c["X"], c["groups"], c["k"]
    if N * X * X > 1 << 30:
        pieces, size = [], max(1, (1 << 28) // (X * X))
        for at in range(0, N, size):
            part = {n: t[at:at + size] if n in ("logits", "grad_weight") else t for n, t in st.items()}
            pieces.append(_exact_route(dict(c, N=min(size, N - at)), part))
        return tuple(torch.cat(t) if t[0] is not None else None for t in zip(*pieces))

    def before(v):  # how many come before each: larger, or as large with a smaller index
        n = v.shape[1]
        lower = torch.arange(n, device=v.device)
        ahead = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (lower[None, :] < lower[:, None]))
        return ahead.sum(2)

    with torch.enable_grad():
        logits = st["logits"].double().requires_grad_(c["train"])
        s = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)) if c["score"] == "softmax" \
            else 1.0 / (1.0 + torch.exp(-logits))
        v = logits.detach() if st["bias"] is None and G == 1 else s.detach()
        if st["bias"] is not None:
            v = v + st["bias"].double()
        if G > 1:
            member = v.reshape(N, G, X // G)
            two = member.amax(2)
            if X // G > 1:
                two = two + member.kthvalue(X // G - 1, dim=2)[0]
            v = torch.where((before(two) < c["top_groups"])[:, :, None], member, -math.inf).reshape(N, X)
        place = before(v)
        idx = torch.stack([(place == j).long().argmax(1) for j in range(k)], 1)
        taken = torch.gather(s, 1, idx)
        weight = 1.5 * (taken / taken.sum(1, keepdim=True) if c["renormalise"] else taken)
        if not c["train"]:
            return None, weight
        grad, = torch.autograd.grad(weight, logits, st["grad_weight"].double())
    return None, weight.detach(), grad


def _exact_expert(c, st):
    N, C, lmax = c["N"], c["C"], c["lmax"]
    h, W = st["h"].double(), st["W"].double()
    out, gh, gW = torch.zeros_like(h), torch.zeros_like(h), torch.zeros_like(W)
    weight = st["weight"].double() if c["gates"] else torch.ones(N, c["k"], dtype=torch.float64, device=h.device)
    gw = torch.zeros_like(weight)
    for e in range(c["X"]):
        n, j = torch.nonzero(st["idx"] == e, as_tuple=True)
        for l in range(lmax + 1):
            m = slice(l * l, (l + 1) * (l + 1))
            x = h[n][:, :, m].transpose(1, 2).reshape(-1, C)  # rows (node, m)
            back = lambda t: t.reshape(n.numel(), 2 * l + 1, C).transpose(1, 2)  # noqa: E731
            y = back(x @ W[e, l].t().contiguous())
            out[n, :, m] += weight[n, j][:, None, None] * y  # (an expert stands once in a node's list)
            if c["train"]:
                g = st["grad_out"].double()[n][:, :, m]
                gw[n, j] += (g * y).sum((1, 2))
                rows = (weight[n, j][:, None, None] * g).transpose(1, 2).reshape(-1, C)
                gh[n, :, m] += back(rows @ W[e, l])
                gW[e, l] = rows.t().contiguous() @ x
    if not c["train"]:
        return out
    return (out, gh, gW, gw) if c["gates"] else (out, gh, gW)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    train = case["train"]
    if case["op"] == "bias":
        E, H, B = case["E"], case["H"], case["B"]
        nbytes = E * (12 + 4 * H) + 4 * B * (H + 1)
        return {"bytes": nbytes + (E * 4 * H + 4 * B * H if train else 0), "flops": E * (6 + (H if train else 0))}
    es = 2 if case["x"] == "bf16" else 4
    if case["op"] == "qk":
        K = (case["lmax"] + 1) ** 2
        size = K * (case["N"] * case["C"] + case["M"] * case["C"] // case["heads"] * case["kv_heads"])
        pos = 4 * (case["N"] + case["M"]) * case["axes"]
        nbytes = 2 * es * size + pos + (2 * es * size + (pos if case["forces"] else 0) if train else 0)
        return {"bytes": nbytes, "flops": size * (8 + (16 if train else 0))}
    if case["op"] == "route":
        N, X, k = case["N"], case["X"], case["k"]
        return {"bytes": N * X * es + 8 * N * k + (N * X * es + 4 * N * k if train else 0), "flops": N * X * (8 + (6 if train else 0))}
    N, C, K, X, k = case["N"], case["C"], (case["lmax"] + 1) ** 2, case["X"], case["k"]
    met = min(X, N * k) * (case["lmax"] + 1) * C * C
    lists = N * k * (4 + (4 if case["gates"] else 0))
    nbytes = 2 * es * N * C * K + es * met + lists
    if train:  # grad_out in; gradients of h (out), the weights (fp32) and the gates
        nbytes += 2 * es * N * C * K + 4 * met + (4 * N * k if case["gates"] else 0)
    return {"bytes": nbytes, "flops": 2 * N * k * K * C * C * (3 if train else 1)}
