"""The operators of an equivariant graph-attention layer as measured work: neighbour attention with
a learned distance-bucket bias and dropout of its probabilities, the distance buckets, the layer
norm of irreps rows and the channel dropout.

Every case has a plain form in elementary torch operations (own = False) and the library's calls
(own = True); `exact` computes the same outputs from the definitions in 64 bits.

Layout, as everywhere in the library: a node row holds the blocks of its irreps in order, inside a
block [channel][m].  Head h of H owns the h-th of H equal parts of every block's channels, which are
contiguous floats, so x_h below is a slice of every block."""
import functools
import math

import numpy as np
import torch

own = False

P_WORDS = 1 << 32
PHILOX_M = (0xD2511F53, 0xCD9E8D57)          # Philox4x32-10: Salmon, Moraes, Dror, Shaw, SC 2011
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
MASK = 0xFFFFFFFF


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a molecule of 24 atoms, 8 neighbours each: inference on one small system, latency alone counts
        dict(name="attn fwd 24 atoms", op="attn", back=False, nodes=24, edges=192, graph="even", hub=False, pad=0,
             qk="4x0e+4x1o", v="4x0e+4x1o", heads=2, buckets=8, p=0.0, fused=False, sorted=True),
        # the training step of a NequIP-sized graph (1,536 atoms, mean degree 30), q|k|v from one linear map
        dict(name="attn step 46k edges", op="attn", back=True, nodes=1536, edges=46080, graph="even", hub=False, pad=0,
             qk="32x0e+32x1o+32x2e", v="32x0e+32x1o+32x2e", heads=4, buckets=32, p=0.1, fused=True, sorted=True),
        # clustered atoms (degrees from a few to hundreds) with one global node that hears and tells all atoms;
        # logits from the scalars alone; the neighbour list is new, so its sender order is built in the pass
        dict(name="attn step global node", op="attn", back=True, nodes=8193, edges=294643, graph="skewed", hub=True,
             pad=0, qk="64x0e", v="32x0e+32x1o+32x2e+32x3o", heads=8, buckets=64, p=0.0, fused=False, sorted=False),
        # odd channel counts, degrees down to zero, and a neighbour list of fixed capacity whose tail is spare
        dict(name="attn step odd sizes", op="attn", back=True, nodes=5003, edges=100003, graph="random", hub=False,
             pad=9973, qk="21x0e+21x1o", v="21x0e+21x1o+21x2e", heads=3, buckets=17, p=0.25, fused=False, sorted=True),
        # inference on 100,000 atoms and 3.0 million edges at 128 channels: rows far beyond the caches
        dict(name="attn fwd 3M edges", op="attn", back=False, nodes=100000, edges=3001138, graph="random", hub=False,
             pad=0, qk="128x0e+128x1o+128x2e", v="128x0e+128x1o+128x2e", heads=8, buckets=32, p=0.0, fused=False,
             sorted=True),
        # the buckets of the two neighbour lists above, once per list
        dict(name="buckets 46k edges", op="buckets", edges=46080, bounds=31),
        dict(name="buckets 3M edges", op="buckets", edges=3001138, bounds=31),
        # node rows of the NequIP-sized graph, forward and backward
        dict(name="norm step 1536 rows", op="norm", back=True, rows=1536, irreps="32x0e+32x1o+32x2e"),
        # the radial network's hidden layer: one row of 64 scalars per edge, forward and backward
        dict(name="norm step 163k x 64", op="norm", back=True, rows=162892, irreps="64x0e"),
        # node rows of the largest graph, inference
        dict(name="norm fwd 100k rows", op="norm", back=False, rows=100000, irreps="128x0e+128x1o+128x2e"),
        # feature dropout of the NequIP-sized graph's rows and of the largest graph's, forward and backward
        dict(name="dropout step 1536 rows", op="dropout", back=True, rows=1536, irreps="32x0e+32x1o+32x2e", p=0.1),
        dict(name="dropout step 100k rows", op="dropout", back=True, rows=100000, irreps="128x0e+128x1o+128x2e", p=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _irreps(rng, mul):
    blocks = [t for t in ("0e", "0o", "1o", "1e", "2e", "3o") if rng.random() < 0.45] or ["0e"]
    return "+".join("%dx%s" % (mul, t) for t in blocks)


def draw(rng):
    op = rng.choice(("attn", "attn", "attn", "buckets", "norm", "dropout"))
    if op == "buckets":
        return dict(op=op, edges=_log_int(rng, 1, 3000000), bounds=rng.randint(1, 255))
    if op != "attn":
        irreps = _irreps(rng, _log_int(rng, 1, 160))
        rows = _log_int(rng, 1, min(400000, 100000 * 1152 // _dim(irreps)))
        case = dict(op=op, back=rng.random() < 0.7, rows=rows, irreps=irreps)
        return case if op == "norm" else dict(case, p=rng.choice((0.05, 0.1, 0.5)))
    heads = rng.choice((1, 2, 3, 4, 8, 16))
    mul = heads * _log_int(rng, 1, max(1, 128 // heads))
    v = _irreps(rng, mul)
    qk = v if rng.random() < 0.6 else "%dx0e" % (heads * rng.randint(1, 24))
    nodes = _log_int(rng, 16, 100000)
    most = int(min(3.0e6, 3.0e9 / (_dim(qk) + _dim(v)), 64.0 * nodes))
    edges = _log_int(rng, max(1, most // 20), max(1, most))
    return dict(op=op, back=rng.random() < 0.7, nodes=nodes + 1, edges=edges, graph=rng.choice(("random", "skewed")),
                hub=rng.random() < 0.3, pad=rng.choice((0, 0, rng.randint(1, 5000))), qk=qk, v=v, heads=heads,
                buckets=rng.randint(2, 128), p=rng.choice((0.0, 0.1, 0.3)), fused=rng.random() < 0.5,
                sorted=rng.random() < 0.7)


# ----------------------------------------------------------------------------------------- layout

@functools.lru_cache(maxsize=None)
def _blocks(irreps):
    """[(channels, 2l + 1, offset, is 0e)]"""
    got, at = [], 0
    for term in irreps.split("+"):
        mul, ir = term.split("x")
        d = 2 * int(ir[:-1]) + 1
        got.append((int(mul), d, at, ir == "0e"))
        at += int(mul) * d
    return got


def _dim(irreps):
    return sum(m * d for m, d, _, _ in _blocks(irreps))


def _channels(irreps):
    return sum(m for m, _, _, _ in _blocks(irreps))


def _edges(case):
    """Edges of the graph, those of the global node among them, without the spare ones."""
    return case["edges"] + (2 * (case["nodes"] - 1) if case["hub"] else 0)


# ---------------------------------------------------------------------------------------- prepare

def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")          # noqa: E731
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")             # noqa: E731
    s = dict(case=case)
    s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C1 % (1 << 63), seed], dtype=torch.int64, device="cuda")
    if case["op"] == "buckets":
        E = case["edges"]
        direction = normal(E, 3)
        length = 6.0 * rand(E, 1).pow(1.0 / 3.0)
        s["vec"] = direction / direction.norm(dim=1, keepdim=True) * length
        s["bounds"] = torch.logspace(math.log10(0.7), math.log10(4.9), case["bounds"], device="cuda")
        n = min(E // 4, case["bounds"])              # distances that lie on a bound, one of zero, one that is lost
        s["vec"][:n] = 0.0
        s["vec"][torch.arange(n, device="cuda"), torch.arange(n, device="cuda") % 3] = s["bounds"][:n]
        s["vec"][n:n + 1] = 0.0
        s["vec"][n + 1:n + 2] = float("nan")
        s["cutoff"] = 5.0
    elif case["op"] == "norm":
        n_scalar = sum(m for m, _, _, e in _blocks(case["irreps"]) if e)
        s["x"] = normal(case["rows"], _dim(case["irreps"])) * (0.25 + rand(case["rows"], 1)) + 0.1
        s["weight"] = 1.0 + 0.2 * normal(_channels(case["irreps"]))
        s["bias"] = 0.2 * normal(n_scalar)
        s["gy"] = normal(case["rows"], _dim(case["irreps"]))
    elif case["op"] == "dropout":
        s["x"] = normal(case["rows"], _dim(case["irreps"]))
        s["gy"] = normal(case["rows"], _dim(case["irreps"]))
    else:
        _prepare_attn(s, case, normal, rand)
    return s


def _prepare_attn(s, case, normal, rand):
    N, E, H, pad = case["nodes"], case["edges"], case["heads"], case["pad"]
    dq, dv, K = _dim(case["qk"]), _dim(case["v"]), case["buckets"]
    long = dict(dtype=torch.int64, device="cuda")
    atoms = N - 1 if case["hub"] else N
    if case["graph"] == "even":
        dst = torch.arange(E, **long) * atoms // E
    elif case["graph"] == "random":
        dst = (rand(E) * atoms).long().clamp_(max=atoms - 1)
    else:
        share = torch.cumsum((rand(atoms).pow(3) + 0.02).double(), 0)
        dst = torch.searchsorted(share, rand(E).double() * share[-1]).clamp_(max=atoms - 1)
    src = (rand(E) * atoms).long().clamp_(max=atoms - 1)
    dist = 5.3 * rand(E).pow(1.0 / 3.0)              # a list with a skin: the edges beyond 5 take no part
    bounds = torch.logspace(math.log10(0.7), math.log10(4.9), K - 1, device="cuda")
    bucket = torch.bucketize(dist, bounds, right=True)
    bucket = torch.where(dist < 5.0, bucket, -1)
    if case["hub"]:                                  # the global node is the last one; its edges have a bucket of their own
        a = torch.arange(atoms, **long)
        top = torch.full((atoms,), atoms, **long)
        dst, src = torch.cat([dst, top, a]), torch.cat([src, a, top])
        bucket = torch.cat([bucket, torch.full((2 * atoms,), K - 1, **long)])
    dst, order = torch.sort(dst, stable=True)
    src, bucket = src[order], bucket[order]
    rowptr = torch.searchsorted(dst, torch.arange(N + 1, **long))
    if pad:                                          # spare places of a list of fixed capacity
        src = torch.cat([src, torch.full((pad,), -1, **long)])
        dst = torch.cat([dst, torch.zeros(pad, **long)])
        bucket = torch.cat([bucket, torch.full((pad,), -1, **long)])
    s.update(dst=dst, rowptr=rowptr.int(), src=src.int(), bucket=bucket.int())
    if case["sorted"]:                               # the sender order that the graph's other layers use too
        by, perm = torch.sort(torch.where(src < 0, N, src), stable=True)
        s.update(perm=perm.int(), colptr=torch.searchsorted(by, torch.arange(N + 1, **long)).int())
    if case["fused"]:
        qkv = normal(N, 2 * dq + dv)
        s.update(q=qkv[:, :dq], k=qkv[:, dq:2 * dq], v=qkv[:, 2 * dq:])
    else:
        s.update(q=normal(N, dq), k=normal(N, dq), v=normal(N, dv))
    s.update(table=0.5 * normal(K, H), gy=normal(N, dv), scale=math.sqrt(H / dq))


# -------------------------------------------------------------------------------------------- run

def run(s):
    if own:
        return _own(s)
    return {"attn": _attn, "buckets": _buckets, "norm": _norm, "dropout": _dropout}[s["case"]["op"]](s)


@functools.lru_cache(maxsize=None)
def _handle(kind, *args):
    """The library's handle of a layer, as a model keeps it (host memory, no data)."""
    import equivariant_tensor_product_b200 as tp
    return getattr(tp, kind)(*args)


def _own(s):
    import equivariant_tensor_product_b200 as tp
    case = s["case"]
    if case["op"] == "buckets":
        return {"bucket": tp.tp_distance_buckets(s["vec"], s["bounds"], s["cutoff"])}
    if case["op"] == "norm":
        norm = _handle("Norm", case["irreps"])
        out = {"y": tp.tp_norm_fwd(norm, s["x"], s["weight"], s["bias"])}
        if case["back"]:
            out["gx"], out["gweight"], out["gbias"] = tp.tp_norm_bwd(norm, s["x"], s["gy"], s["weight"])
        return out
    if case["op"] == "dropout":
        drop = _handle("Dropout", case["irreps"])
        out = {"y": tp.tp_dropout_fwd(drop, s["x"], case["p"], s["rng"])}
        if case["back"]:
            out["gx"] = tp.tp_dropout_bwd(drop, s["gy"], case["p"], s["rng"])
        return out
    attn = _handle("Attention", case["qk"], case["v"], case["heads"], case["buckets"])
    more = dict(bucket=s["bucket"], table=s["table"], scale=s["scale"], p=case["p"], rng=s["rng"])
    y, lse = tp.tp_attn_fwd(attn, s["rowptr"], s["src"], s["q"], s["k"], s["v"], **more)
    if not case["back"]:
        return {"y": y, "lse": lse}
    gq, gk, gv, gtable = tp.tp_attn_bwd(attn, s["rowptr"], s["src"], s["q"], s["k"], s["v"], y, lse, s["gy"],
                                        colptr=s.get("colptr"), perm=s.get("perm"), **more)
    return {"y": y, "lse": lse, "gq": gq, "gk": gk, "gv": gv, "gtable": gtable}


# ------------------------------------------------------------------------------------ plain forms

def _buckets(s):
    """Number of bounds that are not above |vec|, or -1 from the cutoff on (and for NaN).  Squares in 64
    bits: a product of two 32-bit floats is exact there, so no distance changes sides at a bound."""
    x, y, z = s["vec"].double().unbind(1)
    d2 = x * x + y * y + z * z
    n = (d2[:, None] >= s["bounds"].double().square()[None]).sum(1)
    return {"bucket": torch.where(d2 < s["cutoff"] ** 2, n, -1).int()}


def _norm_parts(x, eps=1e-5):
    """Per block: (x centred and scaled to unit mean square, 1 / root mean square) -- 0e blocks lose their
    mean over channels, every other block keeps its direction and is only scaled."""
    return [(lambda c, r: (c * r, r))(c, torch.rsqrt(c.square().mean((1, 2), keepdim=True) + eps)) for c in x]


def _norm(s):
    case, x = s["case"], s["x"]
    blocks = _blocks(case["irreps"])
    first = np.cumsum([0] + [m for m, _, _, _ in blocks])
    zeroth = np.cumsum([0] + [m if e else 0 for m, _, _, e in blocks])
    weight = [s["weight"][first[i]:first[i + 1], None] for i in range(len(blocks))]
    bias = [s["bias"][zeroth[i]:zeroth[i + 1], None] for i in range(len(blocks))]
    cut = lambda t: [t[:, at:at + m * d].reshape(-1, m, d) for m, d, at, _ in blocks]   # noqa: E731
    centre = lambda t, e: t - t.mean((1, 2), keepdim=True) if e else t                  # noqa: E731
    parts = _norm_parts([centre(t, b[3]) for t, b in zip(cut(x), blocks)])
    out = {"y": torch.cat([(n * w + b if e[3] else n * w).flatten(1) for (n, _), w, b, e in zip(parts, weight, bias, blocks)], 1)}
    if case["back"]:
        gy = cut(s["gy"])
        g = [t * w for t, w in zip(gy, weight)]
        out["gx"] = torch.cat([(r * (centre(t, e[3]) - n * (t * n).mean((1, 2), keepdim=True))).flatten(1)
                               for t, (n, r), e in zip(g, parts, blocks)], 1)
        out["gweight"] = torch.cat([(t * n).double().sum((0, 2)) for t, (n, _) in zip(gy, parts)]).float()
        out["gbias"] = torch.cat([t.double().sum((0, 2)) for t, e in zip(gy, blocks) if e[3]]
                                 or [torch.zeros(0, dtype=torch.float64, device=x.device)]).float()
    return out


def _mulhilo(a, b):
    """High and low 32 bits of the product of a 32-bit constant and 32-bit values held in 64-bit ones."""
    low = a * (b & 0xFFFF)
    t = a * (b >> 16) + (low >> 16)
    return t >> 16, ((t & 0xFFFF) << 16) | (low & 0xFFFF)


def _keep(rng, n, p):
    """n truth values from Philox4x32-10: value i is word i mod 4 of the block with counter
    (i div 4, offset) and the seed as key, and is kept when it is not below p 2^32."""
    block = torch.arange((n + 3) // 4, dtype=torch.int64, device=rng.device)
    c = [block & MASK, block >> 32, (rng[1] & MASK).expand_as(block), ((rng[1] >> 32) & MASK).expand_as(block)]
    k = [rng[0] & MASK, (rng[0] >> 32) & MASK]
    for _ in range(10):
        h0, l0 = _mulhilo(PHILOX_M[0], c[0])
        h1, l1 = _mulhilo(PHILOX_M[1], c[2])
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + PHILOX_W[0]) & MASK, (k[1] + PHILOX_W[1]) & MASK]
    return torch.stack(c, 1).reshape(-1)[:n] >= round(p * P_WORDS)


def _dropout(s):
    case = s["case"]
    n = _channels(case["irreps"])
    keep = _keep(s["rng"], case["rows"] * n, case["p"]).reshape(case["rows"], n).float() / (1.0 - case["p"])
    first = np.cumsum([0] + [m for m, _, _, _ in _blocks(case["irreps"])])
    keep = torch.cat([keep[:, first[i]:first[i + 1]].repeat_interleave(d, 1)
                      for i, (_, d, _, _) in enumerate(_blocks(case["irreps"]))], 1)
    out = {"y": s["x"] * keep}
    if case["back"]:
        out["gx"] = s["gy"] * keep
    return out


def _heads(x, irreps, H):
    """[N, dim] -> [N, H, dim / H]"""
    return torch.cat([x[:, at:at + m * d].reshape(-1, H, m * d // H) for m, d, at, _ in _blocks(irreps)], 2)


def _rows(x, irreps):
    """The inverse of _heads."""
    H = x.shape[1]
    parts = torch.split(x, [m * d // H for m, d, _, _ in _blocks(irreps)], 2)
    return torch.cat([t.reshape(x.shape[0], -1) for t in parts], 1)


def _attn(s):
    """p_eh = softmax over the edges e into i of scale q_ih . k_jh + table[bucket_e, h]; y_ih = sum_e r_eh p_eh v_jh
    with r = keep / (1 - p).  An edge without a bucket takes no part; a row without edges is zero."""
    case, N = s["case"], s["q"].shape[0]
    H, dst, src = case["heads"], s["dst"], s["src"].long().clamp(min=0)
    q, k, v = _heads(s["q"], case["qk"], H), _heads(s["k"], case["qk"], H), _heads(s["v"], case["v"], H)
    live = (s["bucket"] >= 0)[:, None]
    bucket = s["bucket"].long().clamp(min=0)
    logit = (q[dst] * k[src]).sum(2) * s["scale"] + s["table"][bucket]
    logit = torch.where(live, logit, -math.inf)
    top = torch.full((N, H), -math.inf, device=q.device).scatter_reduce_(0, dst[:, None].expand(-1, H), logit, "amax")
    top = torch.where(top > -math.inf, top, 0.0)
    total = torch.zeros(N, H, device=q.device).index_add_(0, dst, torch.exp(logit - top[dst]))
    lse = top + torch.log(total)
    prob = torch.where(live, torch.exp(logit - lse[dst]), 0.0)
    drop = prob
    if case["p"]:
        keep = _keep(s["rng"], dst.numel() * H, case["p"]).reshape(-1, H).float() / (1.0 - case["p"])
        drop = prob * keep
    y = torch.zeros_like(v).index_add_(0, dst, drop[:, :, None] * v[src])
    out = {"y": _rows(y, case["v"]), "lse": lse}
    if case["back"]:
        gy = _heads(s["gy"], case["v"], H)
        g = (gy[dst] * v[src]).sum(2)
        g = prob * ((g * keep if case["p"] else g) - (gy * y).sum(2)[dst])
        back = (g * s["scale"])[:, :, None]
        out["gq"] = _rows(torch.zeros_like(q).index_add_(0, dst, back * k[src]), case["qk"])
        out["gk"] = _rows(torch.zeros_like(k).index_add_(0, src, back * q[dst]), case["qk"])
        out["gv"] = _rows(torch.zeros_like(v).index_add_(0, src, drop[:, :, None] * gy[dst]), case["v"])
        out["gtable"] = torch.zeros(s["table"].shape, dtype=torch.float64, device=q.device).index_add_(0, bucket, g.double()).float()
    return out


# ------------------------------------------------------------------------------------------- work

def work(case):
    """Every input read once, every output written once; the products and sums of the formulas."""
    if case["op"] == "buckets":
        return {"bytes": 16 * case["edges"] + 4 * case["bounds"], "flops": 5 * case["edges"]}
    if case["op"] in ("norm", "dropout"):
        n = case["rows"] * _dim(case["irreps"])
        if case["op"] == "dropout":
            return {"bytes": 8 * n * (2 if case["back"] else 1), "flops": n * (2 if case["back"] else 1)}
        return {"bytes": 4 * n * (4 if case["back"] else 2), "flops": n * (18 if case["back"] else 7)}
    N, E, H, dq, dv = case["nodes"], _edges(case), case["heads"], _dim(case["qk"]), _dim(case["v"])
    table = 4 * case["buckets"] * H
    size = 4 * N * (2 * dq + 2 * dv + H) + 4 * (N + 1) + 8 * E + table
    flops = E * (2 * dq + 2 * dv + 6 * H)
    if case["back"]:
        size += 4 * N * (2 * dq + 2 * dv) + table + (4 * (N + 1) + 4 * E if case["sorted"] else 0)
        flops += E * (4 * dq + 4 * dv + 5 * H)
    return {"bytes": size, "flops": flops}


# ------------------------------------------------------------------------------------------ exact

def _exact_keep(seed, offset, n, p):
    """The kept values again, from 64-bit unsigned numbers."""
    u = np.uint64
    low, half = u(MASK), u(32)
    block = np.arange((n + 3) // 4, dtype=u)
    word = [block & low, block >> half, np.full_like(block, offset & MASK), np.full_like(block, offset >> 32)]
    key = [seed & MASK, seed >> 32]
    for r in range(10):
        a, b = word[0] * u(PHILOX_M[0]), word[2] * u(PHILOX_M[1])
        k0, k1 = ((key[i] + r * PHILOX_W[i]) & MASK for i in (0, 1))
        word = [(b >> half) ^ word[1] ^ u(k0), b & low, (a >> half) ^ word[3] ^ u(k1), a & low]
    drop = np.stack(word, 1).reshape(-1)[:n] < u(round(p * P_WORDS))
    return torch.from_numpy(~drop).cuda().double() / (1.0 - p)


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    random = [int(t) for t in s["rng"]]
    if case["op"] == "buckets":
        v = s["vec"].cpu().numpy().astype(np.float64)
        d2 = v[:, 0] ** 2 + v[:, 1] ** 2 + v[:, 2] ** 2
        at = np.searchsorted(s["bounds"].cpu().numpy().astype(np.float64) ** 2, d2, side="right")
        return {"bucket": np.where(d2 < s["cutoff"] ** 2, at, -1).astype(np.int32)}
    if case["op"] == "dropout":
        n = _channels(case["irreps"])
        if case["rows"] * n > 5e7:
            return None
        widths = torch.tensor([d for m, d, _, _ in _blocks(case["irreps"]) for _ in range(m)], device="cuda")
        keep = _exact_keep(*random, case["rows"] * n, case["p"]).reshape(case["rows"], n)
        keep = keep[:, torch.repeat_interleave(torch.arange(n, device="cuda"), widths)]
        return {"y": f["x"] * keep, "gx": f["gy"] * keep} if case["back"] else {"y": f["x"] * keep}
    if case["op"] == "norm":
        return _exact_norm(case, f)
    if _edges(case) * (_dim(case["qk"]) + _dim(case["v"])) > 1.2e9:
        return None
    return _exact_attn(case, s, f, random)


def _exact_norm(case, f):
    """The definition, and its gradients from autograd in 64 bits."""
    leaves = [f[k].requires_grad_(case["back"]) for k in ("x", "weight", "bias")]
    x, weight, bias = leaves
    rows, c, z = [], 0, 0
    for m, d, at, even in _blocks(case["irreps"]):
        b = x[:, at:at + m * d].unflatten(1, (m, d))
        if even:
            b = b - b.sum((1, 2), keepdim=True) / m
        b = b / torch.sqrt((b * b).sum((1, 2), keepdim=True) / (m * d) + 1e-5) * weight[c:c + m].unsqueeze(1)
        if even:
            b = b + bias[z:z + m].unsqueeze(1)
            z += m
        c += m
        rows.append(b.flatten(1))
    y = torch.cat(rows, 1)
    if not case["back"]:
        return {"y": y}
    grads = torch.autograd.grad(y, leaves, f["gy"], allow_unused=True)
    return dict(y=y.detach(), **{k: torch.zeros_like(t) if g is None else g
                                 for k, t, g in zip(("gx", "gweight", "gbias"), leaves, grads)})


def _exact_attn(case, s, f, random):
    """The definition on the live edges, head by head, and its gradients from autograd in 64 bits."""
    H, N, n = case["heads"], case["nodes"], s["dst"].numel()
    keep = _exact_keep(*random, n * H, case["p"]).reshape(n, H) if case["p"] else torch.ones(n, H, device="cuda").double()
    at = torch.nonzero(s["bucket"] >= 0)[:, 0]
    i, j, bucket, keep = s["dst"][at], s["src"][at].long(), s["bucket"][at].long(), keep[at]
    leaves = [f[k].detach().clone().requires_grad_(case["back"]) for k in ("q", "k", "v", "table")]
    q, k, v, table = leaves
    y, lse = torch.zeros_like(v), []
    for h in range(H):
        cols = lambda irreps: torch.cat([torch.arange(at_ + h * m * d // H, at_ + (h + 1) * m * d // H, device="cuda")   # noqa: E731
                                         for m, d, at_, _ in _blocks(irreps)])
        a, b = cols(case["qk"]), cols(case["v"])
        e = torch.exp(s["scale"] * torch.einsum("ec,ec->e", q[i][:, a], k[j][:, a]) + table[bucket, h])
        z = torch.zeros(N, dtype=torch.float64, device="cuda").index_add(0, i, e)
        part = torch.zeros(N, len(b), dtype=torch.float64, device="cuda")
        y = y.index_copy(1, b, part.index_add(0, i, (e * keep[:, h] / z[i])[:, None] * v[j][:, b]))
        lse.append(torch.log(z.detach()))
    out = {"y": y.detach(), "lse": torch.stack(lse, 1)}
    if case["back"]:
        grads = torch.autograd.grad(y, leaves, f["gy"], allow_unused=True)
        out.update({name: torch.zeros_like(t) if g is None else g
                    for name, t, g in zip(("gq", "gk", "gv", "gtable"), leaves, grads)})
    return out
