"""Cases and plain forms of head norms with rotary positions, attention with a sliding window and
sinks, and a cache held in 4 bits.

Eight kinds of case, each one pass as a program calls it:

  norm     queries and keys of a packed projection, each head's row divided by its root mean square
           and weighted, then turned by its position
  grad     the way back: gradients of the rows and of both weights
  nappend  a serving step's new rows: norm and rotation, keys and values into the cache
  fwd      attention over the last ``window`` tokens and the document's first ``sinks``
  train    the same with its gradients: o, lse, dq, dk, dv from q, k, v and do
  tree     new tokens (one, a chain, or a tree of drafts) against a cache, with a window and sinks
  append4  new keys and values into a cache held in 4 bits, and those rows read back as the values
           they stand for
  tree4    new tokens against a cache held in 4 bits

``run`` computes them in elementary torch operations in 32 bits (angles and long sums in 64),
rounded once at the end, or, where ``own`` is true, through exact_attention_23_gb300.

The 4-bit cache. A row of d values is cut into groups of 32. A group's scale is its largest
magnitude over 7, rounded up to five significant bits and kept as bf16; a value is the scale times
a whole number of −7 … 7, the nearest (ties to even) to the value over the scale, kept plus 8 in
four bits. (Any such product is a bf16 number.) Groups whose largest magnitude is below 2⁻¹⁰⁰ are
zeros. In a row's d/2 bytes, read as 32-bit words of eight codes, code 0 in the lowest bits:
  keys    word c·(d/32) + w holds dimensions 32w + 4c + (0, 2, 16, 18, 1, 3, 17, 19), c = 0 … 3
  values  word 8·h + n holds dimensions 64h + n + 8·(0, 1, …, 7), n = 0 … 7
"""

import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # norms and rotation of a training step at the repository's GPT-2 shape, read out of the
        # packed projection
        {"name": "norm_b4_h12_t1024_d64", "kind": "norm", "B": 4, "H": 12, "Hkv": 12, "T": 1024,
         "d": 64, "rot": 64, "interleaved": False, "start": 0, "factor": 1.0},
        # their gradients on a long sequence with shared key heads, half of each head turned
        {"name": "grad_b1_h16_kv4_t16384_d128", "kind": "grad", "B": 1, "H": 16, "Hkv": 4,
         "T": 16384, "d": 128, "rot": 64, "interleaved": True, "start": 100000, "factor": 8.0},
        # one new token for each of eight sequences: pure latency
        {"name": "nappend_b8_h16_kv4_n1_d128", "kind": "nappend", "B": 8, "H": 16, "Hkv": 4, "Tq": 1,
         "ctx": 1000, "cap": 1280, "d": 128, "rot": 128, "interleaved": False, "factor": 1.0},
        # a long prompt that sees the last 1024 tokens and the first four
        {"name": "fwd_w1024_b1_h12_t16384_d64", "kind": "fwd", "B": 1, "H": 12, "Hkv": 12,
         "T": 16384, "d": 64, "window": 1024, "sinks": 4, "softcap": 0.0, "slopes": False, "docs": 0,
         "pad": 0},
        # a training step on packed documents, a short window, ragged length, padded end
        {"name": "train_w200_docs_b2_h12_t1000_d64", "kind": "train", "B": 2, "H": 12, "Hkv": 12,
         "T": 1000, "d": 64, "window": 200, "sinks": 3, "softcap": 0.0, "slopes": False, "docs": 3,
         "pad": 23},
        # a training step on one long sequence, shared key heads, wide heads
        {"name": "train_w1024_b1_h16_kv4_t8192_d128", "kind": "train", "B": 1, "H": 16, "Hkv": 4,
         "T": 8192, "d": 128, "window": 1024, "sinks": 16, "softcap": 0.0, "slopes": False,
         "docs": 0, "pad": 0},
        # single-token decoding over ragged contexts that are longer than the window
        {"name": "tree_w1024_one_b16_h12_ctx8000_d64", "kind": "tree", "B": 16, "H": 12, "Hkv": 12,
         "Tq": 1, "ctx": 8000, "cap": 8100, "d": 64, "drafts": False, "window": 1024, "sinks": 4,
         "softcap": 0.0, "slopes": False},
        # sixteen drafts each over long contexts, shared key heads, wide heads
        {"name": "tree_w4096_n16_b4_h16_kv4_ctx16384_d128", "kind": "tree", "B": 4, "H": 16,
         "Hkv": 4, "Tq": 16, "ctx": 16384, "cap": 16500, "d": 128, "drafts": True, "window": 4096,
         "sinks": 4, "softcap": 0.0, "slopes": False},
        # a prompt's keys and values into a 4-bit cache
        {"name": "append4_b4_kv12_n2048_d64", "kind": "append4", "B": 4, "H": 12, "Hkv": 12,
         "Tq": 2048, "ctx": 300, "cap": 2400, "d": 64},
        # one token for each of eight sequences into a 4-bit cache: latency
        {"name": "append4_b8_kv4_n1_d128", "kind": "append4", "B": 8, "H": 16, "Hkv": 4, "Tq": 1,
         "ctx": 1000, "cap": 1280, "d": 128},
        # single-token decoding over long ragged contexts held in 4 bits
        {"name": "tree4_one_b8_h16_kv4_ctx16384_d128", "kind": "tree4", "B": 8, "H": 16, "Hkv": 4,
         "Tq": 1, "ctx": 16384, "cap": 16400, "d": 128, "drafts": False, "window": 0, "sinks": 0,
         "softcap": 0.0, "slopes": False},
        # eight drafts each, a key head for every query head
        {"name": "tree4_n8_b4_h12_ctx4000_d64", "kind": "tree4", "B": 4, "H": 12, "Hkv": 12, "Tq": 8,
         "ctx": 4000, "cap": 4096, "d": 64, "drafts": True, "window": 0, "sinks": 0, "softcap": 0.0,
         "slopes": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "grad", "nappend", "fwd", "fwd", "train", "train", "tree", "tree",
                       "append4", "tree4", "tree4"])
    d = rng.choice([64, 128])
    H, Hkv = rng.choice([(12, 12), (16, 4), (8, 8), (6, 2), (16, 16), (8, 1), (5, 5)])
    turn = {"rot": rng.choice([d, d // 2, d // 4, d]), "interleaved": rng.random() < 0.5,
            "factor": rng.choice([1.0, 1.0, 4.0, 8.0])}
    base = {"kind": kind, "H": H, "Hkv": Hkv, "d": d}
    if kind in ("norm", "grad"):
        return {**base, **turn, "B": rng.choice([1, 2, 3]), "T": _log(rng, 1, 5000),
                "start": rng.choice([0, 17, 100000, 1000000])}
    if kind in ("nappend", "append4"):
        ctx, n = _log(rng, 4, 1500), _log(rng, 1, 40 if kind == "nappend" else 1000)
        cap = -(-(ctx + n + rng.randrange(40)) // 8) * 8
        c = {**base, "B": _log(rng, 1, 24 if kind == "nappend" else 6), "Tq": n, "ctx": ctx, "cap": cap}
        return {**c, **turn} if kind == "nappend" else c
    cap_at = rng.choice([0.0, 0.0, 30.0, 50.0])
    if kind in ("tree", "tree4"):
        ctx = _log(rng, 16, 16000)
        n = rng.choice([1, 1, 2, 5, 8, 16, 31, 64, 100])
        window = 0 if kind == "tree4" and rng.random() < 0.6 else _log(rng, 8, 8000)
        return {**base, "B": max(1, min(_log(rng, 1, 16), 60000 // ctx)), "Tq": n, "ctx": ctx,
                "cap": -(-(ctx + n + rng.randrange(100)) // 8) * 8, "drafts": rng.random() < 0.6,
                "window": window, "sinks": rng.choice([0, 1, 4, 16, 130]) if window else 0,
                "softcap": cap_at, "slopes": rng.random() < 0.25}
    T = _log(rng, 40, 2900 if kind == "train" else 6000)
    docs = rng.choice([0, 0, 3, 9])
    return {**base, "B": max(1, min(rng.choice([1, 2, 3, 4]), 5000 // T)), "T": T,
            "window": _log(rng, 8, T), "sinks": rng.choice([0, 1, 4, 16, 130]), "softcap": cap_at,
            "slopes": rng.random() < 0.25, "docs": docs, "pad": T // 20 if docs else 0}


# ---------------------------------------------------------------- what the cases are made of

def _doc_lengths(T, docs, pad):
    """Ragged document lengths that fill T − pad tokens (the same for every seed)."""
    w = [1 + (5 * i + 3) % 11 for i in range(docs)]
    n, total = T - pad, sum(w)
    ends = [n * sum(w[:i + 1]) // total for i in range(docs)]
    return [e - s for s, e in zip([0] + ends[:-1], ends)]


def _lengths(B, ctx):
    """Context lengths of a ragged batch: from ctx down to about half of it."""
    return [max(1, ctx - b * ctx // (2 * B)) for b in range(B)]


def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(BF16)


def _inv_freq(rot, factor, device="cuda"):
    """Radians a position for each pair: base 10000, high frequencies as they are and low ones
    stretched by ``factor`` (a ramp over the pair's turns in the first 4096 positions)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if factor != 1.0:
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32,
                        device="cuda")


def _tree(B, n, g):
    """Random draft trees: each node's parent is an earlier node (or the context). Returns the
    visibility [B, n, n] (itself and its ancestors) and the depths [B, n]."""
    r = torch.rand((B, n), generator=g, device="cuda").tolist()
    rows, depths = [], []
    for b in range(B):
        vis, dep = [], []
        for t in range(n):
            p = int(r[b][t] * (t + 1)) - 1
            vis.append((list(vis[p]) if p >= 0 else [0] * n))
            vis[t][t] = 1
            dep.append(dep[p] + 1 if p >= 0 else 0)
        rows.append(vis)
        depths.append(dep)
    return (torch.tensor(rows, dtype=torch.uint8, device="cuda"),
            torch.tensor(depths, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------- 4-bit rows

def _dims(d, keys):
    """The dimensions in the order of a row's codes."""
    if keys:
        return [32 * w + 4 * c + e for c in range(4) for w in range(d // 32)
                for e in (0, 2, 16, 18, 1, 3, 17, 19)]
    return [64 * h + n + 8 * x for h in range(d // 64) for n in range(8) for x in range(8)]


def _quantise(x):
    """Rows [..., d] in float32 -> (whole numbers −7 … 7 [..., d], scales [..., d/32]) in float32."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    # (a quotient of tensors: by a number it is a product with 1/7, which is not exact at multiples of 7)
    bits = (top / torch.full_like(top, 7.0)).view(torch.int32)
    scale = ((bits + ((1 << 19) - 1)) & ~((1 << 19) - 1)).view(torch.float32)
    scale = torch.where(top < 2.0 ** -100, torch.zeros_like(scale), scale)
    over = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    c = torch.where(scale[..., None] > 0, torch.round(g / over), torch.zeros_like(g))
    return c.flatten(-2), scale


def _values(c, scale):
    return (c.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _pack(c, keys):
    order = torch.tensor(_dims(c.shape[-1], keys), device=c.device)
    n = (c[..., order].to(torch.int16) + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(codes, scale, keys):
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.float32) - 8.0
    c = torch.empty_like(n)
    c[..., torch.tensor(_dims(n.shape[-1], keys), device=n.device)] = n
    return _values(c, scale.float())


def _cache4(shape, g):
    """(codes, scales) of a cache of normal rows."""
    out = []
    for keys in (True, False):
        c, scale = _quantise(_randn(shape, g).float())
        out += [_pack(c, keys), scale.to(BF16)]
    return out


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    s = {"c": c}
    if c["kind"] in ("norm", "grad", "nappend"):
        n = c["Tq"] if c["kind"] == "nappend" else c["T"]
        s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"])
        s["mscale"] = 0.1 * math.log(c["factor"]) + 1.0
        # rows of different sizes, as a projection's are
        packed = _randn((B, n, H + 2 * Hkv, d), g)
        packed *= torch.exp(0.5 * torch.randn((B, n, H + 2 * Hkv, 1), generator=g, device="cuda")).to(BF16)
        s["q"] = packed[:, :, :H].transpose(1, 2)
        s["k"] = packed[:, :, H:H + Hkv].transpose(1, 2)
        s["v"] = packed[:, :, H + Hkv:].transpose(1, 2)
        if c["kind"] == "nappend":
            s["k_cache"], s["v_cache"] = (_randn((B, Hkv, c["cap"], d), g) for _ in range(2))
            s["ctx_len"] = torch.tensor(_lengths(B, c["ctx"]), dtype=torch.int32, device="cuda")
            s["positions"] = (s["ctx_len"][:, None] + _tree(B, n, g)[1]).contiguous()
        else:
            s["positions"] = torch.arange(n, device="cuda", dtype=torch.int32) + c["start"]
        if c["kind"] == "grad":
            s["gq"], s["gk"] = _randn((B, H, n, d), g), _randn((B, Hkv, n, d), g)
        return s
    if c["kind"] == "append4":
        s["kc"], s["ks"], s["vc"], s["vs"] = _cache4((B, Hkv, c["cap"], d), g)
        s["k"], s["v"] = (_randn((B, Hkv, c["Tq"], d), g) for _ in range(2))
        s["ctx_len"] = torch.tensor(_lengths(B, c["ctx"]), dtype=torch.int32, device="cuda")
        return s
    s["slopes"] = _slopes(H) if c["slopes"] else None
    # capped models have scores that reach the cap's bend; the others are of unit variance
    std = 4.0 if c["softcap"] else 1.0
    if c["kind"] in ("tree", "tree4"):
        n = c["Tq"]
        s["q"] = _randn((B, H, n, d), g, std)
        if c["kind"] == "tree4":
            s["kc"], s["ks"], s["vc"], s["vs"] = _cache4((B, Hkv, c["cap"], d), g)
        else:
            s["k_cache"], s["v_cache"] = (_randn((B, Hkv, c["cap"], d), g) for _ in range(2))
        s["ctx_len"] = torch.tensor(_lengths(B, c["ctx"]), dtype=torch.int32, device="cuda")
        s["tree"], s["depths"] = _tree(B, n, g) if c["drafts"] else (None, None)
        return s
    T = c["T"]
    s["q"] = _randn((B, H, T, d), g, std)
    s["k"], s["v"] = _randn((B, Hkv, T, d), g), _randn((B, Hkv, T, d), g)
    if c["kind"] == "train":
        s["do"] = _randn((B, H, T, d), g)
    if c["docs"]:
        ids = [i for i, n in enumerate(_doc_lengths(T, c["docs"], c["pad"])) for _ in range(n)]
        ids += [-1] * c["pad"]
        s["doc_ids"] = torch.tensor([ids] * B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

EPS = 1e-6


def _rotate(xf, positions, inv_freq, interleaved, mscale, inverse):
    """Rows in float32, turned (float32)."""
    rot = 2 * inv_freq.numel()
    pos = positions if positions.dim() == 2 else positions[None]
    angle = pos[:, None, :, None].double() * inv_freq
    cos, sin = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    if inverse:
        sin = -sin
    a, b = ((xf[..., 0:rot:2], xf[..., 1:rot:2]) if interleaved
            else (xf[..., :rot // 2], xf[..., rot // 2:rot]))
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = (torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1))
    return torch.cat((turned, xf[..., rot:]), -1)


def _normed(x, w, s):
    xf = x.float()
    y = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, s["positions"], s["inv_freq"], s["c"]["interleaved"], s["mscale"], False).to(BF16)


def _normed_back(g, x, w, s):
    h = _rotate(g.float(), s["positions"], s["inv_freq"], s["c"]["interleaved"], s["mscale"], True)
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    n = xf * r
    dw = (h * n).sum((0, 1, 2), dtype=torch.float64).float()
    dn = h * w
    dx = (dn - n * (dn * n).mean(-1, keepdim=True)) * r
    return dx.to(BF16), dw


def _seen(s, T, window, sinks):
    """[B or 1, 1, 1, T, T] truth values: query i sees key j."""
    at = torch.arange(T, device="cuda")
    i, j = at[:, None], at[None, :]
    ids = s.get("doc_ids")
    if ids is None:
        return ((j <= i) & ((i - j < window) | (j < sinks)))[None, None, None]
    first = torch.cat((torch.ones_like(ids[:, :1], dtype=torch.bool), ids[:, 1:] != ids[:, :-1]), 1)
    run = first.long().cumsum(1)
    start = (at * first).cummax(1).values
    same = (run[:, :, None] == run[:, None, :]) & (ids >= 0)[:, :, None]
    near = (i - j < window)[None] | (j[None] < start[:, :, None] + sinks)
    return ((j <= i)[None] & same & near)[:, None, None]


def _scores(qg, kf, c, seen, distance, slopes, bend=False):
    """Modified scores and, where asked for, the cap's derivative: qg [B, Hkv, G, T, d], kf
    [B, Hkv, 1, S, d], distance a function that makes the distances where there is a bias."""
    z = torch.matmul(qg, kf.transpose(-1, -2)) * (1.0 / math.sqrt(c["d"]))
    slope = None
    if c["softcap"]:
        th = torch.tanh(z / c["softcap"])
        z = th * c["softcap"]
        slope = 1.0 - th * th if bend else None
    if slopes is not None:
        z = z - slopes.view(1, c["Hkv"], -1, 1, 1) * distance()
    return z.masked_fill(~seen, -math.inf), slope


def _softmax(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return p / torch.where(l > 0, l, torch.ones_like(l)), lse.squeeze(-1)


def _plain_attention(s, grads):
    c = s["c"]
    B, H, Hkv, T, d = c["B"], c["H"], c["Hkv"], c["T"], c["d"]
    qg = s["q"].float().view(B, Hkv, H // Hkv, T, d)
    kf, vf = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    at = torch.arange(T, device="cuda", dtype=torch.float32)
    z, bend = _scores(qg, kf, c, _seen(s, T, c["window"], c["sinks"]),
                      lambda: (at[:, None] - at).abs(), s["slopes"], bend=grads)
    p, lse = _softmax(z)
    del z
    o = torch.matmul(p, vf)
    out = {"o": o.view(B, H, T, d).to(BF16), "lse": lse.reshape(B, H, T)}
    if grads:
        do = s["do"].float().view(B, Hkv, H // Hkv, T, d)
        out["dv"] = torch.matmul(p.transpose(-1, -2), do).sum(2).to(BF16)
        ds = torch.matmul(do, vf.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)
        ds = ds * p
        if bend is not None:
            ds = ds * bend
        ds = ds * (1.0 / math.sqrt(d))
        out["dq"] = torch.matmul(ds, kf).view(B, H, T, d).to(BF16)
        out["dk"] = torch.matmul(ds.transpose(-1, -2), qg).sum(2).to(BF16)
    return out


def _plain_tree(s, kf, vf):
    """kf, vf: the caches' rows in float32, as many as any sequence has."""
    c = s["c"]
    B, H, Hkv, n, d = c["B"], c["H"], c["Hkv"], c["Tq"], c["d"]
    S = kf.shape[2]
    qg = s["q"].float().view(B, Hkv, H // Hkv, n, d)
    kf, vf = kf[:, :, None], vf[:, :, None]
    ctx = s["ctx_len"].long()[:, None, None]
    j = torch.arange(S, device="cuda")[None, None, :]
    t = torch.arange(n, device="cuda")
    tree = s["tree"].bool() if s["tree"] is not None else (t[None, :] <= t[:, None]).expand(B, n, n)
    depth = s["depths"].long() if s["depths"] is not None else t.expand(B, n)
    draft = (j - ctx).clamp(0, n - 1)                                     # [B, 1, S]
    in_tree = torch.gather(tree, 2, draft.expand(B, n, S)) & (j >= ctx) & (j < ctx + n)
    seen = (j < ctx) | in_tree
    key_at = torch.where(j < ctx, j.expand(B, 1, S), ctx + torch.gather(depth, 1, draft[:, 0])[:, None])
    away = ctx + depth[:, :, None] - key_at
    if c["window"]:
        seen = seen & ((away < c["window"]) | (key_at < c["sinks"]))
    z, _ = _scores(qg, kf, c, seen[:, None, None], lambda: away.abs().float()[:, None, None], s["slopes"])
    p, lse = _softmax(z)
    return {"o": torch.matmul(p, vf).view(B, H, n, d).to(BF16), "lse": lse.reshape(B, H, n)}


def _rows_of(s):
    """Index of the new rows in a cache: batch, head, row."""
    c = s["c"]
    return (torch.arange(c["B"], device="cuda")[:, None, None],
            torch.arange(c["Hkv"], device="cuda")[None, :, None],
            s["ctx_len"].long()[:, None, None] + torch.arange(c["Tq"], device="cuda"))


def _plain_append4(s):
    at, out = _rows_of(s), {}
    for x, keys in (("k", True), ("v", False)):
        c, scale = _quantise(s[x].float())
        s[x + "c"][at], s[x + "s"][at] = _pack(c, keys), scale.to(BF16)
        out[x] = _unpack(s[x + "c"][at], s[x + "s"][at], keys).to(BF16)
    return out


def run(state):
    s, c = state, state["c"]
    kind = c["kind"]
    if own:
        return _own(s, c, kind)
    if kind == "norm":
        return {"q": _normed(s["q"], s["wq"], s).contiguous(), "k": _normed(s["k"], s["wk"], s).contiguous()}
    if kind == "grad":
        dq, dwq = _normed_back(s["gq"], s["q"], s["wq"], s)
        dk, dwk = _normed_back(s["gk"], s["k"], s["wk"], s)
        return {"dq": dq.contiguous(), "dk": dk.contiguous(), "dwq": dwq, "dwk": dwk}
    if kind == "nappend":
        at = _rows_of(s)
        s["k_cache"][at] = _normed(s["k"], s["wk"], s)
        s["v_cache"][at] = s["v"]
        return {"q": _normed(s["q"], s["wq"], s).contiguous(), "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    if kind == "append4":
        return _plain_append4(s)
    if kind in ("tree", "tree4"):
        S = min(c["cap"], c["ctx"] + c["Tq"])
        if kind == "tree4":
            return _plain_tree(s, _unpack(s["kc"][:, :, :S], s["ks"][:, :, :S], True),
                               _unpack(s["vc"][:, :, :S], s["vs"][:, :, :S], False))
        return _plain_tree(s, s["k_cache"][:, :, :S].float(), s["v_cache"][:, :, :S].float())
    return _plain_attention(s, kind == "train")


def _own(s, c, kind):
    import exact_attention_23_gb300 as fa
    if kind in ("norm", "grad", "nappend"):
        kw = dict(positions=s["positions"], interleaved=c["interleaved"], mscale=s["mscale"], eps=EPS)
        if kind == "norm":
            q, k = fa.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], **kw)
            return {"q": q, "k": k}
        if kind == "grad":
            dq, dk, dwq, dwk = fa.norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"],
                                                s["inv_freq"], **kw)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        q = fa.norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["k_cache"], s["v_cache"],
                                s["ctx_len"], s["inv_freq"], **kw)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if kind in ("append4", "tree4"):
        cache = fa.Cache4(s["kc"], s["ks"], s["vc"], s["vs"])
        if kind == "append4":
            fa.append4(s["k"], s["v"], cache, s["ctx_len"])
            k, v = fa.read4(cache, s["ctx_len"], c["Tq"])
            return {"k": k, "v": v}
        o, lse = fa.fwd_tree4(s["q"], cache, s["ctx_len"], tree=s["tree"], depths=s["depths"],
                              softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
                              sinks=c["sinks"])
        return {"o": o, "lse": lse}
    if kind == "tree":
        o, lse = fa.fwd_tree(s["q"], s["k_cache"], s["v_cache"], s["ctx_len"], tree=s["tree"],
                             depths=s["depths"], softcap=c["softcap"], slopes=s["slopes"],
                             window=c["window"], sinks=c["sinks"])
        return {"o": o, "lse": lse}
    seen = fa.visible(c["B"], c["T"], doc_ids=s.get("doc_ids"), window=c["window"], sinks=c["sinks"],
                      device=s["q"].device)
    rest = torch.empty_like(s["q"]) if kind == "train" else None
    o, lse = fa.fwd_mod(s["q"], s["k"], s["v"], visible=seen, softcap=c["softcap"],
                        slopes=s["slopes"], rest=rest)
    if kind == "fwd":
        return {"o": o, "lse": lse}
    dq, dk, dv = fa.bwd_mod(s["q"], s["k"], s["v"], o, lse, s["do"], visible=seen,
                            softcap=c["softcap"], slopes=s["slopes"], rest=rest)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------------------------- work

def _sees(i, window, sinks):
    """How many keys the token at place i of its document sees."""
    return min(i + 1, window) + min(sinks, max(0, i + 1 - window))


def work(case):
    c = case
    kind, B, H, Hkv, d = c["kind"], c["B"], c["H"], c["Hkv"], c["d"]
    if kind in ("norm", "grad"):
        rows = B * c["T"] * (H + Hkv)
        if kind == "norm":
            return {"bytes": rows * d * 4, "flops": rows * (4 * d + 3 * c["rot"])}
        return {"bytes": rows * d * 6, "flops": rows * (10 * d + 3 * c["rot"])}
    if kind == "nappend":
        rows = B * c["Tq"]
        return {"bytes": rows * (H + 2 * Hkv) * d * 4, "flops": rows * (H + Hkv) * (4 * d + 3 * c["rot"])}
    if kind == "append4":
        # rows read, written in 4 bits with a scale for 32, and given back
        rows = 2 * B * Hkv * c["Tq"]
        return {"bytes": rows * (d * 4 + d // 2 + d // 16), "flops": rows * d * 4}
    if kind in ("tree", "tree4"):
        n = c["Tq"]
        row = d + d // 8 if kind == "tree4" else d * 4  # K and V of one key
        keys = sum(min(L, c["window"] - 1 + c["sinks"]) if c["window"] else L for L in _lengths(B, c["ctx"])) + B * n
        return {"bytes": keys * Hkv * row + B * H * n * (d * 4 + 4), "flops": 4.0 * d * H * n * keys}
    T = c["T"]
    runs = _doc_lengths(T, c["docs"], c["pad"]) if c["docs"] else [T]
    pairs = sum(_sees(i, c["window"], c["sinks"]) for n in runs for i in range(n))
    q, kv = B * H * T * d * 2, B * Hkv * T * d * 2
    if kind == "fwd":
        return {"bytes": 2 * q + 2 * kv + B * H * T * 4, "flops": 4.0 * d * B * H * pairs}
    return {"bytes": 4 * q + 4 * kv + B * H * T * 4, "flops": 14.0 * d * B * H * pairs}


# --------------------------------------------------------------------------------- exact

def _exact_turn(y, positions, inv_freq, interleaved, mscale, inverse):
    """Rows in 64 bits turned as products of complex numbers."""
    rot = 2 * inv_freq.numel()
    pos = positions.double()
    angle = (pos if pos.dim() == 2 else pos.unsqueeze(0)).unsqueeze(-1) * inv_freq
    w = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle).unsqueeze(1)
    y = y.clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_norm(x, w):
    return x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w


def _exact_head(q, k, v, allowed, bias, softcap):
    """One head's (o, lse) in 64 bits, differentiable; rows that see nothing give 0 and −inf."""
    x = q @ k.T / math.sqrt(q.shape[1])
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if bias is not None:
        x = x + bias
    some = allowed.any(1)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    x = torch.where(allowed, x, torch.full((), -1e300, dtype=torch.float64, device=x.device))
    lse = torch.logsumexp(x, 1)
    w = torch.where(allowed & some[:, None], torch.exp(x - lse[:, None]), zero)
    return w @ v, torch.where(some, lse, torch.full_like(lse, -math.inf))


def _exact_rows4(x):
    """Rows as the 4-bit cache holds them, from the format's definition with powers of two in 64 bits."""
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top / torch.full_like(top, 7.0), torch.ones_like(top)))) - 4)
    scale = torch.ceil(top / step / torch.full_like(top, 7.0)) * step
    scale = torch.where(top < 2.0 ** -100, torch.zeros_like(scale), scale)
    n = torch.round(g / torch.where(scale > 0, scale, torch.ones_like(scale)))
    return (n * scale).flatten(-2)


def _exact_read4(codes, scales, keys):
    """A 4-bit cache's values in 64 bits, a dimension at a time."""
    d = 2 * codes.shape[-1]
    out = torch.empty((*codes.shape[:-1], d), dtype=torch.float64, device=codes.device)
    for at, dim in enumerate(_dims(d, keys)):
        n = (codes[..., at // 2] >> (4 * (at % 2))) & 15
        out[..., dim] = (n.double() - 8.0) * scales[..., dim // 32].double()
    return out


def _exact_allowed(c):
    T = c["T"]
    allowed = torch.zeros((T, T), dtype=torch.bool, device="cuda")
    at = 0
    for n in (_doc_lengths(T, c["docs"], c["pad"]) if c["docs"] else [T]):
        block = torch.ones((n, n), dtype=torch.bool, device="cuda").tril().triu(1 - c["window"])
        block[:, :c["sinks"]] = True
        allowed[at:at + n, at:at + n] = block.tril()
        at += n
    return allowed


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    kind, B, H, Hkv, d = c["kind"], c["B"], c["H"], c["Hkv"], c["d"]
    if kind in ("norm", "grad", "nappend"):
        turn = lambda y, back: _exact_turn(y, s["positions"], s["inv_freq"], c["interleaved"],
                                           s["mscale"], back)
        if kind == "grad":
            out = {}
            for x in ("q", "k"):
                rows = s[x].double().requires_grad_(True)
                w = s["w" + x].double().requires_grad_(True)
                with torch.enable_grad():
                    _exact_norm(rows, w).backward(turn(s["g" + x].double(), True))
                out["d" + x], out["dw" + x] = rows.grad, w.grad
            return {n: out[n] for n in ("dq", "dk", "dwq", "dwk")}
        q, k = (turn(_exact_norm(s[x].double(), s["w" + x].double()), False) for x in ("q", "k"))
        if kind == "norm":
            return {"q": q, "k": k}
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, at in enumerate(_lengths(B, c["ctx"])):
            kc[b, :, at:at + c["Tq"]] = k[b]
            vc[b, :, at:at + c["Tq"]] = s["v"][b].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if kind == "append4":
        return {"k": _exact_rows4(s["k"]), "v": _exact_rows4(s["v"])}
    G = H // Hkv
    if kind in ("tree", "tree4"):
        n = c["Tq"]
        if kind == "tree4":
            k_all, v_all = _exact_read4(s["kc"], s["ks"], True), _exact_read4(s["vc"], s["vs"], False)
        else:
            k_all, v_all = s["k_cache"], s["v_cache"]
        o = torch.zeros((B, H, n, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, H, n), dtype=torch.float64, device="cuda")
        for b, at in enumerate(_lengths(B, c["ctx"])):
            drafts = (s["tree"][b].bool() if s["tree"] is not None
                      else torch.ones((n, n), dtype=torch.bool, device="cuda").tril())
            allowed = torch.cat((torch.ones((n, at), dtype=torch.bool, device="cuda"), drafts), 1)
            depth = (s["depths"][b].double() if s["depths"] is not None
                     else torch.arange(n, dtype=torch.float64, device="cuda"))
            place = torch.cat((torch.arange(at, dtype=torch.float64, device="cuda"), depth + at))
            behind = depth[:, None] + at - place[None, :]
            if c["window"]:
                allowed &= (behind < c["window"]) | (place < c["sinks"])[None]
            for h in range(H):
                bias = -behind.abs() * s["slopes"][h].double() if s["slopes"] is not None else None
                o[b, h], lse[b, h] = _exact_head(s["q"][b, h].double(), k_all[b, h // G, :at + n].double(),
                                                 v_all[b, h // G, :at + n].double(), allowed, bias,
                                                 c["softcap"])
        return {"o": o, "lse": lse}
    T, train = c["T"], kind == "train"
    if (14.0 if train else 4.0) * d * B * H * T * T > 6e12:
        return None
    q, k, v = (s[x].double().requires_grad_(train) for x in ("q", "k", "v"))
    os, lses, allowed = [], [], _exact_allowed(c)
    place = torch.arange(T, dtype=torch.float64, device="cuda")
    gap = -(place[:, None] - place[None, :]).abs() if s["slopes"] is not None else None
    for b in range(B):
        for h in range(H):
            bias = gap * s["slopes"][h].double() if gap is not None else None
            qh, kh, vh = q[b, h], k[b, h // G], v[b, h // G]
            with torch.set_grad_enabled(train):
                oh, lh = _exact_head(qh, kh, vh, allowed, bias, c["softcap"])
                if train:
                    oh.backward(s["do"][b, h].double())
            os.append(oh.detach())
            lses.append(lh.detach())
            del oh, lh
    out = {"o": torch.stack(os).view(B, H, T, d), "lse": torch.stack(lses).view(B, H, T)}
    if train:
        out |= {"dq": q.grad, "dk": k.grad, "dv": v.grad}
    return out
