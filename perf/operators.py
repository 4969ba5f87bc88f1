"""Cases and plain forms of the rotary, modified-score and cached-tree operators.

Five kinds of case, each one pass through one operator as a program calls it:

  rope    rotary positions on the queries and keys of a packed projection, or (``grad``) the
          same rotation taken back on their gradients
  append  a serving step's new rows: queries and keys rotated at their positions, keys and
          values written into the cache behind each sequence's context
  fwd     attention with modified scores (a tanh cap, a bias by distance, documents, a prefix)
  train   the same with its gradients: o, lse, dq, dk, dv from q, k, v and do
  tree    new tokens (one, a chain, or a tree of drafts) against a cache with a context length
          of its own for each sequence

``run`` computes them in elementary torch operations in 32 bits (angles in 64), rounded once at
the end, or, where ``own`` is true, through exact_attention_23_gb300.
"""

import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # rotary positions of a training step at the repository's GPT-2 shape: queries and keys
        # read out of the packed projection [B, T, 3·H·d]
        {"name": "rope_b4_h12_t1024_d64", "kind": "rope", "B": 4, "H": 12, "Hkv": 12, "T": 1024,
         "d": 64, "rot": 64, "interleaved": False, "grad": False, "start": 0, "factor": 1.0},
        # the way back on a long sequence with shared key heads, half of each head rotated, the
        # interleaved layout, angles stretched by 8 for a long context
        {"name": "rope_grad_b1_h16_kv4_t16384_d128", "kind": "rope", "B": 1, "H": 16, "Hkv": 4,
         "T": 16384, "d": 128, "rot": 64, "interleaved": True, "grad": True, "start": 100000,
         "factor": 8.0},
        # one new token for each of eight sequences: pure latency
        {"name": "append_b8_h16_kv4_n1_d128", "kind": "append", "B": 8, "H": 16, "Hkv": 4, "Tq": 1,
         "ctx": 1000, "cap": 1280, "d": 128, "rot": 128, "interleaved": False, "factor": 1.0},
        # sixteen drafted tokens for each of sixteen sequences
        {"name": "append_b16_h12_n16_d64", "kind": "append", "B": 16, "H": 12, "Hkv": 12, "Tq": 16,
         "ctx": 700, "cap": 1024, "d": 64, "rot": 32, "interleaved": True, "factor": 4.0},
        # the smallest forward: a short prompt, latency
        {"name": "fwd_cap_b1_h2_t256_d64", "kind": "fwd", "B": 1, "H": 2, "Hkv": 2, "T": 256,
         "d": 64, "causal": True, "softcap": 30.0, "slopes": False, "docs": 0, "prefix": 0,
         "pad": 0},
        # a long prompt, capped scores, causal
        {"name": "fwd_cap_b1_h12_t16384_d64", "kind": "fwd", "B": 1, "H": 12, "Hkv": 12,
         "T": 16384, "d": 64, "causal": True, "softcap": 50.0, "slopes": False, "docs": 0,
         "prefix": 0, "pad": 0},
        # a training step on packed documents with a distance bias: ragged length, padded end
        {"name": "train_docs_bias_b2_h12_t1000_d64", "kind": "train", "B": 2, "H": 12, "Hkv": 12,
         "T": 1000, "d": 64, "causal": True, "softcap": 0.0, "slopes": True, "docs": 7,
         "prefix": 0, "pad": 23},
        # a training step with a prompt that sees all of itself (prefix mask)
        {"name": "train_prefix_b4_h12_t2048_d64", "kind": "train", "B": 4, "H": 12, "Hkv": 12,
         "T": 2048, "d": 64, "causal": True, "softcap": 0.0, "slopes": False, "docs": 0,
         "prefix": 700, "pad": 0},
        # a long packed sequence, shared key heads, wide heads, capped scores
        {"name": "train_cap_docs_b1_h16_kv4_t8192_d128", "kind": "train", "B": 1, "H": 16,
         "Hkv": 4, "T": 8192, "d": 128, "causal": True, "softcap": 30.0, "slopes": False,
         "docs": 5, "prefix": 0, "pad": 0},
        # single-token decoding over ragged contexts, capped scores
        {"name": "tree_one_b8_h12_ctx1000_d64", "kind": "tree", "B": 8, "H": 12, "Hkv": 12,
         "Tq": 1, "ctx": 1000, "cap": 1100, "d": 64, "drafts": False, "softcap": 30.0,
         "slopes": False},
        # sixteen drafts each over long contexts, shared key heads, wide heads
        {"name": "tree_n16_b4_h16_kv4_ctx16384_d128", "kind": "tree", "B": 4, "H": 16, "Hkv": 4,
         "Tq": 16, "ctx": 16384, "cap": 16500, "d": 128, "drafts": True, "softcap": 0.0,
         "slopes": False},
        # a wide tree over middling contexts with a distance bias: 256 rows a key head
        {"name": "tree_n64_b8_h16_kv4_ctx4096_d64", "kind": "tree", "B": 8, "H": 16, "Hkv": 4,
         "Tq": 64, "ctx": 4096, "cap": 4200, "d": 64, "drafts": True, "softcap": 0.0,
         "slopes": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "fwd", "fwd", "train", "train", "tree", "tree"])
    d = rng.choice([64, 128])
    H, Hkv = rng.choice([(12, 12), (16, 4), (8, 8), (6, 2), (16, 16), (8, 1), (5, 5)])
    factor = rng.choice([1.0, 1.0, 4.0, 8.0])
    rot = rng.choice([d, d // 2, d // 4, d])
    if kind == "rope":
        return {"kind": kind, "B": rng.choice([1, 2, 3]), "H": H, "Hkv": Hkv,
                "T": _log(rng, 16, 5000), "d": d, "rot": rot, "interleaved": rng.random() < 0.5,
                "grad": rng.random() < 0.5, "start": rng.choice([0, 17, 100000, 1000000]),
                "factor": factor}
    if kind == "append":
        ctx, n = _log(rng, 4, 1500), _log(rng, 1, 40)
        return {"kind": kind, "B": _log(rng, 1, 24), "H": H, "Hkv": Hkv, "Tq": n, "ctx": ctx,
                "cap": ctx + n + rng.randrange(40), "d": d, "rot": rot,
                "interleaved": rng.random() < 0.5, "factor": factor}
    if kind == "tree":
        ctx = _log(rng, 16, 16000)
        n = rng.choice([1, 1, 2, 5, 8, 16, 31, 64, 100])
        B = max(1, min(_log(rng, 1, 16), 60000 // ctx))
        return {"kind": kind, "B": B, "H": H, "Hkv": Hkv, "Tq": n, "ctx": ctx,
                "cap": ctx + n + rng.randrange(100), "d": d, "drafts": rng.random() < 0.7,
                "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]), "slopes": rng.random() < 0.3}
    T = _log(rng, 40, 2900 if kind == "train" else 6000)
    B = max(1, min(rng.choice([1, 2, 3, 4]), 5000 // T))
    docs = rng.choice([0, 0, 3, 9])
    causal = rng.random() < 0.8
    return {"kind": kind, "B": B, "H": H, "Hkv": Hkv, "T": T, "d": d, "causal": causal,
            "softcap": rng.choice([0.0, 20.0, 50.0]), "slopes": rng.random() < 0.4, "docs": docs,
            "prefix": rng.choice([0, 0, T // 3]) if causal else 0,
            "pad": T // 20 if docs else 0}


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


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    s = {"c": c}
    if c["kind"] == "rope":
        T = c["T"]
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"])
        s["mscale"] = 0.1 * math.log(c["factor"]) + 1.0
        s["positions"] = (torch.arange(T, device="cuda", dtype=torch.int32) + c["start"])
        if c["grad"]:
            s["q"], s["k"] = _randn((B, H, T, d), g), _randn((B, Hkv, T, d), g)
        else:
            packed = _randn((B, T, H + 2 * Hkv, d), g)
            s["q"] = packed[:, :, :H].transpose(1, 2)
            s["k"] = packed[:, :, H:H + Hkv].transpose(1, 2)
        return s
    if c["kind"] == "append":
        n = c["Tq"]
        packed = _randn((B, n, H + 2 * Hkv, d), g)
        s["q"] = packed[:, :, :H].transpose(1, 2)
        s["k"] = packed[:, :, H:H + Hkv].transpose(1, 2)
        s["v"] = packed[:, :, H + Hkv:].transpose(1, 2)
        s["k_cache"], s["v_cache"] = (_randn((B, Hkv, c["cap"], d), g) for _ in range(2))
        s["ctx_len"] = torch.tensor(_lengths(B, c["ctx"]), dtype=torch.int32, device="cuda")
        s["positions"] = (s["ctx_len"][:, None] + _tree(B, n, g)[1]).contiguous()
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"])
        s["mscale"] = 0.1 * math.log(c["factor"]) + 1.0
        return s
    s["slopes"] = _slopes(H) if c["slopes"] else None
    # capped models have scores that reach the cap's bend; the others are of unit variance
    std = 4.0 if c["softcap"] else 1.0
    if c["kind"] == "tree":
        n = c["Tq"]
        s["q"] = _randn((B, H, n, d), g, std)
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
    if c["prefix"]:
        s["prefix_len"] = torch.full((B,), c["prefix"], dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

def _rotate(x, positions, inv_freq, interleaved, mscale, inverse):
    rot = 2 * inv_freq.numel()
    pos = positions if positions.dim() == 2 else positions[None]
    angle = pos[:, None, :, None].double() * inv_freq
    cos, sin = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    if inverse:
        sin = -sin
    xf = x.float()
    a, b = ((xf[..., 0:rot:2], xf[..., 1:rot:2]) if interleaved
            else (xf[..., :rot // 2], xf[..., rot // 2:rot]))
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = (torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1))
    return torch.cat((turned, xf[..., rot:]), -1).to(x.dtype)


def _seen(s, T, B, causal):
    """[B, 1, 1, T, T] truth values: query i sees key j."""
    i = torch.arange(T, device="cuda")[:, None]
    j = torch.arange(T, device="cuda")[None, :]
    ids = s.get("doc_ids")
    if ids is None:
        start = torch.zeros((B, T), dtype=torch.int64, device="cuda")
        same = torch.ones((1, 1, 1), dtype=torch.bool, device="cuda")
    else:
        first = torch.cat((torch.ones_like(ids[:, :1], dtype=torch.bool),
                           ids[:, 1:] != ids[:, :-1]), 1)
        run = first.long().cumsum(1)
        start = (torch.arange(T, device="cuda") * first).cummax(1).values
        same = (run[:, :, None] == run[:, None, :]) & (ids >= 0)[:, :, None]
    if not causal:
        return same.expand(B, T, T)[:, None, None]
    ok = (j <= i)[None]
    prefix = s.get("prefix_len")
    if prefix is not None:
        ok = ok | (j[None] < start[:, :, None] + prefix[:, None, None])
    return (ok & same).expand(B, T, T)[:, None, None]


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
    G = H // Hkv
    qg = s["q"].float().view(B, Hkv, G, T, d)
    kf, vf = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    at = torch.arange(T, device="cuda", dtype=torch.float32)
    z, bend = _scores(qg, kf, c, _seen(s, T, B, c["causal"]), lambda: (at[:, None] - at).abs(),
                      s["slopes"], bend=grads)
    p, lse = _softmax(z)
    del z
    o = torch.matmul(p, vf)
    out = {"o": o.view(B, H, T, d).to(BF16), "lse": lse.reshape(B, H, T)}
    if grads:
        do = s["do"].float().view(B, Hkv, G, T, d)
        out["dv"] = torch.matmul(p.transpose(-1, -2), do).sum(2).to(BF16)
        ds = torch.matmul(do, vf.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)
        ds = ds * p
        if bend is not None:
            ds = ds * bend
        ds = ds * (1.0 / math.sqrt(d))
        out["dq"] = torch.matmul(ds, kf).view(B, H, T, d).to(BF16)
        out["dk"] = torch.matmul(ds.transpose(-1, -2), qg).sum(2).to(BF16)
    return out


def _plain_tree(s):
    c = s["c"]
    B, H, Hkv, n, d = c["B"], c["H"], c["Hkv"], c["Tq"], c["d"]
    S = min(c["cap"], c["ctx"] + n)
    qg = s["q"].float().view(B, Hkv, H // Hkv, n, d)
    kf, vf = s["k_cache"][:, :, :S].float()[:, :, None], s["v_cache"][:, :, :S].float()[:, :, None]
    ctx = s["ctx_len"].long()[:, None, None]
    j = torch.arange(S, device="cuda")[None, None, :]
    t = torch.arange(n, device="cuda")
    tree = s["tree"].bool() if s["tree"] is not None else (t[None, :] <= t[:, None]).expand(B, n, n)
    depth = s["depths"].long() if s["depths"] is not None else t.expand(B, n)
    draft = (j - ctx).clamp(0, n - 1)                                     # [B, 1, S]
    in_tree = torch.gather(tree, 2, draft.expand(B, n, S)) & (j >= ctx) & (j < ctx + n)
    seen = ((j < ctx) | in_tree)[:, None, None]
    key_at = torch.where(j < ctx, j.expand(B, 1, S), ctx + torch.gather(depth, 1, draft[:, 0])[:, None])
    z, _ = _scores(qg, kf, c, seen,
                   lambda: (ctx + depth[:, :, None] - key_at).abs().float()[:, None, None],
                   s["slopes"])
    p, lse = _softmax(z)
    return {"o": torch.matmul(p, vf).view(B, H, n, d).to(BF16), "lse": lse.reshape(B, H, n)}


def _plain_append(s):
    c = s["c"]
    q = _rotate(s["q"], s["positions"], s["inv_freq"], c["interleaved"], s["mscale"], False)
    k = _rotate(s["k"], s["positions"], s["inv_freq"], c["interleaved"], s["mscale"], False)
    b = torch.arange(c["B"], device="cuda")[:, None, None]
    h = torch.arange(c["Hkv"], device="cuda")[None, :, None]
    row = s["ctx_len"].long()[:, None, None] + torch.arange(c["Tq"], device="cuda")
    s["k_cache"][b, h, row] = k
    s["v_cache"][b, h, row] = s["v"]
    return {"q": q.contiguous(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    s, c = state, state["c"]
    if own:
        import exact_attention_23_gb300 as fa
        if c["kind"] == "rope":
            q, k = fa.rope(s["q"], s["k"], s["inv_freq"], positions=s["positions"],
                           interleaved=c["interleaved"], inverse=c["grad"], mscale=s["mscale"])
            return {"q": q, "k": k}
        if c["kind"] == "append":
            q = fa.rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["ctx_len"],
                               s["inv_freq"], positions=s["positions"],
                               interleaved=c["interleaved"], mscale=s["mscale"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if c["kind"] == "tree":
            o, lse = fa.fwd_tree(s["q"], s["k_cache"], s["v_cache"], s["ctx_len"], tree=s["tree"],
                                 depths=s["depths"], softcap=c["softcap"], slopes=s["slopes"])
            return {"o": o, "lse": lse}
        seen = None
        if c["docs"] or c["prefix"]:
            seen = fa.visible(c["B"], c["T"], causal=c["causal"], doc_ids=s.get("doc_ids"),
                              prefix_len=s.get("prefix_len"), device=s["q"].device)
        rest = torch.empty_like(s["q"]) if c["kind"] == "train" else None
        o, lse = fa.fwd_mod(s["q"], s["k"], s["v"], visible=seen, causal=c["causal"],
                            softcap=c["softcap"], slopes=s["slopes"], rest=rest)
        if c["kind"] == "fwd":
            return {"o": o, "lse": lse}
        dq, dk, dv = fa.bwd_mod(s["q"], s["k"], s["v"], o, lse, s["do"], visible=seen,
                                causal=c["causal"], softcap=c["softcap"], slopes=s["slopes"],
                                rest=rest)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if c["kind"] == "rope":
        return {x: _rotate(s[x], s["positions"], s["inv_freq"], c["interleaved"], s["mscale"],
                           c["grad"]).contiguous() for x in ("q", "k")}
    if c["kind"] == "append":
        return _plain_append(s)
    if c["kind"] == "tree":
        return _plain_tree(s)
    return _plain_attention(s, c["kind"] == "train")


# ---------------------------------------------------------------------------------- work

def work(case):
    c = case
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] == "rope":
        rows = B * c["T"] * (H + Hkv)
        return {"bytes": rows * d * 4, "flops": rows * c["rot"] * 3}
    if c["kind"] == "append":
        rows = B * c["Tq"]
        return {"bytes": rows * (H + 2 * Hkv) * d * 4, "flops": rows * (H + Hkv) * c["rot"] * 3}
    if c["kind"] == "tree":
        n = c["Tq"]
        keys = sum(_lengths(B, c["ctx"])) + B * n
        return {"bytes": keys * Hkv * d * 4 + B * H * n * (d * 4 + 4),
                "flops": 4.0 * d * H * n * keys}
    T = c["T"]
    runs = _doc_lengths(T, c["docs"], c["pad"]) if c["docs"] else [T]
    if c["causal"]:
        pairs = sum(n * (n + 1) // 2 + min(n, c["prefix"]) * max(0, min(n, c["prefix"]) - 1) // 2
                    for n in runs)
    else:
        pairs = sum(n * n for n in runs)
    q, kv = B * H * T * d * 2, B * Hkv * T * d * 2
    if c["kind"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + B * H * T * 4, "flops": 4.0 * d * B * H * pairs}
    return {"bytes": 4 * q + 4 * kv + B * H * T * 4, "flops": 14.0 * d * B * H * pairs}


# --------------------------------------------------------------------------------- exact

def _exact_rotate(x, positions, inv_freq, interleaved, mscale, inverse):
    """The rotation as a product of complex numbers in 64 bits."""
    rot = 2 * inv_freq.numel()
    pos = positions.double()
    angle = (pos if pos.dim() == 2 else pos.unsqueeze(0)).unsqueeze(-1) * inv_freq
    w = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle).unsqueeze(1)
    y = x.double().clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_head(q, k, v, allowed, bias, softcap):
    """One head's (o, lse) in 64 bits, differentiable; rows that see nothing give 0 and −inf."""
    x = q @ k.T / math.sqrt(q.shape[1])
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if bias is not None:
        x = x + bias
    some = allowed.any(1)
    x = torch.where(allowed, x, torch.full((), -1e300, dtype=torch.float64, device=x.device))
    lse = torch.logsumexp(x, 1)
    w = torch.where(allowed, torch.exp(x - lse[:, None]), torch.zeros((), dtype=torch.float64, device=x.device))
    w = torch.where(some[:, None], w, torch.zeros((), dtype=torch.float64, device=x.device))
    return w @ v, torch.where(some, lse, torch.full_like(lse, -math.inf))


def _exact_allowed(c):
    T = c["T"]
    allowed = torch.zeros((T, T), dtype=torch.bool, device="cuda")
    at = 0
    for n in (_doc_lengths(T, c["docs"], c["pad"]) if c["docs"] else [T]):
        block = torch.ones((n, n), dtype=torch.bool, device="cuda")
        if c["causal"]:
            block = block.tril()
            block[:, :min(n, c["prefix"])] = True
        allowed[at:at + n, at:at + n] = block
        at += n
    return allowed


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] == "rope":
        return {x: _exact_rotate(s[x], s["positions"], s["inv_freq"], c["interleaved"],
                                 s["mscale"], c["grad"]) for x in ("q", "k")}
    if c["kind"] == "append":
        q, k = (_exact_rotate(s[x], s["positions"], s["inv_freq"], c["interleaved"], s["mscale"],
                              False) for x in ("q", "k"))
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, at in enumerate(_lengths(B, c["ctx"])):
            kc[b, :, at:at + c["Tq"]] = k[b]
            vc[b, :, at:at + c["Tq"]] = s["v"][b].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    G = H // Hkv
    if c["kind"] == "tree":
        n = c["Tq"]
        o = torch.zeros((B, H, n, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, H, n), dtype=torch.float64, device="cuda")
        for b, at in enumerate(_lengths(B, c["ctx"])):
            drafts = (s["tree"][b].bool() if s["tree"] is not None
                      else torch.ones((n, n), dtype=torch.bool, device="cuda").tril())
            allowed = torch.cat((torch.ones((n, at), dtype=torch.bool, device="cuda"), drafts), 1)
            depth = (s["depths"][b].double() if s["depths"] is not None
                     else torch.arange(n, dtype=torch.float64, device="cuda"))
            place = torch.cat((torch.arange(at, dtype=torch.float64, device="cuda"), depth + at))
            gap = -(depth[:, None] + at - place[None, :]).abs()
            for h in range(H):
                bias = gap * s["slopes"][h].double() if s["slopes"] is not None else None
                o[b, h], lse[b, h] = _exact_head(
                    s["q"][b, h].double(), s["k_cache"][b, h // G, :at + n].double(),
                    s["v_cache"][b, h // G, :at + n].double(), allowed, bias, c["softcap"])
        return {"o": o, "lse": lse}
    T, train = c["T"], c["kind"] == "train"
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
