"""Cases of the operators around the verify of drafted trees in a serving
step: norms of queries and keys with the position rotation, append to and
attention over a cache held in 8 bits, and the verify of a tree against the
target's probabilities.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare` makes a case's inputs on the GPU, `run` makes one pass (the plain
form, or with `own` the library's calls), `exact` is the definition in 64
bits and `work` what a pass cannot do without.

Head layouts are those of the repository's model pair (28 query and 4 KV
heads of 128 for the target, 14 and 2 of 64 for its draft) and generic ones;
vocabularies are its 152064 and 151936.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}          # the largest code of each kind
LEAST, MOST = 2.0 ** -50, 2.0 ** 50         # of a scale that is not 0
EPS = 1e-6                                  # of the norms


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One token of the draft model (no norms) at a far position: latency, once a layer and draft step.
        dict(name="rope_token", kind="rope", N=1, hq=14, hkv=2, D=64, R=64, norm=False, pairs=False, far=131000,
             dtype="bf16"),
        # The nodes of 32 chains of 9: the ordinary verify forward.
        dict(name="rope_chains", kind="rope", N=288, hq=16, hkv=8, D=128, R=64, norm=True, pairs=True, far=16384,
             dtype="f16"),
        # A batch of prompts, queries and keys inside one projection's output: the largest.
        dict(name="rope_prompts", kind="rope", N=16411, hq=28, hkv=4, D=128, R=128, norm=True, pairs=False, far=32768,
             dtype="bf16"),
        # The tokens that a verify kept of 32 trees, appended to int8 blocks that are in part full.
        dict(name="append_kept", kind="append", B=32, T=16, kept=6, hkv=4, D=128, lo=5000, hi=16384, page=16, block=16,
             code="i8", dtype="bf16"),
        # Prompts appended after their prefill, e4m3 with larger blocks.
        dict(name="append_prompts", kind="append", B=8, T=4099, kept=0, hkv=8, D=128, lo=0, hi=100, page=64, block=64,
             code="e4m3", dtype="f16"),
        # One token of the draft model, one request: the call whose latency a draft step waits for.
        dict(name="qattn_token", kind="attention", B=1, T=1, tree=False, hq=14, hkv=2, D=64, lo=517, hi=517, page=16,
             block=16, window=0, sinks=0, code="i8", dtype="bf16"),
        # A verify forward of 32 requests with a chain of 8 drafts each over an e4m3 cache.
        dict(name="qattn_chain_batch", kind="attention", B=32, T=9, tree=False, hq=28, hkv=4, D=128, lo=500, hi=16384,
             page=32, block=32, window=0, sinks=0, code="e4m3", dtype="bf16"),
        # Ragged trees in fp16 through a window with sinks, contexts from one slot to thirty thousand.
        dict(name="qattn_window", kind="attention", B=23, T=21, tree=True, hq=16, hkv=8, D=128, lo=1, hi=30001, page=16,
             block=16, window=4099, sinks=5, code="i8", dtype="f16"),
        # Trees of 64 nodes over long contexts: the largest verify forward.
        dict(name="qattn_tree_long", kind="attention", B=16, T=64, tree=True, hq=28, hkv=4, D=128, lo=16384, hi=32768,
             page=64, block=64, window=0, sinks=0, code="i8", dtype="bf16"),
        # One request with a sampled tree of 16 nodes: latency.
        dict(name="sample_single", kind="sample", B=1, T=16, V=151936, drafts="again"),
        # 64 requests, children drawn without replacement.
        dict(name="sample_batch", kind="sample", B=64, T=20, V=152064, drafts="once"),
        # 48 requests whose trees come from a beam: no draft probabilities.
        dict(name="sample_beams", kind="sample", B=48, T=20, V=152064, drafts="beam"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attention", "attention", "sample"])
    c = {"kind": kind}
    if kind != "sample":
        c["hq"], c["hkv"], c["D"] = rng.choice([(14, 2, 64), (28, 4, 128), (16, 8, 128), (8, 8, 64), (32, 8, 128)])
        c["dtype"] = rng.choice(["bf16", "f16"])
    if kind == "rope":
        c["N"] = _log(rng, 1, 14000)
        c["R"] = rng.choice([c["D"], c["D"] // 2, 16])
        c["norm"], c["pairs"] = rng.random() < 0.7, rng.random() < 0.4
        c["far"] = _log(rng, 16, 1000000)
        return c
    if kind == "sample":
        c["B"], c["T"] = _log(rng, 1, 64), _log(rng, 1, 20)
        c["V"] = rng.choice([151936, 152064, _log(rng, 1000, 152064)])
        c["drafts"] = rng.choice(["again", "once", "beam"])
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    c["block"] = rng.choice([b for b in (16, 32, 64, 128) if b <= c["page"]])
    c["code"] = rng.choice(["i8", "e4m3"])
    c["B"] = _log(rng, 1, 32)
    if kind == "append":
        del c["hq"]
        c["kept"] = rng.choice([0, rng.randint(1, 9)])
        c["T"] = _log(rng, c["kept"], 64) if c["kept"] else _log(rng, 1, max(1, 32000 // c["B"] // c["hkv"] * 4))
        c["hi"] = _log(rng, 1, 8192)
        c["lo"] = rng.randint(0, c["hi"])
        return c
    c["T"] = _log(rng, 1, 64)
    c["tree"] = rng.random() < 0.6
    c["hi"] = _log(rng, 16, max(16, min(32768, (100000 if c["hkv"] == 8 else 200000) // c["B"])))
    c["lo"] = rng.randint(1, c["hi"])
    c["window"] = rng.choice([0, _log(rng, 1, 8192)])
    c["sinks"] = rng.randint(0, 9) if c["window"] else 0
    return c


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _lens(lo, hi, n):
    """n lengths over [lo, hi], in no order; the same for every seed of a case."""
    return [lo + (((i * 37 + 3) % n) * (hi - lo)) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _nodes(case):
    """Nodes (or new tokens) of each request: the full number for most, fewer for some."""
    T, B = case["T"], case["B"]
    return [T if b % 3 != 2 else max(1, T - (b * 5) % T) for b in range(B)]


def _paths(case):
    """Number of nodes kept of each request's tree (root and accepted nodes)."""
    return [min(n, 1 + (b * 3 + case["kept"] - 1) % case["kept"]) for b, n in enumerate(_nodes(case))]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _parents(np_rng, n, kids=None):
    """A drafted tree: node 0 the root, each node's parent among the few before it."""
    up, count = [-1], [0] * n
    for i in range(1, n):
        free = [j for j in range(max(0, i - 6), i) if kids is None or count[j] < kids]
        up.append(free[int(np_rng.randint(len(free)))])
        count[up[-1]] += 1
    return up


def _codes(x, scale, code):
    """fp32 values as codes of their scales (nearest, ties to even)."""
    x = x * torch.where(scale > 0, 1.0 / scale, 0.0)
    x = x.clamp(-TOP[code], TOP[code])
    return x.round().to(torch.int8) if code == "i8" else x.to(torch.float8_e4m3fn)


def _scale(amax, code):
    """A block's scale for its largest magnitude, in fp32."""
    s = (amax / torch.full_like(amax, TOP[code])).clamp(LEAST, MOST)
    return torch.where(amax > 0, s, 0.0)


def _cache(case, g, room):
    """Pool of pages in codes with their scales, and each request's table: pages in no order, some unused."""
    B, page, H, D, block = case["B"], case["page"], case["hkv"], case["D"], case["block"]
    per = -(-(case["hi"] + room) // page)
    pool = B * per + 3
    table = torch.randperm(pool, generator=g, device="cuda")[: B * per].reshape(B, per).to(torch.int32)
    got = []
    for _ in range(2):
        # magnitudes of heads and stretches of tokens differ
        x = _randn(g, (pool, H, page // block, block, D), torch.float32)
        x *= torch.exp(torch.randn((pool, H, page // block, 1, 1), generator=g, device="cuda") * 0.3)
        s = _scale(x.abs().amax((3, 4)), case["code"])
        got += [_codes(x, s[..., None, None], case["code"]).reshape(pool, H, page, D), s]
    return got[0], got[2], got[1], got[3], table


def prepare(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    kind, s = case["kind"], {"case": case}
    if kind == "rope":
        N, hq, hkv, D, dt = case["N"], case["hq"], case["hkv"], case["D"], DTYPES[case["dtype"]]
        x = _randn(g, (N, hq + 2 * hkv, D), dt, 1.7)      # a projection's output: queries, keys, values
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hkv]
        s["positions"] = torch.randint(0, case["far"], (N,), generator=g, device="cuda").to(torch.int32)
        j = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = (1e6 ** (-2.0 * j / case["R"])).float()
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if case["norm"] else None
        return s
    B, nodes = case["B"], _nodes(case)
    N = sum(nodes)
    s["offsets"], s["max_nodes"] = _ints(np.cumsum([0] + nodes)), case["T"]
    # row and place of each node in the padded [B][T] grid of the plain forms
    s["row"] = torch.tensor(np.repeat(np.arange(B), nodes), device="cuda")
    s["col"] = torch.tensor(np.concatenate([np.arange(n) for n in nodes]), device="cuda")
    if kind == "sample":
        return _prepare_sample(case, s, g, r, nodes)
    D, H, dt = case["D"], case["hkv"], DTYPES[case["dtype"]]
    lens = _lens(case["lo"], case["hi"], B)
    s["lens"] = _ints(lens)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"] = _cache(
        case, g, case["T"] if kind == "append" else 0)
    s["k_new"], s["v_new"] = _randn(g, (N, H, D), dt), _randn(g, (N, H, D), dt)
    if kind == "append":
        s["out_lens"] = torch.zeros_like(s["lens"])
        s["path"] = s["path_lens"] = None
        if case["kept"]:
            path = np.full((B, case["T"]), -1, dtype=np.int32)
            for b, (n, m) in enumerate(zip(nodes, _paths(case))):
                path[b, :m] = [0] + sorted(r.choice(np.arange(1, n), m - 1, replace=False).tolist()) if m > 1 else [0]
            s["path"], s["path_lens"] = _ints(path), _ints(_paths(case))
        return s
    s["q"] = _randn(g, (N, case["hq"], D), dt, 2.5)      # peaked softmaxes, as attention's are
    s["scale"] = 1.0 / math.sqrt(D)
    s["parents"] = _ints(np.concatenate([_parents(r, n) for n in nodes])) if case["tree"] else None
    return s


KIDS = 4


def _prepare_sample(case, s, g, r, nodes):
    """Target and draft rows that agree as a model pair's do, and trees whose children were drawn from the draft's
    rows (from the target's highest for a beam's)."""
    B, V, N = case["B"], case["V"], sum(nodes)
    ld = -(-V // 4) * 4
    parents = np.concatenate([_parents(r, n, KIDS) for n in nodes])
    z = torch.randn((N, ld), generator=g, device="cuda")[:, :V]
    p = torch.empty((N, ld), device="cuda")[:, :V]
    # vocabularies of a real row: few tokens carry most of the weight
    p.copy_(torch.softmax(z * 4.5, -1))
    q = torch.empty((N, ld), device="cuda")[:, :V]
    q.copy_(torch.softmax(z * 4.2 + 1.2 * torch.randn((N, V), generator=g, device="cuda"), -1))
    off = np.cumsum([0] + nodes)
    first = np.repeat(off[:-1], nodes)
    up = np.where(parents >= 0, parents + first, -1)
    k = min(KIDS, V)
    if case["drafts"] == "beam":
        drawn = (q + 1e-30).log().topk(k, -1).indices
    else:
        drawn = torch.multinomial(q, k, replacement=case["drafts"] == "again", generator=g)
    drawn = drawn.cpu().numpy()
    tokens, count = np.zeros(N, dtype=np.int64), np.zeros(N, dtype=np.int64)
    rank = np.zeros(N, dtype=np.int64)
    for i in range(N):
        if up[i] >= 0:
            tokens[i], rank[i] = drawn[up[i], count[up[i]]], count[up[i]]
            count[up[i]] += 1
    child = np.full((N, KIDS), -1, dtype=np.int64)
    on = up >= 0
    child[up[on], rank[on]] = np.arange(N)[on]
    s["p"], s["q"] = p, None if case["drafts"] == "beam" else q
    s["tokens"], s["parents"] = _ints(tokens), _ints(parents)
    s["child"], s["up"] = torch.tensor(child, device="cuda"), torch.tensor(up, device="cuda")
    s["u"] = torch.rand(N, generator=g, device="cuda")
    s["v"] = torch.rand(B, generator=g, device="cuda")
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _turned(s, x, w):
    c = s["case"]
    R = c["R"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()      # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["pairs"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


def _rope(s):
    return {"q": _turned(s, s["q"], s["wq"]), "k": _turned(s, s["k"], s["wk"])}


def _append_one(s, codes, scales, new, b, slot, lens):
    """Rows `new` appended to slots `slot` of requests `b`."""
    c = s["case"]
    page, block, code, H = c["page"], c["block"], c["code"], c["hkv"]
    per = page // block
    at, blk = s["table"][b, slot // page].long(), (slot % page) // block
    x = new.float()
    key = (at * per + blk)[:, None] * H + torch.arange(H, device="cuda")
    amax = torch.zeros(codes.shape[0] * per * H, device="cuda")
    amax.scatter_reduce_(0, key.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
    fresh = _scale(amax, code).reshape(-1, per, H).transpose(1, 2)
    # blocks that were in part full keep their scale where it suffices; where it grows, their codes are rounded again
    every = torch.arange(lens.shape[0], device="cuda")
    start = lens // block * block
    open_ = (lens > start) & torch.zeros_like(lens, dtype=torch.bool).index_fill_(0, b, True)
    here = s["table"][every, (start // page).clamp(max=s["table"].shape[1] - 1)].long()
    oblk = (start % page) // block
    old = torch.where(open_[:, None], scales[here, :, oblk], 0.0)
    grown = torch.maximum(old, fresh[here, :, oblk])
    j = torch.arange(block, device="cuda")
    place = (start % page)[:, None] + j
    was = codes[here[:, None], :, place]                                  # [B][block][H][D]
    again = _codes(was.float() * old[:, None, :, None], grown[:, None, :, None], code)
    turn = (open_[:, None] & (grown > old))[:, None, :, None] & ((start[:, None] + j) < lens[:, None])[..., None, None]
    raw = torch.int8 if code == "i8" else torch.uint8
    kept = torch.where(turn, again.view(raw), was.view(raw))
    store = codes.view(raw)
    on = open_.nonzero(as_tuple=True)[0]
    store[here[on, None], :, place[on]] = kept[on]
    touched = torch.zeros(codes.shape[0] * per * H, dtype=torch.bool, device="cuda")
    touched[key.reshape(-1)] = True
    scales.copy_(torch.where(touched.reshape(-1, per, H).transpose(1, 2), fresh, scales))
    scales[here[on], :, oblk[on]] = grown[on]
    store[at, :, slot % page] = _codes(x, scales[at, :, blk][..., None], code).view(raw)


def _append(s):
    c = s["case"]
    lens = s["lens"].long()
    if s["path"] is None:
        b, i, rows = s["row"], s["col"], slice(None)
        count = (s["offsets"][1:] - s["offsets"][:-1])
    else:
        on = torch.arange(c["T"], device="cuda") < s["path_lens"][:, None]
        b, i = on.nonzero(as_tuple=True)
        rows = s["offsets"][b].long() + s["path"][b, i].long()
        count = s["path_lens"]
    slot = lens[b] + i
    _append_one(s, s["k_cache"], s["k_scale"], s["k_new"][rows], b, slot, lens)
    _append_one(s, s["v_cache"], s["v_scale"], s["v_new"][rows], b, slot, lens)
    s["out_lens"].copy_(s["lens"] + count)
    # codes as they are held: whole numbers, or float8 values
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "out_lens")}


def _dense(s, codes, scales):
    """[B][Hkv][slots][D] of a request's pages in order, as fp32 values."""
    t, c = s["table"].long(), s["case"]
    x = codes[t].float().unflatten(3, (-1, c["block"])) * scales[t][..., None, None]
    B, P, H = x.shape[:3]
    return x.reshape(B, P, H, c["page"], -1).permute(0, 2, 1, 3, 4).reshape(B, H, P * c["page"], -1)


def _grid(s, x, fill=0):
    """Packed node rows in the padded [B][T] grid, `fill` elsewhere."""
    c = s["case"]
    out = torch.full((c["B"], c["T"]) + x.shape[1:], fill, dtype=x.dtype, device=x.device)
    out[s["row"], s["col"]] = x
    return out


def _grouped(s, x):
    """[B][T][Hq][D] as [B][Hkv][T * G][D]: the rows that share a KV head."""
    c = s["case"]
    B, T = x.shape[:2]
    x = x.reshape(B, T, c["hkv"], c["hq"] // c["hkv"], -1).permute(0, 2, 1, 3, 4)
    return x.reshape(B, c["hkv"], -1, x.shape[-1])


def _lineage(up, T):
    """[B][T][T]: which nodes are a node's ancestors or itself, from parents [B][T]."""
    a = (up[..., None] == torch.arange(T, device="cuda")) | torch.eye(T, device="cuda").bool()
    a = a.float()
    a = ((a @ a) > 0).float()          # paths of up to 2, 4, .. 64 steps
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    return (a @ a) > 0


def _attention(s):
    c = s["case"]
    B, T, hkv, D = c["B"], c["T"], c["hkv"], c["D"]
    G, n, W = c["hq"] // hkv, c["hi"], c["window"] or (1 << 31)
    k, v = (_dense(s, s[x + "_cache"], s[x + "_scale"])[:, :, :n] for x in "kv")
    kn, vn = (_grid(s, s[x].float()).transpose(1, 2) for x in ("k_new", "v_new"))
    q = _grouped(s, _grid(s, s["q"].float()))
    x = torch.cat([q @ k.transpose(2, 3), q @ kn.transpose(2, 3)], -1) * s["scale"]
    if s["parents"] is None:
        sees = torch.ones((T, T), device="cuda").tril().bool().expand(B, T, T)
    else:
        sees = _lineage(_grid(s, s["parents"].long(), -1), T)
    lens = s["lens"].long()[:, None]
    place = lens + sees.sum(-1) - 1                                      # [B][T] positions of the nodes
    at = torch.cat([torch.arange(n, device="cuda").expand(B, n), place], 1)
    near = (at[:, None] < c["sinks"]) | (place[..., None] - at[:, None] < W)
    there = torch.cat([(torch.arange(n, device="cuda") < lens)[:, None].expand(B, T, n), sees], -1) & near
    x.masked_fill_(~there[:, :, None].expand(B, T, G, n + T).reshape(B, 1, T * G, n + T), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x[..., :n] @ v + x[..., n:] @ vn) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.reshape(B, hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, c["hq"], D)
    lse = lse.reshape(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, c["hq"])
    return {"out": o[s["row"], s["col"]].to(s["q"].dtype), "lse": lse[s["row"], s["col"]]}


def _children(s, p, q, u):
    """The test of every node's children in order, in 64 bits (values next to a border): the child taken or -1, and
    what the draw after the last one needs: c (with draft rows), or the tokens left out."""
    c = s["case"]
    N = p.shape[0]
    every = torch.arange(N, device="cuda")
    taken = torch.full((N,), -1, dtype=torch.long, device="cuda")
    Z = torch.ones(N, dtype=torch.float64, device="cuda")
    cut, gone = torch.zeros_like(Z), torch.zeros_like(Z)
    out = torch.zeros((N, KIDS), dtype=torch.bool, device="cuda")
    token = torch.where(s["child"] >= 0, s["tokens"].long()[s["child"].clamp(min=0)], 0)
    for k in range(KIDS):
        on = (s["child"][:, k] >= 0) & (taken < 0)
        x, i = token[:, k], s["child"][:, k].clamp(min=0)
        px = p[every, x].double()
        if q is None:
            px = torch.where((out[:, :k] & (token[:, :k] == x[:, None])).any(-1), 0.0, px)
            yes = on & (u[i] * Z < px)
            no = on & ~yes
            Z = torch.where(no, Z - px, Z)
            out[:, k] = no
        else:
            qx = q[every, x].double()
            left = 1.0 - gone
            rate = torch.where(left > 0, 1.0 / left, 0.0) if c["drafts"] == "once" else torch.ones_like(left)
            yes = on & (u[i] * (qx * rate) * Z < (px - cut * qx).clamp(min=0))
            no = on & ~yes
            gone = torch.where(no, gone + qx, gone)
            cut = torch.where(no, cut + Z * rate, cut)
            Z = torch.where(no, (p.double() - cut[:, None] * q.double()).clamp(min=0).sum(-1), Z)
        taken = torch.where(yes, i, taken)
    return taken, cut, out, token


def _sample(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    p, q, u = s["p"], s["q"], s["u"].double()
    taken, cut, out, token = _children(s, p, q, u)
    # a node lies on the walk if it and all its ancestors are the child that their parents took
    ok = torch.where(s["up"] < 0, True, taken[s["up"].clamp(min=0)] == torch.arange(p.shape[0], device="cuda"))
    bad = ~_grid(s, ok, False)
    on = ~(_lineage(_grid(s, s["parents"].long(), -1), T) & bad[:, None, :]).any(-1) & ~bad
    here = torch.arange(T, device="cuda")
    path = torch.sort(torch.where(on, here, T), -1).values
    on = path < T
    count = on.sum(1)
    first = s["offsets"][:-1].long()
    last = first + path.gather(1, count[:, None] - 1).squeeze(1)
    w = p[last].double()
    if q is None:
        gone = torch.zeros((B, V), device="cuda")
        w = torch.where(gone.scatter_add_(1, token[last], out[last].float()) > 0, 0.0, w)
    else:
        w = (w - cut[last][:, None] * q[last].double()).clamp(min=0)
    total = w.cumsum(-1)
    drawn = (total <= s["v"].double()[:, None] * total[:, -1:]).sum(-1).clamp(max=V - 1)
    tok = _grid(s, s["tokens"], -1)
    res = torch.where(on, tok.gather(1, path.clamp(max=T - 1)), -1)
    res = torch.cat([res[:, 1:], torch.full_like(res[:, :1], -1)], 1)
    res.scatter_(1, count[:, None] - 1, drawn[:, None].to(torch.int32))
    return {"accepted": (count - 1).to(torch.int32), "path": torch.where(on, path, -1).to(torch.int32),
            "tokens": res.to(torch.int32)}


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _own(s):
    import speculative_sampling_verify_temp_amd as sdv
    c = s["case"]
    kind = c["kind"]
    if kind == "rope":
        q, k = sdv.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                                eps=EPS, interleaved=c["pairs"])
        return {"q": q, "k": k}
    if kind == "append":
        sdv.quant_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                         s["lens"], s["offsets"], s["max_nodes"], s["out_lens"], path=s["path"],
                         path_lens=s["path_lens"])
        return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "out_lens")}
    if kind == "attention":
        out, lse = sdv.quant_attention(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"],
                                       s["v_scale"], s["table"], s["lens"], s["offsets"], s["max_nodes"],
                                       parents=s["parents"], window=c["window"], sinks=c["sinks"], scale=s["scale"],
                                       want_lse=True)
        return {"out": out, "lse": lse}
    accepted, path, tokens = sdv.tree_verify_sample(s["p"], s["tokens"], s["parents"], s["offsets"], s["max_nodes"],
                                                    s["u"], s["v"], draft_probs=s["q"],
                                                    flags=sdv.SD_NO_REPLACEMENT if c["drafts"] == "once" else 0)
    return {"accepted": accepted, "path": path, "tokens": tokens}


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope, "append": _append, "attention": _attention, "sample": _sample}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_rope(s):
    c, got = s["case"], {}
    R = c["R"]
    for name in "qk":
        x, w = s[name].double(), s["w" + name]
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS) * w.double()
        z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                        s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
        y = x.clone()
        i = torch.arange(R // 2, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + R // 2)
        t = torch.complex(x[..., lo], x[..., hi]) * z
        y[..., lo], y[..., hi] = t.real, t.imag
        got[name] = y
    return got


def _exact_append(s):
    """Scales and codes block by block; int8 codes are whole numbers and have no such value."""
    c = s["case"]
    page, block, top = c["page"], c["block"], TOP[c["code"]]
    off, lens, got = s["offsets"].tolist(), s["lens"].tolist(), {"out_lens": None}
    for name in "kv":
        codes, scales = s[name + "_cache"].double(), s[name + "_scale"].double()
        for b in range(c["B"]):
            rows = list(range(off[b], off[b + 1]))
            if s["path"] is not None:
                rows = [off[b] + i for i in s["path"][b, :int(s["path_lens"][b])].tolist()]
            new, table = s[name + "_new"][rows].double().transpose(0, 1), s["table"][b].tolist()
            done = 0
            while done < len(rows):
                slot = lens[b] + done
                page_, place = table[slot // page], slot % page
                blk, inside = place // block, place % block
                m = min(block - inside, len(rows) - done)
                x = new[:, done:done + m]
                old = scales[page_, :, blk] if inside else torch.zeros(c["hkv"], dtype=torch.float64, device="cuda")
                fresh = x.abs().amax((1, 2)) / top
                scale = torch.maximum(old, fresh)
                if inside:
                    span = codes[page_, :, place - inside:place]
                    codes[page_, :, place - inside:place] = span * (old / scale)[:, None, None]
                codes[page_, :, place:place + m] = x / scale[:, None, None]
                scales[page_, :, blk] = scale
                done += m
        got[name + "_cache"] = None if c["code"] == "i8" else codes
        got[name + "_scale"] = scales
    return got


def _exact_attention(s):
    c = s["case"]
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    up = None if s["parents"] is None else s["parents"].tolist()
    G, page, block = c["hq"] // c["hkv"], c["page"], c["block"]
    outs, lses = [], []
    for b in range(c["B"]):
        lo, hi, n = off[b], off[b + 1], lens[b]
        sees, deep = np.zeros((hi - lo, hi - lo), dtype=bool), np.zeros(hi - lo, dtype=np.int64)
        for i in range(hi - lo):
            j = i - 1 if up is None else up[lo + i]
            sees[i, i] = True
            if j >= 0:
                sees[i] |= sees[j]
                deep[i] = deep[j] + 1
        at, place = np.concatenate([np.arange(n), n + deep]), n + deep
        seen = np.concatenate([np.ones((hi - lo, n), dtype=bool), sees], 1)
        if c["window"]:
            seen &= (at[None] < c["sinks"]) | (at[None] > place[:, None] - c["window"])
        hidden = torch.tensor(~seen, device="cuda")
        i = torch.arange(n, device="cuda")
        pages, spot = s["table"][b].long()[i // page], i % page
        o, e = [], []
        for h in range(c["hq"]):
            kv = h // G
            k, v = (torch.cat([s[x + "_cache"][pages, kv, spot].double() * s[x + "_scale"][pages, kv, spot // block]
                               .double()[:, None], s[x + "_new"][lo:hi, kv].double()]) for x in "kv")
            x = (s["q"][lo:hi, h].double() @ k.t() * s["scale"]).masked_fill(hidden, -math.inf)
            e.append(torch.logsumexp(x, 1))
            o.append(torch.softmax(x, 1) @ v)
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    if case["kind"] == "sample":      # whole numbers only
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attention": _exact_attention}[case["kind"]](s)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c, kind = case, case["kind"]
    if kind == "rope":
        heads = c["hq"] + c["hkv"]
        return {"bytes": 4 * c["N"] * heads * c["D"] + 4 * c["N"], "flops": 8 * c["N"] * heads * c["D"]}
    B, nodes = c["B"], _nodes(c)
    if kind == "append":
        count = sum(_paths(c) if c["kept"] else nodes)
        return {"bytes": 2 * count * c["hkv"] * c["D"] * 3, "flops": 6 * count * c["hkv"] * c["D"]}
    if kind == "attention":
        lens, D, new = _lens(c["lo"], c["hi"], B), c["D"], sum(nodes)
        # slots that some row sees: through the window the root sees the earliest
        seen = [n if not c["window"] else min(n, c["window"] - 1 + min(c["sinks"], max(0, n - c["window"] + 1)))
                for n in lens]
        moved = 2 * sum(seen) * c["hkv"] * (D + 4 / c["block"]) + 4 * new * (c["hkv"] + c["hq"]) * D
        return {"bytes": moved + 4 * new * c["hq"],
                "flops": 4 * D * c["hq"] * sum(t * (m + t / 2) for t, m in zip(nodes, seen))}
    # the rows of the node where the walk ends
    rows = 1 if c["drafts"] == "beam" else 2
    return {"bytes": 4 * rows * B * c["V"], "flops": 2 * rows * B * c["V"]}
