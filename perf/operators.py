"""Cases of the tree-drafting operators: attention of a drafted tree over a
paged cache, the append of the accepted branch with the weights it gave to
the cached tokens, eviction by those weights, a beam step and the greedy
verify of a tree.

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

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One token of the draft model, one request: the call whose latency a draft step waits for.
        dict(name="attn_draft_token", kind="attention", B=1, T=1, tree=False, hq=14, hkv=2, D=64, lo=517, hi=517,
             page=16, dtype="bf16"),
        # A verify forward of 32 requests with a chain of 8 drafts each: the ordinary batch.
        dict(name="attn_chain_batch", kind="attention", B=32, T=9, tree=False, hq=28, hkv=4, D=128, lo=500, hi=4096,
             page=16, dtype="bf16"),
        # Ragged trees in fp16 over short and odd contexts, some of one slot.
        dict(name="attn_tree_ragged", kind="attention", B=7, T=23, tree=True, hq=16, hkv=8, D=128, lo=1, hi=3001,
             page=32, dtype="f16"),
        # Trees of 64 nodes over long contexts: the largest verify forward.
        dict(name="attn_tree_long", kind="attention", B=16, T=64, tree=True, hq=28, hkv=4, D=128, lo=16384, hi=32768,
             page=64, dtype="bf16"),
        # One request, two tokens kept, short context: the append after each verify of a single user.
        dict(name="commit_single", kind="commit", B=1, T=8, hq=14, hkv=2, D=64, lo=701, hi=701, kept=2, page=16,
             dtype="bf16"),
        # 32 requests with long contexts, up to 6 tokens kept of 16-node trees.
        dict(name="commit_batch", kind="commit", B=32, T=16, hq=28, hkv=4, D=128, lo=5000, hi=16384, kept=6, page=16,
             dtype="bf16"),
        # One request a few tokens over its budget: the steady state of a bounded cache.
        dict(name="evict_steady", kind="evict", B=1, hkv=4, D=128, lo=2053, hi=2053, budget=2048, recent=256, sinks=4,
             page=16, dtype="bf16"),
        # Long prompts cut to a quarter after their prefill.
        dict(name="evict_prompt", kind="evict", B=16, hkv=4, D=128, lo=20000, hi=32768, budget=8192, recent=1024,
             sinks=4, page=64, dtype="bf16"),
        # One request, 4 beams over fp32 logits, a small draft state: the smallest beam step.
        dict(name="beam_single", kind="beam", B=1, W=4, V=151936, dtype="f32", ended=False, layers=4, segs=4, L=256,
             E=64, lo=101, hi=101),
        # 32 requests of 8 beams over bf16 logits with the key/value states of a draft of 4 layers.
        dict(name="beam_batch", kind="beam", B=32, W=8, V=152064, dtype="bf16", ended=True, layers=4, segs=4, L=512,
             E=64, lo=60, hi=512),
        # One request with a tree of 16 nodes over fp32 logits: latency.
        dict(name="verify_single", kind="verify", B=1, T=16, V=151936, dtype="f32"),
        # 64 requests with trees of 64 nodes.
        dict(name="verify_batch", kind="verify", B=64, T=64, V=152064, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "commit", "evict", "beam", "verify"])
    c = {"kind": kind}
    if kind in ("attention", "commit", "evict"):
        c["hq"], c["hkv"], c["D"] = rng.choice([(14, 2, 64), (28, 4, 128), (16, 8, 128), (8, 8, 64), (32, 8, 128)])
        c["page"] = rng.choice([16, 32, 64])
        c["dtype"] = rng.choice(["bf16", "f16"])
        c["B"] = _log(rng, 1, 32)
        c["hi"] = _log(rng, 16, max(16, min(32768, (100000 if c["hkv"] == 8 else 200000) // c["B"])))
        c["lo"] = rng.randint(1, c["hi"])
    if kind == "attention":
        c["T"] = _log(rng, 1, 64)
        c["tree"] = rng.random() < 0.6
    elif kind == "commit":
        c["T"] = _log(rng, 1, 64)
        c["kept"] = rng.randint(1, min(c["T"], 9))
    elif kind == "evict":
        del c["hq"]
        c["budget"] = max(1, rng.randint(c["hi"] // 8, c["hi"]))
        c["recent"] = rng.randint(0, c["budget"] // 2)
        c["sinks"] = rng.randint(0, min(8, c["budget"] - c["recent"]))
    elif kind == "beam":
        c["B"], c["W"] = _log(rng, 1, 32), rng.randint(1, 8)
        c["V"] = rng.choice([151936, 152064, _log(rng, 1000, 152064)])
        c["dtype"] = rng.choice(["bf16", "f32"])
        c["ended"] = rng.random() < 0.5
        c["layers"], c["segs"], c["E"] = rng.randint(1, 4), rng.choice([1, 2, 4]), rng.choice([8, 24, 64])
        c["L"] = _log(rng, 8, 512)
        c["hi"] = rng.randint(1, c["L"])
        c["lo"] = rng.randint(0, c["hi"])
    else:
        c["B"], c["T"] = _log(rng, 1, 64), _log(rng, 1, 64)
        c["V"] = rng.choice([151936, 152064, _log(rng, 1000, 152064)])
        c["dtype"] = rng.choice(["bf16", "f32"])
        if c["dtype"] == "f32":
            c["B"] = min(c["B"], 32)
    return c


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _lens(lo, hi, n):
    """n lengths over [lo, hi], in no order; the same for every seed of a case."""
    return [lo + (((i * 37 + 3) % n) * (hi - lo)) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _nodes(case):
    """Nodes of each request: the full tree for most, fewer for some."""
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


def _parents(np_rng, n):
    """A drafted tree: node 0 the root, each node's parent among the few before it."""
    return [-1] + [int(np_rng.randint(max(0, i - 6), i)) for i in range(1, n)]


def _cache(case, g, room):
    """Pool of pages and each request's table: pages in no order, some unused."""
    B, page = case["B"], case["page"]
    per = -(-(case["hi"] + room) // page)
    pool = B * per + 3
    table = torch.randperm(pool, generator=g, device="cuda")[: B * per].reshape(B, per).to(torch.int32)
    shape, dt = (pool, case["hkv"], page, case["D"]), DTYPES[case["dtype"]]
    return _randn(g, shape, dt), _randn(g, shape, dt), table


def prepare(case, seed):
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, kind, s = case["B"], case["kind"], {"case": case}
    if kind in ("attention", "commit"):
        nodes = _nodes(case)
        N, D, dt = sum(nodes), case["D"], DTYPES[case["dtype"]]
        lens = _lens(case["lo"], case["hi"], B)
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, g, 0 if kind == "attention" else case["kept"])
        s["lens"], s["offsets"] = _ints(lens), _ints(np.cumsum([0] + nodes))
        s["q"] = _randn(g, (N, case["hq"], D), dt, 2.5)      # peaked softmaxes, as attention's are
        s["k_new"], s["v_new"] = _randn(g, (N, case["hkv"], D), dt), _randn(g, (N, case["hkv"], D), dt)
        s["scale"] = 1.0 / math.sqrt(D)
        s["max_nodes"] = case["T"]
        # row and place of each node in the padded [B][T] grid of the plain form
        s["row"] = torch.tensor(np.repeat(np.arange(B), nodes), device="cuda")
        s["col"] = torch.tensor(np.concatenate([np.arange(n) for n in nodes]), device="cuda")
        if kind == "attention":
            s["parents"] = _ints(np.concatenate([_parents(r, n) for n in nodes])) if case["tree"] else None
            return s
        paths = _paths(case)
        path = np.full((B, case["T"]), -1, dtype=np.int32)
        for b, (n, m) in enumerate(zip(nodes, paths)):
            path[b, :m] = [0] + sorted(r.choice(np.arange(1, n), m - 1, replace=False).tolist()) if m > 1 else [0]
        s["path"], s["path_lens"] = _ints(path), _ints(paths)
        L = s["table"].shape[1] * case["page"]
        s["mass_in"] = torch.rand((B, case["hkv"], L), generator=g, device="cuda") * 4
        s["mass_out"] = torch.zeros_like(s["mass_in"])
        s["positions"] = torch.full((B, case["hkv"], L), -1, dtype=torch.int32, device="cuda")
        s["seen"] = s["lens"] + 5
        s["out_lens"] = torch.zeros_like(s["lens"])
        s["decay"] = 0.9375
        # the log-sum-exp that the attention of these rows left (rows off the path are not used)
        s["lse"] = torch.zeros((N, case["hq"]), device="cuda")
        G, off = case["hq"] // case["hkv"], np.cumsum([0] + nodes)
        for b in range(B):
            rows = torch.tensor(off[b] + path[b, :paths[b]], device="cuda")
            k = _dense(s["k_cache"], s["table"][b:b + 1])[0][:, :lens[b]].float()
            kn = s["k_new"][rows].float().transpose(0, 1)
            q = s["q"][rows].float().reshape(len(rows), case["hkv"], G, D).permute(1, 2, 0, 3)
            x = (q.reshape(case["hkv"], -1, D) @ torch.cat([k, kn], 1).transpose(1, 2)) * s["scale"]
            x = x.reshape(case["hkv"], G, len(rows), -1)
            x[..., lens[b]:].masked_fill_(torch.ones(len(rows), len(rows), device="cuda").triu(1).bool(), -math.inf)
            s["lse"][rows] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(len(rows), -1)
        return s
    if kind == "evict":
        lens = _lens(case["lo"], case["hi"], B)
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, g, 0)
        L = s["table"].shape[1] * case["page"]
        s["lens"] = _ints(lens)
        # accumulated weights span many decades; some tokens never got any
        m = torch.exp(2.5 * torch.randn((B, case["hkv"], L), generator=g, device="cuda") - 3.0)
        m[torch.rand(m.shape, generator=g, device="cuda") < 0.02] = 0.0
        s["mass_in"], s["mass_out"] = m, torch.zeros_like(m)
        # slots hold tokens in no order of position after earlier evictions
        s["seen"] = s["lens"] + 100
        noise = torch.rand((B, case["hkv"], L), generator=g, device="cuda")
        noise.masked_fill_(torch.arange(L, device="cuda") >= s["lens"][:, None, None], 2.0)
        rank = torch.argsort(torch.argsort(noise, -1), -1)
        s["pos_in"] = (rank + 100 * (rank >= 4)).to(torch.int32)
        s["pos_out"] = torch.full_like(s["pos_in"], -1)
        s["out_lens"] = torch.zeros_like(s["lens"])
        return s
    V, dt = case["V"], DTYPES[case["dtype"]]
    ld = -(-V // 8) * 8
    if kind == "beam":
        W = case["W"]
        s["logits"] = _randn(g, (B, W, ld), dt, 3.0)[..., :V]
        s["scores"] = -torch.rand((B, W), generator=g, device="cuda") * 6
        s["ended"] = (torch.rand((B, W), generator=g, device="cuda") < 0.2).to(torch.uint8) if case["ended"] else None
        s["cache"] = _randn(g, (case["layers"], B, W, case["segs"], case["L"], case["E"]), torch.bfloat16)
        s["lens"] = _ints(_lens(case["lo"], case["hi"], B))
        return s
    T, nodes = case["T"], _nodes(case)
    off = np.cumsum([0] + nodes)
    s["logits"] = _randn(g, (sum(nodes), ld), dt, 3.0)[..., :V]
    s["offsets"], s["max_nodes"] = _ints(off), T
    best = s["logits"].argmax(-1).cpu().numpy()
    tokens, parents = r.randint(0, V, sum(nodes)), []
    for b, n in enumerate(nodes):      # the target agrees with the draft along one branch of the tree
        parents.append(_parents(r, n))
        cur, left = 0, _accepted(b)
        while left > 0:
            kids = [i for i in range(cur + 1, n) if parents[b][i] == cur]
            if not kids:
                break
            child = kids[int(r.randint(len(kids)))]
            tokens[off[b] + child] = best[off[b] + cur]
            cur, left = child, left - 1
    s["tokens"], s["parents"] = _ints(tokens), _ints(np.concatenate(parents))
    s["row"] = torch.tensor(np.repeat(np.arange(B), nodes), device="cuda")
    s["col"] = torch.tensor(np.concatenate([np.arange(n) for n in nodes]), device="cuda")
    return s


def _accepted(b):
    """Levels on which request b's target agrees with its tree, where the tree is that deep."""
    return (b * 5 + 3) % 7


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _dense(cache, table):
    """[B][Hkv][slots][D] of a request's pages in order."""
    x = cache[table.long()]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4])


def _grid(s, x):
    """Packed node rows in the padded [B][T] grid, zeros elsewhere."""
    c = s["case"]
    out = torch.zeros((c["B"], c["T"]) + x.shape[1:], dtype=x.dtype, device=x.device)
    out[s["row"], s["col"]] = x
    return out


def _grouped(s, x):
    """[B][T][Hq][D] as [B][Hkv][T * G][D]: the rows that share a KV head."""
    c = s["case"]
    B, T = x.shape[:2]
    x = x.reshape(B, T, c["hkv"], c["hq"] // c["hkv"], -1).permute(0, 2, 1, 3, 4)
    return x.reshape(B, c["hkv"], -1, x.shape[-1])


def _sees(s):
    """[B][T][T]: which nodes a node sees."""
    c = s["case"]
    T = c["T"]
    if s["parents"] is None:
        return torch.ones((T, T), device="cuda").tril().bool().expand(c["B"], T, T)
    up = torch.full((c["B"], T), -1, dtype=torch.long, device="cuda")
    up[s["row"], s["col"]] = s["parents"].long()
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
    G = c["hq"] // hkv
    n = c["hi"]
    k, v = (_dense(s[x], s["table"])[:, :, :n].float() for x in ("k_cache", "v_cache"))
    kn, vn = (_grid(s, s[x].float()).transpose(1, 2) for x in ("k_new", "v_new"))
    q = _grouped(s, _grid(s, s["q"].float()))
    x = torch.cat([q @ k.transpose(2, 3), q @ kn.transpose(2, 3)], -1) * s["scale"]
    out_of = torch.arange(n, device="cuda") >= s["lens"][:, None]
    hidden = ~_sees(s)[:, :, None].expand(B, T, G, T).reshape(B, T * G, T)
    x.masked_fill_(torch.cat([out_of[:, None].expand(B, T * G, n), hidden], -1)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x[..., :n] @ v + x[..., n:] @ vn) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.reshape(B, hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, c["hq"], D)
    lse = lse.reshape(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, c["hq"])
    return {"out": o[s["row"], s["col"]].to(s["q"].dtype), "lse": lse[s["row"], s["col"]]}


def _commit(s):
    c = s["case"]
    B, T, hkv, D, page = c["B"], c["T"], c["hkv"], c["D"], c["page"]
    G, P = c["hq"] // hkv, c["kept"]
    path, lens = s["path"][:, :P].long(), s["lens"].long()
    on = torch.arange(P, device="cuda") < s["path_lens"][:, None]
    rows = torch.where(on, s["offsets"][:-1, None].long() + path, 0)
    q = _grouped(s, s["q"][rows].float())
    lse = _grouped(s, s["lse"][rows][..., None])
    kn = s["k_new"][rows]
    n = c["hi"]
    k = _dense(s["k_cache"], s["table"])[:, :, :n].float()
    live = on[:, :, None].expand(B, P, G).reshape(B, 1, P * G, 1)
    w = torch.where(live, ((q @ k.transpose(2, 3)) * s["scale"] - lse).exp(), 0.0).sum(2)
    wn = ((q @ kn.float().permute(0, 2, 3, 1)) * s["scale"] - lse).exp()
    causal = torch.ones((P, P), device="cuda").tril().bool()[:, None].expand(P, G, P).reshape(P * G, P)
    wn = torch.where(live & causal & on[:, None, None], wn, 0.0).sum(2)
    # the weights of the slots in use, then those of the appended ones
    used = (torch.arange(n, device="cuda") < lens[:, None])[:, None].expand(B, hkv, n)
    s["mass_out"][:, :, :n] = torch.where(used, s["decay"] * s["mass_in"][:, :, :n] + w, s["mass_out"][:, :, :n])
    b, i = on.nonzero(as_tuple=True)
    slot = lens[b] + i
    at = s["table"][b, slot // page].long()
    s["mass_out"][b, :, slot] = wn[b, :, i]
    s["positions"][b, :, slot] = (s["seen"][b] + i)[:, None].to(torch.int32)
    s["k_cache"][at, :, slot % page] = kn[b, i]
    s["v_cache"][at, :, slot % page] = s["v_new"][rows][b, i]
    s["out_lens"].copy_(s["lens"] + s["path_lens"])
    return {x: s[x] for x in ("k_cache", "v_cache", "mass_out", "positions", "out_lens")}


def _evict(s):
    c = s["case"]
    page, m = c["page"], c["budget"]
    L = s["mass_in"].shape[-1]
    i = torch.arange(L, device="cuda")
    n = s["lens"].long()[:, None, None]
    key = torch.where((s["pos_in"] < c["sinks"]) | (s["pos_in"] >= s["seen"][:, None, None] - c["recent"]),
                      math.inf, s["mass_in"])
    key = torch.where(i < n, key, -math.inf)
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, i.expand_as(order))
    kept = (rank < m) & (i < n)
    hole, late = ~kept & (i < m) & (i < n), kept & (i >= m)
    # the j-th late survivor goes to the j-th hole of its request and head
    b, h, src = late.nonzero(as_tuple=True)
    dst = hole.nonzero(as_tuple=True)[2]
    stay = kept & (i < m)
    s["mass_out"].copy_(torch.where(stay, s["mass_in"], s["mass_out"]))
    s["pos_out"].copy_(torch.where(stay, s["pos_in"], s["pos_out"]))
    s["mass_out"][b, h, dst] = s["mass_in"][b, h, src]
    s["pos_out"][b, h, dst] = s["pos_in"][b, h, src]
    to, at = s["table"][b, dst // page].long(), s["table"][b, src // page].long()
    s["k_cache"][to, h, dst % page] = s["k_cache"][at, h, src % page]
    s["v_cache"][to, h, dst % page] = s["v_cache"][at, h, src % page]
    s["out_lens"].copy_(s["lens"].clamp(max=m))
    return {x: s[x] for x in ("k_cache", "v_cache", "mass_out", "pos_out", "out_lens")}


EOS = 2


def _beam(s):
    c = s["case"]
    B, W, V = c["B"], c["W"], c["V"]
    z = s["logits"].double()           # candidates of different beams lie close: their order needs 64 bits
    top = z.amax(-1, keepdim=True)
    z = z - (top + (z - top).exp().sum(-1, keepdim=True).log()) + s["scores"].double()[..., None]
    if s["ended"] is not None:
        done = s["ended"].bool()
        z = torch.where(done[..., None], -math.inf, z)
        z[..., EOS] = torch.where(done, s["scores"].double(), z[..., EOS])
    z = z.reshape(B, W * V)
    edge = z.topk(W, -1).values[:, -1:]
    over, at = z > edge, z == edge
    chosen = over | (at & (at.cumsum(-1) <= W - over.sum(-1, keepdim=True)))
    flat = chosen.nonzero(as_tuple=True)[1].reshape(B, W)
    best, order = torch.sort(z.gather(1, flat), dim=-1, descending=True, stable=True)
    flat = flat.gather(1, order)
    parents, tokens = (flat // V).to(torch.int32), (flat % V).to(torch.int32)
    used = torch.arange(c["L"], device="cuda")[:, None] < s["lens"][:, None, None, None, None]
    moved = s["cache"][:, torch.arange(B, device="cuda")[:, None], parents.long()]
    s["cache"] = torch.where(used, moved, s["cache"])
    return {"scores": best.float(), "parents": parents, "tokens": tokens, "cache": s["cache"]}


def _verify(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    z = s["logits"]
    at = torch.arange(V, dtype=torch.int32, device="cuda")
    best = torch.where(z == z.amax(-1, keepdim=True), at, V).amin(-1)      # the lowest of equal maxima
    grid = torch.full((B, T), -1, dtype=torch.long, device="cuda")
    up, tok, win = grid.clone(), grid.clone(), grid.clone()
    up[s["row"], s["col"]], tok[s["row"], s["col"]] = s["parents"].long(), s["tokens"].long()
    win[s["row"], s["col"]] = best.long()
    # a node continues its parent's branch if it is the first child with the parent's best token
    here = torch.arange(T, device="cuda")
    fits = (up[:, None, :] == here[:, None]) & (tok[:, None, :] == win[..., None])
    first = torch.where(fits, here, T).amin(-1)
    fits = (up >= 0) & (first.gather(1, up.clamp(min=0)) == here)
    fits[:, 0] = True
    # the walk visits a node if every node from the root to it does so
    on = (up >= 0) | (here == 0)
    on &= ~(_sees(s) & ~fits[:, None, :]).any(-1)
    path = torch.sort(torch.where(on, here, T), -1).values
    on = path < T
    count = on.sum(1)
    win, tok = torch.cat([win, grid[:, :1]], 1), torch.cat([tok, grid[:, :1]], 1)
    out = torch.cat([tok.gather(1, path)[:, 1:], grid[:, :1]], 1)
    last = path.gather(1, count[:, None] - 1)
    out.scatter_(1, count[:, None] - 1, win.gather(1, last))
    return {"accepted": (count - 1).to(torch.int32), "path": torch.where(on, path, -1).to(torch.int32),
            "tokens": out.to(torch.int32)}


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _own(s):
    import speculative_sampling_verify_temp_amd as sdv
    c = s["case"]
    kind = c["kind"]
    if kind == "attention":
        out, lse = sdv.tree_attention(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"],
                                      s["lens"], s["offsets"], s["max_nodes"], parents=s["parents"],
                                      scale=s["scale"], want_lse=True)
        return {"out": out, "lse": lse}
    if kind == "commit":
        sdv.cache_commit(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["offsets"],
                         s["max_nodes"], s["path"], s["path_lens"], s["out_lens"], q=s["q"], lse=s["lse"],
                         scale=s["scale"], mass_in=s["mass_in"], mass_out=s["mass_out"], decay=s["decay"],
                         positions=s["positions"], seen=s["seen"])
        return {x: s[x] for x in ("k_cache", "v_cache", "mass_out", "positions", "out_lens")}
    if kind == "evict":
        sdv.cache_evict(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["mass_in"], s["mass_out"], s["pos_in"],
                        s["pos_out"], s["seen"], s["out_lens"], budget=c["budget"], recent=c["recent"],
                        sinks=c["sinks"])
        return {x: s[x] for x in ("k_cache", "v_cache", "mass_out", "pos_out", "out_lens")}
    if kind == "beam":
        scores, parents, tokens = sdv.beam_select(s["logits"], s["scores"], c["W"], ended=s["ended"], eos_id=EOS)
        sdv.beam_reorder(s["cache"], parents, lengths=s["lens"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "cache": s["cache"]}
    accepted, path, tokens = sdv.tree_verify_greedy(s["logits"], s["tokens"], s["parents"], s["offsets"],
                                                    s["max_nodes"])
    return {"accepted": accepted, "path": path, "tokens": tokens}


def run(state):
    if own:
        return _own(state)
    return {"attention": _attention, "commit": _commit, "evict": _evict, "beam": _beam,
            "verify": _verify}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------
# The definitions in 64 bits, request by request
# --------------------------------------------------------------------------

def _slots(s, b, n):
    """Page and place of slots 0..n-1 of request b."""
    i = torch.arange(n, device="cuda")
    return s["table"][b].long()[i // s["case"]["page"]], i % s["case"]["page"]


def _exact_attention(s):
    c = s["case"]
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    up = None if s["parents"] is None else s["parents"].tolist()
    G = c["hq"] // c["hkv"]
    outs, lses = [], []
    for b in range(c["B"]):
        lo, hi = off[b], off[b + 1]
        sees = np.zeros((hi - lo, hi - lo), dtype=bool)
        for i in range(hi - lo):
            if up is None:
                sees[i, :i + 1] = True
            else:
                sees[i, i] = True
                if up[lo + i] >= 0:
                    sees[i] |= sees[up[lo + i]]
        pages, at = _slots(s, b, lens[b])
        hidden = torch.tensor(~sees, device="cuda")
        o, e = [], []
        for h in range(c["hq"]):
            kv = h // G
            k = torch.cat([s["k_cache"][pages, kv, at], s["k_new"][lo:hi, kv]]).double()
            v = torch.cat([s["v_cache"][pages, kv, at], s["v_new"][lo:hi, kv]]).double()
            x = s["q"][lo:hi, h].double() @ k.t() * s["scale"]
            x[:, lens[b]:][hidden] = -math.inf
            e.append(torch.logsumexp(x, 1))
            o.append(torch.softmax(x, 1) @ v)
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_commit(s):
    c = s["case"]
    off, lens, m = s["offsets"].tolist(), s["lens"].tolist(), s["path_lens"].tolist()
    G = c["hq"] // c["hkv"]
    mass = s["mass_out"].double()
    for b in range(c["B"]):
        rows = [off[b] + i for i in s["path"][b, :m[b]].tolist()]
        pages, at = _slots(s, b, lens[b])
        for h in range(c["hkv"]):
            k = torch.cat([s["k_cache"][pages, h, at], s["k_new"][rows, h]]).double()
            total = torch.zeros(lens[b] + m[b], dtype=torch.float64, device="cuda")
            for i, row in enumerate(rows):
                q = s["q"][row, h * G:(h + 1) * G].double()
                e = s["lse"][row, h * G:(h + 1) * G].double()
                seen = lens[b] + i + 1
                total[:seen] += torch.exp(k[:seen] @ q.t() * s["scale"] - e).sum(1)
            total[:lens[b]] += s["decay"] * s["mass_in"][b, h, :lens[b]].double()
            mass[b, h, :len(total)] = total
    return {"k_cache": None, "v_cache": None, "mass_out": mass, "positions": None, "out_lens": None}


def _exact_beam(s):
    c = s["case"]
    best = []
    for b in range(c["B"]):
        rows = []
        for w in range(c["W"]):
            if s["ended"] is not None and int(s["ended"][b, w]):
                rows.append(s["scores"][b, w:w + 1].double())
            else:
                rows.append(torch.log_softmax(s["logits"][b, w].double(), 0).topk(min(c["W"], c["V"])).values
                            + s["scores"][b, w].double())
        best.append(torch.sort(torch.cat(rows), descending=True).values[:c["W"]])
    return {"scores": torch.stack(best), "parents": None, "tokens": None, "cache": None}


def exact(case, seed):
    if case["kind"] in ("evict", "verify"):      # no computed floating outputs: rows moved, whole numbers
        return None
    s = prepare(case, seed)
    return {"attention": _exact_attention, "commit": _exact_commit, "beam": _exact_beam}[case["kind"]](s)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c, kind, B = case, case["kind"], case["B"]
    es = 4 if c["dtype"] == "f32" else 2
    if kind == "attention":
        lens, nodes, D = _lens(c["lo"], c["hi"], B), _nodes(c), c["D"]
        new = sum(nodes)
        moved = 2 * (sum(lens) + new) * c["hkv"] * D * es + 2 * new * c["hq"] * D * es + 4 * new * c["hq"]
        return {"bytes": moved, "flops": 4 * D * c["hq"] * sum(n * (m + n / 2) for n, m in zip(nodes, lens))}
    if kind == "commit":
        lens, kept, D = _lens(c["lo"], c["hi"], B), _paths(c), c["D"]
        moved = sum(lens) * c["hkv"] * (D * es + 8) + sum(kept) * (4 * c["hkv"] + c["hq"]) * D * es
        return {"bytes": moved, "flops": 2 * D * c["hq"] * sum(m * n for m, n in zip(kept, lens))}
    if kind == "evict":
        lens = _lens(c["lo"], c["hi"], B)
        # slots ranked at random: this share of the kept ones lies behind the budget
        moves = sum(min(c["budget"], n) * max(0, n - c["budget"]) / n for n in lens)
        return {"bytes": c["hkv"] * (sum(8 * n + 8 * min(n, c["budget"]) for n in lens) + moves * 4 * c["D"] * es),
                "flops": c["hkv"] * sum(lens)}
    if kind == "beam":
        lens, W = _lens(c["lo"], c["hi"], B), c["W"]
        rows = W * (1 - 1 / W)         # beams whose parent is another one, on average
        row = c["layers"] * c["segs"] * c["E"] * 2
        return {"bytes": B * W * c["V"] * es + 2 * rows * row * sum(lens), "flops": 3 * B * W * c["V"]}
    # the rows that the walk visits; a tree of n nodes is rarely deeper than the levels counted here
    seen = sum(min(n, 1 + _accepted(b)) for b, n in enumerate(_nodes(c)))
    return {"bytes": seen * c["V"] * es, "flops": seen * c["V"]}
