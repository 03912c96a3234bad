"""sd_tree_verify_greedy on the GPU against the fp64 oracle, and the operators
of tree drafting run together."""
import numpy as np
import pytest

import oracle
from treetools import dev, random_tree, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _agreeing(rng, z, parents, offsets, depth):
    """Tokens that follow the rows' argmax down one branch for up to depth levels."""
    tokens = rng.integers(0, z.shape[1], z.shape[0]).astype(np.int32)
    for b in range(len(offsets) - 1):
        lo, n = offsets[b], offsets[b + 1] - offsets[b]
        cur = 0
        for _ in range(int(rng.integers(0, depth + 1))):
            kids = [c for c in range(cur + 1, n) if parents[lo + c] == cur]
            if not kids:
                break
            c = kids[int(rng.integers(len(kids)))]
            tokens[lo + c] = int(np.argmax(z[lo + cur]))
            cur = c
    return tokens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,V", [([1], 1), ([3, 1, 64], 7), ([5, 9, 2], 1000), ([64] * 70, 333), ([16, 33], 20011),
                                     ([2, 7], 152064), ([8] * 300, 2050), ([1, 4] * 40, 9001),
                                     # enough rows that only the visited ones are read
                                     ([1] * 330, 20011), ([4, 2, 3, 1] * 150, 30001), ([9] * 330, 20011)])
def test_walks_match_the_oracle(nodes, V, dtype):
    rng = np.random.default_rng(len(nodes) + V)
    off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    parents = np.concatenate([random_tree(rng, n)[:n] for n in nodes]).astype(np.int32)
    z = rounded(rng.standard_normal((off[-1], V)) * 3, dtype)      # bf16 rows have equal maxima
    if V > 1:
        z[0, 0], z[0, V - 1] = 99, 99
    tokens = _agreeing(rng, z, parents, off, 7)
    ld = -(-V // 8) * 8 + 8
    full = np.full((off[-1], ld), np.nan)
    full[:, :V] = z
    x = dev(full, torch_dtype(dtype))[:, :V]
    for flags in (0, 1):
        print(f"verify {len(nodes)} x {nodes[0]} V {V} {dtype} flags {flags}", flush=True)
        got = _sdv().tree_verify_greedy(x, dev(tokens), dev(parents), dev(off), max(nodes), flags=flags)
        want = oracle.tree_verify_greedy_ref(z, tokens, parents, off, max(nodes), no_bonus=flags == 1)
        for g, w, name in zip(got, want, ("accepted", "path", "tokens")):
            assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("B,T,V,dtype", [(48, 16, 152064, "bf16"), (64, 30, 152063, "bf16"), (9, 64, 151936, "f32"),
                                         (700, 5, 40000, "f32")])
def test_large_batches_against_every_row(B, T, V, dtype):
    """Batches whose walks read their own rows, against the argmax of every row
    on the device."""
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(B)
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    z = torch.randn((B * T, -(-V // 8) * 8), generator=g, device="cuda").to(torch_dtype(dtype))[:, :V] * 3
    z = torch.nn.functional.pad(z, (0, -V % 8), value=float("nan"))[:, :V]      # rows padded with NaN
    best = torch.where(z == z.amax(1, keepdim=True), torch.arange(V, device="cuda", dtype=torch.int32), V).amin(1)
    best = best.cpu().numpy()
    off = (np.arange(B + 1) * T).astype(np.int32)
    parents = np.concatenate([random_tree(rng, T) for _ in range(B)]).astype(np.int32)
    tokens = rng.integers(0, V, B * T).astype(np.int32)
    for i in range(B * T):                      # most nodes continue their parent's best token
        if parents[i] >= 0 and rng.random() < 0.7:
            tokens[i] = best[i // T * T + parents[i]]
    acc, path, tok = sdv.tree_verify_greedy(z, dev(tokens), dev(parents), dev(off), T)
    a, p = np.zeros(B, np.int32), np.full((B, T), -1, np.int32)
    for b in range(B):
        cur, n = 0, 0
        while True:
            p[b, n] = cur
            kids = [c for c in range(cur + 1, T) if parents[b * T + c] == cur and tokens[b * T + c] == best[b * T + cur]]
            if not kids:
                break
            cur, n = kids[0], n + 1
        a[b] = n
    assert np.array_equal(acc.cpu().numpy(), a) and np.array_equal(path.cpu().numpy(), p)
    want = np.where(p >= 0, best[np.arange(B)[:, None] * T + np.maximum(p, 0)], -1)
    assert np.array_equal(tok.cpu().numpy(), want)
    assert a.max() >= 3 or T < 6


@pytest.mark.parametrize("B", [1, 90, 1600])
def test_a_deep_chain_is_walked_to_its_end(B):
    rng = np.random.default_rng(2)
    T, V = 64, 516
    z = rng.standard_normal((B * T, V)).astype(np.float32)
    parents = np.tile(np.arange(-1, T - 1), B).astype(np.int32)
    tokens = np.concatenate([[0], z.argmax(1)[:-1]]).astype(np.int32)
    off = (np.arange(B + 1) * T).astype(np.int32)
    acc, path, tok = _sdv().tree_verify_greedy(dev(z), dev(tokens), dev(parents), dev(off), T)
    assert (acc == T - 1).all()
    assert np.array_equal(path.cpu().numpy(), np.tile(np.arange(T), (B, 1)))
    assert np.array_equal(tok.cpu().numpy(), z.argmax(1).reshape(B, T))


@pytest.mark.parametrize("copies", [1, 60, 700])
def test_defects_are_reported_request_by_request(copies):
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(3)
    V, T, R = 600, 4, 9
    z = rng.standard_normal((R * T, V)).astype(np.float32)
    parents = np.tile([-1, 0, 1, 2], R).astype(np.int32)
    tokens = rng.integers(0, V, R * T).astype(np.int32)
    tokens[0] = -7                                   # a root's token is not used
    z[1 * T, 5] = np.nan                             # the root's row: visited
    z[2 * T + 3, 5] = np.nan                         # a row that the walk does not reach
    tokens[3 * T + 2] = V
    tokens[4 * T + 1] = -1
    parents[5 * T + 2] = 2                           # its own parent
    parents[6 * T] = 1                               # a root with a parent
    z[7 * T] = -np.inf                               # all masked: the first token
    tokens[7 * T + 1] = 0
    z[8 * T + 2, V - 1] = np.nan                     # a NaN two steps down the walk
    tokens[8 * T + 1], tokens[8 * T + 2] = int(z[8 * T].argmax()), int(z[8 * T + 1].argmax())
    z, parents, tokens = np.tile(z, (copies, 1)), np.tile(parents, copies), np.tile(tokens, copies)
    off = (np.arange(R * copies + 1) * T).astype(np.int32)
    st = torch.full((R * copies,), -1, dtype=torch.int32, device="cuda")
    acc, path, tok = sdv.tree_verify_greedy(dev(z), dev(tokens), dev(parents), dev(off), T, status=st)
    want = [0, sdv.SD_ST_NONFINITE, 0, sdv.SD_ST_BAD_DRAFT_ID, sdv.SD_ST_BAD_DRAFT_ID, sdv.SD_ST_BAD_TREE,
            sdv.SD_ST_BAD_TREE, 0, sdv.SD_ST_NONFINITE]
    assert st.tolist() == want * copies
    acc = acc.cpu().numpy().reshape(copies, R)
    assert (acc[:, [1, 3, 4, 8]] == -1).all() and (acc[:, [0, 2, 5, 6]] >= 0).all() and (acc[:, 7] >= 1).all()
    bad = np.isin(np.arange(R * copies) % R, (1, 3, 4, 8))
    assert (path.cpu().numpy()[bad] == -1).all() and (tok.cpu().numpy()[bad] == -1).all()
    # node offsets that decrease, pass N, or give a request too many nodes or none
    off2 = np.array([0, 4, 3, 4, 4, 10, 14, R * T * copies + 1], dtype=np.int32)
    st = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    acc, _, _ = sdv.tree_verify_greedy(dev(z), dev(np.clip(tokens, 0, V - 1)), dev(parents), dev(off2), T, status=st)
    bad = [1, 3, 4, 6]
    assert all(st[b].item() & sdv.SD_ST_BAD_NODES and acc[b].item() == -1 for b in bad)
    assert not any(st[b].item() & sdv.SD_ST_BAD_NODES for b in (0, 2, 5))


def test_a_walk_that_is_given_up_is_reported():
    """The bounded waits of walks that read their own rows, forced to run out at
    once: such requests are -1 with a status of their own, the others stand, and
    the next call on the same workspace is whole."""
    import ctypes
    import torch
    import speculative_sampling_verify_temp_amd.tree as tree
    sdv = _sdv()
    rng = np.random.default_rng(5)
    B, T, V = 400, 8, 20011
    ld = -(-V // 4) * 4
    nodes = [T] * B
    nodes[9] = 1                                      # a single node needs no row without a bonus
    off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    N = int(off[-1])
    x = torch.randn((N, ld), device="cuda")[:, :V]
    parents = np.concatenate([np.arange(-1, n - 1) for n in nodes]).astype(np.int32)
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[5 * T + 3] = -1                            # an invalid request says why it is so
    t, p, o = dev(tokens), dev(parents), dev(off)
    a = tree._TREE_VERIFY.pack(x.data_ptr(), ld, t.data_ptr(), p.data_ptr(), o.data_ptr(), 0, B, N, V, T, 1)
    n = tree._tree_verify_bytes(a)
    ws = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")
    out = dict(accepted=torch.full((B,), 7, dtype=torch.int32, device="cuda"),
               path=torch.full((B, T), 7, dtype=torch.int32, device="cuda"),
               tokens=torch.full((B, T), 7, dtype=torch.int32, device="cuda"))
    st = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    P = ctypes.c_void_p
    rc = sdv.lib.sd_debug_tree_verify_polls(ctypes.c_char_p(a), P(ws.data_ptr()), ctypes.c_size_t(n), P(out["accepted"].data_ptr()),
                                            P(out["path"].data_ptr()), P(out["tokens"].data_ptr()), P(st.data_ptr()),
                                            ctypes.c_int32(0), P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    want = np.full(B, sdv.SD_ST_UNFINISHED)
    want[5], want[9] = sdv.SD_ST_BAD_DRAFT_ID, 0
    assert np.array_equal(st.cpu().numpy(), want)
    assert sdv.SD_ST_UNFINISHED & sdv.SD_ST_TREE_INVALID_MASK
    acc = out["accepted"].cpu().numpy()
    assert acc[9] == 0 and (np.delete(acc, 9) == -1).all()
    assert out["path"][9].tolist() == [0] + [-1] * (T - 1)
    bad = torch.arange(B, device="cuda") != 9
    assert (out["path"][bad] == -1).all() and (out["tokens"] == -1).all()
    got = sdv.tree_verify_greedy(x, t, p, o, T, flags=1, status=st, out=out, workspace=ws)
    want[want == sdv.SD_ST_UNFINISHED] = 0
    assert np.array_equal(st.cpu().numpy(), want)
    ref = sdv.tree_verify_greedy(x, t, p, o, T, flags=1)
    assert all(torch.equal(r, g) for r, g in zip(ref, got)) and (np.delete(got[0].cpu().numpy(), 5) >= 0).all()


def test_verify_in_a_graph():
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(4)
    for B in (2, 100, 700):
        T, V = 6, 5000
        parents = np.concatenate([random_tree(rng, T) for _ in range(B)]).astype(np.int32)
        off = (np.arange(B + 1) * T).astype(np.int32)
        x = dev(rng.standard_normal((B * T, V)).astype(np.float32))
        tok, par, o = dev(rng.integers(0, V, B * T).astype(np.int32)), dev(parents), dev(off)
        out = {n: torch.zeros(s, dtype=torch.int32, device="cuda")
               for n, s in (("accepted", (B,)), ("path", (B, T)), ("tokens", (B, T)))}
        sdv.tree_verify_greedy(x, tok, par, o, T, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sdv.tree_verify_greedy(x, tok, par, o, T, out=out)
        for _ in range(4):
            x.copy_(torch.randn_like(x))
            tok.copy_(x.argmax(1).roll(1).to(torch.int32))
            want = sdv.tree_verify_greedy(x, tok, par, o, T)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(w, out[n]) for w, n in zip(want, ("accepted", "path", "tokens")))


def test_tree_drafting_end_to_end():
    """Several rounds as a serving loop runs them on one attention layer: the
    tree grown by beam steps, its attention over the paged cache, the greedy
    verify of its logits, the branch committed with its weights, the cache cut
    to a budget.  Every step is checked against the oracle on the state that
    the step before left."""
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(6)
    B, Hq, H, D, page, V, W, L = 3, 8, 2, 64, 16, 500, 3, 128
    pool = B * (L // page) + 2
    k = torch.full((pool, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    table_np = rng.permutation(pool)[: B * (L // page)].reshape(B, -1).astype(np.int32)
    table = dev(table_np)
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    seen = torch.zeros(B, dtype=torch.int32, device="cuda")
    mass, pos = torch.zeros((B, H, L), device="cuda"), torch.full((B, H, L), -1, dtype=torch.int32, device="cuda")
    emb = rounded(rng.standard_normal((V, (Hq + 2 * H) * D)), "bf16")
    head = dev(rounded(rng.standard_normal((Hq * D, V)) * 0.3, "bf16"), torch.float32)
    draft = rng.standard_normal((V, V)) * 2
    root = [1, 2, 3]
    rows = [[] for _ in range(B)]                 # every committed token
    for step in range(6):
        # grow: two beam steps of W beams each, a tree of 1 + 2 W nodes
        z0 = np.stack([draft[[t] * W] for t in root]).astype(np.float32)
        sc0 = np.tile([0.0] + [-np.inf] * (W - 1), (B, 1)).astype(np.float32)
        s1, p1, t1 = sdv.beam_select(dev(z0), dev(sc0), W)
        t1n = t1.cpu().numpy()
        z1 = draft[t1n].astype(np.float32)
        s2, p2, t2 = sdv.beam_select(dev(z1), s1, W)
        state = torch.arange(B * W, dtype=torch.int64, device="cuda").reshape(1, B, W, 1, 1, 1).repeat(1, 1, 1, 1, 1, 2)
        state = sdv.beam_reorder(state, p2)
        assert (state[0, :, :, 0, 0, 0].cpu().numpy() == np.arange(B)[:, None] * W + p2.cpu().numpy()).all()
        tokens = np.concatenate([[root[b], *t1n[b], *t2[b].tolist()] for b in range(B)]).astype(np.int32)
        parents = np.concatenate([[-1] + [0] * W + [1 + p for p in p2[b].tolist()] for b in range(B)]).astype(np.int32)
        T = 1 + 2 * W
        off = (np.arange(B + 1) * T).astype(np.int32)
        x = dev(emb[tokens], torch.bfloat16).reshape(B * T, Hq + 2 * H, D)
        q, kn, vn = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        lens = ctx.tolist()
        kc, vc = k.double().cpu().numpy(), v.double().cpu().numpy()
        out, lse = sdv.tree_attention(q, kn, vn, k, v, table, ctx, dev(off), T, parents=dev(parents), want_lse=True)
        qd, knd, vnd = (t.double().cpu().numpy() for t in (q, kn, vn))
        o, e, mag = oracle.tree_attention_ref(qd, knd, vnd, kc, vc, table_np, lens, off, D ** -0.5, parents=parents)
        # scores here reach |q| |k| / 8 = 10 and more: their fp32 error and two half steps of bf16
        assert (np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-3) * mag + 1e-6).all()
        assert np.abs(lse.double().cpu().numpy() - e).max() < 1e-4
        logits = out.reshape(B * T, Hq * D).float() @ head
        acc, path, tok = sdv.tree_verify_greedy(logits, dev(tokens), dev(parents), dev(off), T)
        want = oracle.tree_verify_greedy_ref(logits.double().cpu().numpy(), tokens, parents, off, T)
        for g, w in zip((acc, path, tok), want):
            assert np.array_equal(g.cpu().numpy(), w)
        before = mass.double().cpu().numpy()
        new = torch.empty_like(ctx)
        sdv.cache_commit(kn, vn, k, v, table, ctx, dev(off), T, path, acc + 1, new, q=q, lse=lse, mass_out=mass,
                         positions=pos, seen=seen)
        G = Hq // H
        for b in range(B):
            kept = [off[b] + int(i) for i in path[b, : int(acc[b]) + 1]]
            for h in range(H):
                w = oracle.commit_weights_ref(qd[:, h * G:(h + 1) * G], lse.double().cpu().numpy()[:, h * G:(h + 1) * G],
                                              knd, kc, table_np[b], lens[b], kept, h, D ** -0.5)
                w[: lens[b]] += before[b, h, : lens[b]]
                np.testing.assert_allclose(mass[b, h, : len(w)].cpu().numpy(), w, rtol=2e-4, atol=1e-7)
            rows[b] += kept
            root[b] = int(tok[b, int(acc[b])])
        assert new.tolist() == [n + int(a) + 1 for n, a in zip(lens, acc)]
        seen += acc + 1
        ctx = new
        # cut
        m0, p0, n0 = mass.cpu().numpy(), pos.cpu().numpy(), ctx.tolist()
        cut = torch.empty_like(ctx)
        sdv.cache_evict(k, v, table, ctx, mass, mass, pos, pos, seen, cut, 6, 2, 1)
        for b in range(B):
            for h in range(H):
                src = oracle.evict_ref(m0[b, h], p0[b, h], n0[b], int(seen[b]), 6, 2, 1)
                assert pos[b, h, : len(src)].tolist() == [int(p0[b, h, s]) for s in src]
        ctx = cut
        assert max(ctx.tolist()) <= 6
    assert min(seen.tolist()) >= 6
