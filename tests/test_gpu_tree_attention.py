"""sd_tree_attention on the GPU against the fp64 oracle."""
import numpy as np
import pytest

from treetools import Cached, dev, random_tree

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _run(c, **kw):
    out, lse = _sdv().tree_attention(**c.attention_args(), max_nodes=kw.pop("max_nodes", max(1, max(c.nodes))),
                                     scale=c.scale, want_lse=True, **kw)
    return out, lse


CASES = [
    # lens, nodes, Hq, Hkv, D, page
    ([1], [1], 2, 1, 64, 1),
    ([0], [1], 4, 4, 128, 16),
    ([517], [1], 14, 2, 64, 16),
    ([63, 64, 65, 0, 1], [1, 2, 3, 4, 1], 8, 8, 64, 16),
    ([127, 128, 129, 31, 33], [9, 9, 9, 9, 9], 7, 1, 128, 32),
    ([200, 3, 511], [64, 0, 17], 8, 4, 64, 8),
    ([1000, 77], [33, 64], 28, 4, 128, 64),
    ([300, 301], [5, 12], 32, 1, 64, 4),
    ([130, 700, 64], [16, 31, 64], 7, 1, 128, 256),
    ([2500], [2], 4, 4, 128, 16),
    ([90] * 11, [1, 2, 3, 4, 5, 6, 7, 8, 16, 17, 9], 6, 2, 64, 16),
    ([150, 600], [64, 5], 32, 1, 64, 16),
    ([700], [64], 32, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chains_and_trees_match_the_oracle(case, dtype):
    lens, nodes, Hq, Hkv, D, page = CASES[case]
    c = Cached(100 + case, lens, nodes, Hq, Hkv, D, page, dtype, slot_major=case % 2 == 1, packed=case % 3 == 1,
               sigma=2.0)
    print(f"chain {CASES[case]} {dtype}", flush=True)
    c.check_attention(*_run(c), c.reference())
    parents = np.concatenate([random_tree(c.rng, n)[:n] for n in nodes]).astype(np.int32)
    print("tree", flush=True)
    c.check_attention(*_run(c, parents=dev(parents)), c.reference(parents=parents))


@pytest.mark.parametrize("longest", [90, 1100])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 14)])
def test_many_requests(D, Hq, longest):
    """More requests than a wave has lanes, some without nodes or slots, in a
    short table and in one with room for long contexts."""
    rng = np.random.default_rng(D)
    lens = rng.integers(0, 90, 150).tolist()
    lens[70], lens[149] = longest * 2 // 3, longest
    nodes = rng.integers(0, 4, 150).tolist()
    c = Cached(41, lens, nodes, Hq, 2, D, 16, "bf16")
    c.check_attention(*_run(c), c.reference())


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.3])
def test_other_scales(scale):
    """Scales of zero (a plain mean) and below."""
    for D in (64, 128):
        c = Cached(42, [100, 0, 600], [3, 2, 30], 8, 2, D, 16, "f16")
        c.scale = scale
        c.check_attention(*_run(c), c.reference())


@pytest.mark.parametrize("D", [64, 128])
def test_masks_and_what_hides_behind_them(D):
    """Arbitrary masks: rows that see nothing, bits past the tree, and nodes
    that hold NaN and infinities, seen by no row or by some."""
    import torch
    for dtype in ("bf16", "f16"):
        c = Cached(7, [70, 0, 5, 0], [20, 6, 64, 3], 8, 2, D, 16, dtype)
        rng = np.random.default_rng(8)
        mask = rng.integers(0, 1 << 62, c.N, dtype=np.int64)
        mask[20] = 0                      # no cache and no node: an empty row
        mask[21] = ~np.int64(63)          # only bits past its request's 6 nodes
        mask[26:90] |= np.int64(-1) << 40
        hidden = (3, 21, 30)              # packed nodes nobody sees
        off = c.offsets
        for r in hidden:
            b = int(np.searchsorted(off, r, side="right")) - 1
            mask[off[b]:off[b + 1]] &= ~(np.int64(1) << (r - off[b]))
            c.d["k_new"][r] = float("nan")
            c.d["v_new"][r] = float("inf")
        print(f"masks {dtype} D {D}", flush=True)
        c.check_attention(*_run(c, tree_mask=dev(mask)), c.reference(mask=mask))
        # a value of NaN that some rows see: those rows are NaN, the others are not
        c.d["v_new"][10, :, 5] = float("nan")
        c.d["v_new"][40, :, 6] = float("-inf")
        out, lse = _run(c, tree_mask=dev(mask))
        o, e, mag = c.reference(mask=mask)
        got = out.float().cpu().numpy()
        sees = np.array([(int(mask[i]) >> 10) & 1 for i in range(20)], dtype=bool)
        assert np.isnan(got[:20][sees][:, :, 5]).all() and np.isfinite(got[:20][~sees]).all()
        seen2 = np.array([(int(mask[26 + i]) >> 14) & 1 for i in range(64)], dtype=bool)
        assert (got[26:90][seen2][:, :, 6] == -np.inf).all() and np.isfinite(got[26:90][~seen2]).all()
        keep = np.ones(got.shape, dtype=bool)
        keep[:20, :, 5][sees] = False
        keep[26:90, :, 6][seen2] = False
        patched = torch.where(torch.from_numpy(keep).cuda(), out.double(), torch.from_numpy(np.nan_to_num(o)).cuda())
        c.check_attention(patched, lse, (o, e, mag))


def test_queries_and_keys_of_large_scores():
    """Scores of several hundred: the running maximum moves by more than
    exp's range from tile to tile."""
    for D in (64, 128):
        c = Cached(9, [400, 65], [3, 40], 8, 2, D, 16, "bf16", sigma=60.0)
        for t in range(400):              # keys grow along the context
            f = 0.05 + t / 100
            p, s = c.table[0, t // 16], t % 16
            c.k[p, :, s] = np.float32(1) * np.round(c.k[p, :, s] * f * 8) / 8
        import torch
        c.d["k_cache"].copy_(dev(c.k, torch.bfloat16))
        c.k = c.d["k_cache"].double().cpu().numpy()
        c.check_attention(*_run(c), c.reference())


@pytest.mark.parametrize("below", [14.0, 20.0, 26.0])
@pytest.mark.parametrize("Hq,T", [(2, 1), (8, 9), (8, 64)])
def test_small_weights_of_many_keys_beside_a_dominating_one(Hq, T, below):
    """fp16: a first key that every query likes, its value zero, and 30000 keys
    whose weights are 2^-below of its weight each and carry all of the result."""
    import torch
    n, page, H, D = 30000, 64, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    k = (torch.randn((-(-n // page), H, page, D), generator=g, device="cuda") * 0.05).half()
    v = (torch.randn(k.shape, generator=g, device="cuda") + 3.0).half()
    k[:, :, :, 0] = 0.0
    k[0, :, 0, 0], v[0, :, 0] = 8.0, 0.0
    q = (torch.randn((T, Hq, D), generator=g, device="cuda")).half()
    q[:, :, 0] = below * 0.6931 / 8.0 * D ** 0.5
    kn, vn = torch.zeros((T, H, D), device="cuda").half(), torch.zeros((T, H, D), device="cuda").half()
    kn[:, :, 0], kn[:, :, 1] = -8.0, 0.0
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    print(f"tail {Hq} {T} {below}", flush=True)
    out, lse = _sdv().tree_attention(q, kn, vn, k, v, table, lens, off, T, want_lse=True)
    for head in range(Hq):
        h = head * H // Hq
        kk, vv = (x[:, h].reshape(-1, D)[:n].double() for x in (k, v))
        x = torch.cat([q[:, head].double() @ kk.t(), q[:, head].double() @ kn[:, h].double().t()], 1) * D ** -0.5
        x[:, n:][torch.ones((T, T), device="cuda").triu(1).bool()] = float("-inf")
        p = torch.softmax(x, 1)
        vv = torch.cat([vv, vn[:, h].double()])
        o, mag = p @ vv, p @ vv.abs()
        # half a step for the result; each weight w of the largest one is off by
        # half a step, 2^-11 w, or 2^-25 of the scale 2^7 that weights are held at;
        # the scores by (D + 4) 2^-24 of the sum of magnitudes (under 30), the
        # exponent's argument by 2^-24 of its own; fp32 sums of n terms by n 2^-24
        scores = (2 * 68 * 30 + 60) * 2.0 ** -24
        tol = 2.0 ** -11 * o.abs() + (2.0 ** -11 + scores + n * 2.0 ** -24) * 1.01 * mag \
            + 2.0 ** -32 * p.amax(1, keepdim=True) * vv.abs().sum(0) + 2.0 ** -25
        err = (out[:, head].double() - o).abs()
        assert (err <= tol).all(), (head, (err / o.abs()).max())
        assert ((lse[:, head].double() - torch.logsumexp(x, 1)).abs() <= scores + n * 2.0 ** -24 + 2e-5).all()


def test_bad_pages_lengths_and_nodes_are_reported():
    sdv = _sdv()
    c = Cached(11, [100, 100, 100, 100], [4, 4, 4, 4], 8, 2, 128, 16, "bf16", behind=5)
    n_pages = c.k.shape[0]
    import torch
    table = c.table.copy()
    table[0, 2], table[0, 6], table[1, 7] = -1, n_pages, 1 << 30    # the last one is not in use
    c.table = table
    c.d["page_table"] = dev(table)
    parents = np.array([-1, 0, 5, 1] + [-1, 0, 1, 2] * 3 + [0] * 5, dtype=np.int32)
    fixed = parents.copy()
    fixed[2] = -1
    out = torch.full((c.N + 5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.N + 5, 8), 7.0, device="cuda")
    status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    _run(c, parents=dev(parents), out=out, lse=lse, status=status)
    assert status.tolist() == [sdv.SD_ST_BAD_PAGE | sdv.SD_ST_BAD_TREE, 0, 0, 0]
    assert (out[c.N:] == 7).all() and (lse[c.N:] == 7).all()        # rows of no request
    c.check_attention(out, lse, c.reference(parents=fixed))
    # wrong lengths and offsets: zeros and -inf for the former, nothing written for the latter
    c.d["context_lens"] = dev(np.array([100, -1, 10 ** 6, 100], dtype=np.int32))
    off = c.offsets.copy()
    off[4] = c.N + 100
    c.d["node_offsets"] = dev(off)
    out.fill_(7.0)
    lse.fill_(7.0)
    _run(c, parents=dev(parents), out=out, lse=lse, status=status)
    st = status.tolist()
    assert st[0] == sdv.SD_ST_BAD_PAGE | sdv.SD_ST_BAD_TREE and st[1] == st[2] == sdv.SD_ST_BAD_LEN
    assert st[3] == sdv.SD_ST_BAD_NODES
    assert (out[4:12] == 0).all() and (lse[4:12] == float("-inf")).all()
    assert (out[12:] == 7).all() and (lse[12:] == 7).all()


def test_same_bits_on_every_call_and_stream_and_in_a_graph():
    import torch
    sdv = _sdv()
    c = Cached(13, [900, 40, 0, 333], [9, 9, 2, 64], 28, 4, 128, 16, "bf16")
    a, la = _run(c)
    b, lb = _run(c)
    assert torch.equal(a, b) and torch.equal(la, lb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, lb = _run(c, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    args = sdv.make_tree_attention_args(**c.attention_args(), max_nodes=64, scale=c.scale)
    ws = torch.empty(max(16, sdv.tree_attention_workspace_bytes(args)), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(a), torch.zeros_like(la)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(c, out=out, lse=lse, workspace=ws)
    for i in range(4):
        c.d["context_lens"].copy_(torch.tensor([900 - 100 * i, 40 - i, 0, 333], dtype=torch.int32))
        want, lwant = _run(c)
        out.zero_()
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lwant)


def test_interleaved_caches_and_wide_tables():
    """Keys and values of a page side by side in one tensor, padded rows, a
    table that is a part of a wider one, and a query shared by all heads."""
    import torch
    c = Cached(17, [300, 20, 77], [5, 9, 2], 8, 2, 64, 16, "bf16")
    pool = c.k.shape[0]
    kv = torch.full((pool, 2, 2, 16, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    kv[:, 0, :, :, :64], kv[:, 1, :, :, :64] = c.d["k_cache"], c.d["v_cache"]
    c.d["k_cache"], c.d["v_cache"] = kv[:, 0, :, :, :64], kv[:, 1, :, :, :64]
    wide = torch.full((3, c.table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table.shape[1]] = c.d["page_table"]
    c.d["page_table"] = wide[:, 2:2 + c.table.shape[1]]
    c.check_attention(*_run(c), c.reference())
    c.d["q"] = c.d["q"][:, :1].expand(-1, 8, -1)
    c.q = np.repeat(c.q[:, :1], 8, 1)
    c.check_attention(*_run(c), c.reference())


@pytest.mark.parametrize("lens,nodes", [([40, 7], [64, 3]), ([3000, 0, 900], [9, 64, 17]), ([9000], [2])])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (28, 4, 128), (32, 1, 64)])
def test_results_in_place_of_the_queries(lens, nodes, Hq, Hkv, D):
    import torch
    c = Cached(20, lens, nodes, Hq, Hkv, D, 16, "bf16")
    want, lse = _run(c)
    got, e = _run(c, out=c.d["q"])
    assert got.data_ptr() == c.d["q"].data_ptr() and torch.equal(got, want) and torch.equal(e, lse)


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own."""
    import torch
    a, b = Cached(18, [3000, 500], [9, 64], 28, 4, 128, 16, "bf16"), Cached(19, [2500], [64], 8, 2, 64, 16, "f16")
    wa, wb = _run(a), _run(b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((_run(a, stream=s), _run(b, stream=t)))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert all(torch.equal(x, y) for x, y in zip((*ga, *gb), (*wa, *wb)))


def test_a_pool_past_four_gigabytes():
    """Pages whose byte offsets pass 32 bits."""
    import torch
    c = Cached(15, [100], [5], 8, 2, 128, 16, "bf16", spare=0)
    pool = 600000                                   # 600000 pages of 8 KiB: 4.9 GB
    hi = np.arange(c.k.shape[0]) * 7 + pool - 7 * c.k.shape[0]
    big = []
    for x in (c.d["k_cache"], c.d["v_cache"]):
        y = torch.empty((pool, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
        y[torch.from_numpy(hi).cuda()] = x
        big.append(y)
    c.d["k_cache"], c.d["v_cache"] = big
    c.d["page_table"] = dev(hi[c.table].astype(np.int32))
    c.check_attention(*_run(c), c.reference())


def test_long_context_few_rows():
    """A long axis split over the chip and joined: against a dense product in
    fp64 on the device."""
    import torch
    for dtype, T, Hq, H, D in (("bf16", 1, 4, 1, 128), ("f16", 64, 8, 2, 64), ("bf16", 20, 28, 4, 128)):
        n, page = 30011, 64
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
        pages = -(-n // page)
        k, v = rnd(pages, H, page, D), rnd(pages, H, page, D)
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        q, kn, vn = rnd(T, Hq, D) * 3, rnd(T, H, D), rnd(T, H, D)
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        out, lse = _sdv().tree_attention(q, kn, vn, k, v, table, lens, off, T, want_lse=True)
        hide = torch.ones((T, T), device="cuda").triu(1).bool()
        for head in range(Hq):
            h = head * H // Hq
            kk = torch.cat([k[table[0].long(), h].reshape(-1, D)[:n], kn[:, h]]).double()
            vv = torch.cat([v[table[0].long(), h].reshape(-1, D)[:n], vn[:, h]]).double()
            x = q[:, head].double() @ kk.t() * D ** -0.5
            x[:, n:][hide] = float("-inf")
            p = torch.softmax(x, 1)
            eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
            # half a step for the result and for each weight; fp32 sums of n terms
            mag = p @ vv.abs()
            tol = eps * (p @ vv).abs() + (eps + 1e-4) * 1.01 * mag
            if dtype == "f16":
                tol = tol + n * 2.0 ** -25 * vv.abs().max()      # weights below fp16's normal numbers
            assert ((out[:, head].double() - p @ vv).abs() <= tol).all(), (dtype, head)
            assert ((lse[:, head].double() - torch.logsumexp(x, 1)).abs() <= 2e-5).all()
