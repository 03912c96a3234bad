"""sd_cache_commit and sd_cache_evict on the GPU against the fp64 oracle."""
import numpy as np
import pytest

import oracle
from treetools import Cached, dev

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _branch(rng, n, m):
    return [0] + sorted(rng.choice(np.arange(1, n), m - 1, replace=False).tolist()) if m else []


def _commit(c, paths, decay, L, seed, status=None, in_place=False, weights=True, positions=True, **over):
    """One commit; returns the mass before, its device arrays and the new lengths."""
    import torch
    rng = np.random.default_rng(seed)
    B = len(c.lens)
    cols = max(max(c.nodes), 1) + 2
    path = np.full((B, cols), 99, dtype=np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    mass = rng.random((B, c.H, L)).astype(np.float32) * 3
    kw = dict(k_new=c.d["k_new"], v_new=c.d["v_new"], k_cache=c.d["k_cache"], v_cache=c.d["v_cache"],
              page_table=c.d["page_table"], context_lens=c.d["context_lens"], node_offsets=c.d["node_offsets"],
              max_nodes=max(1, max(c.nodes)), path=dev(path), path_lens=dev(np.array([len(p) for p in paths], np.int32)),
              out_context=torch.full((B,), -5, dtype=torch.int32, device="cuda"), status=status)
    if weights:
        _, e, _ = c.reference()
        m_in = dev(mass)
        kw.update(q=c.d["q"], lse=dev(np.nan_to_num(e).astype(np.float32)), scale=c.scale, decay=decay,
                  mass_in=m_in, mass_out=m_in if in_place else torch.full_like(m_in, -3.0))
        c.lse = kw["lse"].double().cpu().numpy()
    if positions:
        kw.update(positions=torch.full((B, c.H, L), -9, dtype=torch.int32, device="cuda"),
                  seen=dev(np.array([n + 11 for n in c.lens], dtype=np.int32)))
    kw.update(over)
    _sdv().cache_commit(**kw)
    return mass, kw


def _check_commit(c, paths, decay, mass, kw, in_place):
    """Weights: each of the m G terms exp(x) is off by the score's error, the
    rounding of x in base 2 (its magnitude, 40 at most here, times 2^-23) and
    an ulp; the fp32 sum by m G 2^-24 of itself; decay by two roundings."""
    G = c.Hq // c.H
    for b, p in enumerate(paths):
        n, m = c.lens[b], len(p)
        rows = [c.offsets[b] + i for i in p]
        for h in range(c.H):
            w = oracle.commit_weights_ref(c.q[:, h * G:(h + 1) * G], c.lse[:, h * G:(h + 1) * G], c.kn, c.k, c.table[b],
                                          n, rows, h, c.scale)
            tol = w * (2 * c.score_error() + 50 * 2.0 ** -23 + (m * G + 4) * 2.0 ** -24) + 1e-30
            old = decay * mass[b, h, :n].astype(np.float64)
            w[:n] += old
            tol[:n] += np.abs(w[:n]) * 2.0 ** -23
            got = kw["mass_out"][b, h].double().cpu().numpy()
            assert (np.abs(got[:n + m] - w) <= tol).all(), (b, h, np.abs(got[:n + m] - w).max())
            rest = mass[b, h, n + m:] if in_place else -3.0
            assert (got[n + m:] == rest).all()
        pos = kw["positions"][b].cpu().numpy()
        assert (pos[:, n:n + m] == n + 11 + np.arange(m)).all()
        assert (np.delete(pos, np.arange(n, n + m), 1) == -9).all()
    assert kw["out_context"].tolist() == [n + len(p) for n, p in zip(c.lens, paths)]
    k, v = c.k_dev.copy(), c.v_dev.copy()
    for b, p in enumerate(paths):
        for i, node in enumerate(p):
            t = c.lens[b] + i
            k[c.table[b, t // c.page], :, t % c.page] = c.kn[c.offsets[b] + node]
            v[c.table[b, t // c.page], :, t % c.page] = c.vn[c.offsets[b] + node]
    np.testing.assert_array_equal(c.d["k_cache"].double().cpu().numpy(), k)     # NaN where nothing was
    np.testing.assert_array_equal(c.d["v_cache"].double().cpu().numpy(), v)


CASES = [
    # lens, nodes, kept, Hq, Hkv, D, page
    ([1], [1], [1], 2, 1, 64, 1),
    ([0, 5], [3, 4], [2, 0], 4, 4, 128, 16),
    ([517], [8], [2], 14, 2, 64, 16),
    ([63, 64, 65, 15, 127], [9, 9, 9, 9, 9], [1, 2, 9, 3, 4], 28, 4, 128, 16),
    ([300, 20], [64, 64], [64, 33], 7, 1, 128, 32),
    ([1200, 0, 31], [16, 5, 1], [5, 5, 1], 32, 1, 64, 8),
    ([400, 90], [64, 64], [64, 20], 32, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_commit_matches_the_oracle(case, dtype):
    lens, nodes, kept, Hq, Hkv, D, page = CASES[case]
    c = Cached(200 + case, lens, nodes, Hq, Hkv, D, page, dtype, slot_major=case % 2 == 0, packed=case % 3 == 2, room=70)
    paths = [list(range(m)) if case % 2 else _branch(c.rng, n, m) for n, m in zip(nodes, kept)]
    L = c.table.shape[1] * page + 3
    decay, in_place = (0.75, False) if case % 2 else (1.0, True)
    # lse comes from the chain's attention: a weight may pass one where the branch leaves nodes out
    print(f"commit {CASES[case]} {dtype}", flush=True)
    mass, kw = _commit(c, paths, decay, L, case, in_place=in_place)
    _check_commit(c, paths, decay, mass, kw, in_place)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,kept", [(64, 4, 2, 1), (128, 28, 4, 3), (128, 16, 1, 1), (64, 32, 1, 5)])
def test_infinite_keys_have_no_weight_where_their_scores_are_minus_infinity(D, Hq, Hkv, kept, dtype):
    """Cached and drafted keys with an infinite element, against queries that all
    have the other sign there: weight zero, whatever the number of rows."""
    c = Cached(224, [150, 20], [6, 6], Hq, Hkv, D, 16, dtype, room=8)
    c.q[:, :, 3] = -np.abs(c.q[:, :, 3]) - 1.0
    c.d["q"].copy_(dev(c.q, c.d["q"].dtype))
    c.q = c.d["q"].double().cpu().numpy()
    paths = [list(range(kept)), [0]]
    for b, t in ((0, 0), (0, 77), (0, 149), (1, 19)):
        for x in (c.k, c.k_dev):
            x[c.table[b, t // 16], :, t % 16, 3] = np.inf
        c.d["k_cache"][int(c.table[b, t // 16]), :, t % 16, 3] = float("inf")
    c.kn[kept - 1, :, 3] = np.inf
    c.d["k_new"][kept - 1, :, 3] = float("inf")
    # finite magnitudes for the bound of the scores' errors
    bound = Cached.score_error(type("", (), dict(scale=c.scale, D=D, q=c.q, k=np.nan_to_num(c.k, posinf=0.0),
                                                 kn=np.nan_to_num(c.kn, posinf=0.0)))())
    c.score_error = lambda: bound
    L = c.table.shape[1] * 16
    print(f"infinite keys {D} {Hq} {Hkv} {kept} {dtype}", flush=True)
    mass, kw = _commit(c, paths, 0.5, L, 3)
    assert np.isfinite(c.lse).all()
    _check_commit(c, paths, 0.5, mass, kw, False)
    for t in (0, 77, 149):
        np.testing.assert_array_equal(kw["mass_out"][0, :, t].cpu().numpy(), 0.5 * mass[0, :, t])


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (32, 2), (28, 4)])
def test_rows_that_saw_nothing_give_no_weight(Hq, Hkv):
    """An lse of -inf, as attention leaves it for a row whose mask is empty."""
    c = Cached(225, [0, 40], [4, 4], Hq, Hkv, 64, 16, "bf16", room=8)
    _, e, _ = c.reference()
    e[0] = -np.inf
    e[5, 1::2] = -np.inf
    mass, kw = _commit(c, [[0, 1, 3], [0, 1]], 0.5, c.table.shape[1] * 16, 1, lse=dev(e.astype(np.float32)))
    c.lse = kw["lse"].double().cpu().numpy()
    _check_commit(c, [[0, 1, 3], [0, 1]], 0.5, mass, kw, False)


def test_a_branch_may_name_a_node_twice():
    c = Cached(223, [40, 3], [4, 4], 4, 2, 64, 16, "bf16", room=8)
    L = c.table.shape[1] * 16
    mass, kw = _commit(c, [[0, 2, 2], [3, 1]], 1.0, L, 1, in_place=True)
    _check_commit(c, [[0, 2, 2], [3, 1]], 1.0, mass, kw, True)


def test_commit_and_evict_in_a_graph():
    """A commit and an eviction captured once and replayed on states that the
    program changes in between."""
    import torch
    sdv = _sdv()
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    B, H, Hq, D, page, n, T, budget = 3, 2, 8, 64, 16, 300, 4, 200
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cols = 20
    k, v = rnd(B * cols, H, page, D), rnd(B * cols, H, page, D)
    table = torch.randperm(B * cols, generator=g, device="cuda").to(torch.int32).reshape(B, cols)
    q, kn, vn = rnd(B * T, Hq, D), rnd(B * T, H, D), rnd(B * T, H, D)
    lse = torch.full((B * T, Hq), 6.0, device="cuda")
    off = torch.arange(B + 1, device="cuda", dtype=torch.int32) * T
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 1, 3, -1]] * B, dtype=torch.int32, device="cuda")
    plen = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    mass = torch.rand((B, H, cols * page), generator=g, device="cuda")
    pos = torch.arange(cols * page, dtype=torch.int32, device="cuda").repeat(B, H, 1)
    seen = ctx.clone()
    mid, out = torch.zeros_like(ctx), torch.zeros_like(ctx)
    m2, p2 = mass.clone(), pos.clone()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        sdv.cache_commit(kn, vn, k, v, table, ctx, off, T, path, plen, mid, q=q, lse=lse, mass_in=mass, mass_out=m2,
                         positions=p2, seen=seen)
        sdv.cache_evict(k, v, table, mid, m2, m2, p2, p2, seen, out, budget, 20, 4, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for x in (k, v, q, kn, vn):
            x.copy_(rnd(*x.shape))
        mass.copy_(torch.rand(mass.shape, generator=g, device="cuda"))
        plen.copy_(torch.tensor([i % 4, 1, 2], dtype=torch.int32))
        state = [x.clone() for x in (k, v)]
        m2.copy_(mass)
        p2.copy_(pos)
        step()
        want = [x.clone() for x in (k, v, m2, p2, mid, out)]
        for x, y in zip((k, v), state):
            x.copy_(y)
        m2.copy_(mass)
        p2.copy_(pos)
        ws.fill_(0xEE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((k, v, m2, p2, mid, out), want))


def test_decay_zero_reads_no_old_weight():
    import torch
    c = Cached(220, [40, 3], [4, 4], 4, 2, 64, 16, "bf16", room=8)
    L = c.table.shape[1] * 16
    m = torch.full((2, 2, L), float("nan"), device="cuda")
    mass, kw = _commit(c, [[0, 2], [0]], 0.0, L, 1, mass_in=m, mass_out=torch.full_like(m, -3.0))
    _check_commit(c, [[0, 2], [0]], 0.0, np.zeros_like(mass), kw, False)


def test_commit_without_weights_or_positions():
    c = Cached(221, [40, 3], [4, 4], 4, 2, 64, 16, "f16", room=8)
    _, kw = _commit(c, [[0, 2, 3], []], 0.0, 64, 1, weights=False, positions=False)
    assert kw["out_context"].tolist() == [43, 3]
    got = c.d["k_cache"].double().cpu().numpy()
    for i, node in enumerate([0, 2, 3]):
        t = 40 + i
        assert (got[c.table[0, t // 16], :, t % 16] == c.kn[node]).all()


def test_commit_refuses_defects_request_by_request():
    import torch
    sdv = _sdv()
    c = Cached(222, [40, 40, 40, 40, 40, 40, 40], [4] * 7, 4, 2, 64, 16, "bf16", room=8)
    cap = c.table.shape[1] * 16
    lens = np.array([40, 40, -2, cap - 1, 40, 40, 40], dtype=np.int32)
    c.d["context_lens"] = dev(lens)
    table = c.table.copy()
    table[4, 1], table[6, 2] = -3, c.k.shape[0]        # a bad page under the context, one under the appended slots
    c.d["page_table"] = dev(table)
    status = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    before = c.d["k_cache"].clone()
    L = cap
    path_lens = torch.tensor([1, 5, 1, 2, 2, 2, 1], dtype=torch.int32, device="cuda")
    mass, kw = _commit(c, [[0], [0, 1, 2, 3], [0], [0, 1], [0, 1], [0, 4], [0]], 1.0, L, 2, status=status,
                       path_lens=path_lens)
    assert status.tolist() == [0, sdv.SD_ST_BAD_PATH, sdv.SD_ST_BAD_LEN, sdv.SD_ST_BAD_LEN, sdv.SD_ST_BAD_PAGE,
                               sdv.SD_ST_BAD_PATH, sdv.SD_ST_BAD_PAGE]
    assert kw["out_context"].tolist() == [41, 40, -2, cap - 1, 42, 40, 41]
    out = kw["mass_out"].cpu().numpy()
    for b in (1, 2, 3, 5):
        assert (out[b] == -3).all() and (kw["positions"][b] == -9).all()
    np.testing.assert_array_equal(out[4, :, 16:32], mass[4, :, 16:32])     # absent slots gained nothing
    after = c.d["k_cache"].clone()
    for b, m in ((0, 1), (4, 2)):
        for i in range(m):
            p, s = int(table[b, (40 + i) // 16]), (40 + i) % 16
            assert torch.equal(after[p, :, s], c.d["k_new"][4 * b + i])
            after[p, :, s] = before[p, :, s]
    assert torch.equal(after.view(torch.int16), before.view(torch.int16))


# ---- eviction ----

def _evict(seed, lens, H, D, page, budget, recent, sinks, dtype="bf16", kind="random", positions=True, in_place=False,
           bad=False, status=None):
    import torch
    rng = np.random.default_rng(seed)
    c = Cached(seed, lens, [1] * len(lens), H, H, D, page, dtype)
    B, L = len(lens), c.table.shape[1] * page + 5
    mass = np.exp(3 * rng.standard_normal((B, H, L))).astype(np.float32)
    if kind == "ties":
        mass = rng.integers(0, 3, (B, H, L)).astype(np.float32)
    if kind == "equal":
        mass[:] = 0.25
    if kind == "odd":       # not numbers, infinities, zeros of both signs, values below zero
        for value in (np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 1e-42):
            mass[rng.random((B, H, L)) < 0.1] = value
    pos = np.full((B, H, L), -77, dtype=np.int32)
    seen = np.array([n + 40 for n in lens], dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            pos[b, h, :n] = rng.permutation(np.concatenate([np.arange(min(n, 3)), np.arange(min(n, 3), n) + 40]))
    if bad:
        c.table[0, 1] = -1
        c.d["page_table"] = dev(c.table)
    m_in, p_in = dev(mass), dev(pos)
    m_out = m_in if in_place else torch.full_like(m_in, -3.0)
    p_out = p_in if in_place else torch.full_like(p_in, -9)
    out = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    k0, v0 = c.d["k_cache"].clone(), c.d["v_cache"].clone()
    _sdv().cache_evict(c.d["k_cache"], c.d["v_cache"], c.d["page_table"], c.d["context_lens"], m_in, m_out,
                       p_in if positions else None, p_out if positions else None, dev(seen) if positions else None,
                       out, budget, recent, sinks, status=status)
    torch.cuda.synchronize()
    want = [k0.view(torch.int16).cpu().numpy().copy(), v0.view(torch.int16).cpu().numpy().copy()]
    wm = mass.copy() if in_place else np.full_like(mass, -3.0)
    wp = pos.copy() if in_place else np.full_like(pos, -9)
    old = [w.copy() for w in want]
    for b, n in enumerate(lens):
        for h in range(H):
            src = oracle.evict_ref(mass[b, h], pos[b, h] if positions else None, n, seen[b], budget, recent, sinks)
            for t, s in enumerate(src):
                wm[b, h, t], wp[b, h, t] = mass[b, h, s], pos[b, h, s]
                a, z = c.table[b, t // page], c.table[b, s // page]
                if t != s and a >= 0 and z >= 0:
                    for w, o in zip(want, old):
                        w[a, h, t % page] = o[z, h, s % page]
    np.testing.assert_array_equal(m_out.cpu().numpy(), wm)
    if positions:
        np.testing.assert_array_equal(p_out.cpu().numpy(), wp)
    for x, w in zip((c.d["k_cache"], c.d["v_cache"]), want):
        np.testing.assert_array_equal(x.view(torch.int16).cpu().numpy(), w)
    assert out.tolist() == [min(n, budget) for n in lens]


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,H,D,page,budget,recent,sinks", [
    ([1], 1, 64, 16, 1, 0, 0),
    ([2, 1, 0], 2, 64, 1, 1, 1, 0),
    ([100, 64, 65, 63], 2, 128, 16, 64, 8, 3),
    ([700, 1300, 20], 3, 64, 32, 500, 500, 0),
    ([1025, 1024, 2049], 2, 128, 64, 1000, 17, 2),
    ([4099], 4, 64, 16, 4096, 64, 4),
    ([5000, 3], 1, 128, 16, 7, 2, 2),
])
def test_evict_matches_the_oracle(lens, H, D, page, budget, recent, sinks, kind):
    print(f"evict {lens} {H} {D} {page} {budget} {kind}", flush=True)
    _evict(300 + len(lens) + budget, lens, H, D, page, budget, recent, sinks, kind=kind,
           dtype="f16" if H == 2 else "bf16", in_place=kind in ("ties", "odd"))


@pytest.mark.parametrize("n", [70, 5000])
@pytest.mark.parametrize("recent,sinks", [(0, 0), (0, 2), (3, 1), (20, 0)])
def test_evict_protects_positions_at_or_past_seen(n, recent, sinks):
    """`seen` before it counts the last eight tokens; with and without a window of
    recent ones, and with more protected slots than the budget."""
    import torch
    rng = np.random.default_rng(n + recent)
    H, page = 2, 16
    c = Cached(324, [n], [1], H, H, 64, page, "bf16")
    L = c.table.shape[1] * page
    pos = np.zeros((1, H, L), dtype=np.int32)
    for h in range(H):
        pos[0, h, :n] = rng.permutation(n)
    mass = rng.random((1, H, L)).astype(np.float32)
    mass[pos >= n - 8] = -1.0                     # the just appended: no weight yet
    for budget in (24, 40):
        m, p, out = dev(mass), dev(pos), torch.zeros(1, dtype=torch.int32, device="cuda")
        _sdv().cache_evict(c.d["k_cache"], c.d["v_cache"], c.d["page_table"], c.d["context_lens"], m, m, p, p,
                           dev(np.array([n - 8], np.int32)), out, budget, recent, sinks)
        for h in range(H):
            src = oracle.evict_ref(mass[0, h], pos[0, h], n, n - 8, budget, recent, sinks)
            assert p[0, h, :budget].tolist() == [int(pos[0, h, s]) for s in src], (h, budget)
            assert set(range(n - 8, n)) <= set(p[0, h, :budget].tolist()) or recent + sinks + 8 > budget


def test_evict_without_positions_and_with_bad_pages():
    import torch
    sdv = _sdv()
    _evict(320, [300, 30], 2, 64, 16, 50, 0, 0, positions=False)
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    _evict(321, [300, 30], 2, 64, 16, 50, 4, 2, bad=True, status=status)
    assert status.tolist() == [sdv.SD_ST_BAD_PAGE, 0]


def test_evict_moves_masses_and_positions_but_not_rows_of_bad_pages():
    """One slot on a bad page moves into a hole of a good one, and one of a good
    page into a hole of a bad one: the bookkeeping follows the ranking, no row of
    either move is touched."""
    import torch
    sdv = _sdv()
    c = Cached(323, [64], [1], 1, 1, 64, 16, "bf16")
    c.table[0, 0], c.table[0, 3] = -1, c.k.shape[0]                    # slots 0..15 and 48..63
    c.d["page_table"] = dev(c.table)
    mass = torch.arange(80, dtype=torch.float32, device="cuda").flip(0).reshape(1, 1, 80).contiguous()
    mass[0, 0, [3, 20, 21, 40, 41, 50]] = torch.tensor([-1.0, -2.0, -3.0, 99.0, 98.0, 97.0], device="cuda")
    pos = torch.arange(80, dtype=torch.int32, device="cuda").reshape(1, 1, 80).contiguous()
    want = list(range(32))
    want[3], want[20], want[21] = 40, 41, 50
    m0, k0, v0 = mass[0, 0].clone(), c.d["k_cache"].clone(), c.d["v_cache"].clone()
    out, st = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    sdv.cache_evict(c.d["k_cache"], c.d["v_cache"], c.d["page_table"], c.d["context_lens"], mass, mass, pos, pos,
                    dev(np.array([64], np.int32)), out, 32, status=st)
    assert st.tolist() == [sdv.SD_ST_BAD_PAGE] and out.tolist() == [32]
    assert pos[0, 0, :32].tolist() == want and torch.equal(mass[0, 0, :32], m0[want])
    p, q = int(c.table[0, 1]), int(c.table[0, 2])
    k0[p, 0, 4], v0[p, 0, 4] = k0[q, 0, 9], v0[q, 0, 9]                # 41 -> 20: both pages are good
    assert torch.equal(c.d["k_cache"].view(torch.int16), k0.view(torch.int16))
    assert torch.equal(c.d["v_cache"].view(torch.int16), v0.view(torch.int16))


def test_evict_leaves_a_request_of_wrong_length_alone():
    import torch
    sdv = _sdv()
    c = Cached(322, [60, 60], [1, 1], 2, 2, 64, 16, "bf16")
    c.d["context_lens"] = dev(np.array([-1, 1000], dtype=np.int32))
    L = c.table.shape[1] * 16
    mass, pos = torch.rand(2, 2, L, device="cuda"), torch.zeros((2, 2, L), dtype=torch.int32, device="cuda")
    m0, k0 = mass.clone(), c.d["k_cache"].clone()
    out, st = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    sdv.cache_evict(c.d["k_cache"], c.d["v_cache"], c.d["page_table"], c.d["context_lens"], mass, mass, pos, pos,
                    out.clone(), out, 8, status=st)
    assert st.tolist() == [sdv.SD_ST_BAD_LEN] * 2 and out.tolist() == [-1, 1000]
    assert torch.equal(mass, m0) and torch.equal(c.d["k_cache"].view(torch.int16), k0.view(torch.int16))


def test_long_caches_against_sorting():
    """32768 and 40000 slots (more than LDS holds) to 5000, random and with many
    equal weights: the survivors against a stable sort on the device."""
    import torch
    sdv = _sdv()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    B, H, D, page, budget = 2, 2, 64, 64, 5000
    for n, equal in ((32768, False), (32768, True), (40000, False), (40000, True)):
        k = torch.randn((B * n // page, H, page, D), generator=g, device="cuda").to(torch.bfloat16)
        v = -k
        table = torch.randperm(B * n // page, generator=g, device="cuda").to(torch.int32).reshape(B, -1)
        lens = torch.tensor([n, n - 13], dtype=torch.int32, device="cuda")
        mass = torch.exp(2 * torch.randn((B, H, n), generator=g, device="cuda"))
        if equal:
            mass = (mass * 2).floor()
        pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, H, 1)
        m_out, p_out, out = torch.zeros_like(mass), torch.zeros_like(pos), torch.zeros_like(lens)
        k0 = k.clone()
        sdv.cache_evict(k, v, table, lens, mass, m_out, pos, p_out, lens, out, budget, 100, 4)
        for b in range(B):
            m = int(lens[b])
            for h in range(H):
                key = mass[b, h, :m].clone()
                key[:4] = float("inf")
                key[m - 100:] = float("inf")
                kept = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
                got = p_out[b, h, :budget].long()
                assert torch.equal(got.sort().values, kept)
                stay = kept[kept < budget]
                assert torch.equal(got[stay], stay)
                mask = torch.ones(budget, dtype=torch.bool, device="cuda")
                mask[stay] = False
                assert torch.equal(got[mask], kept[kept >= budget])
                assert torch.equal(m_out[b, h, :budget], mass[b, h, got])
                dense = lambda x: x[table[b].long(), h].reshape(-1, D)  # noqa: E731
                assert torch.equal(dense(k)[:budget], dense(k0)[got])
                assert torch.equal(dense(v)[:budget], -dense(k0)[got])
