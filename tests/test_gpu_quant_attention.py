"""sd_quant_attention on the GPU against the fp64 oracle."""
import numpy as np
import pytest

import oracle
from servetools import Quantised, code_dev, random_cache
from treetools import EPS, dev, random_tree, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _parents(s):
    return np.concatenate([random_tree(s.rng, n)[:n] for n in s.nodes]).astype(np.int32)


def _run(s, parents=None, **kw):
    return _sdv().quant_attention(**s.attention_args(), max_nodes=max(s.nodes),
                                  parents=None if parents is None else dev(parents), want_lse=True, **kw)


@pytest.mark.parametrize("code,dtype", [("i8", "bf16"), ("i8", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,D,page,block,tree", [
    ([517], [1], 14, 2, 64, 16, 16, False), ([1], [1], 4, 1, 128, 16, 16, False), ([0, 0], [3, 1], 4, 2, 64, 16, 16, True),
    ([15, 16, 17, 127, 128, 129], [1] * 6, 7, 1, 128, 16, 16, False),
    ([300, 0, 77, 1025], [9, 4, 1, 7], 28, 4, 128, 32, 16, False),
    ([700, 64, 31], [23, 5, 64], 4, 4, 64, 64, 64, True),
    ([2000, 999], [64, 33], 14, 2, 64, 128, 32, True),
    ([1100, 10], [64, 64], 28, 4, 128, 64, 64, True),
    ([40] * 70, [2] * 70, 2, 1, 64, 16, 16, False), ([3000], [2], 32, 1, 128, 1024, 256, False)])
def test_rows_match_the_oracle(lens, nodes, Hq, Hkv, D, page, block, tree, code, dtype):
    s = Quantised(7, lens, nodes, Hq=Hq, Hkv=Hkv, D=D, page=page, block=block, code=code, dtype=dtype, sigma=1.5)
    parents = _parents(s) if tree else None
    print(f"attention {lens[:4]} {nodes[:4]} {Hq}/{Hkv} {D} {page}/{block} {code} {dtype}", flush=True)
    out, lse = _run(s, parents)
    s.check(out, lse, s.reference(parents))


@pytest.mark.parametrize("code,dtype", [("i8", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 1), (5, 0), (17, 40), (130, 4), (513, 200), (700, 129),
                                          (2 ** 31 - 1, 7)])
def test_windows_and_sinks(window, sinks, code, dtype):
    lens, nodes = [1500, 0, 3, 640, 129, 20, 1281], [7, 20, 12, 1, 16, 9, 3]
    s = Quantised(8, lens, nodes, Hq=8, Hkv=2, D=64, page=32, block=16, code=code, dtype=dtype)
    for parents in (None, _parents(s)):
        out, lse = _run(s, parents, window=window, sinks=sinks)
        s.check(out, lse, s.reference(parents, window, sinks))


def test_many_rows_through_a_window():
    lens, nodes = [4000, 2777, 90], [64, 40, 64]
    s = Quantised(9, lens, nodes, Hq=14, Hkv=2, D=128, page=64, block=32)
    parents = _parents(s)
    out, lse = _run(s, parents, window=1025, sinks=5)
    s.check(out, lse, s.reference(parents, 1025, 5))


def test_what_a_window_hides_is_not_read():
    """Pages outside the window and the sinks may be gone: their table entries are
    not followed, and nothing is reported."""
    import torch
    s = Quantised(10, [2000, 900], [4, 1], Hq=4, Hkv=2, D=64)
    ref = s.reference(None, 300, 20)
    t = s.table.copy()
    t[0, 2:106] = -5
    t[1, 2:37] = 10 ** 6
    s.d["page_table"] = dev(t)
    st = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    out, lse = _run(s, window=300, sinks=20, status=st)
    s.check(out, lse, ref)
    assert st.tolist() == [0, 0]


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales_of_any_sign(scale):
    s = Quantised(11, [200, 33], [5, 2], Hq=4, Hkv=2, D=64, sigma=0.7)
    out, lse = _run(s, scale=scale)
    s.check(out, lse, s.reference(scale=scale), scale)


def test_scales_far_apart():
    """Value scales over 2^80: what a token of a small one adds is as exact as its
    share, and rows that see only small ones are whole."""
    for D in (64, 128):
        s = Quantised(12, [96, 48], [3, 2], Hq=4, Hkv=2, D=D)
        for b, p in enumerate(s.table[:, :6].tolist()):
            for i, page in enumerate(p):
                e = [0, 40, -40, 12, -30, 25][i] if b == 0 else -45 - i
                s.vs[page] = np.float32(2.0) ** e
        s.d["v_scale"] = dev(s.vs)
        # the second request's own values would drown its cache's
        s.vn[3:] *= 0
        s.d["v_new"] = dev(s.vn, torch_dtype("bf16"))
        out, lse = _run(s)
        o, e, mag = s.reference()
        got = out.double().cpu().numpy()
        # n weights below 2^-32 of the largest w = p vs each, the rest as elsewhere
        es = s.score_error()
        tol = (2.0 ** -8 + 2.0 ** -11 + 2 * es + 200 * 2.0 ** -24) * mag + 160 * 2.0 ** -32 * 128 * mag.max(-1, keepdims=True)
        assert (np.abs(got - o) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - e) <= es + 2.0 ** -16).all()


def test_blocks_of_zeros_and_unsound_scales():
    import torch
    sdv = _sdv()
    s = Quantised(13, [130, 64, 32], [4, 1, 2], Hq=4, Hkv=2, D=64)
    p = s.table
    s.ks[p[0, 1], 0] = 0                       # keys of zeros: scores 0
    s.vs[p[0, 2], 1] = 0                       # values of zeros, whatever the codes
    s.ks[p[0, 3], 1] = np.nan
    s.vs[p[0, 5], 0] = np.inf
    s.vs[p[1, 0], 0] = -1.0
    s.ks[p[1, 3], 1] = 2.0 ** -51
    s.d["k_scale"], s.d["v_scale"] = dev(s.ks), dev(s.vs)
    st = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    out, lse = _run(s, status=st)
    ref = s.reference()
    for x in (s.ks, s.vs):
        x[~(np.abs(x) < 1e6)] = 1.0
    s.check(out, lse, ref)
    assert st.tolist() == [sdv.SD_ST_BAD_SCALE, sdv.SD_ST_BAD_SCALE, 0]


@pytest.mark.parametrize("D", [64, 128])
def test_e4m3_codes_that_are_not_numbers_count_as_zero(D):
    s = Quantised(14, [300, 50], [3, 2], Hq=8, Hkv=2, D=D, code="e4m3", page=32, block=32)
    p = s.table
    s.k[p[0, 1], 0, 5, 7] = np.nan
    s.v[p[0, 4], 1, 30, D - 1] = np.nan
    s.v[p[1, 0], 0, 0] = np.nan
    s.d["k_cache"], s.d["v_cache"] = code_dev(s.k, "e4m3"), code_dev(s.v, "e4m3")
    for window in (0, 40):
        out, lse = _run(s, window=window)
        s.check(out, lse, s.reference(None, window))


def test_values_that_are_not_finite_stay_with_the_rows_that_see_them():
    import torch
    s = Quantised(15, [60, 20], [6, 3], Hq=4, Hkv=2, D=64)
    parents = np.array([-1, 0, 0, 1, 2, 4, -1, 0, 0], dtype=np.int32)
    ref = s.reference(parents)
    s.vn[3, 0, 5], s.vn[4, 1, 6] = np.inf, np.nan
    s.vn[7, 1, 0] = -np.inf
    s.kn[8, 0, 3] = np.nan
    s.d["v_new"], s.d["k_new"] = dev(s.vn, torch.bfloat16), dev(s.kn, torch.bfloat16)
    out, lse = _run(s, parents)
    o = out.double().cpu().numpy()
    touched = np.zeros(o.shape, dtype=bool)
    touched[3, :2, 5] = touched[4, 2:, 6] = touched[5, 2:, 6] = touched[7, 2:, 0] = True
    assert (o[3, :2, 5] == np.inf).all() and np.isnan(o[4:6, 2:, 6]).all() and (o[7, 2:, 0] == -np.inf).all()
    assert np.isnan(o[8, :2]).all() and torch.isnan(lse[8, :2]).all()
    touched[8, :2] = True
    clean = np.where(touched, ref[0], o)
    lse = lse.clone()
    lse[8, :2] = torch.from_numpy(ref[1][8, :2]).float().cuda()
    s.vn, s.kn = np.nan_to_num(s.vn, posinf=1, neginf=-1), np.nan_to_num(s.kn)
    s.check(torch.from_numpy(clean), lse, ref)


def test_defects_and_rows_of_no_request():
    import torch
    sdv = _sdv()
    s = Quantised(16, [100, 40, 64, 30, 20], [4, 3, 2, 1, 5], Hq=4, Hkv=2, D=64, behind=3)
    t = s.table.copy()
    t[0, 1] = -1                                            # bad pages are left out
    t[2, :4] = 10 ** 6
    s.table = t
    s.d["page_table"] = dev(t)
    parents = np.concatenate([_parents(s), [-1, 0, 0]]).astype(np.int32)
    parents[s.offsets[4] + 2] = 2                           # its own parent: a root
    ref_parents = parents.copy()
    ref = s.reference(ref_parents)
    ctx = np.array(s.lens, dtype=np.int32)
    ctx[1] = 10 ** 6
    s.d["context_lens"] = dev(ctx)
    st = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((s.N + 3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.N + 3, 4), 7.0, device="cuda")
    _sdv().quant_attention(**s.attention_args(), max_nodes=5, parents=dev(parents), out=out, lse=lse, status=st)
    assert st.tolist() == [sdv.SD_ST_BAD_PAGE, sdv.SD_ST_BAD_LEN, sdv.SD_ST_BAD_PAGE, 0, sdv.SD_ST_BAD_TREE]
    assert (out[s.N:] == 7).all() and (lse[s.N:] == 7).all()
    lo, hi = s.offsets[1], s.offsets[2]
    assert (out[lo:hi] == 0).all() and (lse[lo:hi] == -np.inf).all()
    ref[0][lo:hi], ref[1][lo:hi], ref[2][lo:hi] = 0, -np.inf, 0
    s.check(out, lse, ref)
    off = np.array([0, 4, 2, 9, 10, 99], dtype=np.int32)    # decreasing, too many, past N
    st.fill_(-1)
    out.fill_(7.0)
    s.d["node_offsets"], s.d["context_lens"] = dev(off), dev(np.array(s.lens, dtype=np.int32))
    _sdv().quant_attention(**s.attention_args(), max_nodes=5, out=out, status=st)
    N = sdv.SD_ST_BAD_NODES
    assert [x & N for x in st.tolist()] == [0, N, N, 0, N]
    assert (out[4:9] == 7).all() and (out[10:] == 7).all() and not (out[:4] == 7).all()


def test_in_place_of_queries_and_strided_caches():
    import torch
    for kw in (dict(slot_major=True), dict(packed=True)):
        s = Quantised(17, [90, 300], [6, 2], Hq=4, Hkv=2, D=128, **kw)
        out, lse = _run(s)
        s.check(out, lse, s.reference())
    q = s.d["q"] = s.d["q"].contiguous()
    got, lse2 = _run(s, out=q)
    assert got is q and torch.equal(got, out) and torch.equal(lse, lse2)


def test_results_repeat_and_graphs_replay():
    import torch
    sdv = _sdv()
    s = Quantised(18, [3000, 170, 1200], [9, 3, 5], Hq=8, Hkv=2, D=128)
    a = s.attention_args()
    out, lse = _run(s)
    again, lse2 = _run(s)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    n = sdv.quant_attention_workspace_bytes(sdv.make_quant_attention_args(**a, max_nodes=9))
    assert n > 0
    ws = [torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2)]
    res = [torch.zeros_like(out) for _ in range(2)]
    graphs = []
    for w, r in zip(ws, res):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sdv.quant_attention(**a, max_nodes=9, out=r, workspace=w, window=0 if r is res[0] else 700)
        graphs.append(g)
    for _ in range(3):
        a["q"].copy_(torch.randn_like(a["q"]))
        want = [sdv.quant_attention(**a, max_nodes=9, window=w)[0] for w in (0, 700)]
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], res[0]) and torch.equal(want[1], res[1])


@pytest.mark.parametrize("far", ["pages", "heads"])
def test_caches_past_4_gib(far):
    """Pages, or heads, further apart than 32 bits reach: appended to and attended as
    the same cache close together, on a stream of its own."""
    import torch
    sdv = _sdv()
    names = ("k_cache", "v_cache", "k_scale", "v_scale")
    s = Quantised(19, [150, 61], [9, 5], Hq=4, Hkv=2, D=128, page=32, block=16, room=16)
    near = s.d
    pool, H, page, D = near["k_cache"].shape
    wide = dict(near)
    stride = (5 << 30) // (pool if far == "pages" else 1) & -16
    strides = (stride, page * D, D, 1) if far == "pages" else (page * D, stride, D, 1)
    for n in names[:2]:
        buf = torch.empty(stride * ((pool if far == "pages" else H) - 1) + pool * H * page * D, dtype=torch.int8, device="cuda")
        wide[n] = buf.as_strided(near[n].shape, strides)
        wide[n].copy_(near[n])
    for n in names[2:]:
        wide[n] = near[n].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res = []
    for d, st in ((near, None), (wide, side)):
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        sdv.quant_append(d["k_new"], d["v_new"], *(d[n] for n in names), d["page_table"], d["context_lens"],
                         d["node_offsets"], 9, lens, stream=st)
        res.append(sdv.quant_attention(d["q"], d["k_new"], d["v_new"], *(d[n] for n in names), d["page_table"], lens,
                                       d["node_offsets"], 9, want_lse=True, stream=st))
        torch.cuda.synchronize()
        assert lens.tolist() == [159, 66]
    for n in names:
        assert torch.equal(near[n].contiguous().view(torch.uint8), wide[n].contiguous().view(torch.uint8)), n
    assert all(torch.equal(a, b) for a, b in zip(*res)) and torch.isfinite(res[0][0]).all()


def test_requests_that_share_pages_and_calls_at_once():
    """A prefix held once for all requests, and calls on streams and workspaces of
    their own at the same time."""
    import torch
    s = Quantised(20, [700] * 5, [3] * 5, Hq=14, Hkv=2, D=64, page=64, block=64, code="e4m3")
    s.table[:, :6] = s.table[0, :6]
    s.d["page_table"].copy_(dev(s.table))
    out, lse = _run(s)
    s.check(out, lse, s.reference())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(3):
        got = [_run(s, stream=st) for st in streams]
        torch.cuda.synchronize()
        for o, e in got:
            assert torch.equal(o, out) and torch.equal(e, lse)


@pytest.mark.parametrize("nodes,Hq,Hkv", [([13, 20, 27], 14, 2), ([64, 33, 5], 8, 2), ([64, 1, 50], 3, 1)])
def test_more_rows_than_a_row_tile(nodes, Hq, Hkv):
    """65 to 256 rows a KV head: codes that are not numbers in the cache, infinities
    and NaN in nodes that only their descendants see, in place of the queries."""
    import torch
    s = Quantised(21, [900, 300, 2000], nodes, Hq=Hq, Hkv=Hkv, D=128, code="e4m3", page=32, block=32)
    parents = _parents(s)
    for b in range(3):      # the last node: nobody else sees it
        parents[s.offsets[b + 1] - 1] = 0 if nodes[b] > 1 else -1
    p = s.table
    s.k[p[0, 3], 0, 5, 7] = np.nan
    s.v[p[2, 40], Hkv - 1, 30, 127] = np.nan
    s.d["k_cache"], s.d["v_cache"] = code_dev(s.k, "e4m3"), code_dev(s.v, "e4m3")
    ref = s.reference(parents)
    last = [int(o) - 1 for o in s.offsets[1:]]
    s.vn[last[0], 0, 5], s.vn[last[2], Hkv - 1, 127] = np.inf, np.nan
    s.d["v_new"] = dev(s.vn, torch.bfloat16)
    out, lse = _run(s, parents)
    o = out.double().cpu().numpy()
    G = Hq // Hkv
    touched = np.zeros(o.shape, dtype=bool)
    touched[last[0], :G, 5] = touched[last[2], Hq - G:, 127] = True
    assert (o[last[0], :G, 5] == np.inf).all() and np.isnan(o[last[2], Hq - G:, 127]).all()
    s.vn = np.nan_to_num(s.vn, posinf=1)
    s.check(torch.from_numpy(np.where(touched, ref[0], o)), lse, ref)
    q = s.d["q"] = s.d["q"].contiguous()
    got, again = _run(s, parents, out=q)
    assert torch.equal(got.nan_to_num(), out.nan_to_num()) and torch.equal(again, lse)


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_near_the_largest_of_their_type(D, code):
    """bf16 queries of up to 2^126 over small keys: scores of 2^80 and more, but numbers.
    One key has all the weight: its value, off by half a step of the result and of the
    weight in fp16, 2^-20 for the rest; lse within the scores' error."""
    import torch
    s = Quantised(30, [300, 45], [3, 1], Hq=8, Hkv=2, D=D, code=code, page=32, block=16)
    for x in (s.ks, s.vs):
        x[~np.isfinite(x)] = 1.0
    s.ks = (s.ks * np.float32(2.0 ** -43)).astype(np.float32)
    big = 2.0 ** np.array([110.0, 121.0, 123.0, 124.0])
    s.q = rounded(s.q * big[:, None, None], "bf16")
    s.kn = rounded(s.kn * 2.0 ** -100, "bf16")
    s.d.update(q=dev(s.q, torch.bfloat16), k_new=dev(s.kn, torch.bfloat16), k_scale=dev(s.ks))
    out, lse = _run(s)
    o, e, mag = s.reference()
    es = (D + 8) * 2.0 ** -24 * s.scale * D * np.abs(s.q).max(-1) * s.ks.max() * oracle.serve.TOP[code]
    assert (e > 2.0 ** 60).all() and np.isfinite(e).all()
    assert (np.abs(mag - np.abs(o)) <= 2.0 ** -40 * mag).all()       # one key alone, by far
    got = out.double().cpu().numpy()
    assert (np.abs(got - o) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * np.abs(o)).all()
    assert (np.abs(lse.double().cpu().numpy() - e) <= es + 2.0 ** -22 * e).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,D", [
    ([0, 0, 0], [2, 5, 64], 4, 2, 64), ([0, 0], [64, 33], 14, 2, 128), ([0, 0], [1, 40], 6, 2, 128),
    ([1, 3, 20], [1, 4, 16], 14, 2, 64), ([2000, 40], [9, 64], 28, 4, 128)])
def test_values_that_are_all_alike_are_their_average(lens, nodes, Hq, Hkv, D, dtype):
    """Whatever the weights are: those of the nodes are exact to 16 bits and those of the
    cache to fp16's 11, far from what half a step of the values' type would need."""
    import torch
    s = Quantised(31, lens, nodes, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, sigma=1.2)
    dt = torch_dtype(dtype)
    if max(lens):
        if dtype == "f16":       # (its cached weights may be off by more than half a step)
            lens = s.lens = [0] * len(lens)
            s.d["context_lens"].zero_()
        s.d["k_scale"].mul_(0.5)
        s.d["v_cache"].fill_(64)
        s.d["v_scale"].fill_(2.0 ** -6)
        values = torch.ones(D)
    else:
        values = torch.tensor(rounded(s.rng.uniform(0.25, 4, D), dtype))
    s.d["v_new"] = values.to(dt).cuda().expand(s.N, Hkv, D).contiguous()
    for parents in (None, _parents(s)):
        out, _ = _run(s, parents)
        assert torch.equal(out, values.to(dt).cuda().expand_as(out))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_node_that_dominates_is_as_exact_as_its_value(D, dtype):
    """One slot whose score is 0 and a node, both of value 127: their average is 127
    whatever the weights, so a weight that is off by more than half a step of the
    result's type shows."""
    import torch
    s = Quantised(38, [1] * 20, [1] * 20, Hq=28, Hkv=4, D=D, dtype=dtype, sigma=4.0)
    dt = torch_dtype(dtype)
    s.d["k_scale"].zero_()
    s.d["v_cache"].fill_(127)
    s.d["v_scale"].fill_(1.0)
    s.d["v_new"].fill_(127)
    out, lse = _run(s)
    x = np.einsum("nhgd,nhd->nhg", s.q.reshape(20, 4, 7, D), s.kn).reshape(20, 28) * s.scale
    assert ((x > 2) & (x < 5.5)).mean() > 0.1        # nodes of 2^3 to 2^8 times the slot's weight
    assert torch.equal(out, torch.full_like(out, 127))
    assert (np.abs(lse.double().cpu().numpy() - np.logaddexp(0, x)) <= s.score_error() + 2.0 ** -20).all()


def test_unsound_scales_that_no_row_sees_are_not_reported():
    """Blocks outside the window and the sinks, on pages of which a part is seen."""
    import torch
    sdv = _sdv()
    s = Quantised(32, [400, 400, 400, 120], [3, 1, 2, 2], Hq=4, Hkv=2, D=64, page=128, block=16)
    # the window of 100 shows slots from 301 on (block 2 of page 2), the 20 sinks blocks 0 and 1
    t = s.table
    ref = s.reference(None, 100, 20)
    for p, blk in ((0, 2), (0, 7), (2, 1), (1, 3)):
        s.ks[t[0, p], 1, blk] = np.nan
        s.vs[t[0, p], 0, blk] = -2.0
    s.vs[t[1, 2], 1, 2] = np.inf             # seen by the window
    s.ks[t[2, 0], 0, 1] = -1.0               # seen among the sinks
    s.ks[t[3, 0], 0, 7] = np.inf             # the last one in use
    s.d["k_scale"], s.d["v_scale"] = dev(s.ks), dev(s.vs)
    st = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    out, lse = _run(s, window=100, sinks=20, status=st)
    bad = sdv.SD_ST_BAD_SCALE
    assert st.tolist() == [0, bad, bad, bad]
    rows = slice(0, int(s.offsets[1]))
    s2 = Quantised(32, [400, 400, 400, 120], [3, 1, 2, 2], Hq=4, Hkv=2, D=64, page=128, block=16)
    clean, clean_lse = _run(s2, window=100, sinks=20)
    assert torch.equal(out[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows])
    s2.check(clean, clean_lse, ref)
    _run(s, status=st)                       # without a window everything is seen
    assert st.tolist() == [bad] * 4


def test_strides_of_axes_of_one_say_nothing():
    """One node of a fused projection in place; a cache of one head and one page whose
    strides along them are anything."""
    import torch
    s = Quantised(33, [90], [1], Hq=4, Hkv=2, D=64, packed=True)
    out, lse = _run(s)
    s.check(out, lse, s.reference())
    q = s.d["q"]
    assert q.is_contiguous() and q.stride(0) != q.shape[1] * q.shape[2]
    got, again = _run(s, out=q)
    assert got is q and torch.equal(got, out) and torch.equal(lse, again)
    s = Quantised(34, [50], [3], Hq=4, Hkv=1, D=64, page=64, block=32, packed=True)
    s.table[:] = 0
    s.k, s.v, s.ks, s.vs = (x[:1] for x in (s.k, s.v, s.ks, s.vs))
    d = s.d
    d["page_table"].zero_()
    for n, x in (("k_cache", s.k), ("v_cache", s.v), ("k_scale", s.ks), ("v_scale", s.vs)):
        d[n] = code_dev(x, "i8") if "cache" in n else dev(x)
    out, lse = _run(s)
    s.check(out, lse, s.reference())
    for n in ("k_cache", "v_cache"):
        d[n] = d[n].as_strided((1, 1, 64, 64), (3, 5, 64, 1))
    for n in ("k_new", "v_new"):
        d[n] = d[n].contiguous().as_strided((3, 1, 64), (64, 7, 1))
    got, again = _run(s)
    assert torch.equal(got, out) and torch.equal(lse, again)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    _sdv().quant_append(*(d[n] for n in ("k_new", "v_new", "k_cache", "v_cache", "k_scale", "v_scale", "page_table",
                                         "context_lens", "node_offsets")), 3, lens)
    assert lens.tolist() == [53]


@pytest.mark.parametrize("code,dtype", [("i8", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,D,page", [
    ([3000, 1], [1, 1], 14, 2, 64, 16), ([3000, 0, 1700, 2999], [1, 1, 1, 0], 28, 4, 128, 32),
    ([3000, 800], [4, 2], 14, 2, 64, 64), ([1500, 3001, 77], [3, 4, 4], 28, 4, 128, 16)])
def test_few_rows_over_many_tiles(lens, nodes, Hq, Hkv, D, page, code, dtype):
    """Decoding in tables of more tiles than one workgroup takes: 16 and 32 rows of a KV
    head, split over workgroups and joined."""
    import torch
    s = Quantised(35, lens, nodes, Hq=Hq, Hkv=Hkv, D=D, page=page, block=16, code=code, dtype=dtype, sigma=1.5)
    n = _sdv().quant_attention_workspace_bytes(_sdv().make_quant_attention_args(**s.attention_args(), max_nodes=max(nodes)))
    assert n > 0
    out, lse = _run(s, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
    s.check(out, lse, s.reference())


@pytest.mark.parametrize("code,T,Hq", [("i8", 1, 2), ("e4m3", 4, 8), ("i8", 20, 2), ("e4m3", 30, 3)])
def test_many_requests_in_split_tables(code, T, Hq):
    """Three times 64 requests, most of them short, some without nodes, some long."""
    import torch
    rng = np.random.default_rng(36)
    B = 135
    lens, nodes = rng.integers(0, 50, B), rng.integers(0, T + 1, B)
    lens[[3, 63, 64, 66, 130, 134]] = [1500, 700, 1490, 64, 1333, 900]
    nodes[[3, 64, 130, 134]] = T
    nodes[[0, 62, 65, 127, 128]] = 0
    s = Quantised(36, lens.tolist(), nodes.tolist(), Hq=Hq, Hkv=1, D=64, page=64, block=32, code=code)
    n = _sdv().quant_attention_workspace_bytes(_sdv().make_quant_attention_args(**s.attention_args(), max_nodes=T))
    assert n > 0
    parents = _parents(s)
    out, lse = _run(s, parents, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
    s.check(out, lse, s.reference(parents))


@pytest.mark.parametrize("T,G", [(2, 2), (4, 7), (20, 2), (48, 2)])
@pytest.mark.parametrize("code,dtype,D", [("i8", "bf16", 64), ("e4m3", "bf16", 128), ("i8", "f16", 128), ("e4m3", "f16", 64)])
def test_runs_of_more_tiles_than_are_looked_up_at_once(T, G, code, dtype, D):
    """A large batch of long contexts, whose workgroups go through more than 32 tiles on
    end: scales that differ from block to block, unsound ones and codes that are not
    numbers all along.  Every row against a softmax in 64 bits."""
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(37)
    B, H, page, block, pool = 66, 8, 128, 32, 150
    lens = rng.integers(4300, 6000, B)
    nodes = rng.integers(1, T + 1, B)
    nodes[[0, 1, 65]] = T
    nodes[40] = 0
    off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    N, Hq = int(off[-1]), H * G
    table = rng.integers(0, pool, (B, 47)).astype(np.int32)      # (requests share pages)
    k, ks = random_cache(rng, pool, H, page, D, block, code, 0.3)
    v, vs = random_cache(rng, pool, H, page, D, block, code, 0.3)
    kd, vd = code_dev(k, code), code_dev(v, code)
    if code == "e4m3":
        kd[5, 3, 17, 9] = float("nan")
        vd[77, 1, 100, D - 2] = float("nan")
    for x, value in ((ks, np.nan), (ks, -1.0), (vs, np.inf), (vs, 2.0 ** -60)):
        x[rng.random(x.shape) < 0.005] = value
    dt = torch_dtype(dtype)
    q, kn, vn = (dev(rng.standard_normal((N, h, D)) * sigma, dt) for h, sigma in ((Hq, 2.0), (H, 1.0), (H, 1.0)))
    t = {n: dev(x) for n, x in (("ks", ks), ("vs", vs), ("table", table), ("lens", lens.astype(np.int32)), ("off", off))}
    args = (q, kn, vn, kd, vd, t["ks"], t["vs"], t["table"], t["lens"], t["off"], T)
    out, lse = sdv.quant_attention(*args, want_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # the definition, a request and head at a time
    sound = lambda x: (x == 0) | ((x >= 2.0 ** -50) & (x <= 2.0 ** 50))  # noqa: E731
    there = (sound(t["ks"]) & sound(t["vs"]))
    key, val = (torch.nan_to_num(c.double()) * torch.where(there, x, 0).double().repeat_interleave(block, 2)[..., None]
                for c, x in ((kd, t["ks"]), (vd, t["vs"])))
    there = there.repeat_interleave(block, 2)
    top = oracle.serve.TOP[code]
    n = 6000 + T + 64
    qmax, big = q.double().abs().max(), max(np.nanmax(np.where(np.isfinite(vs), vs, 0)) * top, vn.abs().max().item())
    eps = EPS[dtype]
    es = (D + 8) * 2.0 ** -24 * D ** 0.5 * qmax.item() * max(np.nanmax(ks) * top, kn.abs().max().item()) + 2.0 ** -20
    more = n * 2.0 ** -24 * 255 * np.nanmax(np.where(np.isfinite(vs), vs, 0)) if code == "i8" else 0.0
    for b in range(B):
        lo, hi, m = int(off[b]), int(off[b + 1]), int(lens[b])
        if lo == hi:
            continue
        at = t["table"][b].long()
        for h in range(H):
            rows = lambda x: x[at, h].reshape(-1, *x.shape[3:])[:m]  # noqa: E731
            kk, vv = torch.cat([rows(key), kn[lo:hi, h].double()]), torch.cat([rows(val), vn[lo:hi, h].double()])
            sees = torch.cat([rows(there).expand(hi - lo, m), torch.ones((hi - lo, hi - lo), device="cuda").tril().bool()], 1)
            for g in range(h * G, (h + 1) * G):
                x = (q[lo:hi, g].double() @ kk.t() * D ** -0.5).masked_fill(~sees, -np.inf)
                w = torch.softmax(x, 1)
                o, mag = w @ vv, w @ vv.abs()
                tol = eps * o.abs() + (eps + 2 * es + n * 2.0 ** -24) * (1 + eps) * mag + n * 2.0 ** -32 * big + 2.0 ** -24 + more
                assert ((out[lo:hi, g].double() - o).abs() <= tol).all(), (b, h, g)
                e = torch.logsumexp(x, 1)
                assert ((lse[lo:hi, g].double() - e).abs() <= es + n * 2.0 ** -24 + 2.0 ** -22 * (1 + e.abs())).all(), (b, h, g)
