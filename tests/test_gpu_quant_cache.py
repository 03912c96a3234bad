"""sd_quant_append on the GPU against the oracle: scales and codes are equal, since
the definition is in fp32 and both follow it."""
import numpy as np
import pytest

import oracle
from servetools import Quantised, code_np
from treetools import dev, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _append(s, path=None, path_lens=None, max_new=None, status=None, **over):
    import torch
    d = {**s.d, **over}
    out = torch.full((len(s.lens),), -7, dtype=torch.int32, device="cuda")
    got = _sdv().quant_append(d["k_new"], d["v_new"], d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"],
                              d["page_table"], d["context_lens"], d["node_offsets"], max_new or max(s.nodes), out,
                              path=path, path_lens=path_lens, status=status)
    assert got is out
    return out


def _same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def _expect(s, rows):
    """The cache after appending these packed rows, request by request."""
    k, v, ks, vs = code_np(s.d["k_cache"]), code_np(s.d["v_cache"]), s.d["k_scale"].cpu().numpy(), s.d["v_scale"].cpu().numpy()
    for b, r in enumerate(rows):
        oracle.quant_append_ref(s.kn[r].astype(np.float32), k, ks, s.table[b], s.lens[b], s.block, s.code)
        oracle.quant_append_ref(s.vn[r].astype(np.float32), v, vs, s.table[b], s.lens[b], s.block, s.code)
    return k, v, ks, vs


def _state(s):
    return code_np(s.d["k_cache"]), code_np(s.d["v_cache"]), s.d["k_scale"].cpu().numpy(), s.d["v_scale"].cpu().numpy()


@pytest.mark.parametrize("code,dtype", [("i8", "bf16"), ("i8", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("lens,nodes,page,block,D,H", [
    ([0], [1], 16, 16, 64, 1), ([5, 16, 31], [1, 1, 1], 16, 16, 128, 2), ([0, 3, 40, 15], [70, 1, 33, 17], 16, 16, 64, 3),
    ([0, 100, 63], [200, 29, 65], 64, 32, 128, 2), ([1, 64], [131, 64], 64, 64, 128, 1), ([7, 0], [300, 256], 128, 128, 128, 2),
    ([9, 1000], [1500, 1100], 1024, 1024, 64, 1), ([17], [600], 512, 256, 128, 2)])
def test_rows_match_the_oracle(lens, nodes, page, block, D, H, code, dtype):
    s = Quantised(1, lens, nodes, Hq=H, Hkv=H, D=D, page=page, block=block, code=code, dtype=dtype, room=max(nodes))
    want = _expect(s, [range(s.offsets[b], s.offsets[b + 1]) for b in range(len(lens))])
    out = _append(s)
    assert out.tolist() == [n + m for n, m in zip(lens, nodes)]
    for g, w, name in zip(_state(s), want, ("k", "v", "k_scale", "v_scale")):
        assert _same(g, w), name


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_paths_and_strides(code):
    """The kept branch alone, out of a packed projection into a cache whose slots lie
    outside the heads; other rows of the pages stay as they were."""
    lens, nodes = [10, 33, 0, 47], [9, 4, 6, 1]
    s = Quantised(2, lens, nodes, Hq=4, Hkv=2, D=128, code=code, room=9, slot_major=True, packed=True)
    paths = [[0, 3, 8], [], [0, 1, 2, 3, 4, 5], [0]]
    path = np.full((4, 9), -1, dtype=np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    want = _expect(s, [[s.offsets[b] + i for i in p] for b, p in enumerate(paths)])
    out = _append(s, dev(path), dev(np.array([len(p) for p in paths], dtype=np.int32)))
    assert out.tolist() == [n + len(p) for n, p in zip(lens, paths)]
    for g, w, name in zip(_state(s), want, ("k", "v", "k_scale", "v_scale")):
        assert _same(g, w), name


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_token_by_token_is_the_definition_repeated(code):
    """A block filled one token at a time, its scale growing on the way: after each
    step within one rounding of every growth, and equal to the oracle's."""
    import torch
    rng = np.random.default_rng(3)
    s = Quantised(3, [0, 5], [1, 1], Hq=1, Hkv=1, D=64, code=code, room=40)
    for step in range(20):
        s.kn = rounded(rng.standard_normal((2, 1, 64)) * 1.25 ** step, "bf16")
        s.vn = rounded(rng.standard_normal((2, 1, 64)) * 0.8 ** step, "bf16")
        s.d["k_new"], s.d["v_new"] = dev(s.kn, torch.bfloat16), dev(s.vn, torch.bfloat16)
        want = _expect(s, [[0], [1]])
        out = _append(s)
        for g, w in zip(_state(s), want):
            assert _same(g, w)
        s.lens = out.tolist()
        s.d["context_lens"] = out
    assert s.lens == [20, 25]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_zeros_tiny_huge_and_unsound_values(code):
    import torch
    sdv = _sdv()
    lens, nodes = [0, 0, 3, 0, 0, 4], [16, 16, 5, 17, 1, 2]
    s = Quantised(4, lens, nodes, Hq=1, Hkv=1, D=64, code=code, room=20)
    o = s.offsets
    s.kn[o[0]:o[1]] = 0                                      # a block of zeros: scale 0
    s.kn[o[1]:o[2]] = rounded(s.kn[o[1]:o[2]] * 1e-20, "bf16")        # below the least scale
    s.kn[o[2], 0, 7], s.kn[o[2] + 1, 0, 3], s.kn[o[2] + 2, 0, 1] = np.nan, np.inf, -np.inf
    s.kn[o[3]:o[4]] = rounded(s.kn[o[3]:o[4]] * 1e25, "bf16")         # above the largest
    s.vn[o[4]] = np.nan                                      # nothing that is finite
    ks = s.d["k_scale"]
    ks[s.table[5, 0]] = float("nan")                         # an old scale that is none
    s.ks[s.table[5, 0]] = np.nan
    s.d["k_new"], s.d["v_new"] = dev(s.kn, torch.bfloat16), dev(s.vn, torch.bfloat16)
    want = _expect(s, [range(o[b], o[b + 1]) for b in range(6)])
    st = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    _append(s, status=st)
    for g, w, name in zip(_state(s), want, ("k", "v", "k_scale", "v_scale")):
        assert _same(g, w), name
    assert st.tolist() == [0, 0, sdv.SD_ST_NONFINITE, 0, sdv.SD_ST_NONFINITE, 0]
    assert ks[s.table[0, 0], 0, 0] == 0 and ks[s.table[1, 0], 0, 0] == 2.0 ** -50 and ks[s.table[3, 0], 0, 0] == 2.0 ** 50


def test_defects_append_nothing():
    import torch
    sdv = _sdv()
    lens, nodes = [3, 4, 5, 6, 20, 9], [4] * 6
    s = Quantised(5, lens, nodes, Hq=2, Hkv=2, D=64, room=12)
    path = np.tile(np.array([0, 1, 2, 3], dtype=np.int32), (6, 1))
    path[0, 1] = 4                                          # past the request's nodes
    path[1, 2] = -1
    m = np.array([2, 3, 5, 3, 1, 0], dtype=np.int32)        # request 2: longer than its nodes
    table = s.table.copy()
    table[3, 0] = 10 ** 6                                   # a bad page
    cap = table.shape[1] * s.page
    ctx = np.array(lens, dtype=np.int32)
    ctx[4] = cap                                            # no room for one more
    before = _state(s)
    st = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    out = _append(s, dev(path), dev(m), status=st, page_table=dev(table), context_lens=dev(ctx))
    assert st.tolist() == [sdv.SD_ST_BAD_PATH] * 3 + [sdv.SD_ST_BAD_PAGE, sdv.SD_ST_BAD_LEN, 0]
    assert out.tolist() == [3, 4, 5, 9, cap, 9]
    for g, w in zip(_state(s), before):
        assert _same(g, w)
    # offsets that decrease or give a request too many nodes; lengths outside the table
    off = np.array([0, 4, 2, 8, 25, 24, 24], dtype=np.int32)
    ctx = np.array([-1, 4, 5, 6, 7, cap + 1], dtype=np.int32)
    st.fill_(-1)
    out = _append(s, max_new=4, status=st, node_offsets=dev(off), context_lens=dev(ctx))
    N, L = sdv.SD_ST_BAD_NODES, sdv.SD_ST_BAD_LEN
    assert st.tolist() == [L, N, N, N, N, L]
    assert out.tolist() == ctx.tolist()
    for g, w in zip(_state(s), before):
        assert _same(g, w)


def test_append_in_a_graph():
    """Captured and replayed with new rows and lengths: each replay as an eager call."""
    import torch
    sdv = _sdv()
    s = Quantised(6, [0, 0], [24, 24], Hq=2, Hkv=2, D=128, page=32, block=32, room=200)
    d = s.d
    out, ctx = torch.zeros(2, dtype=torch.int32, device="cuda"), d["context_lens"]
    names = ("k_cache", "v_cache", "k_scale", "v_scale")
    call = lambda x: sdv.quant_append(d["k_new"], d["v_new"], *(x[n] for n in names), d["page_table"], ctx,  # noqa: E731
                                      d["node_offsets"], 24, out)
    call(d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d)
    ctx.zero_()
    eager = {n: d[n].clone() for n in names}
    for _ in range(4):
        d["k_new"].copy_(torch.randn_like(d["k_new"]))
        d["v_new"].copy_(torch.randn_like(d["v_new"]))
        call(eager)
        g.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(d[n].view(torch.uint8), eager[n].view(torch.uint8)), n
        ctx.copy_(out)
    assert ctx.tolist() == [96, 96]


def test_path_and_its_lengths_come_together():
    """One without the other is refused, and nothing is appended."""
    import torch
    s = Quantised(8, [5, 9], [3, 2], Hq=2, Hkv=2, D=64, room=8)
    before = _state(s)
    path, m = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for kw in (dict(path=path), dict(path_lens=m)):
        with pytest.raises(ValueError, match="path"):
            _append(s, **kw)
    for g, w in zip(_state(s), before):
        assert _same(g, w)
