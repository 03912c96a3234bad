"""sd_beam_select and sd_beam_reorder on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest

import oracle
from treetools import dev, rounded, torch_dtype

pytestmark = pytest.mark.gpu

# A candidate's score: the fp32 exponentials of a row are off by 2^-23 of the
# magnitude of their exponent (under 24 for what a sum can notice) and an ulp,
# so its log-sum-exp by 26 * 2^-23; the result is rounded to fp32.
LSE_ERR = 26 * 2.0 ** -23


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _check(z, scores, n_out, got, ended=None, eos=-1):
    s, par, tok = (t.cpu().numpy() for t in got[:3])
    exact = 0
    for b in range(z.shape[0]):
        ref = oracle.beam_select_ref(z[b], scores[b], n_out + 1, None if ended is None else ended[b], eos)
        for j in range(n_out):
            if j >= len(ref):
                assert s[b, j] == -np.inf and par[b, j] == -1 and tok[b, j] == -1
                continue
            x, w, t = ref[j]
            tol = LSE_ERR + abs(x) * 2.0 ** -23
            assert abs(s[b, j] - x) <= tol, (b, j, s[b, j], x)
            # beams within twice the error of each other may swap; the order within a beam is exact
            near = any(abs(ref[i][0] - x) <= 2 * tol and ref[i][1] != w for i in (j - 1, j + 1) if 0 <= i < len(ref))
            if not near:
                assert (par[b, j], tok[b, j]) == (w, t), (b, j, ref[max(0, j - 1):j + 2])
                exact += 1
    return exact


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,n_out", [(1, 1, 1, 1), (2, 3, 5, 4), (3, 4, 1000, 8), (2, 8, 20011, 8), (1, 64, 300, 64),
                                         (1, 5, 152064, 10), (2, 2, 8192, 64), (1, 3, 4099, 64), (40, 2, 257, 3)])
def test_select_matches_the_oracle(B, W, V, n_out, dtype):
    rng = np.random.default_rng(B * W + V)
    z = rounded(rng.standard_normal((B, W, V)) * 3, dtype)
    sc = (-rng.random((B, W)) * 5).astype(np.float32)
    ld = -(-V // 8) * 8 + 8
    full = np.full((B, W, ld), np.nan)
    full[..., :V] = z
    x = dev(full, torch_dtype(dtype))[..., :V]
    print(f"select {B} {W} {V} {n_out} {dtype}", flush=True)
    got = _sdv().beam_select(x, dev(sc), n_out)
    exact = _check(z, sc, n_out, got)
    assert exact >= 0.9 * min(n_out, W * V) * B


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_go_to_the_lowest_beam_and_token(dtype):
    """Rows of few distinct values, rows all equal, equal rows in several beams
    and sorted rows."""
    import torch
    V = 5000
    rng = np.random.default_rng(3)
    z = np.zeros((5, 4, V))
    z[0] = 1.0
    z[1] = rng.integers(0, 3, (4, V))
    z[2] = rng.standard_normal(V)[None]
    z[3] = np.arange(V)[None] / 64.0
    z[4] = -np.arange(V)[None] / 64.0
    z = rounded(z, dtype)
    sc = np.zeros((5, 4), dtype=np.float32)
    got = _sdv().beam_select(dev(z, torch_dtype(dtype)), dev(sc), 40)
    s, par, tok = (t.cpu().numpy() for t in got)
    for b in range(5):
        same = [w for w in range(4) if (z[b, w] == z[b, 0]).all()]
        if len(same) == 4:      # equal rows have equal sums: the flat order is exact
            order = np.argsort(-np.concatenate([z[b, w] for w in range(4)]), kind="stable")[:40]
            assert list(zip(par[b], tok[b])) == [(i // V, i % V) for i in order], b
    _check(z, sc, 40, got)
    assert torch.equal(got[0], _sdv().beam_select(dev(z, torch_dtype(dtype)), dev(sc), 40)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", ["lowest", -1e30, -1e20, -1e10])
def test_masked_vocabularies(dtype, value):
    """Finite mask values over runs of neighbouring tokens, the end of the
    vocabulary, or all tokens but a few: the sums of the others stand, and the
    masked tokens are candidates behind them."""
    import torch
    rng = np.random.default_rng(11)
    B, W, V, n = 4, 3, 9001, 12
    low = float(torch.finfo(torch_dtype(dtype)).min) if value == "lowest" else value
    z = rng.standard_normal((B, W, V)) * 3
    z[0, :, 64:4000] = low                        # a run
    z[1, :, 7000:] = low                          # a padded vocabulary
    keep = rng.integers(0, V, (W, 3))             # a constraint that leaves three tokens
    few = np.full((W, V), low)
    for w in range(W):
        few[w, keep[w]] = z[2, w, keep[w]]
    z[2] = few
    z[3, :, ::2] = low                            # every other one
    z = rounded(z, dtype)
    sc = (-rng.random((B, W)) * 2).astype(np.float32)
    ld = -(-V // 8) * 8
    full = np.full((B, W, ld), np.nan)
    full[..., :V] = z
    status = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    print(f"masked {dtype} {value}", flush=True)
    got = _sdv().beam_select(dev(full, torch_dtype(dtype))[..., :V], dev(sc), n, status=status)
    assert status.tolist() == [0] * B
    assert _check(z, sc, n, got) >= 3 * B


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_do_not_depend_on_the_level_of_the_logits(dtype):
    """Rows far from zero, another level for every beam: a score is a
    difference, as exact there as anywhere."""
    rng = np.random.default_rng(12)
    B, W, V, n = 3, 6, 20011, 10
    z = rng.standard_normal((B, W, V)) * 3
    z[0] += np.array([1000.0, -5000.0, 0.0, 30.0, 100.0, -77.0])[:, None]
    z[1] += 1000.0
    z[2] -= np.array([4000.0, 4100.0, 1e5, 2e4, 3e4, 5e4])[:, None]
    z[2, 3, 77] += 400.0                          # one token that dominates
    z = rounded(z, dtype)
    sc = (-rng.random((B, W)) * 2).astype(np.float32)
    ld = -(-V // 8) * 8
    full = np.full((B, W, ld), np.nan)
    full[..., :V] = z
    print(f"levels {dtype}", flush=True)
    got = _sdv().beam_select(dev(full, torch_dtype(dtype))[..., :V], dev(sc), n)
    assert _check(z, sc, n, got) >= n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_nothing_but_masks_are_uniform(dtype):
    """A beam whose logits are all the same mask value spreads its score evenly,
    -log V each, whatever that value: it does not outrank a beam that chose."""
    import torch
    rng = np.random.default_rng(13)
    V, n = 5003, 9
    low = float(torch.finfo(torch_dtype(dtype)).min)
    z = rng.standard_normal((6, 3, V)) * 3
    for b, value in enumerate((low, -1e30, -1e20, -1e10, 1e30, -low)):
        z[b, 1] = value
    z[0, 2, 1:] = low                             # one token left
    z = rounded(z, dtype)
    sc = np.zeros((6, 3), dtype=np.float32)
    sc[:, 0], sc[:, 2] = -5.0, -6.0
    ld = -(-V // 8) * 8
    full = np.full((6, 3, ld), np.nan)
    full[..., :V] = z
    got = _sdv().beam_select(dev(full, torch_dtype(dtype))[..., :V], dev(sc), n)
    assert _check(z, sc, n, got) >= 3 * 6
    s, par, _ = (t.cpu().numpy() for t in got)
    assert np.abs(s[par == 1] + math.log(V)).max() < 1e-5


def test_single_beams_of_any_layout():
    """[B][1][V] logits made of padded rows and of the last position of each request."""
    import torch
    rng = np.random.default_rng(14)
    z = rounded(rng.standard_normal((5, 3, 1001)) * 3, "f32")
    x = torch.full((5, 3, 1004), float("nan"), device="cuda")
    x[..., :1001] = dev(z, torch.float32)
    sc = -rng.random((5, 1)).astype(np.float32)
    assert _check(z[:, 2:], sc, 4, _sdv().beam_select(x[:, -1:, :1001], dev(sc), 4)) == 20
    assert _check(z[:, 1:2], sc, 4, _sdv().beam_select(x[:, 1, :1001].unsqueeze(1), dev(sc), 4)) == 20


def test_ended_inactive_and_bad_beams():
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(4)
    B, W, V, n = 8, 3, 700, 6
    z = rng.standard_normal((B, W, V)).astype(np.float32).astype(np.float64)
    sc = -rng.random((B, W)).astype(np.float32)
    ended = np.zeros((B, W), dtype=np.uint8)
    ended[0, 1] = 1
    ended[1] = 1                                 # all ended: three candidates
    sc[2, 1:] = -np.inf                          # the first step: one live beam
    sc[3] = -np.inf                              # none
    z[0, 1] = np.nan                             # an ended beam's logits are not examined
    z[2, 1] = np.nan                             # nor those of one at -inf
    z[4, 2, 17] = np.nan
    z[5, 0, 699] = np.inf
    z[6, 1] = -np.inf
    sc[7, 0] = np.nan
    z[1, 0, 5:] = -np.inf
    x = z.copy()
    x[2, 0, 3:] = -np.inf                        # three tokens left
    status = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    oe = torch.full((B, n), 9, dtype=torch.uint8, device="cuda")
    got = sdv.beam_select(dev(x.astype(np.float32)), dev(sc), n, ended=dev(ended), eos_id=2, out_ended=oe, status=status)
    st = status.tolist()
    assert st[:4] == [0, 0, 0, 0] and st[4:7] == [sdv.SD_ST_NONFINITE] * 3 and st[7] == sdv.SD_ST_BAD_PARAM
    _check(np.nan_to_num(x[:4], nan=0.0, neginf=-np.inf, posinf=np.inf), sc[:4], n, [t[:4] for t in got], ended[:4], 2)
    s, par, tok = (t.cpu().numpy() for t in got)
    assert (par[4:] == -1).all() and (tok[4:] == -1).all() and (s[4:] == -np.inf).all()
    assert (tok[1, :3] == 2).all() and (par[1, 3:] == -1).all()
    want = [[int(p >= 0 and (ended[b, p] or t == 2)) for p, t in zip(par[b], tok[b])] for b in range(B)]
    assert oe.tolist() == want


def test_select_in_a_graph_and_on_a_stream():
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(5)
    x, sc = dev(rng.standard_normal((3, 4, 30000)).astype(np.float32)), dev(np.zeros((3, 4), np.float32))
    out = dict(scores=torch.zeros(3, 4, device="cuda"), parents=torch.zeros((3, 4), dtype=torch.int32, device="cuda"),
               tokens=torch.zeros((3, 4), dtype=torch.int32, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = sdv.beam_select(x, sc, 4)
    torch.cuda.synchronize()
    side = sdv.beam_select(x, sc, 4, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdv.beam_select(x, sc, 4, out=out)
    for i in range(4):
        x.add_(torch.randn_like(x))
        want = sdv.beam_select(x, sc, 4)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, out[k]) for a, k in zip(want, ("scores", "parents", "tokens")))


@pytest.mark.parametrize("layers,B,W,segs,L,E", [(1, 1, 1, 1, 1, 8), (2, 3, 4, 2, 33, 8), (3, 2, 8, 4, 100, 64),
                                                 (1, 2, 64, 1, 7, 24), (2, 1, 17, 3, 20, 16), (1, 5, 5, 1, 1000, 8)])
@pytest.mark.parametrize("in_place", [True, False])
def test_reorder_is_a_gather(layers, B, W, segs, L, E, in_place):
    import torch
    rng = np.random.default_rng(W + L)
    x = rng.integers(-30000, 30000, (layers, B, W, segs, L, E)).astype(np.int16)
    W_out = W if in_place else min(64, W + 2)
    par = rng.integers(0, W, (B, W_out)).astype(np.int32)
    par[0, 0] = -1 if W > 1 else 0
    if B > 1:
        par[1] = np.arange(W_out) % W
        par[1, -1] = W                            # no such beam
    lens = rng.integers(0, L + 1, B).astype(np.int32)
    lens[-1] = L + 9                              # clamped
    old = np.full((layers, B, W_out, segs, L, E), 77, dtype=np.int16)
    for lengths in (None, lens):
        want = x.copy() if in_place else old.copy()
        for b in range(B):
            n = L if lengths is None else min(L, int(lens[b]))
            for w in range(W_out):
                if 0 <= par[b, w] < W:
                    want[:, b, w, :, :n] = x[:, b, par[b, w], :, :n]
        src = dev(x)
        out = None if in_place else dev(old)
        got = _sdv().beam_reorder(src, dev(par), None if lengths is None else dev(lens), out=out)
        assert np.array_equal(got.cpu().numpy(), want)
        if not in_place:
            assert np.array_equal(src.cpu().numpy(), x)


def test_reorder_whatever_axes_of_one_say():
    """States with a single unit, layer, beam or segment whose strides come from
    other shapes."""
    import torch
    rng = np.random.default_rng(10)
    x = rng.integers(-9, 9, (2, 3, 4, 1, 5, 8)).astype(np.int16)
    par = rng.integers(0, 4, (3, 4)).astype(np.int32)
    for view in (lambda t: t.transpose(3, 4), lambda t: t.as_strided(t.shape, (480, 160, 40, 7, 8, 1)),
                 lambda t: t[:1].as_strided((1, *t.shape[1:]), (3, 160, 40, 40, 8, 1)),
                 lambda t: t[:, :, :, :, :1].as_strided((2, 3, 4, 1, 1, 8), (480, 160, 40, 40, 5, 1))):
        t = dev(x)
        want = t.clone()
        w = view(want)
        w.copy_(w.clone()[:, torch.arange(3, device="cuda")[:, None], dev(par).long()])
        _sdv().beam_reorder(view(t), dev(par))
        assert torch.equal(t, want)
    with pytest.raises(ValueError):
        _sdv().beam_reorder(dev(x).transpose(4, 5), dev(par))


def test_reorder_of_a_broadcast_state():
    """One prompt's state for all requests and beams, spread into their own."""
    rng = np.random.default_rng(15)
    x = rng.integers(-9, 9, (2, 1, 1, 2, 10, 8)).astype(np.int16)
    par = np.zeros((3, 4), dtype=np.int32)
    old = dev(np.full((2, 3, 4, 2, 10, 8), 5, dtype=np.int16))
    got = _sdv().beam_reorder(dev(x).expand(2, 3, 2, 2, 10, 8), dev(par), dev(np.array([10, 3, 0], np.int32)), out=old)
    want = np.full((2, 3, 4, 2, 10, 8), 5, dtype=np.int16)
    want[:, 0], want[:, 1, :, :, :3] = x[:, 0], x[:, 0, :, :, :3]
    assert np.array_equal(got.cpu().numpy(), want)


def test_reorder_of_strided_states():
    """Beams that are not the outermost rows: [B][W][layers][segs] in memory."""
    import torch
    rng = np.random.default_rng(9)
    x = rng.integers(-9, 9, (2, 3, 4, 2, 10, 8)).astype(np.int16)
    par = rng.integers(0, 3, (2, 3)).astype(np.int32)
    t = dev(x)
    state = t.permute(2, 0, 1, 3, 4, 5)
    _sdv().beam_reorder(state, dev(par))
    assert np.array_equal(t.cpu().numpy(), x[np.arange(2)[:, None], par])
