"""sd_tree_verify_sample on the GPU against the fp64 oracle."""
import ctypes

import numpy as np
import pytest

import oracle
from treetools import dev

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _padded(x):
    """Rows of any length in a tensor whose rows are 16-byte aligned, NaN behind them."""
    import torch
    return torch.nn.functional.pad(dev(x), (0, 4 + -x.shape[1] % 4), value=float("nan"))[:, :x.shape[1]]


class Trees:
    """Random trees whose children were drawn from draft rows that agree with the
    target's to some degree; NaN wherever nothing may be read."""

    def __init__(self, seed, nodes, V, drafts="again", Vd=None, peak=3.0, reach=5, behind=0):
        rng = np.random.default_rng(seed)
        self.nodes, self.V = nodes, V
        self.off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        N = self.N = int(self.off[-1])
        z = rng.standard_normal((N, V)) * peak
        self.p = _softmax(z)
        Vd = self.Vd = Vd or V
        q = _softmax((z * 0.9 + 0.5 * peak * rng.standard_normal((N, V)))[:, :Vd])
        self.parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, n)]
                                       for n in nodes]).astype(np.int32)
        self.tokens = rng.integers(0, V, N).astype(np.int32)
        for b, n in enumerate(nodes):
            lo = self.off[b]
            for c in range(n):
                kids = [i for i in range(c + 1, n) if self.parents[lo + i] == c]
                row = q[lo + c].astype(np.float64)
                if drafts == "beam":
                    best = np.argsort(-(z[lo + c] + rng.standard_normal(V)))
                    self.tokens[[lo + i for i in kids]] = best[np.arange(len(kids)) % V]
                    continue
                k = min(len(kids), Vd) if drafts == "once" else len(kids)
                drawn = rng.choice(Vd, k, replace=drafts == "again", p=row / row.sum())
                for i, t in zip(kids, drawn):
                    self.tokens[lo + i] = t
        self.q = None if drafts == "beam" else q
        self.u, self.v = rng.random(N).astype(np.float32), rng.random(len(nodes)).astype(np.float32)
        self.no_replacement = drafts == "once"

    def device(self):
        p, q = _padded(self.p), None if self.q is None else _padded(self.q)
        if q is not None:      # rows of nodes without children are not read
            has = np.zeros(self.N, dtype=bool)
            for b, n in enumerate(self.nodes):
                lo = self.off[b]
                has[[lo + c for c in self.parents[lo:lo + n] if c >= 0]] = True
            q[dev(~has)] = float("nan")
        return dict(target_probs=p, tokens=dev(self.tokens), parents=dev(self.parents), node_offsets=dev(self.off),
                    max_nodes=max(self.nodes), accept_uniforms=dev(self.u), draw_uniforms=dev(self.v), draft_probs=q)

    def check(self, flags=0, status=None):
        sdv = _sdv()
        got = sdv.tree_verify_sample(**self.device(), flags=flags | (sdv.SD_NO_REPLACEMENT if self.no_replacement else 0),
                                     status=status)
        want = oracle.tree_sample_ref(self.p, self.q, self.tokens, self.parents, self.off, max(self.nodes), self.u, self.v,
                                      no_bonus=bool(flags & 1), no_replacement=self.no_replacement)
        # sums of V products in 64 bits: decisions nearer than this could go either way
        sure = want[3] > self.V * 2.0 ** -50
        assert sure.mean() > 0.9
        for g, w, name in zip(got, want, ("accepted", "path", "tokens")):
            assert np.array_equal(g.cpu().numpy()[sure], w[sure]), name
        return want


@pytest.mark.parametrize("drafts", ["again", "once", "beam"])
@pytest.mark.parametrize("nodes,V,Vd", [
    ([1], 1, 0), ([2, 1, 5], 2, 0), ([3, 1, 64], 7, 5), ([5, 9, 2], 1000, 0), ([64] * 20, 333, 0), ([16, 33], 20011, 19999),
    ([2, 7], 152064, 151936), ([8] * 300, 2050, 0), ([1, 4] * 40, 9001, 8000), ([6] * 700, 64, 0), ([20], 151936, 0),
    ([4] * 1100, 515, 514)])
def test_walks_match_the_oracle(nodes, V, Vd, drafts):
    t = Trees(len(nodes) + V, nodes, V, drafts, Vd or None)
    for flags in (0, 1):
        print(f"sample {len(nodes)} x {nodes[0]} V {V} {drafts} flags {flags}", flush=True)
        t.check(flags)


@pytest.mark.parametrize("drafts", ["again", "once", "beam"])
def test_wide_and_deep_trees(drafts):
    """A star of 63 children rejected one after another, and a chain that is kept."""
    for reach, peak in ((64, 0.3), (1, 3.0)):
        t = Trees(5, [64] * 6, 700, drafts, peak=peak, reach=reach)
        if reach == 64:
            t.parents[:] = 0
            t.parents[t.off[:-1]] = -1
            t.u[:] = np.float32(1 - 2.0 ** -24)
            rng = np.random.default_rng(6)
            if drafts == "once":
                for b in range(6):
                    t.tokens[t.off[b] + 1:t.off[b + 1]] = rng.choice(700, 63, replace=False)
        else:
            t.u[:] = 0.0
        acc = t.check()[0]
        assert reach == 64 or acc.max() == 63


@pytest.mark.parametrize("drafts", ["again", "once", "beam"])
def test_first_tokens_keep_the_targets_law(drafts):
    """Histogram of the first token emitted over many requests against p: chi-square
    with V - 1 degrees of freedom, below its mean by 6 standard deviations or less."""
    rng = np.random.default_rng(7)
    V, B, T = 12, 60000, 4
    z = rng.standard_normal(V)
    p, q = _softmax(z), _softmax(0.5 * z + rng.standard_normal(V))
    off = (np.arange(B + 1) * T).astype(np.int32)
    parents = np.tile([-1, 0, 0, 0], B).astype(np.int32)
    tokens = np.zeros((B, T), dtype=np.int32)
    qd = q.astype(np.float64) / q.astype(np.float64).sum()
    if drafts == "again":
        tokens[:, 1:] = rng.choice(V, (B, 3), p=qd)
    elif drafts == "once":
        tokens[:, 1:] = np.argsort(-(np.log(qd) + rng.gumbel(size=(B, V))), axis=1)[:, :3]
    else:
        tokens[:, 1:] = np.argsort(-q)[:3]
    sdv = _sdv()
    rows = dev(np.tile(p, (B * T, 1)))
    acc, _, tok = sdv.tree_verify_sample(
        rows, dev(tokens.reshape(-1)), dev(parents), dev(off), T, dev(rng.random(B * T).astype(np.float32)),
        dev(rng.random(B).astype(np.float32)), draft_probs=None if drafts == "beam" else dev(np.tile(q, (B * T, 1))),
        flags=sdv.SD_NO_REPLACEMENT if drafts == "once" else 0)
    # accepted: with given children the sum of their p; else at least the first child's
    # share, the sum of min(p, q), both within 6 standard deviations
    share = float(p[tokens[0, 1:]].sum()) if drafts == "beam" else float(np.minimum(p, q).sum())
    got, off_by = acc.double().mean().item(), 6 * np.sqrt(share * (1 - share) / B)
    assert got > share - off_by and (drafts != "beam" or got < share + off_by), (got, share)
    count = np.bincount(tok[:, 0].cpu().numpy(), minlength=V)
    want = B * p.astype(np.float64) / p.astype(np.float64).sum()
    chi = ((count - want) ** 2 / want).sum()
    assert chi < (V - 1) + 6 * np.sqrt(2 * (V - 1)), chi


def test_borders_of_the_random_numbers():
    """u = 0 accepts whatever has weight; v = 0 draws the first token with weight, the
    largest v below 1 the last one."""
    sdv = _sdv()
    V, T = 1003, 3
    rng = np.random.default_rng(8)
    p = np.zeros((4 * T, V), dtype=np.float32)
    for r in p:
        at = np.sort(rng.choice(np.arange(5, V - 5), 6, replace=False))
        r[at] = np.array([0.25, 0.125, 0.125, 0.25, 0.125, 0.125])
    tok = np.array([0, 1, 2] * 4, dtype=np.int32)                    # children with p = 0: never accepted
    tok[4] = np.flatnonzero(p[3])[3]                                 # request 1: a child with weight
    parents = np.tile([-1, 0, 0], 4).astype(np.int32)
    off = (np.arange(5) * T).astype(np.int32)
    last = np.float32(1 - 2.0 ** -24)
    v = np.array([0, 0, last, last], dtype=np.float32)
    acc, path, out = sdv.tree_verify_sample(_padded(p), dev(tok), dev(parents), dev(off), T, dev(np.zeros(12, dtype=np.float32)),
                                            dev(v))
    assert acc.tolist() == [0, 1, 0, 0]
    first = lambda r: int(np.flatnonzero(p[r])[0])      # noqa: E731
    end = lambda r: int(np.flatnonzero(p[r])[-1])       # noqa: E731
    assert out[:, 0].tolist() == [first(0), int(tok[4]), end(6), end(9)]
    assert out[1].tolist() == [int(tok[4]), first(4), -1] and path[1].tolist() == [0, 1, -1]
    # a rejected token is not drawn, though it holds nearly all of p and v = 0 points at it
    p[:] = 0
    p[:, 5], p[:, 900] = np.float32(1 - 2.0 ** -24), np.float32(2.0 ** -24)
    tok[:] = 5
    u = np.full(12, last, dtype=np.float32)
    p[0:3, 5] = 0.5
    p[0:3, 900] = 0.5
    acc, _, out = sdv.tree_verify_sample(_padded(p), dev(tok), dev(parents), dev(off), T, dev(u), dev(v))
    assert acc.tolist() == [0, 0, 0, 0] and out[:, 0].tolist() == [900] * 4


def test_equal_rows_leave_nothing_to_draw_from():
    """p = q: a test cannot fail but by rounding; here u q Z < p is false since p and
    q are 0 at the token, and the residual is 0: reported, and the draw is from p."""
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(9)
    for B in (1, 600):
        V = 501
        p = np.tile(_softmax(rng.standard_normal((1, V)) * 2), (2 * B, 1))
        p[:, 7] = 0
        off = (np.arange(B + 1) * 2).astype(np.int32)
        tok = np.tile([0, 7], B).astype(np.int32)
        parents = np.tile([-1, 0], B).astype(np.int32)
        v = rng.random(B).astype(np.float32)
        st = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        acc, _, out = sdv.tree_verify_sample(_padded(p), dev(tok), dev(parents), dev(off), 2, dev(np.full(2 * B, 0.5, np.float32)),
                                             dev(v), draft_probs=_padded(p), status=st)
        assert (st == sdv.SD_ST_RESID_ZERO | sdv.SD_ST_Q_ZERO).all() and (acc == 0).all()
        C = np.cumsum(p[0].astype(np.float64))
        want = np.searchsorted(C, v.astype(np.float64) * C[-1], side="right")
        assert np.array_equal(out[:, 0].cpu().numpy(), want)


@pytest.mark.parametrize("copies", [1, 80])
def test_defects_are_reported_request_by_request(copies):
    import torch
    sdv = _sdv()
    rng = np.random.default_rng(10)
    V, T, R = 600, 4, 12
    p, q = _softmax(rng.standard_normal((R * T, V))), _softmax(rng.standard_normal((R * T, V)))
    parents = np.tile([-1, 0, 1, 2], R).astype(np.int32)
    tokens = rng.integers(0, V, R * T).astype(np.int32)
    u, v = np.full(R * T, 0.5, dtype=np.float32), np.full(R, 0.5, dtype=np.float32)
    q[np.arange(1, R * T) - 1, tokens[1:]] = 0.9     # first children are rejected
    p[np.arange(1, R * T) - 1, tokens[1:]] = 1e-6
    tokens[0] = -7                                   # a root's token is not used
    p[1 * T, 5] = np.nan                             # the root's row: summed up
    q[2 * T, 5] = -0.5
    p[3 * T + 3, 5] = np.nan                         # a row that the walk does not reach
    tokens[4 * T + 2] = V
    tokens[5 * T + 1] = -1
    parents[6 * T + 2] = 2                           # its own parent
    u[7 * T + 1] = 1.0
    v[8] = np.nan
    u[9 * T + 2] = -3.0                              # not used: the child before it is rejected
    p[10 * T, tokens[10 * T + 1]] = np.inf           # the tested token's own
    q[11 * T, tokens[11 * T + 1]] = 0.0              # accepted, since p > 0: its children are tested
    u[11 * T + 2] = 2.0
    tile = lambda x: np.tile(x, (copies,) + (1,) * (x.ndim - 1))  # noqa: E731
    off = (np.arange(R * copies + 1) * T).astype(np.int32)
    st = torch.full((R * copies,), -1, dtype=torch.int32, device="cuda")
    acc, path, tok = sdv.tree_verify_sample(dev(tile(p)), dev(tile(tokens)), dev(tile(parents)), dev(off), T, dev(tile(u)),
                                            dev(tile(v)), draft_probs=dev(tile(q)), status=st)
    NF, ID, BP = sdv.SD_ST_NONFINITE, sdv.SD_ST_BAD_DRAFT_ID, sdv.SD_ST_BAD_PARAM
    want = [0, NF, NF, 0, ID, ID, sdv.SD_ST_BAD_TREE, BP, BP, 0, NF, BP | sdv.SD_ST_Q_ZERO]
    assert st.tolist() == want * copies
    bad = np.array([bool(s & sdv.SD_ST_TREE_INVALID_MASK) for s in want] * copies)
    assert (acc.cpu().numpy() == np.where(bad, -1, 0)).all()
    assert (path.cpu().numpy()[bad] == -1).all() and (tok.cpu().numpy()[bad] == -1).all()
    assert (tok.cpu().numpy()[~bad, 0] >= 0).all()


def test_a_walk_that_is_given_up_is_reported():
    """The bounded waits forced to run out at once: requests that need a pass are -1
    with a status of their own, the others stand, and the next call is whole."""
    import torch
    import speculative_sampling_verify_temp_amd.serve as serve
    sdv = _sdv()
    t = Trees(11, [5] * 50 + [1], 20011, "once")
    t.u[t.off[3]:t.off[4]] = 0.0                      # request 3 accepts down to a leaf
    d = t.device()
    B, T = 51, 5
    p, q = d["target_probs"], d["draft_probs"]
    a = serve._TREE_SAMPLE.pack(p.data_ptr(), q.data_ptr(), p.stride(0), q.stride(0), d["tokens"].data_ptr(),
                                d["parents"].data_ptr(), d["node_offsets"].data_ptr(), d["accept_uniforms"].data_ptr(),
                                d["draw_uniforms"].data_ptr(), B, t.N, 20011, 20011, T, 5)
    n = serve._tree_sample_bytes(a)
    ws = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")
    out = dict(accepted=torch.full((B,), 7, dtype=torch.int32, device="cuda"),
               path=torch.full((B, T), 7, dtype=torch.int32, device="cuda"),
               tokens=torch.full((B, T), 7, dtype=torch.int32, device="cuda"))
    st = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    P = ctypes.c_void_p
    rc = sdv.lib.sd_debug_tree_sample_polls(ctypes.c_char_p(a), P(ws.data_ptr()), ctypes.c_size_t(n),
                                            P(out["accepted"].data_ptr()), P(out["path"].data_ptr()),
                                            P(out["tokens"].data_ptr()), P(st.data_ptr()), ctypes.c_int32(0),
                                            P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    s = st.cpu().numpy()
    # requests whose walk needs no pass end in any case; another one stands where each of
    # its workgroups found the others' sums at its first look
    acc, path, tok, _ = oracle.tree_sample_ref(t.p, t.q, t.tokens, t.parents, t.off, T, t.u, t.v, True, True)
    passes = np.zeros(B, dtype=int)
    for b in range(B):
        lo, n = t.off[b], t.off[b + 1] - t.off[b]
        for i in range(acc[b] + 1):
            kids = [c for c in range(n) if t.parents[lo + c] == path[b, i]]
            passes[b] += kids.index(path[b, i + 1]) if i < acc[b] else len(kids)
    assert passes[3] == passes[50] == 0 and (passes > 1).any()
    lost = (s & sdv.SD_ST_UNFINISHED) != 0
    assert lost.any() and not lost[passes == 0].any()
    for o, r in ((out["accepted"], acc), (out["path"], path), (out["tokens"], tok)):
        o = o.cpu().numpy()
        assert (o[lost] == -1).all() and np.array_equal(o[~lost], r[~lost])
    d = {**d, "flags": 5}
    got = sdv.tree_verify_sample(**d, out=out, status=st, workspace=ws)
    ref = sdv.tree_verify_sample(**d)
    assert all(torch.equal(r, g) for r, g in zip(ref, got)) and (got[0] >= 0).all()


def test_many_calls_at_once():
    """Calls on streams and workspaces of their own, more than the chip holds teams of:
    slices whose workgroups do not come are taken over, and results stay the same."""
    import torch
    sdv = _sdv()
    d = Trees(13, [9] * 32, 20011, "again").device()
    ref = sdv.tree_verify_sample(**d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    got = [None] * len(streams)
    for r in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = sdv.tree_verify_sample(**d)
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(x, y) for x, y in zip(ref, g))


def test_in_a_graph_and_on_a_stream():
    import torch
    sdv = _sdv()
    for drafts, nodes in (("again", [6] * 3), ("beam", [6] * 100), ("once", [9] * 700)):
        t = Trees(12, nodes, 3001 if len(nodes) < 200 else 400, drafts)
        d = t.device()
        B, T = len(nodes), nodes[0]
        out = {n: torch.zeros(s, dtype=torch.int32, device="cuda")
               for n, s in (("accepted", (B,)), ("path", (B, T)), ("tokens", (B, T)))}
        sdv.tree_verify_sample(**d, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sdv.tree_verify_sample(**d, out=out)
        s = torch.cuda.Stream()
        for _ in range(4):
            d["accept_uniforms"].copy_(torch.rand_like(d["accept_uniforms"]))
            d["draw_uniforms"].copy_(torch.rand_like(d["draw_uniforms"]))
            s.wait_stream(torch.cuda.current_stream())
            want = sdv.tree_verify_sample(**d, stream=s)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(w, out[n]) for w, n in zip(want, ("accepted", "path", "tokens")))


def test_rows_past_2_to_the_32_elements():
    import torch
    t = Trees(14, [5, 1], 1500, "again")
    d = t.device()
    ref = _sdv().tree_verify_sample(**d)
    ld = (1 << 30) + 4      # row 4 begins past 2^32 elements, row 1 past 2^32 bytes
    buf = torch.empty(5 * ld + 4096, dtype=torch.float32, device="cuda")
    for name, at in (("target_probs", 0), ("draft_probs", 2048)):
        x = buf.as_strided((t.N, 1500), (ld, 1), at)
        x.copy_(d[name])
        d[name] = x
    for flags in (0, 1):
        got = _sdv().tree_verify_sample(**d, flags=flags)
        want = _sdv().tree_verify_sample(**{**d, "target_probs": _padded(t.p), "draft_probs": t.device()["draft_probs"]}, flags=flags)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert all(torch.equal(g, w) for g, w in zip(_sdv().tree_verify_sample(**d), ref))


@pytest.mark.parametrize("V", [1003, 20011])
def test_a_beams_row_whose_whole_support_was_drafted(V):
    """Without draft rows Z is 1 less the rejected p, and a row's fp32 numbers sum to 1
    only within rounding: the last of its tokens can be rejected too, and nothing is left
    to draw from.  Reported, and the draw is from p."""
    import torch
    sdv = _sdv()
    B, T = 40, 4
    last = np.float32(1 - 2.0 ** -24)
    p = np.zeros((B * T, V), dtype=np.float32)
    a, b = 3, V - 2
    p[:, a], p[:, b] = 0.5, np.float32(0.5 - 2.0 ** -25)
    parents = np.tile([-1, 0, 0, 0], B).astype(np.int32)
    tokens = np.tile([0, a, b, a], B).astype(np.int32)      # (one of them twice)
    u = np.full(B * T, last, dtype=np.float32)
    for r in range(0, B, 4):       # the same below the root's first child
        parents[r * T + 2], parents[r * T + 3] = 1, 1
        u[r * T + 1] = 0.0
        tokens[r * T + 2:r * T + 4] = a, b
    rows = p.copy()                # the oracle's
    p[7 * T] = 0                   # nothing to draw from even so
    off = (np.arange(B + 1) * T).astype(np.int32)
    v = np.random.default_rng(15).random(B).astype(np.float32)
    st = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    for B2 in (B, 2):
        n = B2 * T
        acc, path, tok = sdv.tree_verify_sample(_padded(p[:n]), dev(tokens[:n]), dev(parents[:n]), dev(off[:B2 + 1]), T,
                                                dev(u[:n]), dev(v[:B2]), status=st[:B2])
        want = oracle.tree_sample_ref(rows[:n], None, tokens[:n], parents[:n], off[:B2 + 1], T, u[:n], v[:B2])
        ok = np.arange(B2) != 7
        for g, w in zip((acc, path, tok), want):
            assert np.array_equal(g.cpu().numpy()[ok], w[ok])
            assert (g.cpu().numpy()[~ok] == -1).all()
        assert (st[:B2].cpu().numpy()[ok] == sdv.SD_ST_RESID_ZERO).all()
        assert all(s & sdv.SD_ST_NONFINITE for s in st[:B2].cpu().numpy()[~ok])
        deep = np.arange(B2) % 4 == 0
        assert (want[0] == deep)[ok].all() and set(want[2][np.arange(B2), want[0]][ok]) <= {a, b}


@pytest.mark.parametrize("drafts", ["again", "once", "beam"])
@pytest.mark.parametrize("nodes,V", [([20], 151936), ([9] * 7, 20011), ([6] * 100, 9001), ([33] * 16, 60000)])
def test_slices_that_are_taken_over(nodes, V, drafts):
    """Half of a team's workgroups are not there: their slices are taken over, so that
    workgroups hold several, lose some to each other and make sums again for the draw.
    Without that, requests would be unfinished; the results are the oracle's."""
    import torch
    import speculative_sampling_verify_temp_amd.serve as serve
    sdv = _sdv()
    t = Trees(16, nodes, V, drafts, peak=1.5)
    t.u[:] = 1 - (1 - t.u) * np.float32(0.25)         # many rejections
    d = t.device()
    B, T = len(nodes), max(nodes)
    p, q = d["target_probs"], d["draft_probs"]
    ld = p.stride(0) if t.N > 1 else (V + 3) // 4 * 4
    a = serve._TREE_SAMPLE.pack(p.data_ptr(), 0 if q is None else q.data_ptr(), ld, ld, d["tokens"].data_ptr(),
                                d["parents"].data_ptr(), d["node_offsets"].data_ptr(), d["accept_uniforms"].data_ptr(),
                                d["draw_uniforms"].data_ptr(), B, t.N, V, V, T, sdv.SD_NO_REPLACEMENT if drafts == "once" else 0)
    n = serve._tree_sample_bytes(a)
    want = oracle.tree_sample_ref(t.p, t.q, t.tokens, t.parents, t.off, T, t.u, t.v, no_replacement=drafts == "once")
    sure = want[3] > V * 2.0 ** -50
    assert sure.mean() > 0.9
    usual = sdv.tree_verify_sample(**d, flags=sdv.SD_NO_REPLACEMENT if drafts == "once" else 0)
    P = ctypes.c_void_p
    for _ in range(3):
        ws = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")
        out = [torch.full(s, 7, dtype=torch.int32, device="cuda") for s in ((B,), (B, T), (B, T), (B,))]
        rc = sdv.lib.sd_debug_tree_sample_polls(ctypes.c_char_p(a), P(ws.data_ptr()), ctypes.c_size_t(n),
                                                *(P(o.data_ptr()) for o in out), ctypes.c_int32(-1),
                                                P(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        torch.cuda.synchronize()
        assert not (out[3] & sdv.SD_ST_TREE_INVALID_MASK).any()
        for o, w, x in zip(out, want, usual):
            assert np.array_equal(o.cpu().numpy()[sure], w[sure]) and torch.equal(o, x)
        # a slice's claims are counted: one for each pass, whoever made it
        claims = ws.cpu().numpy().view(np.uint32).reshape(B, -1)[:, 256:320]
        slices = int((claims[0] > 0).sum())
        assert slices > 1 and (claims[:, :slices] == claims[:, :1]).all() and not claims[:, slices:].any()
