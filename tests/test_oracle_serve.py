"""The oracle of include/sd_serve.h against closed forms, identities and brute force
(CPU only)."""
import itertools
import math

import numpy as np
import pytest

import oracle


def test_norm_and_rotation_identities():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    freq = (100.0 ** (-np.arange(4) / 4.0)).astype(np.float32)
    pos = np.array([0, 1, 7, 100, -3])
    for pairs in (False, True):
        y = oracle.norm_rope_ref(x, None, pos, freq, 0.0, pairs)
        assert np.allclose(y[0], x[0])                             # position 0 turns nothing
        assert np.array_equal(y[..., 8:], x[..., 8:])              # nor what lies past rot
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        # q . k depends on the distance of the positions alone
        q, k = rng.standard_normal((2, 1, 1, 16))
        f = lambda v, p: oracle.norm_rope_ref(v, None, [p], freq, 0.0, pairs)[0, 0]  # noqa: E731
        assert np.isclose(f(q, 9) @ f(k, 4), f(q, 105) @ f(k, 100))
        # one pair of a known angle
        e = np.zeros((1, 1, 16))
        e[0, 0, 0] = 1
        b = 1 if pairs else 4
        g = f(e[0:1], 2)
        assert np.isclose(g[0], math.cos(2.0)) and np.isclose(g[b], math.sin(2.0))
    n = oracle.norm_rope_ref(x, np.full(16, 2.0), pos, freq, 0.0)
    assert np.allclose((n * n).mean(-1), 4.0)


def test_rotation_of_far_positions():
    """Sines and cosines of products that fp64 rounds, against 64-bit mantissas, which hold
    positions of 31 bits times fp32 frequencies exactly; 2 pi in them is off by 2^-63, so
    2^29 turns by 2^-34."""
    assert np.finfo(np.longdouble).nmant >= 63
    two_pi = 8 * np.arctan(np.longdouble(1))
    rng = np.random.default_rng(3)
    pos = np.concatenate([rng.integers(2 ** 30, 2 ** 31, 40), [2 ** 31 - 1, -2 ** 31]])
    freq = rng.uniform(0.5, 1.0, 8).astype(np.float32)
    x = np.zeros((len(pos), 1, 16))
    x[..., :8] = 1
    y = oracle.norm_rope_ref(x, None, pos, freq, 0.0)[:, 0]
    t = pos[:, None].astype(np.longdouble) * freq.astype(np.longdouble)
    t = t - np.rint(t / two_pi) * two_pi
    assert (np.abs(y[:, :8] - np.cos(t)) < 2.0 ** -32).all() and (np.abs(y[:, 8:] - np.sin(t)) < 2.0 ** -32).all()


def test_e4m3_values_against_the_whole_format():
    """Nearest of all 253 finite values, ties to the even code, by brute force."""
    import torch
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    assert len(vals) == 253 and vals[-1] == 448
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(3000) * 10.0 ** rng.integers(-4, 3, 3000), (vals[1:] + vals[:-1]) / 2, vals])
    x = np.clip(x, -448, 448)
    got = oracle.e4m3_round(x)
    assert np.isin(got, vals).all()
    assert (np.abs(got - x) <= np.abs(vals[:, None] - x).min(0) + 0).all()
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    exact32 = x == x.astype(np.float32)      # (others are rounded to fp32 first)
    assert np.array_equal(got[exact32], want[exact32])


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_append_is_its_definition(code):
    rng = np.random.default_rng(2)
    page, block, H, D, m, ctx = 32, 16, 2, 8, 41, 21
    codes, scales = np.zeros((4, H, page, D)), np.zeros((4, H, 2), dtype=np.float32)
    table = [2, 0, 3, 1]
    first = rng.standard_normal((ctx, H, D)).astype(np.float32)
    oracle.quant_append_ref(first, codes, scales, table, 0, block, code)
    new = (rng.standard_normal((m, H, D)) * 3).astype(np.float32)
    oracle.quant_append_ref(new, codes, scales, table, ctx, block, code)
    top = oracle.serve.TOP[code]
    x = np.concatenate([first, new]).astype(np.float64)
    for t in range(ctx + m):
        s = scales[table[t // page], :, t % page // block].astype(np.float64)[:, None]
        c = codes[table[t // page], :, t % page]
        assert np.abs(c).max() <= top
        # half a step, twice where the block was rounded again
        step = s if code == "i8" else np.maximum(np.abs(x[t]) / 8, s * 2.0 ** -9)
        assert (np.abs(c * s - x[t]) <= (1.0 if 16 <= t < ctx else 0.5) * step * (1 + 1e-5)).all()
    for b in range(0, ctx + m, block):
        amax = np.abs(x[b:min(b + block, ctx + m)]).max((0, 2))
        assert np.allclose(scales[table[b // page], :, b % page // block], amax / top, rtol=1e-6)


def _tiny(seed, T=4, lens=(9, 0)):
    rng = np.random.default_rng(seed)
    H, G, D, page, block = 2, 2, 8, 16, 16
    k, v = rng.integers(-127, 128, (2, 6, H, page, D)).astype(np.float64)
    ks, vs = rng.random((2, 6, H, 1)).astype(np.float32) * 0.01 + 0.001
    table = np.array([[1, 4], [5, 0]])
    N = T * len(lens)
    q = rng.standard_normal((N, H * G, D))
    kn, vn = rng.standard_normal((2, N, H, D))
    return q, kn, vn, k, v, ks, vs, table, list(lens), np.arange(len(lens) + 1) * T, block, 0.4


def test_attention_is_the_16_bit_one_of_its_values():
    a = _tiny(3)
    q, kn, vn, k, v, ks, vs, table, lens, off, block, scale = a
    parents = np.array([-1, 0, 0, 2] * 2)
    kk, vv = k * ks[..., None], v * vs[..., None]
    want = oracle.tree_attention_ref(q, kn, vn, kk, vv, table, lens, off, scale, parents)
    got = oracle.quant_attention_ref(*a, parents=parents)
    for g, w in zip(got, want):
        assert np.allclose(g, w)


def test_windows():
    a = _tiny(4)
    q, kn, vn, k, v, ks, vs, table, lens, off, block, scale = a
    whole = oracle.quant_attention_ref(*a)
    for g, w in zip(oracle.quant_attention_ref(*a, window=13), whole):      # as wide as all positions
        assert np.allclose(g, w)
    for g, w in zip(oracle.quant_attention_ref(*a, window=1, sinks=50), whole):      # all are sinks
        assert np.allclose(g, w)
    o, lse, _ = oracle.quant_attention_ref(*a, window=1)                   # itself alone
    for i in range(8):
        for g in range(4):
            assert np.allclose(o[i, g], vn[i, g // 2])
            assert np.isclose(lse[i, g], scale * q[i, g] @ kn[i, g // 2])
    # a row by hand: position 11 of request 0, window 5, 2 sinks: slots 0, 1, 7, 8 and nodes 0 .. 2
    o, lse, _ = oracle.quant_attention_ref(*a, window=5, sinks=2)
    keys = np.concatenate([k[1, 0, [0, 1, 7, 8]] * ks[1, 0], kn[:3, 0]])
    vals = np.concatenate([v[1, 0, [0, 1, 7, 8]] * vs[1, 0], vn[:3, 0]])
    x = scale * keys @ q[2, 0]
    p = np.exp(x - x.max())
    assert np.allclose(o[2, 0], p @ vals / p.sum()) and np.isclose(lse[2, 0], np.log(np.exp(x).sum()))


def _law(p, q, children, no_replacement):
    """Law of the first emitted token for given children tokens, by the textbook:
    each test against the normalised residual."""
    law = np.zeros(len(p))
    left, alive, dq = p.copy(), 1.0, q.copy()
    for x in children:
        acc = min(1.0, left[x] / dq[x]) if dq[x] > 0 else float(left[x] > 0)
        law[x] += alive * acc
        alive *= 1 - acc
        left = np.maximum(left - dq, 0)
        if left.sum() == 0:
            return law
        left /= left.sum()
        if no_replacement:
            dq = dq.copy()
            dq[x] = 0
            dq = dq / dq.sum() if dq.sum() > 0 else dq
    return law + alive * left


@pytest.mark.parametrize("no_replacement", [False, True])
def test_sampled_walks_follow_the_textbook_and_keep_the_law(no_replacement):
    """Over a grid of random numbers the oracle's first token has the textbook's law
    given the children; over the children's own law, the target's."""
    rng = np.random.default_rng(5)
    V = 4
    p, q = rng.dirichlet(np.ones(V), 2)
    total = np.zeros(V)
    grid = (np.arange(40) + 0.5) / 40
    for kids in itertools.product(range(V), repeat=2):
        if no_replacement:
            if kids[0] == kids[1]:
                continue
            weight = q[kids[0]] * q[kids[1]] / (1 - q[kids[0]])
        else:
            weight = q[kids[0]] * q[kids[1]]
        law = _law(p, q, kids, no_replacement)
        total += weight * law
        n = len(grid)
        u1, u2 = (g.ravel() for g in np.meshgrid(grid, grid, indexing="ij"))
        count = np.zeros(V)
        for v in grid[::4]:
            B = n * n
            u = np.stack([np.zeros(B), u1, u2], 1).reshape(-1)
            tok = np.tile([0, *kids], B)
            _, _, out, _ = oracle.tree_sample_ref(np.tile(p, (3 * B, 1)), np.tile(q, (3 * B, 1)), tok,
                                                  np.tile([-1, 0, 0], B), np.arange(B + 1) * 3, 3, u, np.full(B, v),
                                                  no_replacement=no_replacement)
            count += np.bincount(out[:, 0], minlength=V)
        assert np.abs(count / count.sum() - law).max() < 0.15      # a grid of 10 draws: steps of 0.1
    assert np.allclose(total, p, atol=1e-12)


def test_given_children_keep_the_law():
    """Point masses: accepted with p, in order, the rest of p drawn from."""
    p = np.array([[0.5, 0.2, 0.1, 0.2]] * 3)
    tok, up, off = np.array([0, 0, 2]), np.array([-1, 0, 0]), np.array([0, 3])
    call = lambda u1, u2, v: oracle.tree_sample_ref(p, None, tok, up, off, 3, np.array([0, u1, u2]), np.array([v]))  # noqa: E731
    assert call(0.49, 0, 0)[2][0].tolist() == [0, 0, -1] and call(0.49, 0, 0)[0][0] == 1
    assert call(0.51, 0.19, 0.0)[2][0, 0] == 2          # 0.19 * 0.5 < 0.1
    assert call(0.51, 0.21, 0.0)[2][0, 0] == 1          # what is left: 0.2 and 0.2
    assert call(0.51, 0.21, 0.51)[2][0, 0] == 3
    acc, path, out, _ = oracle.tree_sample_ref(p, None, tok, up, off, 3, np.array([0, 0.1, 0]), np.array([0.6]), no_bonus=True)
    assert acc[0] == 1 and path[0].tolist() == [0, 1, -1] and out[0].tolist() == [0, -1, -1]


def test_given_children_that_are_all_of_p():
    """The last of them can be rejected where p sums up to less than 1: the draw is from p."""
    p = np.array([[0.5, 0.0, 0.5 - 2.0 ** -25]] * 3)
    tok, up, off = np.array([0, 0, 2]), np.array([-1, 0, 0]), np.array([0, 3])
    u = np.array([0, 1 - 2.0 ** -24, 1 - 2.0 ** -24])
    for v, want in ((0.0, 0), (0.4, 0), (0.6, 2), (1 - 2.0 ** -24, 2)):
        acc, path, out, _ = oracle.tree_sample_ref(p, None, tok, up, off, 3, u, np.array([v]))
        assert acc[0] == 0 and path[0].tolist() == [0, -1, -1] and out[0].tolist() == [want, -1, -1]
