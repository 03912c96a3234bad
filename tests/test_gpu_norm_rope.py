"""sd_qk_norm_rope on the GPU against the fp64 oracle."""
import numpy as np
import pytest

import oracle
from treetools import EPS, dev, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


def _freq(rot, base=1e6):
    return (base ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


def _check(got, x, w, pos, freq, eps, pairs, dtype):
    """Half a step for the result; the norm's sum of D squares, its root, quotient
    and two products, (D / 2 + 8) 2^-24 of the element; the angle, off by 2^-26 turns
    from its rounding to fp32, a sine's 2 units in the last place and three more
    roundings: 2^-21 of the pair's length."""
    want = oracle.norm_rope_ref(x, w, pos, freq, eps, pairs)
    D, half = x.shape[-1], len(freq)
    got = got.double().cpu().numpy()
    r = np.abs(want)
    if pairs:
        r[..., :2 * half] = np.repeat(np.hypot(want[..., 0:2 * half:2], want[..., 1:2 * half:2]), 2, -1)
    else:
        h = np.hypot(want[..., :half], want[..., half:2 * half])
        r[..., :half], r[..., half:2 * half] = h, h
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0       # half a step of fp16's subnormal numbers
    tol = EPS[dtype] * np.abs(want) + ((D / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) * r + tiny
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,Hq,Hk,D,rot,pairs,norm", [
    (1, 1, 0, 64, 64, False, True), (1, 14, 2, 64, 64, False, False), (3, 14, 2, 64, 16, True, True),
    (33, 28, 4, 128, 128, False, True), (17, 8, 8, 128, 64, True, True), (7, 32, 8, 128, 16, False, False),
    (5, 3, 1, 256, 256, False, True), (9, 1, 1, 256, 96, True, True), (130, 1, 1, 64, 32, False, True),
    (2, 70, 1, 128, 112, True, False), (515, 4, 2, 64, 64, True, True)])
def test_heads_match_the_oracle(N, Hq, Hk, D, rot, pairs, norm, dtype):
    rng = np.random.default_rng(N + D + rot)
    q, k = (rounded(rng.standard_normal((N, h, D)) * 3, dtype) for h in (Hq, Hk))
    wq, wk = (rounded(1 + 0.3 * rng.standard_normal(D), dtype) if norm else None for _ in range(2))
    pos = rng.integers(0, 40000, N).astype(np.int32)
    freq = _freq(rot)
    dt = torch_dtype(dtype)
    dv = lambda x: None if x is None else dev(x, dt)  # noqa: E731
    oq, ok = _sdv().qk_norm_rope(dv(q), dv(k) if Hk else None, dev(pos), dev(freq), q_weight=dv(wq),
                                 k_weight=dv(wk) if Hk else None, eps=1e-5, interleaved=pairs)
    _check(oq, q, wq, pos, freq, 1e-5, pairs, dtype)
    if Hk:
        _check(ok, k, wk, pos, freq, 1e-5, pairs, dtype)
    else:
        assert ok is None


def test_far_and_negative_positions():
    """Angles of up to 2^31 radians: off by 2^-52 of themselves in 64 bits."""
    rng = np.random.default_rng(0)
    pos = np.array([0, 1, -1, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31], dtype=np.int32)
    q = rounded(rng.standard_normal((len(pos), 2, 64)), "f16")
    freq = _freq(64, 1e4)
    oq, _ = _sdv().qk_norm_rope(dev(q, torch_dtype("f16")), None, dev(pos), dev(freq))
    _check(oq, q, None, pos, freq, 0.0, False, "f16")


@pytest.mark.parametrize("pairs", [False, True])
def test_in_place_inside_a_projection(pairs):
    """Queries and keys turned where a fused projection left them; its values, and
    what lies between rows, stay."""
    import torch
    rng = np.random.default_rng(1)
    N, Hq, Hk, D = 37, 6, 2, 128
    x = rounded(rng.standard_normal((N, Hq + 2 * Hk + 1, D)), "bf16")
    t = dev(x, torch.bfloat16)
    before = t.clone()
    w = rounded(1 + 0.3 * rng.standard_normal(D), "bf16")
    pos, freq = rng.integers(0, 9999, N).astype(np.int32), _freq(64)
    q, k = t[:, :Hq], t[:, Hq:Hq + Hk]
    oq, ok = _sdv().qk_norm_rope(q, k, dev(pos), dev(freq), q_weight=dev(w, torch.bfloat16), eps=1e-6, interleaved=pairs,
                                 out_q=q, out_k=k)
    assert oq is q and ok is k
    _check(q, x[:, :Hq], w, pos, freq, 1e-6, pairs, "bf16")
    _check(k, x[:, Hq:Hq + Hk], None, pos, freq, 1e-6, pairs, "bf16")
    assert torch.equal(t[:, Hq + Hk:], before[:, Hq + Hk:])
    # strided results beside strided inputs: [heads][N][D]
    out = torch.full((Hq, N, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got, _ = _sdv().qk_norm_rope(before[:, :Hq], None, dev(pos), dev(freq), q_weight=dev(w, torch.bfloat16), eps=1e-6,
                                 interleaved=pairs, out_q=out)
    assert got is out and torch.equal(out, t[:, :Hq])


def test_rows_of_zeros_and_infinities():
    """A row of zeros stays zero (eps keeps the root); an infinity stays in its row."""
    import torch
    q = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    q[1, 1, 5] = float("inf")
    q[2, 0] = 1.0
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    pos, freq = torch.tensor([5, 6, 0], dtype=torch.int32, device="cuda"), dev(_freq(64))
    o, _ = _sdv().qk_norm_rope(q, None, pos, freq, q_weight=w, eps=1e-6)
    assert (o[0] == 0).all() and (o[1, 0] == 0).all() and (o[2, 1] == 0).all()
    assert torch.isnan(o[1, 1]).any()
    assert torch.allclose(o[2, 0], torch.ones_like(o[2, 0]))


def test_in_a_graph_and_on_a_stream():
    import torch
    sdv = _sdv()
    q, k = torch.randn((40, 8, 128), device="cuda").bfloat16(), torch.randn((40, 2, 128), device="cuda").bfloat16()
    pos, freq = torch.arange(40, dtype=torch.int32, device="cuda"), dev(_freq(128))
    oq, ok = sdv.qk_norm_rope(q, k, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sq, sk = sdv.qk_norm_rope(q, k, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(sq, oq) and torch.equal(sk, ok)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdv.qk_norm_rope(q, k, pos, freq, out_q=oq, out_k=ok)
    for i in range(3):
        q.copy_(torch.randn_like(q))
        pos.add_(i)
        want = sdv.qk_norm_rope(q, k, pos, freq)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], oq) and torch.equal(want[1], ok)
