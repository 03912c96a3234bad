"""Inputs for the GPU tests of include/sd_serve.h: numpy arrays for the oracle and
the same values on the device, with codes that are not numbers (or large ones)
wherever nothing may be read."""
import numpy as np

import oracle
from treetools import EPS, dev, rounded, torch_dtype

CODE = {"i8": "int8", "e4m3": "float8_e4m3fn"}


def code_dev(x, code):
    """Codes as the device holds them; NaN becomes 0x7f in e4m3."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(getattr(torch, CODE[code]))


def code_np(t):
    return t.float().double().cpu().numpy()


def random_cache(rng, pool, H, page, D, block, code, spread=0.5):
    """Random values [pool][H][page][D] quantised: (codes fp64, scales fp32)."""
    x = rng.standard_normal((pool, H, page // block, block, D)).astype(np.float32)
    x *= np.exp(rng.standard_normal((pool, H, page // block, 1, 1)) * spread).astype(np.float32)
    top = np.float32(oracle.serve.TOP[code])
    s = np.abs(x).max(axis=(3, 4)) / top
    y = np.clip(x / s[..., None, None], -top, top).astype(np.float64)
    c = np.rint(y) if code == "i8" else oracle.e4m3_round(y)
    return c.reshape(pool, H, page, D), s


class Quantised:
    """Requests with a paged 8-bit cache and packed tree nodes."""

    def __init__(self, seed, lens, nodes, Hq=4, Hkv=2, D=64, page=16, block=16, code="i8", dtype="bf16", room=0, behind=0,
                 sigma=1.0, spread=0.5, slot_major=False, packed=False):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.nodes, self.D, self.Hq, self.H, self.page, self.block = lens, nodes, D, Hq, Hkv, page, block
        self.code, self.dtype = code, dtype
        B = len(lens)
        cols = max(1, max(-(-(n + room) // page) for n in lens)) + 1
        pool = B * cols + 2
        self.table = rng.permutation(pool)[: B * cols].reshape(B, cols).astype(np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.N = sum(nodes)
        N = self.N + behind
        dt = torch_dtype(dtype)
        self.k, self.ks = random_cache(rng, pool, Hkv, page, D, block, code, spread)
        self.v, self.vs = random_cache(rng, pool, Hkv, page, D, block, code, spread)
        self.q = rounded(rng.standard_normal((N, Hq, D)) * sigma, dtype)
        self.kn = rounded(rng.standard_normal((N, Hkv, D)), dtype)
        self.vn = rounded(rng.standard_normal((N, Hkv, D)), dtype)
        used = np.zeros((pool, page), dtype=bool)
        for b, n in enumerate(lens):
            for t in range(n):
                used[self.table[b, t // page], t % page] = True
        junk = np.nan if code == "e4m3" else -128.0      # what lies in slots that are not in use
        kd, vd, ks, vs = self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy()
        for x in (kd, vd):
            x.transpose(0, 2, 1, 3)[~used] = junk
        whole = used.reshape(pool, page // block, block).any(-1)      # scales of blocks without a slot in use
        for x in (ks, vs):
            x.transpose(0, 2, 1)[~whole] = np.nan

        def cache(x):
            if slot_major:
                return code_dev(x.transpose(0, 2, 1, 3), code).transpose(1, 2)
            return code_dev(x, code)

        self.d = dict(k_cache=cache(kd), v_cache=cache(vd), k_scale=dev(ks), v_scale=dev(vs), page_table=dev(self.table),
                      context_lens=dev(np.array(lens, dtype=np.int32)), node_offsets=dev(self.offsets))
        if packed:      # one tensor of queries, keys and values, as a projection leaves it
            x = dev(np.concatenate([self.q, self.kn, self.vn], 1), dt)
            self.d["q"], self.d["k_new"], self.d["v_new"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.d["q"], self.d["k_new"], self.d["v_new"] = (dev(x, dt) for x in (self.q, self.kn, self.vn))
        self.scale = D ** -0.5
        assert torch.isfinite(self.d["q"]).all()

    def attention_args(self):
        return {k: self.d[k] for k in ("q", "k_new", "v_new", "k_cache", "v_cache", "k_scale", "v_scale", "page_table",
                                       "context_lens", "node_offsets")}

    def reference(self, parents=None, window=0, sinks=0, scale=None):
        return oracle.quant_attention_ref(self.q, self.kn, self.vn, self.k, self.v, self.ks, self.vs, self.table, self.lens,
                                          self.offsets, self.block, self.scale if scale is None else scale, parents, window,
                                          sinks)

    def score_error(self, scale=None):
        """Bound of a score's error: products of a code and an element have at most
        19 bits, exact in fp32, so D additions and three more roundings, each off by
        2^-24 of the sum of magnitudes; log2 of a value scale (below 2^5 in magnitude)
        and its sum with the score add 2^-20."""
        scale = abs(self.scale if scale is None else scale)
        top = max(self.ks.max() * oracle.serve.TOP[self.code], np.abs(self.kn).max())
        mag = scale * self.D * np.abs(self.q).max() * top
        return (self.D + 8) * 2.0 ** -24 * mag + 2.0 ** -20

    def check(self, out, lse, ref, scale=None):
        """|out - ref|: half a step for the result; for each weight half a step of
        the type it enters the product in (fp16 for the cache, the queries' for the
        nodes), and twice the scores' error, all times the weighted mean of |v|; fp32
        sums over n keys add n 2^-24 of the same; fp16 weights far below the largest
        lose at most 2^-32 of it each.  int8 codes are summed up as code + 128, so n
        additions are off by n 2^-24 of a sum of up to 255 scales times the weights
        where |v| would be less."""
        o, e, mag = ref
        n = max(self.lens) + max(self.nodes) + 64
        out, lse = out.double().cpu().numpy()[: self.N], lse.double().cpu().numpy()[: self.N]
        o, e, mag = o[: self.N], e[: self.N], mag[: self.N]
        eps, es = EPS[self.dtype], self.score_error(scale)
        big = max((self.vs.max() * oracle.serve.TOP[self.code]), np.abs(self.vn).max())
        tol = eps * np.abs(o) + (eps + 2 * es + n * 2.0 ** -24) * (1 + eps) * mag + n * 2.0 ** -32 * big + 2.0 ** -24
        if self.code == "i8":
            tol = tol + n * 2.0 ** -24 * 255 * np.nan_to_num(self.vs).max()
        bad = ~(np.abs(out - o) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], np.nanmax(np.abs(out - o)))
        none = np.isinf(e)
        assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
        d = np.abs(lse[~none] - e[~none])
        assert (d <= es + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(e[~none]))).all(), d.max()
