"""Inputs for the tree-drafting GPU tests: numpy arrays for the oracle and the
same values on the device, with NaN wherever nothing may be read."""
import numpy as np

import oracle

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}    # half a step, relative


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def rounded(x, dtype):
    """Values of x in the type, as fp64 (what the device holds, exactly)."""
    import torch
    return torch.from_numpy(x).to(torch_dtype(dtype)).double().numpy()


def random_tree(rng, T):
    return [-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, T)]


class Cached:
    """Requests with a paged cache and packed tree nodes."""

    def __init__(self, seed, lens, nodes, Hq=4, Hkv=2, D=64, page=16, dtype="bf16", slot_major=False, packed=False,
                 spare=2, behind=0, sigma=1.0, room=0):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.nodes, self.dtype, self.D, self.Hq, self.H, self.page = lens, nodes, dtype, D, Hq, Hkv, page
        B = len(lens)
        cols = max(1, max(-(-(n + room) // page) for n in lens)) + 1
        pool = B * cols + spare
        self.table = rng.permutation(pool)[: B * cols].reshape(B, cols).astype(np.int32)
        self.N = sum(nodes)
        N = self.N + behind
        self.offsets = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        dt = torch_dtype(dtype)
        self.k = rounded(rng.standard_normal((pool, Hkv, page, D)), dtype)
        self.v = rounded(rng.standard_normal((pool, Hkv, page, D)), dtype)
        self.q = rounded(rng.standard_normal((N, Hq, D)) * sigma, dtype)
        self.kn = rounded(rng.standard_normal((N, Hkv, D)), dtype)
        self.vn = rounded(rng.standard_normal((N, Hkv, D)), dtype)
        used = np.zeros((pool, page), dtype=bool)
        for b, n in enumerate(lens):
            for t in range(n):
                used[self.table[b, t // page], t % page] = True
        self.k_dev, self.v_dev = self.k.copy(), self.v.copy()
        for x in (self.k_dev, self.v_dev):
            x.transpose(0, 2, 1, 3)[~used] = np.nan

        def cache(x):
            if slot_major:
                return dev(x.transpose(0, 2, 1, 3), dt).transpose(1, 2)
            return dev(x, dt)

        self.d = dict(k_cache=cache(self.k_dev), v_cache=cache(self.v_dev), page_table=dev(self.table),
                      context_lens=dev(np.array(lens, dtype=np.int32)), node_offsets=dev(self.offsets))
        if packed:      # one tensor of queries, keys and values, as a projection leaves it
            x = dev(np.concatenate([self.q, self.kn, self.vn], 1), dt)
            self.d["q"], self.d["k_new"], self.d["v_new"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.d["q"], self.d["k_new"], self.d["v_new"] = (dev(x, dt) for x in (self.q, self.kn, self.vn))
        self.scale = D ** -0.5
        assert torch.isfinite(self.d["q"]).all()

    def attention_args(self):
        return {k: self.d[k] for k in ("q", "k_new", "v_new", "k_cache", "v_cache", "page_table", "context_lens",
                                       "node_offsets")}

    def reference(self, parents=None, mask=None):
        return oracle.tree_attention_ref(self.q, self.kn, self.vn, self.k, self.v, self.table, self.lens,
                                         self.offsets, self.scale, parents, mask)

    def score_error(self):
        """Bound of a score's error: products of 8- or 11-bit numbers are exact
        in fp32, so D additions and the scaling, each off by 2^-24 of the sum
        of magnitudes; the exponent's argument in base 2 adds two more."""
        scale = abs(self.scale)
        mag = scale * self.D * np.abs(self.q).max() * max(np.abs(self.k).max(), np.abs(self.kn).max())
        top = scale * np.linalg.norm(self.q, axis=-1).max() * \
            max(np.linalg.norm(self.k, axis=-1).max(), np.linalg.norm(self.kn, axis=-1).max())
        return (self.D + 4) * 2.0 ** -24 * min(mag, 4 * top)

    def check_attention(self, out, lse, ref):
        """|out - ref|: half a step for the result; half a step of the element
        type for each weight p (they are rounded for the matrix product), and
        twice the scores' error, all times the weighted mean of |v|; fp32
        sums over n keys add n 2^-24 of the same."""
        o, e, mag = ref
        n = max(self.lens) + max(self.nodes) + 64
        out, lse = out.double().cpu().numpy()[: self.N], lse.double().cpu().numpy()[: self.N]
        eps, es = EPS[self.dtype], self.score_error()
        tol = eps * np.abs(o) + (eps + 2 * es + n * 2.0 ** -24) * (1 + eps) * mag + 2.0 ** -24
        if self.dtype == "f16":
            # weights below fp16's smallest normal number lose relative
            # precision: at most 2^-25 each
            tol = tol + n * 2.0 ** -25 * np.abs(np.nan_to_num(self.v)).max()
        bad = np.abs(out - o[: self.N]) > tol[: self.N]
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(out - o[: self.N]).max())
        assert np.isfinite(out).all()
        none = np.isinf(e[: self.N])
        assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
        d = np.abs(lse[~none] - e[: self.N][~none])
        assert (d <= es + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(e[: self.N][~none]))).all(), d.max()
