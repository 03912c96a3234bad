"""Serving steps of drafted trees over a cache in 8 bits, the operators of
include/sd_serve.h one after another as a server calls them: the tree's queries and
keys are normed and turned, attend, give the target's probabilities, the tree is
verified against them and the kept branch appended.  Each result against the fp64
oracle of what went in, and all of them again through replayed graphs."""
import numpy as np
import pytest

import oracle
from servetools import Quantised, code_np
from test_gpu_norm_rope import _check as check_rotation
from treetools import dev, random_tree, rounded, torch_dtype

pytestmark = pytest.mark.gpu

V, T, STEPS, EPS = 997, 7, 4, 1e-5


def _sdv():
    import speculative_sampling_verify_temp_amd as sdv
    return sdv


class Server:
    """Requests in prefill and then in steps; a model of one layer with random weights."""

    def __init__(self, seed, code, dtype, window, prompts=(0, 5, 33, 90)):
        import torch
        self.window, self.prompts, self.B = window, prompts, len(prompts)
        self.s = s = Quantised(seed, [0] * self.B, [T] * self.B, Hq=6, Hkv=2, D=64, code=code, dtype=dtype,
                               room=max(prompts) + STEPS * T)
        rng = np.random.default_rng(seed)
        self.dt = dt = torch_dtype(dtype)
        self.heads = s.Hq + 2 * s.H
        norm = lambda *n: rounded(rng.standard_normal(n), dtype)  # noqa: E731
        self.embed, self.proj = dev(norm(V, 32), dt), dev(norm(32, self.heads * s.D), dt)
        self.head = dev(norm(s.Hq * s.D, V), dt)
        self.wq, self.wk = (rounded(1 + 0.2 * rng.standard_normal(s.D), dtype) for _ in range(2))
        self.dwq, self.dwk = dev(self.wq, dt), dev(self.wk, dt)
        self.freq = (1e4 ** (-np.arange(s.D // 2) / (s.D // 2))).astype(np.float32)
        self.dfreq = dev(self.freq)
        # what a step reads, in place for the graphs
        N = self.B * T
        z = lambda *n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
        self.qkv, self.pos = z(N, self.heads, s.D, t=dt), z(N)
        self.tokens, self.parents = z(N), z(N)
        self.draft, self.probs = (z(N, V + 3, t=torch.float32)[:, :V] for _ in range(2))
        self.u, self.v = z(N, t=torch.float32), z(self.B, t=torch.float32)
        self.ctx, self.now = s.d["context_lens"], z(self.B)
        self.status = [z(self.B) for _ in range(3)]
        self.cache = {k: s.d[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "page_table")}
        self.rng = np.random.default_rng(seed + 1)
        self.prefill()

    def project(self, tokens):
        return (self.embed[tokens.long()] @ self.proj).view(-1, self.heads, self.s.D) / 6

    def rotate(self, qkv, pos):
        h = self.s.Hq + self.s.H
        return _sdv().qk_norm_rope(qkv[:, :self.s.Hq], qkv[:, self.s.Hq:h], pos, self.dfreq, self.dwq, self.dwk, EPS,
                                   out_q=qkv[:, :self.s.Hq], out_k=qkv[:, self.s.Hq:h])

    def prefill(self):
        """The prompts' keys and values, all requests in one call."""
        import torch
        off = np.concatenate([[0], np.cumsum(self.prompts)]).astype(np.int32)
        pos = dev(np.concatenate([np.arange(n) for n in self.prompts]).astype(np.int32))
        qkv = self.project(dev(self.rng.integers(0, V, off[-1]))).contiguous()
        raw = qkv.clone()
        q, k = self.rotate(qkv, pos)
        Hq, H = self.s.Hq, self.s.H
        self.check_rotation(raw, q, k, pos)
        want = self.state()
        self.expect(want, k, qkv[:, Hq + H:], [range(off[b], off[b + 1]) for b in range(self.B)])
        _sdv().quant_append(k, qkv[:, Hq + H:], **self.cache, context_lens=self.ctx, node_offsets=dev(off),
                            max_new=max(self.prompts), out_context=self.now, status=self.status[0])
        assert self.now.tolist() == list(self.prompts) and not self.status[0].any()
        self.same(want)
        self.ctx.copy_(self.now)
        torch.cuda.synchronize()

    def draft_trees(self):
        """Children drawn from random draft rows; the root is the last token emitted."""
        import torch
        off = self.s.offsets
        z = self.rng.standard_normal((self.B * T, V)) * 2
        q = np.exp(z) / np.exp(z).sum(1, keepdims=True)
        up = np.concatenate([random_tree(self.rng, T) for _ in range(self.B)]).astype(np.int32)
        tok = self.rng.integers(0, V, self.B * T).astype(np.int32)
        deep = np.zeros(self.B * T, dtype=np.int32)
        for b in range(self.B):
            for i in range(1, T):
                c = off[b] + up[off[b] + i]
                deep[off[b] + i] = deep[c] + 1
                tok[off[b] + i] = self.rng.choice(V, p=q[c])
        self.tokens.copy_(dev(tok)), self.parents.copy_(dev(up)), self.draft.copy_(dev(q.astype(np.float32)))
        self.u.copy_(dev(self.rng.random(self.B * T).astype(np.float32)))
        self.v.copy_(dev(self.rng.random(self.B).astype(np.float32)))
        self.pos.copy_(self.ctx.repeat_interleave(T) + dev(deep))
        self.qkv.copy_(self.project(self.tokens))
        torch.cuda.synchronize()

    def attend(self):
        s, Hq, h = self.s, self.s.Hq, self.s.Hq + self.s.H
        q, k = self.rotate(self.qkv, self.pos)
        self.out, self.lse = _sdv().quant_attention(
            q, k, self.qkv[:, h:], **self.cache, context_lens=self.ctx, node_offsets=s.d["node_offsets"], max_nodes=T,
            parents=self.parents, window=self.window, sinks=2 if self.window else 0, want_lse=True, status=self.status[0])

    def target(self):
        logits = (self.out.view(self.B * T, -1) @ self.head).float() / 4
        self.probs.copy_(logits.softmax(-1))

    def keep(self):
        s, Hq, h = self.s, self.s.Hq, self.s.Hq + self.s.H
        self.got = _sdv().tree_verify_sample(self.probs, self.tokens, self.parents, s.d["node_offsets"], T, self.u, self.v,
                                             draft_probs=self.draft, status=self.status[1])
        _sdv().quant_append(self.qkv[:, Hq:h], self.qkv[:, h:], **self.cache, context_lens=self.ctx,
                            node_offsets=s.d["node_offsets"], max_new=T, out_context=self.now, path=self.got[1],
                            path_lens=self.got[0] + 1, status=self.status[2])
        self.ctx.copy_(self.now)

    # ---- against the oracle ----

    def state(self):
        return tuple(code_np(self.cache[k]) if "cache" in k else self.cache[k].cpu().numpy()
                     for k in ("k_cache", "v_cache", "k_scale", "v_scale"))

    def same(self, want):
        for g, w in zip(self.state(), want):
            assert np.array_equal(g, w, equal_nan=True)

    def expect(self, state, k, v, rows):
        k, v = k.float().cpu().numpy(), v.float().cpu().numpy()
        kc, vc, ks, vs = state
        for b, (r, n) in enumerate(zip(rows, self.ctx.tolist())):
            oracle.quant_append_ref(k[list(r)], kc, ks, self.s.table[b], n, self.s.block, self.s.code)
            oracle.quant_append_ref(v[list(r)], vc, vs, self.s.table[b], n, self.s.block, self.s.code)

    def check_rotation(self, raw, q, k, pos):
        Hq, H = self.s.Hq, self.s.H
        raw, pos = raw.double().cpu().numpy(), pos.cpu().numpy()
        check_rotation(q, raw[:, :Hq], self.wq, pos, self.freq, EPS, False, self.s.dtype)
        check_rotation(k, raw[:, Hq:Hq + H], self.wk, pos, self.freq, EPS, False, self.s.dtype)

    def checked_step(self):
        s, Hq, h = self.s, self.s.Hq, self.s.Hq + self.s.H
        raw, before, lens = self.qkv.clone(), self.state(), self.ctx.tolist()
        self.attend()
        num = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.check_rotation(raw, self.qkv[:, :Hq], self.qkv[:, Hq:h], self.pos)
        assert np.array_equal(num(raw[:, h:]), num(self.qkv[:, h:]))
        s.q, s.kn, s.vn = num(self.qkv[:, :Hq]), num(self.qkv[:, Hq:h]), num(self.qkv[:, h:])
        s.lens, (s.k, s.v, s.ks, s.vs) = lens, before
        up = self.parents.cpu().numpy()
        ref = s.reference(up, self.window, 2 if self.window else 0)
        ks, vs = s.ks, s.vs
        s.ks, s.vs = np.nan_to_num(ks), np.nan_to_num(vs)      # (scales of blocks not in use, for the bound alone)
        s.check(self.out, self.lse, ref)
        s.ks, s.vs = ks, vs
        self.target()
        self.keep()
        acc, path, tok, margin = oracle.tree_sample_ref(self.probs.cpu().numpy(), self.draft.cpu().numpy(),
                                                        self.tokens.cpu().numpy(), up, s.offsets, T, self.u.cpu().numpy(),
                                                        self.v.cpu().numpy())
        sure = margin > V * 2.0 ** -50
        for g, w in zip(self.got, (acc, path, tok)):
            assert np.array_equal(g.cpu().numpy()[sure], w[sure])
        acc, path, _ = (g.cpu().numpy() for g in self.got)
        self.ctx.copy_(dev(np.array(lens, dtype=np.int32)))
        self.expect(before, self.qkv[:, Hq:h], self.qkv[:, h:],
                    [[s.offsets[b] + path[b, i] for i in range(acc[b] + 1)] for b in range(self.B)])
        self.same(before)
        assert self.now.tolist() == [n + a + 1 for n, a in zip(lens, acc)]
        self.ctx.copy_(self.now)
        assert not any(st.any() for st in self.status)
        return [t.clone() for t in (self.out, self.lse, *self.got, self.now)]


@pytest.mark.parametrize("code,dtype,window", [("i8", "bf16", 0), ("e4m3", "f16", 0), ("i8", "f16", 21), ("e4m3", "bf16", 40)])
def test_steps_match_the_oracle_and_replay(code, dtype, window):
    import torch
    one = Server(3, code, dtype, window)
    steps, kept = [], 0
    for _ in range(STEPS):
        one.draft_trees()
        steps.append(one.checked_step())
        kept += int(steps[-1][2].sum())
    print(f"{code} {dtype}: {kept} drafted tokens kept", flush=True)

    # the same steps again, each in two graphs around the model's own products
    two = Server(3, code, dtype, window)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    lens = two.ctx.clone()
    with torch.cuda.graph(first):
        two.attend()
    two.probs.copy_(torch.ones_like(two.probs) / V)
    with torch.cuda.graph(second):
        two.keep()
    assert torch.equal(lens, two.ctx)
    for want in steps:
        two.draft_trees()
        first.replay()
        two.target()
        second.replay()
        torch.cuda.synchronize()
        for g, w in zip((two.out, two.lse, *two.got, two.now), want):
            assert torch.equal(g, w)
    for k in ("k_cache", "v_cache", "k_scale", "v_scale"):
        a, b = one.cache[k], two.cache[k]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
