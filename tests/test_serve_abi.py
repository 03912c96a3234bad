"""The entry points of include/sd_serve.h on the host (CPU only, nothing is
launched): struct layouts, exports, and every refusal of a bad argument."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sd_serve.h")

P = ctypes.c_void_p
OUT = P(0x900000)


@pytest.fixture(scope="module")
def sdv():
    import speculative_sampling_verify_temp_amd as m
    return m


def _serve():
    import speculative_sampling_verify_temp_amd.serve as s
    return s


def test_every_declared_symbol_is_exported(sdv):
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sd_[a-z_0-9]+)\s*\(", txt)))
    assert len(names) == 7
    for n in names:
        assert hasattr(sdv.lib, n), n


STRUCTS = [("SdQkNormRopeArgs", "sd_qk_norm_rope_args_t", "_NORM_ROPE"), ("SdQuantCache", "sd_quant_cache_t", None),
           ("SdQuantAttentionArgs", "sd_quant_attention_args_t", "_QUANT_ATTENTION"),
           ("SdQuantAppendArgs", "sd_quant_append_args_t", "_QUANT_APPEND"),
           ("SdTreeSampleArgs", "sd_tree_sample_args_t", "_TREE_SAMPLE")]


@pytest.mark.parametrize("cls,name,packed", STRUCTS)
def test_struct_layouts_match_the_header(cls, name, packed, tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    A = getattr(_serve(), cls)
    fields = [f[0] for f in A._fields_]
    src = tmp_path / "t.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"sd_serve.h\"\nint main(void){"
                   f"printf(\"%zu\", sizeof({name}));" +
                   "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields) + "return 0;}\n")
    exe = tmp_path / "t"
    subprocess.run([gcc, "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(A)] + [getattr(A, f).offset for f in fields]


@pytest.mark.parametrize("cls,name,packed", [s for s in STRUCTS if s[2]])
def test_packed_arguments_are_the_structs(cls, name, packed):
    """The binding packs argument structs as bytes: every value lands in its field."""
    S = _serve()
    A, pk = getattr(S, cls), getattr(S, packed)
    fields = []
    for n, kind in A._fields_:
        fields += [(True, f[0]) for f in kind._fields_] if kind is S.SdQuantCache else [(False, n)]
    assert pk.size == ctypes.sizeof(A)
    a = A.from_buffer_copy(pk.pack(*range(1, len(fields) + 1)))
    assert [getattr(a.cache if inner else a, n) for inner, n in fields] == list(range(1, len(fields) + 1))


def _cache():
    return _serve().SdQuantCache(0x100000, 0x200000, 0x280000, 0x290000, 4 * 16 * 128, 16 * 128, 128, 4, 1, 0x300000, 10,
                                 0x310000, 3, 2, 4, 128, 16, 16, 20, 10)


CACHE_DEFECTS = [
    ("k", None, -1), ("v", None, -1), ("k", 0x100008, -1), ("k_scale", None, -1), ("v_scale", 0x290002, -1),
    ("page_table", None, -1), ("context_lens", None, -1), ("code", 1, -1), ("code", 5, -1), ("B", 0, -1),
    ("H_kv", 0, -1), ("D", 0, -1), ("D", 80, -4), ("page_size", 0, -1), ("page_size", 24, -4), ("page_size", 8, -4),
    ("page_size", 2048, -4), ("block", 0, -1), ("block", 8, -4), ("block", 32, -4), ("block", 24, -4),
    ("num_pages", 0, -1), ("max_pages", 0, -1), ("ld_table", 9, -1), ("page_stride", -16, -1), ("head_stride", 8, -1),
    ("slot_stride", 112, -1), ("slot_stride", 136, -1), ("slot_stride", 1 << 21, -4), ("scale_page", -1, -1),
    ("scale_head", -1, -1), ("B", 70000, -4), ("H_kv", 32768, -4),
]


def _rope():
    return _serve().SdQkNormRopeArgs(0x100000, 0x200000, 0x300000, 0x400000, 1024, 128, 512, 128, 1024, 128, 512, 128,
                                     0x500000, 0x510000, 0x520000, 0x530000, 1, 6, 8, 4, 128, 64, 0, 1e-6)


def _attention():
    return _serve().SdQuantAttentionArgs(_cache(), 0x400000, 0x410000, 0x420000, 1024, 128, 512, 128, 512, 128,
                                         0x430000, None, 1, 6, 3, 8, 0, 0, 0.5)


def _append():
    return _serve().SdQuantAppendArgs(_cache(), 0x410000, 0x420000, 512, 128, 512, 128, 0x430000, 0x440000, 3, 0x450000,
                                      1, 6, 3)


def _sample():
    return _serve().SdTreeSampleArgs(0x100000, 0x180000, 1000, 1000, 0x200000, 0x210000, 0x220000, 0x230000, 0x240000,
                                     2, 6, 1000, 1000, 3, 0)


MAKE = dict(rope=_rope, attention=_attention, append=_append, sample=_sample)


def _call(sdv, kind, a, ws=P(0xA00000), n=1 << 40, out=OUT, st=None):
    lib, r = sdv.lib, ctypes.byref(a)
    if kind == "rope":
        return lib.sd_qk_norm_rope(r, None)
    if kind == "attention":
        return lib.sd_quant_attention(r, ws, n, out, None, st, None)
    if kind == "append":
        return lib.sd_quant_append(r, out, st, None)
    return lib.sd_tree_verify_sample(r, ws, n, out, P(0x910000), P(0x920000), st, None)


@pytest.mark.parametrize("kind", ["attention", "append"])
@pytest.mark.parametrize("field,value,code", CACHE_DEFECTS)
def test_cache_defects_are_refused(sdv, kind, field, value, code):
    a = MAKE[kind]()
    setattr(a.cache, field, value)
    if field == "H_kv" and value > 4:
        a.H_q = value
    assert _call(sdv, kind, a) == code


@pytest.mark.parametrize("kind,field,value,code", [
    ("rope", "q", None, -1), ("rope", "q", 0x100008, -1), ("rope", "k", None, -1), ("rope", "q_out", None, -1),
    ("rope", "k_out", 0x400004, -1), ("rope", "q_node", 1020, -1), ("rope", "k_head", -128, -1),
    ("rope", "q_weight", 0x500002, -1), ("rope", "positions", None, -1), ("rope", "inv_freq", None, -1),
    ("rope", "dtype", 0, -1), ("rope", "dtype", 3, -1), ("rope", "N", 0, -1), ("rope", "H_q", 0, -1),
    ("rope", "H_k", -1, -1), ("rope", "D", 80, -4), ("rope", "D", 32, -1), ("rope", "rot", 0, -1),
    ("rope", "rot", 24, -1), ("rope", "rot", 144, -1), ("rope", "eps", -1.0, -1), ("rope", "eps", float("nan"), -1),
    ("rope", "eps", float("inf"), -1), ("rope", "H_q", 65535, -4), ("rope", "q_out_head", 0, -1),
    ("rope", "q_out_head", 64, -1), ("rope", "q_out_node", 1000, -1), ("rope", "k_out_node", 0, -1),
    ("attention", "q", None, -1), ("attention", "k_new", 0x410004, -1), ("attention", "v_new", None, -1),
    ("attention", "q_node", 1020, -1), ("attention", "k_head", -128, -1), ("attention", "node_offsets", None, -1),
    ("attention", "dtype", 3, -1), ("attention", "N", 0, -1), ("attention", "max_nodes", 0, -1),
    ("attention", "max_nodes", 65, -4), ("attention", "H_q", 6, -1), ("attention", "H_q", 0, -1),
    ("attention", "H_q", 4 * 33, -4), ("attention", "scale", float("nan"), -1), ("attention", "scale", float("inf"), -1),
    ("attention", "window", -1, -1), ("attention", "sinks", -1, -1), ("attention", "sinks", 4, -1),
    ("append", "k_new", None, -1), ("append", "v_node", 4, -1), ("append", "node_offsets", None, -1),
    ("append", "path_lens", None, -1), ("append", "ld_path", 2, -1), ("append", "dtype", 0, -1), ("append", "N", 0, -1),
    ("append", "max_new", 0, -1),
    ("sample", "target_probs", None, -1), ("sample", "target_probs", 0x100008, -1), ("sample", "draft_probs", 0x180004, -1),
    ("sample", "ld_target", 996, -1), ("sample", "ld_target", 1002, -1), ("sample", "ld_draft", 999, -1),
    ("sample", "tokens", None, -1), ("sample", "parents", None, -1), ("sample", "node_offsets", None, -1),
    ("sample", "accept_uniforms", None, -1), ("sample", "draw_uniforms", None, -1), ("sample", "B", 0, -1),
    ("sample", "N", 0, -1), ("sample", "V", 0, -1), ("sample", "V_draft", 0, -1), ("sample", "V_draft", 1001, -1),
    ("sample", "max_nodes", 0, -1), ("sample", "max_nodes", 65, -4), ("sample", "flags", 2, -1), ("sample", "B", 65536, -4),
])
def test_bad_arguments_are_refused(sdv, kind, field, value, code):
    a = MAKE[kind]()
    setattr(a, field, value)
    assert _call(sdv, kind, a) == code


def test_grids_beyond_the_limits_are_refused(sdv):
    """More workgroups than a grid holds: neither call writes anything."""
    a = _rope()
    a.N = 2 ** 31 - 1
    assert _call(sdv, "rope", a) == -4
    a = _append()
    a.path, a.max_new = None, 2 ** 28
    a.cache.max_pages = a.cache.ld_table = 2 ** 26
    assert _call(sdv, "append", a) == -4


def test_sizes_beyond_the_limits_are_refused(sdv):
    a = _append()
    a.max_new = a.ld_path = 65
    assert _call(sdv, "append", a) == -4
    a = _sample()
    a.V = a.V_draft = a.ld_target = a.ld_draft = 1 << 28
    assert _call(sdv, "sample", a) == -4
    n = ctypes.c_size_t()
    for kind, f in (("attention", sdv.lib.sd_quant_attention_workspace_bytes),):
        a = MAKE[kind]()
        a.cache.page_size = a.cache.block = 1024
        a.cache.max_pages = a.cache.ld_table = 1 << 20
        a.cache.B = 65535
        assert f(ctypes.byref(a), ctypes.byref(n)) == -4
        a.window, a.sinks = 100, 5      # few key tiles through a window
        assert f(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
        a.cache.max_pages = a.cache.ld_table = (1 << 20) + 1
        assert f(ctypes.byref(a), ctypes.byref(n)) == -4


@pytest.mark.parametrize("kind", ["sample", "attention"])
def test_missing_outputs_and_small_workspaces_are_refused(sdv, kind):
    a = MAKE[kind]()
    if kind == "attention":
        a.cache.max_pages = a.cache.ld_table = 1000
    assert _call(sdv, kind, a, out=None) == -1
    assert _call(sdv, kind, a, ws=None) == sdv.SD_EWORKSPACE
    assert _call(sdv, kind, a, n=7) == sdv.SD_EWORKSPACE
    assert _call(sdv, kind, a, ws=P(0xA00004)) == sdv.SD_EWORKSPACE


def test_outputs_that_may_not_be_inputs_are_refused(sdv):
    for field in ("q_weight", "k_weight", "positions", "inv_freq", "k", "k_out"):
        a = _rope()
        a.q_out = getattr(a, field)
        assert _call(sdv, "rope", a) == -1, field
    a = _rope()
    a.k_out = a.q
    assert _call(sdv, "rope", a) == -1
    for s in ("q", "k"):      # in place only with equal strides
        a = _rope()
        setattr(a, s + "_out", getattr(a, s))
        setattr(a, s + "_node", 2048)
        assert _call(sdv, "rope", a) == -1
    assert _call(sdv, "attention", _attention(), out=P(0x900008)) == -1
    for field in ("k_new", "v_new"):
        a = _attention()
        assert _call(sdv, "attention", a, out=P(getattr(a, field))) == -1, field
    for field in ("k", "v"):
        a = _attention()
        assert _call(sdv, "attention", a, out=P(getattr(a.cache, field))) == -1, field
    for field, value in (("q_node", 1032), ("q_head", 136), ("q_head", 0)):      # rows of others' queries
        a = _attention()
        setattr(a, field, value)
        assert _call(sdv, "attention", a, out=P(a.q)) == -1, field
    for out in (None, P(0x310000), P(0x300000), P(0x430000), P(0x440000), P(0x450000)):
        assert _call(sdv, "append", _append(), out=out) == -1
    assert _call(sdv, "append", _append(), st=OUT) == -1
    for out in (0x100000, 0x180000, 0x200000, 0x210000, 0x220000, 0x230000, 0x240000, 0x910000):
        assert _call(sdv, "sample", _sample(), out=P(out)) == -1, hex(out)
    assert _call(sdv, "sample", _sample(), st=OUT) == -1


def test_rows_that_share_memory_are_not_written(sdv):
    for field in ("page_stride", "head_stride", "scale_page", "scale_head"):
        a = _append()
        setattr(a.cache, field, 0)
        assert _call(sdv, "append", a) == -1, field
    for x, y in (("k", "v"), ("k_scale", "v_scale")):
        a = _append()
        setattr(a.cache, y, getattr(a.cache, x))
        assert _call(sdv, "append", a) == -1


def test_the_binding_refuses_what_it_can_see(sdv):
    """Tensors that are not on the current GPU, wrong types, shapes and strides raise
    before any call (CPU tensors here)."""
    import torch
    k = torch.zeros(20, 4, 32, 64, dtype=torch.int8)
    sc = torch.zeros(20, 4, 2)
    table, lens, off = torch.zeros(2, 10, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), \
        torch.tensor([0, 3, 6], dtype=torch.int32)
    q, kn = torch.zeros(6, 8, 64, dtype=torch.bfloat16), torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    make = lambda **o: sdv.make_quant_attention_args(**{**dict(  # noqa: E731
        q=q, k_new=kn, v_new=kn, k_cache=k, v_cache=k, k_scale=sc, v_scale=sc, page_table=table, context_lens=lens,
        node_offsets=off, max_nodes=3), **o})
    a = make(window=7, sinks=2)
    c = a.cache
    assert (c.code, c.B, c.H_kv, c.D, c.page_size, c.block, c.num_pages, c.max_pages) == (3, 2, 4, 64, 32, 16, 20, 10)
    assert (a.dtype, a.N, a.H_q, a.window, a.sinks, a.scale) == (1, 6, 8, 7, 2, 0.125)
    e = make(k_cache=k.to(torch.float8_e4m3fn), v_cache=k.to(torch.float8_e4m3fn))
    assert e.cache.code == 4
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(k_new=kn[:5]), dict(k_new=kn.half()),
                dict(v_cache=k[:, :, :16]), dict(v_cache=k.view(torch.uint8)), dict(k_scale=sc.double()),
                dict(k_scale=sc[:, :2], v_scale=sc[:, :2]), dict(k_scale=torch.zeros(20, 4, 3), v_scale=torch.zeros(20, 4, 3)),
                dict(k_scale=sc[..., :1]), dict(k_scale=torch.zeros(20, 4, 4)[..., ::2], v_scale=torch.zeros(20, 4, 4)[..., ::2]),
                dict(page_table=table.long()), dict(page_table=table.t()), dict(context_lens=lens.long()),
                dict(node_offsets=off[:2]), dict(parents=off), dict(k_cache=k.transpose(2, 3), v_cache=k.transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            make(**bad)
    with pytest.raises(TypeError):
        make(k_cache=k.half(), v_cache=k.half())
    for call in (lambda: sdv.quant_attention(q, kn, kn, k, k, sc, sc, table, lens, off, 3),
                 lambda: sdv.quant_append(kn, kn, k, k, sc, sc, table, lens, off, 3, lens),
                 lambda: sdv.qk_norm_rope(q, kn, torch.zeros(6, dtype=torch.int32), torch.zeros(32)),
                 lambda: sdv.tree_verify_sample(torch.zeros(6, 100), torch.zeros(6, dtype=torch.int32),
                                                torch.zeros(6, dtype=torch.int32), off, 3, torch.zeros(6), torch.zeros(2))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_strides_of_axes_of_one_are_not_looked_at(sdv):
    """One packed node in place of its query, wherever it lies; the binding's strides of
    axes of one are those of no tensor."""
    import torch
    n = ctypes.c_size_t()
    a = _attention()
    a.N, a.max_nodes, a.q_node = 1, 1, 2048
    a.cache.max_pages = a.cache.ld_table = 1000
    assert _call(sdv, "attention", a, out=P(a.q), ws=None) == sdv.SD_EWORKSPACE      # all but the workspace is fine
    a.N = 2
    assert _call(sdv, "attention", a, out=P(a.q), ws=None) == -1
    k = torch.zeros(64 * 64, dtype=torch.int8)
    kc, vc = k.as_strided((1, 1, 64, 64), (3, 5, 64, 1)), k.as_strided((1, 1, 64, 64), (48, 7, 64, 1))
    sc = torch.zeros(2)
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    got = sdv.make_quant_attention_args(
        x[0, :1], x[0, :1, :1].as_strided((1, 1, 64), (3, 5, 1)), x[0, :1, :1], kc, vc, sc.as_strided((1, 1, 2), (9, 4, 1)),
        sc.as_strided((1, 1, 2), (2, 6, 1)), torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
        torch.tensor([0, 1], dtype=torch.int32), 1)
    c = got.cache
    assert (c.page_stride, c.head_stride, c.slot_stride, c.scale_page, c.scale_head) == (0, 0, 64, 0, 0)
    assert got.k_node % 8 == got.k_head % 8 == 0
    assert sdv.lib.sd_quant_attention_workspace_bytes(ctypes.byref(got), ctypes.byref(n)) == 0
    for bad in (kc.as_strided((1, 1, 32, 64), (3, 5, 128, 1)), kc[:, :, :32]):      # strides of other axes
        with pytest.raises(ValueError):
            sdv.make_quant_attention_args(x[0, :1], x[0, :1, :1], x[0, :1, :1], kc, bad, sc.reshape(1, 1, 2), sc.reshape(1, 1, 2),
                                          torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                          torch.tensor([0, 1], dtype=torch.int32), 1)


def test_outputs_of_the_attention_that_may_not_be_inputs_are_refused(sdv):
    """Every output against every input, the other outputs and the workspace."""
    a = _attention()
    a.parents = 0x440000
    a.cache.max_pages = a.cache.ld_table = 1000
    ws, out, lse, st = 0xA00000, 0x900000, 0x910000, 0x920000
    call = lambda o, e, s: sdv.lib.sd_quant_attention(ctypes.byref(a), P(ws), 7, P(o), P(e), P(s), None)  # noqa: E731
    assert call(out, lse, st) == sdv.SD_EWORKSPACE      # nothing but the workspace's size
    ins = [a.k_new, a.v_new, a.cache.k, a.cache.v, a.cache.k_scale, a.cache.v_scale, a.cache.page_table,
           a.cache.context_lens, a.node_offsets, a.parents, ws]
    for x in ins:
        assert call(x, lse, st) == call(out, x, st) == call(out, lse, x) == -1, hex(x)
    assert call(out, a.q, st) == call(out, lse, a.q) == -1
    assert call(out, out, st) == call(out, lse, out) == call(out, lse, lse) == -1
    assert call(a.q, lse, st) == sdv.SD_EWORKSPACE
