"""The tree-drafting entry points on the host (CPU only, nothing is launched):
struct layouts, exports, and every refusal of a bad argument."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sd_tree.h")

P = ctypes.c_void_p
OUT = P(0x900000)


@pytest.fixture(scope="module")
def sdv():
    import speculative_sampling_verify_temp_amd as m
    return m


def _tree():
    import speculative_sampling_verify_temp_amd.tree as t
    return t


def test_every_declared_symbol_is_exported(sdv):
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sd_[a-z_0-9]+)\s*\(", txt)))
    assert len(names) == 10
    for n in names:
        assert hasattr(sdv.lib, n), n


@pytest.mark.parametrize("cls,name", [
    ("SdKvCache", "sd_kv_cache_t"), ("SdTreeAttentionArgs", "sd_tree_attention_args_t"),
    ("SdTreeVerifyArgs", "sd_tree_verify_args_t"), ("SdCacheCommitArgs", "sd_cache_commit_args_t"),
    ("SdCacheEvictArgs", "sd_cache_evict_args_t"), ("SdBeamSelectArgs", "sd_beam_select_args_t"),
    ("SdBeamReorderArgs", "sd_beam_reorder_args_t")])
def test_struct_layouts_match_the_header(cls, name, tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    A = getattr(_tree(), cls)
    fields = [f[0] for f in A._fields_]
    src = tmp_path / "t.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"sd_tree.h\"\nint main(void){"
                   f"printf(\"%zu\", sizeof({name}));" +
                   "".join(f'printf(" %zu", offsetof({name}, {f.rstrip("_")}));' for f in fields) +
                   "return 0;}\n")
    exe = tmp_path / "t"
    subprocess.run([gcc, "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(A)] + [getattr(A, f).offset for f in fields]


@pytest.mark.parametrize("cls,packed", [
    ("SdTreeAttentionArgs", "_TREE_ATTENTION"), ("SdTreeVerifyArgs", "_TREE_VERIFY"),
    ("SdCacheCommitArgs", "_CACHE_COMMIT"), ("SdCacheEvictArgs", "_CACHE_EVICT"),
    ("SdBeamSelectArgs", "_BEAM_SELECT"), ("SdBeamReorderArgs", "_BEAM_REORDER")])
def test_packed_arguments_are_the_structs(cls, packed):
    """The binding packs argument structs as bytes: every value lands in its
    field."""
    T = _tree()
    A, S = getattr(T, cls), getattr(T, packed)
    fields = []
    for name, kind in A._fields_:
        if kind is T.SdKvCache:
            fields += [("cache", f[0]) for f in kind._fields_]
        else:
            fields.append((None, name))
    assert S.size == ctypes.sizeof(A)
    a = A.from_buffer_copy(S.pack(*range(1, len(fields) + 1)))
    got = [getattr(a.cache if outer else a, name) for outer, name in fields]
    assert got == list(range(1, len(fields) + 1))


def _cache():
    return _tree().SdKvCache(0x100000, 0x200000, 4 * 16 * 128, 16 * 128, 128, 0x300000, 10, 0x310000,
                             1, 2, 4, 128, 16, 20, 10)


CACHE_DEFECTS = [
    ("k", None, -1), ("v", None, -1), ("k", 0x100008, -1), ("page_table", None, -1),
    ("context_lens", None, -1), ("dtype", 0, -1), ("dtype", 5, -1), ("B", 0, -1), ("H_kv", 0, -1),
    ("D", 0, -1), ("D", 80, -4), ("page_size", 0, -1), ("page_size", 24, -4), ("page_size", 2048, -4),
    ("num_pages", 0, -1), ("max_pages", 0, -1), ("ld_table", 9, -1), ("page_stride", -8, -1),
    ("head_stride", 12, -1), ("slot_stride", 120, -1), ("slot_stride", 132, -1), ("B", 70000, -4),
]


def _attention():
    return _tree().SdTreeAttentionArgs(_cache(), 0x400000, 0x410000, 0x420000, 1024, 128, 512, 128, 512, 128,
                                       0x430000, None, None, 6, 3, 8, 0.5)


def _commit():
    return _tree().SdCacheCommitArgs(_cache(), 0x410000, 0x420000, 512, 128, 512, 128, 0x430000, 0x440000, 3,
                                     0x450000, 6, 3, 0x400000, 1024, 128, 0x460000, 8, 0.5, 1.0, 0x470000,
                                     0x470000, 160, 0x480000, 0x490000)


def _evict():
    return _tree().SdCacheEvictArgs(_cache(), 0x400000, 0x400000, 0x410000, 0x410000, 160, 0x420000, 64, 8, 4)


def _verify():
    return _tree().SdTreeVerifyArgs(0x100000, 1008, 0x200000, 0x210000, 0x220000, 1, 2, 6, 1000, 3, 0)


def _select():
    return _tree().SdBeamSelectArgs(0x100000, 1008, 0x200000, None, 1, 2, 4, 1000, 4, 2)


def _reorder():
    return _tree().SdBeamReorderArgs(0x100000, 0x100000, 4096, 2048, 512, 256, 4096, 2048, 512, 256, 0x200000, None,
                                     32, 2, 2, 4, 4, 2, 8)


def _call(sdv, kind, a, ws=P(0xA00000), n=1 << 40, out=OUT):
    lib, r = sdv.lib, ctypes.byref(a)
    if kind == "attention":
        return lib.sd_tree_attention(r, ws, n, out, None, None, None)
    if kind == "commit":
        return lib.sd_cache_commit(r, out, None, None)
    if kind == "evict":
        return lib.sd_cache_evict(r, ws, n, out, None, None)
    if kind == "verify":
        return lib.sd_tree_verify_greedy(r, ws, n, out, OUT, OUT, None, None)
    if kind == "select":
        return lib.sd_beam_select(r, ws, n, out, OUT, OUT, None, None, None)
    return lib.sd_beam_reorder(r, None)


MAKE = dict(attention=_attention, commit=_commit, evict=_evict, verify=_verify, select=_select, reorder=_reorder)


@pytest.mark.parametrize("kind", ["attention", "commit", "evict"])
@pytest.mark.parametrize("field,value,code", CACHE_DEFECTS)
def test_cache_defects_are_refused(sdv, kind, field, value, code):
    a = MAKE[kind]()
    setattr(a.cache, field, value)
    if kind == "evict" and field in ("max_pages", "page_size") and code == -4:
        a.ld_mass = 1 << 20
    assert _call(sdv, kind, a) == code


def test_a_table_beyond_31_bits_of_slots_is_refused(sdv):
    a = _attention()
    a.cache.page_size, a.cache.max_pages, a.cache.ld_table = 1024, 1 << 21, 1 << 21
    assert _call(sdv, "attention", a) == -4


@pytest.mark.parametrize("kind,field,value,code", [
    ("attention", "q", None, -1), ("attention", "k_new", 0x410004, -1), ("attention", "v_new", None, -1),
    ("attention", "q_node", 1020, -1), ("attention", "k_head", -128, -1), ("attention", "node_offsets", None, -1),
    ("attention", "N", 0, -1), ("attention", "max_nodes", 0, -1), ("attention", "max_nodes", 65, -4),
    ("attention", "H_q", 6, -1), ("attention", "H_q", 0, -1), ("attention", "H_q", 4 * 33, -4),
    ("attention", "scale", float("nan"), -1), ("attention", "scale", float("inf"), -1),
    ("commit", "k_new", None, -1), ("commit", "v_node", 4, -1), ("commit", "path", None, -1),
    ("commit", "path_lens", None, -1), ("commit", "ld_path", 2, -1), ("commit", "max_nodes", 65, -4),
    ("commit", "q", None, -1), ("commit", "lse", None, -1), ("commit", "H_q", 7, -1),
    ("commit", "scale", float("inf"), -1), ("commit", "decay", float("nan"), -1),
    ("commit", "mass_in", None, -1), ("commit", "ld_mass", 0, -1), ("commit", "seen", None, -1),
    ("commit", "positions", None, -1), ("commit", "N", 0, -1),
    ("evict", "mass_in", None, -1), ("evict", "mass_out", None, -1), ("evict", "positions_in", None, -1),
    ("evict", "positions_out", None, -1), ("evict", "seen", None, -1), ("evict", "budget", 0, -1),
    ("evict", "recent", -1, -1), ("evict", "sinks", -1, -1), ("evict", "recent", 61, -1),
    ("evict", "ld_mass", 159, -1),
    ("verify", "logits", None, -1), ("verify", "logits", 0x100008, -1), ("verify", "tokens", None, -1),
    ("verify", "parents", None, -1), ("verify", "node_offsets", None, -1), ("verify", "ld", 999, -1),
    ("verify", "ld", 1004, -1), ("verify", "dtype", 2, -1), ("verify", "B", 0, -1), ("verify", "N", 0, -1),
    ("verify", "V", 0, -1), ("verify", "max_nodes", 0, -1), ("verify", "max_nodes", 65, -4),
    ("verify", "flags", 2, -1),
    ("select", "logits", None, -1), ("select", "logits", 0x100002, -1), ("select", "scores", None, -1),
    ("select", "ld", 999, -1), ("select", "dtype", 3, -1), ("select", "B", 0, -1), ("select", "W", 0, -1),
    ("select", "W", 65, -4), ("select", "n_out", 0, -1), ("select", "n_out", 65, -4), ("select", "V", 0, -1),
    ("reorder", "in_", None, -1), ("reorder", "out", None, -1), ("reorder", "parents", None, -1),
    ("reorder", "in_", 0x100004, -1), ("reorder", "in_beam", 520, -1), ("reorder", "out_seg", -16, -1),
    ("reorder", "unit_bytes", 24, -1), ("reorder", "unit_bytes", 0, -1), ("reorder", "layers", 0, -1),
    ("reorder", "W_in", 0, -1), ("reorder", "W_out", 5, -1), ("reorder", "out_request", 4096, -1),
    ("reorder", "max_units", 0, -1),
])
def test_bad_arguments_are_refused(sdv, kind, field, value, code):
    a = MAKE[kind]()
    setattr(a, field, value)
    assert _call(sdv, kind, a) == code


def test_reorder_sizes_beyond_the_limits_are_refused(sdv):
    a = _reorder()
    a.W_in = a.W_out = 65
    assert _call(sdv, "reorder", a) == -4


@pytest.mark.parametrize("kind,sizes,code", [
    ("select", dict(B=1 << 18, W=64), -4), ("select", dict(B=(1 << 18) - 1, W=64), 0), ("select", dict(B=1 << 20, W=16), -4),
    ("select", dict(B=1 << 20, W=15), 0), ("select", dict(B=(1 << 20) + 1, W=1), -4),
    ("verify", dict(N=1 << 24, V=3, ld=8), -4), ("verify", dict(N=(1 << 24) - 1, V=3, ld=8), 0),
    ("verify", dict(N=1 << 24, V=1000), -4)])
def test_grids_beyond_the_hardware_are_refused(sdv, kind, sizes, code):
    """A grid dimension holds less than 2^32 threads: what would pass that is
    refused with the sizes, not at the launch."""
    a = MAKE[kind]()
    for k, v in sizes.items():
        setattr(a, k, v)
    n = ctypes.c_size_t()
    f = sdv.lib.sd_beam_select_workspace_bytes if kind == "select" else sdv.lib.sd_tree_verify_workspace_bytes
    assert f(ctypes.byref(a), ctypes.byref(n)) == code
    if code:
        assert _call(sdv, kind, a) == code


def test_short_tables_of_very_many_heads_are_split(sdv):
    """One workgroup per (request, KV head, row tile) needs no workspace; where
    these pass a grid dimension the work is cut into runs instead."""
    n = ctypes.c_size_t()
    for heads, whole in ((8, True), (255, True), (2048, False)):
        a = _attention()
        a.cache.B, a.cache.H_kv, a.H_q, a.cache.page_size, a.cache.max_pages = 65535, heads, heads, 16, 1
        assert sdv.lib.sd_tree_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
        assert (n.value == 0) == whole, heads


def test_evictions_of_more_heads_than_31_bits_count_are_refused(sdv):
    n = ctypes.c_size_t()
    for heads, code in ((32768, 0), (32769, -4), (65535, -4)):
        a = _evict()
        a.cache.B, a.cache.H_kv, a.cache.page_size, a.cache.max_pages = 65535, heads, 1, 1
        a.budget, a.recent, a.sinks = 1, 0, 0
        assert sdv.lib.sd_cache_evict_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == code, heads
        if code:
            assert _call(sdv, "evict", a) == code


@pytest.mark.parametrize("kind", ["verify", "select", "evict"])
def test_missing_outputs_and_small_workspaces_are_refused(sdv, kind):
    assert _call(sdv, kind, MAKE[kind](), out=None) == -1
    assert _call(sdv, kind, MAKE[kind](), ws=None) == sdv.SD_EWORKSPACE
    assert _call(sdv, kind, MAKE[kind](), n=7) == sdv.SD_EWORKSPACE


def test_outputs_that_may_not_be_inputs_are_refused(sdv):
    assert _call(sdv, "attention", _attention(), out=None) == -1
    assert _call(sdv, "attention", _attention(), out=P(0x900008)) == -1
    for kind in ("commit", "evict"):
        assert _call(sdv, kind, MAKE[kind](), out=None) == -1
        assert _call(sdv, kind, MAKE[kind](), out=P(0x310000)) == -1      # context_lens itself
    assert _call(sdv, "select", _select(), out=P(0x200000)) == -1         # the scores


def test_rows_of_logits_however_their_axes_came_about():
    """The row stride of logits, whatever an axis of one says of itself."""
    import torch
    rows = lambda t: _tree()._logits(t, "logits")[1]  # noqa: E731
    x = torch.zeros(6, 1008)
    assert rows(x) == 1008 and rows(x[:, :1000]) == 1008
    y = x[:, :1000]
    assert rows(y.unsqueeze(1)) == rows(y.unsqueeze(0)) == rows(y.reshape(6, 1, 1000).contiguous()) + 8 == 1008
    assert rows(y.view(2, 3, 1000)) == 1008
    z = torch.zeros(4, 7, 1008)
    assert rows(z[:, -1:]) == rows(z[:, -1:, :1000]) == 7 * 1008       # the last position of each request
    assert rows(z[:, -1]) == 7 * 1008
    assert rows(z[:1, 2:5]) == 1008 and rows(z[3:, 6:]) == 1008
    for bad in (z[:, :3], z.transpose(0, 1), x[:, ::2]):
        with pytest.raises(ValueError):
            rows(bad)


@pytest.mark.parametrize("kind,inputs", [
    ("attention", ("k_new", "v_new")), ("verify", ("tokens", "parents", "node_offsets")),
    ("commit", ("node_offsets", "path", "path_lens", "seen"))])
def test_an_output_that_is_an_input_is_refused(sdv, kind, inputs):
    """Other workgroups still read it while its first results are written."""
    for field in inputs:
        a = MAKE[kind]()
        assert _call(sdv, kind, a, out=P(getattr(a, field))) == -1, field
    if kind == "attention":
        for field in ("k", "v"):
            a = MAKE[kind]()
            assert _call(sdv, kind, a, out=P(getattr(a.cache, field))) == -1, field
        for field, value in (("q_node", 1032), ("q_head", 136), ("q_head", 0)):      # rows of others' queries
            a = MAKE[kind]()
            setattr(a, field, value)
            assert _call(sdv, kind, a, out=P(a.q)) == -1, field
    if kind == "verify":
        a = MAKE[kind]()
        for outs in ((OUT, P(a.tokens), P(0x910000)), (OUT, P(0x910000), P(a.parents))):
            assert sdv.lib.sd_tree_verify_greedy(ctypes.byref(a), P(0xA00000), 1 << 40, *outs, None, None) == -1


def test_rows_that_share_memory_are_not_written(sdv):
    """Expanded caches and states: the rows of one would be written over another's."""
    for field in ("head_stride", "page_stride"):
        a = _evict()
        setattr(a.cache, field, 0)
        assert _call(sdv, "evict", a) == -1, field
    for field in ("layer", "request", "beam", "seg"):
        a = _reorder()
        setattr(a, "in_" + field, 0)
        setattr(a, "out_" + field, 0)
        assert _call(sdv, "reorder", a) == -1, field


def test_the_binding_refuses_what_it_can_see(sdv):
    """Tensors that are not on the current GPU, wrong types, shapes and
    strides raise before any call (CPU tensors here)."""
    import torch
    k = torch.zeros(20, 4, 16, 64, dtype=torch.bfloat16)
    table, lens, off = torch.zeros(2, 10, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), \
        torch.tensor([0, 3, 6], dtype=torch.int32)
    q, kn = torch.zeros(6, 8, 64, dtype=torch.bfloat16), torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    make = lambda **o: sdv.make_tree_attention_args(**{**dict(  # noqa: E731
        q=q, k_new=kn, v_new=kn, k_cache=k, v_cache=k, page_table=table, context_lens=lens,
        node_offsets=off, max_nodes=3), **o})
    a = make()
    assert (a.cache.B, a.cache.H_kv, a.cache.D, a.cache.page_size, a.cache.num_pages, a.H_q, a.N) == \
        (2, 4, 64, 16, 20, 8, 6)
    assert a.scale == 0.125
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(k_new=kn[:5]), dict(v_new=kn.transpose(1, 2)),
                dict(v_cache=k[:, :, :8]), dict(v_cache=k.half()), dict(page_table=table.long()),
                dict(page_table=table.t()), dict(context_lens=lens.long()), dict(context_lens=lens[:1]),
                dict(node_offsets=off[:2]), dict(parents=off), dict(tree_mask=torch.zeros(6, dtype=torch.int32)),
                dict(k_cache=k.transpose(2, 3), v_cache=k.transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            make(**bad)
    with pytest.raises(TypeError):
        make(k_cache=k.float(), v_cache=k.float())
    with pytest.raises(ValueError):
        sdv.tree_attention(q, kn, kn, k, k, table, lens, off, 3)
    with pytest.raises(ValueError):
        sdv.beam_select(torch.zeros(2, 4, 100), torch.zeros(2, 4), 4)
    with pytest.raises(ValueError):
        sdv.cache_commit(kn, kn, k, k, table, lens, off, 3, torch.zeros(2, 3, dtype=torch.int32), lens, lens,
                         mass_out=torch.zeros(2, 4, 160))
