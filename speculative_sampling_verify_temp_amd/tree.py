"""Tree drafting on MI355X: Python binding of include/sd_tree.h.

Functions mirror the C entry points; like the rest of the package they only
check and marshal arguments.
    tree_attention(...)      -> sd_tree_attention
    tree_verify_greedy(...)  -> sd_tree_verify_greedy
    cache_commit(...)        -> sd_cache_commit
    cache_evict(...)         -> sd_cache_evict
    beam_select(...)         -> sd_beam_select
    beam_reorder(...)        -> sd_beam_reorder

The cache is a pair of tensors [pages][H_kv][page_size][D] (any strides with
contiguous rows, the same for both), with a page table [B][max_pages] and the
slots in use [B], both int32.  With `stream` given, outputs and workspaces that
are not passed in are allocated on that stream too, as in a
`with torch.cuda.stream(stream)` block.
"""
import ctypes
import struct

import torch

from . import SD_BF16, SD_F32, SD_OK, SD_ST_INVALID_MASK, SdVerifyError, lib

SD_F16 = 2
SD_MAX_NODES = 64
SD_MAX_BEAMS = 64
SD_MAX_PAGE_SIZE = 1024
SD_MAX_GROUP = 32
SD_ST_BAD_LEN, SD_ST_BAD_NODES, SD_ST_BAD_PAGE = 1 << 8, 1 << 9, 1 << 10
SD_ST_BAD_TREE, SD_ST_BAD_PATH, SD_ST_UNFINISHED = 1 << 11, 1 << 12, 1 << 13
SD_ST_TREE_INVALID_MASK = (SD_ST_INVALID_MASK | SD_ST_BAD_LEN | SD_ST_BAD_NODES | SD_ST_BAD_PATH |
                           SD_ST_UNFINISHED)

_P, _I32, _I64, _U32, _F, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                 ctypes.c_float, ctypes.c_size_t)


class SdKvCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("page_stride", _I64), ("head_stride", _I64),
                ("slot_stride", _I64), ("page_table", _P), ("ld_table", _I64),
                ("context_lens", _P), ("dtype", _I32), ("B", _I32), ("H_kv", _I32), ("D", _I32),
                ("page_size", _I32), ("num_pages", _I32), ("max_pages", _I32)]


class SdTreeAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", SdKvCache), ("q", _P), ("k_new", _P), ("v_new", _P),
                ("q_node", _I64), ("q_head", _I64), ("k_node", _I64), ("k_head", _I64),
                ("v_node", _I64), ("v_head", _I64), ("node_offsets", _P), ("parents", _P),
                ("tree_mask", _P), ("N", _I32), ("max_nodes", _I32), ("H_q", _I32), ("scale", _F)]


class SdTreeVerifyArgs(ctypes.Structure):
    _fields_ = [("logits", _P), ("ld", _I64), ("tokens", _P), ("parents", _P),
                ("node_offsets", _P), ("dtype", _I32), ("B", _I32), ("N", _I32), ("V", _I32),
                ("max_nodes", _I32), ("flags", _U32)]


class SdCacheCommitArgs(ctypes.Structure):
    _fields_ = [("cache", SdKvCache), ("k_new", _P), ("v_new", _P), ("k_node", _I64),
                ("k_head", _I64), ("v_node", _I64), ("v_head", _I64), ("node_offsets", _P),
                ("path", _P), ("ld_path", _I64), ("path_lens", _P), ("N", _I32),
                ("max_nodes", _I32), ("q", _P), ("q_node", _I64), ("q_head", _I64), ("lse", _P),
                ("H_q", _I32), ("scale", _F), ("decay", _F), ("mass_in", _P), ("mass_out", _P),
                ("ld_mass", _I64), ("positions", _P), ("seen", _P)]


class SdCacheEvictArgs(ctypes.Structure):
    _fields_ = [("cache", SdKvCache), ("mass_in", _P), ("mass_out", _P), ("positions_in", _P),
                ("positions_out", _P), ("ld_mass", _I64), ("seen", _P), ("budget", _I32),
                ("recent", _I32), ("sinks", _I32)]


class SdBeamSelectArgs(ctypes.Structure):
    _fields_ = [("logits", _P), ("ld", _I64), ("scores", _P), ("ended", _P), ("dtype", _I32),
                ("B", _I32), ("W", _I32), ("V", _I32), ("n_out", _I32), ("eos_id", _I32)]


class SdBeamReorderArgs(ctypes.Structure):
    _fields_ = [("in_", _P), ("out", _P), ("in_layer", _I64), ("in_request", _I64),
                ("in_beam", _I64), ("in_seg", _I64), ("out_layer", _I64), ("out_request", _I64),
                ("out_beam", _I64), ("out_seg", _I64), ("parents", _P), ("lengths", _P),
                ("unit_bytes", _I64), ("layers", _I32), ("B", _I32), ("W_in", _I32),
                ("W_out", _I32), ("segs", _I32), ("max_units", _I32)]


# The argument structs as bytes: packing them costs a call a tenth of what
# filling a ctypes.Structure does.  Native alignment is the C compiler's; 0q
# pads the end to that of an 8-byte field.
_CACHE = "QQqqqQqQiiiiiii"
_TREE_ATTENTION = struct.Struct(_CACHE + "QQQqqqqqqQQQiiif0q")
_TREE_VERIFY = struct.Struct("QqQQQiiiiiI0q")
_CACHE_COMMIT = struct.Struct(_CACHE + "QQqqqqQQqQiiQqqQiffQQqQQ0q")
_CACHE_EVICT = struct.Struct(_CACHE + "QQQQqQiii0q")
_BEAM_SELECT = struct.Struct("QqQQiiiiii0q")
_BEAM_REORDER = struct.Struct("QQqqqqqqqqQQqiiiiii0q")


def _entry(name, *rest):
    f = lib[name]
    f.argtypes = [ctypes.c_char_p, *rest]
    f.restype = ctypes.c_int
    return f


def _size_entry(name):
    f = _entry(name, ctypes.POINTER(_SZ))

    def size(a):
        n = _SZ()
        rc = f(a, n)
        if rc != SD_OK:
            raise SdVerifyError(rc, name)
        return n.value
    return size


_tree_attention = _entry("sd_tree_attention", _P, _SZ, _P, _P, _P, _P)
_tree_verify = _entry("sd_tree_verify_greedy", _P, _SZ, _P, _P, _P, _P, _P)
_cache_commit = _entry("sd_cache_commit", _P, _P, _P)
_cache_evict = _entry("sd_cache_evict", _P, _SZ, _P, _P, _P)
_beam_select = _entry("sd_beam_select", _P, _SZ, _P, _P, _P, _P, _P, _P)
_beam_reorder = _entry("sd_beam_reorder", _P)
_tree_attention_bytes = _size_entry("sd_tree_attention_workspace_bytes")
_tree_verify_bytes = _size_entry("sd_tree_verify_workspace_bytes")
_cache_evict_bytes = _size_entry("sd_cache_evict_workspace_bytes")
_beam_select_bytes = _size_entry("sd_beam_select_workspace_bytes")


# ---- argument checks ----

def _here(first, *rest):
    """All tensors on the current GPU, which is where the call's work goes."""
    dev = first.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must be on the current GPU")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call must be on the same GPU")


def _plain(t, dtype, name, shape):
    """Pointer of a contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
    return t.data_ptr()


def _output(t, dtype, name, shape, like):
    """The given output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _plain(t, dtype, name, shape)
    return t


def _status(status, B):
    return None if status is None else _plain(status, torch.int32, "status", (B,))


def _on(stream, f, args):
    """f with these keyword arguments, and what it allocates, on the stream."""
    with torch.cuda.stream(stream):
        return f(**{**args, "stream": None})


def _stream():
    """The current stream's handle, without building a Stream object, which
    takes longer than the rest of the argument checks."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream().cuda_stream
    return raw(torch.cuda.current_device())


def _rows(t, name, like, N, H, D):
    """Packed node rows [N][H][D] of the cache's element type: (pointer, strides)."""
    if t.dtype is not like.dtype or t.shape != (N, H, D):
        raise ValueError(f"{name} must be {like.dtype} of shape {[N, H, D]}")
    node, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), node, head


def _cache(k, v, table, lens):
    """The fields of sd_kv_cache_t."""
    if k.dtype is torch.bfloat16:
        code = SD_BF16
    elif k.dtype is torch.float16:
        code = SD_F16
    else:
        raise TypeError(f"the cache must be bfloat16 or float16 (got {k.dtype})")
    strides = k.stride()
    if len(strides) != 4 or k.shape != v.shape or v.dtype is not k.dtype or strides != v.stride():
        raise ValueError("k_cache and v_cache must be [pages][H_kv][page_size][D] with the same "
                         "type, shape and strides")
    pages, H, page, D = k.shape
    ps, hs, ss, es = strides
    if es != 1 and D > 1:
        raise ValueError("the elements of a cache row must be contiguous")
    if table.dtype is not torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("page_table must be int32 [B][max_pages] with contiguous rows")
    B, cols = table.shape
    return (k.data_ptr(), v.data_ptr(), ps, hs, ss, table.data_ptr(),
            table.stride(0) if B > 1 else max(cols, table.stride(0)),
            _plain(lens, torch.int32, "context_lens", (B,)), code, B, H, D, page, pages, cols)


def _workspace(size, a, given, like):
    """The given workspace or a new one, if one is needed: (tensor, pointer, bytes)."""
    if given is not None:
        if not given.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        _here(like, given)
        return given, given.data_ptr(), given.numel() * given.element_size()
    n = size(a)
    if n == 0:
        return None, None, 0
    ws = torch.empty(n, dtype=torch.uint8, device=like.device)
    return ws, ws.data_ptr(), n


def _done(rc, name):
    if rc != SD_OK:
        raise SdVerifyError(rc, name)


# ---- attention of a drafted tree ----

def _attention_args(q, k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets,
                    max_nodes, parents, tree_mask, scale):
    c = _cache(k_cache, v_cache, page_table, context_lens)
    B, H = c[9:11]
    N, Hq, D = q.shape
    if c[11] != D:
        raise ValueError("queries and cache must have the same head size")
    qp, qn, qh = _rows(q, "q", k_cache, N, Hq, D)
    kp, kn, kh = _rows(k_new, "k_new", k_cache, N, H, D)
    vp, vn, vh = _rows(v_new, "v_new", k_cache, N, H, D)
    return _TREE_ATTENTION.pack(
        *c, qp, kp, vp, qn, qh, kn, kh, vn, vh,
        _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)),
        0 if parents is None else _plain(parents, torch.int32, "parents", (N,)),
        0 if tree_mask is None else _plain(tree_mask, torch.int64, "tree_mask", (N,)), N, max_nodes,
        Hq, D ** -0.5 if scale is None else scale)


def make_tree_attention_args(q, k_new, v_new, k_cache, v_cache, page_table, context_lens,
                             node_offsets, max_nodes, parents=None, tree_mask=None, scale=None):
    """sd_tree_attention_args_t from tensors: q [N][H_q][D], k_new and v_new
    [N][H_kv][D], node_offsets [B + 1], parents [N] int32 or tree_mask [N]
    int64 (bit j: node j of the request is seen) or neither (a chain); scale
    defaults to 1 / sqrt(D)."""
    return SdTreeAttentionArgs.from_buffer_copy(_attention_args(
        q, k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets, max_nodes,
        parents, tree_mask, scale))


def tree_attention_workspace_bytes(args):
    """Bytes of workspace tree_attention needs for a filled argument struct."""
    return _tree_attention_bytes(bytes(args))


def tree_attention(q, k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets,
                   max_nodes, parents=None, tree_mask=None, scale=None, want_lse=False, out=None,
                   lse=None, status=None, workspace=None, stream=None):
    """Attention of the packed nodes of B drafted trees over the paged cache
    and each other; returns (out [N][H_q][D], lse [N][H_q] or None).

    out, lse: optional preallocated contiguous outputs; status: optional [B]
    int32 tensor for the per-request bits."""
    if stream is not None:
        return _on(stream, tree_attention, locals())
    _here(q, k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets, parents,
          tree_mask, out, lse, status)
    a = _attention_args(q, k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets,
                        max_nodes, parents, tree_mask, scale)
    shape = q.shape
    out = _output(out, q.dtype, "out", shape, q)
    if want_lse or lse is not None:
        lse = _output(lse, torch.float32, "lse", shape[:2], q)
    ws, wp, n = _workspace(_tree_attention_bytes, a, workspace, q)
    rc = _tree_attention(a, wp, n, out.data_ptr(), None if lse is None else lse.data_ptr(),
                         _status(status, page_table.shape[0]), _stream())
    _done(rc, "sd_tree_attention")
    return out, lse


# ---- greedy verify of a tree ----

def _logits(t, name):
    """Rows with unit element stride: (pointer, row stride, type code)."""
    if t.dtype == torch.float32:
        code = SD_F32
    elif t.dtype == torch.bfloat16:
        code = SD_BF16
    else:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    V = t.shape[-1]
    if V > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the logits of a row must be contiguous")
    ld = t.stride(-2)
    if t.dim() == 3 and t.shape[0] > 1:
        if t.shape[1] == 1:      # the stride of an axis of one says nothing
            ld = t.stride(0)
        elif t.stride(0) != t.shape[1] * ld:
            raise ValueError(f"{name} must have its rows back to back")
    rows = t.numel() // max(1, V)
    return t.data_ptr(), (ld if rows > 1 else max(ld, V)), code


def tree_verify_greedy(logits, tokens, parents, node_offsets, max_nodes, flags=0, status=None,
                       out=None, workspace=None, stream=None):
    """Greedy verify of B drafted trees: logits [N][V], tokens and parents
    [N], node_offsets [B + 1].  Returns (accepted [B], path [B][max_nodes],
    tokens [B][max_nodes]).

    out: optional dict of preallocated outputs (accepted, path, tokens)."""
    if stream is not None:
        return _on(stream, tree_verify_greedy, locals())
    if logits.dim() != 2:
        raise ValueError("logits must be [N][V]")
    N, V = logits.shape
    B = node_offsets.numel() - 1
    o = out or {}
    acc, path, tok = o.get("accepted"), o.get("path"), o.get("tokens")
    _here(logits, tokens, parents, node_offsets, status, acc, path, tok)
    ptr, ld, code = _logits(logits, "logits")
    a = _TREE_VERIFY.pack(ptr, ld, _plain(tokens, torch.int32, "tokens", (N,)),
                          _plain(parents, torch.int32, "parents", (N,)),
                          _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)), code, B, N, V,
                          max_nodes, flags)
    ws, wp, n = _workspace(_tree_verify_bytes, a, workspace, logits)

    acc = _output(acc, torch.int32, "accepted", (B,), logits)
    path = _output(path, torch.int32, "path", (B, max_nodes), logits)
    tok = _output(tok, torch.int32, "tokens", (B, max_nodes), logits)
    rc = _tree_verify(a, wp, n, acc.data_ptr(), path.data_ptr(), tok.data_ptr(),
                      _status(status, B), _stream())
    _done(rc, "sd_tree_verify_greedy")
    return acc, path, tok


# ---- append to and eviction from the cache ----

def cache_commit(k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets, max_nodes,
                 path, path_lens, out_context, q=None, lse=None, scale=None, mass_in=None,
                 mass_out=None, decay=1.0, positions=None, seen=None, status=None, stream=None):
    """Append the nodes path[b][: path_lens[b]] to the cache; out_context [B]
    receives the new lengths.

    With mass_out [B][H_kv][L] the attention weight of these rows is
    accumulated from q, lse (of tree_attention) and mass_in (mass_out's own
    values when None); positions [B][H_kv][L] and seen [B] record where the
    appended tokens stand."""
    if stream is not None:
        return _on(stream, cache_commit, locals())
    if mass_out is not None and (q is None or lse is None):
        raise ValueError("weights need q and lse")
    if mass_out is not None and mass_in is None:
        mass_in = mass_out
    _here(k_new, v_new, k_cache, v_cache, page_table, context_lens, node_offsets, path, path_lens,
          out_context, q, lse, mass_in, mass_out, positions, seen, status)
    c = _cache(k_cache, v_cache, page_table, context_lens)
    N = k_new.shape[0]
    B, H, D = c[9:12]
    kp, kn, kh = _rows(k_new, "k_new", k_cache, N, H, D)
    vp, vn, vh = _rows(v_new, "v_new", k_cache, N, H, D)
    L = 0
    weights = (0, 0, 0, 0, 0, 0.0, 0.0, 0, 0)
    if mass_out is not None:
        L, Hq = mass_out.shape[-1], q.shape[1]
        weights = (*_rows(q, "q", k_cache, N, Hq, D), _plain(lse, torch.float32, "lse", (N, Hq)), Hq,
                   D ** -0.5 if scale is None else scale, decay,
                   _plain(mass_in, torch.float32, "mass_in", (B, H, L)),
                   _plain(mass_out, torch.float32, "mass_out", (B, H, L)))
    places = (0, 0)
    if positions is not None:
        if seen is None:
            raise ValueError("positions need seen")
        L = L or positions.shape[-1]
        places = (_plain(positions, torch.int32, "positions", (B, H, L)),
                  _plain(seen, torch.int32, "seen", (B,)))
    cols = path.shape[-1]
    a = _CACHE_COMMIT.pack(*c, kp, vp, kn, kh, vn, vh,
                           _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)),
                           _plain(path, torch.int32, "path", (B, cols)), cols,
                           _plain(path_lens, torch.int32, "path_lens", (B,)), N, max_nodes,
                           *weights, L, *places)
    rc = _cache_commit(a, _plain(out_context, torch.int32, "out_context", (B,)),
                       _status(status, B), _stream())
    _done(rc, "sd_cache_commit")
    return out_context


def cache_evict(k_cache, v_cache, page_table, context_lens, mass_in, mass_out, positions_in,
                positions_out, seen, out_context, budget, recent=0, sinks=0, status=None,
                workspace=None, stream=None):
    """Cut every request's cache to its `budget` slots of the largest mass,
    keeping positions below `sinks` and the last `recent` ones; out_context
    [B] receives the new lengths.  mass_* [B][H_kv][L] float32 and positions_*
    [B][H_kv][L] int32 (or None, None, with recent = sinks = 0); outputs may
    be the inputs."""
    if stream is not None:
        return _on(stream, cache_evict, locals())
    _here(k_cache, v_cache, page_table, context_lens, mass_in, mass_out, positions_in,
          positions_out, seen, out_context, status)
    c = _cache(k_cache, v_cache, page_table, context_lens)
    B, H = c[9:11]
    L = mass_in.shape[-1]
    if (positions_in is None) != (positions_out is None):
        raise ValueError("positions_in and positions_out go together")
    places = (0, 0)
    if positions_in is not None:
        places = (_plain(positions_in, torch.int32, "positions_in", (B, H, L)),
                  _plain(positions_out, torch.int32, "positions_out", (B, H, L)))
    a = _CACHE_EVICT.pack(*c, _plain(mass_in, torch.float32, "mass_in", (B, H, L)),
                          _plain(mass_out, torch.float32, "mass_out", (B, H, L)), *places, L,
                          0 if seen is None else _plain(seen, torch.int32, "seen", (B,)), budget,
                          recent, sinks)
    ws, wp, n = _workspace(_cache_evict_bytes, a, workspace, k_cache)
    rc = _cache_evict(a, wp, n, _plain(out_context, torch.int32, "out_context", (B,)),
                      _status(status, B), _stream())
    _done(rc, "sd_cache_evict")
    return out_context


# ---- a beam step ----

def beam_select(logits, scores, n_out, ended=None, eos_id=-1, out_ended=None, status=None,
                out=None, workspace=None, stream=None):
    """The n_out best continuations over the beams of each request: logits
    [B][W][V] (float32 or bfloat16), scores [B][W] float32, ended [B][W] uint8
    or None.  Returns (scores [B][n_out], parents [B][n_out], tokens
    [B][n_out]); out_ended: optional [B][n_out] uint8 output.

    out: optional dict of preallocated outputs (scores, parents, tokens)."""
    if stream is not None:
        return _on(stream, beam_select, locals())
    if logits.dim() != 3:
        raise ValueError("logits must be [B][W][V]")
    B, W, V = logits.shape
    o = out or {}
    sc, par, tok = o.get("scores"), o.get("parents"), o.get("tokens")
    _here(logits, scores, ended, out_ended, status, sc, par, tok)
    ptr, ld, code = _logits(logits, "logits")
    a = _BEAM_SELECT.pack(ptr, ld, _plain(scores, torch.float32, "scores", (B, W)),
                          0 if ended is None else _plain(ended, torch.uint8, "ended", (B, W)), code,
                          B, W, V, n_out, eos_id)
    oe = None if out_ended is None else _plain(out_ended, torch.uint8, "out_ended", (B, n_out))
    ws, wp, n = _workspace(_beam_select_bytes, a, workspace, logits)

    sc = _output(sc, torch.float32, "scores", (B, n_out), logits)
    par = _output(par, torch.int32, "parents", (B, n_out), logits)
    tok = _output(tok, torch.int32, "tokens", (B, n_out), logits)
    rc = _beam_select(a, wp, n, sc.data_ptr(), par.data_ptr(), tok.data_ptr(), oe,
                      _status(status, B), _stream())
    _done(rc, "sd_beam_select")
    return sc, par, tok


def beam_reorder(state, parents, lengths=None, out=None, stream=None):
    """Move beam states to the beams that continue them: state
    [layers][B][W][segs][units][..] (the trailing part of a unit contiguous,
    a multiple of 16 bytes), parents [B][W_out] int32, lengths [B] int32 units
    in use or None.  In place without `out`; returns the tensor written."""
    if stream is not None:
        return _on(stream, beam_reorder, locals())
    if state.dim() < 5:
        raise ValueError("state must be [layers][B][W][segs][units][..]")
    dst = state if out is None else out
    _here(state, dst, parents, lengths)
    shape = state.shape
    layers, B, W, segs, units = shape[:5]
    if parents.dim() != 2 or parents.shape[0] != B:
        raise ValueError("parents must be [B][W_out]")
    W_out = parents.shape[1]
    if dst.dtype is not state.dtype or dst.shape != (layers, B, W_out, segs, *shape[4:]):
        raise ValueError("out must have state's type and shape, with W_out beams")
    es = state.element_size()
    unit = es
    for n in shape[5:]:
        unit *= n
    strides = []
    for t in (state, dst):
        s = t.stride()
        want = es
        for n, step in zip(shape[:3:-1], s[:3:-1]):
            if n > 1 and step * es != want:      # (the stride of an axis of one says nothing)
                raise ValueError("the units of a state row must be contiguous")
            want *= n
        strides += [step * es if n > 1 else 0 for n, step in zip(t.shape, s[:4])]
    a = _BEAM_REORDER.pack(state.data_ptr(), dst.data_ptr(), *strides,
                           _plain(parents, torch.int32, "parents", (B, W_out)),
                           0 if lengths is None else _plain(lengths, torch.int32, "lengths", (B,)), unit,
                           layers, B, W, W_out, segs, units)
    _done(_beam_reorder(a, _stream()), "sd_beam_reorder")
    return dst
