"""A serving step of drafted trees on MI355X: Python binding of
include/sd_serve.h.

Functions mirror the C entry points; like the rest of the package they only
check and marshal arguments.
    qk_norm_rope(...)        -> sd_qk_norm_rope
    quant_attention(...)     -> sd_quant_attention
    quant_append(...)        -> sd_quant_append
    tree_verify_sample(...)  -> sd_tree_verify_sample

The 8-bit cache is a pair of tensors [pages][H_kv][page_size][D] of int8 or
float8_e4m3fn (any strides with contiguous rows, the same for both) with fp32
scales [pages][H_kv][page_size / block], a page table [B][max_pages] and the
slots in use [B], both int32.  With `stream` given, outputs and workspaces that
are not passed in are allocated on that stream too, as in a
`with torch.cuda.stream(stream)` block.
"""
import ctypes
import struct

import torch

from . import SD_BF16
from .tree import (SD_F16, _done, _entry, _here, _on, _output, _plain, _size_entry, _status, _stream,
                   _workspace)

SD_I8, SD_E4M3 = 3, 4
SD_MIN_BLOCK = 16
SD_NO_REPLACEMENT = 4
SD_ST_BAD_SCALE = 1 << 14

_P, _I32, _I64, _U32, _F, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                 ctypes.c_float, ctypes.c_size_t)


class SdQkNormRopeArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("q_out", _P), ("k_out", _P),
                ("q_node", _I64), ("q_head", _I64), ("k_node", _I64), ("k_head", _I64),
                ("q_out_node", _I64), ("q_out_head", _I64), ("k_out_node", _I64),
                ("k_out_head", _I64), ("q_weight", _P), ("k_weight", _P), ("positions", _P),
                ("inv_freq", _P), ("dtype", _I32), ("N", _I32), ("H_q", _I32), ("H_k", _I32),
                ("D", _I32), ("rot", _I32), ("interleaved", _I32), ("eps", _F)]


class SdQuantCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("page_stride", _I64),
                ("head_stride", _I64), ("slot_stride", _I64), ("scale_page", _I64),
                ("scale_head", _I64), ("page_table", _P), ("ld_table", _I64), ("context_lens", _P),
                ("code", _I32), ("B", _I32), ("H_kv", _I32), ("D", _I32), ("page_size", _I32),
                ("block", _I32), ("num_pages", _I32), ("max_pages", _I32)]


class SdQuantAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", SdQuantCache), ("q", _P), ("k_new", _P), ("v_new", _P),
                ("q_node", _I64), ("q_head", _I64), ("k_node", _I64), ("k_head", _I64),
                ("v_node", _I64), ("v_head", _I64), ("node_offsets", _P), ("parents", _P),
                ("dtype", _I32), ("N", _I32), ("max_nodes", _I32), ("H_q", _I32), ("window", _I32),
                ("sinks", _I32), ("scale", _F)]


class SdQuantAppendArgs(ctypes.Structure):
    _fields_ = [("cache", SdQuantCache), ("k_new", _P), ("v_new", _P), ("k_node", _I64),
                ("k_head", _I64), ("v_node", _I64), ("v_head", _I64), ("node_offsets", _P),
                ("path", _P), ("ld_path", _I64), ("path_lens", _P), ("dtype", _I32), ("N", _I32),
                ("max_new", _I32)]


class SdTreeSampleArgs(ctypes.Structure):
    _fields_ = [("target_probs", _P), ("draft_probs", _P), ("ld_target", _I64), ("ld_draft", _I64),
                ("tokens", _P), ("parents", _P), ("node_offsets", _P), ("accept_uniforms", _P),
                ("draw_uniforms", _P), ("B", _I32), ("N", _I32), ("V", _I32), ("V_draft", _I32),
                ("max_nodes", _I32), ("flags", _U32)]


# The argument structs as bytes (cheaper a call than filling a ctypes.Structure).
_CACHE = "QQQQqqqqqQqQiiiiiiii"
_NORM_ROPE = struct.Struct("QQQQqqqqqqqqQQQQiiiiiiif0q")
_QUANT_ATTENTION = struct.Struct(_CACHE + "QQQqqqqqqQQiiiiiif0q")
_QUANT_APPEND = struct.Struct(_CACHE + "QQqqqqQQqQiii0q")
_TREE_SAMPLE = struct.Struct("QQqqQQQQQiiiiiI0q")

_norm_rope = _entry("sd_qk_norm_rope", _P)
_quant_attention = _entry("sd_quant_attention", _P, _SZ, _P, _P, _P, _P)
_quant_append = _entry("sd_quant_append", _P, _P, _P)
_tree_sample = _entry("sd_tree_verify_sample", _P, _SZ, _P, _P, _P, _P, _P)
_quant_attention_bytes = _size_entry("sd_quant_attention_workspace_bytes")
_tree_sample_bytes = _size_entry("sd_tree_sample_workspace_bytes")


# ---- argument checks ----

def _element(t, name):
    if t.dtype is torch.bfloat16:
        return SD_BF16
    if t.dtype is torch.float16:
        return SD_F16
    raise TypeError(f"{name} must be bfloat16 or float16 (got {t.dtype})")


def _heads(t, name, like, N, D):
    """Rows [N][H][D] of this type: (pointer, strides, H); strides of axes of one
    say nothing."""
    if t.dim() != 3 or t.dtype is not like.dtype or t.shape[0] != N or t.shape[2] != D:
        raise ValueError(f"{name} must be {like.dtype} of shape [{N}, heads, {D}]")
    node, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    H = t.shape[1]
    return t.data_ptr(), (node if N > 1 else H * D), (head if H > 1 else D), H


def _rows(t, name, like, N, H, D):
    """Rows [N][H][D] of this type and number of heads: (pointer, strides)."""
    p, node, head, heads = _heads(t, name, like, N, D)
    if heads != H:
        raise ValueError(f"{name} must be {like.dtype} of shape {[N, H, D]}")
    return p, node, head


def _alike(a, b):
    """Whether strides are the same; those of axes of one say nothing."""
    return a.stride() == b.stride() or all(x == y for x, y, n in zip(a.stride(), b.stride(), a.shape) if n > 1)


def _cache(k, v, k_scale, v_scale, table, lens):
    """The fields of sd_quant_cache_t."""
    if k.dtype is torch.int8:
        code = SD_I8
    elif k.dtype is torch.float8_e4m3fn:
        code = SD_E4M3
    else:
        raise TypeError(f"the cache must be int8 or float8_e4m3fn (got {k.dtype})")
    strides = k.stride()
    if len(strides) != 4 or k.shape != v.shape or v.dtype is not k.dtype or not _alike(k, v):
        raise ValueError("k_cache and v_cache must be [pages][H_kv][page_size][D] with the same "
                         "type, shape and strides")
    pages, H, page, D = k.shape
    ps, hs, ss, es = strides
    if es != 1 and D > 1:
        raise ValueError("the elements of a cache row must be contiguous")
    sst = k_scale.stride()
    if (k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 or len(sst) != 3 or
            k_scale.shape != v_scale.shape or not _alike(k_scale, v_scale) or k_scale.shape[:2] != (pages, H)):
        raise ValueError("k_scale and v_scale must be float32 [pages][H_kv][page_size / block] with "
                         "the same shape and strides")
    blocks = k_scale.shape[2]
    if blocks < 1 or page % blocks or (blocks > 1 and sst[2] != 1):
        raise ValueError("the scales of a page and head must be contiguous and divide the page")
    if table.dtype is not torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("page_table must be int32 [B][max_pages] with contiguous rows")
    B, cols = table.shape
    scale_page, scale_head, _ = sst
    if pages == 1:
        ps = scale_page = 0
    if H == 1:
        hs = scale_head = 0
    return (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), ps, hs, ss, scale_page, scale_head,
            table.data_ptr(), table.stride(0) if B > 1 else max(cols, table.stride(0)),
            _plain(lens, torch.int32, "context_lens", (B,)), code, B, H, D, page, page // blocks, pages, cols)


# ---- norms and rotation ----

def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, out_q=None, out_k=None, stream=None):
    """Norm of each head of q [N][H_q][D] and k [N][H_k][D] (or None) and its
    rotation by positions [N] (int32) times inv_freq [rot / 2] (float32).
    Returns (q, k) as new tensors, or in out_q and out_k, which may be q and k.

    q_weight, k_weight: [D] of the element type; None leaves out the norm.
    interleaved: the pairs are (2 j, 2 j + 1) instead of (j, j + rot / 2)."""
    if stream is not None:
        return _on(stream, qk_norm_rope, locals())
    _here(q, k, positions, inv_freq, q_weight, k_weight, out_q, out_k)
    code = _element(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [N][H_q][D]")
    N, _, D = q.shape
    qp, qn, qh, Hq = _heads(q, "q", q, N, D)
    if out_q is None:
        out_q = q.new_empty(q.shape)
    elif out_q.shape != q.shape:
        raise ValueError("out_q must have q's shape")
    oqp, oqn, oqh, _ = _heads(out_q, "out_q", q, N, D)
    key = (0, 0, 0, 0)
    if k is None:
        if out_k is not None or k_weight is not None:
            raise ValueError("out_k and k_weight need k")
        okp = okn = okh = 0
    else:
        key = _heads(k, "k", q, N, D)
        if out_k is None:
            out_k = k.new_empty(k.shape)
        elif out_k.shape != k.shape:
            raise ValueError("out_k must have k's shape")
        okp, okn, okh, _ = _heads(out_k, "out_k", q, N, D)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    half = inv_freq.shape[0]
    a = _NORM_ROPE.pack(qp, key[0], oqp, okp, qn, qh, key[1], key[2], oqn, oqh, okn, okh,
                        0 if q_weight is None else _plain(q_weight, q.dtype, "q_weight", (D,)),
                        0 if k_weight is None else _plain(k_weight, q.dtype, "k_weight", (D,)),
                        _plain(positions, torch.int32, "positions", (N,)),
                        _plain(inv_freq, torch.float32, "inv_freq", (half,)), code, N, Hq, key[3], D,
                        2 * half, bool(interleaved), eps)
    _done(_norm_rope(a, _stream()), "sd_qk_norm_rope")
    return out_q, out_k


# ---- the 8-bit cache ----

def _attention_args(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens,
                    node_offsets, max_nodes, parents, window, sinks, scale):
    c = _cache(k_cache, v_cache, k_scale, v_scale, page_table, context_lens)
    B, H = c[13:15]
    N, Hq, D = q.shape
    if c[15] != D:
        raise ValueError("queries and cache must have the same head size")
    code = _element(q, "q")
    return _QUANT_ATTENTION.pack(
        *c, *_interleave(_rows(q, "q", q, N, Hq, D), _rows(k_new, "k_new", q, N, H, D),
                         _rows(v_new, "v_new", q, N, H, D)),
        _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)),
        0 if parents is None else _plain(parents, torch.int32, "parents", (N,)), code, N, max_nodes,
        Hq, window, sinks, D ** -0.5 if scale is None else scale)


def _interleave(*rows):
    """Pointers of all rows, then their strides."""
    return [r[0] for r in rows] + [s for r in rows for s in r[1:]]


def make_quant_attention_args(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table,
                              context_lens, node_offsets, max_nodes, parents=None, window=0, sinks=0,
                              scale=None):
    """sd_quant_attention_args_t from tensors, as quant_attention takes them."""
    return SdQuantAttentionArgs.from_buffer_copy(_attention_args(
        q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens, node_offsets,
        max_nodes, parents, window, sinks, scale))


def quant_attention_workspace_bytes(args):
    """Bytes of workspace quant_attention needs for a filled argument struct."""
    return _quant_attention_bytes(bytes(args))


def quant_attention(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens,
                    node_offsets, max_nodes, parents=None, window=0, sinks=0, scale=None,
                    want_lse=False, out=None, lse=None, status=None, workspace=None, stream=None):
    """Attention of the packed nodes of B drafted trees (q [N][H_q][D], k_new and
    v_new [N][H_kv][D], node_offsets [B + 1], parents [N] int32 or None for
    chains) over the 8-bit cache and each other; returns (out [N][H_q][D], lse
    [N][H_q] or None).

    window > 0: only keys less than `window` positions back are seen, and the
    first `sinks` positions.  scale defaults to 1 / sqrt(D).  out, lse: optional
    preallocated contiguous outputs; status: optional [B] int32 tensor for the
    per-request bits."""
    if stream is not None:
        return _on(stream, quant_attention, locals())
    _here(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens, node_offsets,
          parents, out, lse, status)
    a = _attention_args(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens,
                        node_offsets, max_nodes, parents, window, sinks, scale)
    shape = q.shape
    out = _output(out, q.dtype, "out", shape, q)
    if want_lse or lse is not None:
        lse = _output(lse, torch.float32, "lse", shape[:2], q)
    ws, wp, n = _workspace(_quant_attention_bytes, a, workspace, q)
    rc = _quant_attention(a, wp, n, out.data_ptr(), None if lse is None else lse.data_ptr(),
                          _status(status, page_table.shape[0]), _stream())
    _done(rc, "sd_quant_attention")
    return out, lse


def quant_append(k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens,
                 node_offsets, max_new, out_context, path=None, path_lens=None, status=None,
                 stream=None):
    """Quantise and append the nodes path[b][: path_lens[b]] of each request, or
    with path None all of its nodes (up to max_new, a prompt's tokens) in order;
    out_context [B] receives the new lengths."""
    if stream is not None:
        return _on(stream, quant_append, locals())
    _here(k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, context_lens, node_offsets,
          out_context, path, path_lens, status)
    c = _cache(k_cache, v_cache, k_scale, v_scale, page_table, context_lens)
    N = k_new.shape[0]
    B, H, D = c[13:16]
    code = _element(k_new, "k_new")
    kept = (0, 0, 0)
    if (path is None) != (path_lens is None):
        raise ValueError("path and path_lens are given together")
    if path is not None:
        cols = path.shape[-1]
        kept = (_plain(path, torch.int32, "path", (B, cols)), cols,
                _plain(path_lens, torch.int32, "path_lens", (B,)))
    a = _QUANT_APPEND.pack(*c, *_interleave(_rows(k_new, "k_new", k_new, N, H, D),
                                            _rows(v_new, "v_new", k_new, N, H, D)),
                           _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)), *kept, code, N,
                           max_new)
    rc = _quant_append(a, _plain(out_context, torch.int32, "out_context", (B,)), _status(status, B),
                       _stream())
    _done(rc, "sd_quant_append")
    return out_context


# ---- sampled verify of a tree ----

def _probs(t, name, N):
    """Rows [N][V] of float32: (pointer, row stride, V)."""
    if t.dtype is not torch.float32 or t.dim() != 2 or t.shape[0] != N:
        raise ValueError(f"{name} must be float32 [{N}][V]")
    V = t.shape[1]
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the probabilities of a row must be contiguous")
    return t.data_ptr(), (t.stride(0) if N > 1 else (max(V, t.stride(0)) + 3) // 4 * 4), V


def tree_verify_sample(target_probs, tokens, parents, node_offsets, max_nodes, accept_uniforms,
                       draw_uniforms, draft_probs=None, flags=0, status=None, out=None,
                       workspace=None, stream=None):
    """Verify of B drafted trees that keeps the target's distribution:
    target_probs [N][V] and draft_probs [N][V_draft] (or None for trees whose
    children were not drawn) float32, tokens and parents [N], node_offsets
    [B + 1], accept_uniforms [N] and draw_uniforms [B] float32 in [0, 1).
    Returns (accepted [B], path [B][max_nodes], tokens [B][max_nodes]).

    flags: SD_NO_BONUS, SD_NO_REPLACEMENT; out: optional dict of preallocated
    outputs (accepted, path, tokens)."""
    if stream is not None:
        return _on(stream, tree_verify_sample, locals())
    N = tokens.numel()
    B = node_offsets.numel() - 1
    o = out or {}
    acc, path, tok = o.get("accepted"), o.get("path"), o.get("tokens")
    _here(target_probs, draft_probs, tokens, parents, node_offsets, accept_uniforms, draw_uniforms,
          status, acc, path, tok)
    p, ld, V = _probs(target_probs, "target_probs", N)
    q, ld_q, Vd = (0, 0, V) if draft_probs is None else _probs(draft_probs, "draft_probs", N)
    a = _TREE_SAMPLE.pack(p, q, ld, ld_q, _plain(tokens, torch.int32, "tokens", (N,)),
                          _plain(parents, torch.int32, "parents", (N,)),
                          _plain(node_offsets, torch.int32, "node_offsets", (B + 1,)),
                          _plain(accept_uniforms, torch.float32, "accept_uniforms", (N,)),
                          _plain(draw_uniforms, torch.float32, "draw_uniforms", (B,)), B, N, V, Vd,
                          max_nodes, flags)
    ws, wp, n = _workspace(_tree_sample_bytes, a, workspace, target_probs)
    acc = _output(acc, torch.int32, "accepted", (B,), target_probs)
    path = _output(path, torch.int32, "path", (B, max_nodes), target_probs)
    tok = _output(tok, torch.int32, "tokens", (B, max_nodes), target_probs)
    rc = _tree_sample(a, wp, n, acc.data_ptr(), path.data_ptr(), tok.data_ptr(), _status(status, B),
                      _stream())
    _done(rc, "sd_tree_verify_sample")
    return acc, path, tok
