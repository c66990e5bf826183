"""ctypes binding of include/spec_tree.h (argument marshalling only): drafted
trees verified over a paged key/value cache."""
from __future__ import annotations

import ctypes as C

import torch

from ._binding import _check, _dt, _on, lib

F16 = 2
MAX_NODES = 1024

_vp, _i32, _i64 = C.c_void_p, C.c_int, C.c_int64
# the current stream's handle, without an object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _AppendArgs(C.Structure):
    _fields_ = [("src", _vp * 2), ("cache", _vp * 2), ("src_layer", _i64 * 2),
                ("src_row", _i64 * 2), ("src_head", _i64 * 2), ("cache_layer", _i64 * 2),
                ("cache_page", _i64 * 2), ("cache_token", _i64 * 2), ("cache_head", _i64 * 2),
                ("slots", _vp), ("layers", _i32), ("N", _i32), ("H", _i32), ("D", _i32),
                ("num_pages", _i32), ("page_size", _i32), ("elem_bytes", _i32)]


class _AttentionArgs(C.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "v", "k_cache", "v_cache", "out", "out_lse",
                                    "block_table", "lens", "parents", "cu_nodes")]
                + [(n, _i64) for n in ("q_node", "q_head", "k_node", "k_head", "v_node", "v_head",
                                       "kc_page", "kc_token", "kc_head", "vc_page", "vc_token",
                                       "vc_head", "table_row")]
                + [(n, _i32) for n in ("B", "N", "Hq", "Hkv", "D", "num_pages", "page_size",
                                       "table_width", "dtype")]
                + [("scale", C.c_float)])


_ready = None


def _lib():
    global _ready
    L = lib()
    if _ready is not L:
        L.spec_verify_probs.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                        _vp]
        L.spec_verify_probs.restype = _i32
        L.spec_verify_tree.argtypes = [_vp] * 7 + [_i32] * 5 + [_vp] * 4
        L.spec_verify_tree.restype = _i32
        L.spec_kv_slots.argtypes = ([_vp] * 4 + [_i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32,
                                                 _i32] + [_vp] * 5)
        L.spec_kv_slots.restype = _i32
        L.spec_kv_append.argtypes = [C.POINTER(_AppendArgs), _vp]
        L.spec_kv_append.restype = _i32
        L.spec_tree_attention_workspace_size.argtypes = [_i32, _i32, _i32]
        L.spec_tree_attention_workspace_size.restype = C.c_size_t
        L.spec_tree_attention.argtypes = [C.POINTER(_AttentionArgs), _vp, C.c_size_t, _vp]
        L.spec_tree_attention.restype = _i32
        _ready = L
    return L


# The argument checks run on every call of a serving step, some of which take
# a few microseconds on the device: one pass over (tensor, name, type, shape,
# dense) rows, details on failure.
def _device(t):
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors (no CPU path)")
    return t.device


def _dims(t, name, n):
    """The shape of an argument that must have n axes."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} axes, got {list(shape)}")
    return shape


def _want(device, *checks):
    for t, name, dtype, shape, dense in checks:
        if (t.dtype is dtype and t.shape == shape and t.device == device
                and (not dense or t.is_contiguous())):
            continue
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
        if t.dtype is dtype and t.shape == shape:
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} must be {str(dtype).removeprefix('torch.')} {list(shape)}, got "
                         f"{str(t.dtype).removeprefix('torch.')} {list(t.shape)}")


def _rows(table, B, W):
    if B > 0 and W > 1 and table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")


def _p(t):
    return None if t is None else t.data_ptr()


def _call(device, stream, body):
    """body(stream handle) with the tensors' device current and with the
    stream that the kernels run on current too, since that is where outputs and
    scratch space are allocated."""
    if stream is None and torch.cuda.current_device() == device.index:
        return body(_raw_stream(device.index))
    if stream is not None and stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    with _on(device):
        if stream is None:
            return body(torch.cuda.current_stream(device).cuda_stream)
        with torch.cuda.stream(stream):
            return body(stream.cuda_stream)


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(device, (t, name, dtype, shape, True))
    return t


def spec_verify_probs(target, draft, tokens, uniforms, draw_uniforms, *, out_accept_len=None,
                      out_tokens=None, stream=None):
    """Verify chains against given probabilities with given uniforms: target
    [B, g+1, V], draft [B, g, V] (fp32 or bf16; None for point drafts), tokens
    [B, g] int32, uniforms [B, g] and draw_uniforms [B] fp32 in [0, 1).
    Token x at position i is accepted when u q(x) < p(x); the first rejection's
    correction token is drawn from max(p - q, 0) by draw_uniforms, the bonus
    token from target row g.  Returns (accept_len [B], tokens [B, g+1])."""
    dev, dt = _device(target), _dt(target)
    B, g1, V = _dims(target, "target", 3)
    g = g1 - 1
    _want(dev, (target, "target", target.dtype, (B, g1, V), True),
          (tokens, "tokens", torch.int32, (B, g), True),
          (uniforms, "uniforms", torch.float32, (B, g), True),
          (draw_uniforms, "draw_uniforms", torch.float32, (B,), True))
    if draft is not None:
        _want(dev, (draft, "draft", target.dtype, (B, g, V), True))

    def body(s):
        acc = _out(out_accept_len, "out_accept_len", torch.int32, (B,), dev)
        tok = _out(out_tokens, "out_tokens", torch.int32, (B, g1), dev)
        _check(_lib().spec_verify_probs(_p(target), _p(draft), _p(tokens), _p(uniforms),
                                        _p(draw_uniforms), B, g, V, dt, _p(acc), _p(tok), s))
        return acc, tok

    return _call(dev, stream, body)


def spec_verify_tree(target, draft, tokens, parents, cu_nodes, uniforms, draw_uniforms, *,
                     max_nodes: int, out_accept_len=None, out_tokens=None, out_path=None,
                     stream=None):
    """Verify drafted trees against given probabilities with given uniforms.
    The nodes of all B sequences are packed (cu_nodes [B+1] int32, parents [N]
    int32 within the sequence, node 0 the root with parent -1); target [N, V]:
    the law of the token after every node; draft [N, V]: the law its children
    were drawn from (None for point drafts); tokens [N] int32, uniforms [N],
    draw_uniforms [B] fp32; max_nodes: the most nodes a sequence has.
    Returns (accept_len [B], tokens [B, max_nodes], path [B, max_nodes])."""
    dev, dt = _device(target), _dt(target)
    N, V = _dims(target, "target", 2)
    B, = _dims(draw_uniforms, "draw_uniforms", 1)
    _want(dev, (target, "target", target.dtype, (N, V), True),
          (tokens, "tokens", torch.int32, (N,), True),
          (parents, "parents", torch.int32, (N,), True),
          (cu_nodes, "cu_nodes", torch.int32, (B + 1,), True),
          (uniforms, "uniforms", torch.float32, (N,), True),
          (draw_uniforms, "draw_uniforms", torch.float32, (B,), True))
    if draft is not None:
        _want(dev, (draft, "draft", target.dtype, (N, V), True))

    def body(s):
        acc = _out(out_accept_len, "out_accept_len", torch.int32, (B,), dev)
        tok = _out(out_tokens, "out_tokens", torch.int32, (B, max_nodes), dev)
        path = _out(out_path, "out_path", torch.int32, (B, max_nodes), dev)
        _check(_lib().spec_verify_tree(_p(target), _p(draft), _p(tokens), _p(parents),
                                       _p(cu_nodes), _p(uniforms), _p(draw_uniforms), B, N,
                                       max_nodes, V, dt, _p(acc), _p(tok), _p(path), s))
        return acc, tok, path

    return _call(dev, stream, body)


def kv_slots(lens, add, cu_rows, block_table, free_pages, free_count, *, rows: int,
             page_size: int, path=None, out_slots=None, out_start=None, out_lens=None,
             out_free_count=None, stream=None):
    """Block tables and slot maps from request lengths, on the device: lens [B]
    tokens held, add [B] tokens joining (-1 releases the request), cu_rows
    [B+1] bounds of the requests' packed rows (`rows` in all), block_table
    [B, W] and free_pages [P] (updated in place), free_count [1]; path [B, w]:
    the rows that are kept (out_path of spec_verify_tree), None for the first
    add[b].  All int32.  Returns (slots [rows], start [B], new lens [B], new
    free_count [1]); slots is -1 for rows not kept, start -1 for a request that
    was refused (no pages, table row too short) or released.  out_lens and
    out_free_count may be lens and free_count."""
    dev = _device(lens)
    B, = _dims(lens, "lens", 1)
    W = _dims(block_table, "block_table", 2)[1]
    pool, = _dims(free_pages, "free_pages", 1)
    width = 0
    _want(dev, (lens, "lens", torch.int32, (B,), True), (add, "add", torch.int32, (B,), True),
          (cu_rows, "cu_rows", torch.int32, (B + 1,), True),
          (block_table, "block_table", torch.int32, (B, W), False),
          (free_pages, "free_pages", torch.int32, (pool,), True),
          (free_count, "free_count", torch.int32, (1,), True))
    _rows(block_table, B, W)
    if path is not None:
        width = _dims(path, "path", 2)[1]
        _want(dev, (path, "path", torch.int32, (B, width), True))

    def body(s):
        if out_slots is out_start is out_lens is out_free_count is None:  # one allocation
            slots, start, new, count = torch.empty(
                rows + 2 * B + 1, dtype=torch.int32, device=dev).split((rows, B, B, 1))
        else:
            slots = _out(out_slots, "out_slots", torch.int32, (rows,), dev)
            start = _out(out_start, "out_start", torch.int32, (B,), dev)
            new = _out(out_lens, "out_lens", torch.int32, (B,), dev)
            count = _out(out_free_count, "out_free_count", torch.int32, (1,), dev)
        _check(_lib().spec_kv_slots(
            _p(lens), _p(add), _p(cu_rows), _p(path), width, _p(block_table),
            block_table.stride(0) if B > 1 else W, W, _p(free_pages), pool, _p(free_count), B,
            rows, page_size, _p(slots), _p(start), _p(new), _p(count), s))
        return slots, start, new, count

    return _call(dev, stream, body)


def append_args(k, v, k_cache, v_cache):
    """kv_append's rows and caches, checked, as its argument block without the
    slots; None where there is nothing to copy."""
    dev, dt = _device(k), k.dtype
    shape = k.shape
    if len(shape) not in (3, 4):
        raise ValueError(f"k must be [N, H, D] or [layers, N, H, D], got {list(shape)}")
    lead = tuple(shape[:-3])
    N, H, D = shape[-3:]
    pages, page = _dims(k_cache, "k_cache", len(shape) + 1)[-4:-2]
    cache = lead + (pages, page, H, D)
    _want(dev, (v, "v", dt, shape, False), (k_cache, "k_cache", dt, cache, False),
          (v_cache, "v_cache", dt, cache, False))
    es = k.element_size()
    if es not in (1, 2, 4):
        raise ValueError(f"elements of 1, 2 or 4 bytes are copied, got {k.dtype}")
    if k.numel() == 0 or k_cache.numel() == 0:
        return None
    ks, vs, kcs, vcs = k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
    if D > 1 and not ks[-1] == vs[-1] == kcs[-1] == vcs[-1] == 1:
        raise ValueError("the last axis of k, v and the caches must be contiguous")
    two = _i64 * 2
    layered = bool(lead)
    return _AppendArgs(
        (_vp * 2)(k.data_ptr(), v.data_ptr()), (_vp * 2)(k_cache.data_ptr(), v_cache.data_ptr()),
        two(ks[0], vs[0]) if layered else two(), two(ks[-3], vs[-3]), two(ks[-2], vs[-2]),
        two(kcs[0], vcs[0]) if layered else two(), two(kcs[-4], vcs[-4]), two(kcs[-3], vcs[-3]),
        two(kcs[-2], vcs[-2]), None, lead[0] if layered else 1, N, H, D, pages, page, es)


def append_rows(args, slots, device, stream):
    """kv_append of checked arguments."""
    if args is None:
        return
    args.slots = slots.data_ptr()
    _call(device, stream, lambda s: _check(_lib().spec_kv_append(C.byref(args), s)))


def kv_append(k, v, slots, k_cache, v_cache, *, stream=None):
    """Keys and values written into the paged cache: row i of k, v
    [N, H, D] goes to slot slots[i] of k_cache, v_cache [pages, page_size, H,
    D]; slots (int32) outside the cache skip the row.  With a leading layer
    axis on all four, every layer at once.  Strides are free but for the last
    axis; k, v must not overlap the caches.  Returns None."""
    args = append_args(k, v, k_cache, v_cache)
    _want(k.device, (slots, "slots", torch.int32, (k.shape[-3],), True))
    append_rows(args, slots, k.device, stream)


def tree_attention_workspace_size(Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace tree_attention needs (0 for head layouts it refuses)."""
    return int(_lib().spec_tree_attention_workspace_size(Hq, Hkv, D))


def tree_attention(q, k, v, k_cache, v_cache, block_table, lens, parents, cu_nodes, *,
                   scale: float | None = None, with_lse: bool = False, out=None, out_lse=None,
                   workspace=None, stream=None):
    """Attention of drafted nodes over their sequence's paged context and
    their own ancestors.  q [N, Hq, D], k, v [N, Hkv, D] (bf16 or fp16): the
    nodes of all B sequences, packed as cu_nodes [B+1] says; k_cache, v_cache
    [pages, page_size, Hkv, D]; block_table [B, W], lens [B] (cached tokens),
    parents [N] int32.  Strides are free but for the last axis.  scale
    defaults to D ** -0.5.  Returns (out [N, Hq, D], lse [N, Hq] fp32 or
    None).  `workspace`: a uint8 tensor of tree_attention_workspace_size
    bytes, of any content; calls that may run at once need one each."""
    dev = _device(q)
    dt = q.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dt}")
    N, Hq, D = _dims(q, "q", 3)
    Hkv = _dims(k, "k", 3)[1]
    pages, page = _dims(k_cache, "k_cache", 4)[:2]
    B, = _dims(lens, "lens", 1)
    W = _dims(block_table, "block_table", 2)[1]
    nodes, cache = (N, Hkv, D), (pages, page, Hkv, D)
    _want(dev, (k, "k", dt, nodes, False), (v, "v", dt, nodes, False),
          (k_cache, "k_cache", dt, cache, False), (v_cache, "v_cache", dt, cache, False),
          (lens, "lens", torch.int32, (B,), True),
          (cu_nodes, "cu_nodes", torch.int32, (B + 1,), True),
          (parents, "parents", torch.int32, (N,), True),
          (block_table, "block_table", torch.int32, (B, W), False))
    _rows(block_table, B, W)
    qs, ks, vs, kcs, vcs = q.stride(), k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
    if N > 0 and not qs[2] == ks[2] == vs[2] == kcs[3] == vcs[3] == 1:
        raise ValueError("the last axis of q, k, v and the caches must be contiguous")

    def body(s):
        o = _out(out, "out", dt, (N, Hq, D), dev)
        lse = out_lse
        if with_lse or lse is not None:
            lse = _out(lse, "out_lse", torch.float32, (N, Hq), dev)
        ws = workspace
        if ws is not None:
            if ws.device != dev or not ws.is_contiguous():
                raise ValueError(f"workspace must be contiguous on {dev}")
        else:
            ws = torch.empty(max(tree_attention_workspace_size(Hq, Hkv, D), 256),
                             dtype=torch.uint8, device=dev)
        a = _AttentionArgs(
            _p(q), _p(k), _p(v), _p(k_cache), _p(v_cache), _p(o), _p(lse), _p(block_table),
            _p(lens), _p(parents), _p(cu_nodes), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], kcs[0],
            kcs[1], kcs[2], vcs[0], vcs[1], vcs[2], block_table.stride(0), B, N, Hq, Hkv, D,
            pages, page, W, 1 if dt is torch.bfloat16 else F16,
            D ** -0.5 if scale is None else scale)
        _check(_lib().spec_tree_attention(C.byref(a), ws.data_ptr(),
                                          ws.numel() * ws.element_size(), s))
        return o, lse

    return _call(dev, stream, body)
