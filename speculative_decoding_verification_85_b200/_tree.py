"""ctypes binding of include/spec_tree.h (argument marshalling only): drafted
trees verified over a paged key/value cache."""
from __future__ import annotations

import ctypes as C

import torch

from ._binding import _check, _dt, _on, lib

F16 = 2
MAX_NODES = 1024

_vp, _i32, _i64 = C.c_void_p, C.c_int, C.c_int64


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


def _same_device(first, **rest):
    if not first.is_cuda:
        raise ValueError("tensors must be CUDA tensors (no CPU path)")
    for name, t in rest.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} must be on {first.device}, got {t.device}")


def _want(t, name, dtype, *shape, contiguous=True):
    """Shape, type and contiguity of one argument; None in `shape` matches any size."""
    if t.dtype != dtype or t.dim() != len(shape) or any(
            s is not None and s != n for s, n in zip(shape, t.shape)):
        want = ", ".join("*" if s is None else str(s) for s in shape)
        raise ValueError(f"{name} must be {str(dtype).removeprefix('torch.')} [{want}], got "
                         f"{str(t.dtype).removeprefix('torch.')} {list(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _p(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


class _Call:
    """The device, the stream and the allocations of one call: outputs and
    scratch space are allocated on the stream that the kernels run on."""

    def __init__(self, device, stream):
        self._dev = _on(device)
        self.stream = torch.cuda.current_stream(device) if stream is None else stream
        self._ctx = torch.cuda.stream(self.stream)

    def __enter__(self):
        self._dev.__enter__()
        self._ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        self._ctx.__exit__(*exc)
        self._dev.__exit__(*exc)


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, dtype, *shape)
    return t


def spec_verify_probs(target, draft, tokens, uniforms, draw_uniforms, *, out_accept_len=None,
                      out_tokens=None, stream=None):
    """Verify chains against given probabilities with given uniforms: target
    [B, g+1, V], draft [B, g, V] (fp32 or bf16; None for point drafts), tokens
    [B, g] int32, uniforms [B, g] and draw_uniforms [B] fp32 in [0, 1).
    Token x at position i is accepted when u q(x) < p(x); the first rejection's
    correction token is drawn from max(p - q, 0) by draw_uniforms, the bonus
    token from target row g.  Returns (accept_len [B], tokens [B, g+1])."""
    _same_device(target, draft=draft, tokens=tokens, uniforms=uniforms,
                 draw_uniforms=draw_uniforms, out_accept_len=out_accept_len,
                 out_tokens=out_tokens)
    dt = _dt(target)
    _want(target, "target", target.dtype, None, None, None)
    B, g1, V = target.shape
    if draft is not None:
        _want(draft, "draft", target.dtype, B, g1 - 1, V)
    _want(tokens, "tokens", torch.int32, B, g1 - 1)
    _want(uniforms, "uniforms", torch.float32, B, g1 - 1)
    _want(draw_uniforms, "draw_uniforms", torch.float32, B)
    dev = target.device
    with _Call(dev, stream) as s:
        acc = _out(out_accept_len, "out_accept_len", torch.int32, (B,), dev)
        tok = _out(out_tokens, "out_tokens", torch.int32, (B, g1), dev)
        _check(_lib().spec_verify_probs(_p(target), _p(draft), _p(tokens), _p(uniforms),
                                        _p(draw_uniforms), B, g1 - 1, V, dt, _p(acc), _p(tok), s))
    return acc, tok


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
    _same_device(target, draft=draft, tokens=tokens, parents=parents, cu_nodes=cu_nodes,
                 uniforms=uniforms, draw_uniforms=draw_uniforms, out_accept_len=out_accept_len,
                 out_tokens=out_tokens, out_path=out_path)
    dt = _dt(target)
    _want(target, "target", target.dtype, None, None)
    N, V = target.shape
    if draft is not None:
        _want(draft, "draft", target.dtype, N, V)
    for t, n in ((tokens, "tokens"), (parents, "parents")):
        _want(t, n, torch.int32, N)
    _want(uniforms, "uniforms", torch.float32, N)
    _want(draw_uniforms, "draw_uniforms", torch.float32, None)
    B = draw_uniforms.shape[0]
    _want(cu_nodes, "cu_nodes", torch.int32, B + 1)
    dev = target.device
    with _Call(dev, stream) as s:
        acc = _out(out_accept_len, "out_accept_len", torch.int32, (B,), dev)
        tok = _out(out_tokens, "out_tokens", torch.int32, (B, max_nodes), dev)
        path = _out(out_path, "out_path", torch.int32, (B, max_nodes), dev)
        _check(_lib().spec_verify_tree(_p(target), _p(draft), _p(tokens), _p(parents),
                                       _p(cu_nodes), _p(uniforms), _p(draw_uniforms), B, N,
                                       max_nodes, V, dt, _p(acc), _p(tok), _p(path), s))
    return acc, tok, path


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
    _same_device(lens, add=add, cu_rows=cu_rows, block_table=block_table, free_pages=free_pages,
                 free_count=free_count, path=path, out_slots=out_slots, out_start=out_start,
                 out_lens=out_lens, out_free_count=out_free_count)
    _want(lens, "lens", torch.int32, None)
    B = lens.shape[0]
    _want(add, "add", torch.int32, B)
    _want(cu_rows, "cu_rows", torch.int32, B + 1)
    _want(block_table, "block_table", torch.int32, B, None, contiguous=False)
    W = block_table.shape[1]
    if B > 0 and W > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    _want(free_pages, "free_pages", torch.int32, None)
    _want(free_count, "free_count", torch.int32, 1)
    if path is not None:
        _want(path, "path", torch.int32, B, None)
    dev = lens.device
    with _Call(dev, stream) as s:
        slots = _out(out_slots, "out_slots", torch.int32, (rows,), dev)
        start = _out(out_start, "out_start", torch.int32, (B,), dev)
        new = _out(out_lens, "out_lens", torch.int32, (B,), dev)
        count = _out(out_free_count, "out_free_count", torch.int32, (1,), dev)
        _check(_lib().spec_kv_slots(
            _p(lens), _p(add), _p(cu_rows), _p(path), 0 if path is None else path.shape[1],
            _p(block_table), block_table.stride(0) if B > 1 else W, W, _p(free_pages),
            free_pages.shape[0], _p(free_count), B, rows, page_size, _p(slots), _p(start), _p(new),
            _p(count), s))
    return slots, start, new, count


def kv_append(k, v, slots, k_cache, v_cache, *, stream=None):
    """Keys and values written into the paged cache: row i of k, v
    [N, H, D] goes to slot slots[i] of k_cache, v_cache [pages, page_size, H,
    D]; slots (int32) outside the cache skip the row.  With a leading layer
    axis on all four, every layer at once.  Strides are free but for the last
    axis; k, v must not overlap the caches.  Returns None."""
    _same_device(k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache)
    if k.dim() not in (3, 4):
        raise ValueError(f"k must be [N, H, D] or [layers, N, H, D], got {list(k.shape)}")
    lead = tuple(k.shape[:k.dim() - 3])
    N, H, D = k.shape[-3:]
    _want(v, "v", k.dtype, *lead, N, H, D, contiguous=False)
    _want(k_cache, "k_cache", k.dtype, *lead, None, None, H, D, contiguous=False)
    pages, page = k_cache.shape[-4:-2]
    _want(v_cache, "v_cache", k.dtype, *lead, pages, page, H, D, contiguous=False)
    _want(slots, "slots", torch.int32, N)
    es = k.element_size()
    if es not in (1, 2, 4):
        raise ValueError(f"elements of 1, 2 or 4 bytes are copied, got {k.dtype}")
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if D > 1 and t.stride(-1) != 1:
            raise ValueError(f"{n}'s last axis must be contiguous")
    if N == 0 or H == 0 or D == 0 or pages == 0 or page == 0 or 0 in lead:
        return
    a = _AppendArgs(slots=_p(slots), layers=lead[0] if lead else 1, N=N, H=H, D=D,
                    num_pages=pages, page_size=page, elem_bytes=es)
    for w, (x, cache) in enumerate(((k, k_cache), (v, v_cache))):
        a.src[w], a.cache[w] = x.data_ptr(), cache.data_ptr()
        a.src_layer[w] = x.stride(0) if lead else 0
        a.cache_layer[w] = cache.stride(0) if lead else 0
        a.src_row[w], a.src_head[w] = x.stride(-3), x.stride(-2)
        a.cache_page[w], a.cache_token[w], a.cache_head[w] = cache.stride()[-4:-1]
    with _Call(k.device, stream) as s:
        _check(_lib().spec_kv_append(C.byref(a), s))


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
    _same_device(q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, block_table=block_table,
                 lens=lens, parents=parents, cu_nodes=cu_nodes, out=out, out_lse=out_lse,
                 workspace=workspace)
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    _want(q, "q", q.dtype, None, None, None, contiguous=False)
    N, Hq, D = q.shape
    _want(k, "k", q.dtype, N, None, D, contiguous=False)
    Hkv = k.shape[1]
    _want(v, "v", q.dtype, N, Hkv, D, contiguous=False)
    _want(k_cache, "k_cache", q.dtype, None, None, Hkv, D, contiguous=False)
    pages, page = k_cache.shape[:2]
    _want(v_cache, "v_cache", q.dtype, pages, page, Hkv, D, contiguous=False)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.stride(-1) != 1 and t.numel() > 0:
            raise ValueError(f"{n}'s last axis must be contiguous")
    _want(lens, "lens", torch.int32, None)
    B = lens.shape[0]
    _want(cu_nodes, "cu_nodes", torch.int32, B + 1)
    _want(parents, "parents", torch.int32, N)
    _want(block_table, "block_table", torch.int32, B, None, contiguous=False)
    W = block_table.shape[1]
    if B > 0 and W > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    dev = q.device
    with _Call(dev, stream) as s:
        out = _out(out, "out", q.dtype, (N, Hq, D), dev)
        if with_lse or out_lse is not None:
            out_lse = _out(out_lse, "out_lse", torch.float32, (N, Hq), dev)
        if workspace is None:
            workspace = torch.empty(max(tree_attention_workspace_size(Hq, Hkv, D), 256),
                                    dtype=torch.uint8, device=dev)
        a = _AttentionArgs(
            _p(q), _p(k), _p(v), _p(k_cache), _p(v_cache), _p(out), _p(out_lse),
            _p(block_table), _p(lens), _p(parents), _p(cu_nodes), *q.stride()[:2],
            *k.stride()[:2], *v.stride()[:2], *k_cache.stride()[:3], *v_cache.stride()[:3],
            block_table.stride(0), B, N, Hq, Hkv, D, pages, page, W,
            1 if q.dtype == torch.bfloat16 else F16, D ** -0.5 if scale is None else scale)
        _check(_lib().spec_tree_attention(C.byref(a), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), s))
    return out, out_lse
