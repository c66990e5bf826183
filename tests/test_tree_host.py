"""CPU checks of the drafted-tree entry points: what they refuse, before any
CUDA call."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
from speculative_decoding_verification_85_b200 import _tree

FAKE = ctypes.c_void_p(1 << 20)


def _err(rc, status, text):
    assert rc == status
    assert text in sv.lib().spec_verify_last_error()


def test_verify_arguments():
    L = _tree._lib()

    def probs(B=2, g=3, V=10, dtype=sv.BF16, t=FAKE, x=FAKE):
        return L.spec_verify_probs(t, None, x, FAKE, FAKE, B, g, V, dtype, FAKE, FAKE, None)

    assert probs(B=0, t=None) == 0
    _err(probs(B=-1), 1, b"B must be in")
    _err(probs(g=0), 1, b"draft length")
    _err(probs(g=65), 1, b"draft length")
    _err(probs(V=0), 1, b"V must be")
    _err(probs(dtype=2), 1, b"dtype")
    _err(probs(t=None), 1, b"NULL")
    _err(probs(x=ctypes.c_void_p(3)), 1, b"aligned")

    def tree(B=2, N=4, width=3, V=10, dtype=sv.F32, t=FAKE, cu=FAKE):
        return L.spec_verify_tree(t, FAKE, FAKE, FAKE, cu, FAKE, FAKE, B, N, width, V, dtype,
                                  FAKE, FAKE, None, None)

    assert tree(B=0) == 0
    _err(tree(B=65537), 1, b"B must be in")
    _err(tree(N=-1), 1, b"N must be")
    _err(tree(width=0), 1, b"max_nodes")
    _err(tree(V=0), 1, b"V must be")
    _err(tree(dtype=5), 1, b"dtype")
    _err(tree(t=None), 1, b"NULL")
    _err(tree(cu=None), 1, b"NULL")
    _err(tree(t=ctypes.c_void_p(2)), 1, b"aligned")


def test_slots_arguments():
    L = _tree._lib()

    def slots(B=2, N=4, page=16, W=3, row=3, pool=5, lens=FAKE, count=FAKE):
        return L.spec_kv_slots(lens, FAKE, FAKE, None, 0, FAKE, row, W, FAKE, pool, count, B, N,
                               page, FAKE, FAKE, FAKE, FAKE, None)

    _err(slots(B=-1), 1, b"B must be in")
    _err(slots(N=-1), 1, b"N must be")
    _err(slots(page=0), 1, b"page_size")
    _err(slots(W=-1), 1, b"table_width")
    _err(slots(row=2), 1, b"overlap")
    _err(slots(pool=-1), 1, b"pool")
    _err(slots(lens=None), 1, b"NULL")
    _err(slots(count=None), 1, b"NULL")
    _err(slots(count=ctypes.c_void_p(6)), 1, b"aligned")


def test_append_arguments():
    L = _tree._lib()

    def append(**kw):
        a = _tree._AppendArgs(slots=FAKE, layers=1, N=2, H=2, D=8, num_pages=3, page_size=4,
                              elem_bytes=2)
        for w in range(2):
            a.src[w] = a.cache[w] = 1 << 20
        for k, x in kw.items():
            setattr(a, k, x)
        return L.spec_kv_append(ctypes.byref(a), None)

    assert append(N=0) == 0 and append(layers=0) == 0 and append(num_pages=0) == 0
    for k in ("layers", "N", "num_pages"):
        _err(append(**{k: -1}), 1, b"sizes out of range")
    for k in ("H", "D", "page_size"):
        _err(append(**{k: 0}), 1, b"sizes out of range")
    _err(append(elem_bytes=8), 1, b"elem_bytes")
    _err(append(slots=None), 1, b"NULL")
    _err(append(D=2**20, H=2**12), 1, b"too large")
    _err(L.spec_kv_append(None, None), 1, b"NULL")


def test_python_checks():
    t = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_probs(t, None, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
                             torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_tree(t[0], None, torch.zeros(3, dtype=torch.int32),
                            torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                            torch.zeros(3), torch.zeros(1), max_nodes=3)
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_slots(z, z, z, z[None], z, z[:1], rows=1, page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_append(t, t, z, t[None], t[None])


def test_attention_arguments():
    L = _tree._lib()
    assert sv.tree_attention_workspace_size(32, 8, 128) > 0
    for heads in ((32, 7, 128), (4, 8, 64), (129, 1, 64), (8, 0, 64), (8, 2, 136), (8, 2, 12)):
        assert sv.tree_attention_workspace_size(*heads) == 0

    def call(ws=FAKE, ws_bytes=1 << 30, **kw):
        a = _tree._AttentionArgs()
        for n, t in _tree._AttentionArgs._fields_:
            if t is ctypes.c_void_p:
                setattr(a, n, 1 << 20)
            elif t is ctypes.c_int64:
                setattr(a, n, 1024)
        sizes = dict(B=2, N=4, Hq=8, Hkv=2, D=64, num_pages=9, page_size=16, table_width=5,
                     dtype=1, scale=0.1)
        for n, x in {**sizes, **kw}.items():
            setattr(a, n, x)
        return L.spec_tree_attention(ctypes.byref(a), ws, ws_bytes, None)

    assert call(B=0) == 0 and call(N=0) == 0
    for kw, status, text in [
            (dict(dtype=0), 1, b"dtype"), (dict(B=-1), 1, b"B must be"),
            (dict(N=-1), 1, b"N must be"), (dict(Hkv=3), 1, b"multiple of Hkv"),
            (dict(Hq=512, Hkv=2), 1, b"multiple of Hkv"), (dict(D=12), 2, b"D must be"),
            (dict(D=256), 2, b"D must be"), (dict(page_size=24), 2, b"page_size"),
            (dict(page_size=1), 2, b"page_size"), (dict(page_size=192), 2, b"page_size"),
            (dict(num_pages=0), 1, b"num_pages"), (dict(table_width=2**28), 1, b"too long"),
            (dict(scale=0.0), 1, b"scale"), (dict(scale=float("nan")), 1, b"scale"),
            (dict(scale=float("inf")), 1, b"scale"), (dict(q=None), 1, b"NULL"),
            (dict(block_table=None), 1, b"NULL"), (dict(v_cache=(1 << 20) + 8), 1, b"16-byte"),
            (dict(out=(1 << 20) + 2), 1, b"16-byte"), (dict(lens=(1 << 20) + 1), 1, b"aligned"),
            (dict(q_node=12), 1, b"strides"), (dict(kc_token=0), 1, b"strides"),
            (dict(vc_page=-8), 1, b"strides"), (dict(ws=None), 4, b"workspace"),
            (dict(ws=ctypes.c_void_p(64)), 4, b"aligned"), (dict(ws_bytes=100), 4, b"too small")]:
        _err(call(**kw), status, text)
    _err(L.spec_tree_attention(None, FAKE, 1 << 30, None), 1, b"NULL")


def test_attention_python_checks():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.tree_attention(x, x, x, x[None], x[None], z[None], z[:1], z, z)
