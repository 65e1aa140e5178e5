"""Refusals of the entry points of drafted and branching sequences, without a GPU: bad arguments are
answered on the host with the documented status before CUDA is touched."""
import ctypes

import pytest
import torch

from gemm_conv_chains_gb300 import ops

from test_decoder_boundary import ALIGN, CUDA, FAKE, MIS, NULL, OK, SHAPE, UNSUP, Cache, cache, f32, i32, i64, vp


@pytest.fixture(scope="module")
def L():
    L = ctypes.CDLL(ops.lib()._name)
    cp = ctypes.POINTER(Cache)
    L.b2b_cache_tree_attention_workspace.argtypes = [cp, i64, i32, ctypes.POINTER(i64)]
    L.b2b_cache_tree_attention.argtypes = [i32, cp, i64, vp, i64, i32, vp, i32, vp, f32, f32, vp, vp, vp, i64, vp]
    L.b2b_cache_pages_workspace.argtypes = [i64, i32, ctypes.POINTER(i64)]
    L.b2b_cache_pages.argtypes = [i32, i64, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]
    L.b2b_cache_copy.argtypes = [cp, i64, vp, vp]
    L.b2b_cache_compact.argtypes = [cp, vp, vp, i32, vp, vp]
    return L


def tree(L, c=None, dt=0, T=2, q=FAKE, ldq=256, q_heads=4, masks=FAKE, words=1, positions=None, scale=0.1,
         cap=0.0, slopes=None, out=0x90000, ws=None, ws_bytes=0):
    return L.b2b_cache_tree_attention(dt, c or cache(), T, q, ldq, q_heads, masks, words, positions, scale,
                                      cap, slopes, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=2), UNSUP), (dict(T=-1), SHAPE), (dict(q_heads=3), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(cap=-1.0), SHAPE), (dict(ldq=260), ALIGN), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(masks=None), NULL), (dict(masks=FAKE + 4), ALIGN), (dict(positions=FAKE + 2), ALIGN),
    (dict(words=0), SHAPE), (dict(words=-1), SHAPE), (dict(words=1 << 25), UNSUP), (dict(ws=MIS), ALIGN),
    (dict(slopes=FAKE + 2), ALIGN), (dict(T=0, q=None, out=None, masks=None), OK),
])
def test_tree_refusals(L, kw, expect):
    assert tree(L, **kw) == expect


@pytest.mark.parametrize("kw", [dict(masks=0x90000), dict(masks=0x8FFF8), dict(masks=0x90008, words=3),
                                dict(positions=0x90000), dict(positions=0x8FFFC)])
def test_tree_output_over_what_is_read(L, kw):
    assert tree(L, **kw) == UNSUP


def test_tree_masks_need_a_bit_per_new_token(L):
    c = cache(batch=1, max_new=65)
    assert tree(L, c, T=65, words=1) == SHAPE
    n = ctypes.c_int64(-1)
    assert L.b2b_cache_tree_attention_workspace(None, 2, 4, ctypes.byref(n)) == NULL
    assert L.b2b_cache_tree_attention_workspace(cache(), 2, 4, None) == NULL
    assert L.b2b_cache_tree_attention_workspace(cache(head_dim=72), 2, 4, ctypes.byref(n)) == UNSUP
    assert L.b2b_cache_tree_attention_workspace(cache(), 0, 4, ctypes.byref(n)) == OK and n.value == 0


A = 0x100000     # fake operands, 64 KB apart


def pages(L, **kw):
    a = dict(page_size=16, pages=100, batch=4, width=8, table=A, lens=A + 0x10000, rows=4, parents=None,
             kept=None, new=None, table_out=A + 0x20000, lens_out=A + 0x30000, copies=A + 0x40000,
             left=A + 0x50000, ws=None, ws_bytes=0)
    a.update(kw)
    return L.b2b_cache_pages(a["page_size"], a["pages"], a["batch"], a["width"], a["table"], a["lens"],
                             a["rows"], a["parents"], a["kept"], a["new"], a["table_out"], a["lens_out"],
                             a["copies"], a["left"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP), (dict(page_size=24), UNSUP), (dict(pages=-1), SHAPE),
    (dict(pages=2 ** 31), UNSUP), (dict(batch=-1), SHAPE), (dict(width=-1), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=5), SHAPE), (dict(rows=4097, parents=FAKE), UNSUP), (dict(width=2 ** 28), UNSUP),
    (dict(rows=4096, parents=FAKE, width=2 ** 20), UNSUP), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(table_out=None), NULL), (dict(lens_out=None), NULL), (dict(copies=None), NULL), (dict(left=None), NULL),
    (dict(table=A + 2), ALIGN), (dict(kept=FAKE + 1), ALIGN), (dict(left=A + 0x50001), ALIGN),
    (dict(table_out=A), UNSUP), (dict(table_out=A + 124), UNSUP), (dict(lens_out=A + 0x10000), UNSUP),
    (dict(copies=A + 0x20000), UNSUP), (dict(left=A + 0x4002C), UNSUP), (dict(new=A + 0x3000C), UNSUP),
    (dict(pages=400000), NULL), (dict(pages=400000, ws=A + 0x60000, ws_bytes=16), SHAPE),
    (dict(pages=400000, ws=MIS, ws_bytes=1600000), ALIGN),
    (dict(pages=400000, ws=A - 0x10000, ws_bytes=1600000), UNSUP),
])
def test_pages_refusals(L, kw, expect):
    assert pages(L, **kw) == expect


def test_pages_workspace(L):
    n = ctypes.c_int64(-1)
    assert L.b2b_cache_pages_workspace(40960, 128, ctypes.byref(n)) == OK and n.value == 0
    assert L.b2b_cache_pages_workspace(40961, 4, ctypes.byref(n)) == OK and n.value == 163856 + 64
    assert L.b2b_cache_pages_workspace(9, 129, ctypes.byref(n)) == OK and n.value == 48 + 129 * 16
    assert L.b2b_cache_pages_workspace(-1, 4, ctypes.byref(n)) == SHAPE
    assert L.b2b_cache_pages_workspace(5, 5000, ctypes.byref(n)) == UNSUP
    assert L.b2b_cache_pages_workspace(5, 4, None) == NULL


@pytest.mark.parametrize("kw,expect", [
    (dict(pages=-1), SHAPE), (dict(heads=0), SHAPE), (dict(head_dim=80), UNSUP), (dict(page_size=48), UNSUP),
    (dict(k=None), NULL), (dict(v_scale=None), NULL), (dict(v=MIS), ALIGN), (dict(k_scale=FAKE + 2), ALIGN),
    (dict(pages=2 ** 31), UNSUP),
])
def test_pool_refusals(L, kw, expect):
    c = cache(**kw)
    assert L.b2b_cache_copy(c, 3, FAKE, None) == expect
    assert L.b2b_cache_compact(c, FAKE, FAKE, 3, FAKE, None) == expect


def test_copy_and_compact_refusals(L):
    assert L.b2b_cache_copy(None, 3, FAKE, None) == NULL
    assert L.b2b_cache_copy(cache(), -1, FAKE, None) == SHAPE
    assert L.b2b_cache_copy(cache(), 2 ** 31, FAKE, None) == UNSUP
    assert L.b2b_cache_copy(cache(), 3, None, None) == NULL
    assert L.b2b_cache_copy(cache(), 3, FAKE + 2, None) == ALIGN
    assert L.b2b_cache_copy(cache(), 0, None, None) == OK
    assert L.b2b_cache_compact(None, FAKE, FAKE, 3, FAKE, None) == NULL
    for args, expect in (((None, FAKE, 3, FAKE), NULL), ((FAKE, None, 3, FAKE), NULL), ((FAKE, FAKE, 3, None), NULL),
                         ((FAKE, FAKE, -1, FAKE), SHAPE), ((FAKE + 2, FAKE, 3, FAKE), ALIGN),
                         ((FAKE, FAKE + 1, 3, FAKE), ALIGN), ((FAKE, FAKE, 0, FAKE), OK)):
        assert L.b2b_cache_compact(cache(), *args, None) == expect
    assert L.b2b_cache_compact(cache(batch=0), FAKE, FAKE, 3, FAKE, None) == OK
    assert L.b2b_cache_compact(cache(batch=-1), FAKE, FAKE, 3, FAKE, None) == SHAPE
    assert L.b2b_cache_compact(cache(lens=None), FAKE, FAKE, 3, FAKE, None) == NULL
    assert L.b2b_cache_compact(cache(max_pages=2 ** 28), FAKE, FAKE, 3, FAKE, None) == UNSUP
    assert L.b2b_cache_compact(cache(max_pages=0), FAKE, FAKE, 3, FAKE, None) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_without_a_device_report_a_cuda_error(L):
    assert tree(L) == CUDA
    assert pages(L) == CUDA
    assert L.b2b_cache_copy(cache(), 3, FAKE, None) == CUDA
    assert L.b2b_cache_compact(cache(), FAKE, FAKE, 3, FAKE, None) == CUDA


def test_binding_refusals():
    q = torch.zeros(2, 2, 64, dtype=torch.float16)
    k = torch.zeros(3, 2, 16, 64).to(torch.float8_e4m3fn)
    s = torch.zeros(3, 2)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    masks = torch.zeros(2, 1, dtype=torch.int64)
    for call in (lambda: ops.cache_tree_attention(q, masks, k, k, s, s, table, lens),
                 lambda: ops.cache_tree_attention_workspace(2, 2, k, k, s, s, table, lens),
                 lambda: ops.cache_pages(table, lens, 3, 16), lambda: ops.cache_copy(k, k, s, s, table),
                 lambda: ops.cache_compact(k, k, s, s, table, lens, lens, table, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="out must have four tensors"):
        ops.cache_pages(table, lens, 3, 16, out=(table, lens))
    with pytest.raises(TypeError):
        ops.cache_copy(None, k, s, s, table)
