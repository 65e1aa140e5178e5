"""Refusals of the decoder-block entry points, without a GPU: bad arguments are answered on the
host with the documented status before CUDA is touched."""
import ctypes

import pytest
import torch

from gemm_conv_chains_gb300 import ops

OK, NULL, SHAPE, ALIGN, UNSUP, CUDA = 0, 1, 2, 3, 4, 5
FAKE, MIS = 0x10000, 0x10008


i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class Cache(ctypes.Structure):
    """b2b_cache (include/b2b.h)."""
    _fields_ = [("k", vp), ("v", vp), ("k_scale", vp), ("v_scale", vp), ("pages", i64),
                ("heads", i32), ("page_size", i32), ("head_dim", i32), ("batch", i32),
                ("page_table", vp), ("max_pages", i32), ("max_new", i32), ("lens", vp),
                ("starts", vp)]


@pytest.fixture(scope="module")
def L():
    L = ctypes.CDLL(ops.lib()._name)
    cp = ctypes.POINTER(Cache)
    L.b2b_rotary_table.argtypes = ops.lib().b2b_rotary_table.argtypes
    L.b2b_rotary.argtypes = [i32, i64, i32, i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, i64, vp]
    L.b2b_cache_append.argtypes = [i32, cp, i64, vp, i64, vp, i64, vp, i64, i32, i32, vp, i64, i32,
                                   vp, i64, vp]
    L.b2b_cache_attention_workspace.argtypes = [cp, i64, i32, ctypes.POINTER(i64)]
    L.b2b_cache_attention.argtypes = [i32, cp, i64, vp, i64, i32, f32, f32, vp, vp, vp, i64, vp]
    return L


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=10, heads=2, page_size=16,
             head_dim=64, batch=2, page_table=FAKE, max_pages=4, max_new=1, lens=FAKE, starts=None)
    a.update(kw)
    return Cache(*[a[n] for n, _ in Cache._fields_])


def attend(L, c=None, dt=0, T=2, q=FAKE, ldq=256, q_heads=4, scale=0.1, cap=0.0, slopes=None,
           out=FAKE, ws=None, ws_bytes=0):
    return L.b2b_cache_attention(dt, c or cache(), T, q, ldq, q_heads, scale, cap, slopes, out, ws,
                                 ws_bytes, None)


CACHE_REFUSALS = [
    (dict(pages=-1), SHAPE), (dict(heads=0), SHAPE), (dict(batch=0), SHAPE), (dict(batch=-1), SHAPE),
    (dict(head_dim=80), UNSUP), (dict(head_dim=512), UNSUP), (dict(page_size=8), UNSUP),
    (dict(page_size=48), UNSUP), (dict(page_size=512), UNSUP), (dict(max_new=0), SHAPE),
    (dict(max_new=3), SHAPE), (dict(pages=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=2 ** 28), UNSUP), (dict(k=None), NULL), (dict(v_scale=None), NULL),
    (dict(lens=None), NULL), (dict(page_table=None), NULL), (dict(k=MIS), ALIGN),
    (dict(k_scale=FAKE + 2), ALIGN), (dict(starts=FAKE + 1), ALIGN), (dict(batch=3), SHAPE),
]


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS)
def test_cache_refusals(L, kw, expect):
    c = cache(**kw)
    assert attend(L, c, q_heads=4, ldq=4 * kw.get("head_dim", 64)) == expect
    assert L.b2b_cache_append(0, c, 2, FAKE, 2 * 512, FAKE, 2 * 512, None, 0, 0, 0, None, 0, 0, None,
                              0, None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=2), UNSUP), (dict(T=-1), SHAPE), (dict(q_heads=3), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(cap=-1.0), SHAPE), (dict(cap=float("inf")), SHAPE),
    (dict(ldq=248), SHAPE), (dict(ldq=260), ALIGN), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(q=MIS), ALIGN), (dict(slopes=FAKE + 2), ALIGN), (dict(ws=MIS), ALIGN),
    (dict(T=0, q=None, out=None), OK),
])
def test_attention_refusals(L, kw, expect):
    assert attend(L, **kw) == expect


def test_null_cache_and_workspace_query(L):
    n = ctypes.c_int64(-1)
    assert L.b2b_cache_attention_workspace(None, 2, 4, ctypes.byref(n)) == NULL
    assert L.b2b_cache_attention_workspace(cache(), 2, 4, None) == NULL
    assert L.b2b_cache_attention_workspace(cache(head_dim=72), 2, 4, ctypes.byref(n)) == UNSUP
    assert L.b2b_cache_attention_workspace(cache(), 0, 4, ctypes.byref(n)) == OK and n.value == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=-1), UNSUP), (dict(ldk=120), SHAPE), (dict(ldv=132), ALIGN), (dict(k=None), NULL),
    (dict(v=MIS), ALIGN), (dict(table=FAKE, rot=0), SHAPE), (dict(table=FAKE, rot=72), SHAPE),
    (dict(table=FAKE, rot=40), ALIGN), (dict(table=FAKE, layout=2), UNSUP),
    (dict(table=FAKE, P=-1), SHAPE), (dict(table=MIS), ALIGN),
    (dict(q=FAKE, qo=FAKE), NULL),                                     # queries without a table
    (dict(table=FAKE, q=FAKE), NULL), (dict(table=FAKE, q=FAKE, qo=FAKE, Hq=0), SHAPE),
    (dict(table=FAKE, q=FAKE, qo=FAKE, ldq=64), SHAPE),
    (dict(table=FAKE, q=MIS, qo=FAKE), ALIGN), (dict(T=0, k=None, v=None), OK),
])
def test_append_refusals(L, kw, expect):
    a = dict(dt=0, T=2, k=FAKE, ldk=128, v=FAKE, ldv=128, table=None, P=9, rot=64, layout=0, q=None,
             ldq=256, Hq=4, qo=None, ldqo=256)
    a.update(kw)
    assert L.b2b_cache_append(a["dt"], cache(), a["T"], a["k"], a["ldk"], a["v"], a["ldv"],
                              a["table"], a["P"], a["rot"], a["layout"], a["q"], a["ldq"], a["Hq"],
                              a["qo"], a["ldqo"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=3), UNSUP), (dict(inverse=2), UNSUP), (dict(T=-1), SHAPE), (dict(H=0), SHAPE),
    (dict(D=60), ALIGN), (dict(rot=24), ALIGN), (dict(rot=80), SHAPE), (dict(layout=-1), UNSUP),
    (dict(ldx=100), SHAPE), (dict(ldo=132), ALIGN), (dict(x=None), NULL), (dict(table=None), NULL),
    (dict(pos=None), NULL), (dict(out=MIS), ALIGN), (dict(P=-1), SHAPE), (dict(T=2 ** 31), UNSUP),
    (dict(T=0, x=None, out=None, pos=None), OK),
])
def test_rotary_refusals(L, kw, expect):
    a = dict(dt=1, T=3, H=2, D=64, rot=64, layout=0, inverse=0, x=FAKE, ldx=128, table=FAKE, P=10,
             pos=FAKE, out=FAKE, ldo=128)
    a.update(kw)
    assert L.b2b_rotary(a["dt"], a["T"], a["H"], a["D"], a["rot"], a["layout"], a["inverse"], a["x"],
                        a["ldx"], a["table"], a["P"], a["pos"], a["out"], a["ldo"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), SHAPE), (dict(rot=0), SHAPE), (dict(rot=20), ALIGN), (dict(base=0.0), SHAPE),
    (dict(scaling=3), UNSUP), (dict(factor=0.0), SHAPE), (dict(gain=float("nan")), SHAPE),
    (dict(scaling=2, original=0), SHAPE), (dict(scaling=2, low=4.0, high=4.0), SHAPE),
    (dict(n=2 ** 40), UNSUP), (dict(table=None), NULL), (dict(n=0, table=None), OK),
])
def test_rotary_table_refusals(L, kw, expect):
    a = dict(n=8, rot=32, base=1e4, scaling=0, factor=1.0, original=10, low=1.0, high=32.0, gain=1.0,
             table=FAKE)
    a.update(kw)
    assert L.b2b_rotary_table(a["n"], a["rot"], a["base"], a["scaling"], a["factor"], a["original"],
                              a["low"], a["high"], a["gain"], a["table"], None) == expect


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_without_a_device_report_a_cuda_error(L):
    assert attend(L) == CUDA
    assert L.b2b_get_cache_error(None) == CUDA


def test_binding_refusals():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    table, pos = torch.zeros(4, 32, 2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ops.rotary(x, table, pos)
    with pytest.raises(TypeError, match="expected float16 or bfloat16, got torch.float32"):
        ops.rotary(x.float(), table, pos)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        ops.rotary(None, table, pos)
    with pytest.raises(ValueError, match="three dimensions"):
        ops.rotary(x[0], table, pos)
    with pytest.raises(ValueError, match="layout"):
        ops.rotary(x, table, pos, layout="pairs")
    with pytest.raises(ValueError, match="scaling"):
        ops.rotary_table(4, 32, scaling="other")
    with pytest.raises(ValueError, match="CUDA"):
        ops.rotary_table(4, 32, device="cpu")
    k = torch.zeros(3, 2, 16, 64).to(torch.float8_e4m3fn)
    s = torch.zeros(3, 2)
    pages, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.cache_append(x, x, k, k, s, s, pages, lens)
    with pytest.raises(ValueError, match="CUDA"):
        ops.cache_attention(x, k, k, s, s, pages, lens)
    with pytest.raises(ValueError, match="CUDA"):
        ops.cache_attention_workspace(2, 2, k, k, s, s, pages, lens)
    with pytest.raises(TypeError):
        ops.cache_attention(x)
