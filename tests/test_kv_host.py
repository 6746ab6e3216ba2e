"""Refusals of the key/value cache's entry points, before anything runs on a
device: the C ABI's status codes and the binding's exceptions."""
import ctypes

import pytest
import torch

import mxfp4_block_scaled_fos_b200 as F
from mxfp4_block_scaled_fos_b200 import build as fbuild
from mxfp4_block_scaled_fos_b200 import kv


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return kv._lib()


NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE, ARG = 1, 2, 3, 4, 5, 7


def _cache(**kw):
    c = dict(k_codes=64, k_scales=128, v_codes=192, v_scales=256, k_tensor_scale=320, v_tensor_scale=384,
             num_pages=4, page_size=16, heads=2, head_dim=64, codes_page_stride=1024, scales_page_stride=128)
    c.update(kw)
    return kv._CacheC(*(c[n] for n, _ in kv._CacheC._fields_))


BAD_POOLS = [
    (dict(k_codes=None), NULL), (dict(v_tensor_scale=None), NULL), (dict(v_scales=136), ALIGN),
    (dict(k_codes=72), ALIGN), (dict(k_tensor_scale=322), ALIGN), (dict(codes_page_stride=1000), SHAPE),
    (dict(codes_page_stride=1032), ALIGN), (dict(codes_page_stride=1 << 32), SHAPE), (dict(scales_page_stride=64), SHAPE), (dict(scales_page_stride=136), ALIGN),
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(heads=0), SHAPE), (dict(num_pages=-1), SHAPE), (dict(num_pages=1 << 31), SHAPE),
]


def _append(L, cache=None, fmt=0, k=16, k_ld=128, v=16, tokens=3, slots=8, rot=None, q=None, q_ld=256, q_out=None,
            q_heads=4):
    c = cache or _cache()
    return L.fos_kv_append(ctypes.byref(c), fmt, k, k_ld, v, 128, tokens, slots,
                           None if rot is None else ctypes.byref(rot), q, q_ld, q_out, 256, q_heads, None, None)


def _attention(L, cache=None, q=16, q_ld=256, total=5, q_heads=4, cu=4, batch=2, pages=4, max_pages=3, kv_len=4,
               max_q=3, scale=0.1, causal=1, window=0, out=16, out_ld=256, lse=None, ws=16, wsb=1 << 40):
    c = cache or _cache()
    return L.fos_kv_attention(ctypes.byref(c), q, q_ld, total, q_heads, cu, batch, pages, max_pages, kv_len, max_q,
                              scale, causal, window, out, out_ld, lse, ws, wsb, None, None)


@pytest.mark.parametrize("bad,code", BAD_POOLS)
def test_pools(L, bad, code):
    c = _cache(**bad)
    assert _append(L, c) == code
    assert L.fos_kv_read(ctypes.byref(c), 8, 3, 16, 16, None, None) == code
    assert _attention(L, c) == code


def test_append_refusals(L):
    rot = kv._RotaryC(16, 4, 10, 64, 0)
    assert L.fos_kv_append(None, 0, 16, 128, 16, 128, 3, 8, None, None, 0, None, 0, 0, None, None) == NULL
    assert _append(L, fmt=3) == ARG and _append(L, fmt=-1) == ARG and _append(L, fmt=2) == UNSUPPORTED
    assert _append(L, k=None) == NULL and _append(L, v=None) == NULL and _append(L, slots=None) == NULL
    assert _append(L, k=24) == ALIGN and _append(L, k_ld=132) == ALIGN and _append(L, k_ld=120) == SHAPE
    assert _append(L, slots=12) == ALIGN
    assert _append(L, tokens=-1) == SHAPE and _append(L, tokens=1 << 31) == SHAPE
    assert _append(L, q=16, q_out=16) == ARG                        # queries without a rotation
    assert _append(L, rot=rot, q=16) == NULL and _append(L, rot=rot, q_out=16) == NULL
    assert _append(L, rot=rot, q=16, q_out=16, q_ld=248) == SHAPE
    assert _append(L, rot=rot, q=16, q_out=16, q_heads=0) == SHAPE
    assert _append(L, rot=rot, q=16, q_out=24) == ALIGN
    for bad, code in ((dict(table=None), NULL), (dict(positions=None), NULL), (dict(dim=24), SHAPE),
                      (dict(dim=0), SHAPE), (dict(dim=80), SHAPE), (dict(max_positions=-1), SHAPE),
                      (dict(interleaved=2), ARG), (dict(table=8), ALIGN), (dict(positions=2), ALIGN)):
        r = dict(table=16, positions=4, max_positions=10, dim=64, interleaved=0)
        r.update(bad)
        assert _append(L, rot=kv._RotaryC(*(r[n] for n, _ in kv._RotaryC._fields_))) == code, bad
    assert _append(L, tokens=0) == 0


def test_read_refusals(L):
    c = _cache()
    read = lambda slots=8, t=3, k=16, v=16: L.fos_kv_read(ctypes.byref(c), slots, t, k, v, None, None)  # noqa: E731
    assert read(slots=None) == NULL and read(k=None) == NULL and read(v=None) == NULL
    assert read(slots=4) == ALIGN and read(k=8) == ALIGN and read(v=8) == ALIGN
    assert read(t=-1) == SHAPE and read(t=0) == 0


def test_attention_refusals(L):
    for name in ("q", "cu", "pages", "kv_len", "out"):
        assert _attention(L, **{name: None}) == NULL, name
    assert _attention(L, q=8) == ALIGN and _attention(L, q_ld=260) == ALIGN and _attention(L, q_ld=248) == SHAPE
    assert _attention(L, out=8) == ALIGN and _attention(L, out_ld=248) == SHAPE
    assert _attention(L, cu=2) == ALIGN and _attention(L, lse=2) == ALIGN
    assert _attention(L, q_heads=3) == SHAPE and _attention(L, q_heads=0) == SHAPE
    assert _attention(L, total=-1) == SHAPE and _attention(L, batch=-1) == SHAPE and _attention(L, max_pages=-1) == SHAPE
    assert _attention(L, max_pages=1 << 28) == SHAPE
    assert _attention(L, causal=2) == ARG and _attention(L, window=-1) == ARG
    assert _attention(L, causal=0, window=5) == ARG and _attention(L, max_q=-1) == ARG
    assert _attention(L, scale=float("nan")) == ARG and _attention(L, scale=float("inf")) == ARG
    assert _attention(L, batch=0) == 0 and _attention(L, total=0) == 0


def test_binding_refuses_what_is_no_cache():
    t = torch.zeros
    with pytest.raises(TypeError):
        F.KVCache(t(2, 1, 16, 32, dtype=torch.uint8), t(2, 1, 16, 4, dtype=torch.uint8),
                  t(2, 1, 16, 32, dtype=torch.uint8), t(2, 1, 16, 4, dtype=torch.uint8), t(1), t(1))
    with pytest.raises(ValueError):
        F.KVCache(t(2, 1, 16, 32, dtype=torch.uint8), None, None, None, None, None, fmt="mxfp4")
    with pytest.raises(ValueError):
        F.KVCache(t(2, 16, 32, dtype=torch.uint8), None, None, None, None, None)


def test_buffers_of_a_call_on_another_stream_are_that_streams(L, monkeypatch):
    """What a call with stream= allocates (outputs and workspace) comes from that
    stream's memory, and the current stream's use of the outputs is recorded."""
    inside, theirs, mine, recorded, calls = [], [], [], [], []

    class On:
        def __init__(self, stream):
            assert stream == "side"

        def __enter__(self):
            inside.append(1)

        def __exit__(self, *_):
            inside.pop()

    def watch(make):
        def f(*a, **kw):
            t = make(*a, **kw)
            (theirs if inside else mine).append(t)
            return t
        return f

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "new_empty", watch(torch.Tensor.new_empty))
    monkeypatch.setattr(torch, "empty_like", watch(torch.empty_like))
    monkeypatch.setattr(torch, "empty", watch(torch.empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(kv, "_call", lambda cache, what, fn, stream, args: calls.append((what, stream, args)))

    class Cache:
        heads, head_dim, page_size, _dev, _fmt, _ref, _scale = 1, 64, 16, -1, 0, None, 0.125

    c, i32 = Cache(), torch.int32
    x, slots = torch.zeros(3, 1, 64, dtype=torch.bfloat16), torch.arange(3)
    pos, table = torch.zeros(3, dtype=i32), torch.zeros(4, 64)
    got = [kv.kv_append(c, x, x, slots, pos, table, q=x, stream="side")]
    got += kv.kv_read(c, slots, stream="side")
    got += kv.kv_attention(c, x, torch.tensor([0, 3], dtype=i32), torch.zeros(1, 40, dtype=i32),
                           torch.zeros(1, dtype=i32), 3, return_lse=True, stream="side")
    assert [w for w, *_ in calls] == ["fos_kv_append", "fos_kv_read", "fos_kv_attention"]
    assert all(s == "side" for _, s, _ in calls) and not mine
    ptrs = {t.data_ptr() for t in theirs}
    workspace = calls[2][2][17]
    assert workspace in ptrs and all(any(t.data_ptr() <= g.data_ptr() < t.data_ptr() + t.nbytes for t in theirs)
                                     for g in got)
    assert set(recorded) == {(p, "current") for p in ptrs - {workspace}}


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_tables_whose_tokens_pass_32_bits_are_refused(L, page_size):
    """Up to the largest length that counts past the last token's tile still fit in 32 bits for."""
    c = _cache(page_size=page_size, codes_page_stride=1 << 14, scales_page_stride=1 << 11)
    most = ((1 << 31) - 65536) // page_size
    assert _attention(L, c, max_pages=most, batch=0) == 0
    for pages in (most + 1, (1 << 31) // page_size - 1, (1 << 31) // page_size):
        assert _attention(L, c, max_pages=pages) == SHAPE
        assert _attention(L, c, max_pages=pages, max_q=300, total=300) == SHAPE


def test_a_table_width_whose_product_wraps_is_refused(L):
    for pages in (1 << 60, (1 << 60) + 1, (1 << 63) - 1):
        assert _attention(L, max_pages=pages) == SHAPE


def test_the_fields_of_a_cache_are_fixed():
    """A tensor or format put in a field's place would not be the one that calls use."""
    c = object.__new__(F.KVCache)
    c.__dict__.update(k_tensor_scale=torch.ones(1), fmt="nvfp4_46", page_size=16)
    for name, value in (("k_tensor_scale", torch.zeros(1)), ("fmt", "nvfp4_6"), ("page_size", 32)):
        with pytest.raises(AttributeError):
            setattr(c, name, value)
    c.layer = 3                           # what is no field is the user's
    assert c.fmt == "nvfp4_46" and bool(c.k_tensor_scale == 1) and c.layer == 3
