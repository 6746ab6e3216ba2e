"""The key/value cache in 4 bits (mxfp4_block_scaled_fos_b200/kv.py): append
and read against the oracle bit for bit, attention against a 64-bit
computation on the same codes with the bound derived in kv_reference.py."""
import math

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fos_b200 as F
import kv_reference as R

from helpers import require_gpu

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _table(n, rot):
    angle = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _random_cache(pages, page, heads, dim, seed, gap=0):
    """A cache of quantized normal values; `gap` bytes of 16 between its pages."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed)
    ref = {}
    pools = []
    for name in "kv":
        x = torch.randn(pages * page, heads, dim, generator=g).to(torch.bfloat16)
        amax = np.array([5.1 + 0.37 * h for h in range(heads)], np.float32)
        c, s = R.quantize(x, amax, False)
        for y, kind in ((c, "c"), (s, "s")):
            y = np.ascontiguousarray(y.reshape(pages, page, heads, -1).transpose(0, 2, 1, 3))
            ref[name + kind] = y
            n = y[0].size
            whole = torch.full((pages, n + 16 * gap), 0xFF, dtype=torch.uint8, device=dev)
            t = whole[:, :n].unflatten(1, y.shape[1:])
            t.copy_(torch.from_numpy(y))
            pools.append(t)
        st = torch.from_numpy(amax) / 1792.0
        ref[name + "st"] = st.numpy()
        ref[name + "dev"] = st.to(dev)
    cache = F.KVCache(*pools, ref["kdev"], ref["vdev"])
    return cache, ref


@pytest.mark.parametrize("dim,page,rot,inter,fmt,tokens,heads,q_heads", [
    (128, 16, 128, False, "nvfp4_46", 1, 1, 1),
    (128, 16, 128, False, "nvfp4_46", 37, 8, 32),
    (128, 64, 64, False, "nvfp4_6", 130, 2, 3),
    (128, 128, 16, True, "nvfp4_46", 5, 3, 24),
    (64, 16, 64, True, "nvfp4_6", 33, 5, 5),
    (64, 32, 48, False, "nvfp4_46", 64, 1, 7),
    (64, 64, 16, False, "nvfp4_46", 1300, 2, 2),
    (64, 16, 0, False, "nvfp4_46", 50, 4, 0),
])
def test_append_and_read_match_the_oracle(dim, page, rot, inter, fmt, tokens, heads, q_heads):
    dev = require_gpu()
    g = torch.Generator().manual_seed(tokens + dim)
    n = -(-tokens // page) + 3
    k_amax = torch.rand(heads, generator=g) * 3 + 2
    cache = F.KVCache.empty(n, page, heads, dim, k_amax.to(dev), 2.9, fmt=fmt, device=dev)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    # one projection's output: tokens further apart than their heads
    x = (torch.randn(tokens, q_heads + 2 * heads + 1, dim, generator=g)).to(torch.bfloat16)
    x[0, -2:, :16] = 0
    q, k, v = x[:, :q_heads], x[:, q_heads:q_heads + heads], x[:, q_heads + heads:q_heads + 2 * heads]
    # 32-byte aligned rows, or (odd numbers of tokens) rows that are only 16-byte aligned
    pad = 8 * (tokens % 2)
    xd = torch.zeros(tokens, x.shape[1] * dim + pad, dtype=torch.bfloat16, device=dev)[:, pad:].unflatten(1, x.shape[1:])
    xd.copy_(x)
    qd, kd, vd = (xd[:, a:b] for a, b in ((0, q_heads), (q_heads, q_heads + heads),
                                          (q_heads + heads, q_heads + 2 * heads)))
    slots = torch.randperm(n * page, generator=g)[:tokens].to(torch.int64)
    slots[tokens // 2::5] = -1 - slots[tokens // 2::5]
    status = torch.zeros(1, dtype=I32, device=dev)
    kw, want_q, want_k = {}, q, k
    if rot:
        pos = torch.randint(0, 99, (tokens,), generator=g).to(I32)
        table = _table(99, rot)
        want_q, want_k = R.rotate(q, pos, table, inter), R.rotate(k, pos, table, inter)
        kw = dict(positions=pos.to(dev), cos_sin=table.to(dev), interleaved=inter, q=qd)
    got_q = F.kv_append(cache, kd, vd, slots.to(dev), status=status, **kw)
    if rot:
        assert torch.equal(got_q.cpu().view(torch.int16), want_q.view(torch.int16))
    else:
        assert got_q is None
    assert int(status) == 0
    live = slots >= 0
    assert int(live.sum()) == len(set(slots[live].tolist()))
    out_k, out_v = F.kv_read(cache, slots.to(dev))
    for want, amax, codes, scales, st, out in (
            (want_k, k_amax, cache.k_codes, cache.k_scales, cache.k_tensor_scale, out_k),
            (v, torch.full((heads,), 2.9), cache.v_codes, cache.v_scales, cache.v_tensor_scale, out_v)):
        c, s = R.quantize(want, amax.numpy(), fmt == "nvfp4_6")
        for mine, theirs in ((codes, c), (scales, s)):
            all_rows = np.full((n * page, heads, theirs.shape[-1]), 0xA5, np.uint8)
            all_rows[slots[live].numpy()] = theirs[live.numpy()]
            got = mine.transpose(1, 2).reshape(n * page, heads, -1).cpu().numpy()
            assert np.array_equal(got, all_rows)   # the other slots as they were
        st = st.cpu().numpy()
        y = (R.values(c, s).astype(np.float32) * st[:, None]).astype(np.float32)
        y[~live.numpy()] = 0
        assert torch.equal(out.cpu(), torch.from_numpy(y).to(torch.bfloat16))


def test_append_rotates_queries_in_place_and_reports_bad_indexes():
    dev = require_gpu()
    cache = F.KVCache.empty(2, 16, 2, 128, 4.0, 4.0, device=dev)
    cache.k_codes.fill_(7)
    x = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    xd, table = x.to(dev), _table(10, 128)
    pos = torch.tensor([3, 10, -1, 9], dtype=I32)     # 10 and -1 are outside the table
    slots = torch.tensor([5, 6, 7, 32])               # 32 is outside the pool
    status = torch.zeros(1, dtype=I32, device=dev)
    q = xd[:, :4]
    got = F.kv_append(cache, xd[:, 4:6], xd[:, 6:], slots.to(dev), pos.to(dev), table.to(dev), q=q, q_out=q,
                      status=status)
    assert got is q and int(status) == F.STATUS_INDEX
    want = x[:, :4].clone()
    ok = [0, 3]
    want[ok] = R.rotate(x[ok, :4], pos[ok], table, False)
    assert torch.equal(q.cpu().view(torch.int16), want.view(torch.int16))
    assert torch.equal(xd[:, 4:].cpu(), x[:, 4:])
    rows = cache.k_codes.transpose(1, 2).reshape(32, -1)
    assert bool((rows[[i for i in range(32) if i != 5]] == 7).all()) and not bool((rows[5] == 7).all())
    status.zero_()
    k, v = F.kv_read(cache, torch.tensor([32, 5, -1], device=dev), status=status)
    assert int(status) == F.STATUS_INDEX and not k[0].any() and not v[2].any() and bool(k[1].any())
    status.zero_()
    bad = xd.clone()
    bad[1, 6, 77] = math.inf
    F.kv_append(cache, bad[:, 4:6], bad[:, 6:], torch.arange(4, device=dev), status=status)
    assert int(status) == F.STATUS_NONFINITE


def _check(cache, ref, q, cu, pages, kv_len, causal=True, window=0, scale=None, max_q=None, **kw):
    dev = require_gpu()
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse, bound, lbound = R.attention(q, ref["kc"], ref["ks"], ref["vc"], ref["vs"], ref["kst"], ref["vst"],
                                          cu, pages, kv_len, causal, window, scale)
    status = torch.zeros(1, dtype=I32, device=dev)
    n = [b - a for a, b in zip(cu, cu[1:])]
    got, gl = F.kv_attention(cache, q.to(dev), torch.tensor(cu, dtype=I32, device=dev),
                             torch.as_tensor(np.asarray(pages), dtype=I32).to(dev),
                             torch.tensor(kv_len, dtype=I32, device=dev), max(n) if max_q is None else max_q,
                             causal=causal, window=window, scale=scale, return_lse=True, status=status, **kw)
    got, gl = got.cpu().double().numpy(), gl.cpu().double().numpy()
    assert int(status) == 0
    rows = slice(cu[0], cu[-1])
    off = np.abs(got - out)[rows] - bound[rows]
    assert np.isfinite(got[rows]).all() and (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:5])
    none = np.isinf(lse[rows])
    assert np.array_equal(np.isneginf(gl[rows]), none)
    assert (np.abs(gl[rows][~none] - lse[rows][~none]) <= lbound[rows][~none]).all()
    return got, gl


def _paged(kv_len, page, seed, spare=1):
    """A block table of distinct pages in random order, -1 beyond each length."""
    need = [-(-m // page) for m in kv_len]
    order = np.random.RandomState(seed).permutation(sum(need) + spare)
    table = np.full((len(kv_len), max(1, max(need) + 1)), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, sum(need) + spare


def _queries(total, heads, dim, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(total, heads, dim, generator=g) * gain).to(torch.bfloat16)


# ragged single tokens and drafts: q_heads / heads of 1 to 8, odd lengths, pages that end inside a tile
@pytest.mark.parametrize("dim,page,heads,group,q_len,kv_len,window", [
    (128, 16, 2, 4, [1, 1, 1], [1, 300, 17], 0),
    (128, 64, 1, 8, [1, 1], [129, 64], 0),
    (128, 128, 3, 1, [1, 1, 1, 1], [5, 1000, 16, 15], 0),
    (64, 32, 2, 3, [4, 1, 5], [40, 333, 5], 0),
    (64, 16, 1, 7, [2, 3], [700, 48], 100),
    (128, 16, 1, 16, [1, 2], [260, 31], 0),
    (128, 32, 2, 5, [3, 1], [90, 257], 33),
    (64, 64, 2, 4, [1] * 9, [9, 1, 2, 900, 64, 65, 63, 31, 33], 0),
])
def test_attention_single_tokens(dim, page, heads, group, q_len, kv_len, window):
    pages, n = _paged(kv_len, page, 3)
    cache, ref = _random_cache(n, page, heads, dim, 5, gap=1)
    cu = [0] + np.cumsum(q_len).tolist()
    _check(cache, ref, _queries(cu[-1], heads * group, dim, 7, 2.0), cu, pages, kv_len, window=window)


# prompts: lengths around the tiles' borders, a history, windows, a query longer than its keys
@pytest.mark.parametrize("dim,page,heads,group,q_len,kv_len,window,causal", [
    (128, 16, 1, 4, [130, 1, 64], [130, 40, 200], 0, True),
    (64, 64, 2, 1, [200], [200], 0, True),
    (128, 32, 1, 3, [45, 97], [333, 97], 50, True),
    (64, 16, 1, 5, [77, 0, 31], [256, 10, 31], 0, True),
    (64, 128, 2, 2, [40, 70, 33], [129, 0, 500], 0, False),
    (128, 64, 1, 1, [257], [255], 0, True),
    (64, 32, 1, 8, [60, 17], [30, 0], 0, True),
    (128, 16, 1, 1, [300], [383], 128, True),
    # long enough for several CTAs to share a row tile's tokens; one of the sequences is short, one empty
    (128, 64, 1, 2, [70, 3, 40], [2300, 5, 0], 0, True),
    (64, 16, 1, 3, [100], [1700], 600, True),
    (128, 128, 1, 1, [90, 66], [1290, 700], 0, False),
])
def test_attention_prompts(dim, page, heads, group, q_len, kv_len, window, causal):
    pages, n = _paged(kv_len, page, 4)
    cache, ref = _random_cache(n, page, heads, dim, 6)
    cu = [0] + np.cumsum(q_len).tolist()
    _check(cache, ref, _queries(cu[-1], heads * group, dim, 8, 2.0), cu, pages, kv_len, window=window, causal=causal)


@pytest.mark.parametrize("max_q", [1, 200])
def test_attention_leaves_other_rows_and_nan_stays_in_its_row(max_q):
    dev = require_gpu()
    kv_len, cu = [70, 0, 33], [2, 3, 5, 45]
    pages, n = _paged(kv_len, 16, 9)
    cache, ref = _random_cache(n, 16, 2, 64, 10)
    # what lies behind the last token of a page is garbage: NaN scales
    for b, m in enumerate(kv_len):
        if m % 16:
            for t in (cache.k_scales, cache.v_scales, cache.k_codes, cache.v_codes):
                t[int(pages[b, m // 16]), :, m % 16:] = 0xFF
    q = _queries(50, 4, 64, 11)
    out = torch.full((50, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((50, 4), 3.0, device=dev)
    _check(cache, ref, q, cu, pages, kv_len, out=out, lse=lse, max_q=max_q)
    edge = [0, 1, 45, 46, 47, 48, 49]
    assert bool((out[edge] == 3.0).all()) and bool((lse[edge] == 3.0).all())
    clean = out.clone()
    q[7, 1, 5] = math.nan
    q[9, 3, 0] = math.inf
    got = F.kv_attention(cache, q.to(dev), torch.tensor(cu, dtype=I32, device=dev),
                         torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev), max_q,
                         out=out.clone())
    # queries 7 and 9 of the last sequence see no key (33 keys, 40 queries): masked, so zeros; 30 sees some
    assert torch.equal(got, clean)
    q[30, 1, 5] = math.nan
    q[31, 3, 0] = -math.inf
    got = F.kv_attention(cache, q.to(dev), torch.tensor(cu, dtype=I32, device=dev),
                         torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev), max_q,
                         out=out.clone())
    assert bool(got[30, 1].isnan().all()) and bool(got[31, 3].isnan().all())
    got[30, 1], got[31, 3] = clean[30, 1], clean[31, 3]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("max_q", [1, 100])
def test_attention_reports_bad_pages_and_lengths(max_q):
    dev = require_gpu()
    cache, ref = _random_cache(4, 16, 1, 64, 12)
    q = _queries(3, 2, 64, 13)
    pages = np.array([[0, 1], [2, 99], [3, -7]], np.int32)
    cu = [0, 1, 2, 3]

    def run(pages, kv_len, cu):
        status = torch.zeros(1, dtype=I32, device=dev)
        out = F.kv_attention(cache, q.to(dev), torch.tensor(cu, dtype=I32, device=dev),
                             torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev), max_q,
                             status=status, out=torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev))
        return out, int(status)

    good, ok = run(pages, [32, 16, 16], cu)
    assert ok == 0
    out, bad = run(pages, [32, 20, 16], cu)     # page 99 holds visible tokens: they do not count
    assert bad == F.STATUS_INDEX and torch.equal(out, good)
    out, bad = run(pages, [32, 16, 32], cu)
    assert bad == F.STATUS_INDEX and torch.equal(out, good)
    out, bad = run(pages, [33, 16, -1], cu)     # clamped to the table, and to nothing
    assert bad == F.STATUS_INDEX and torch.equal(out[:2], good[:2]) and not out[2].any()
    for broken in ([0, 1, 4, 3], [0, 1, 0, 3], [-1, 1, 2, 3], [0, 1, 2, 9]):
        out, bad = run(pages, [32, 16, 16], broken)
        assert bad & F.STATUS_INDEX and bool(out.isfinite().all())


@pytest.mark.parametrize("max_q", [1, 100])
def test_attention_of_extreme_values(max_q):
    """Scores far apart, a dominant late key, tiny and huge queries, a zero query and zero scales."""
    dev = require_gpu()
    kv_len = [400]
    pages, n = _paged(kv_len, 16, 20)
    cache, ref = _random_cache(n, 16, 1, 128, 21)
    q = _queries(6, 8, 128, 22)
    q[0] *= 60.0
    q[1] *= 2.0 ** -100
    q[2] = 0
    q[3, :, ::2] *= 2.0 ** -30
    _check(cache, ref, q, [0, 6], pages, kv_len, max_q=max_q)
    _check(cache, ref, q[4:], [0, 2], pages, kv_len, scale=-0.3, max_q=max_q)
    _check(cache, ref, q[4:], [0, 2], pages, kv_len, scale=0.0, max_q=max_q)


def test_same_call_same_bits_and_another_stream():
    dev = require_gpu()
    kv_len, cu = [900, 33, 410], [0, 1, 2, 3]
    pages, n = _paged(kv_len, 16, 30)
    cache, _ = _random_cache(n, 16, 2, 128, 31)
    q = _queries(3, 8, 128, 32).to(dev)
    args = (cache, q, torch.tensor(cu, dtype=I32, device=dev), torch.from_numpy(pages).to(dev),
            torch.tensor(kv_len, dtype=I32, device=dev), 1)
    a = F.kv_attention(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [F.kv_attention(*args, stream=side) for _ in range(3)] + [F.kv_attention(*args) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, x) for x in got)


def test_decoding_steps_captured_and_replayed():
    """Append and attention of a growing batch, captured once and replayed:
    every step equals the same calls made outside a graph, and the last one
    the 64-bit computation."""
    dev = require_gpu()
    B, H, HQ, D, P = 3, 2, 8, 128, 16
    start, steps = [14, 0, 47], 4
    pages = np.array([[3, 1, 9, 8], [0, 6, 7, 2], [4, 10, 5, 11]], np.int32)
    cu = torch.arange(B + 1, dtype=I32, device=dev)
    pd, table = torch.from_numpy(pages).to(dev), _table(100, D).to(dev)
    g = torch.Generator().manual_seed(40)
    x = torch.randn(steps, B, HQ + 2 * H, D, generator=g).to(torch.bfloat16).to(dev)

    def make():
        c, ref = _random_cache(12, P, H, D, 41)
        buf = {"x": torch.zeros_like(x[0]), "len": torch.tensor(start, dtype=I32, device=dev),
               "y": torch.zeros(B, HQ, D, dtype=torch.bfloat16, device=dev)}
        return c, buf

    def step(c, buf):
        pos = buf["len"].clone()
        at = pos.long()
        slots = pd.long().gather(1, (at // P)[:, None]).squeeze(1) * P + at % P
        q = F.kv_append(c, buf["x"][:, HQ:HQ + H], buf["x"][:, HQ + H:], slots, pos, table, q=buf["x"][:, :HQ])
        buf["len"] += 1
        F.kv_attention(c, q, cu, pd, buf["len"], 1, out=buf["y"])
        return q

    eager, be = make()
    want = []
    for i in range(steps):
        be["x"].copy_(x[i])
        q_last = step(eager, be)
        want.append(be["y"].clone())
    c, buf = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*make())                     # warm up outside the capture, on other buffers
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, buf)
    buf["len"].copy_(torch.tensor(start, dtype=I32))
    for i in range(steps):
        buf["x"].copy_(x[i])
        graph.replay()
        assert torch.equal(buf["y"], want[i]), i
    for a, b in ((c.k_codes, eager.k_codes), (c.v_scales, eager.v_scales)):
        assert torch.equal(a, b)
    np_ = lambda t: t.cpu().numpy()  # noqa: E731
    out, _, bound, _ = R.attention(q_last.cpu(), np_(c.k_codes), np_(c.k_scales), np_(c.v_codes), np_(c.v_scales),
                                   np_(c.k_tensor_scale), np_(c.v_tensor_scale), [0, 1, 2, 3], pages,
                                   [m + steps for m in start], True, 0, 1 / math.sqrt(D))
    assert (np.abs(np_(want[-1].double()) - out) <= bound).all()


def test_prompt_and_then_tokens_agree():
    """A prompt appended and attended in one call, and token by token, over
    the same cache: the same keys, so the same answers within both bounds."""
    dev = require_gpu()
    T, H, HQ, D, P = 75, 1, 4, 64, 32
    g = torch.Generator().manual_seed(50)
    x = torch.randn(T, HQ + 2 * H, D, generator=g).to(torch.bfloat16).to(dev)
    table = _table(T, D).to(dev)
    pages = torch.tensor([[2, 0, 1]], dtype=I32, device=dev)
    pos = torch.arange(T, dtype=I32, device=dev)
    slots = pages[0].long()[pos.long() // P] * P + pos.long() % P
    cache = F.KVCache.empty(3, P, H, D, 5.0, 5.0, device=dev)
    q = F.kv_append(cache, x[:, HQ:HQ + H], x[:, HQ + H:], slots, pos, table, q=x[:, :HQ])
    whole = F.kv_attention(cache, q, torch.tensor([0, T], dtype=I32, device=dev), pages,
                           torch.tensor([T], dtype=I32, device=dev), T)
    other = F.KVCache.empty(3, P, H, D, 5.0, 5.0, device=dev)
    rows, qs = [], []
    for i in range(T):
        s = slice(i, i + 1)
        qs.append(F.kv_append(other, x[s, HQ:HQ + H], x[s, HQ + H:], slots[s], pos[s], table, q=x[s, :HQ]))
        rows.append(F.kv_attention(other, qs[-1], torch.tensor([0, 1], dtype=I32, device=dev), pages,
                                   torch.tensor([i + 1], dtype=I32, device=dev), 1))
    assert torch.equal(torch.cat(qs), q)
    np_ = lambda t: t.cpu().numpy()  # noqa: E731
    out, _, bound, _ = R.attention(q.cpu(), np_(cache.k_codes), np_(cache.k_scales), np_(cache.v_codes),
                                   np_(cache.v_scales), np_(cache.k_tensor_scale), np_(cache.v_tensor_scale),
                                   [0, T], np_(pages), [T], True, 0, 1 / 8)
    for got in (whole, torch.cat(rows)):
        assert (np.abs(np_(got.double()) - out) <= bound).all()


def test_empty_calls():
    dev = require_gpu()
    cache = F.KVCache.empty(1, 16, 1, 64, 1.0, 1.0, device=dev)
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=dev)
    assert F.kv_append(cache, none, none, torch.empty(0, dtype=torch.int64, device=dev)) is None
    k, v = F.kv_read(cache, torch.empty(0, dtype=torch.int64, device=dev))
    assert k.shape == v.shape == (0, 1, 64)
    zero = torch.zeros(1, dtype=I32, device=dev)
    out = F.kv_attention(cache, none, zero, torch.empty(0, 3, dtype=I32, device=dev), zero[:0], 0)
    assert out.shape == (0, 1, 64)
    # a table without columns: no keys
    one = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=dev)
    out, lse = F.kv_attention(cache, one, torch.tensor([0, 1], dtype=I32, device=dev),
                              torch.empty(1, 0, dtype=I32, device=dev), zero, 1, return_lse=True)
    assert not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_q", [1, 200])
def test_one_key_gives_its_values_for_every_code(dim, max_q):
    """With a single visible key the answer is its values as kv_read gives
    them, bit for bit: every byte of codes in every place of a row."""
    dev = require_gpu()
    n = 256
    cache = F.KVCache.empty(n, 16, 2, dim, 3.0, 3.0, device=dev)
    byte = torch.arange(n, device=dev)[:, None] + torch.arange(dim // 2, device=dev) * 37
    for t in (cache.k_codes, cache.v_codes):
        t.copy_((byte % 256).to(torch.uint8)[:, None, None])
    for t in (cache.k_scales, cache.v_scales):
        t.copy_((torch.arange(n, device=dev) % 0x7f).to(torch.uint8)[:, None, None, None])
    slots = torch.arange(n, device=dev) * 16 + torch.arange(n, device=dev) % 16
    pages = torch.arange(n, dtype=I32, device=dev)[:, None].contiguous()
    kv_len = (torch.arange(n, device=dev) % 16 + 1).to(I32)
    q = _queries(n, 4, dim, 60).to(dev)
    got = F.kv_attention(cache, q, torch.arange(n + 1, dtype=I32, device=dev), pages, kv_len, max_q, window=1)
    want = F.kv_read(cache, slots)[1].repeat_interleave(2, 1)
    assert torch.equal(got, want)


# both kernels, whatever sizes would choose: max_q is a hint (a small one takes the kernel for few queries)
@pytest.mark.parametrize("max_q", [1, 1 << 20])
@pytest.mark.parametrize("dim,page,heads,group,q_len,kv_len,window,causal,gap", [
    (128, 16, 1, 4, [70, 1, 64], [130, 40, 200], 0, True, 1),
    (64, 64, 2, 1, [200, 3], [200, 700], 0, True, 3),
    (128, 32, 1, 3, [45, 97], [333, 97], 50, True, 0),
    (64, 16, 1, 5, [77, 0, 31], [256, 10, 31], 0, True, 0),
    (64, 128, 2, 2, [40, 70, 33], [129, 0, 500], 0, False, 1),
    (128, 64, 1, 2, [257], [255], 0, True, 0),
    (64, 32, 1, 8, [60, 17], [30, 0], 0, True, 2),
    (128, 64, 1, 2, [70, 3, 40], [2300, 5, 0], 0, True, 0),
    (64, 16, 1, 3, [100], [1700], 600, True, 1),
    (128, 128, 1, 1, [90, 66], [1290, 700], 0, False, 0),
    (128, 16, 2, 1, [1, 129, 1], [1, 129, 2], 1, True, 0),
])
def test_attention_by_either_kernel(dim, page, heads, group, q_len, kv_len, window, causal, gap, max_q):
    pages, n = _paged(kv_len, page, 14)
    cache, ref = _random_cache(n, page, heads, dim, 16, gap=gap)
    cu = [0] + np.cumsum(q_len).tolist()
    _check(cache, ref, _queries(cu[-1], heads * group, dim, 18, 2.0), cu, pages, kv_len, window=window, causal=causal,
           max_q=max_q)


@pytest.mark.parametrize("max_q", [1, 1 << 20])
def test_pages_far_apart(max_q):
    """Pools whose pages lie 2^32 - 16 bytes apart: offsets past 32 bits in all three operators."""
    dev = require_gpu()
    stride, n, page, heads, dim = (1 << 32) - 16, 3, 16, 2, 64
    whole = torch.empty(2 * stride + (1 << 20), dtype=torch.uint8, device=dev)
    pools = [torch.as_strided(whole, (n, heads, page, dim // d), (stride, page * dim // d, dim // d, 1), at << 14)
             for at, d in enumerate((2, 16, 2, 16))]
    st = torch.full((heads,), 5.0 / 1792.0, device=dev)
    far = F.KVCache(*pools, st, st)
    near = F.KVCache.empty(n, page, heads, dim, 5.0, 5.0, device=dev)
    near.k_tensor_scale.copy_(st)
    near.v_tensor_scale.copy_(st)
    g = torch.Generator().manual_seed(70)
    x = torch.randn(n * page, 2 * heads, dim, generator=g).to(torch.bfloat16).to(dev)
    slots = torch.arange(n * page, device=dev)
    for c in (far, near):
        F.kv_append(c, x[:, :heads], x[:, heads:], slots)
    for a, b in zip(F.kv_read(far, slots), F.kv_read(near, slots)):
        assert torch.equal(a, b)
    q = _queries(9, 4, dim, 71).to(dev)
    args = (q, torch.tensor([0, 2, 9], dtype=I32, device=dev),
            torch.tensor([[2, 0, 1], [1, 2, -1]], dtype=I32, device=dev), torch.tensor([47, 32], dtype=I32, device=dev),
            max_q)
    assert torch.equal(F.kv_attention(far, *args), F.kv_attention(near, *args))


@pytest.mark.parametrize("max_q", [1, 1 << 20])
def test_many_sequences(max_q):
    """More sequences than a block has threads, some empty: a bundle of single
    tokens equals the same sequences one at a time."""
    dev = require_gpu()
    B, page, dim = 611, 16, 64
    rng = np.random.RandomState(80)
    q_len = rng.randint(0, 3, B)
    kv_len = [int(m) for m in rng.randint(0, 60, B)]
    kv_len[7] = 400
    cache, _ = _random_cache(40, page, 1, dim, 81)
    pages = rng.randint(0, 40, (B, 25)).astype(np.int32)     # pages shared by sequences
    cu = np.concatenate(([0], np.cumsum(q_len))).astype(np.int32)
    q = _queries(int(cu[-1]), 2, dim, 82).to(dev)
    pd, ld = torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev)
    got, lse = F.kv_attention(cache, q, torch.from_numpy(cu).to(dev), pd, ld, max_q, return_lse=True)
    for b in list(range(0, B, 37)) + [7, B - 1]:
        if not q_len[b]:
            continue
        s = slice(int(cu[b]), int(cu[b + 1]))
        one, l1 = F.kv_attention(cache, q[s], torch.tensor([0, q_len[b]], dtype=I32, device=dev), pd[b:b + 1],
                                 ld[b:b + 1], 1, return_lse=True)
        # either answer is within 2^-8 of the other's bf16 and the weights' 2^-11 (values below 6)
        assert torch.allclose(got[s].float(), one.float(), rtol=2.0 ** -7, atol=6 * 2.0 ** -9), b
        assert torch.allclose(lse[s], l1, rtol=1e-5, atol=1e-4, equal_nan=True), b


@pytest.mark.parametrize("max_q", [1, 1 << 20])
def test_pages_before_a_window_are_not_read(max_q):
    dev = require_gpu()
    kv_len, n_q, window = [500], 6, 40
    pages, n = _paged(kv_len, 16, 90)
    cache, ref = _random_cache(n, 16, 1, 128, 91)
    q = _queries(n_q, 2, 128, 92)
    want, _ = _check(cache, ref, q, [0, n_q], pages, kv_len, window=window, max_q=max_q)
    gone = pages.copy()
    gone[0, :(500 - n_q + 1 - window) // 16] = 1 << 30       # would set the status
    status = torch.zeros(1, dtype=I32, device=dev)
    got = F.kv_attention(cache, q.to(dev), torch.tensor([0, n_q], dtype=I32, device=dev),
                         torch.from_numpy(gone).to(dev), torch.tensor(kv_len, dtype=I32, device=dev), max_q,
                         window=window, status=status)
    assert int(status) == 0 and np.array_equal(got.cpu().double().numpy(), want)


def test_calls_at_once_and_graphs_of_both_kernels():
    """Both kernels, with workspaces of their own, on two streams at once; and
    each captured, the graphs replayed in turn and at once."""
    dev = require_gpu()
    kv_len = [3000, 17, 900]
    pages, n = _paged(kv_len, 64, 100)
    cache, _ = _random_cache(n, 64, 2, 128, 101)
    pd, ld = torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev)
    calls = []
    for each, seed in ((1, 102), (90, 103)):
        q = _queries(3 * each, 8, 128, seed).to(dev)
        cu = torch.arange(4, dtype=I32, device=dev) * each
        assert F.kv_attention_workspace_size(cache, 3 * each, 3, 8, each, pages.shape[1]) > 0
        calls.append(lambda q=q, cu=cu, each=each: F.kv_attention(cache, q, cu, pd, ld, each, return_lse=True))
    want = [f() for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(4):
        for s, f in zip(streams, calls):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    for i, (y, l) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for y, l in outs:
            y.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for k, i in enumerate(order):
            with torch.cuda.stream(streams[k if order[0] != order[1] else 0]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_prompt_graph_follows_new_lengths():
    """A captured call of many queries serves other lengths and pages of the same shapes."""
    dev = require_gpu()
    cache, ref = _random_cache(40, 16, 1, 64, 110)
    cu = torch.tensor([0, 100, 130], dtype=I32, device=dev)
    pages, lens = torch.zeros(2, 40, dtype=I32, device=dev), torch.zeros(2, dtype=I32, device=dev)
    q = _queries(130, 4, 64, 111)
    qd = q.to(dev)
    F.kv_attention(cache, qd, cu, pages, lens, 1 << 20)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = F.kv_attention(cache, qd, cu, pages, lens, 1 << 20)
    for seed, n_cu, n_len in ((1, [0, 100, 130], [600, 30]), (2, [0, 30, 130], [10, 639]), (3, [0, 0, 130], [5, 200])):
        order = np.random.RandomState(seed).permutation(40).astype(np.int32)
        table = np.stack((order, order[::-1]))
        cu.copy_(torch.tensor(n_cu, dtype=I32))
        pages.copy_(torch.from_numpy(table.copy()))
        lens.copy_(torch.tensor(n_len, dtype=I32))
        g.replay()
        want, _, bound, _ = R.attention(q, ref["kc"], ref["ks"], ref["vc"], ref["vs"], ref["kst"], ref["vst"], n_cu,
                                        table, n_len, True, 0, 1 / 8)
        assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()


def test_binding_refusals():
    dev = require_gpu()
    c = F.KVCache.empty(4, 16, 2, 64, 1.0, 1.0, device=dev)
    bf = dict(dtype=torch.bfloat16, device=dev)
    k, slots = torch.zeros(3, 2, 64, **bf), torch.arange(3, device=dev)
    table, pos = _table(9, 64).to(dev), torch.zeros(3, dtype=I32, device=dev)
    append = lambda *a, **kw: F.kv_append(c, *a, **kw)  # noqa: E731
    for bad in ((k.float(), k, slots), (k.cpu(), k, slots), (k, k, slots.int()), (k, k, slots.cpu())):
        with pytest.raises(TypeError):
            append(*bad)
    for bad in ((k[:2], k, slots), (k, k, slots[:2]), (k[:, :1], k, slots), (k[..., :32], k, slots),
                (k.transpose(0, 1).contiguous().transpose(0, 1), k, slots)):
        with pytest.raises(ValueError):
            append(*bad)
    for kw in (dict(cos_sin=table), dict(positions=pos), dict(q=k), dict(q_out=k),
               dict(cos_sin=table, positions=pos[:2]), dict(cos_sin=table[0], positions=pos)):
        with pytest.raises(ValueError):
            append(k, k, slots, **kw)
    with pytest.raises(TypeError):
        append(k, k, slots, cos_sin=table.double(), positions=pos)
    with pytest.raises(F.FosError):
        append(k, k, slots, cos_sin=_table(9, 24).to(dev), positions=pos)
    with pytest.raises(TypeError):
        append(k, k, slots, status=torch.zeros(1, device=dev))
    q, cu = torch.zeros(3, 4, 64, **bf), torch.tensor([0, 3], dtype=I32, device=dev)
    pages, lens = torch.zeros(1, 2, dtype=I32, device=dev), torch.ones(1, dtype=I32, device=dev)
    att = lambda q=q, cu=cu, pages=pages, lens=lens, n=3, **kw: F.kv_attention(c, q, cu, pages, lens, n, **kw)  # noqa: E731
    att()
    for kw in (dict(q=q.half()), dict(cu=cu.long()), dict(pages=pages.long()), dict(lens=lens.float()),
               dict(lse=torch.zeros(3, 4, **bf))):
        with pytest.raises(TypeError):
            att(**kw)
    for kw in (dict(q=q[:, :3]), dict(q=q[0]), dict(pages=pages[0]), dict(lens=lens.expand(2)), dict(window=-1),
               dict(window=5, causal=False), dict(out=q[:2]), dict(cu=cu[:0]),
               dict(workspace=torch.zeros(1, dtype=torch.uint8, device=dev).expand(1 << 24))):
        with pytest.raises(ValueError):
            att(**kw)
    for kw in (dict(n=-1), dict(scale=math.nan), dict(workspace=torch.zeros(16, dtype=torch.uint8, device=dev))):
        with pytest.raises(F.FosError):
            att(**kw)
    with pytest.raises(ValueError):
        F.kv_read(c, slots, out=(k[:2], k))
    with pytest.raises(TypeError):
        F.kv_read(c, slots.int())


def test_a_buffer_longer_than_its_sequences_needs_no_workspace_for_the_rest():
    """Rows of no sequence (a padded buffer) do not make the workspace grow with the CTAs of a row."""
    cache = F.KVCache.empty(1, 64, 1, 128, 1.0, 1.0, device=require_gpu())
    size = lambda rows: F.kv_attention_workspace_size(cache, rows, 1, 8, 300, 1 << 12)  # noqa: E731
    assert 0 < size(300) and size(1 << 20) <= 4 * 148 * 256 * 130 * 4


# the kernel for many queries, one CTA for all tokens of its rows (no workspace): whole row tiles that see no key,
# of an empty sequence or of more queries than keys, beside others
@pytest.mark.parametrize("dim,page,heads,group,q_len,kv_len,causal", [
    (128, 64, 2, 2, [150, 400, 3, 260], [300, 0, 0, 500], False),
    (128, 16, 2, 1, [600, 150], [40, 860], True),
    (128, 128, 8, 4, [200, 129], [0, 0], False),
    (64, 32, 2, 2, [150, 400, 3, 260], [300, 0, 0, 500], False),
    (64, 16, 2, 1, [600, 150], [40, 860], True),
])
def test_rows_without_keys_in_every_run(dim, page, heads, group, q_len, kv_len, causal):
    dev = require_gpu()
    pages, n = _paged(kv_len, page, 120)
    cache, ref = _random_cache(n, page, heads, dim, 121)
    cu = [0] + np.cumsum(q_len).tolist()
    q = _queries(cu[-1], heads * group, dim, 122, 2.0)
    assert F.kv_attention_workspace_size(cache, cu[-1], len(q_len), heads * group, max(q_len), pages.shape[1]) == 0
    first, _ = _check(cache, ref, q, cu, pages, kv_len, causal=causal)
    none = torch.cat([torch.arange(m) < max(0, m - k) if causal else torch.full((m,), k == 0)
                      for m, k in zip(q_len, kv_len)]).to(dev)
    assert int(none.sum()) >= 256 // group
    args = (cache, q.to(dev), torch.tensor(cu, dtype=I32, device=dev), torch.from_numpy(pages).to(dev),
            torch.tensor(kv_len, dtype=I32, device=dev), max(q_len))
    first = torch.from_numpy(first).to(dev, torch.bfloat16)
    for _ in range(300):
        out, lse = torch.full_like(first, 3.0), torch.full((cu[-1], heads * group), 3.0, device=dev)
        F.kv_attention(*args, causal=causal, out=out, lse=lse)
        assert torch.equal(out, first) and not out[none].any() and bool((lse[none] == -math.inf).all())


@pytest.mark.parametrize("max_q", [1, 100])
def test_calls_that_overlap_share_no_buffers(max_q):
    """A call on another stream while one on the current stream still runs,
    with no wait between the streams: workspaces and outputs that the calls
    allocate are not the other's."""
    dev = require_gpu()
    kv_len = [4000, 3000]
    pages, n = _paged(kv_len, 64, 130)
    cache, _ = _random_cache(n, 64, 2, 128, 131)
    pd, ld = torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev)
    cu = torch.tensor([0, max_q, 2 * max_q], dtype=I32, device=dev)
    qs = [_queries(2 * max_q, 8, 128, 132 + i).to(dev) for i in range(2)]
    assert F.kv_attention_workspace_size(cache, 2 * max_q, 2, 8, max_q, pages.shape[1]) > 0
    call = lambda q, **kw: F.kv_attention(cache, q, cu, pd, ld, max_q, return_lse=True, **kw)  # noqa: E731
    slots = pd[0].long().clamp(min=0) * 64
    want = [call(q) for q in qs] + [F.kv_read(cache, slots)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = [call(qs[0]) if i % 2 == 0 else call(qs[1], stream=side) for i in range(6)]
        got.append(F.kv_read(cache, slots, stream=side))
        torch.cuda.synchronize()
        for i, pair in enumerate(got):
            for a, b in zip(pair, want[2 if i == 6 else i % 2]):
                assert torch.equal(a, b), i
    # outputs that are dropped while the current stream still reads them
    total = torch.zeros((), dtype=torch.float64, device=dev)
    for _ in range(50):
        y, _ = call(qs[1], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        total += y.double().sum()
        del y
    torch.cuda.synchronize()
    one = torch.zeros((), dtype=torch.float64, device=dev)
    for _ in range(50):
        one += want[1][0].double().sum()
    assert torch.equal(total, one)


@pytest.mark.parametrize("max_q", [1, 1 << 20])
@pytest.mark.parametrize("batch,broken", [
    (3, {1: 7}), (3, {3: 3}), (3, {2: 0, 3: 0}),       # outside; descending; a batch padded with zeros
    (32, {31: 7}), (32, {31: 70}), (32, {32: 5}), (33, {17: 0}), (33, {32: 5, 33: 5}),
    (700, {512: 3}), (700, {0: -1}), (700, {512: 4000}), (700, {i: 0 for i in range(300, 701)}),
])
def test_offsets_that_descend_or_leave_the_queries(batch, broken, max_q):
    """Such a sequence has no queries and the others are answered, unless they
    overlap and have more queries than there are: then none is. A status either way."""
    dev = require_gpu()
    cache, _ = _random_cache(3, 16, 2, 64, 140)
    good = list(range(0, 2 * batch + 2, 2))
    total = good[-1]
    q = _queries(total, 4, 64, 141).to(dev)
    pages = torch.zeros(batch, 2, dtype=I32, device=dev)
    lens = torch.full((batch,), 20, dtype=I32, device=dev)      # the same keys for every sequence

    def run(cu):
        status = torch.zeros(1, dtype=I32, device=dev)
        out = torch.full((total, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((total, 4), 3.0, device=dev)
        F.kv_attention(cache, q, torch.tensor(cu, dtype=I32, device=dev), pages, lens, max_q, causal=False, out=out,
                       lse=lse, status=status)
        return out, lse, int(status)

    want, want_lse, status = run(good)
    assert status == 0 and not bool((want == 3.0).all(2).any())
    cu = [broken.get(i, x) for i, x in enumerate(good)]
    kept = [range(x, y) for x, y in zip(cu, cu[1:]) if 0 <= x <= y <= total]
    rows = torch.zeros(total, dtype=torch.bool, device=dev)
    if sum(map(len, kept)) <= total:
        rows[[i for r in kept for i in r]] = True
    out, lse, status = run(cu)
    assert status == F.STATUS_INDEX
    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])
    assert bool((out[~rows] == 3.0).all()) and bool((lse[~rows] == 3.0).all())


@pytest.mark.parametrize("max_q", [1, 1 << 14])
def test_overlapping_sequences_whose_rows_pass_32_bits(max_q):
    """65537 sequences, every other one with all 2^24 rows: 2^39 rows, counted
    in 32 bits for a grid that has room for 2^24."""
    dev = require_gpu()
    batch, total, heads = 65537, 1 << 14, 1 << 10
    cache, _ = _random_cache(1, 16, 1, 64, 150)
    cu = torch.zeros(batch + 1, dtype=I32, device=dev)
    cu[1::2] = total
    q = torch.ones(total, heads, 64, dtype=torch.bfloat16, device=dev)
    out, status = torch.full_like(q, 3.0), torch.zeros(1, dtype=I32, device=dev)
    F.kv_attention(cache, q, cu, torch.zeros(batch, 1, dtype=I32, device=dev), torch.ones(batch, dtype=I32, device=dev),
                   max_q, out=out, status=status)
    assert int(status) == F.STATUS_INDEX and bool((out == 3.0).all())


@pytest.mark.parametrize("max_q", [1, 6, 1 << 20])
@pytest.mark.parametrize("dim,n_q,kv_len", [(128, 6, 4), (64, 6, 3), (64, 303, 41), (128, 1501, 1400)])
def test_a_query_without_keys_is_zero_beside_a_cached_nan(dim, n_q, kv_len, max_q):
    """NaN scales in the first token: the queries before it, in one row tile with others, still get 0 and -inf."""
    dev = require_gpu()
    pages, n = _paged([kv_len], 16, 160)
    cache, _ = _random_cache(n, 16, 1, dim, 161)
    for t in (cache.k_scales, cache.v_scales):
        t[int(pages[0, 0]), :, 0] = 0x7F
    out, lse = F.kv_attention(cache, _queries(n_q, 2, dim, 162).to(dev), torch.tensor([0, n_q], dtype=I32, device=dev),
                              torch.from_numpy(pages).to(dev), torch.tensor([kv_len], dtype=I32, device=dev), max_q,
                              return_lse=True)
    none = n_q - kv_len
    assert not out[:none].any() and bool(torch.isneginf(lse[:none]).all()) and bool(out[none:].isnan().all())


# many long sequences: a CTA walks tens of tiles of one item, past every reuse of a stage and of the page ids' window
@pytest.mark.parametrize("dim,page,heads,group,q_len,batch,longest,window,causal,gain", [
    (64, 16, 2, 8, 1, 128, 9000, 0, True, 2.0),        # 8 rows
    (128, 16, 2, 4, 2, 128, 9000, 0, True, 6.0),       # 8 rows, maxima that rise late
    (128, 64, 1, 3, 1, 200, 12000, 0, True, 2.0),      # 3 rows
    (64, 32, 1, 16, 1, 100, 12000, 0, True, 6.0),      # 16 rows
    (128, 16, 2, 4, 4, 60, 9000, 0, True, 2.0),        # 16 rows
    (128, 128, 1, 8, 4, 60, 9000, 0, True, 2.0),       # 32 rows in two tiles
    (64, 64, 2, 2, 3, 120, 9000, 7000, True, 6.0),     # a window over most of them
    (128, 32, 1, 9, 1, 120, 9000, 0, False, 2.0),
])
def test_attention_of_many_tiles_a_cta(dim, page, heads, group, q_len, batch, longest, window, causal, gain):
    dev = require_gpu()
    rng = np.random.RandomState(170)
    kv_len = [int(m) for m in rng.randint(longest // 2, longest, batch)]
    kv_len[batch // 3], kv_len[1], kv_len[2] = q_len, longest, 0 if not causal else q_len
    cache, ref = _random_cache(4096 // page, page, heads, dim, 171)
    pages = rng.randint(0, 4096 // page, (batch, -(-longest // page))).astype(np.int32)   # shared by sequences
    cu = np.arange(batch + 1) * q_len
    q = _queries(batch * q_len, heads * group, dim, 172, gain)
    status = torch.zeros(1, dtype=I32, device=dev)
    out, lse = F.kv_attention(cache, q.to(dev), torch.from_numpy(cu.astype(np.int32)).to(dev),
                              torch.from_numpy(pages).to(dev), torch.tensor(kv_len, dtype=I32, device=dev), q_len,
                              causal=causal, window=window, return_lse=True, status=status)
    assert int(status) == 0
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b in (0, 1, 2, batch // 3, batch // 2, batch - 1):
        s = slice(int(cu[b]), int(cu[b + 1]))
        want, wl, bound, lbound = R.attention(q[s], ref["kc"], ref["ks"], ref["vc"], ref["vs"], ref["kst"], ref["vst"],
                                              [0, q_len], pages[b:b + 1], kv_len[b:b + 1], causal, window,
                                              1 / math.sqrt(dim))
        assert (np.abs(out[s] - want) <= bound).all(), (b, (np.abs(out[s] - want) - bound).max())
        none = np.isinf(wl)
        assert np.array_equal(np.isneginf(lse[s]), none)
        assert (np.abs(lse[s][~none] - wl[~none]) <= lbound[~none]).all(), b


# more tokens than the grid has CTAs for, in place; more lanes than a CTA (64 + 8 + 8 heads); rows of 16 and 32
# bytes' alignment; half pairs that are not whole blocks apart at both head sizes
@pytest.mark.parametrize("dim,page,rot,inter,fmt,tokens,heads,q_heads,aligned", [
    (128, 64, 128, False, "nvfp4_46", 5001, 2, 4, 32),
    (128, 16, 128, True, "nvfp4_46", 4003, 2, 4, 32),
    (128, 16, 64, False, "nvfp4_46", 3001, 1, 8, 16),
    (64, 32, 64, False, "nvfp4_6", 6007, 2, 3, 16),
    (64, 64, 32, True, "nvfp4_46", 6001, 1, 1, 16),
    (128, 128, 128, False, "nvfp4_46", 2003, 8, 64, 32),
    (128, 16, 48, True, "nvfp4_46", 1501, 8, 64, 16),
    (128, 16, 0, False, "nvfp4_46", 5003, 2, 0, 32),
    (128, 32, 48, False, "nvfp4_46", 803, 2, 5, 16),
    (128, 32, 16, False, "nvfp4_6", 803, 3, 4, 32),
    (64, 32, 48, False, "nvfp4_46", 803, 2, 4, 32),
])
def test_append_of_many_tokens_in_place(dim, page, rot, inter, fmt, tokens, heads, q_heads, aligned):
    dev = require_gpu()
    g = torch.Generator().manual_seed(180 + tokens)
    n = -(-tokens // page) + 2
    cache = F.KVCache.empty(n, page, heads, dim, 3.3, 2.9, fmt=fmt, device=dev)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    x = torch.randn(tokens, q_heads + 2 * heads, dim, generator=g).to(torch.bfloat16)
    pad = aligned // 2 % 16
    xd = torch.zeros(tokens, x.shape[1] * dim + pad, dtype=torch.bfloat16, device=dev)[:, pad:].unflatten(1, x.shape[1:])
    xd.copy_(x)
    assert all(xd.data_ptr() % a == 0 for a in (16, aligned)) and (xd.stride(0) % 16 == 0) == (aligned == 32)
    slots = torch.randperm(n * page, generator=g)[:tokens].to(torch.int64)
    slots[3::7] = -1
    status = torch.zeros(1, dtype=I32, device=dev)
    want, kw = x.clone(), {}
    if rot:
        pos, table = torch.randint(0, 777, (tokens,), generator=g).to(I32), _table(777, rot)
        want[:, :q_heads + heads] = R.rotate(x[:, :q_heads + heads], pos, table, inter)
        kw = dict(positions=pos.to(dev), cos_sin=table.to(dev), interleaved=inter, q=xd[:, :q_heads],
                  q_out=xd[:, :q_heads])
    F.kv_append(cache, xd[:, q_heads:q_heads + heads], xd[:, q_heads + heads:], slots.to(dev), status=status, **kw)
    assert int(status) == 0
    assert torch.equal(xd[:, :q_heads].cpu().view(torch.int16), want[:, :q_heads].view(torch.int16))
    assert torch.equal(xd[:, q_heads:].cpu().view(torch.int16), x[:, q_heads:].view(torch.int16))
    live = slots >= 0
    for y, amax, codes, scales in ((want[:, q_heads:q_heads + heads], 3.3, cache.k_codes, cache.k_scales),
                                   (want[:, q_heads + heads:], 2.9, cache.v_codes, cache.v_scales)):
        c, s = R.quantize(y, np.full(heads, amax, np.float32), fmt == "nvfp4_6")
        for mine, theirs in ((codes, c), (scales, s)):
            rows = np.full((n * page, heads, theirs.shape[-1]), 0xA5, np.uint8)
            rows[slots[live].numpy()] = theirs[live.numpy()]
            assert np.array_equal(mine.transpose(1, 2).reshape(n * page, heads, -1).cpu().numpy(), rows)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("each,lens", [(1, [700, 33, 0]), (3, [700, 33, 5]), (90, [700, 33, 95]), (90, [3000, 5, 95])])
def test_strided_queries_and_outputs_and_a_callers_workspace(each, lens, dim):
    """Queries out of a wider projection, outputs into a wider buffer, a
    workspace that is larger than asked for and full of NaN: the same bits as
    with dense tensors, and nothing else written."""
    dev = require_gpu()
    B, H, HQ = 3, 2, 6
    pages, n = _paged(lens, 16, 190)
    cache, _ = _random_cache(n, 16, H, dim, 191)
    q = _queries(B * each, HQ, dim, 192).to(dev)
    args = (torch.arange(B + 1, dtype=I32, device=dev) * each, torch.from_numpy(pages).to(dev),
            torch.tensor(lens, dtype=I32, device=dev), each)
    want, wl = F.kv_attention(cache, q, *args, return_lse=True)
    wide = torch.full((B * each, (HQ + 5) * dim), 5.0, dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + HQ * dim] = q.flatten(1)
    out = torch.full((B * each + 2, (HQ + 1) * dim + 24), 3.0, dtype=torch.bfloat16, device=dev)
    mine = out[1:-1, 16:16 + HQ * dim].unflatten(1, (HQ, dim))
    size = F.kv_attention_workspace_size(cache, B * each, B, HQ, each, pages.shape[1])
    ws = torch.full((size // 4 + 64,), math.nan, device=dev)
    got, gl = F.kv_attention(cache, wide[:, 8:8 + HQ * dim].unflatten(1, (HQ, dim)), *args, out=mine, return_lse=True,
                             workspace=ws)
    assert got is mine and torch.equal(mine, want) and torch.equal(gl, wl)
    mine.fill_(3.0)
    assert bool((out == 3.0).all()) and bool(ws[size // 4:].isnan().all())


@pytest.mark.parametrize("max_q", [None, 1, 1 << 20])
def test_a_mixed_batch_in_one_call_or_two(max_q):
    """A prompt beside single tokens and drafts: one call, and two over parts of
    cu_q into the same outputs, each within the bound."""
    dev = require_gpu()
    q_len, kv_len = [150, 1, 3, 1, 0, 1], [210, 800, 33, 1, 5, 0]
    pages, n = _paged(kv_len, 32, 200)
    cache, ref = _random_cache(n, 32, 2, 128, 201)
    cu = [0] + np.cumsum(q_len).tolist()
    q = _queries(cu[-1], 6, 128, 202, 2.0)
    want, _ = _check(cache, ref, q, cu, pages, kv_len, max_q=max_q)
    qd, cd, pd = q.to(dev), torch.tensor(cu, dtype=I32, device=dev), torch.from_numpy(pages).to(dev)
    ld = torch.tensor(kv_len, dtype=I32, device=dev)
    out, lse = torch.empty_like(qd), torch.empty(cu[-1], 6, device=dev)
    F.kv_attention(cache, qd, cd[:2], pd[:1], ld[:1], 150, out=out, lse=lse)
    F.kv_attention(cache, qd, cd[1:], pd[1:], ld[1:], 3, out=out, lse=lse)
    exact, el, bound, lbound = R.attention(q, ref["kc"], ref["ks"], ref["vc"], ref["vs"], ref["kst"], ref["vst"], cu,
                                           pages, kv_len, True, 0, 1 / math.sqrt(128))
    assert (np.abs(out.cpu().double().numpy() - exact) <= bound).all()
    none = np.isinf(el)
    got = lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(got), none) and (np.abs(got[~none] - el[~none]) <= lbound[~none]).all()


def test_new_scales_are_copied_into_a_cache():
    dev = require_gpu()
    cache = F.KVCache.empty(1, 16, 2, 64, 1.0, 1.0, device=dev)
    with pytest.raises(AttributeError):
        cache.k_tensor_scale = torch.ones(2, device=dev)
    g = torch.Generator().manual_seed(210)
    x = (3 * torch.randn(16, 2, 64, generator=g)).to(torch.bfloat16)
    amax = np.array([11.0, 13.0], np.float32)
    cache.k_tensor_scale.copy_(torch.from_numpy(amax) / 1792.0)
    F.kv_append(cache, x.to(dev), x.to(dev), torch.arange(16, device=dev))
    codes, scales = R.quantize(x, amax, False)
    assert np.array_equal(cache.k_codes[0].transpose(0, 1).cpu().numpy(), codes)
    assert np.array_equal(cache.k_scales[0].transpose(0, 1).cpu().numpy(), scales)
