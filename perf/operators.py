"""The key/value cache operators, measured: append, read back, attention.

The cache holds keys and values of a decoder (or of an encoder, for cross
attention) in 4 bits: packed E2M1 codes with one E4M3 scale for each 16
values of a head and one FP32 scale for each head, in pages of `page` tokens.

  append     the position rotation of new queries and keys, and the new keys
             and values quantized into the cache; what the cache then holds
             for them is read back and returned with the rotated queries
  read       the keys and values of many slots, as bf16
  attention  ragged queries over the pages of their sequences, causal (with
             or without a sliding window) or over the whole of an encoder

A case's lengths follow from the case alone, its values and the order of its
pages from the seed.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HELD = 0.5 + 1.0 / 16   # bytes of the cache for each value


# ------------------------------------------------------------------ cases
def _append(name, tokens, q_heads, heads, dim, page, rot, interleaved, six, skip):
    c = {"op": "append", "tokens": tokens, "q_heads": q_heads, "heads": heads, "dim": dim, "page": page,
         "rot": rot, "interleaved": interleaved, "six": six, "skip": skip}
    return dict(c, name=name) if name else c


def _read(name, tokens, heads, dim, page):
    c = {"op": "read", "tokens": tokens, "heads": heads, "dim": dim, "page": page}
    return dict(c, name=name) if name else c


def _attention(name, batch, q_len, kv_len, even, q_heads, heads, dim, page, causal, window):
    c = {"op": "attention", "batch": batch, "q_len": q_len, "kv_len": kv_len, "even": even, "q_heads": q_heads,
         "heads": heads, "dim": dim, "page": page, "causal": causal, "window": window}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step of 64 sequences
        _append("append_step", 64, 32, 8, 128, 16, 128, False, False, 0),
        # a long prompt
        _append("append_prompt", 16384, 32, 8, 128, 64, 128, False, False, 0),
        # a padded batch of a model that rotates a part of each head, plain NVFP4
        _append("append_partial", 1237, 12, 3, 64, 32, 32, True, True, 13),
        # a shared prefix handed to another worker
        _read("read_prefix", 500, 8, 128, 16),
        # a long context handed over
        _read("read_long", 131072, 8, 128, 64),
        # one sequence, one token: latency
        _attention("decode_one", 1, 1, 1000, True, 32, 8, 128, 16, True, 0),
        # a serving batch of ragged contexts
        _attention("decode_batch", 64, 1, 16384, False, 32, 8, 128, 16, True, 0),
        # few long contexts, eight query heads for each key/value head
        _attention("decode_long", 4, 1, 131072, False, 64, 8, 128, 64, True, 0),
        # drafted tokens verified, odd heads, a sliding window
        _attention("verify_window", 48, 5, 5000, False, 15, 5, 64, 32, True, 1000),
        # a prompt
        _attention("prompt", 1, 8192, 8192, True, 32, 8, 128, 64, True, 0),
        # chunks of prompts behind their history, a sliding window
        _attention("chunks_window", 6, 1501, 6007, False, 20, 4, 64, 16, True, 2048),
        # a decoder's tokens over encoders of other lengths
        _attention("cross", 8, 448, 1500, False, 16, 16, 64, 64, False, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    dim = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    heads = rng.choice((1, 2, 3, 4, 5, 8))
    q_heads = heads * rng.choice((1, 2, 3, 4, 5, 7, 8))
    op = rng.choice(("append", "append", "read", "decode", "decode", "prompt", "prompt", "cross"))
    if op == "append":
        rot = rng.choice((dim, dim, dim // 2, dim // 4))
        return _append(None, _log(rng, 1, 16384), q_heads, heads, dim, page, rot, rng.random() < 0.5,
                       rng.random() < 0.3, rng.choice((0, 0, 7)))
    if op == "read":
        return _read(None, _log(rng, 1, 131072), heads, dim, page)
    if op == "decode":
        batch = _log(rng, 1, 128)
        most = min(131072, (1 << 29) // (batch * heads * dim))
        return _attention(None, batch, rng.choice((1, 1, 1, 2, 4)), _log(rng, 5, most), rng.random() < 0.3, q_heads,
                          heads, dim, page, True, rng.choice((0, 0, 300)))
    batch = _log(rng, 1, 8)
    kv_len = _log(rng, 40, int(8192 / math.sqrt(batch)))
    q_len = max(1, min(kv_len, _log(rng, 17, 8192)))
    q_heads = min(q_heads, 32 // heads * heads)
    return _attention(None, batch, q_len, kv_len, rng.random() < 0.3, q_heads, heads, dim, page, op == "prompt",
                      rng.choice((0, 0, 700)) if op == "prompt" else 0)


def _lengths(c):
    """(query tokens, cached tokens) of each sequence; the first is the longest, a ragged batch has an empty one."""
    b = c["batch"]
    if c["even"]:
        return [c["q_len"]] * b, [c["kv_len"]] * b
    r = random.Random("%d %d %d" % (b, c["q_len"], c["kv_len"]))
    q = [c["q_len"]] + [r.randint(1, c["q_len"]) for _ in range(b - 1)]
    kv = [c["kv_len"]] + [r.randint(1, c["kv_len"]) for _ in range(b - 1)]
    if c["causal"]:
        kv = [max(x, y) for x, y in zip(q, kv)]   # the queries' own keys are in the cache
    elif b > 1:
        kv[b // 2] = 0                            # an encoder that gave nothing
    return q, kv


def work(case):
    t, h, d = case.get("tokens", 0), case["heads"], case["dim"]
    if case["op"] == "append":
        kept = t - (t // case["skip"] if case["skip"] else 0)
        new = kept * h * d * 2
        return {"bytes": 4.0 * t * case["q_heads"] * d + new * 2 + new * HELD + new * HELD + new * 2
                + t * 12.0 + t * 4.0 * case["rot"],
                "flops": 3.0 * t * (case["q_heads"] + h) * case["rot"] + 20.0 * new}
    if case["op"] == "read":
        return {"bytes": t * h * d * 2 * (HELD + 2.0) + 8.0 * t, "flops": 4.0 * t * h * d}
    q, kv = _lengths(case)
    pairs = seen = 0
    for n, m in zip(q, kv):
        if not case["causal"]:
            pairs, seen = pairs + n * m, seen + m
            continue
        last = [m - n + 1 + i for i in range(n)]  # keys before and at each query
        w = case["window"] or m
        pairs += sum(min(x, w) for x in last)
        seen += m - max(0, last[0] - w)
    return {"bytes": sum(q) * case["q_heads"] * (4.0 * d + 4.0) + seen * h * d * 2 * HELD,
            "flops": 4.0 * pairs * case["q_heads"] * d}


# ------------------------------------------------------------- plain forms
def _e2m1(v):
    """Magnitude codes 0..7 of v >= 0: nearest, ties to even, saturating at 6."""
    c = (v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0)
    return c.to(torch.uint8)


def _try(w, s, st):
    """One candidate scale code (E4M3) of each block: codes with sign, and the squared error."""
    e = s.float() * st
    inv = torch.where(e == 0, torch.zeros_like(e), (1.0 / e).clamp(max=torch.finfo(torch.float32).max))
    code = _e2m1(w.abs() * inv)
    q = torch.tensor(E2M1, device=w.device)[code.long()]
    q = torch.where(torch.signbit(w), -q, q)
    d = (w.double() - q.double() * e.double()).float()   # one rounding
    t = d * d
    t = t[..., 0::2] + t[..., 1::2]
    t = t[..., 0::2] + t[..., 1::2]
    t = t[..., 0::2] + t[..., 1::2]
    return code + 8 * torch.signbit(w).to(torch.uint8), t[..., 0::2] + t[..., 1::2]


def _quantize(x, st, six):
    """bf16 x [tokens, heads, dim] -> packed codes and scale bytes; st [heads]."""
    w = x.float().unflatten(-1, (-1, 16))
    st = st[None, :, None, None]
    r = (w.abs().amax(-1, keepdim=True) / st).clamp(max=torch.finfo(torch.float32).max)
    s6 = (r / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    code, err = _try(w, s6, st)
    s = s6.view(torch.uint8)
    if not six:
        s4 = (r / 4.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        code4, err4 = _try(w, s4, st)
        code = torch.where(err4 < err, code4, code)
        s = torch.where(err4 < err, s4.view(torch.uint8), s)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.squeeze(-1)


def _values(codes, scales, st):
    """Packed codes [..., heads, dim/2] and scale bytes back to the 32-bit values that they stand for."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = scales.view(torch.float8_e4m3fn).float()
    return (grid[q].unflatten(-1, (-1, 16)) * s[..., None] * st[:, None, None]).flatten(-2)


def _rotate(x, cs, interleaved):
    """The first cs.shape[-1] values of each head rotated; x [tokens, heads, dim] bf16, cs [tokens, rot] (cos, sin)."""
    rot = cs.shape[-1]
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y = x.float()
    z, rest = y[..., :rot], y[..., rot:]
    a, b = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., : rot // 2], z[..., rot // 2:])
    u, v = a * c - b * s, b * c + a * s
    z = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((z, rest), -1).to(torch.bfloat16)


def _gather(codes, scales, page, offset):
    """Rows of a paged pool [pages, heads, page, n] at (page, offset), any shape: [..., heads, n]."""
    return codes[page, :, offset], scales[page, :, offset]


def _run_append(s):
    c = s["case"]
    k = _rotate(s["k"], s["table"][s["positions"].long()], c["interleaved"])
    q = _rotate(s["q"], s["table"][s["positions"].long()], c["interleaved"])
    at = (s["slots"] >= 0).nonzero().squeeze(1)
    page, off = s["slots"][at] // c["page"], s["slots"][at] % c["page"]
    for_k, for_ks = _quantize(k[at], s["k_st"], c["six"])
    for_v, for_vs = _quantize(s["v"][at], s["v_st"], c["six"])
    s["kc"][page, :, off], s["ks"][page, :, off] = for_k, for_ks
    s["vc"][page, :, off], s["vs"][page, :, off] = for_v, for_vs
    return q, *_run_read(s)


def _run_read(s):
    c = s["case"]
    empty = (s["slots"] < 0)[:, None, None]
    at = s["slots"].clamp(min=0)
    page, off = at // c["page"], at % c["page"]
    k = _values(*_gather(s["kc"], s["ks"], page, off), s["k_st"]).masked_fill(empty, 0.0)
    v = _values(*_gather(s["vc"], s["vs"], page, off), s["v_st"]).masked_fill(empty, 0.0)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _run_attention(s):
    c, cu, lens = s["case"], s["cu"].long(), s["lens"].long()
    b, h, g = c["batch"], c["heads"], c["q_heads"] // c["heads"]
    n, m = s["max_q"], s["max_kv"]
    j = torch.arange(m, device=cu.device)
    page = s["pages"][:, j // c["page"]].long().clamp(min=0)
    off = (j % c["page"])[None].expand(b, m)
    k = _values(*_gather(s["kc"], s["ks"], page, off), s["k_st"]).permute(0, 2, 3, 1)   # [b, h, d, m]
    v = _values(*_gather(s["vc"], s["vs"], page, off), s["v_st"]).permute(0, 2, 1, 3)   # [b, h, m, d]
    i = torch.arange(n, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (h, g)).permute(0, 2, 1, 3, 4)                 # [b, h, n, g, d]
    x = (q.reshape(b, h, n * g, -1) @ k).unflatten(2, (n, g)) * s["scale"]
    last = (lens - (cu[1:] - cu[:-1]))[:, None] + i if c["causal"] else (lens - 1)[:, None].expand(b, n)
    off = (j > last[..., None]) | (j >= lens[:, None, None])
    if c["window"]:
        off = off | (j <= last[..., None] - c["window"])
    x.masked_fill_(off[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    y = (p.flatten(2, 3) @ v).unflatten(2, (n, g)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + total.log()
    at, i = s["row_seq"], s["row_pos"]
    y = y.permute(0, 2, 1, 3, 4).flatten(2, 3)[at, i]
    return y.to(torch.bfloat16), lse.squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)[at, i]


# ----------------------------------------------------------- the operators
def _run_own(s):
    import mxfp4_block_scaled_fos_b200 as fos
    c = s["case"]
    if c["op"] == "append":
        q = fos.kv_append(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"], cos_sin=s["table"],
                          interleaved=c["interleaved"], q=s["q"])
        return q, *fos.kv_read(s["cache"], s["slots"])
    if c["op"] == "read":
        return fos.kv_read(s["cache"], s["slots"])
    return fos.kv_attention(s["cache"], s["q"], s["cu"], s["pages"], s["lens"], s["max_q"], causal=c["causal"],
                            window=c["window"], scale=s["scale"], return_lse=True)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _run_append(state) if op == "append" else _run_read(state) if op == "read" else _run_attention(state)


# ---------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _channels(g, heads, dim):
    """Keys have a few channels of larger values in each head, values hardly."""
    return 1.0 + 4.0 * (torch.rand(1, heads, dim, generator=g, device="cuda") < 0.03)


def _cache(g, c, pages):
    """Pools of `pages` pages filled with quantized values, with the scales of the heads."""
    h, d, p = c["heads"], c["dim"], c["page"]
    s = {}
    for name, gain in (("k", _channels(g, h, d)), ("v", torch.ones(1, h, d, device="cuda"))):
        most = (5.0 + torch.rand(h, generator=g, device="cuda")) * gain.amax((0, 2))   # a calibration's largest values
        st = most / (2688.0 if c.get("six") else 1792.0)
        codes = torch.empty(pages, h, p, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, h, p, d // 16, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 25) // (h * p * d))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = (_normal(g, n * p, h, d) * gain).to(torch.bfloat16)
            a, b = _quantize(x, st, c.get("six", False))
            codes[i:i + n] = a.unflatten(0, (n, p)).transpose(1, 2)
            scales[i:i + n] = b.unflatten(0, (n, p)).transpose(1, 2)
        s.update({name + "c": codes, name + "s": scales, name + "_st": st, name + "_gain": gain})
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, dev = dict(case), "cuda"
    h, d, page = c["heads"], c["dim"], c["page"]
    if c["op"] != "attention":
        t = c["tokens"]
        n = -(-t // page) + 2
        s = _cache(g, c, n)
        s["slots"] = torch.randperm(n, generator=g, device=dev)[:, None] * page + torch.arange(page, device=dev)
        s["slots"] = s["slots"].flatten()[1:t + 1].contiguous()
    else:
        q, kv = _lengths(c)
        t, most = sum(q), max(kv)
        need = [-(-m // page) for m in kv]
        s = _cache(g, c, sum(need) + 1)
        order = torch.randperm(sum(need) + 1, generator=g, device=dev).to(torch.int32)
        table = torch.full((len(q), max(1, max(need))), -1, dtype=torch.int32, device=dev)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at:at + m]
            at += m
        cu = torch.tensor([0] + q).cumsum(0)
        s |= {"pages": table, "cu": cu.to(torch.int32).to(dev), "lens": torch.tensor(kv, dtype=torch.int32, device=dev),
              "max_q": max(q), "max_kv": max(1, most), "scale": 1.0 / math.sqrt(d),
              "q": _normal(g, t, c["q_heads"], d).to(torch.bfloat16),
              "row_seq": torch.arange(len(q)).repeat_interleave(torch.tensor(q)).to(dev)}
        s["row_pos"] = torch.arange(t, device=dev) - s["cu"].long()[s["row_seq"]]
    if c["op"] == "append":
        qkv = _normal(g, t, c["q_heads"] + 2 * h, d)         # queries, keys and values of one projection
        qkv[:, c["q_heads"]:c["q_heads"] + h] *= s["k_gain"]
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv.split((c["q_heads"], h, h), 1)
        if c["skip"]:
            s["slots"][c["skip"] - 1::c["skip"]] = -1        # the batch's padding
        first = int(torch.randint(0, 1000, (1,), generator=g, device=dev))
        s["positions"] = (torch.arange(t, device=dev) + first).to(torch.int32)
        angle = torch.arange(t + 1000, dtype=torch.float64, device=dev)[:, None] * \
            10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    s["case"] = c
    if own:
        import mxfp4_block_scaled_fos_b200 as fos
        s["cache"] = fos.KVCache(s["kc"], s["ks"], s["vc"], s["vs"], s["k_st"], s["v_st"],
                                 fmt="nvfp4_6" if c.get("six") else "nvfp4_46")
    return s


# ------------------------------------------------------------- in 64 bits
def _nearest(x, grid):
    """The grid's value nearest to x >= 0 (ties to an even place), in 64 bits; grid ascending from 0."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    a, b = x - grid[hi - 1], grid[hi] - x
    down = (a < b) | ((a == b) & ((hi - 1) % 2 == 0))
    return torch.where(down, grid[hi - 1], grid[hi])


def _held(x, st, six):
    """What the cache holds for x [tokens, heads, dim] by the definition, in 64 bits."""
    e4m3 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    w = x.double().reshape(*x.shape[:2], -1, 16)
    t = st.double()[:, None, None]
    got = []
    for most in (6.0,) if six else (6.0, 4.0):
        e = _nearest(w.abs().amax(-1, keepdim=True) / t / most, e4m3) * t
        y = torch.sign(w) * _nearest(torch.where(e > 0, w.abs() / e, 0.0), e2m1) * e
        got.append((y, ((w - y) ** 2).sum(-1, keepdim=True)))
    y = got[0][0] if six else torch.where(got[1][1] < got[0][1], got[1][0], got[0][0])
    return y.reshape(x.shape)


def _turned(x, pos, table, interleaved):
    """Rotation as a product of complex numbers."""
    rot = table.shape[1]
    t = table.double()[pos.long()]
    unit = torch.complex(t[:, : rot // 2], t[:, rot // 2:])[:, None]
    z = x[..., :rot].double().reshape(*x.shape[:2], *((rot // 2, 2) if interleaved else (2, rot // 2)))
    pair = (z[..., 0], z[..., 1]) if interleaved else (z[..., 0, :], z[..., 1, :])
    y = torch.complex(*(p.contiguous() for p in pair)) * unit
    y = torch.stack((y.real, y.imag), -1 if interleaved else -2).flatten(-2)
    return torch.cat((y, x[..., rot:].double()), -1)


def _stored(codes, scales, st, slots, page):
    """The values of slots of a pool, in 64 bits."""
    rows, sc = codes.transpose(1, 2).flatten(0, 1)[slots], scales.transpose(1, 2).flatten(0, 1)[slots]
    n = torch.stack((rows % 16, rows // 16), -1).flatten(-2)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[(n % 8).long()]
    mag = torch.where(n >= 8, -mag, mag)
    return mag * (sc.view(torch.float8_e4m3fn).double() * st.double()[:, None]).repeat_interleave(16, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "read":
        return [_stored(s[n + "c"], s[n + "s"], s[n + "_st"], s["slots"], c["page"]) for n in "kv"]
    if c["op"] == "append":
        q = _turned(s["q"], s["positions"], s["table"], c["interleaved"])
        k = _turned(s["k"], s["positions"], s["table"], c["interleaved"]).to(torch.bfloat16)
        gone = (s["slots"] < 0)[:, None, None]
        return [q, _held(k, s["k_st"], c["six"]).masked_fill(gone, 0.0),
                _held(s["v"], s["v_st"], c["six"]).masked_fill(gone, 0.0)]
    q_len, kv_len = _lengths(c)
    g, at = c["q_heads"] // c["heads"], 0
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), []
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        j = torch.arange(m, device="cuda")
        slots = s["pages"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
        k, v = (_stored(s[x + "c"], s[x + "s"], s[x + "_st"], slots, c["page"]) for x in "kv")
        i = torch.arange(n, device="cuda")[:, None] + (m - n)
        seen = ((j <= i) & ((j > i - c["window"]) | (c["window"] == 0))) if c["causal"] else torch.ones(n, m, device="cuda").bool()
        one = []
        for h in range(c["q_heads"]):
            x = s["q"][at:at + n, h].double() @ k[:, h // g].T * s["scale"]
            x = x.masked_fill(~seen, -math.inf)
            one.append(torch.logsumexp(x, 1) if m else torch.full((n,), -math.inf, dtype=torch.float64, device="cuda"))
            w = (x - one[-1][:, None]).exp().nan_to_num(0.0)
            out[at:at + n, h] = w @ v[:, h // g]
        lse.append(torch.stack(one, 1))
        at += n
    return [out, torch.cat(lse)]
