"""The key/value cache operators in 64 bits, for the tests: numpy and the
oracle's quantizer only."""
from __future__ import annotations

import numpy as np
import torch

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)
E4M3 = np.array([oracle.e4m3_decode(c) for c in range(256)], np.float64)


def rotate(x: torch.Tensor, positions, table, interleaved: bool) -> torch.Tensor:
    """bf16 [T, H, D] turned by the definition's binary32 steps, then bf16."""
    y = x.float().numpy().copy()
    rot = table.shape[1]
    cs = table.numpy()[positions.numpy()][:, None, :]
    c, s = cs[..., : rot // 2], cs[..., rot // 2:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s      # float32 arrays: every step rounds
    y[..., ib] = b * c + a * s
    return torch.from_numpy(y).to(torch.bfloat16)


def quantize(x: torch.Tensor, amax: np.ndarray, six: bool):
    """bf16 [T, H, D] -> codes uint8 [T, H, D/2], scales [T, H, D/16] (the oracle, a head at a time)."""
    codes, scales = [], []
    for h in range(x.shape[1]):
        r = oracle.quantize(x[:, h].contiguous().view(torch.int16).numpy().view(np.uint16)[None],
                            fmt=1 if six else 0, amax_in=np.array([amax[h]], np.float32))
        codes.append(r["r_codes"][0])
        scales.append(r["r_scales"][0])
    return np.stack(codes, 1), np.stack(scales, 1)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """q * s in 64 bits: [..., D/2], [..., D/16] -> [..., D]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return E2M1[nib] * np.repeat(E4M3[scales], 16, axis=-1)


def attention(q, kc, ks, vc, vs, kst, vst, cu, pages, kv_len, causal, window, scale):
    """(out, lse, bound) in 64 bits for [total_q, Hq, D]; the bound is on
    |kernel - out| before and after its rounding to bf16.

    With n keys, e = 2^-24: a score sums D products (any order: D e times the
    sum of their magnitudes) and takes a few more roundings, and a query may
    be rounded to integers with its largest value in [2^22, 2^23), off by
    1/2 <= 2^-23 max |q| = 2 e max |q|, so a score is off by ds <=
    e |scale St| ((D + 8) sum |q k| + 2 max |q| sum |k|); its exponential by
    2 ds (score and maximum) + 2^-21 (exp2 and the reduced argument); a weight is rounded to f16 (2^-11, or 2^-25 of the largest
    where it is subnormal); the sums over n keys add n e.  The result is
    rounded to bf16 (2^-8)."""
    q = q.double().numpy()
    T, HQ, D = q.shape
    P, H = kc.shape[2], kc.shape[1]
    out = np.zeros((T, HQ, D))
    lse = np.full((T, HQ), -np.inf)
    bound = np.zeros((T, HQ, D))
    lbound = np.zeros((T, HQ))
    for b in range(len(kv_len)):
        n, m = int(cu[b + 1] - cu[b]), int(kv_len[b])
        j = np.arange(m)
        page, off = np.asarray(pages[b])[j // P].astype(np.int64), j % P
        for i in range(n):
            hi = m - n + i + 1 if causal else m
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            pg, of = page[lo:hi], off[lo:hi]
            for h in range(HQ):
                g = h * H // HQ
                k = values(kc[pg, g, of], ks[pg, g, of]) * float(kst[g])
                v = values(vc[pg, g, of], vs[pg, g, of]) * float(vst[g])
                x = k @ q[cu[b] + i, h] * scale
                top = x.max()
                p = np.exp(x - top)
                total = p.sum()
                p /= total
                t = cu[b] + i
                out[t, h] = p @ v
                lse[t, h] = top + np.log(total)
                ds = ((D + 8) * (np.abs(k) @ np.abs(q[t, h])) + 2 * np.abs(q[t, h]).max() * np.abs(k).sum(1)).max()
                ds *= 2.0 ** -24 * abs(scale)
                rel = 2 * ds + 2.0 ** -21 + (hi - lo) * 2.0 ** -23
                mag = p @ np.abs(v)
                bound[t, h] = (np.expm1(rel) + 2.0 ** -11) * mag * 1.01 + 2.0 ** -25 * np.abs(v).sum(0) / total
                bound[t, h] += 2.0 ** -8 * (np.abs(out[t, h]) + bound[t, h]) + 1e-37
                lbound[t, h] = rel + 2.0 ** -22 * abs(lse[t, h]) + 1e-6
    return out, lse, bound, lbound
