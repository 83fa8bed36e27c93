"""CPU oracles of the masked attention over a route and of the paged, quantised
cache -- TEST INFRASTRUCTURE ONLY, in fp64, from the definitions in
include/rr_attention.h and include/rr_cache.h.

Sums run over token positions with the number of times the route names each
(a repeated entry counts once per occurrence), so no expansion of the route is
shared with the kernels.
"""
from __future__ import annotations

import math

import numpy as np


def softmax_rows(x, count, v):
    """(out, lse, mean_abs): rows of softmax(x) v with key s counted
    count[t, s] times; mean_abs is the same mean of |v|.  Masked rows of v
    (count 0 for every t) may hold anything."""
    x = np.where(count > 0, x, -np.inf)
    top = x.max(axis=1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(invalid="ignore"):
        p = np.where(count > 0, np.exp(x - base[:, None]), 0.0) * count
    total = p.sum(axis=1)
    some = total != 0        # a NaN score makes the row NaN
    p = np.where(some[:, None], p / np.where(some, total, 1.0)[:, None], 0.0)
    clean = np.zeros_like(v)
    out = np.zeros((x.shape[0], v.shape[1]))
    mean = np.zeros_like(out)
    bad = ~np.isfinite(v).all(axis=1)
    clean[~bad] = v[~bad]
    out, mean = p @ clean, p @ np.abs(clean)
    for s in np.nonzero(bad)[0]:
        for t in np.nonzero(count[:, s] > 0)[0]:
            out[t] += p[t, s] * v[s]
    with np.errstate(divide="ignore"):
        lse = np.log(total) + base
    return out, lse, mean


def scores(q, k, scale, cap, slope, pos, key):
    """Logits of one head: q [t, dh], k [s, dh], positions of both."""
    with np.errstate(invalid="ignore"):
        x = q @ k.T * scale
    if cap:
        x = cap * np.tanh(x / cap)
    return x - slope * np.abs(pos[:, None] - key[None, :]) if slope else x


def masked_attention(q, k, v, route, chunk, causal=False, scale=None, soft_cap=0.0, slopes=None, doc_q=None,
                     doc_k=None, prefix=None, q_offset=0):
    """(out, lse, mean_abs) of q [b, hq, nq, dh], k and v [b, hkv, nk, dh],
    route [b, hr, query chunks, width], all fp64."""
    b, hq, nq, dh = q.shape
    hkv, nk = k.shape[1:3]
    hr = route.shape[1]
    scale = 1.0 / math.sqrt(dh) if scale is None else scale
    out, lse, mean = np.zeros((b, hq, nq, dh)), np.zeros((b, hq, nq)), np.zeros((b, hq, nq, dh))
    key = np.arange(nk)
    for ib in range(b):
        for h in range(hq):
            kh = h * hkv // hq
            for i in range(-(-nq // chunk)):
                t = np.arange(i * chunk, min(nq, (i + 1) * chunk))
                pos = t + q_offset
                count = np.zeros(nk)
                for j in route[ib, h * hr // hq, i]:
                    if j >= 0:
                        count[j * chunk:(j + 1) * chunk] += 1
                see = np.ones((t.size, nk), dtype=bool)
                if causal:
                    see = key[None, :] <= pos[:, None]
                    if prefix is not None:
                        see |= key[None, :] < prefix[ib]
                if doc_q is not None:
                    see &= (doc_q[ib, t][:, None] == doc_k[ib][None, :]) & (doc_q[ib, t][:, None] >= 0)
                x = scores(q[ib, h, t], k[ib, kh], scale, soft_cap, 0.0 if slopes is None else slopes[h], pos, key)
                out[ib, h, t], lse[ib, h, t], mean[ib, h, t] = softmax_rows(x, see * count, v[ib, kh])
    return out, lse, mean


# ---- the cache ---------------------------------------------------------------------

E4M3 = np.array([(1 if c < 128 else -1) * (np.nan if c & 127 == 127 else
                                           (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else
                                           (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def store_row(x, fmt):
    """(codes, scales) of one row of fp64 elements, one element at a time: the
    least power of two by trial, the nearest code with ties to the even one."""
    width, largest, values = (x.size, 448.0, E4M3[:127]) if fmt == "e4m3" else (32, 6.0, E2M1[:8])
    codes, scales = [], []
    for group in x.reshape(-1, width):
        if not np.isfinite(group).all():
            codes += [0] * width
            scales.append(255)
            continue
        e = -127
        while np.abs(group).max() > largest * 2.0 ** e:
            e += 1
        scales.append(e + 127)
        for y in group * 2.0 ** -e:
            gap = np.abs(values - abs(y))
            near = np.nonzero(gap == gap.min())[0]
            code = int(near[near % 2 == 0][0] if near.size > 1 else near[0])
            codes.append(code + ((len(values) + 1) // 8 * 8 if np.signbit(y) else 0))
    codes = np.array(codes, dtype=np.uint8)
    if fmt == "e2m1":
        codes = codes[0::2] | codes[1::2] << 4
    return codes, np.array(scales, dtype=np.uint8)


def read_rows(codes, scales, fmt):
    """Values in fp64 of code rows [..., R] with scales [..., G]."""
    if fmt == "e4m3":
        y = E4M3[codes]
    else:
        y = E2M1[np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return y * np.repeat(s, y.shape[-1] // s.shape[-1], axis=-1)


def cached_attention(codes, scales, fmt, q, lens, table, route=None, scale=None, soft_cap=0.0, slopes=None):
    """(out, lse, mean_abs) of q [b, qt, hq, dh] over the cache."""
    b, qt, hq, dh = q.shape
    heads, chunk = codes.shape[1], codes.shape[3]
    scale = 1.0 / math.sqrt(dh) if scale is None else scale
    out, lse, mean = np.zeros(q.shape), np.full((b, qt, hq), -np.inf), np.zeros(q.shape)
    for ib in range(b):
        n = max(0, min(int(lens[ib]), table.shape[1] * chunk))
        if n == 0:
            continue
        key = np.arange(n)
        pos = int(lens[ib]) - qt + np.arange(qt)
        page = table[ib, key // chunk]
        there = (page >= 0) & (page < codes.shape[0])
        at = np.where(there, page, 0)
        for h in range(heads):
            if codes.shape[0] == 0:
                continue
            k = read_rows(codes[at, h, 0, key % chunk], scales[at, h, 0, key % chunk], fmt)
            v = read_rows(codes[at, h, 1, key % chunk], scales[at, h, 1, key % chunk], fmt)
            times = np.ones(n)
            if route is not None:
                times[:] = 0
                for j in route[ib, h]:
                    if j >= 0:
                        times[j * chunk:(j + 1) * chunk] += 1
            count = (key[None, :] <= pos[:, None]) * (times * there)[None, :]
            for i in range(h * (hq // heads), (h + 1) * (hq // heads)):
                x = scores(q[ib, :, i], k, scale, soft_cap, 0.0 if slopes is None else slopes[i], pos, key)
                out[ib, :, i], lse[ib, :, i], mean[ib, :, i] = softmax_rows(x, count, v)
    return out, lse, mean
