"""Masked attention over a route (rr_masked_attention, include/rr_attention.h)
against the fp64 oracle (oracle/masked.py).

Tolerance, from the arithmetic: inputs are exact in fp32 and so is each product
q_d k_d; an fp32 sum of dh of them is off by at most dh 2^-24 of the sum of
their magnitudes, and scaling, cap and bias add a few roundings of the score:
    delta = 2^-24 (dh scale max sum |q_d k_d| + 8 max |x|)
(the cap's tanh is good to 2^-21 absolutely, hence cap 2^-21 more).  A weight is
then off by the factor e^delta at most, numerator and normaliser alike, and
rounded once to the inputs' type (half a step: eps / 2 of it; f16 weights below
2^-14 by at most 2^-25 of the largest weight); the result is rounded once:
    |o - o*| <= (2 delta + eps / 2) mean |v| + eps / 2 |o*| + n 2^-25 max |v| (f16)
with 2^-12 of slack on the first factor for the fp32 sums of weights.
The log of the sum: delta + 2^-21 (1 + |lse|).
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import masked as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def rr():
    import cross_layer_route_b200 as rr
    torch.cuda.set_device(0)
    return rr


def _np(x):
    return x.detach().double().cpu().numpy()


def make(b=2, hq=4, hkv=2, hr=None, nq=100, nk=None, dh=64, chunk=16, width=5, dtype=BF, seed=0, q_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    nk = nq if nk is None else nk
    hr = hkv if hr is None else hr
    mk = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    q = (torch.randn(b, hq, nq, dh, generator=g) * q_scale).to(dtype).to(DEV)
    k, v = mk(b, hkv, nk, dh), mk(b, hkv, nk, dh)
    nqc, nkc = -(-nq // chunk), max(1, -(-nk // chunk))
    route = torch.randint(-1, nkc + 1, (b, hr, nqc, width), generator=g, dtype=torch.int32)
    own = (torch.arange(nqc) * chunk + nk - nq).clamp(0) // chunk
    route[..., width // 2] = own.clamp(max=nkc - 1).int()
    return q, k, v, route.to(DEV)


def check(got, q, k, v, route, chunk, **kw):
    out, lse = got
    opt = {n: _np(x) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    qn, kn, vn = _np(q), _np(k), _np(v)
    ref, ref_lse, mean = M.masked_attention(qn, kn, vn, route.cpu().numpy(), chunk, **opt)
    eps = torch.finfo(q.dtype).eps
    dh, cap = q.shape[3], opt.get("soft_cap", 0.0)
    scale = opt.get("scale") or dh ** -0.5
    clean = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)
    a = max(((clean(qn[b, h]) @ clean(kn[b, h * kn.shape[1] // qn.shape[1]]).T).max(initial=0.0)
             for b in range(q.shape[0]) for h in range(q.shape[1])), default=0.0)
    delta = 2.0 ** -24 * (dh + 8) * scale * a + cap * 2.0 ** -21
    big = clean(vn).max(initial=0.0)
    bound = (2 * delta + eps / 2 + 2.0 ** -12) * mean + eps / 2 * np.abs(ref) + 1e-7
    if q.dtype == HF:
        bound = bound + route.shape[3] * chunk * 2.0 ** -25 * big
    o, s = _np(out), _np(lse)
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(o[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    err = np.abs(np.where(fine, o - ref, 0.0))
    assert (err <= np.where(fine, bound, 1.0)).all(), (err.max(), np.unravel_index(np.argmax(err - bound), err.shape))
    seen = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(s), np.isneginf(ref_lse))
    e = np.abs(np.where(seen, s - np.where(seen, ref_lse, 0.0), 0.0))
    assert (e <= delta + 2.0 ** -21 * (1 + np.abs(np.where(seen, ref_lse, 0.0)))).all(), e.max()
    assert (o[np.isneginf(ref_lse)] == 0).all()


def masks(kind, b, hq, nq, nk, seed=1):
    g = torch.Generator().manual_seed(seed)
    kw = {}
    if "c" in kind:
        kw.update(causal=True, q_offset=nk - nq)
    if "t" in kind:
        kw["soft_cap"] = 20.0
    if "s" in kind:
        kw["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]).to(DEV)
    if "d" in kind:
        doc = torch.sort(torch.randint(0, 3, (b, nk), generator=g), dim=1).values.int()
        doc[:, nk // 3:nk // 3 + 2] = -1
        kw["doc_k"] = doc.to(DEV)
        kw["doc_q"] = doc[:, nk - nq:].contiguous().to(DEV)
    if "p" in kind:
        kw["prefix"] = torch.randint(0, nk + 1, (b,), generator=g, dtype=torch.int32).to(DEV)
    return kw


SHAPES = [dict(), dict(nq=1, nk=1), dict(nq=1, nk=50, hq=8), dict(nq=33, nk=130, chunk=32, dtype=HF),
          dict(nq=200, chunk=64, dh=128, hq=8, width=3), dict(nq=129, nk=300, chunk=128, dh=128, dtype=HF, width=2),
          dict(nq=64, chunk=16, hq=3, hkv=1, b=1, dtype=HF), dict(nq=257, chunk=64, hq=4, hkv=1, b=1, width=7),
          dict(nq=140, chunk=32, dh=128, hq=16, hkv=2, b=1, width=40), dict(nq=96, chunk=16, hq=8, hkv=1, hr=4, b=1),
          dict(nq=150, nk=400, chunk=64, dh=128, hq=12, hkv=2, b=1, dtype=HF, width=4),
          dict(nq=70, chunk=128, hq=2, hkv=2, b=1, width=1), dict(nq=300, chunk=128, dh=128, hq=3, hkv=3, b=1, width=4)]


@pytest.mark.parametrize("kind", ["", "c", "ct", "cs", "cdp", "tsdp", "ctsdp"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_the_oracle(rr, shape, kind):
    s = SHAPES[shape]
    chunk = s.get("chunk", 16)
    q, k, v, route = make(seed=shape, q_scale=4.0 if "t" in kind else 1.0, **s)
    kw = masks(kind, q.shape[0], q.shape[1], q.shape[2], k.shape[2])
    check(rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw), q, k, v, route, chunk, **kw)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", [dict(chunk=16), dict(chunk=64, hq=8, hkv=2, dh=128, nq=190)])
def test_what_masked_rows_hold_is_not_read(rr, dtype, shape):
    q, k, v, route = make(dtype=dtype, b=1, seed=5, **shape)
    nq, chunk = q.shape[2], shape["chunk"]
    doc = torch.zeros(1, nq, dtype=torch.int32)
    doc[:, 40:47] = -1            # rows that nothing sees, in the middle of chunks
    doc[:, 70:] = 1
    k[:, :, 40:43], v[:, :, 40:43] = float("nan"), float("inf")
    k[:, :, 43:47], v[:, :, 43:47] = float("-inf"), float("nan")
    v[:, 0, 20, 3] = float("nan")                 # seen by later rows only, under the causal mask
    v[:, -1, 85, 7] = float("inf")
    kw = dict(doc_q=doc.to(DEV), doc_k=doc.to(DEV), causal=True)
    got = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
    check(got, q, k, v, route, chunk, **kw)
    assert torch.isfinite(got[0][:, :, :16]).all()


@pytest.mark.parametrize("chunk,hq,dh", [(16, 2, 64), (64, 4, 64), (64, 8, 128)])
def test_means_at_the_top_of_f16(rr, chunk, hq, dh):
    # weights of 2^6 (1 + 1.2 2^-11), which f16 rounds up to 2^6 (1 + 2^-10), and one of 2^7:
    # their product with values of 65504 over their sum is 65529, past the last number of f16
    q, k, v, _ = make(b=1, hq=hq, hkv=2, nq=64, nk=256, dh=dh, chunk=chunk, dtype=HF)
    route = torch.arange(256 // chunk, dtype=torch.int32).expand(1, 2, 64 // chunk, -1).contiguous().to(DEV)
    q.zero_()
    k.zero_()
    q[..., 0], k[:, :, 1:, 0] = 1.0, -1.0
    v.fill_(65504.0)
    v[..., 1::2] = -65504.0
    scale = math.log(2.0 / (1.0 + 1.2 * 2.0 ** -11))
    kw = dict(scale=scale)
    got = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
    assert torch.isfinite(got[0]).all()
    check(got, q, k, v, route, chunk, **kw)
    k[0, 0, 3, 0] = float("nan")      # a NaN is not a large number
    v[0, 1, 3, 1] = float("inf")
    got = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
    assert torch.isnan(got[0][:, :hq // 2]).all() and (got[0][:, hq // 2:, :, 1] == float("inf")).all()
    assert torch.isfinite(got[0][:, hq // 2:, :, 2:]).all()


@pytest.mark.parametrize("chunk,hq,dh", [(16, 2, 64), (64, 4, 64), (64, 8, 128)])
def test_means_at_the_top_of_bf16(rr, chunk, hq, dh):
    # sums of such values pass the last number of fp32, their means do not
    q, k, v, route = make(b=1, hq=hq, hkv=2, nq=130, dh=dh, chunk=chunk, seed=7)
    top = float(torch.finfo(BF).max)
    v.copy_(v.clamp(-3, 3) * 2.0 ** 126)
    v[:, :, 20:90] = top
    v[:, :, 20:90, 1::2] = -top
    v[:, :, :, 2] = 2.0 ** -100
    for kw in (dict(), dict(causal=True)):
        got = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
        assert torch.isfinite(got[0]).all() and (got[0][..., 2] <= 2.0 ** -100).all()
        check(got, q, k, v, route, chunk, **kw)


@pytest.mark.parametrize("chunk,hq,dh", [(16, 2, 64), (64, 4, 64), (64, 8, 128)])
def test_infinities_of_small_weights(rr, chunk, hq, dh):
    # a weight of 2^-120 times an infinity is one
    q, k, v, _ = make(b=1, hq=hq, hkv=2, nq=64, dh=dh, chunk=chunk)
    route = torch.arange(64 // chunk, dtype=torch.int32).expand(1, 2, 64 // chunk, -1).contiguous().to(DEV)
    q.zero_()
    k.zero_()
    q[..., 0], k[:, :, 9, 0] = 1.0, -120.0
    v[:, :, 9, 5], v[:, :, 9, 6] = float("inf"), float("-inf")
    kw = dict(scale=math.log(2.0))
    got = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
    check(got, q, k, v, route, chunk, **kw)
    assert (got[0][..., 5] == float("inf")).all() and (got[0][..., 6] == float("-inf")).all()


# units of one tile of 64 to 128 rows, whose tiles of 128 keys two groups of warps take in turn
ONE_TILE = [dict(nq=130, chunk=64, width=1), dict(nq=130, chunk=64, width=2), dict(nq=130, chunk=64, width=3),
            dict(nq=200, chunk=64, width=6, dtype=HF), dict(nq=200, nk=500, chunk=128, dh=128, hq=2, width=4),
            dict(nq=100, chunk=32, dh=128, hq=6, width=13, dtype=HF), dict(nq=90, chunk=16, hq=14, width=9),
            dict(nq=190, chunk=64, hq=2, dh=128, width=5), dict(nq=40, nk=700, chunk=16, hq=8, hkv=1, b=1, width=40),
            dict(nq=1, nk=300, chunk=128, hq=1, hkv=1, width=3)]


@pytest.mark.parametrize("kind", ["", "ct", "cs", "cdp", "ctsdp"])
@pytest.mark.parametrize("shape", range(len(ONE_TILE)))
def test_units_of_one_tile(rr, shape, kind):
    s = ONE_TILE[shape]
    q, k, v, route = make(seed=shape + 50, q_scale=4.0 if "t" in kind else 1.0, **s)
    kw = masks(kind, q.shape[0], q.shape[1], q.shape[2], k.shape[2])
    check(rr.masked_attention(q, k, v, route, s["chunk"], return_lse=True, **kw), q, k, v, route, s["chunk"], **kw)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", [dict(chunk=64, nq=190, width=3), dict(chunk=32, hq=8, dh=128, nq=190, width=9),
                                   dict(chunk=16, hq=12, nq=150, width=30)])
def test_what_masked_rows_hold_is_not_read_by_units_of_one_tile(rr, dtype, shape):
    test_what_masked_rows_hold_is_not_read(rr, dtype, shape)


def test_halves_of_a_row_that_see_nothing(rr):
    # of the unit's two tiles of keys the rows of one document see the first alone, of
    # the other the second, and of a third none; the tiles hold no numbers elsewhere
    q, k, v, _ = make(b=1, nq=64, nk=256, chunk=64, seed=9)
    doc_q = (torch.arange(64) % 3)[None].int().to(DEV)
    doc_k = torch.tensor([0] * 128 + [1] * 128)[None].int().to(DEV)
    route = torch.arange(4, dtype=torch.int32).expand(1, 2, 1, 4).contiguous().to(DEV)
    for spoil in (None, 0, 1):
        if spoil is not None:
            v[:, :, 128 * spoil + 5] = float("nan")
            k[:, :, 128 * spoil + 9] = float("inf")
        got = rr.masked_attention(q, k, v, route, 64, doc_q=doc_q, doc_k=doc_k, return_lse=True)
        check(got, q, k, v, route, 64, doc_q=doc_q, doc_k=doc_k)
        assert torch.count_nonzero(got[0][:, :, 2::3]) == 0
        if spoil == 0:
            assert torch.isfinite(got[0][:, :, 1::3]).all()


@pytest.mark.parametrize("hq", [1, 2])
def test_blocks_outlast_rows_computed_on_their_own(rr, hq):
    # the first unit's rows, at the widest route, meet a NaN in a value row that nobody sees
    # and take 1.3 s; the rest of their block's units, the last one among them, come after
    chunk, nqc, width, dh = 128, 149, 1024, 128
    q, k, v, _ = make(b=1, hq=hq, hkv=1, nq=nqc * chunk, nk=4 * chunk, dh=dh, chunk=chunk, seed=11)
    route = torch.full((1, 1, nqc, width), -1, dtype=torch.int32)
    route[:, :, 0] = torch.arange(width) % 4
    route[:, :, 1:, 0] = torch.arange(1, nqc) % 3 + 1
    doc = torch.zeros(1, 4 * chunk, dtype=torch.int32)
    doc[:, 5] = -1
    v[:, :, 5] = float("nan")
    kw = dict(doc_q=torch.zeros(1, nqc * chunk, dtype=torch.int32, device=DEV), doc_k=doc.to(DEV))
    got = rr.masked_attention(q, k, v, route.to(DEV), chunk, return_lse=True, **kw)
    assert torch.isfinite(got[0]).all()
    check(got, q, k, v, route, chunk, **kw)


def test_rows_that_see_nothing(rr):
    q, k, v, route = make(nq=50, nk=80)
    doc_q = torch.full((2, 50), 3, dtype=torch.int32, device=DEV)
    doc_k = torch.zeros((2, 80), dtype=torch.int32, device=DEV)
    cases = [dict(doc_q=doc_q, doc_k=doc_k), dict(width=0), dict(slopes=torch.ones(4, device=DEV), width=0)]
    for kw in cases:
        out, lse = rr.masked_attention(q, k, v, route, 16, return_lse=True, **kw)
        assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()
    none = k[:, :, :0]
    out, lse = rr.masked_attention(q, none, none, route, 16, return_lse=True)
    assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()
    assert rr.masked_attention(q[:, :, :0], k, v, route[:, :, :0].contiguous(), 16).shape == (2, 4, 0, 64)
    assert rr.masked_attention(q[:0], k[:0], v[:0], route[:0].contiguous(), 16).shape == (0, 4, 50, 64)


@pytest.mark.parametrize("shape", [dict(chunk=16), dict(chunk=64, hq=8, hkv=2, nq=128, dh=128)])
def test_repeated_entries_count_each_time(rr, shape):
    q, k, v, _ = make(b=1, seed=3, **shape)
    chunk = shape["chunk"]
    route = torch.tensor([1, 0, 1, 1, -1], dtype=torch.int32, device=DEV).expand(
        1, k.shape[1], -(-q.shape[2] // chunk), 5).contiguous()
    for kw in (dict(), dict(causal=True)):
        check(rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw), q, k, v, route, chunk, **kw)


@pytest.mark.parametrize("shape", [dict(chunk=16), dict(chunk=64, hq=8, hkv=2, dh=128)])
def test_bias_of_far_positions_keeps_the_scores(rr, shape):
    # every key is 2^23 positions away: slope * distance alone has a step of 1/2 in fp32
    q, k, v, route = make(b=1, nq=40, nk=128, width=8, seed=9, **shape)
    kw = dict(causal=True, q_offset=1 << 23, slopes=torch.full((q.shape[1],), 0.5, device=DEV))
    got = rr.masked_attention(q, k, v, route, shape["chunk"], return_lse=True, **kw)
    ref, lse, mean = M.masked_attention(_np(q), _np(k), _np(v), route.cpu().numpy(), shape["chunk"], causal=True,
                                        q_offset=1 << 23, slopes=[0.5] * q.shape[1])
    assert (np.abs(_np(got[0]) - ref) <= (2.0 ** -8 + 2.0 ** -12) * mean + 2.0 ** -8 * np.abs(ref) + 1e-7).all()
    # the documents hide the near chunk: the nearest visible key is what counts
    doc = torch.zeros(1, 128, dtype=torch.int32, device=DEV)
    doc[:, 60:] = 7
    kw.update(doc_q=torch.zeros(1, 40, dtype=torch.int32, device=DEV), doc_k=doc)
    got = rr.masked_attention(q, k, v, route, shape["chunk"], return_lse=True, **kw)
    ref, lse, mean = M.masked_attention(_np(q), _np(k), _np(v), route.cpu().numpy(), shape["chunk"], causal=True,
                                        q_offset=1 << 23, slopes=[0.5] * q.shape[1],
                                        doc_q=np.zeros((1, 40)), doc_k=_np(doc))
    assert (np.abs(_np(got[0]) - ref) <= (2.0 ** -8 + 2.0 ** -12) * mean + 2.0 ** -8 * np.abs(ref) + 1e-7).all()
    seen = np.isfinite(lse)
    assert np.abs(_np(got[1])[seen] / lse[seen] - 1).max(initial=0) < 2.0 ** -22


def test_strides_and_views(rr):
    b, hq, hkv, nq, dh, chunk = 2, 8, 2, 130, 64, 32
    _, _, _, route = make(b=b, hq=hq, hkv=hkv, nq=nq, dh=dh, chunk=chunk)
    g = torch.Generator().manual_seed(4)
    fused = torch.randn(b, nq, hq + 2 * hkv, dh, generator=g).to(BF).to(DEV)      # a fused projection
    q, k, v = (x.transpose(1, 2) for x in fused.split([hq, hkv, hkv], dim=2))
    got = rr.masked_attention(q, k, v, route, chunk, causal=True, return_lse=True)
    check(got, q, k, v, route, chunk, causal=True)
    flat = rr.masked_attention(q.contiguous(), k.contiguous(), v.contiguous(), route, chunk, causal=True)
    assert torch.equal(flat, got[0])
    # broadcast keys and queries, and a result inside a larger buffer whose other rows stay
    q1, k1 = q[:1].expand(b, -1, -1, -1), k[:, :1].expand(-1, hkv, -1, -1)
    room = torch.full((b, nq + 3, hq + 1, dh), 7.0, dtype=BF, device=DEV)
    out = room[:, 1:nq + 1, :hq].transpose(1, 2)
    got = rr.masked_attention(q1, k1, v, route, chunk, out=out, return_lse=True)
    assert got[0] is out
    check(got, q1, k1, v, route, chunk)
    assert (room[:, 0] == 7).all() and (room[:, nq + 1:] == 7).all() and (room[:, :, hq] == 7).all()


@pytest.mark.parametrize("chunk,group", [(16, 1), (64, 8)])
def test_strides_of_a_size_of_one(rr, chunk, group):
    q, k, v, route = make(b=1, hq=group, hkv=1, nq=1, dh=64, chunk=chunk)
    want = rr.masked_attention(q, k, v, route, chunk)
    odd = [x.as_strided(x.shape, (3, 64 if x.shape[1] > 1 else 5, 7, 1)) for x in (q, k, v)]
    out = torch.zeros(group, 64, dtype=q.dtype, device=DEV)
    rr.masked_attention(*odd, route, chunk, out=out.as_strided((1, group, 1, 64), (9, 64, 11, 1)))
    assert torch.equal(out, want.view(group, 64)) and out.any()


@pytest.mark.parametrize("shape", [dict(chunk=16), dict(chunk=64, hq=8, hkv=2, dh=128)])
def test_streams_and_graphs(rr, shape):
    q, k, v, route = make(seed=2, nq=150, **shape)
    chunk = shape["chunk"]
    want = rr.masked_attention(q, k, v, route, chunk, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rr.masked_attention(q, k, v, route, chunk, causal=True, stream=side)
    handle = rr.masked_attention(q, k, v, route, chunk, causal=True, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(handle, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = rr.masked_attention(q, k, v, route, chunk, causal=True, return_lse=True)
    q.copy_(torch.randn_like(q))
    graph.replay()
    torch.cuda.synchronize()
    check((out, lse), q, k, v, route, chunk, causal=True)


FIRST_CALLS = """
import threading
import torch
import cross_layer_route_b200 as rr
torch.cuda.set_device(0)
g = torch.Generator().manual_seed(1)
q, k, v = (torch.randn(1, 2, 256, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
route = torch.arange(2, dtype=torch.int32).expand(1, 2, 2, 2).contiguous().cuda()
torch.cuda.synchronize()
start, got = threading.Barrier(16), [None] * 16
def call(i):
    stream = torch.cuda.Stream()
    start.wait()
    got[i] = rr.masked_attention(q, k, v, route, 128, causal=True, return_lse=True, stream=stream)
threads = [threading.Thread(target=call, args=(i,)) for i in range(16)]
for t in threads:
    t.start()
for t in threads:
    t.join()
want = rr.masked_attention(q, k, v, route, 128, causal=True, return_lse=True)
torch.cuda.synchronize()
assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))
print("same bits")
"""


def test_first_calls_of_many_threads_give_the_same_bits():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        run = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=120)
        assert run.returncode == 0 and "same bits" in run.stdout, run.stderr[-2000:]


def test_two_calls_give_the_same_bits(rr):
    q, k, v, route = make(nq=300, hq=16, hkv=4, dh=128, chunk=64, width=6)
    first = rr.masked_attention(q, k, v, route, 64, causal=True, return_lse=True)
    for _ in range(3):
        again = rr.masked_attention(q, k, v, route, 64, causal=True, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype,dh,chunk,hq,hkv,nq,width", [(HF, 64, 32, 8, 8, 1301, 16), (BF, 128, 16, 4, 2, 3300, 24),
                                                            (BF, 64, 64, 4, 4, 1500, 24), (HF, 128, 16, 16, 16, 700, 20)])
@pytest.mark.parametrize("kind", ["", "ctsdp"])
def test_large_calls_equal_their_parts(rr, dtype, dh, chunk, hq, hkv, nq, width, kind):
    # units of under 128 rows: a large call copies its keys by TMA, its parts by
    # cp.async, and both compute the same sums in the same order
    b = 4
    q, k, v, route = make(b=b, hq=hq, hkv=hkv, nq=nq, dh=dh, chunk=chunk, width=width, dtype=dtype, seed=chunk)
    kw = masks(kind, b, hq, nq, nq)
    whole = rr.masked_attention(q, k, v, route, chunk, return_lse=True, **kw)
    for i in range(b):
        one = {n: x[i:i + 1].contiguous() if n in ("doc_q", "doc_k", "prefix") else x for n, x in kw.items()}
        part = rr.masked_attention(q[i:i + 1], k[i:i + 1], v[i:i + 1], route[i:i + 1].contiguous(), chunk, return_lse=True,
                                   **one)
        assert torch.equal(whole[0][i:i + 1], part[0]) and torch.equal(whole[1][i:i + 1], part[1])
    # broadcast keys and values, and rows of several heads side by side
    wide = torch.randn(b, nq, hkv, 2 * dh, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV).transpose(1, 2)
    k2, v2 = wide[:1, ..., :dh].expand(b, -1, -1, -1), wide[:, :1, :, dh:].expand(-1, hkv, -1, -1)
    whole = rr.masked_attention(q, k2, v2, route, chunk, causal=True)
    part = rr.masked_attention(q, k2.contiguous(), v2.contiguous(), route, chunk, causal=True)
    assert torch.equal(whole, part)


def test_overlapping_and_repeated_rows(rr):
    # keys that overlap one another (a window over a signal), one key for all tokens, queries likewise
    for hq, chunk in ((2, 16), (8, 64)):
        nq, dh = 100, 64
        _, _, _, route = make(b=1, hq=hq, hkv=2, nq=nq, chunk=chunk)
        signal = torch.randn(2, nq * 8 + dh, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
        k = signal.as_strided((1, 2, nq, dh), (0, signal.stride(0), 8, 1))
        v = signal[:, :dh].reshape(1, 2, 1, dh).expand(1, 2, nq, dh)
        q = signal[:1, :dh].reshape(1, 1, 1, dh).expand(1, hq, nq, dh)
        for args in ((q, k, k), (q, k, v), (k[:, :1].expand(1, hq, nq, dh), v, k)):
            got = rr.masked_attention(*args, route, chunk, causal=True, return_lse=True)
            check(got, *args, route, chunk, causal=True)


def test_agrees_with_the_plain_sparse_attention(rr):
    q, k, v, route = make(b=1, hq=4, hkv=4, nq=256, dh=128, chunk=64)
    a = rr.sparse_attention(q[0], k[0], v[0], route[0], 64, causal=True)
    out = rr.masked_attention(q, k, v, route, 64, causal=True)
    # both round the weights once; this one also the result
    mean = M.masked_attention(_np(q), _np(k), _np(v), route.cpu().numpy(), 64, causal=True)[2][0]
    assert (np.abs(_np(out[0]) - _np(a)) <= (2.0 ** -7 + 2.0 ** -11) * mean + 2.0 ** -8 * np.abs(_np(a)) + 1e-6).all()


def test_ledger_routes_in_place(rr):
    import rr_workloads as W
    from rr_parity import config_of
    w = W.C5.with_(bh=4, n=48, layers=1)
    led = rr.RouteLedger(config_of(w, rr), DEV)
    _, _, qs, ks = W.LayerStream(w, "cpu").next()
    led.layer(qs.to(DEV), ks.to(DEV), 0)
    nq = 48 * 16 - 5
    q, k, v, _ = make(b=2, hq=8, hkv=2, nq=nq, chunk=16)
    got = led.masked_attention(q, k, v, 16, soft_cap=25.0, return_lse=True)
    ids = led.read()["ids"][:, :, :w.k].reshape(2, 2, 48, w.k).contiguous().to(DEV)
    check(got, q, k, v, ids, 16, soft_cap=25.0, causal=bool(w.causal))
    with pytest.raises(ValueError):
        led.masked_attention(q, k, v, 16, causal=False)
    with pytest.raises(ValueError):
        led.masked_attention(q[:, :, :100], k, v, 16)
    with pytest.raises(ValueError):
        led.masked_attention(q, k, v, 16, route_heads=3)


def test_binding_refuses_wrong_tensors(rr):
    q, k, v, route = make()
    bad = [(q.float(), k, v, route), (q, k.half(), v, route), (q, k, v[:, :1], route), (q, k, v, route.long()),
           (q, k, v, route[:, :, :-1].contiguous()), (q.cpu(), k, v, route), (q, k, v, route.transpose(2, 3)),
           (q[..., ::2], k, v, route)]
    for args in bad:
        with pytest.raises(ValueError):
            rr.masked_attention(*args, 16)
    for kw in (dict(width=9), dict(slopes=torch.ones(3, device=DEV)), dict(doc_q=torch.zeros(2, 100, device=DEV)),
               dict(prefix=torch.zeros(3, dtype=torch.int32, device=DEV)), dict(out=torch.empty_like(q).float()),
               dict(doc_k=torch.zeros(2, 100, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rr.masked_attention(q, k, v, route, 16, **kw)
    odd = torch.zeros(2, 4, 100, 68, dtype=BF, device=DEV)[..., :64]      # rows 8 bytes off 16
    for kw in (dict(soft_cap=-1.0), dict(soft_cap=float("nan")), dict(scale=float("inf")), dict(q_offset=-1),
               dict(q_offset=1 << 24)):
        with pytest.raises(rr.RRError):
            rr.masked_attention(q, k, v, route, 16, **kw)
    with pytest.raises(rr.RRError):
        rr.masked_attention(odd, k, v, route, 16)
    with pytest.raises((rr.RRError, ValueError)):
        rr.masked_attention(q, k, v, route, 24)


def test_numbers_that_fit_no_field_are_refused(rr):
    q, k, v, route = make()
    for kw in (dict(q_offset=1 << 31), dict(q_offset=-(1 << 40)), dict(q_offset=2.5), dict(scale="1"), dict(soft_cap=10 ** 400)):
        with pytest.raises(ValueError):
            rr.masked_attention(q, k, v, route, 16, **kw)
    for kw in (dict(soft_cap=1e39), dict(scale=-1e300)):      # infinities in fp32
        with pytest.raises(rr.RRError):
            rr.masked_attention(q, k, v, route, 16, **kw)
