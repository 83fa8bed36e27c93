"""Host-side checks of the masked attention's and the cache's entry points
(include/rr_attention.h, include/rr_cache.h), and of their oracle against
closed forms.  No GPU needed: refused calls return before any CUDA call."""
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import cross_layer_route_b200 as rr
from oracle import masked as M

P = 0x7F00_0000_0000      # never dereferenced by these tests


def masked_cfg(**kw):
    base = dict(batch=2, q_heads=8, kv_heads=2, route_heads=4, nq_tokens=100, nk_tokens=100, dh=64, chunk=16, width=4,
                route_stride=8, causal=1, dtype=rr.RR_BF16, q_offset=0, scale=0.0, soft_cap=0.0, q_stride=(51200, 6400, 64),
                k_stride=(12800, 6400, 64), v_stride=(12800, 6400, 64), out_stride=(51200, 6400, 64))
    base.update(kw)
    c = rr.rr_masked_attn_config()
    for n, x in base.items():
        setattr(c, n, getattr(c, n).__class__(*x) if isinstance(x, tuple) else x)
    return c


def masked_args(**kw):
    base = dict(q=P, k=P, v=P, route=P, out=P)
    base.update(kw)
    return rr.rr_masked_attn_args(**base)


def refused(call, *args, status=None):
    with pytest.raises(rr.RRError) as e:
        call(*args)
    assert e.value.status == (rr.RR_EINVAL if status is None else status)


@pytest.mark.parametrize("bad", [
    dict(dh=96), dict(chunk=48), dict(kv_heads=0), dict(kv_heads=3), dict(route_heads=3), dict(route_heads=16),
    dict(nq_tokens=-1), dict(nk_tokens=-1), dict(batch=-1), dict(width=-1), dict(width=1025, route_stride=1025),
    dict(route_stride=3), dict(dtype=rr.RR_F32), dict(dtype=7), dict(q_offset=-1), dict(q_offset=(1 << 24) - 99),
    dict(nk_tokens=(1 << 24) + 1), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(soft_cap=-1.0),
    dict(soft_cap=1e-4), dict(soft_cap=math.inf), dict(soft_cap=math.nan), dict(q_stride=(51200, 6400, 60)),
    dict(k_stride=(-8, 6400, 64)), dict(v_stride=(1 << 41, 6400, 64)), dict(out_stride=(51200, 0, 64)),
    dict(batch=1 << 20, q_heads=1 << 16, kv_heads=1, route_heads=1 << 12),
    dict(batch=1, nq_tokens=1, q_heads=1 << 27, kv_heads=1, route_heads=1, chunk=128),      # 2^34 rows to a unit
])
def test_masked_attention_refuses_bad_shapes(bad):
    refused(rr.rr_masked_attention, masked_cfg(**bad), masked_args(), 0)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(v=0), dict(route=0), dict(out=0), dict(q=P + 8), dict(k=P + 2), dict(v=P + 4),
    dict(out=P + 8), dict(route=P + 2), dict(slopes=P + 1), dict(doc_q=P), dict(doc_k=P), dict(doc_q=P, doc_k=P + 2),
    dict(prefix=P + 3), dict(lse=P + 2),
])
def test_masked_attention_refuses_bad_pointers(bad):
    refused(rr.rr_masked_attention, masked_cfg(), masked_args(**bad), 0)


def test_strides_of_a_size_of_one_count_nothing():
    # looked at before the pointers, so that a call that gets past them is refused for its null ones
    odd = dict(q_stride=(-3, 7, 1), k_stride=(-3, 7, 1), v_stride=(-3, 7, 1), out_stride=(-3, 7, 1))
    one = masked_cfg(batch=1, q_heads=1, kv_heads=1, route_heads=1, nq_tokens=0, nk_tokens=1, **odd)
    rr.rr_masked_attention(one, masked_args(), 0)
    one.nk_tokens = 2
    refused(rr.rr_masked_attention, one, masked_args(), 0)
    pool = rr.rr_cache_pool(P, P)
    for call in (rr.rr_cache_write, rr.rr_cache_read):
        call(cache(heads=1), pool, rows(rows=1, batch=0), P, (-3, 7), P, (1, 1), rr.RR_BF16, 0)
        refused(call, cache(heads=1), pool, rows(rows=2, batch=0), P, (-3, 7), P, (64, 1), rr.RR_BF16, 0)
    rr.rr_cached_attention(cache(heads=1), pool, attn(batch=1, q_heads=1, q_tokens=0, q_stride=(-3, 9, 1)), attn_args(), 0, 0, 0)
    refused(rr.rr_cached_attention, cache(heads=1), pool, attn(batch=1, q_heads=2, q_tokens=0, q_stride=(-3, 9, 1)),
            attn_args(), 0, 0, 0)


@pytest.mark.parametrize("out", [(51200, 6400, 8), (51200, 64, 64), (6400, 6400, 64), (51200, 6392, 64), (51192, 6400, 64),
                                 (1 << 40, 1 << 40, 64)])
def test_masked_attention_refuses_results_on_top_of_one_another(out):
    refused(rr.rr_masked_attention, masked_cfg(out_stride=out), masked_args(), 0)


@pytest.mark.parametrize("none", ["batch", "nq_tokens"])
def test_masked_attention_takes_results_in_any_order(none):
    # two dimensions at a time: calls of nothing return after the check of the others' strides
    n0, n1, d0, d1 = (2, 8, 0, 1) if none == "nq_tokens" else (8, 100, 1, 2)
    for s0, s1 in ((64 * n1, 64), (64, 64 * n0), (64 * n1 + 8, 64), (72, 72 * n0), (1 << 40, 64), (64 * n1 - 8, 64), (64, 64),
                   (64, 64 * n0 - 8), (56, 1 << 20), (1 << 20, 8), (128, 192)):
        out = [8] * 3
        out[d0], out[d1] = s0, s1
        places = sorted(i * s0 + j * s1 for i in range(n0) for j in range(n1))
        apart = min(y - x for x, y in zip(places, places[1:])) >= 64
        cfg = masked_cfg(out_stride=tuple(out), **{none: 0})
        if apart:
            rr.rr_masked_attention(cfg, masked_args(), 0)
        else:
            refused(rr.rr_masked_attention, cfg, masked_args(), 0)


def test_masked_attention_with_nothing_to_do():
    rr.rr_masked_attention(masked_cfg(batch=0), masked_args(), 0)
    rr.rr_masked_attention(masked_cfg(nq_tokens=0), masked_args(q=0, out=0), 0)


def cache(**kw):
    base = dict(pages=10, heads=4, dh=64, chunk=16, format=rr.RR_E4M3)
    base.update(kw)
    return rr.rr_cache_config(**base)


def rows(**kw):
    base = dict(batch=2, rows=30, cu=P, start=P, page_table=P, table_width=3, table_stride=3)
    base.update(kw)
    return rr.rr_cache_rows(**base)


BAD_CACHES = [dict(pages=-1), dict(heads=0), dict(heads=65536), dict(dh=32), dict(chunk=8), dict(format=2)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches(bad):
    c, pool, s = cache(**bad), rr.rr_cache_pool(P, P), (256, 64)
    assert rr.rr_cache_codes_bytes(c) == 0 and rr.rr_cache_scales_bytes(c) == 0
    refused(rr.rr_cache_write, c, pool, rows(), P, s, P, s, rr.RR_BF16, 0)
    refused(rr.rr_cache_read, c, pool, rows(), P, s, P, s, rr.RR_BF16, 0)
    refused(rr.rr_cached_attention, c, pool, attn(), attn_args(), P, 1 << 40, 0)


def test_cache_sizes():
    assert rr.rr_cache_codes_bytes(cache()) == 10 * 4 * 2 * 16 * 64
    assert rr.rr_cache_scales_bytes(cache()) == 10 * 4 * 2 * 16
    assert rr.rr_cache_codes_bytes(cache(format=rr.RR_E2M1, dh=128, pages=1 << 20)) == (1 << 20) * 4 * 2 * 16 * 64
    assert rr.rr_cache_scales_bytes(cache(format=rr.RR_E2M1, dh=128)) == 10 * 4 * 2 * 16 * 4


def test_cache_rows_refusals():
    pool, s = rr.rr_cache_pool(P, P), (256, 64)
    for call in (rr.rr_cache_write, rr.rr_cache_read):
        for r in (rows(batch=-1), rows(rows=-1), rows(table_width=-1), rows(table_stride=2), rows(cu=0), rows(start=0),
                  rows(page_table=0), rows(cu=P + 2), rows(start=P + 1), rows(page_table=P + 2)):
            refused(call, cache(), pool, r, P, s, P, s, rr.RR_BF16, 0)
        refused(call, cache(), rr.rr_cache_pool(0, P), rows(), P, s, P, s, rr.RR_BF16, 0)
        refused(call, cache(), rr.rr_cache_pool(P, P + 4), rows(), P, s, P, s, rr.RR_BF16, 0)
        for k, ks in ((P + 8, s), (P, (256, 60)), (P, (-256, 64))):
            refused(call, cache(), pool, rows(), k, ks, P, s, rr.RR_BF16, 0)
            refused(call, cache(), pool, rows(), P, s, k, ks, rr.RR_BF16, 0)
        refused(call, cache(), pool, rows(), P, s, P, s, 3, 0)
        refused(call, cache(), pool, rows(), P, (256, 66), P, s, rr.RR_F32, 0)
        call(cache(), pool, rows(rows=0), P, s, P, s, rr.RR_BF16, 0)
        call(cache(), pool, rows(batch=0), P, s, P, s, rr.RR_BF16, 0)
    refused(rr.rr_cache_write, cache(), pool, rows(), None, s, P, s, rr.RR_BF16, 0)
    refused(rr.rr_cache_read, cache(), pool, rows(), P, (0, 64), P, s, rr.RR_BF16, 0)     # rows on top of one another
    rr.rr_cache_read(cache(), pool, rows(), None, s, None, s, rr.RR_BF16, 0)


def test_cache_read_refuses_results_on_top_of_one_another():
    # rows [30, 4] of 64; a call of no sequences returns after the check of the strides
    pool, s = rr.rr_cache_pool(P, P), (256, 64)
    for bad in ((248, 64), (64, 64), (192, 64), (64, 64 * 29), (256, 56), (56, 1 << 20), (128, 192)):
        for k, v in ((bad, s), (s, bad)):
            refused(rr.rr_cache_read, cache(), pool, rows(batch=0), P, k, P, v, rr.RR_BF16, 0)
        rr.rr_cache_write(cache(), pool, rows(batch=0), P, bad, P, bad, rr.RR_BF16, 0)      # read only: any
    for good in ((256, 64), (512, 64), (320, 72), (64, 64 * 30), (72, 72 * 30), (1 << 40, 64), (128, 128 * 29 + 64)):
        rr.rr_cache_read(cache(), pool, rows(batch=0), P, good, P, good, rr.RR_BF16, 0)
    rr.rr_cache_read(cache(heads=1), pool, rows(batch=0), P, (64, 0), P, (64, 8), rr.RR_BF16, 0)
    rr.rr_cache_read(cache(), pool, rows(rows=1, batch=0), P, (0, 64), P, (8, 64), rr.RR_BF16, 0)


def attn(**kw):
    base = dict(batch=2, q_tokens=1, q_heads=8, dtype=rr.RR_BF16, table_width=64, table_stride=64, width=0,
                route_stride=1, scale=0.0, soft_cap=0.0, q_stride=(512, 512, 64))
    base.update(kw)
    c = rr.rr_cached_attn_config()
    for n, x in base.items():
        setattr(c, n, getattr(c, n).__class__(*x) if isinstance(x, tuple) else x)
    return c


def attn_args(**kw):
    base = dict(q=P, seq_lens=P, page_table=P, out=P)
    base.update(kw)
    return rr.rr_cached_attn_args(**base)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=16384), dict(q_tokens=-1), dict(q_tokens=129), dict(q_heads=6), dict(q_heads=0),
    dict(dtype=rr.RR_F32), dict(table_width=-1), dict(table_stride=63), dict(table_width=1 << 21, table_stride=1 << 21),
    dict(width=-1), dict(width=4, route_stride=3), dict(route_stride=0), dict(scale=math.nan), dict(scale=-0.5),
    dict(soft_cap=-3.0), dict(soft_cap=math.inf), dict(q_stride=(512, 512, 63)), dict(q_stride=(-512, 512, 64)),
])
def test_cached_attention_refuses_bad_shapes(bad):
    assert rr.rr_cached_attention_workspace_bytes(cache(), attn(**bad), False) == 0
    refused(rr.rr_cached_attention, cache(), rr.rr_cache_pool(P, P), attn(**bad), attn_args(), P, 1 << 40, 0)


def test_cached_attention_refuses_bad_pointers_and_workspaces():
    pool = rr.rr_cache_pool(P, P)
    for bad in (dict(q=0), dict(q=P + 8), dict(out=0), dict(out=P + 2), dict(seq_lens=0), dict(seq_lens=P + 1),
                dict(page_table=0), dict(page_table=P + 2), dict(route=P + 2), dict(slopes=P + 1), dict(lse=P + 2)):
        refused(rr.rr_cached_attention, cache(), pool, attn(), attn_args(**bad), P, 1 << 40, 0)
    assert rr.rr_cached_attention_workspace_bytes(cache(), attn(), False) == 0     # a few blocks share a sequence
    long = attn(batch=1, table_width=4096, table_stride=4096)
    need = rr.rr_cached_attention_workspace_bytes(cache(), long, False)
    assert need > 0 and need % (8 * (64 + 4) * 4) == 0
    refused(rr.rr_cached_attention, cache(), pool, long, attn_args(), P, need - 1, 0, status=rr.RR_ENOMEM)
    refused(rr.rr_cached_attention, cache(), pool, long, attn_args(), P + 16, need, 0)
    refused(rr.rr_cached_attention, cache(), pool, long, attn_args(), 0, need, 0)
    refused(rr.rr_cached_attention, cache(), rr.rr_cache_pool(0, P), attn(), attn_args(), P, need, 0)
    rr.rr_cached_attention(cache(), pool, attn(batch=0), attn_args(), 0, 0, 0)
    rr.rr_cached_attention(cache(), pool, attn(q_tokens=0), attn_args(), 0, 0, 0)


def test_bindings_refuse_host_tensors():
    q = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    route = torch.zeros(1, 2, 1, 4, dtype=torch.int32)
    codes, scales = torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, 16, 1, dtype=torch.uint8)
    ints = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rr.masked_attention(q, q, q, route, 16)
    with pytest.raises(ValueError):
        rr.cache_write(codes, scales, q[0], q[0], ints, ints[:1], table)
    with pytest.raises(ValueError):
        rr.cache_read(codes, scales, ints, ints[:1], table, 2, 64)
    with pytest.raises(ValueError):
        rr.cached_attention(codes, scales, q, ints[:1], table)
    with pytest.raises(ValueError):
        rr.cache_empty(4, 2, 16, 64, fmt="int8")
    with pytest.raises(rr.RRError):
        rr.cache_empty(4, 2, 24, 64)


def test_cache_empty_takes_any_name_of_a_device(monkeypatch):
    named = []
    monkeypatch.setattr(rr.torch, "zeros", lambda shape, dtype, device: named.append(device))
    for device in (0, 1, "cuda:1", None):
        rr.cache_empty(1, 1, 16, 64, device=device)
    assert named == [0, 0, 1, 1, "cuda:1", "cuda:1", "cuda", "cuda"]


def test_a_ledger_refuses_chunks_of_no_tokens():
    ledger = SimpleNamespace(cfg=rr.Config(bh=2, nq=2, nk=2, d=64, k=2, m_near=0, r_rand=0))
    for chunk in (0, -16):
        with pytest.raises(ValueError):
            rr.RouteLedger._route_of(ledger, 2, chunk, 32, 32)


# ---- the oracle against closed forms ------------------------------------------------

def test_oracle_of_the_masked_attention():
    # equal keys: the mean of the visible values, and the log of their number plus the score
    q, k = np.ones((1, 1, 4, 64)), np.ones((1, 1, 40, 64))
    v = np.arange(40.0)[None, None, :, None] * np.ones(64)
    route = np.array([[[[0, 2, 2, -1, 9]]]])
    out, lse, _ = M.masked_attention(q, k, v, route, 16)
    keys = list(range(16)) + 2 * list(range(32, 40))
    assert np.allclose(out, np.mean(keys)) and np.allclose(lse, math.log(32) + 8)
    out, lse, _ = M.masked_attention(q, k, v, route, 16, causal=True, q_offset=2, soft_cap=4.0)
    assert np.allclose(out[0, 0, :, 0], [1, 1.5, 2, 2.5])
    assert np.allclose(lse[0, 0], np.log([3, 4, 5, 6]) + 4 * math.tanh(2))
    out, _, _ = M.masked_attention(q, k, v, route, 16, causal=True, prefix=np.array([40]))
    assert np.allclose(out, np.mean(keys))
    doc = np.zeros((1, 40))
    doc[:, 4:] = -1
    out, lse, _ = M.masked_attention(q, k, v, route, 16, doc_q=np.array([[0, 0, 1, -1]]), doc_k=doc,
                                     slopes=[math.log(2.0)])
    assert np.allclose(out[0, 0, 0, 0], (0 + 1 / 2 + 2 / 4 + 3 / 8) / (1 + 1 / 2 + 1 / 4 + 1 / 8))
    assert (out[0, 0, 2:] == 0).all() and np.isneginf(lse[0, 0, 2:]).all()


def test_oracle_of_the_cache_formats():
    y = M.E4M3[:127]
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double(), torch.tensor(y))
    rng = np.random.default_rng(0)
    for fmt, step in (("e4m3", 2.0 ** -4), ("e2m1", 2.0 ** -2)):
        x = rng.standard_normal(64)
        codes, scales = M.store_row(x, fmt)
        back = M.read_rows(codes, scales, fmt)
        top = np.repeat(np.abs(x.reshape(scales.size, -1)).max(axis=1), 64 // scales.size)
        assert (np.abs(back - x) <= np.maximum(step * np.abs(x), 2 ** -2 * top / 2)).all()
        assert (scales > 100).all()
        again = M.store_row(back, fmt)
        assert np.array_equal(M.read_rows(*again, fmt), back)
    assert np.isnan(M.read_rows(*M.store_row(np.array([np.inf] + [0.0] * 63), "e2m1"), "e2m1")[:32]).all()
