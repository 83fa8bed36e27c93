"""The paged, quantised cache and the attention over it (include/rr_cache.h)
against the fp64 oracle (oracle/masked.py).

Writing and reading are exact: the codes and scales have to equal the oracle's,
the values read back the stored ones rounded once to the output's type.

Attention, from the arithmetic: codes are exact in f16 and so are the queries
(scaled by a power of two); products are exact in fp32, their sum is off by at
most dh 2^-24 of the sum of magnitudes; scaling, cap and bias add a few
roundings of the score:  delta = 2^-24 (dh + 8) max sum |q k| scale + cap 2^-21.
Weights are rounded to f16 (2^-11), below 2^-21 of the largest weight * scale by
at most 2^-32 of it: n 2^-32 max |v| in all.  The result is rounded once:
    |o - o*| <= (2 delta + 2^-11 + 2^-12) mean |v| + eps / 2 |o*| + n 2^-32 max |v|
"""
import numpy as np
import pytest
import torch

from oracle import masked as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def rr():
    import cross_layer_route_b200 as rr
    torch.cuda.set_device(0)
    return rr


def _np(x):
    return x.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def table_of(need, pages, seed=0):
    """Pages in no order, one of each, -1 past a sequence's end."""
    order = np.random.default_rng(seed).permutation(pages)
    t = np.full((len(need), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def batch(lens, starts, chunk, extra=3, seed=0):
    need = [-(-(s + n) // chunk) for s, n in zip(starts, lens)]
    pages = sum(need) + extra
    cu = np.concatenate([[0], np.cumsum(lens)])
    return pages, cu, table_of(need, pages, seed)


def oracle_write(codes, scales, k, v, cu, start, table, fmt):
    chunk = codes.shape[3]
    for b in range(len(start)):
        for r in range(cu[b], cu[b + 1]):
            pos = start[b] + r - cu[b]
            if pos < 0 or pos // chunk >= table.shape[1]:
                continue
            page = table[b, pos // chunk]
            if not 0 <= page < codes.shape[0]:
                continue
            for h in range(codes.shape[1]):
                for w, x in ((0, k), (1, v)):
                    codes[page, h, w, pos % chunk], scales[page, h, w, pos % chunk] = M.store_row(x[r, h], fmt)


WRITES = [("e4m3", 64, 16, 1, BF, [3, 0, 20], [0, 5, 13]), ("e4m3", 128, 64, 3, HF, [70, 1], [60, 0]),
          ("e2m1", 64, 32, 2, FF, [1, 1, 1, 33], [31, 0, 2, 32]), ("e2m1", 128, 128, 5, BF, [5], [126]),
          ("e4m3", 64, 128, 9, FF, [2, 3], [0, 127]), ("e2m1", 128, 16, 8, HF, [18, 0, 0, 7], [0, 0, 3, 9])]


@pytest.mark.parametrize("fmt,dh,chunk,heads,dtype,lens,starts", WRITES)
def test_write_and_read(rr, fmt, dh, chunk, heads, dtype, lens, starts):
    pages, cu, table = batch(lens, starts, chunk)
    rows = int(cu[-1]) + 4                       # rows behind the last sequence
    g = torch.Generator().manual_seed(dh + heads)
    x = torch.randn(rows, 3, heads, dh, generator=g)
    x *= torch.exp2(torch.randint(-12, 12, (rows, 3, heads, 1), generator=g).float())
    x[0, :, 0] = 0.0
    x[1, 1:, 0, 3] = float("nan")
    x[2, 1:, heads - 1, dh - 1] = float("-inf")
    if dtype == FF:
        x[0, 1, 0, :4] = torch.tensor([1e-40, -1e-38, 0.0, 2e-45])
        x[1, 2, heads - 1, :3] = torch.tensor([3e38, -1.0, 1e30])
    x = x.to(dtype).to(DEV)
    k, v = x[:, 1], x[:, 2]                      # views of a fused projection
    codes, scales = rr.cache_empty(pages, heads, chunk, dh, fmt, DEV)
    codes.fill_(0x5A)
    scales.fill_(77)
    ref_c, ref_s = codes.cpu().numpy(), scales.cpu().numpy()
    args = (_i32(cu), _i32(starts), _i32(table))
    rr.cache_write(codes, scales, k, v, *args)
    oracle_write(ref_c, ref_s, _np(k), _np(v), cu, starts, table, fmt)
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    assert np.array_equal(codes.cpu().numpy(), ref_c)
    for out_type in (BF, HF, FF):
        room = torch.full((rows, heads + 1, 2, dh), 9.0, dtype=out_type, device=DEV)
        out = (room[:, :heads, 0], room[:, :heads, 1])
        got = rr.cache_read(codes, scales, *args, rows, dh, out_type, out=out)
        for w in (0, 1):
            for b in range(len(lens)):
                for r in range(cu[b], cu[b + 1]):
                    pos = starts[b] + r - cu[b]
                    at = (table[b, pos // chunk], slice(None), w, pos % chunk)
                    want = torch.tensor(M.read_rows(ref_c[at], ref_s[at], fmt)).to(FF).to(out_type)
                    assert torch.equal(got[w][r].cpu().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))
        assert (room[int(cu[-1]):] == 9).all() and (room[:, heads] == 9).all()
    kk, vv = rr.cache_read(codes, scales, *args, int(cu[-1]), dh, dtype)
    assert kk.shape == vv.shape == (int(cu[-1]), heads, dh)


def test_every_value_of_the_formats_and_every_tie(rr):
    # x / 2^e on each format's grid and half-way between, with the scale held by the largest value
    for fmt, values, dh in (("e4m3", M.E4M3[:127], 128), ("e2m1", M.E2M1[:8], 64)):
        mids = np.concatenate([values, (values[1:] + values[:-1]) / 2, -(values[1:] + values[:-1]) / 2])
        per = (dh if fmt == "e4m3" else 32) - 1
        rows = []
        for i in range(0, mids.size, per):
            part = np.zeros(per)
            part[:mids[i:i + per].size] = mids[i:i + per]
            rows.append(np.concatenate([[values[-1]], part]))
        if fmt == "e2m1":
            rows = [np.concatenate([r, rows[0]]) for r in rows]
        x = torch.tensor(np.array(rows)).float()[:, None].contiguous().to(DEV)
        n = x.shape[0]
        codes, scales = rr.cache_empty(1, 1, 16, dh, fmt, DEV)
        rr.cache_write(codes, scales, x, -x, _i32([0, n]), _i32([0]), _i32([[0]]))
        for r in range(n):
            for w, s in ((0, 1.0), (1, -1.0)):
                want = M.store_row(s * np.array(rows[r]), fmt)
                assert np.array_equal(codes[0, 0, w, r].cpu().numpy(), want[0])
                assert np.array_equal(scales[0, 0, w, r].cpu().numpy(), want[1])


def test_places_without_a_page(rr):
    chunk, dh, heads = 16, 64, 2
    codes, scales = rr.cache_empty(3, heads, chunk, dh, "e4m3", DEV)
    codes.fill_(0x11)
    table = _i32([[0, -1, 2], [7, 1, -5]])                       # 7: past the pool
    cu, start = _i32([0, 40, 60]), _i32([-4, 40])                # before position 0; past the table's end
    k = torch.ones(60, heads, dh, dtype=BF, device=DEV)
    before = codes.clone()
    rr.cache_write(codes, scales, k, k, cu, start, table)
    changed = (codes != before).any(-1).any(2).any(1).cpu().numpy()      # [page, place]
    want = np.zeros((3, chunk), dtype=bool)
    want[0] = True                       # positions 0..15 of sequence 0
    want[2, :4] = True                   # positions 32..35
    # sequence 1: positions 40..47 name page -5, 48..59 lie past its table
    assert np.array_equal(changed, want)
    out = torch.full((60, heads, dh), 5.0, device=DEV)
    kk, _ = rr.cache_read(codes, scales, cu, start, table, 60, dh, FF, out=(out, out.clone()))
    pos = np.concatenate([np.arange(-4, 36), np.arange(40, 60)])
    there = ((pos[:40] >= 0) & (pos[:40] < 16)) | (pos[:40] >= 32)
    assert np.array_equal((kk[:, 0, 0].cpu().numpy() == 1), np.concatenate([there, np.zeros(20, bool)]))
    assert np.array_equal((kk[:, 0, 0].cpu().numpy() == 0), ~np.concatenate([there, np.zeros(20, bool)]))
    # nothing to do
    rr.cache_write(codes, scales, k[:0], k[:0], _i32([0, 0, 0]), start, table)
    rr.cache_write(codes, scales, k, k, _i32([0]), start[:0], table[:0])
    empty = rr.cache_empty(0, heads, chunk, dh, "e4m3", DEV)
    rr.cache_write(*empty, k, k, cu, start, table)
    assert (rr.cache_read(*empty, cu, start, table, 60, dh, FF)[0] == 0).all()


def test_many_short_sequences(rr):
    # the search over cu: more than 32 * 32 sequences, empty ones among them, rows before cu[0]
    rng = np.random.default_rng(3)
    n, chunk, dh = 1500, 16, 64
    lens = rng.integers(0, 4, n)
    cu = 5 + np.concatenate([[0], np.cumsum(lens)])
    start = rng.integers(0, 13, n)
    table = np.arange(n, dtype=np.int32)[:, None]
    rows = int(cu[-1]) + 3
    k = torch.randn(rows, 1, dh, device=DEV, dtype=HF)
    codes, scales = rr.cache_empty(n, 1, chunk, dh, "e4m3", DEV)
    args = (_i32(cu), _i32(start), _i32(table))
    rr.cache_write(codes, scales, k, k, *args)
    out = torch.full((rows, 1, dh), 3.0, device=DEV)
    got, _ = rr.cache_read(codes, scales, *args, rows, dh, FF, out=(out, out.clone()))
    assert (got[:5] == 3).all() and (got[int(cu[-1]):] == 3).all()
    err = (got[5:int(cu[-1])] - k[5:int(cu[-1])].float()).abs()
    # half a step of e4m3, or of its smallest step at the row's scale (amax <= 448 2^e < 2 amax)
    top = k[5:int(cu[-1])].float().abs().amax(-1, keepdim=True)
    assert (err <= torch.maximum(2.0 ** -4 * k[5:int(cu[-1])].float().abs(), top * 2.0 ** -10 * 2 / 224)).all()
    assert int((scales != 0).sum()) == 2 * int(lens.sum())


def fill(pages, heads, chunk, dh, fmt, seed=0, spread=2):
    """A pool of written rows, their scales spread over `spread` binades; unwritten ones are NaN codes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(pages, heads, 2, chunk, dh, generator=g)
    x = x * torch.exp2(torch.randint(-spread, spread + 1, (pages, heads, 2, chunk, 1), generator=g).float())
    width = dh if fmt == "e4m3" else 32
    most = 448.0 if fmt == "e4m3" else 6.0
    y = x.unflatten(-1, (-1, width))
    e = torch.ceil(torch.log2(y.abs().amax(-1) / most)).clamp(-127, 120)
    y = y * torch.exp2(-e)[..., None]
    if fmt == "e4m3":
        codes = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:
        values = torch.tensor(M.E2M1[:8])
        c = (y.double().abs()[..., None] - values).abs().argmin(-1).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
        c = c.flatten(-2)
        codes = c[..., 0::2] | c[..., 1::2] << 4
    return codes.contiguous().to(DEV), (e + 127).to(torch.uint8).contiguous().to(DEV)


def check(got, codes, scales, fmt, q, lens, table, route=None, **kw):
    out, lse = got
    opt = {n: _np(x) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    rn = None if route is None else route.cpu().numpy()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    ref, ref_lse, mean = M.cached_attention(c, s, fmt, _np(q), np.array(lens), table, rn, **opt)
    dh, chunk = q.shape[3], codes.shape[3]
    cap, scale = opt.get("soft_cap", 0.0), opt.get("scale") or dh ** -0.5
    values = np.abs(M.read_rows(c, s, fmt))
    values = np.where(np.isfinite(values), values, 0.0)
    a = np.abs(_np(q)).sum(-1).max(initial=0.0) * values[:, :, 0].max(initial=0.0)
    delta = 2.0 ** -24 * (dh + 8) * scale * a + cap * 2.0 ** -21
    eps = torch.finfo(q.dtype).eps
    n = max(max(lens), (0 if route is None else route.shape[2] * chunk), 1)
    bound = (2 * delta + 2.0 ** -11 + 2.0 ** -12) * mean + eps / 2 * np.abs(ref) \
        + n * 2.0 ** -32 * values[:, :, 1].max(initial=0.0) + 1e-7
    o, got_lse = _np(out), _np(lse)
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    fine = ~np.isnan(ref)
    err = np.abs(np.where(fine, o - ref, 0.0))
    assert (err <= np.where(fine, bound, 1.0)).all(), (err.max(), np.unravel_index(np.argmax(err - bound), err.shape))
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(ref_lse))
    assert np.array_equal(np.isnan(got_lse), np.isnan(ref_lse))
    seen = np.isfinite(ref_lse)
    e = np.abs(np.where(seen, got_lse - np.where(seen, ref_lse, 0.0), 0.0))
    assert (e <= delta + 2.0 ** -21 * (1 + np.abs(np.where(seen, ref_lse, 0.0)))).all(), e.max()
    assert (o[np.isneginf(ref_lse)] == 0).all()


ATTN = [dict(), dict(fmt="e2m1"), dict(lens=[1, 16, 17], dh=128, group=4, heads=1), dict(fmt="e2m1", dh=128, group=4, qt=3),
        dict(lens=[2, 130, 0, 64], qt=4, group=8, heads=2, chunk=64, dtype=HF), dict(lens=[700], dh=128, group=1, chunk=128),
        dict(lens=[900, 3], fmt="e2m1", dh=128, group=16, heads=1, chunk=32), dict(lens=[100, 40], dh=128, qt=9, group=4, chunk=32),
        dict(lens=[33] * 20, heads=4, group=8, qt=4, dh=128), dict(lens=[20, 40] * 10, heads=4, group=8, qt=4, dh=128, fmt="e2m1"),
        dict(lens=[260], heads=1, group=12, qt=7, fmt="e2m1", dtype=HF), dict(lens=[3000, 1500], heads=1, group=3, chunk=64, dh=128)]


def cached_case(lens=(40, 5, 200), fmt="e4m3", dh=64, chunk=16, heads=2, group=2, qt=1, dtype=BF, seed=0, spread=2,
                q_scale=1.0):
    lens = list(lens)
    need = [-(-n // chunk) for n in lens]
    pages = sum(need) + 2
    codes, scales = fill(pages, heads, chunk, dh, fmt, seed, spread)
    table = table_of(need, pages, seed)
    # what lies behind a sequence's end in its last page: NaN codes, NaN scales
    for b, n in enumerate(lens):
        if n % chunk:
            codes[table[b, need[b] - 1], :, :, n % chunk:] = 0x7F
            scales[table[b, need[b] - 1], :, :, n % chunk:] = 255
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), qt, heads * group, dh, generator=g) * q_scale).to(dtype).to(DEV)
    return codes, scales, fmt, q, lens, table


@pytest.mark.parametrize("kind", ["", "r", "t", "s", "rts"])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_matches_the_oracle(rr, case, kind):
    codes, scales, fmt, q, lens, table = cached_case(seed=case, q_scale=4.0 if "t" in kind else 1.0, **ATTN[case])
    heads, chunk, hq = codes.shape[1], codes.shape[3], q.shape[2]
    kw, route = {}, None
    if "r" in kind:
        g = torch.Generator().manual_seed(case)
        route = torch.randint(-2, table.shape[1] + 2, (len(lens), heads, 7), generator=g, dtype=torch.int32)
        route = route.to(DEV)
    if "t" in kind:
        kw["soft_cap"] = 30.0
    if "s" in kind:
        kw["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]).to(DEV)
    got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), route=route, return_lse=True, **kw)
    check(got, codes, scales, fmt, q, lens, table, route, **kw)


@pytest.mark.parametrize("fmt,dh,chunk,heads,group,qt,batch,most", [
    ("e4m3", 64, 64, 4, 2, 1, 40, 3000),      # shares that end inside jobs and hold several
    ("e2m1", 128, 16, 2, 4, 1, 60, 900),
    ("e4m3", 64, 32, 1, 8, 5, 30, 1500),      # ... of two row blocks
    ("e4m3", 64, 16, 2, 8, 4, 24, 3001),      # three blocks to each job
    ("e2m1", 64, 128, 1, 2, 1, 3, 9000)])
def test_ragged_batches(rr, fmt, dh, chunk, heads, group, qt, batch, most):
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(most // 3, most, batch)]
    lens[0], lens[1], lens[-1] = most, 0, 1
    if batch > 5:
        lens[3:5] = [0, 0]
    case = cached_case(lens=lens, fmt=fmt, dh=dh, chunk=chunk, heads=heads, group=group, qt=qt, seed=batch)
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(heads * group)]).to(DEV)
    for kw in (dict(), dict(slopes=slopes)):
        got = rr.cached_attention(*case[:2], case[3], _i32(case[4]), _i32(case[5]), return_lse=True, **kw)
        check(got, *case, **kw)


# tables far wider than the sequences, most of them empty in some: the caller cuts by the
# table's width, so that there are fewer steps of 16 tokens than blocks (up to 296)
@pytest.mark.parametrize("fmt,dh,chunk,heads,group,qt,width,lens,routed", [
    ("e4m3", 128, 64, 8, 4, 1, 2000, [64] * 3, 0), ("e4m3", 128, 64, 8, 4, 1, 64, [500] + [0] * 11, 0),
    ("e2m1", 64, 32, 1, 4, 1, 64, [20] * 100, 0), ("e4m3", 64, 32, 2, 4, 5, 400, [100, 1, 100, 0, 1, 100, 1, 100], 0),
    ("e4m3", 128, 16, 4, 8, 4, 400, [20, 0, 0, 1, 100, 100], 0), ("e2m1", 128, 128, 1, 4, 5, 400, [0, 300, 1], 0),
    ("e2m1", 128, 32, 2, 8, 5, 1000, [1, 1, 0], 0), ("e4m3", 128, 64, 8, 4, 1, 188, [200] + [0] * 62 + [60], 0),
    ("e4m3", 64, 16, 1, 2, 1, 1000, [128] * 36 + [112], 0), ("e2m1", 64, 16, 1, 2, 1, 1000, [128] * 37, 0),
    ("e4m3", 64, 16, 1, 2, 1, 1000, [128] * 36 + [129], 0), ("e4m3", 64, 16, 1, 4, 2, 200, [0] * 99 + [700], 150),
    ("e2m1", 128, 16, 1, 4, 1, 200, [0] * 50 + [700] + [0] * 49, 150), ("e4m3", 64, 32, 2, 4, 5, 60, [0] * 39 + [700], 200),
    ("e2m1", 128, 16, 2, 8, 4, 900, [0] * 24, 0)])
def test_few_tokens_under_a_wide_table(rr, fmt, dh, chunk, heads, group, qt, width, lens, routed):
    batch = len(lens)
    codes, scales, fmt, q, lens, short = cached_case(lens=lens, fmt=fmt, dh=dh, chunk=chunk, heads=heads, group=group, qt=qt,
                                                     seed=width)
    rng = np.random.default_rng(width)
    table = rng.integers(-1, codes.shape[0], (batch, width)).astype(np.int32)     # pages of others behind a sequence's end
    for b, n in enumerate(lens):
        table[b, :-(-n // chunk)] = short[b, :-(-n // chunk)]
    route = _i32(rng.integers(-1, 800 // chunk, (batch, heads, routed))) if routed else None
    cfg = rr.rr_cache_config(codes.shape[0], heads, dh, chunk, rr.RR_E4M3 if fmt == "e4m3" else rr.RR_E2M1)
    attn = rr.rr_cached_attn_config(batch, qt, heads * group, rr.RR_BF16, width, width, routed, max(routed, 1))
    need = rr.rr_cached_attention_workspace_bytes(cfg, attn, routed > 0)
    assert need > 0
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(heads * group)]).to(DEV)
    for kw in (dict(), dict(slopes=slopes)):
        work = torch.full((need,), 255, dtype=torch.uint8, device=DEV)            # NaN wherever nothing is written
        got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), route=route, workspace=work, return_lse=True,
                                  **kw)
        check(got, codes, scales, fmt, q, lens, table, route, **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_scales_that_differ_by_many_binades(rr, fmt):
    case = cached_case(lens=[300, 90], fmt=fmt, dh=128, spread=24, q_scale=2.0 ** -24, group=4)
    got = rr.cached_attention(*case[:2], case[3], _i32(case[4]), _i32(case[5]), return_lse=True)
    check(got, *case)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_extremes_of_the_queries(rr, fmt):
    codes, scales, fmt, q, lens, table = cached_case(lens=[50, 30, 64], fmt=fmt, dh=64, group=4)
    q[0] *= 2.0 ** 60
    scales[table[0, :3], :, 0] -= 58
    q[1, 0, 0] = 0.0
    q[1, 0, 1] *= 2.0 ** -100
    q[2, 0, 3, 5] = float("nan")
    got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
    ref, ref_lse, mean = M.cached_attention(codes.cpu().numpy(), scales.cpu().numpy(), fmt, _np(q), np.array(lens), table)
    assert np.isnan(_np(got[0])[2, 0, 3]).all() and np.isnan(_np(got[1])[2, 0, 3])
    fine = ~np.isnan(ref)
    # scores reach a few times 2^2 |q| |k| scale: the rounding of bf16 outputs dominates
    err = np.abs(np.where(fine, _np(got[0]) - ref, 0))
    assert (err <= np.where(fine, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * mean + 1e-6, 1)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_strides_of_a_size_of_one(rr, fmt):
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn(64, generator=g).to(BF).to(DEV) for _ in range(3))
    codes, scales = rr.cache_empty(1, 1, 16, 64, fmt, DEV)
    zero, cu, table = _i32([0]), _i32([0, 1]), _i32([[0]])
    rr.cache_write(codes, scales, k.as_strided((1, 1, 64), (3, 5, 1)), v.as_strided((1, 1, 64), (1, 7, 1)), cu, zero, table)
    got = tuple(torch.zeros(64, dtype=torch.float32, device=DEV) for _ in range(2))
    rr.cache_read(codes, scales, cu, zero, table, 1, 64, torch.float32,
                  out=tuple(x.as_strided((1, 1, 64), (2, 3, 1)) for x in got))
    back = M.read_rows(codes.cpu().numpy(), scales.cpu().numpy(), fmt)[0, 0, :, 0]
    assert np.array_equal(got[0].cpu().numpy(), back[0]) and np.array_equal(got[1].cpu().numpy(), back[1])
    out = rr.cached_attention(codes, scales, q.as_strided((1, 1, 1, 64), (9, 3, 5, 1)), _i32([1]), table)
    assert torch.equal(out.view(64), got[1].to(BF))      # one token's weight is one


@pytest.mark.parametrize("power", [-96, 90])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_queries_and_keys_at_the_ends_of_their_range(rr, fmt, power):
    # powers of two that cancel in the scores
    codes, scales, fmt, q, lens, table = cached_case(lens=[48, 96], fmt=fmt, dh=64, group=4)
    q *= 2.0 ** power
    assert scales[:, :, 0].max() < 127 + 4 and scales[:, :, 0].min() > 90
    scales[:, :, 0] -= power if power > 0 else 0
    scales[:, :, 0] += -power if power < 0 else 0
    got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
    check(got, codes, scales, fmt, q, lens, table)


@pytest.mark.parametrize("lens", [[48, 96], [9000, 4000]])      # whole jobs, and joined parts
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_values_at_the_small_end_of_their_range(rr, fmt, lens):
    # values' scales down to 2^-126: their results are numbers of bf16 (and what cache_read returns)
    codes, scales, fmt, q, lens, table = cached_case(lens=lens, fmt=fmt, dh=64, group=4, heads=1)
    ref, ref_lse, mean = M.cached_attention(codes.cpu().numpy(), scales.cpu().numpy(), fmt, _np(q), np.array(lens), table)
    values = scales[:, :, 1]
    down = int(values[values != 255].min()) - 1
    assert 100 < down < 126
    scales[:, :, 1] = torch.where(values == 255, values, values - down)
    out = _np(rr.cached_attention(codes, scales, q, _i32(lens), _i32(table))) * 2.0 ** down
    # as in check(), delta below 2^-24 (64 + 8) 8 max |q| max |k|; and half a step of bf16's smallest numbers, 2^-134
    delta = 2.0 ** -24 * 72 * 8 * float(q.abs().max()) * 64
    bound = (2 * delta + 2.0 ** -11 + 2.0 ** -12) * mean + 2.0 ** -8 * np.abs(ref) + max(lens) * 2.0 ** -32 * 64 + 2.0 ** (down - 134)
    assert (np.abs(out - ref) <= bound).all(), np.abs(out - ref).max()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_groups_that_hold_no_number(rr, fmt):
    # a NaN scale reaches the rows that see it, of its own dims for the values, and no others
    codes, scales, fmt, q, lens, table = cached_case(lens=[40, 33], fmt=fmt, dh=128, qt=4, group=2)
    page = lambda b, p: table[b, p // 16]
    scales[page(0, 38), 0, 1, 38 % 16, -1] = 255      # a value that the first two query tokens do not see
    scales[page(1, 31), 1, 0, 31 % 16, 0] = 255       # a key likewise
    got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
    check(got, codes, scales, fmt, q, lens, table)
    assert torch.isfinite(got[0][0, :2]).all() and torch.isnan(got[0][0, 2:, :2, 96:]).all()


def test_sequences_without_tokens_or_pages(rr):
    codes, scales, fmt, q, lens, table = cached_case(lens=[0, 1, 20, 90], qt=2, chunk=16)
    table[2, 0] = -1
    table[3, 1], table[3, 2], table[3, 5] = 99, -1, -3
    for route in (None, _i32(np.full((4, 2, 3), -1)), _i32(np.array([[[0, 5, 5], [1, 2, 0]]] * 4))):
        got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), route=route, return_lse=True)
        check(got, codes, scales, fmt, q, lens, table, route)
    # a length past the table: what has no place is not seen; a negative one sees nothing
    long = [-3, 500, 20, 90]
    got = rr.cached_attention(codes, scales, q, _i32(long), _i32(table), return_lse=True)
    check(got, codes, scales, fmt, q, long, table)
    none = torch.zeros(4, 0, dtype=torch.int32, device=DEV)
    got = rr.cached_attention(codes, scales, q, _i32(lens), none, return_lse=True)
    assert (got[0] == 0).all() and torch.isneginf(got[1]).all()
    empty = rr.cache_empty(0, 2, 16, 64, "e4m3", DEV)
    got = rr.cached_attention(*empty, q, _i32(lens), _i32(table), return_lse=True)
    assert (got[0] == 0).all() and torch.isneginf(got[1]).all()
    assert rr.cached_attention(codes, scales, q[:0], _i32([]), _i32(table)[:0]).shape == (0, 2, 4, 64)
    assert rr.cached_attention(codes, scales, q[:, :0], _i32(lens), _i32(table)).shape == (4, 0, 4, 64)


@pytest.mark.parametrize("kw", [dict(), dict(width=0)])
def test_routes_of_no_entries_see_nothing(rr, kw):
    codes, scales, fmt, q, lens, table = cached_case(lens=[40, 700])
    for stride in (0,) if not kw else (0, 5):
        route = torch.zeros(2, 2, stride, dtype=torch.int32, device=DEV)
        out, lse = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), route=route, return_lse=True, **kw)
        assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()
        assert rr.cached_attention(codes, scales, q[:0], _i32([]), _i32(table)[:0], route=route[:0], **kw).shape == (0, 1, 4, 64)


def test_bias_of_far_positions_keeps_the_scores(rr):
    # the route names only the far end of a long sequence
    chunk, dh = 128, 64
    lens = [1 << 22]
    codes, scales = fill(4, 1, chunk, dh, "e4m3")
    table = np.full((1, (1 << 22) // chunk), -1, dtype=np.int32)
    table[0, :3] = [2, 0, 3]
    q = torch.randn(1, 2, 4, dh, device=DEV).to(HF)
    slopes = torch.full((4,), 0.5, device=DEV)
    for route in (_i32([[[2, 0, 1]]]), None):
        got = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), route=route, slopes=slopes, return_lse=True)
        short = table[:, :3]
        # the oracle on the keys that have pages, at their positions
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        key = np.arange(3 * chunk)
        k = M.read_rows(c[short[0, key // chunk], 0, 0, key % chunk], s[short[0, key // chunk], 0, 0, key % chunk], "e4m3")
        v = M.read_rows(c[short[0, key // chunk], 0, 1, key % chunk], s[short[0, key // chunk], 0, 1, key % chunk], "e4m3")
        for h in range(4):
            pos = lens[0] - 2 + np.arange(2)
            ref, lse, mean = M.softmax_rows(M.scores(_np(q)[0, :, h], k, dh ** -0.5, 0.0, 0.5, pos, key), np.ones((2, key.size)), v)
            assert (np.abs(_np(got[0])[0, :, h] - ref) <= 2.0 ** -10 * mean + 2.0 ** -11 * np.abs(ref) + 1e-6).all()
            assert np.abs(_np(got[1])[0, :, h] / lse - 1).max() < 2.0 ** -22


def test_streams_graphs_and_workspaces(rr):
    codes, scales, fmt, q, lens, table = cached_case(lens=[20000, 300], group=4, heads=1, dh=128, chunk=64)
    args = (_i32(lens), _i32(table))
    want = rr.cached_attention(codes, scales, q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [rr.cached_attention(codes, scales, q, *args, stream=s) for s in (side, side.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    cfg = rr.rr_cache_config(codes.shape[0], codes.shape[1], 128, codes.shape[3], rr.RR_E4M3)
    n = rr.rr_cached_attn_config(2, 1, 4, rr.RR_BF16, table.shape[1], table.shape[1], 0, 1)
    work = torch.empty(rr.rr_cached_attention_workspace_bytes(cfg, n, False), dtype=torch.uint8, device=DEV)
    assert work.numel() > 0
    assert torch.equal(rr.cached_attention(codes, scales, q, *args, workspace=work), want)
    with pytest.raises(rr.RRError) as e:
        rr.cached_attention(codes, scales, q, *args, workspace=work[:-256])
    assert e.value.status == rr.RR_ENOMEM
    # two graphs on one workspace, replayed in turn; lengths and cache change between replays
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, rr.cached_attention(codes, scales, q, *args, workspace=work, return_lse=True)))
    args[0].copy_(_i32([17001, 1]))
    q.copy_(torch.randn_like(q))
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        check(got, codes, scales, fmt, q, [17001, 1], table)


def test_a_turn_written_read_and_attended(rr):
    """A prompt and two steps of decoding: cache_write, then cached_attention
    over the whole cache and over a route, against masked_attention over what
    cache_read returns for the same tokens."""
    chunk, dh, heads, group = 16, 64, 2, 2
    lens = [37, 50]
    pages = 12
    codes, scales = rr.cache_empty(pages, heads, chunk, dh, "e4m3", DEV)
    table = _i32(table_of([6, 6], pages))
    cu = _i32([0, 37, 87])
    x = torch.randn(87, 2, heads, dh, device=DEV).to(BF)
    rr.cache_write(codes, scales, x[:, 0], x[:, 1], cu, _i32([0, 0]), table)
    for step in range(2):
        kv = torch.randn(2, 2, heads, dh, device=DEV).to(BF)
        rr.cache_write(codes, scales, kv[:, 0], kv[:, 1], _i32([0, 1, 2]), _i32(lens), table)
        lens = [n + 1 for n in lens]
        q = torch.randn(2, 1, heads * group, dh, device=DEV).to(BF)
        route = _i32([[[2, 0], [1, 2]], [[3, 1], [0, 3]]])
        for r in (None, route):
            out = rr.cached_attention(codes, scales, q, _i32(lens), table, route=r)
            for b in range(2):
                k, v = rr.cache_read(codes, scales, _i32([0, lens[b]]), _i32([0]), table[b:b + 1].contiguous(), lens[b],
                                     dh, BF)
                ids = _i32(list(range(6))).expand(1, heads, 1, 6).contiguous() if r is None else r[b][None, :, None]
                want = rr.masked_attention(q[b].transpose(0, 1)[None], k.transpose(0, 1)[None], v.transpose(0, 1)[None],
                                           ids.contiguous(), chunk, causal=True, q_offset=lens[b] - 1)
                err = (out[b].float() - want[0].transpose(0, 1).float()).abs()
                assert (err <= 2.0 ** -7 * v.float().abs().max()).all()
    # the dense call agrees with the oracle too
    check(rr.cached_attention(codes, scales, q, _i32(lens), table, return_lse=True), codes, scales, "e4m3", q, lens,
          table.cpu().numpy())


def test_ledger_routes_in_place(rr):
    b, heads, nk, chunk, dh, width = 3, 2, 40, 16, 64, 8
    cfg = rr.Config(bh=b * heads, nq=1, nk=nk, d=64, k=width, m_near=4, r_rand=2, dtype="bf16")
    led = rr.RouteLedger(cfg, DEV)
    led.layer(torch.randn(b * heads, 1, 64, device=DEV).to(BF), torch.randn(b * heads, nk, 64, device=DEV).to(BF), 0)
    lens = [nk * chunk - 3, 500, 640]
    codes, scales = fill(b * nk, heads, chunk, dh, "e2m1")
    table = np.arange(b * nk, dtype=np.int32).reshape(b, nk)
    q = torch.randn(b, 1, 4, dh, device=DEV).to(BF)
    got = led.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
    ids = led.read()["ids"][:, 0, :width].reshape(b, heads, width).contiguous().to(DEV)
    check(got, codes, scales, "e2m1", q, lens, table, ids)
    with pytest.raises(ValueError):
        led.cached_attention(codes, scales, q[:2], _i32(lens[:2]), _i32(table[:2]))
    with pytest.raises(ValueError):
        led.cached_attention(codes, scales, q, _i32(lens), _i32(table), width=3)


def test_two_calls_give_the_same_bits(rr):
    codes, scales, fmt, q, lens, table = cached_case(lens=[5000, 100, 2500], group=8, dh=128, chunk=64)
    first = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
    for _ in range(3):
        again = rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refuses_wrong_tensors(rr):
    codes, scales, fmt, q, lens, table = cached_case()
    ln, tb = _i32(lens), _i32(table)
    bad = [(codes.float(), scales, q, ln, tb), (codes, scales[:-1], q, ln, tb), (codes, scales, q.float(), ln, tb),
           (codes[..., :48].contiguous(), scales, q, ln, tb), (codes, scales, q, ln.long(), tb),
           (codes, scales, q, ln[:2], tb), (codes, scales, q, ln, tb[:2]), (codes, scales, q, ln, tb.t()),
           (codes, scales, q.cpu(), ln, tb), (codes.transpose(0, 1), scales, q, ln, tb)]
    for args in bad:
        with pytest.raises(ValueError):
            rr.cached_attention(*args)
    for kw in (dict(route=tb), dict(width=3), dict(slopes=torch.ones(4)), dict(out=q.float()),
               dict(route=_i32(np.zeros((3, 2, 4))), width=5), dict(workspace=torch.empty(8, device=DEV))):
        with pytest.raises(ValueError):
            rr.cached_attention(codes, scales, q, ln, tb, **kw)
    k = torch.zeros(10, 2, 64, dtype=BF, device=DEV)
    cu, start = _i32([0, 4, 8, 10]), _i32([0, 0, 0])
    for args in ((k.double(), k, cu, start, tb), (k, k.half(), cu, start, tb), (k[:, :1], k, cu, start, tb),
                 (k, k, cu[:-1], start, tb), (k, k, cu, start[:2], tb), (k, k, cu, start, tb.long())):
        with pytest.raises(ValueError):
            rr.cache_write(codes, scales, *args)
    with pytest.raises(ValueError):
        rr.cache_read(codes, scales, cu, start, tb, 10, 64, torch.float64)
    with pytest.raises(ValueError):
        rr.cache_read(codes, scales, cu, start, tb, 10, 96)
    with pytest.raises(ValueError):
        rr.cache_read(codes, scales, cu, start, tb, 10, 64, BF, out=(k, k[:9]))


def test_numbers_that_fit_no_field_are_refused(rr):
    codes, scales, fmt, q, lens, table = cached_case()
    for kw, error in ((dict(scale="1"), ValueError), (dict(soft_cap=10 ** 400), ValueError), (dict(soft_cap=1e39), rr.RRError),
                      (dict(scale=-1e300), rr.RRError)):
        with pytest.raises(error):
            rr.cached_attention(codes, scales, q, _i32(lens), _i32(table), **kw)
    with pytest.raises(ValueError):
        rr.cache_read(codes, scales, _i32([0, 1]), _i32([0]), _i32([[0]]), 1 << 31, 64)
