"""Measured cases of the attention and cache operators that follow a route.

Four operators that a serving program runs after the router has chosen its
chunks:

  masked    attention of a prompt over its routes, with capped scores, a bias
            by distance, a document mask and a prefix mask
  write     a step's keys and values quantised into a paged cache
  read      cached keys and values gathered back (after a write in `turn`)
  cached    attention of a sequence's newest tokens over the paged cache,
            dense or over a route

Each case is a dict of plain values.  run() computes it in plain torch
operations, or, with `own` set, with the calls that a user makes.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a short prompt in a chat: a handful of chunks, where the call itself is what counts
        {"name": "masked_short", "kind": "masked", "b": 1, "hq": 8, "hkv": 2, "nq": 77, "nk": 77, "dh": 64, "chunk": 16,
         "width": 4, "dtype": "bf16", "causal": True, "cap": 30.0, "slopes": False, "docs": 0, "prefix": False, "tokens_first": True},
        # four prompts with a bidirectional prefix and a bias by distance, one key head to each query head
        {"name": "masked_prefix_bias", "kind": "masked", "b": 4, "hq": 8, "hkv": 8, "nq": 2501, "nk": 2501, "dh": 64, "chunk": 32,
         "width": 24, "dtype": "f16", "causal": True, "cap": 0.0, "slopes": True, "docs": 0, "prefix": True, "tokens_first": False},
        # the next piece of two long prompts that are processed in pieces, scores capped
        {"name": "masked_piece_cap", "kind": "masked", "b": 2, "hq": 32, "hkv": 8, "nq": 2048, "nk": 30000, "dh": 128, "chunk": 64,
         "width": 48, "dtype": "bf16", "causal": True, "cap": 30.0, "slopes": False, "docs": 0, "prefix": False, "tokens_first": True},
        # one long packed sequence of documents, the routing path's largest chunk size and route width
        {"name": "masked_long_docs", "kind": "masked", "b": 1, "hq": 16, "hkv": 4, "nq": 65536, "nk": 65536, "dh": 128, "chunk": 64,
         "width": 32, "dtype": "bf16", "causal": True, "cap": 0.0, "slopes": False, "docs": 5, "prefix": False, "tokens_first": False},
        # one decoding step of 64 sequences
        {"name": "write_step", "kind": "write", "format": "e4m3", "heads": 8, "dh": 128, "chunk": 64, "batch": 64, "most": 1, "before": 4000,
         "spare": 0, "dtype": "bf16"},
        # eight prompts of different lengths, with unused rows at the end of the batch
        {"name": "write_prompts", "kind": "write", "format": "e4m3", "heads": 8, "dh": 128, "chunk": 64, "batch": 8, "most": 8191, "before": 0,
         "spare": 37, "dtype": "bf16"},
        # pieces of three conversations: written, and read back for the attention over them
        {"name": "turn", "kind": "turn", "format": "e2m1", "heads": 4, "dh": 64, "chunk": 16, "batch": 3, "most": 1500, "before": 700,
         "spare": 5, "dtype": "f16"},
        # the cached history of four long prompts, read for the attention of their next piece
        {"name": "read_history", "kind": "read", "format": "e2m1", "heads": 8, "dh": 128, "chunk": 64, "batch": 4, "most": 32000, "before": 0,
         "spare": 0, "dtype": "bf16"},
        # one sequence, one token: the latency of a single stream
        {"name": "cached_one", "kind": "cached", "format": "e4m3", "heads": 8, "group": 4, "dh": 128, "chunk": 64, "batch": 1, "qt": 1,
         "most": 4096, "width": 0, "dtype": "bf16", "cap": 0.0, "slopes": False},
        # a full batch of ragged sequences, every page read
        {"name": "cached_batch", "kind": "cached", "format": "e4m3", "heads": 8, "group": 4, "dh": 128, "chunk": 64, "batch": 64, "qt": 1,
         "most": 12001, "width": 0, "dtype": "bf16", "cap": 0.0, "slopes": False},
        # long sequences through their routes, scores capped, the cache in four bits
        {"name": "cached_routed", "kind": "cached", "format": "e2m1", "heads": 8, "group": 4, "dh": 128, "chunk": 64, "batch": 16, "qt": 1,
         "most": 100000, "width": 128, "dtype": "bf16", "cap": 30.0, "slopes": False},
        # four drafted tokens of each sequence checked at once, a bias by distance, small pages
        {"name": "cached_drafts", "kind": "cached", "format": "e4m3", "heads": 2, "group": 8, "dh": 64, "chunk": 16, "batch": 24, "qt": 4,
         "most": 3001, "width": 0, "dtype": "f16", "cap": 0.0, "slopes": True},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["masked", "masked", "write", "turn", "read", "cached", "cached"])
    if kind == "masked":
        while True:
            hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 4, 8])
            nq = _spread(rng, 1, 20000)
            c = {"kind": kind, "b": rng.choice([1, 1, 2, 3]), "hq": hkv * group, "hkv": hkv, "nq": nq,
                 "nk": nq + rng.choice([0, 0, _spread(rng, 1, 20000)]), "dh": rng.choice([64, 128]), "chunk": rng.choice([16, 32, 64, 128]),
                 "width": _spread(rng, 1, 64), "dtype": rng.choice(["bf16", "f16"]), "causal": rng.random() < 0.8,
                 "cap": rng.choice([0.0, 20.0, 50.0]), "slopes": rng.random() < 0.4, "docs": rng.choice([0, 0, 3, 9]),
                 "prefix": rng.random() < 0.3, "tokens_first": rng.random() < 0.5}
            if c["b"] * c["hq"] * c["nq"] * c["width"] * c["chunk"] * c["dh"] <= 6e10:
                return c
    c = {"kind": kind, "format": rng.choice(["e4m3", "e2m1"]), "heads": rng.choice([1, 2, 4, 8]), "dh": rng.choice([64, 128]),
         "chunk": rng.choice([16, 32, 64, 128]), "batch": _spread(rng, 1, 48), "dtype": rng.choice(["bf16", "f16"])}
    if kind == "cached":
        c.update(group=rng.choice([1, 2, 4, 8]), qt=rng.choice([1, 1, 1, 2, 5]), most=_spread(rng, 16, 16000), width=rng.choice([0, 0, 8, 48]),
                 cap=rng.choice([0.0, 0.0, 30.0]), slopes=rng.random() < 0.3)
        return c
    if kind == "write":
        c["format"] = "e4m3"
    c.update(most=_spread(rng, 1, 200000 // c["batch"] // c["heads"]), before=rng.choice([0, _spread(rng, 1, 3000)]), spare=rng.choice([0, 0, 9]))
    return c


# ---- lengths and documents of a case, the same for every seed ---------------------------------------------------------------

def _lengths(c):
    """Tokens of each sequence: ragged, the longest first, from a step's single token up to `most`."""
    r = random.Random(17 * c["batch"] + c["most"])
    return [c["most"]] + [max(1, r.randint(c["most"] // 3, c["most"])) for _ in range(c["batch"] - 1)]


def _befores(c):
    """Tokens already cached before each sequence's new ones."""
    r = random.Random(c["before"] + 1)
    return [r.randint(0, c["before"]) for _ in range(c["batch"])]


def _doc_starts(c):
    r = random.Random(c["docs"])
    return [0] + sorted(r.randrange(c["nk"]) for _ in range(c["docs"] - 1))


def _chunks(n, chunk):
    return -(-n // chunk)


def _routed_tokens(c):
    """Visible (query, key) pairs of one head as the routes of prepare() have them, diagonal chunks counted by half."""
    ch, off = c["chunk"], c["nk"] - c["nq"]
    starts = _doc_starts(c) if c["docs"] else [0]
    ends = starts[1:] + [c["nk"]]
    pairs = 0
    for i in range(_chunks(c["nq"], ch)):
        rows = min(ch, c["nq"] - i * ch)
        first = off + i * ch
        low, high = [(s, e) for s, e in zip(starts, ends) if s <= first][-1] if c["docs"] else (0, c["nk"])
        high = min(high, first + rows) if c["causal"] else high
        keys = min(c["width"] * ch, max(0, high - low))
        pairs += rows * keys - (rows * min(rows, keys) // 2 if c["causal"] else 0)
    return pairs


def work(c):
    if c["kind"] == "masked":
        rows, keys = c["b"] * c["hq"] * c["nq"], c["b"] * c["hkv"] * c["nk"]
        nqc = _chunks(c["nq"], c["chunk"])
        route = c["b"] * c["hkv"] * nqc * c["width"] * 4
        small = (c["b"] * (c["nq"] + c["nk"]) * 4 if c["docs"] else 0) + (4 * c["b"] if c["prefix"] else 0) + (4 * c["hq"] if c["slopes"] else 0)
        reads = min(keys, c["b"] * c["hkv"] * nqc * c["width"] * c["chunk"])
        return {"bytes": 2 * 2 * rows * c["dh"] + 2 * 2 * reads * c["dh"] + 4 * rows + route + small,
                "flops": 4 * c["dh"] * c["b"] * c["hq"] * _routed_tokens(c)}
    groups = 1 if c["format"] == "e4m3" else c["dh"] // 32
    row = (c["dh"] if c["format"] == "e4m3" else c["dh"] // 2) + groups
    lens = _lengths(c)
    if c["kind"] == "cached":
        have = [min(n, c["width"] * c["chunk"]) if c["width"] else n for n in lens]
        rows = c["batch"] * c["qt"] * c["heads"] * c["group"]
        table = 4 * sum(_chunks(n, c["chunk"]) for n in have) + (4 * c["batch"] * c["heads"] * c["width"])
        return {"bytes": 2 * row * c["heads"] * sum(have) + 4 * rows * c["dh"] + 4 * rows + table,
                "flops": 4 * c["dh"] * c["heads"] * c["group"] * c["qt"] * sum(have)}
    rows = 2 * c["heads"] * sum(lens)
    passes = 2 if c["kind"] == "turn" else 1
    return {"bytes": passes * rows * (row + 2 * c["dh"]), "flops": passes * 2 * rows * c["dh"]}


# ---- inputs --------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _routes(g, c):
    """Distinct chunks for each query chunk, its own one among them, those of its document first; -1 where there are no more."""
    ch, off = c["chunk"], c["nk"] - c["nq"]
    nqc, nkc = _chunks(c["nq"], ch), _chunks(c["nk"], ch)
    first = off + ch * torch.arange(nqc, device="cuda")
    last = torch.clamp(first + ch - 1, max=c["nk"] - 1)
    ids = torch.arange(nkc, device="cuda")
    bonus = ((ids >= first[:, None] // ch) & (ids <= last[:, None] // ch)).float() * 4
    if c["docs"]:
        starts = torch.tensor(_doc_starts(c), device="cuda")
        doc = lambda t: torch.searchsorted(starts, t, right=True)
        bonus = bonus + 2 * ((doc(ids * ch) <= doc(first)[:, None]) & (doc(torch.clamp(ids * ch + ch, max=c["nk"]) - 1) >= doc(first)[:, None])).float()
    outside = ids * ch > last[:, None] if c["causal"] else torch.zeros(nqc, nkc, dtype=torch.bool, device="cuda")
    score = torch.rand(c["b"], c["hkv"], nqc, nkc, generator=g, device="cuda") + bonus
    top, at = score.masked_fill(outside, -1.0).topk(min(c["width"], nkc), dim=-1)
    route = torch.where(top >= 0, at, -1).int()
    return torch.nn.functional.pad(route, (0, c["width"] - route.shape[-1]), value=-1).contiguous()


def _split(x, c):
    """[b, heads, n, dh], as a view of rows that hold all heads where the case says so."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if c["tokens_first"] else x


def _power(e):
    """2^e in 32 bits, from its bits."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _quantised(x, fmt):
    """(codes as the values they stand for, exponents) of rows in the cache's formats: the smallest power of two that holds a
    row's (e4m3) or 32 elements' (e2m1) largest value, and the elements divided by it, rounded to nearest, ties to even."""
    most, width = (448.0, x.shape[-1]) if fmt == "e4m3" else (6.0, 32)
    x = x.float().unflatten(-1, (-1, width))
    m, e = torch.frexp(x.abs().amax(-1))
    # amax = 2 m * 2^(e - 1) with 2 m in [1, 2); 448 = 1.75 * 2^8 and 6 = 1.5 * 2^2
    top, power = (1.75, 8) if fmt == "e4m3" else (1.5, 2)
    e = torch.where(m > 0, e - 1 - power + (2 * m > top).int(), -127).clamp(min=-127)
    y = x * _power(-e)[..., None]
    if fmt == "e4m3":
        y = y.to(torch.float8_e4m3fn).float()
    else:
        a = y.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        y = torch.copysign((a / step).round() * step, y)
    return y.flatten(-2), e


def _e2m1_codes(y):
    a = y.abs()
    code = sum((a >= v).to(torch.uint8) for v in E2M1[1:]) + 8 * torch.signbit(y).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2]


def _store(x, fmt):
    """(codes, scales) of rows as the cache holds them."""
    y, e = _quantised(x, fmt)
    return (y.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else _e2m1_codes(y)), (e + 127).to(torch.uint8)


def _values(codes, scales, dh):
    """What codes and scales of the cache stand for, in 32 bits."""
    if codes.shape[-1] == dh:
        y = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        y = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    e = _power(scales.int() - 127)
    return (y.unflatten(-1, (e.shape[-1], -1)) * e[..., None]).flatten(-2)


def _pool(g, c, pages, fill):
    row, groups = (c["dh"], 1) if c["format"] == "e4m3" else (c["dh"] // 2, c["dh"] // 32)
    codes = torch.zeros(pages, c["heads"], 2, c["chunk"], row, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, c["heads"], 2, c["chunk"], groups, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (c["heads"] * 2 * c["chunk"] * c["dh"]))
    for p in range(0, pages if fill else 0, step):
        n = min(step, pages - p)
        codes[p:p + n], scales[p:p + n] = _store(_normal(g, n, c["heads"], 2, c["chunk"], c["dh"]).bfloat16(), c["format"])
    return codes, scales


def _table(g, need):
    """Pages of a pool handed out in no order, -1 past a sequence's end."""
    pages, width = sum(need), max(need)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def prepare(c, seed):
    g = _gen(seed)
    if c["kind"] == "masked":
        t = DTYPES[c["dtype"]]
        q = (_normal(g, c["b"], c["hq"], c["nq"], c["dh"]) * (4.0 if c["cap"] else 1.0)).to(t)
        k = _normal(g, c["b"], c["hkv"], c["nk"], c["dh"]).to(t)
        v = _normal(g, c["b"], c["hkv"], c["nk"], c["dh"]).to(t)
        s = {"case": c, "q": _split(q, c), "k": _split(k, c), "v": _split(v, c), "route": _routes(g, c),
             "slopes": None, "doc_q": None, "doc_k": None, "prefix": None}
        if c["slopes"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda")
        if c["docs"]:
            starts = torch.tensor(_doc_starts(c), device="cuda")
            doc = torch.searchsorted(starts, torch.arange(c["nk"], device="cuda"), right=True).int()
            s["doc_k"] = doc.repeat(c["b"], 1)
            s["doc_q"] = s["doc_k"][:, c["nk"] - c["nq"]:].contiguous()
        if c["prefix"]:
            s["prefix"] = torch.randint(0, c["nk"] // 2 + 1, (c["b"],), generator=g, device="cuda", dtype=torch.int32)
        return s
    lens = _lengths(c)
    if c["kind"] == "cached":
        need = [_chunks(n, c["chunk"]) for n in lens]
        codes, scales = _pool(g, c, sum(need), True)
        q = (_normal(g, c["batch"], c["qt"], c["heads"] * c["group"], c["dh"]) * (4.0 if c["cap"] else 1.0)).to(DTYPES[c["dtype"]])
        s = {"case": c, "codes": codes, "scales": scales, "q": q, "lens": _int32(lens), "table": _table(g, need), "route": None, "slopes": None}
        if c["slopes"]:
            h = c["heads"] * c["group"]
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")
        if c["width"]:
            # the last chunk, and distinct others from the whole length
            n = torch.tensor(need, device="cuda")[:, None, None]
            ids = torch.arange(max(need), device="cuda")
            score = torch.rand(c["batch"], c["heads"], max(need), generator=g, device="cuda") + (ids == n - 1) * 2.0
            top, at = score.masked_fill(ids >= n, -1.0).topk(min(c["width"], max(need)), dim=-1)
            route = torch.where(top >= 0, at, -1).int()
            s["route"] = torch.nn.functional.pad(route, (0, c["width"] - route.shape[-1]), value=-1).contiguous()
        return s
    before = _befores(c)
    need = [_chunks(a + n, c["chunk"]) for a, n in zip(before, lens)]
    codes, scales = _pool(g, c, sum(need), c["kind"] == "read")
    used = sum(lens)
    s = {"case": c, "codes": codes, "scales": scales, "table": _table(g, need), "start": _int32(before), "used": used,
         "cu": _int32([sum(lens[:i]) for i in range(len(lens) + 1)]), "rows": used + c["spare"]}
    if c["kind"] != "read":
        # a layer's fused projection: queries, keys and values of a token side by side
        x = _normal(g, s["rows"], 3, c["heads"], c["dh"]).to(DTYPES[c["dtype"]])
        s["k"], s["v"] = x[:, 1], x[:, 2]
    return s


# ---- the operators in their plain form ---------------------------------------------------------------------------------------

def _attend(q, k, v, logits_more, visible, distance, slopes, cap):
    """softmax over the last axis of q k^T (scaled by logits_more) under `visible`; out and log of the sum."""
    s = (q @ k.transpose(-1, -2)) * logits_more
    if cap:
        s = cap * torch.tanh(s / cap)
    shift = 0.0
    if slopes is not None:
        # the bias relative to the row's nearest visible key: far positions keep their last bits
        near = torch.where(visible, distance, 1 << 30).amin(-1, keepdim=True)
        near = torch.where(near == 1 << 30, 0, near)
        s = s - slopes * (distance - near)
        shift = -(slopes * near)[..., 0]
    s = s.masked_fill(~visible, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, torch.log(total[..., 0]) + top[..., 0] + shift


def _masked_plain(s):
    c, ch = s["case"], s["case"]["chunk"]
    b, hq, nq, dh = s["q"].shape
    hkv, nk = s["k"].shape[1:3]
    nqc, nkc, group, off = _chunks(nq, ch), _chunks(nk, ch), hq // hkv, nk - nq
    pad = lambda x, n: torch.nn.functional.pad(x.float(), (0, 0, 0, n * ch - x.shape[2]))
    q = pad(s["q"], nqc).view(b, hkv, group, nqc, ch, dh).transpose(2, 3)
    ids = s["route"].long()
    there = (ids >= 0) & (ids < nkc)
    ids = ids.clamp(0, nkc - 1)
    at = (torch.arange(b, device="cuda")[:, None, None, None], torch.arange(hkv, device="cuda")[None, :, None, None], ids)
    flat = lambda x: pad(x, nkc).view(b, hkv, nkc, ch, dh)[at].flatten(3, 4)[:, :, :, None]
    k, v = flat(s["k"]), flat(s["v"])
    key = (ids[..., None] * ch + torch.arange(ch, device="cuda")).int()
    visible = (there[..., None] & (key < nk)).flatten(3)[:, :, :, None, None, :]
    key = key.flatten(3)[:, :, :, None, None, :]
    row = torch.arange(nqc * ch, device="cuda", dtype=torch.int32).view(nqc, 1, ch, 1)
    if c["causal"]:
        seen = key <= row + off
        if s["prefix"] is not None:
            seen = seen | (key < s["prefix"].view(b, 1, 1, 1, 1, 1))
        visible = visible & seen
    if s["doc_q"] is not None:
        doc_q = torch.nn.functional.pad(s["doc_q"], (0, nqc * ch - nq), value=-1).view(b, 1, nqc, 1, ch, 1)
        doc_k = s["doc_k"][torch.arange(b, device="cuda").view(b, 1, 1, 1, 1, 1), key.clamp(max=nk - 1).long()]
        visible = visible & (doc_q == doc_k) & (doc_q >= 0)
    slopes = None if s["slopes"] is None else s["slopes"].view(hkv, 1, group, 1, 1)
    distance = None if slopes is None else (row + off - key).abs()
    out, lse = _attend(q, k, v, dh ** -0.5, visible, distance, slopes, c["cap"])
    out = out.transpose(2, 3).reshape(b, hq, nqc * ch, dh)[:, :, :nq]
    return {"out": out.to(s["q"].dtype).contiguous(), "lse": lse.transpose(2, 3).reshape(b, hq, nqc * ch)[:, :, :nq].contiguous()}


def _places(s, rows):
    """(page, place in the page) of the first `rows` rows of a ragged batch."""
    c = s["case"]
    i = torch.arange(rows, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], i, right=True) - 1
    at = s["start"][seq] + i - s["cu"][seq]
    return s["table"][seq, (at // c["chunk"]).long()].long(), (at % c["chunk"]).long()


def _write_plain(s):
    c, n = s["case"], s["used"]
    page, place = _places(s, n)
    codes, scales = _store(torch.stack((s["k"][:n], s["v"][:n]), 2), c["format"])
    head = torch.arange(c["heads"], device="cuda")[None, :, None]
    which = torch.arange(2, device="cuda")[None, None, :]
    s["codes"][page[:, None, None], head, which, place[:, None, None]] = codes
    s["scales"][page[:, None, None], head, which, place[:, None, None]] = scales


def _read_plain(s):
    c = s["case"]
    page, place = _places(s, s["used"])
    head = torch.arange(c["heads"], device="cuda")[None, :]
    at = lambda x, which: x[page[:, None], head, which, place[:, None]]
    k, v = (_values(at(s["codes"], w), at(s["scales"], w), c["dh"]).to(DTYPES[c["dtype"]]) for w in (0, 1))
    return {"k": k, "v": v}


def _cached_plain(s):
    c, ch = s["case"], s["case"]["chunk"]
    b, h, group, qt, dh = c["batch"], c["heads"], c["group"], c["qt"], c["dh"]
    q = s["q"].float().view(b, qt, h, group, dh).permute(0, 2, 1, 3, 4).reshape(b, h, qt * group, dh)
    width = s["table"].shape[1]
    ids = s["route"].long() if s["route"] is not None else torch.arange(width, device="cuda").expand(b, h, width)
    lens = s["lens"].view(b, 1, 1)
    there = (ids >= 0) & (ids * ch < lens)
    ids = ids.clamp(0, width - 1)
    page = s["table"][torch.arange(b, device="cuda")[:, None, None], ids].clamp(min=0).long()
    head = torch.arange(h, device="cuda")[None, :, None]
    k, v = (_values(s["codes"][page, head, w], s["scales"][page, head, w], dh).flatten(2, 3) for w in (0, 1))
    key = (ids[..., None] * ch + torch.arange(ch, device="cuda")).int()
    row = (lens - qt + torch.arange(qt, device="cuda")).repeat_interleave(group, -1)[..., None].int()
    visible = (there[..., None] & (key >= 0)).flatten(2)[:, :, None, :] & (key.flatten(2)[:, :, None, :] <= row)
    slopes = None if s["slopes"] is None else s["slopes"].view(h, 1, group).expand(h, qt, group).reshape(h, qt * group, 1)
    distance = None if slopes is None else row - key.flatten(2)[:, :, None, :]
    out, lse = _attend(q, k, v, dh ** -0.5, visible, distance, slopes, c["cap"])
    out = out.view(b, h, qt, group, dh).permute(0, 2, 1, 3, 4).reshape(b, qt, h * group, dh)
    return {"out": out.to(s["q"].dtype), "lse": lse.view(b, h, qt, group).permute(0, 2, 1, 3).reshape(b, qt, h * group)}


def run(s):
    c = s["case"]
    if own:
        import cross_layer_route_b200 as rr
        scale = {"soft_cap": c["cap"], "slopes": s["slopes"]} if "cap" in c else {}
        if c["kind"] == "masked":
            out, lse = rr.masked_attention(s["q"], s["k"], s["v"], s["route"], c["chunk"], causal=c["causal"], doc_q=s["doc_q"], doc_k=s["doc_k"],
                                           prefix=s["prefix"], q_offset=c["nk"] - c["nq"], return_lse=True, **scale)
            return {"out": out, "lse": lse}
        if c["kind"] == "cached":
            out, lse = rr.cached_attention(s["codes"], s["scales"], s["q"], s["lens"], s["table"], route=s["route"], return_lse=True, **scale)
            return {"out": out, "lse": lse}
        if c["kind"] != "read":
            rr.cache_write(s["codes"], s["scales"], s["k"], s["v"], s["cu"], s["start"], s["table"])
        if c["kind"] != "write":
            k, v = rr.cache_read(s["codes"], s["scales"], s["cu"], s["start"], s["table"], s["used"], c["dh"], DTYPES[c["dtype"]])
            return {"k": k, "v": v}
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if c["kind"] == "masked":
        return _masked_plain(s)
    if c["kind"] == "cached":
        return _cached_plain(s)
    if c["kind"] != "read":
        _write_plain(s)
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]} if c["kind"] == "write" else _read_plain(s)


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------------------

def _softmax64(logits, count, values):
    """Rows of softmax(logits) values, each key counted `count` times (0: not visible), and the log of the sums."""
    logits = logits + torch.log(count)
    lse = torch.logsumexp(logits, -1)
    p = torch.exp(logits - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return p @ values, lse


def _score64(q, k, c):
    s = q.double() @ k.double().T / math.sqrt(c["dh"])
    return c["cap"] * torch.tanh(s / c["cap"]) if c["cap"] else s


def _exact_masked(c, s):
    ch, nq, nk, off = c["chunk"], c["nq"], c["nk"], c["nk"] - c["nq"]
    out = torch.empty(c["b"], c["hq"], nq, c["dh"], dtype=torch.float64, device="cuda")
    lse = torch.empty(c["b"], c["hq"], nq, dtype=torch.float64, device="cuda")
    nkc = _chunks(nk, ch)
    token = torch.arange(nk, device="cuda")
    block = ch * max(1, (1 << 27) // (8 * nk * ch))
    for b in range(c["b"]):
        for h in range(c["hq"]):
            hk = h * c["hkv"] // c["hq"]
            ids = s["route"][b, hk].long()
            ok = (ids >= 0) & (ids < nkc)
            times = torch.zeros(ids.shape[0], nkc, device="cuda", dtype=torch.float64).scatter_add_(1, ids.clamp(0, nkc - 1), ok.double())
            for r in range(0, nq, block):
                rows = torch.arange(r, min(nq, r + block), device="cuda")
                count = times[rows // ch][:, token // ch]
                see = torch.ones_like(count, dtype=torch.bool)
                if c["causal"]:
                    see = token[None, :] <= off + rows[:, None]
                    if s["prefix"] is not None:
                        see = see | (token < s["prefix"][b])[None, :]
                if s["doc_q"] is not None:
                    mine = s["doc_q"][b, rows][:, None]
                    see = see & (mine == s["doc_k"][b][None, :]) & (mine >= 0)
                x = _score64(s["q"][b, h, rows], s["k"][b, hk], c)
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (off + rows[:, None] - token[None, :]).abs()
                out[b, h, rows], lse[b, h, rows] = _softmax64(x, count * see, s["v"][b, hk].double())
    return {"out": out, "lse": lse}


def _two(e):
    """2^e in 64 bits, from its bits: a power function's last bit would move ties."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _rows64(c, s, which, b, positions):
    """[positions, heads, dh] of the cache in 64 bits."""
    page = s["table"][b, positions // c["chunk"]].long()
    codes = s["codes"][page, :, which, positions % c["chunk"]].long()
    scales = s["scales"][page, :, which, positions % c["chunk"]].long()
    if c["format"] == "e2m1":
        codes = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
        bits, exponents, bias = 1, 2, 1
    else:
        bits, exponents, bias = 3, 4, 7
    m, e, sign = codes % 2 ** bits, codes // 2 ** bits % 2 ** exponents, codes // 2 ** (bits + exponents)
    x = torch.where(e == 0, m.double() * 2.0 ** (1 - bias - bits), (1 + m.double() / 2 ** bits) * _two(e - bias)) * (1 - 2 * sign)
    return x * _two(scales - 127).repeat_interleave(c["dh"] // scales.shape[-1], -1)


def _exact_cached(c, s):
    shape = (c["batch"], c["qt"], c["heads"] * c["group"])
    out, lse = torch.empty(*shape, c["dh"], dtype=torch.float64, device="cuda"), torch.empty(shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        token = torch.arange(n, device="cuda")
        k, v = _rows64(c, s, 0, b, token), _rows64(c, s, 1, b, token)
        for h in range(c["heads"]):
            times = torch.ones(_chunks(n, c["chunk"]), dtype=torch.float64, device="cuda")
            if s["route"] is not None:
                ids = s["route"][b, h].long()
                times = torch.zeros_like(times).index_add_(0, ids[ids >= 0], torch.ones_like(ids[ids >= 0], dtype=torch.float64))
            for i in range(h * c["group"], (h + 1) * c["group"]):
                at = n - c["qt"] + torch.arange(c["qt"], device="cuda")[:, None]
                x = _score64(s["q"][b, :, i], k[:, h], c)
                if s["slopes"] is not None:
                    x = x - s["slopes"][i].double() * (at - token)
                out[b, :, i], lse[b, :, i] = _softmax64(x, times[token // c["chunk"]] * (token <= at), v[:, h])
    return {"out": out, "lse": lse}


def _rounded64(x, fmt):
    """(elements on their format's grid, exponents) from the definition: the least exponent by trial, the grid by its spacing."""
    most, least, bits, width = (448.0, -6, 3, x.shape[-1]) if fmt == "e4m3" else (6.0, 0, 1, 32)
    x = x.double().unflatten(-1, (-1, width))
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / most)) - 1
    for _ in range(2):
        e = torch.where(top > most * _two(e), e + 1, e)
    e = torch.where(top > 0, e.clamp(min=-127), -127.0)
    y = x * _two(-e)[..., None]
    spacing = _two(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** least))).clamp(min=least) - bits)
    return (y / spacing).round() * spacing, e


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "masked":
        return _exact_masked(c, s)
    if c["kind"] == "cached":
        return _exact_cached(c, s)
    lens = _lengths(c)
    begin = s["start"].tolist()
    if c["kind"] == "read":
        at = [torch.arange(a, a + n, device="cuda") for a, n in zip(begin, lens)]
        return {"k": torch.cat([_rows64(c, s, 0, b, p) for b, p in enumerate(at)]), "v": torch.cat([_rows64(c, s, 1, b, p) for b, p in enumerate(at)])}
    rows = [_rounded64(s[x][:s["used"]], c["format"]) for x in ("k", "v")]
    if c["kind"] == "turn":
        k, v = ((y * _two(e)[..., None]).flatten(-2) for y, e in rows)
        return {"k": k, "v": v}
    codes, r = torch.zeros(s["codes"].shape, dtype=torch.float64, device="cuda"), 0
    for b, n in enumerate(lens):
        p = torch.arange(begin[b], begin[b] + n, device="cuda")
        for w in (0, 1):
            codes[s["table"][b, p // c["chunk"]].long(), :, w, p % c["chunk"]] = rows[w][0].flatten(-2)[r:r + n]
        r += n
    return {"codes": codes, "scales": None}
