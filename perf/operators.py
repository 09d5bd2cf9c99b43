"""Measured cases of the 4-bit key/value cache: writing and reading tokens,
attention over a visible range or over selected token ids, attention that
accumulates each token's weight, and eviction by that weight.

`own` chooses the side: False computes every pass in elementary torch
operations in 32 bits; True makes the calls that a user of the library makes.

The cache holds, per token slot and key/value head, D elements in blocks of
16: a block's scale is s = e4m3(amax / 6), its codes are e2m1(x / s), both
rounded to nearest even, and an element stands for s * e2m1(code).  Codes are
(pages, page_size, heads, D/2) bytes, element 2i in the low nibble; scales are
(pages, page_size, heads, D/16) bytes.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # magnitudes of the codes 0 .. 7


# ------------------------------------------------------------------- cases
def listed():
    heads8 = {"kv_heads": 8, "dim": 128, "page": 64}
    gqa = dict(heads8, group=8, dtype="bf16", cap=0.0, windowed=False)
    return [
        # one decode step of 16 sequences writes a token each
        dict(heads8, name="store_step", op="store", tokens=16, dtype="bf16"),
        # a prompt chunk of 8192 tokens enters the cache
        dict(heads8, name="store_prompt", op="store", tokens=8192, dtype="bf16"),
        # a single user's decode step over a short context: latency
        dict(gqa, name="attend_one", op="attend", rows=1, longest=2048, shortest=2048),
        # the decode batch of 16 rows, contexts of all lengths up to 4 shards of 4096
        dict(gqa, name="attend_step", op="attend", rows=16, longest=16384, shortest=1),
        # a full serving batch
        dict(gqa, name="attend_batch", op="attend", rows=256, longest=8192, shortest=64),
        # two long documents
        dict(gqa, name="attend_long", op="attend", rows=2, longest=131072, shortest=100003),
        # no shared heads, small heads, odd lengths, a sliding window, capped scores
        {"name": "attend_odd", "op": "attend", "rows": 33, "longest": 4097, "shortest": 1,
         "kv_heads": 12, "group": 1, "dim": 64, "page": 16, "dtype": "f16", "cap": 30.0,
         "windowed": True},
        # a decode step that also accumulates the tokens' weights for a later eviction
        dict(gqa, name="attend_weights", op="weights", rows=8, longest=16384, shortest=8192),
        # a decode step over the 2048 ids of the top-K merge, 16 sequences
        dict(gqa, name="select_step", op="select", rows=16, ids=2048, longest=16384,
             shortest=1024, shared=False),
        # a prompt chunk: 1024 query rows of one sequence, each with its own 2048 ids
        dict(gqa, name="select_prompt", op="select", rows=1024, ids=2048, longest=32768,
             shortest=31745, shared=True),
        # one long sequence cut down to 8192 tokens
        dict(heads8, name="evict_long", op="evict", rows=1, longest=131072, shortest=131072,
             budget=8192, sinks=4, recent=1024),
        # a batch of sequences brought back to 4096 tokens each
        dict(heads8, name="evict_batch", op="evict", rows=32, longest=16384, shortest=3000,
             budget=4096, sinks=4, recent=512),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "weights", "select", "select", "evict"])
    c = {"op": op, "kv_heads": rng.choice([1, 2, 4, 5, 8, 12]), "dim": rng.choice([64, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 128])}
    width = c["kv_heads"] * c["dim"]
    if op == "store":
        c.update(tokens=_spread(rng, 1, 8192 * 1024 // max(1024, width)),
                 dtype=rng.choice(["bf16", "f16", "f32"]))
        return c
    if op == "evict":
        c["rows"] = _spread(rng, 1, 32)
        c["longest"] = _spread(rng, 64, min(131072, 16384 * 32 // c["rows"]))
        c["shortest"] = rng.randint(1, c["longest"])
        c["budget"] = _spread(rng, 16, max(16, min(8192, c["longest"])))
        c["sinks"] = rng.choice([0, 4, c["budget"] // 8])
        c["recent"] = rng.choice([0, 1, c["budget"] // 4])
        return c
    c.update(group=rng.choice([1, 2, 3, 4, 7, 8, 16]), dtype=rng.choice(["bf16", "f16"]),
             cap=rng.choice([0.0, 0.0, 30.0]), windowed=rng.random() < 0.25)
    room = 2 ** 28 // (c["kv_heads"] * c["dim"] * max(1, c["group"] // 8))  # rows * tokens
    if op == "select":
        c["shared"] = rng.random() < 0.5
        c["rows"] = _spread(rng, 1, 512)
        c["ids"] = _spread(rng, 1, max(1, min(4096, room // c["rows"])))
        c["longest"] = _spread(rng, c["ids"], max(c["ids"], 32768 if c["shared"]
                                                  else min(131072, room // c["rows"])))
        c["shortest"] = rng.randint(1, c["longest"])
    else:
        c["rows"] = _spread(rng, 1, 256 if op == "attend" else 32)
        c["longest"] = _spread(rng, 1, max(1, min(131072, room // c["rows"])))
        c["shortest"] = rng.randint(1, c["longest"])
    return c


def _lengths(case):
    """The rows' lengths, evenly spaced from the longest to the shortest."""
    n = case["rows"]
    return [case["longest"] - (case["longest"] - case["shortest"]) * i // max(1, n - 1)
            for i in range(n)]


def _window(case, length):
    """First visible token of a row of this length."""
    return length // 3 if case.get("windowed") else 0


# ------------------------------------------------------------------ inputs
def _encode(x):
    """Codes and scales of x (..., D) in the cache's format, in 32 bits."""
    x = x.float().unflatten(-1, (-1, 16))
    a = x.abs()
    s = (a.amax(-1, keepdim=True) / torch.full((), 6.0, device=x.device)).clamp(max=448.0)
    s8 = s.to(torch.float8_e4m3fn)
    s = s8.float()
    code = ((a > 0.25 * s).byte() + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s)
            + (a > 2.5 * s) + (a >= 3.5 * s) + (a > 5.0 * s))
    code = torch.where(s > 0, code + 8 * (x < 0).byte(), 0).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8).squeeze(-1)


def _decode(codes, scales):
    """What codes (..., D/2) and scales (..., D/16) stand for, in 32 bits."""
    grid = torch.tensor(GRID + [-g for g in GRID], device=codes.device)
    pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], -1)  # by byte
    x = pairs[codes.long()].flatten(-2).unflatten(-1, (-1, 16))
    return (x * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    H, D, P = case["kv_heads"], case["dim"], case["page"]

    def normal(*shape):
        # keys and values: a few channels much larger than the rest
        x = torch.randn(*shape, generator=g, device=dev)
        return x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=dev))

    state = {"case": dict(case)}
    if case["op"] == "store":
        n = case["tokens"]
        # keys and values are slices of a fused projection's output
        fused = normal(n, 3 * H, D).to(DTYPES[case["dtype"]])
        pages = -(-n // P) + 1
        # tokens follow each other within pages that lie in any order
        order = torch.randperm(pages, generator=g, device=dev)
        slots = (order[:, None] * P + torch.arange(P, device=dev)).flatten()[:n]
        state.update(k=fused[:, H:2 * H], v=fused[:, 2 * H:], slots=slots)
    else:
        evict = case["op"] == "evict"
        one = bool(case.get("shared"))  # all rows are rows of one sequence
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        if not one:
            lens = lens[torch.randperm(len(lens), generator=g, device=dev)]
        owned = lens.amax().view(1) if one else lens
        per = (owned + P - 1) // P  # pages of each sequence
        first = torch.cumsum(per, 0) - per
        width = -(-case["longest"] // P)
        used = int(per.sum())
        at = torch.arange(width, device=dev)
        order = torch.randperm(used, generator=g, device=dev).int()
        table = torch.where(at < per[:, None], order[(first[:, None] + at).clamp(max=used - 1)], -1)
        pages = used + (case["rows"] * -(-case["budget"] // P) if evict else 0)
        state.update(table=table.int().contiguous(), lens=lens)
    planes = [torch.zeros(pages, P, H, w, dtype=torch.uint8, device=dev)
              for w in (D // 2, D // 2, D // 16, D // 16)]
    state.update(zip(("k_codes", "v_codes", "k_scales", "v_scales"), planes))
    if case["op"] == "store":
        return state
    state["k_codes"][:used], state["k_scales"][:used] = _encode(normal(used, P, H, D).bfloat16())
    state["v_codes"][:used], state["v_scales"][:used] = _encode(normal(used, P, H, D).bfloat16())
    if evict:
        out = torch.arange(used, pages, device=dev, dtype=torch.int32)
        state["out_table"] = out.view(case["rows"], -1)
        state["first_out"] = used
        # accumulated weights: a few heavy tokens, many light ones that tie
        w = torch.rand(case["rows"], case["longest"], generator=g, device=dev)
        state["weights"] = torch.round(w ** 6 * 4096) / 256
        return state
    Hq = H * case["group"]
    fused = torch.randn(case["rows"], Hq + 2 * H, D, generator=g, device=dev)
    state["q"] = (2.0 * fused).to(DTYPES[case["dtype"]])[:, :Hq]
    state["starts"] = (lens // 3).int() if case["windowed"] else None
    if case["op"] == "weights":
        state["weights"] = torch.zeros(case["rows"], case["longest"], device=dev)
    if case["op"] == "select":
        # distinct tokens of each row's visible range in an order of their own, then padding
        order = torch.rand(case["rows"], case["longest"], generator=g, device=dev)
        order[torch.arange(case["longest"], device=dev) >= lens[:, None]] = 2.0
        ids = order.argsort(-1)[:, :case["ids"]].int()
        state["ids"] = torch.where(ids < lens[:, None], ids, -1).contiguous()
        state["owner"] = torch.zeros_like(lens) if one else None
    return state


# ------------------------------------------------------------- plain forms
def _plain_store(s):
    for_k, for_v = _encode(s["k"]), _encode(s["v"])
    at = s["slots"]
    for_all = for_k[:1] + for_v[:1] + for_k[1:] + for_v[1:]
    planes = s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]
    [p.flatten(0, 1).index_copy_(0, at, x) for p, x in zip(planes, for_all)]
    kc, vc, ks, vs = [p.flatten(0, 1)[at] for p in planes]
    return [_decode(kc, ks).to(s["k"].dtype), _decode(vc, vs).to(s["v"].dtype)]


def _tokens_of(s):
    """The rows' tokens as positions (rows, n), whether each is visible, and
    its slot in the cache."""
    c = s["case"]
    if c["op"] == "select":
        pos = s["ids"].long()
    else:
        pos = torch.arange(c["longest"], device=s["lens"].device).expand(c["rows"], -1)
    seen = (pos >= 0) & (pos < s["lens"][:, None])
    if s["starts"] is not None:
        seen = seen & (pos >= s["starts"][:, None])
    table = s["table"].expand(c["rows"], -1) if c.get("shared") else s["table"]
    at = torch.where(seen, pos, 0)
    page = torch.gather(table.long(), 1, at // c["page"])
    slot = torch.where(seen, page * c["page"] + at % c["page"], 0)
    return seen, slot


def _plain_attend(s):
    c = s["case"]
    seen, slot = _tokens_of(s)
    kc, vc, ks, vs = [s[n].flatten(0, 1) for n in ("k_codes", "v_codes", "k_scales", "v_scales")]
    q = s["q"].float().unflatten(1, (c["kv_heads"], c["group"]))  # rows, kv, group, D
    k = _decode(kc[slot], ks[slot]).transpose(1, 2)  # rows, kv, tokens, D
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(c["dim"])
    del k
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total > 0, total, 1.0)
    v = _decode(vc[slot], vs[slot]).transpose(1, 2)
    out = torch.matmul(x, v).flatten(1, 2).to(s["q"].dtype)
    lse = (top + torch.log(total)).flatten(1, 3)
    if c["op"] != "weights":
        return [out, lse]
    s["weights"] += x.sum((1, 2))
    return [out, lse, s["weights"]]


def _plain_evict(s):
    c = s["case"]
    dev = s["lens"].device
    n, budget = s["lens"][:, None].long(), c["budget"]
    pos = torch.arange(c["longest"], device=dev)[None]
    spared = (n <= budget) | (pos < c["sinks"]) | (pos >= n - c["recent"])
    order = torch.where(spared, math.inf, s["weights"])
    order = torch.where(pos < n, order, -math.inf)
    best = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :budget]
    kept_n = n.clamp(max=budget)
    rank = torch.arange(best.shape[1], device=dev)[None]
    kept = torch.where(rank < kept_n, best, c["longest"]).sort(1).values
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[1]), value=c["longest"])
    rank = torch.arange(budget, device=dev)[None]
    live = rank < kept_n
    at = torch.where(live, kept, 0)
    src = torch.gather(s["table"].long(), 1, at // c["page"]) * c["page"] + at % c["page"]
    dst = s["out_table"].long()[:, rank[0] // c["page"]] * c["page"] + rank % c["page"]
    planes = [s[x].flatten(0, 1) for x in ("k_codes", "v_codes", "k_scales", "v_scales")]
    [p.index_copy_(0, dst[live], p[src[live]]) for p in planes]
    return _evicted(s, torch.where(live, kept, -1).int(), kept_n[:, 0].int(),
                    torch.where(live, torch.gather(s["weights"], 1, at), 0.0))


def _evicted(s, kept, lens, weights):
    """An eviction's outputs: the choice, and the pages that it filled.  It
    moves the cache's bytes and computes none of them: they are compared as
    they are."""
    f = s["first_out"]
    return [kept, lens, weights, s["k_codes"][f:], s["v_codes"][f:], s["k_scales"][f:],
            s["v_scales"][f:]]


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"store": _plain_store, "evict": _plain_evict}.get(op, _plain_attend)(state)


def _own(s, op):
    import sparse_attention_indexer_stable_gb300 as dk

    cache = s.get("cache")
    if cache is None:  # the handle that a program makes once beside its pages
        cache = s["cache"] = dk.Kv4Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    if op == "store":
        dk.kv4_append(cache, s["k"], s["v"], s["slots"])
        k, v = dk.kv4_read(cache, s["slots"], dtype=s["k"].dtype)
        return [k, v]
    c = s["case"]
    if op == "evict":
        kept, lens, weights = dk.kv4_evict(cache, s["table"], s["lens"], s["weights"],
                                           s["out_table"], c["budget"], sinks=c["sinks"],
                                           recent=c["recent"])
        return _evicted(s, kept, lens, weights)
    out, lse = dk.kv4_attention(cache, s["q"], s["table"], s["lens"], ids=s.get("ids"),
                                owner=s.get("owner"), starts=s["starts"], softcap=c["cap"],
                                weights=s.get("weights"))
    return [out, lse, s["weights"]] if op == "weights" else [out, lse]


# -------------------------------------------------------------- work, exact
def work(case):
    H, D = case["kv_heads"], case["dim"]
    slot = 2 * H * (D // 2 + D // 16)  # a token's bytes in the cache
    if case["op"] == "store":  # written once, read once; the values in and out
        n = case["tokens"]
        wide = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * slot + 4 * n * H * D * wide + 16 * n, "flops": 0}
    lens = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * slot + 12), "flops": 0}
    seen = [n - _window(case, n) for n in lens]
    extra = 0
    if case["op"] == "select":
        share = [min(1.0, case["ids"] / n) for n in lens]
        seen = [m * f for m, f in zip(seen, share)]
        extra = 4 * case["rows"] * case["ids"]
    tokens = sum(seen)
    if case["op"] == "weights":
        extra = 8 * tokens
    Hq = H * case["group"]
    once = min(tokens, case["longest"]) if case.get("shared") else tokens
    return {"bytes": once * slot + extra + case["rows"] * Hq * (4 * D + 4),
            "flops": 4.0 * tokens * Hq * D}


def _exact_step(a, low, bits):
    """a >= 0 rounded to nearest even with `bits` significant bits and no
    exponent below `low`, in 64 bits."""
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** (low - 4))))
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, torch.where(torch.exp2(e) > a, e - 1, e))
    step = torch.exp2(e.clamp(min=low) - (bits - 1))
    return torch.round(a / step) * step


def _exact_values(x):
    x = x.double().unflatten(-1, (-1, 16))
    s = _exact_step(x.abs().amax(-1, keepdim=True) / 6, -6, 4).clamp(max=448)
    y = _exact_step(x.abs() / torch.where(s > 0, s, 1.0), 0, 2).clamp(max=6)
    return (torch.sign(x) * y * s).flatten(-2)


def _exact_cache(s, which, slots):
    """Elements (n, kv, D) of the slots, in 64 bits."""
    b = s[which + "_codes"].flatten(0, 1)[slots].int()
    c = torch.stack([b % 16, b // 16], -1).flatten(-2)
    e, m = c // 2 % 4, (c % 2).double()
    mag = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
    f = s[which + "_scales"].flatten(0, 1)[slots].int()
    fe, fm = f // 8, (f % 8).double()
    scale = torch.where(fe == 0, fm * 2.0 ** -9, torch.exp2(fe.double() - 7) * (1 + fm / 8))
    return torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(16, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return [_exact_values(s["k"]), _exact_values(s["v"])]
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        rows = []
        for b, n in enumerate(lens):
            w, keep = s["weights"][b, :n], torch.ones(n, dtype=torch.bool, device="cuda")
            if n > case["budget"]:
                lo, hi = case["sinks"], n - case["recent"]
                keep[lo:hi] = False
                take = case["budget"] - case["sinks"] - case["recent"]
                keep[lo + torch.argsort(-w[lo:hi].double(), stable=True)[:take]] = True
            row = torch.zeros(case["budget"], dtype=torch.float64, device="cuda")
            row[:int(keep.sum())] = w[keep].double()
            rows.append(row)
        return [None, None, torch.stack(rows), None, None, None, None]
    out, lse, weights = [], [], []
    for t, n in enumerate(lens):
        if case["op"] == "select":
            pos = s["ids"][t].long()
            pos = pos[(pos >= _window(case, n)) & (pos < n)]
        else:
            pos = torch.arange(_window(case, n), n, device="cuda")
        table = s["table"][0 if case.get("shared") else t].long()
        slots = table[pos // case["page"]] * case["page"] + pos % case["page"]
        k, v = _exact_cache(s, "k", slots), _exact_cache(s, "v", slots)
        q = s["q"][t].double().unflatten(0, (case["kv_heads"], case["group"]))
        x = torch.einsum("hgd,nhd->hgn", q, k) * case["dim"] ** -0.5
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        lse.append(torch.logsumexp(x, -1).flatten())
        p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) if len(pos) else x
        out.append(torch.einsum("hgn,nhd->hgd", p, v).flatten(0, 1))
        w = torch.zeros(case["longest"], dtype=torch.float64, device="cuda")
        w[pos] = p.sum((0, 1))
        weights.append(w)
    got = [torch.stack(out), torch.stack(lse)]
    return got + [torch.stack(weights)] if case["op"] == "weights" else got
