"""Measured cases of a batch's way into the 4-bit key/value cache: pages and
slots for its new tokens, rotary positions of its queries and keys, and
attention over whole prompts.

`own` chooses the side: False computes every pass in elementary torch
operations; True makes the calls that a user of the library makes.

extend   Sequence b holds lens[b] tokens and gets counts[b] more.  It takes the
         pages that these need from a list of free ones, and every new token
         learns its slot, position, sequence and number of visible tokens;
         places behind the last token are padding.
rotary   Elements i and i + R/2 (or 2i and 2i + 1: interleaved) of a head's
         first R turn by position * frequency[i].  The frequencies are
         base^(-2i/R); for long contexts those of few turns over the original
         length are divided by a factor, those of many are kept, with a linear
         blend between, and the turned elements are scaled by `magnitude`.
prompt   Row i of a sequence sees its rows j <= i (all rows where not causal),
         with a window only those with j > i - window.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SLOW, FAST = 1.0, 32.0  # turns over the original length: all of the factor, none of it


# ------------------------------------------------------------------- cases
def listed():
    heads8 = {"kv_heads": 8, "group": 8, "dim": 128, "dtype": "bf16"}
    prompt = dict(heads8, op="prompt", seqs=1, causal=True, window=0, cap=0.0)
    rotary = dict(heads8, op="rotary", turned=128, interleaved=False, factor=1.0, original=0)
    return [
        # a decode step's bookkeeping: 256 sequences, most with one new token, the places of a
        # captured graph's batch
        {"name": "extend_step", "op": "extend", "seqs": 256, "page": 64, "longest": 8192,
         "shortest": 0, "counts": 1, "idle": True, "places": 256},
        # prompts of many lengths join sequences that are under way
        {"name": "extend_prompts", "op": "extend", "seqs": 64, "page": 16, "longest": 30000,
         "shortest": 0, "counts": 2000, "idle": True, "places": 65536},
        # a decode step of 16 rows: latency
        dict(rotary, name="rotary_step", tokens=16, longest=16384),
        # a prompt chunk
        dict(rotary, name="rotary_prompt", tokens=16384, longest=16384),
        # half of each head, interleaved, far positions of a context stretched eightfold
        {"name": "rotary_part", "op": "rotary", "tokens": 4097, "kv_heads": 5, "group": 3,
         "dim": 128, "turned": 64, "dtype": "f16", "interleaved": True, "longest": 1000003,
         "factor": 8.0, "original": 131072},
        # a short question: latency
        dict(prompt, name="prompt_short", longest=100, shortest=100),
        # a chat's prompt
        dict(prompt, name="prompt_chat", longest=2048, shortest=2048),
        # prompts of all lengths packed into one batch
        dict(prompt, name="prompt_packed", seqs=48, longest=1500, shortest=1),
        # a long document
        dict(prompt, name="prompt_long", longest=16384, shortest=16384),
        # wide heads
        dict(prompt, name="prompt_wide", seqs=2, longest=4096, shortest=4001, kv_heads=4, group=4,
             dim=256),
        # no shared heads, small heads, odd lengths, a sliding window, capped scores
        {"name": "prompt_odd", "op": "prompt", "seqs": 33, "longest": 4097, "shortest": 1,
         "kv_heads": 12, "group": 1, "dim": 64, "dtype": "f16", "cap": 30.0, "window": 1000,
         "causal": True},
        # texts that are read as a whole, for a later ranking of them
        {"name": "prompt_both", "op": "prompt", "seqs": 16, "longest": 2048, "shortest": 300,
         "kv_heads": 4, "group": 7, "dim": 64, "dtype": "bf16", "cap": 0.0, "window": 0,
         "causal": False},
    ]


MOST = 4.4e12  # operations of prompt_long


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "rotary", "prompt", "prompt", "prompt"])
    if op == "extend":
        c = {"op": op, "seqs": _spread(rng, 1, 512), "page": rng.choice([1, 16, 32, 64, 128])}
        c["counts"] = 1 if rng.random() < 0.4 else _spread(rng, 1, max(1, 65536 // c["seqs"]))
        c["longest"] = _spread(rng, 1, 32768 if c["page"] > 1 else 4096)
        c["shortest"] = rng.randint(0, c["longest"])
        c["idle"] = rng.random() < 0.5
        c["places"] = c["seqs"] * c["counts"] + rng.choice([0, 0, 1, 37])
        return c
    c = {"op": op, "kv_heads": rng.choice([1, 2, 4, 5, 8, 12]),
         "group": rng.choice([1, 2, 3, 4, 7, 8, 16]), "dim": rng.choice([64, 128, 128, 256])}
    heads = c["kv_heads"] * c["group"]
    if op == "rotary":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["tokens"] = _spread(rng, 1, min(65536, 16384 * 72 * 128 // 2 //
                                          ((heads + c["kv_heads"]) * c["dim"])))
        c["turned"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32, 2])
        c["interleaved"] = rng.random() < 0.5
        c["longest"] = _spread(rng, 1, 2000000)
        c["factor"] = rng.choice([1.0, 1.0, 4.0, 32.0])
        c["original"] = rng.choice([0, 4096, 32768]) if c["factor"] > 1.0 else 0
        return c
    c.update(dtype=rng.choice(["bf16", "f16"]), cap=rng.choice([0.0, 0.0, 0.0, 30.0]),
             causal=rng.random() < 0.75, window=0)
    c["longest"] = _spread(rng, 1, 16384)
    most = 32768 * 64 // max(64, heads)  # rows of the batch
    c["longest"] = min(c["longest"], most)
    c["seqs"] = _spread(rng, 1, max(1, min(64, most // c["longest"])))
    c["shortest"] = rng.randint(0, c["longest"])
    if rng.random() < 0.25:
        c["window"] = _spread(rng, 1, c["longest"])
    while work(c)["flops"] > MOST:
        c["longest"] = c["longest"] * 3 // 4
        c["shortest"] = min(c["shortest"], c["longest"])
    return c


def _lengths(case):
    """The sequences' lengths, evenly spaced from the longest to the shortest."""
    n = case["seqs"]
    return [case["longest"] - (case["longest"] - case["shortest"]) * i // max(1, n - 1)
            for i in range(n)]


def _counts(case):
    """New tokens of each sequence: all lengths up to the most, some none."""
    n, most = case["seqs"], case["counts"]
    return [0 if case["idle"] and i % 5 == 3 else most - (most - 1) * i // max(1, n - 1)
            for i in range(n)]


def _frequencies(case):
    """Radians a position for each pair, and the factor of the turned elements."""
    r, factor = case["turned"], case["factor"]
    f = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    if factor == 1.0:
        return f, 1.0
    if not case["original"]:
        return [x / factor for x in f], 1.0
    keep = [min(1.0, max(0.0, (case["original"] * x / (2.0 * math.pi) - SLOW) / (FAST - SLOW)))
            for x in f]
    return [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    state = {"case": dict(case)}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if case["op"] == "extend":
        P, n = case["page"], case["seqs"]
        lens = i32(_lengths(case))[torch.randperm(n, generator=g, device=dev)]
        counts = i32(_counts(case))[torch.randperm(n, generator=g, device=dev)]
        held = (lens + P - 1) // P
        width = -(-(case["longest"] + case["counts"]) // P)
        owned, spare = int(held.sum()), n * (case["counts"] // P + 1)
        pages = torch.randperm(owned + spare + 7, generator=g, device=dev).int()
        at = torch.arange(width, device=dev)
        first = torch.cumsum(held, 0) - held
        table = torch.where(at < held[:, None], pages[(first[:, None] + at).clamp(max=owned)], -1)
        # seven pages of the list were given away by earlier steps
        state.update(table=table.int().contiguous(), lens=lens, counts=counts, used=i32([7]),
                     free=pages[owned:].contiguous(), pages=owned + spare + 7)
        return state

    H, D, Hq = case["kv_heads"], case["dim"], case["kv_heads"] * case["group"]

    def fused(rows):
        """Queries, keys and values as slices of a fused projection's output, a
        few channels larger than the rest."""
        x = torch.randn(rows, Hq + 2 * H, D, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(D, generator=g, device=dev))
        x[:, :Hq] *= 1.5
        x = x.to(DTYPES[case["dtype"]])
        return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]

    if case["op"] == "rotary":
        state["q"], state["k"], _ = fused(case["tokens"])
        state["positions"] = torch.randint(0, case["longest"], (case["tokens"],), generator=g,
                                           device=dev, dtype=torch.int32)
        state["freq"], state["magnitude"] = _frequencies(case)
        return state
    lens = i32(_lengths(case))[torch.randperm(case["seqs"], generator=g, device=dev)]
    state["lens"] = lens.tolist()
    state["starts"] = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0)).int()
    state["q"], state["k"], state["v"] = fused(sum(state["lens"]))
    return state


# ------------------------------------------------------------- plain forms
def _plain_extend(s):
    c = s["case"]
    P, N, dev = c["page"], c["places"], s["lens"].device
    width, B = s["table"].shape[1], c["seqs"]
    lens = s["lens"].long().clamp(min=0)
    ends = torch.cumsum(s["counts"].long().clamp(min=0), 0).clamp(max=N)
    starts = torch.nn.functional.pad(ends, (1, 0))
    grown = lens + ends - starts[:-1]
    had = ((lens + P - 1) // P).clamp(max=width)
    need = ((grown + P - 1) // P).clamp(max=width) - had
    first = s["used"].long() + torch.cumsum(need, 0) - need
    at = torch.arange(width, device=dev)
    take = first[:, None] + at - had[:, None]
    found = torch.where(take < len(s["free"]), s["free"][take.clamp(0, len(s["free"]) - 1)], -1)
    fresh = (at >= had[:, None]) & (at < (had + need)[:, None])
    table = s["table"]
    table.copy_(torch.where(fresh, found, table))
    t = torch.arange(N, device=dev)
    owner = torch.searchsorted(ends, t, right=True)
    live = owner < B
    b = owner.clamp(max=B - 1)
    position = torch.where(live, lens[b] + t - starts[b], 0)
    page = table[b, (position // P).clamp(max=width - 1)].long()
    ok = live & (position // P < width) & (page >= 0) & (page < s["pages"])
    return [torch.where(ok, page * P + position % P, -1), position.int(),
            torch.where(live, owner, -1).int(), torch.where(live, position + 1, 0).int(),
            starts.int(), grown.int(), (s["used"] + need.sum()).int(), table]


def _turn(x, cos, sin, case):
    """x (n, heads, D) with its first R elements turned."""
    r = case["turned"]
    cos, sin = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rotary(s):
    # angles in 64 bits: 32 would leave a far position's whole turns inexact
    freq = torch.tensor(s["freq"], dtype=torch.float64, device=s["q"].device)
    angle = s["positions"].double()[:, None] * freq
    cos = (torch.cos(angle) * s["magnitude"]).float()
    sin = (torch.sin(angle) * s["magnitude"]).float()
    return [_turn(x.float(), cos, sin, s["case"]).to(x.dtype) for x in (s["q"], s["k"])]


def _seen(case, i, j):
    """Which of the keys j (n,) the rows i (m,) see, (m, n)."""
    ok = torch.ones(len(i), len(j), dtype=torch.bool, device=i.device)
    if case["causal"]:
        ok &= j <= i[:, None]
    if case["window"]:
        ok &= j > i[:, None] - case["window"]
    return ok


def _pieces(case, lens, entries):
    """(first row of the sequence, rows lo..hi, keys from..to) of the batch, each
    with about `entries` scores."""
    at = 0
    heads = case["kv_heads"] * case["group"]
    for n in lens:
        step = min(1024, max(16, entries // (heads * max(1, n))))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            first = max(0, lo - case["window"] + 1) if case["window"] else 0
            yield at, lo, hi, first, hi if case["causal"] else n
        at += n


def _plain_prompt(s):
    c, dev = s["case"], s["q"].device
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    for at, lo, hi, first, last in _pieces(c, s["lens"], 2 ** 30):
        a = q[at + lo:at + hi].float().unflatten(1, (c["kv_heads"], c["group"])).permute(1, 2, 0, 3)
        b = k[at + first:at + last].float().permute(1, 2, 0)[:, None]
        x = torch.matmul(a, b) / math.sqrt(c["dim"])  # kv, group, rows, keys
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        ok = _seen(c, torch.arange(lo, hi, device=dev), torch.arange(first, last, device=dev))
        x.masked_fill_(~ok, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        y = torch.matmul(x, v[at + first:at + last].float().permute(1, 0, 2)[:, None]) / total
        out[at + lo:at + hi] = y.permute(2, 0, 1, 3).flatten(1, 2).to(q.dtype)
        lse[at + lo:at + hi] = (top + torch.log(total))[..., 0].permute(2, 0, 1).flatten(1)
    return [out, lse]


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"extend": _plain_extend, "rotary": _plain_rotary, "prompt": _plain_prompt}[op](state)


def _own(s, op):
    import sparse_attention_indexer_stable_gb300 as dk

    c = s["case"]
    if op == "extend":
        step = dk.kv4_extend(s["table"], s["lens"], s["counts"], s["free"], s["used"],
                             places=c["places"], page_size=c["page"], num_pages=s["pages"])
        return [step.slots, step.positions, step.owner, step.row_lens, step.starts, step.lens,
                step.used, s["table"]]
    if op == "rotary":
        rope = s.get("rope")
        if rope is None:  # the handle that a program makes once
            rope = s["rope"] = dk.Rotary(c["turned"], base=10000.0, interleaved=c["interleaved"],
                                         factor=c["factor"], original=c["original"], slow=SLOW,
                                         fast=FAST)
        return list(dk.rotary(rope, s["positions"], s["q"], s["k"]))
    out, lse = dk.prompt_attention(s["q"], s["k"], s["v"], s["starts"], causal=c["causal"],
                                   window=c["window"], softcap=c["cap"])
    return [out, lse]


# -------------------------------------------------------------- work, exact
def _pairs(case, n):
    """Visible (row, key) pairs of a sequence of n rows."""
    w = min(case["window"] or n, n)
    seen = w * (w + 1) // 2 + (n - w) * w  # j <= i, j > i - w
    if case["causal"]:
        return seen
    return seen + n * (n - 1) // 2


def work(case):
    if case["op"] == "extend":
        P = case["page"]
        new = _counts(case)
        return {"bytes": 20 * case["places"] + 16 * case["seqs"] + 12 * sum(-(-n // P) for n in new),
                "flops": 0}
    H, D, Hq = case["kv_heads"], case["dim"], case["kv_heads"] * case["group"]
    if case["op"] == "rotary":
        wide = 4 if case["dtype"] == "f32" else 2
        n = case["tokens"] * (Hq + H)
        return {"bytes": 2 * n * D * wide + 4 * case["tokens"], "flops": 3 * n * case["turned"]}
    lens = _lengths(case)
    pairs = sum(_pairs(case, n) for n in lens)
    return {"bytes": sum(lens) * (4 * Hq * D + 4 * H * D + 4 * Hq), "flops": 4.0 * pairs * Hq * D}


def exact(case, seed):
    if case["op"] == "extend":
        return None  # whole numbers throughout
    s = prepare(case, seed)
    if case["op"] == "rotary":
        freq = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
        turned = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"),
                             s["positions"].double()[:, None] * freq)[:, None]
        r, got = case["turned"], []
        for x in (s["q"], s["k"]):
            y = x.double()
            head = y[..., :r].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
            first, second = head.unbind(-1 if case["interleaved"] else -2)
            z = torch.complex(first.contiguous(), second.contiguous()) * turned
            z = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).flatten(-2)
            got.append(torch.cat([z, y[..., r:]], -1))
        return got
    if work(case)["flops"] > 6e12:
        return None
    H, G = case["kv_heads"], case["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for at, lo, hi, first, last in _pieces(case, s["lens"], 2 ** 29):
        rows, keys = slice(at + lo, at + hi), slice(at + first, at + last)
        ok = _seen(case, torch.arange(lo, hi, device="cuda"),
                   torch.arange(first, last, device="cuda"))
        for h in range(H):
            a = s["q"][rows, h * G:(h + 1) * G].double().transpose(0, 1)  # group, rows, D
            x = a @ s["k"][keys, h].double().T * case["dim"] ** -0.5
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            x = torch.where(ok, x, -math.inf)
            e = torch.logsumexp(x, -1)
            lse[rows, h * G:(h + 1) * G] = e.T
            out[rows, h * G:(h + 1) * G] = (torch.exp(x - e[..., None])
                                            @ s["v"][keys, h].double()).transpose(0, 1)
    return [out, lse]
