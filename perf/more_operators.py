"""The int8 K/V cache and the attention over shared prefixes, as measured cases.

Five operators, each over the paged cache that the serving calls share:

- ``insert``: K and V of new tokens quantised to int8, one power-of-two scale per token and KV head, as they are written
  into the cache; the rows are read back as the values that they stand for;
- ``gather``: ranges of the requests' contexts read back from the int8 cache as packed bf16 K and V;
- ``shared``: attention of a batch whose requests share long prefixes, over a bf16, E4M3 or int8 cache;
- ``chunk``: attention of each request's new tokens over all its keys in an int8 cache;
- ``sparse``: the decode attention over selected blocks of an int8 cache.

``run`` gives each in its plain form (elementary torch operations in 32 bits; the quantisation is exact in them), or,
where ``own`` is true, as the package's calls.
"""
import math
import random

import torch

own = False

HEADS, KV_HEADS, DIM, PAGE, TOPK = 64, 4, 128, 128, 16
GROUP = HEADS // KV_HEADS
LOG2E = 1.0 / math.log(2.0)


# ---- the cases ------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 requests writes one token each: latency
        {"name": "insert 64 x 1", "op": "insert", "requests": 64, "min_new": 1, "max_new": 1, "mix": 1},
        # a step of prompts in chunks, of odd lengths
        {"name": "insert 9 chunks, 16k", "op": "insert", "requests": 9, "min_new": 1333, "max_new": 2222, "mix": 2},
        # the ends of four chats read back, from inside a page
        {"name": "gather 4, short", "op": "gather", "requests": 4, "min_len": 100, "max_len": 700, "mix": 3},
        # whole contexts read back for a recomputation
        {"name": "gather 8, up to 32k", "op": "gather", "requests": 8, "min_len": 4096, "max_len": 32768, "mix": 4},
        # four chats that begin with the same instructions: the smallest decode step
        {"name": "shared 4 x 1, 2k", "op": "shared", "groups": 1, "requests": 4, "alone": 0, "prefix": 2048, "min_own": 20,
         "max_own": 500, "max_new": 1, "cache": "bf16", "lse": False, "mix": 5},
        # a decode step of 64 requests about one document
        {"name": "shared 64 x 1, 16k", "op": "shared", "groups": 1, "requests": 64, "alone": 0, "prefix": 16421,
         "min_own": 100, "max_own": 2000, "max_new": 1, "cache": "bf16", "lse": False, "mix": 6},
        # many samples of one long prompt, FP8 cache
        {"name": "shared 256 x 1, 32k, E4M3", "op": "shared", "groups": 1, "requests": 256, "alone": 0, "prefix": 32768,
         "min_own": 1, "max_own": 1000, "max_new": 1, "cache": "e4m3", "lse": False, "mix": 7},
        # three prefixes, a few drafted tokens per request, some requests with none in common, log-sum-exp kept
        {"name": "shared 3 groups of 40, int8", "op": "shared", "groups": 3, "requests": 37, "alone": 3, "prefix": 5000,
         "min_own": 10, "max_own": 900, "max_new": 5, "cache": "int8", "lse": True, "mix": 8},
        # prompts in chunks at the end of their contexts
        {"name": "chunk 5 x 333-700, int8", "op": "chunk", "requests": 5, "min_len": 3000, "max_len": 16384,
         "min_new": 333, "max_new": 700, "lse": False, "mix": 9},
        # a decode step of 16 long contexts
        {"name": "chunk 16 x 1, 128k, int8", "op": "chunk", "requests": 16, "min_len": 131072, "max_len": 131072,
         "min_new": 1, "max_new": 1, "lse": True, "mix": 10},
        # a decode step of four short contexts over their selected blocks
        {"name": "sparse 4, 8k", "op": "sparse", "requests": 4, "min_len": 1, "max_len": 8192, "mix": 11},
        # a decode step of 64 requests of 4k to 64k keys over their selected blocks
        {"name": "sparse 64, 4k-64k", "op": "sparse", "requests": 64, "min_len": 4096, "max_len": 65536, "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["insert", "gather", "shared", "shared", "chunk", "sparse"])
    mix = rng.randrange(1000, 1 << 20)
    if op == "insert":
        requests = _log(rng, 1, 512)
        most = _log(rng, 1, max(1, 16384 // requests))
        return {"op": op, "requests": requests, "min_new": rng.choice([0, 1, most]), "max_new": most, "mix": mix}
    if op == "gather":
        requests = _log(rng, 1, 64)
        longest = _log(rng, 2, min(65536, 131072 // requests))
        return {"op": op, "requests": requests, "min_len": max(1, longest // rng.choice([1, 2, 50])), "max_len": longest,
                "mix": mix}
    if op == "shared":
        groups = rng.choice([1, 1, 2, 4])
        requests = _log(rng, 2, 256 // groups)
        prefix, longest = _log(rng, 100, 32768), _log(rng, 1, 4096)
        new = min(longest, rng.choice([1, 1, _log(rng, 2, 8)]))
        alone = rng.choice([0, 0, 2])
        # the largest listed case bounds the scores, and 2^19 the keys that are not shared
        while requests > 2 and (groups * requests * new * (prefix + longest) > 256 * 32768
                                or (groups * requests + alone) * longest > 1 << 19):
            requests = max(2, requests // 2)
        return {"op": op, "groups": groups, "requests": requests, "alone": alone, "prefix": prefix,
                "min_own": max(1, longest // rng.choice([1, 3, 40])), "max_own": longest, "max_new": new,
                "cache": rng.choice(["bf16", "e4m3", "int8"]), "lse": rng.random() < 0.5, "mix": mix}
    requests = _log(rng, 1, 64)
    longest = _log(rng, 130, 131072)
    if op == "sparse":
        while requests * longest > 64 * 65536:
            requests = (requests + 1) // 2
        return {"op": op, "requests": requests, "min_len": max(1, longest // rng.choice([1, 2, 1000])), "max_len": longest,
                "mix": mix}
    new = rng.choice([1, 1, _log(rng, 2, 700)])
    while requests > 1 and (requests * new * longest > 20000000 or requests * longest > 16 * 131072):
        requests = (requests + 1) // 2
    new = min(new, 20000000 // longest, longest)
    return {"op": op, "requests": requests, "min_len": max(1, longest // rng.choice([1, 2, 1000])), "max_len": longest,
            "min_new": min(new, rng.choice([1, new])), "max_new": new, "lse": rng.random() < 0.5, "mix": mix}


def _pages(n):
    return -(-n // PAGE)


def _sizes(case):
    """The requests of a case, from the case alone, as (group or -1, old, new): tokens that are there, and new ones (gather:
    where the range begins, and its length)."""
    rng = random.Random(case["mix"])
    if case["op"] == "insert":
        return [(-1, rng.randint(0, 500), rng.randint(case["min_new"] if r else case["max_new"], case["max_new"]))
                for r in range(case["requests"])]
    if case["op"] == "gather":
        return [(-1, rng.choice([0, rng.randint(0, 300)]), rng.randint(case["min_len"], case["max_len"]))
                for _ in range(case["requests"])]
    if case["op"] == "shared":
        out = []
        for g in range(case["groups"]):
            prefix = case["prefix"] - (case["prefix"] * g) // 7  # (the groups' prefixes differ)
            for _ in range(case["requests"]):
                new = rng.randint(1, case["max_new"])
                out.append((g, prefix + max(0, rng.randint(case["min_own"], case["max_own"]) - new), new))
        for _ in range(case["alone"]):
            new = rng.randint(1, case["max_new"])
            out.append((-1, rng.randint(0, case["max_own"]), new))
        return out
    out = []
    for _ in range(case["requests"]):
        new = rng.randint(case["min_new"], case["max_new"]) if case["op"] == "chunk" else 1
        out.append((-1, max(0, rng.randint(case["min_len"], case["max_len"]) - new), new))
    return out


def _shared_lens(case):
    return [case["prefix"] - (case["prefix"] * g) // 7 for g in range(case["groups"])]


def work(case):
    sizes = _sizes(case)
    t = sum(n for _, _, n in sizes)
    row8 = 2 * KV_HEADS * (DIM + 2)  # K and V of a token in the int8 cache
    row16 = 2 * KV_HEADS * DIM * 2
    if case["op"] == "insert":  # in, and back again
        return {"bytes": t * (2 * row16 + 2 * row8 + 8), "flops": 4 * t * 2 * KV_HEADS * DIM}
    if case["op"] == "gather":
        return {"bytes": t * (row16 + row8), "flops": t * 2 * KV_HEADS * DIM}
    if case["op"] == "sparse":
        keys = sum(min(o + n, (TOPK - 1) * PAGE + (o + n - 1) % PAGE + 1) for _, o, n in sizes)
        return {"bytes": keys * row8 + 2 * 2 * t * HEADS * DIM + 4 * KV_HEADS * t * TOPK, "flops": 4 * keys * HEADS * DIM}
    seen = sum(n * (o + n) - n * (n - 1) // 2 for _, o, n in sizes)  # (query, key) pairs
    row = row8 if case.get("cache", "int8") == "int8" else row16 // (2 if case["cache"] == "e4m3" else 1)
    keys = sum(o + n for _, o, n in sizes if n)
    if case["op"] == "shared":  # each group's common pages once
        for g, length in enumerate(_shared_lens(case)):
            keys -= (sum(1 for x, _, _ in sizes if x == g) - 1) * (length // PAGE * PAGE)
    return {"bytes": 2 * 2 * t * HEADS * DIM + keys * row + (4 * t * HEADS if case["lse"] else 0),
            "flops": 4 * seen * HEADS * DIM}


# ---- what a program has in hand --------------------------------------------------------------------------------

def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _table(case, sizes, gen):
    """A page table whose rows hold pages of a random permutation of the pool's, a group's rows the same common ones."""
    need = [_pages(o + n) for _, o, n in sizes]
    width = max(1, max(need))
    common = [length // PAGE for length in _shared_lens(case)] if case["op"] == "shared" else []
    total = sum(common) + sum(n - (common[g] if g >= 0 else 0) for (g, _, _), n in zip(sizes, need)) + 3
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.zeros(len(sizes), width, dtype=torch.int32, device="cuda")
    at = sum(common)
    starts = _offsets(common)
    for r, ((g, _, _), n) in enumerate(zip(sizes, need)):
        c = common[g] if g >= 0 else 0
        if c:
            table[r, :c] = perm[starts[g]:starts[g] + c]
        table[r, c:n] = perm[at:at + n - c]
        at += n - c
    return table, total


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    def int8_cache(pages):  # rows of normal values whose sizes differ
        cache = randn(pages * PAGE, KV_HEADS, DIM).mul_(40).round_().clamp_(-127, 127).to(torch.int8)
        scales = torch.exp2(torch.randint(-7, -4, (pages, KV_HEADS, PAGE), generator=gen, device="cuda").float())
        return cache, scales.bfloat16()

    sizes = _sizes(case)
    news = [n for _, _, n in sizes]
    table, pages = _table(case, sizes, gen)
    state = {"op": case["op"], "table": table, "max_new": max(news), "tokens": sum(news),
             "cu": _ints(_offsets(news)), "lens": _ints([o + n for _, o, n in sizes]),
             "old": _ints([o for _, o, _ in sizes])}
    kind = case.get("cache", "int8")
    if kind == "int8":
        state["k_cache"], state["k_scales"] = int8_cache(pages)
        state["v_cache"], state["v_scales"] = int8_cache(pages)
    else:
        state["k_cache"], state["v_cache"] = randn(pages * PAGE, KV_HEADS, DIM), randn(pages * PAGE, KV_HEADS, DIM)
        if kind == "e4m3":
            state["k_cache"] = state["k_cache"].to(torch.float8_e4m3fn)
            state["v_cache"] = state["v_cache"].to(torch.float8_e4m3fn)
    state["kind"], state["scale8"] = kind, {"k_scale": 0.5, "v_scale": 0.25} if kind == "e4m3" else {}
    t = sum(news)
    if case["op"] == "insert":
        kv = randn(t, 2 * KV_HEADS, DIM)  # a projection's output: k and v are its heads
        kv *= torch.exp2(torch.randint(-3, 4, (t, 2 * KV_HEADS, 1), generator=gen, device="cuda").float()).bfloat16()
        r = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), _ints(news).long())
        position = state["old"][r] + torch.arange(t, device="cuda") - state["cu"][r]
        page = table[r, position // PAGE].long()
        return dict(state, k=kv[:, :KV_HEADS], v=kv[:, KV_HEADS:], slots=page * PAGE + position % PAGE)
    if case["op"] == "gather":
        return state
    state["q"] = randn(t, HEADS, DIM)
    state["lse"] = case.get("lse", False)
    if case["op"] == "shared":
        n = case["requests"]
        common = _shared_lens(case)
        return dict(state, groups=_ints(_offsets([n] * case["groups"])), shared=_ints(common),
                    group=_ints([g for g, _, _ in sizes], torch.int64), max_group=max(sum(news[g * n:(g + 1) * n]) for g in range(case["groups"])),
                    max_shared=max(c // PAGE for c in common) * PAGE,
                    max_own=max(o + m - (common[g] // PAGE * PAGE if g >= 0 else 0) for g, o, m in sizes))
    if case["op"] == "sparse":  # the blocks that a selection keeps: the last one and the best of the others, in order
        blocks = (state["lens"].long() + PAGE - 1) // PAGE
        score = torch.rand(KV_HEADS, len(sizes), table.shape[1], generator=gen, device="cuda")
        b = torch.arange(table.shape[1], device="cuda")
        score = torch.where(b >= blocks[:, None], -1.0, torch.where(b == blocks[:, None] - 1, 2.0, score))
        if score.shape[-1] < TOPK:
            score = torch.nn.functional.pad(score, (0, TOPK - score.shape[-1]), value=-1.0)
        best = score.topk(TOPK, dim=-1)
        ids = torch.where(best.values < 0, 1 << 30, best.indices).sort(dim=-1).values
        state["q2k"] = torch.where(ids == 1 << 30, -1, ids).int().contiguous()
    return state


# ---- one pass --------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"insert": _insert, "gather": _gather, "shared": _shared, "chunk": _chunk, "sparse": _sparse}[state["op"]](state)


def _own(s):
    import block_sparse_attention_08_gb300 as msa
    cache = (s["k_cache"], s["v_cache"]) + ((s["k_scales"], s["v_scales"]) if s["kind"] == "int8" else ())
    if s["op"] == "insert":
        msa.msa_quantize_insert(s["k"], s["v"], s["slots"], *cache)
    if s["op"] in ("insert", "gather"):
        k, v = msa.msa_dequantize_gather(*cache, s["table"], s["cu"], s["tokens"], starts=s["old"])
        return {"k": k, "v": v}
    if s["op"] == "sparse":
        return {"out": msa.msa_sparse_attend_decode_int8kv(s["q"], *cache, s["q2k"], s["lens"], s["table"])}
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if s["lse"] else None
    if s["op"] == "chunk":
        out = msa.msa_attend_chunk_int8kv(s["q"], *cache, s["lens"], s["table"], s["cu"], lse=lse)
    else:
        call = {"bf16": msa.msa_attend_shared, "e4m3": msa.msa_attend_shared_fp8kv, "int8": msa.msa_attend_shared_int8kv}
        out = call[s["kind"]](s["q"], *cache, s["lens"], s["table"], s["cu"], s["groups"], s["shared"], lse=lse, **s["scale8"])
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def _values(s, slots):
    """K and V [..., kv heads, 128] in 32 bits at those slots."""
    k, v = s["k_cache"][slots].float(), s["v_cache"][slots].float()
    if s["kind"] == "int8":
        page, at = slots // PAGE, slots % PAGE
        return k * s["k_scales"][page, :, at].float()[..., None], v * s["v_scales"][page, :, at].float()[..., None]
    return k * s["scale8"].get("k_scale", 1.0), v * s["scale8"].get("v_scale", 1.0)


def _quantised(x):
    """int8 values and scales of rows of 128."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    # the power of two at or below the largest (its exponent bits), 64 steps to it
    scale = (top.view(torch.int32) & 0x7F800000).view(torch.float32).clamp(min=2.0 ** -127) / 64
    return torch.round(x / scale).clamp(-127, 127).to(torch.int8), scale[..., 0].bfloat16()


def _insert(s):
    page, at = s["slots"] // PAGE, s["slots"] % PAGE
    s["k_cache"][s["slots"]], s["k_scales"][page, :, at] = _quantised(s["k"])
    s["v_cache"][s["slots"]], s["v_scales"][page, :, at] = _quantised(s["v"])
    return _gather(s)


def _gather(s):
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    position = s["old"][r] + t - s["cu"][r]
    k, v = _values(s, s["table"][r, position // PAGE].long() * PAGE + position % PAGE)
    return {"k": k.bfloat16(), "v": v.bfloat16()}


def _part(q, k, v, hidden):
    """Softmax parts of q [n, kv heads, rows, 128] over k and v [n, kv heads, keys, 128]: maximum, sum, sum of values."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(LOG2E / math.sqrt(DIM)).masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp2_()
    return top, x.sum(-1, keepdim=True), torch.matmul(x, v)


def _heads(q, rows, n):
    """Rows [a, n] of q as [a, kv heads, n x 16, 128] in 32 bits."""
    return q[rows.clamp(max=q.shape[0] - 1)].float().view(-1, n, KV_HEADS, GROUP, DIM).transpose(1, 2).flatten(2, 3)


def _own_part(s, skip, keys, n):
    """The parts of each request's new tokens over its keys from position skip [requests] on."""
    cu, news = s["cu"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(n, device="cuda")
    position = skip[:, None] + torch.arange(keys, device="cuda")
    page = s["table"].gather(1, (position // PAGE).clamp(max=s["table"].shape[1] - 1)).long()
    k, v = _values(s, page * PAGE + position % PAGE)
    last = (s["lens"].long() - news)[:, None] + i
    hidden = position[:, None] > last[:, :, None]  # [requests, new, keys]
    hidden = hidden[:, None, :, None].expand(-1, 1, -1, GROUP, -1).flatten(2, 3)
    return _part(_heads(s["q"], cu[:-1, None] + i, n), k.transpose(1, 2), v.transpose(1, 2), hidden)


def _rows(x, a, i, n):
    """x [a, kv heads, n x 16, d] at tokens (a, i) as [tokens, 64, d]."""
    return x.view(x.shape[0], KV_HEADS, n, GROUP, -1)[a, :, i].flatten(1, 2)


def _result(s, top, total, o):
    out = {"out": (o / total).bfloat16()}
    return dict(out, lse=(top + torch.log2(total))[..., 0]) if s["lse"] else out


def _token_request(s):
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    return t, r, t - s["cu"][r]


def _chunk(s):
    n = s["max_new"]
    parts = _own_part(s, torch.zeros_like(s["lens"]).long(), s["table"].shape[1] * PAGE, n)
    _, r, i = _token_request(s)
    return _result(s, *(_rows(x, r, i, n) for x in parts))


def _shared(s):
    n, m = s["max_new"], s["max_group"]
    t, r, i = _token_request(s)
    first = s["groups"][:-1].long()
    length = s["shared"].long() // PAGE * PAGE
    start = s["cu"][first].long()
    # the common keys, once for each group
    position = torch.arange(s["max_shared"], device="cuda")
    k, v = _values(s, s["table"][first][:, position // PAGE].long() * PAGE + position % PAGE)
    hidden = (position >= length[:, None])[:, None, None]
    common = _part(_heads(s["q"], start[:, None] + torch.arange(m, device="cuda"), m), k.transpose(1, 2),
                   v.transpose(1, 2), hidden)
    # each request's own
    group = s["group"]
    mine = _own_part(s, torch.where(group < 0, 0, length[group.clamp(min=0)]), s["max_own"], n)
    g = group[r]
    in_group = (g >= 0)[:, None, None]
    at = torch.where(g < 0, 0, t - start[g.clamp(min=0)])
    top0, sum0, o0 = (_rows(x, g.clamp(min=0), at, m) for x in common)
    top1, sum1, o1 = (_rows(x, r, i, n) for x in mine)
    top = torch.where(in_group, torch.maximum(top0, top1), top1)
    f0, f1 = torch.where(in_group, torch.exp2(top0 - top), 0.0), torch.exp2(top1 - top)
    return _result(s, top, sum0 * f0 + sum1 * f1, o0 * f0 + o1 * f1)


def _sparse(s):
    b = s["q"].shape[0]
    blocks = s["q2k"].permute(1, 0, 2).long()  # [requests, kv heads, 16]
    page = s["table"].long().unsqueeze(1).expand(-1, KV_HEADS, -1).gather(2, blocks.clamp(min=0))
    at = torch.arange(PAGE, device="cuda")
    slots, head = page[..., None] * PAGE + at, torch.arange(KV_HEADS, device="cuda")[:, None, None]
    page, head = page[..., None].expand_as(slots), head.expand(KV_HEADS, TOPK, PAGE)
    k = s["k_cache"][slots, head].float() * s["k_scales"][page, head, at].float()[..., None]
    v = s["v_cache"][slots, head].float() * s["v_scales"][page, head, at].float()[..., None]
    hidden = (blocks[..., None] < 0) | (blocks[..., None] * PAGE + at >= s["lens"].long()[:, None, None, None])
    top, total, o = _part(s["q"].view(b, KV_HEADS, GROUP, DIM).float(), k.flatten(2, 3), v.flatten(2, 3),
                          hidden.flatten(2, 3)[:, :, None])
    return {"out": (o / total).reshape(b, HEADS, DIM).bfloat16()}


# ---- from the definitions, in 64 bits --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    lens, cu, old = s["lens"].tolist(), s["cu"].tolist(), s["old"].tolist()

    def row(r, a, b):
        pos = torch.arange(a, b, device="cuda")
        return s["table"][r].long()[pos // PAGE] * PAGE + pos % PAGE

    def value(name, slot, g):
        x = s[name + "_cache"][slot, g].double()
        if s["kind"] == "int8":
            return x * s[name + "_scales"][slot // PAGE, g, slot % PAGE].double()[:, None]
        return x * s["scale8"].get(name + "_scale", 1.0)

    if case["op"] == "insert":
        # steps of 2^(e - 6), 2^e at or below the row's largest: the nearest multiple, the even one of two, 127 at most
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            top = x.abs().amax(-1, keepdim=True)
            step = top / torch.frexp(top)[0] / 128  # (a number over its mantissa in [0.5, 1) is a power of two, exactly)
            out[name] = torch.minimum(torch.maximum(torch.round(x / step), x.new_tensor(-127.0)), x.new_tensor(127.0)) * step
        return out
    if case["op"] == "gather":
        out = {"k": [], "v": []}
        for r in range(len(lens)):
            slot = row(r, old[r], lens[r])
            for name in out:
                out[name].append(torch.stack([value(name, slot, g) for g in range(KV_HEADS)], 1))
        return {name: torch.cat(x) for name, x in out.items()}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, length in enumerate(lens):
        new = cu[r + 1] - cu[r]
        slots = row(r, 0, length)
        for g in range(KV_HEADS):
            heads = slice(g * GROUP, (g + 1) * GROUP)
            if case["op"] == "sparse":
                keep = torch.zeros(_pages(length), dtype=torch.bool, device="cuda")
                ids = s["q2k"][g, r]
                keep[ids[ids >= 0].long()] = True
                pos = torch.arange(length, device="cuda")[keep.repeat_interleave(PAGE)[:length]]
            else:
                pos = torch.arange(length, device="cuda")
            key, val = value("k", slots[pos], g), value("v", slots[pos], g)
            for a in range(0, new, 256):
                b = min(new, a + 256)
                z = torch.einsum("thd,kd->thk", s["q"][cu[r] + a:cu[r] + b, heads].double(), key) / math.sqrt(DIM)
                ok = pos[None] <= torch.arange(length - new + a, length - new + b, device="cuda")[:, None]
                z = torch.where(ok[:, None], z, -math.inf)
                norm = torch.logsumexp(z, -1)
                out[cu[r] + a:cu[r] + b, heads] = torch.einsum("thk,kd->thd", torch.exp(z - norm[..., None]), val)
                lse[cu[r] + a:cu[r] + b, heads] = norm / math.log(2.0)
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}
