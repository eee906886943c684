"""The operators of chunked serving over a paged K/V cache, as measured cases.

Three operators, in the order in which a serving step calls them:

- ``slots``: page-table rows and the slot of every new token, from the requests' lengths and a stack of free pages;
- ``rotary``: rotary positions with several axes on Q and K, with K and V written into the paged cache at those slots
  (bf16 or E4M3), and the same rotation for training, forward and backward;
- ``attend``: causal attention of each request's new tokens (one, or a chunk) over all its keys in the paged cache.

``run`` gives each in its plain form (elementary torch operations in 32 bits; the angles of the rotation in 64, since a
position times a frequency loses its fraction in 32), or, where ``own`` is true, as the package's calls.
"""
import math
import random

import torch

own = False

HEADS, KV_HEADS, DIM, PAGE = 64, 4, 128, 128
LOG2E = 1.0 / math.log(2.0)


# ---- the cases ------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 64: one new token each, a page is opened for one request in 128
        {"name": "slots, a step of 64", "op": "slots", "requests": 64, "min_len": 4096, "max_len": 65536, "min_new": 1,
         "max_new": 1, "mix": 1, "spare": 0},
        # a large mixed batch in a buffer that is longer than its tokens (a captured graph's)
        {"name": "slots, 509 mixed", "op": "slots", "requests": 509, "min_len": 1, "max_len": 16384, "min_new": 0,
         "max_new": 130, "mix": 2, "spare": 1000},
        # the decode step of 64 requests: latency
        {"name": "insert 64 tokens", "op": "insert", "tokens": 64, "rot": 128, "axes": "0", "interleaved": False,
         "cache": "bf16", "far": 65536},
        # a prompt with images: three axes, half of the head rotated
        {"name": "insert 16384, three axes", "op": "insert", "tokens": 16384, "rot": 64, "axes": "0:12,1:10,2:10",
         "interleaved": False, "cache": "bf16", "far": 1000},
        # an odd chunk far into a long context, pairs side by side, FP8 cache
        {"name": "insert 8191, E4M3", "op": "insert", "tokens": 8191, "rot": 128, "axes": "0:16,1:24,2:24",
         "interleaved": True, "cache": "e4m3", "far": 1000000},
        # a training step's rotation of a 16k document, forward and backward
        {"name": "rotary training, 16384", "op": "train", "tokens": 16384, "rot": 128, "axes": "0:16,1:24,2:24",
         "interleaved": False, "far": 1000},
        # four short chats, one new token each: the smallest call
        {"name": "attend 4 x 1, short", "op": "attend", "requests": 4, "min_len": 300, "max_len": 2000, "min_new": 1,
         "max_new": 1, "mix": 3, "cache": "bf16", "lse": False},
        # a decode step of 64 requests of 4k to 64k keys
        {"name": "attend 64 x 1, 4k-64k", "op": "attend", "requests": 64, "min_len": 4096, "max_len": 65536,
         "min_new": 1, "max_new": 1, "mix": 4, "cache": "bf16", "lse": False},
        # a decode step of 16 long contexts over an FP8 cache, log-sum-exp kept for a merge
        {"name": "attend 16 x 1, 128k, E4M3", "op": "attend", "requests": 16, "min_len": 131072, "max_len": 131072,
         "min_new": 1, "max_new": 1, "mix": 5, "cache": "e4m3", "lse": True},
        # a chunk of 2048 new tokens at the end of 32k keys: the largest product
        {"name": "attend 2048 over 32k", "op": "attend", "requests": 1, "min_len": 32768, "max_len": 32768,
         "min_new": 2048, "max_new": 2048, "mix": 6, "cache": "bf16", "lse": False},
        # decodes and chunks in one batch
        {"name": "attend 17 mixed", "op": "attend", "requests": 17, "min_len": 1, "max_len": 8192, "min_new": 1,
         "max_new": 500, "mix": 7, "cache": "bf16", "lse": True},
        # chunks over an FP8 cache
        {"name": "attend 5 chunks, E4M3", "op": "attend", "requests": 5, "min_len": 3000, "max_len": 16384,
         "min_new": 333, "max_new": 700, "mix": 8, "cache": "e4m3", "lse": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["slots", "insert", "train", "attend", "attend", "attend"])
    mix = rng.randrange(1000, 1 << 20)
    if op == "slots":
        new = _log(rng, 1, 300)
        return {"op": op, "requests": _log(rng, 1, 700), "min_len": 1, "max_len": _log(rng, 300, 65536),
                "min_new": rng.choice([0, 1]), "max_new": new, "mix": mix, "spare": rng.choice([0, 1, 700])}
    if op in ("insert", "train"):
        rot = 16 * rng.randint(1, 8)
        cut = sorted(rng.randint(0, rot // 2) for _ in range(2))
        axes = rng.choice(["0", "0:%d,1:%d,2:%d" % (cut[0], cut[1] - cut[0], rot // 2 - cut[1])])
        case = {"op": op, "tokens": _log(rng, 1, 16384), "rot": rot, "axes": axes,
                "interleaved": rng.random() < 0.5, "far": _log(rng, 1000, 1000000)}
        return dict(case, cache=rng.choice(["bf16", "e4m3"])) if op == "insert" else case
    requests = _log(rng, 1, 64)
    longest = _log(rng, 130, 131072)
    new = rng.choice([1, 1, _log(rng, 2, 2048)])
    # the largest listed case bounds the plain form's scores and the keys in the cache
    while requests > 1 and (requests * new * longest > 2048 * 32768 or requests * longest > 1 << 21):
        requests = (requests + 1) // 2
    new = min(new, 2048 * 32768 // longest, longest)
    return {"op": op, "requests": requests, "min_len": max(1, longest // rng.choice([1, 2, 16, 1000])),
            "max_len": longest, "min_new": min(new, rng.choice([1, new])), "max_new": new, "mix": mix,
            "cache": rng.choice(["bf16", "e4m3"]), "lse": rng.random() < 0.5}


def _lengths(case):
    """(length with the new tokens, new tokens) of each request, from the case alone."""
    rng = random.Random(case["mix"])
    lens, news = [], []
    for r in range(case["requests"]):
        n = _log(rng, max(1, case["min_new"]), case["max_new"]) if r == 0 or rng.random() < 0.9 else case["min_new"]
        length = rng.randint(min(case["min_len"], case["max_len"]), case["max_len"])
        lens.append(max(length, n))
        news.append(n)
    return lens, news


def _pages(n):
    return -(-n // PAGE)


def work(case):
    if case["op"] == "slots":
        lens, news = _lengths(case)
        t = sum(news)
        opened = sum(_pages(n) - _pages(n - m) for n, m in zip(lens, news))
        # lengths in, offsets out; a page id in and out for each opened page; a page id in, slot and position out
        return {"bytes": 12 * len(lens) + 8 * opened + 12 * (t + case["spare"]) + 4 * len(lens), "flops": 0}
    if case["op"] == "insert":
        t, size = case["tokens"], 1 if case["cache"] == "e4m3" else 2
        return {"bytes": t * DIM * (2 * (2 * HEADS + 2 * KV_HEADS) + 2 * KV_HEADS * size),
                "flops": 3 * t * (HEADS + KV_HEADS) * case["rot"]}
    if case["op"] == "train":
        t = case["tokens"]
        return {"bytes": 2 * t * DIM * 2 * 2 * (HEADS + KV_HEADS), "flops": 2 * 3 * t * (HEADS + KV_HEADS) * case["rot"]}
    lens, news = _lengths(case)
    size = 1 if case["cache"] == "e4m3" else 2
    seen = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, news))  # (query, key) pairs
    t = sum(news)
    return {"bytes": 2 * 2 * t * HEADS * DIM + sum(n for n, m in zip(lens, news) if m) * 2 * KV_HEADS * DIM * size
            + (4 * t * HEADS if case["lse"] else 0), "flops": 4 * seen * HEADS * DIM}


# ---- what a program has in hand --------------------------------------------------------------------------------

def _axes(case):
    """The axis of each rotated pair."""
    if ":" not in case["axes"]:
        return (0,) * (case["rot"] // 2)
    return tuple(a for part in case["axes"].split(",") for a, n in [map(int, part.split(":"))] for _ in range(n))


def _tables(lens, news, spare_pages, gen):
    """A page table whose rows hold a random permutation of the pool's pages, and the pages left over."""
    need = torch.tensor([_pages(n) for n in lens])
    total = int(need.sum()) + spare_pages
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    width = max(1, int(need.max()))
    first = (torch.cumsum(need, 0) - need).cuda()[:, None]
    col = torch.arange(width, device="cuda")[None]
    table = torch.where(col < need.cuda()[:, None], perm[(first + col).clamp(max=total - 1)], 0).int()
    return table.contiguous(), perm[int(need.sum()):].contiguous(), total


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    def cache(slots):
        x = randn(slots, KV_HEADS, DIM)
        return x.to(torch.float8_e4m3fn) if case["cache"] == "e4m3" else x

    scales = {"k_scale": 0.5, "v_scale": 0.25} if case.get("cache") == "e4m3" else {}
    if case["op"] == "slots":
        lens, news = _lengths(case)
        old = [n - m for n, m in zip(lens, news)]
        opened = sum(_pages(n) - _pages(o) for n, o in zip(lens, old))
        table, free, total = _tables(old, news, opened + 64, gen)
        width = max(_pages(n) for n in lens)
        wide = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
        wide[:, :min(width, table.shape[1])] = table[:, :width]
        return {"op": "slots", "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
                "news": torch.tensor(news, dtype=torch.int32, device="cuda"), "table": wide, "free": free,
                "num_free": torch.tensor([free.shape[0]], dtype=torch.int32, device="cuda"),
                "capacity": sum(news) + case["spare"], "num_slots": total * PAGE}
    if case["op"] in ("insert", "train"):
        t, rot = case["tokens"], case["rot"]
        start = case["far"] + torch.randint(1000, (1,), generator=gen, device="cuda", dtype=torch.int32)
        i = torch.arange(t, dtype=torch.int32, device="cuda")
        if ":" in case["axes"]:  # text and pictures in turn: a picture's tokens share their time
            inside = i % 1024
            picture = inside >= 400
            positions = torch.stack([torch.where(picture, i - inside + 400, i),
                                     torch.where(picture, i - inside + 400 + (inside - 400) // 24, i),
                                     torch.where(picture, i - inside + 400 + (inside - 400) % 24, i)]) + start
        else:
            positions = (i + start)[None]
        state = {"op": case["op"], "axes": _axes(case), "interleaved": case["interleaved"],
                 "positions": positions.contiguous(),
                 "inv_freq": torch.tensor([1e6 ** (-2.0 * j / rot) for j in range(rot // 2)], device="cuda")}
        if case["op"] == "train":
            return dict(state, q=randn(t, HEADS, DIM).requires_grad_(), k=randn(t, KV_HEADS, DIM).requires_grad_(),
                        gq=randn(t, HEADS, DIM), gk=randn(t, KV_HEADS, DIM))
        qkv = randn(t, HEADS + 2 * KV_HEADS, DIM)  # the projection's output: q, k and v are its heads
        pages = _pages(t) + 3
        perm = torch.randperm(pages, generator=gen, device="cuda")
        slots = perm[(i + 37).long() // PAGE] * PAGE + (i + 37) % PAGE  # a chunk that starts inside a page
        return dict(state, q=qkv[:, :HEADS], k=qkv[:, HEADS:HEADS + KV_HEADS], v=qkv[:, HEADS + KV_HEADS:], slots=slots,
                    k_cache=cache(pages * PAGE), v_cache=cache(pages * PAGE), scales=scales)
    lens, news = _lengths(case)
    table, _, total = _tables(lens, news, 1, gen)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return {"op": "attend", "q": randn(cu[-1], HEADS, DIM), "k_cache": cache(total * PAGE),
            "v_cache": cache(total * PAGE), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "table": table, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "scales": scales,
            "max_new": max(news), "lse": case["lse"]}


# ---- one pass --------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"slots": _slots, "insert": _insert, "train": _train, "attend": _attend}[state["op"]](state)


def _own(s):
    import block_sparse_attention_08_gb300 as msa
    if s["op"] == "slots":
        cu, slots, positions, left = msa.msa_map_slots(s["lens"], s["news"], s["table"], s["free"], s["num_free"],
                                                       num_slots=s["num_slots"], capacity=s["capacity"])
        return {"cu": cu, "slots": slots, "positions": positions, "table": s["table"], "left": left}
    if s["op"] == "insert":
        q = msa.msa_rotary_insert(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"],
                                  s["v_cache"], axes=s["axes"], interleaved=s["interleaved"], **s["scales"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "train":
        q, k = msa.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], axes=s["axes"], interleaved=s["interleaved"])
        dq, dk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["gq"], s["gk"]))
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if s["lse"] else None
    call = msa.msa_attend_chunk_fp8kv if s["scales"] else msa.msa_attend_chunk
    out = call(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["table"], s["cu"], lse=lse, **s["scales"])
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def _slots(s):
    lens, news = s["lens"].long(), s["news"].long()
    old = lens - news
    have, need = (old + PAGE - 1) // PAGE, (lens + PAGE - 1) // PAGE
    before = torch.cumsum(need - have, 0) - (need - have)
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    taken = s["num_free"].long() - 1 - (before[:, None] + col - have[:, None])
    fresh = s["free"][taken.clamp(0, s["free"].shape[0] - 1)]
    s["table"].copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), fresh, s["table"]))
    cu = torch.nn.functional.pad(torch.cumsum(news, 0), (1, 0))
    t = torch.arange(s["capacity"], device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=lens.shape[0] - 1)
    position = old[r] + t - cu[r]
    page = s["table"][r, (position // PAGE).clamp(0, s["table"].shape[1] - 1)].long()
    live = t < cu[-1]
    return {"cu": cu.int(), "slots": torch.where(live, page * PAGE + position % PAGE, -1),
            "positions": torch.where(live, position, 0).int(), "table": s["table"],
            "left": (s["num_free"] - (need - have).sum()).int()}


def _cos_sin(s):
    axes = torch.tensor(s["axes"], device="cuda")
    angle = s["positions"][axes].double().T * s["inv_freq"].double()  # [tokens, pairs]
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotated(x, cos, sin, interleaved):
    """x [tokens, heads, 128] in 32 bits, rotated by the angles."""
    half = cos.shape[-1]
    x = x.float()
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :half], turned[..., half:])
    y = (a * cos - b * sin, a * sin + b * cos)
    return torch.cat([torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1), rest], -1)


def _insert(s):
    cos, sin = _cos_sin(s)
    k = _rotated(s["k"], cos, sin, s["interleaved"]) / s["scales"].get("k_scale", 1.0)
    v = s["v"].float() / s["scales"].get("v_scale", 1.0)
    if s["scales"]:
        k, v = k.clamp(-448, 448), v.clamp(-448, 448)
    s["k_cache"][s["slots"]] = k.to(s["k_cache"].dtype)
    s["v_cache"][s["slots"]] = v.to(s["v_cache"].dtype)
    return {"q": _rotated(s["q"], cos, sin, s["interleaved"]).bfloat16(), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _train(s):
    cos, sin = _cos_sin(s)
    with torch.no_grad():  # the rotation's gradient is the rotation back
        return {"q": _rotated(s["q"], cos, sin, s["interleaved"]).bfloat16(),
                "k": _rotated(s["k"], cos, sin, s["interleaved"]).bfloat16(),
                "dq": _rotated(s["gq"], cos, -sin, s["interleaved"]).bfloat16(),
                "dk": _rotated(s["gk"], cos, -sin, s["interleaved"]).bfloat16()}


def _attend(s):
    q, lens, cu, group = s["q"].float(), s["lens"].long(), s["cu"].long(), HEADS // KV_HEADS
    b, n = s["table"].shape[0], s["max_new"]
    table = s["table"].long()
    # keys and values [requests, kv heads, keys, 128], queries [requests, kv heads, new tokens x 16, 128], both padded
    k = s["k_cache"].view(-1, PAGE, KV_HEADS, DIM)[table].float().flatten(1, 2).transpose(1, 2)
    v = s["v_cache"].view(-1, PAGE, KV_HEADS, DIM)[table].float().flatten(1, 2).transpose(1, 2)
    k, v = k * s["scales"].get("k_scale", 1.0), v * s["scales"].get("v_scale", 1.0)
    i = torch.arange(n, device="cuda")[None]
    news = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    q = q[rows].view(b, n, KV_HEADS, group, DIM).transpose(1, 2).flatten(2, 3)
    x = torch.matmul(q, k.transpose(-1, -2)).view(b, KV_HEADS, n, group, -1).mul_(LOG2E / math.sqrt(DIM))
    last = (lens - news)[:, None] + i  # the position of each query
    hidden = torch.arange(x.shape[-1], device="cuda") > last[:, :, None]
    x.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp2_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).view(b, KV_HEADS, n, group, DIM) / total
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = t - cu[r]
    out = o[r, :, at].reshape(-1, HEADS, DIM).bfloat16()
    if not s["lse"]:
        return {"out": out}
    lse = (top + torch.log2(total))[..., 0]
    return {"out": out, "lse": lse[r, :, at].reshape(-1, HEADS)}


# ---- from the definitions, in 64 bits --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers: compared for equality
    s = prepare(case, seed)
    if case["op"] in ("insert", "train"):
        return _exact_rotary(s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    group = HEADS // KV_HEADS
    for r, length in enumerate(lens):
        new = cu[r + 1] - cu[r]
        pos = torch.arange(length, device="cuda")
        slot = s["table"][r].long()[pos // PAGE] * PAGE + pos % PAGE
        for g in range(KV_HEADS):
            key = s["k_cache"][slot, g].double() * s["scales"].get("k_scale", 1.0)
            value = s["v_cache"][slot, g].double() * s["scales"].get("v_scale", 1.0)
            heads = slice(g * group, (g + 1) * group)
            for a in range(0, new, 256):
                b = min(new, a + 256)
                z = torch.einsum("thd,kd->thk", s["q"][cu[r] + a:cu[r] + b, heads].double(), key) / math.sqrt(DIM)
                ok = pos[None] <= torch.arange(length - new + a, length - new + b, device="cuda")[:, None]
                z = torch.where(ok[:, None], z, -math.inf)
                norm = torch.logsumexp(z, -1)
                out[cu[r] + a:cu[r] + b, heads] = torch.einsum("thk,kd->thd", torch.exp(z - norm[..., None]), value)
                lse[cu[r] + a:cu[r] + b, heads] = norm / math.log(2.0)
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def _exact_rotary(s):
    pairs = len(s["axes"])

    def turn(x, sign):
        x = x.detach().double()
        y = x.clone()
        for j, axis in enumerate(s["axes"]):
            a, b = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + pairs)
            phase = sign * s["positions"][axis].double() * float(s["inv_freq"][j])
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(phase), phase)[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        return y

    if s["op"] == "train":
        return {"q": turn(s["q"], 1), "k": turn(s["k"], 1), "dq": turn(s["gq"], -1), "dk": turn(s["gk"], -1)}
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache[s["slots"]] = turn(s["k"], 1) / s["scales"].get("k_scale", 1.0)
    v_cache[s["slots"]] = s["v"].double() / s["scales"].get("v_scale", 1.0)
    return {"q": turn(s["q"], 1), "k_cache": k_cache, "v_cache": v_cache}
