"""Plain 64-bit implementations and inputs for the chunked-serving tests."""
import math

import torch

H, G, D, PAGE = 64, 4, 128, 128


def pages(n):
    return -(-n // PAGE)


def page_table(lens, *, width=None, spare=1, seed=0, device="cuda"):
    """(table int32 [batch, width], pages in the pool): each request's pages are a random part of
    the pool; entries behind them are 0."""
    need = [pages(n) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
    table = torch.zeros(len(lens), width or max(max(need), 1), dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table.to(device), total


def offsets(news, device="cuda"):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def attend(q, k_cache, v_cache, lens, table, cu, scale, k_scale=1.0, v_scale=1.0, skip=()):
    """(out, lse, spread, reach) in float64: spread = sum_j w_j |v_j| (what a relative error of the
    weights can move an output by), reach = max_j scale * sum_d |q_d k_d| (what the products' order
    can move a score by).  ``skip``: (request, block) pairs whose keys are left out."""
    T, dev = q.shape[0], q.device
    out = torch.zeros(T, H, D, dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    reach = torch.zeros(T, H, dtype=torch.float64, device=dev)
    for r, n in enumerate(lens):
        a, b = int(cu[r]), int(cu[r + 1])
        if a == b:
            continue
        pos = torch.arange(n, device=dev)
        keep = torch.ones(n, dtype=torch.bool, device=dev)
        for rr, block in skip:
            if rr == r:
                keep[block * PAGE:(block + 1) * PAGE] = False
        slot = table[r].long()[pos // PAGE].clamp(0, k_cache.shape[0] // PAGE - 1) * PAGE + pos % PAGE
        ok = (pos[None] <= (n - (b - a) + torch.arange(b - a, device=dev))[:, None]) & keep
        for g in range(G):
            k = k_cache[slot, g].double() * k_scale
            v = v_cache[slot, g].double() * v_scale
            k, v = torch.where(keep[:, None], k, 0.0), torch.where(keep[:, None], v, 0.0)
            hs = slice(16 * g, 16 * g + 16)
            qq = q[a:b, hs].double()
            z = torch.einsum("thd,kd->thk", qq, k) * scale
            z = torch.where(ok[:, None], z, -math.inf)
            norm = torch.logsumexp(z, -1)
            w = torch.where(ok[:, None], torch.exp(z - norm.nan_to_num(0.0, 0.0, 0.0)[..., None]), 0.0)
            out[a:b, hs] = torch.einsum("thk,kd->thd", w, v)
            spread[a:b, hs] = torch.einsum("thk,kd->thd", w, v.abs())
            lse[a:b, hs] = norm / math.log(2.0)
            x = torch.einsum("thd,kd->thk", qq.abs(), k.abs()) * scale
            reach[a:b, hs] = torch.where(ok[:, None], x, 0.0).amax(-1)
    return out, lse, spread, reach


def check_attend(out, lse, ref, keys, weight_bits, vmax=8.0):
    """Compares with attend()'s result.  A score's fp32 dot product of 128 exact products is off by at
    most 128 * 2^-24 of reach (twice: the key's and the maximum's), and 2^-22 for the exponential;
    a weight is then rounded by at most 2^-weight_bits, or 2^-25 absolute where fp16 (11 bits) is
    subnormal; the output once by 2^-8.  lse: the score's error in base 2, the running fp32 sum over the
    blocks, two roundings of the result."""
    r_out, r_lse, spread, reach = ref
    score = 2 * 128 * 2.0 ** -24 * reach
    rel = score + 2.0 ** -22 + 2.0 ** -weight_bits
    tol = 2.0 ** -8 * r_out.abs() + 1.01 * rel[..., None] * spread + keys * 2.0 ** -32 * vmax + 2.0 ** -130
    err = (out.double() - r_out).abs()
    assert torch.isfinite(out.float()).all()
    worst = (err / tol).max()
    assert worst <= 1, f"out is {float(worst):.3g} times its tolerance off"
    if lse is not None:
        fin = torch.isfinite(r_lse)
        assert torch.equal(fin, torch.isfinite(lse)) and bool((lse[~fin] == -math.inf).all())
        tol = (score + (keys / 128 + 32) * 2.0 ** -24 + 2.0 ** -22) * 1.4427 + r_lse.abs() * 2.0 ** -22
        worst = ((lse.double() - r_lse).abs() / tol)[fin]
        assert worst.numel() == 0 or worst.max() <= 1, f"lse is {float(worst.max()):.3g} times its tolerance off"


def rotate(x, positions, inv_freq, axes, interleaved, sign=1):
    """The rotation in float64."""
    x = x.detach().double()
    y = x.clone()
    pairs = len(axes)
    for j, axis in enumerate(axes):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        phase = sign * positions[axis].double() * float(inv_freq[j])
        c, s = torch.cos(phase)[:, None], torch.sin(phase)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def map_slots(lens, news, table, free, num_free, num_slots, capacity):
    """Request by request: (cu, slots, positions, table, num_free, errors)."""
    table = [list(row) for row in table]
    stack = list(free[:num_free]) if 0 <= num_free <= len(free) else []
    cu, slots, positions, errors, full = [0], [], [], set(), False
    for r, (n, m) in enumerate(zip(lens, news)):
        good = 0 <= m <= n and pages(n) <= len(table[r])
        if not good:
            errors.add((3, r))
            m = 0
        opened = pages(n) - pages(n - m) if good else 0
        if not full and (opened > len(stack) or cu[-1] + m > capacity):
            full = True
            errors.add((6, r))
        if full:
            m = opened = 0
        for page in range(pages(n) - opened, pages(n) if opened else 0):
            i = stack.pop()
            table[r][page] = i if 0 <= i < num_slots // PAGE else -1
        for p in range(n - m, n if m else 0):
            page = table[r][p // PAGE]
            ok = 0 <= page < num_slots // PAGE
            if not ok:
                errors.add((1, len(slots)))
            slots.append(page * PAGE + p % PAGE if ok else -1)
            positions.append(p)
        cu.append(cu[-1] + m)
    spare = capacity - len(slots)
    return cu, slots + [-1] * spare, positions + [0] * spare, table, len(stack), errors
