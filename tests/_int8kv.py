"""Plain 64-bit implementations and inputs for the tests of the int8 K/V cache."""
import math

import torch

from _serving import D, G, H, PAGE


def quantise(x):
    """(n int64, scale float64) of rows of 128, from the definition: 2^e at or below the largest magnitude, e >= -127, steps of
    2^(e - 6), the nearest multiple (the even one of two), 127 at most.  A row that is not finite: zeros, NaN."""
    x = x.detach().double().cpu()
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(bad, 0.0, x)
    top = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 1).double()
    e = torch.where(top == 0, -127.0, e).clamp(min=-127)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), e - 6)
    n = torch.round(x / step).clamp(-127, 127)
    return torch.where(bad, 0, n).long(), torch.where(bad, math.nan, step)[..., 0]


def values(cache, scales, dtype=torch.float64):
    """[slots, 4, 128] that an int8 cache stands for."""
    s = scales.to(dtype).transpose(1, 2).reshape(-1, G)  # [slots, 4]
    return cache.to(dtype) * s[..., None]


def cache(pages, seed=0, device="cuda", powers=True):
    """A random int8 cache and its scales: powers of two, or any bf16 numbers."""
    gen = torch.Generator().manual_seed(seed)
    n = torch.randint(-127, 128, (pages * PAGE, G, D), generator=gen, dtype=torch.int32).to(torch.int8)
    s = torch.exp2(torch.randint(-7, -4, (pages, G, PAGE), generator=gen).float())
    if not powers:
        s = s * (1 + torch.rand(s.shape, generator=gen))
    return n.to(device), s.bfloat16().to(device)


def sparse(q, k, v, q2k, lens, table, scale):
    """(out, spread, reach) in float64 of the decode attention over selected blocks (as _serving.attend gives them); k and v
    are the values [slots, 4, 128]."""
    B, dev = q.shape[0], q.device
    out = torch.zeros(B, H, D, dtype=torch.float64, device=dev)
    spread, reach = torch.zeros_like(out), torch.zeros(B, H, dtype=torch.float64, device=dev)
    for r, n in enumerate(lens):
        for g in range(G):
            pos = [p for b in q2k[g, r].tolist() if 0 <= b * PAGE < n for p in range(b * PAGE, min(n, (b + 1) * PAGE))]
            if not pos:
                continue
            pos = torch.tensor(pos, device=dev)
            page = table[r].long()[pos // PAGE]
            pos, page = pos[(page >= 0) & (page < k.shape[0] // PAGE)], page[(page >= 0) & (page < k.shape[0] // PAGE)]
            if not len(pos):
                continue
            slot = page * PAGE + pos % PAGE
            kk, vv, hs = k[slot, g].double(), v[slot, g].double(), slice(16 * g, 16 * g + 16)
            qq = q[r, hs].double()
            w = torch.softmax(qq @ kk.T * scale, -1)
            out[r, hs], spread[r, hs] = w @ vv, w @ vv.abs()
            reach[r, hs] = (qq.abs() @ kk.abs().T * scale).amax(-1)
    return out, spread, reach


def check_sparse(out, ref, powers=True):
    """Compares with sparse()'s result.  A score is off by at most 2 * 128 * 2^-24 of reach (as _serving.check_attend), 2^-22 for
    the exponential and 2^-23 for the scale's products; a weight is rounded by 2^-8, in the sum as well, and with scales that are
    no powers of two once more with the value's scale; the output once by 2^-8."""
    r_out, spread, reach = ref
    rel = 2 * (128 * 2.0 ** -24 * reach + 2.0 ** -22 + 2.0 ** -23 * reach) + (2 if powers else 3) * 2.0 ** -8
    tol = 2.0 ** -8 * r_out.abs() + 1.01 * rel[..., None] * spread + 2.0 ** -130
    assert torch.isfinite(out.float()).all()
    worst = ((out.double() - r_out).abs() / tol).max()
    assert worst <= 1, f"out is {float(worst):.3g} times its tolerance off"
