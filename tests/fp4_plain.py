"""Plain 64-bit forms of the 4-bit cache and of sampling, from their definitions, for the GPU tests.  They run on
the tensors' device and share no code with the library."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]   # 0 .. 448


def f32(t):
    """One rounding to binary32, held in 64 bits."""
    return t.float().double()


def nearest(x, grid):
    """Index into the rising `grid` of the value nearest to each x >= 0; a tie goes to the even index, x above the
    largest value to the last."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - g[lo], g[hi] - x
    return torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantise(y, scale):
    """(codes, scale bytes) of the blocks of 16 along the last axis of y (binary32 values held in 64 bits)."""
    scale = torch.tensor(scale, dtype=torch.float32).double().item()
    b = y.unflatten(-1, (-1, 16))
    odd = ~b.isfinite().all(-1)
    b = torch.where(odd[..., None], torch.zeros_like(b), b)
    s = nearest(f32(f32(b.abs().amax(-1) / 6) / scale), E4M3)
    S = f32(torch.tensor(E4M3, dtype=torch.float64, device=y.device)[s] * scale)[..., None]
    code = nearest(f32(b.abs() / torch.where(S > 0, S, torch.ones_like(S))), E2M1) * (S > 0)
    code = code + 8 * ((b < 0) & (code > 0))
    return code.flatten(-2), torch.where(odd, 127, s)


def pack(code, s, page):
    """The bytes of a cache from codes[slots, Hk, D] and scale bytes[slots, Hk, D / 16]."""
    n, Hk, D = code.shape
    out = torch.empty(n // page, Hk, page * (D // 2 + D // 16), dtype=torch.uint8, device=code.device)
    at = lambda t: t.unflatten(0, (-1, page)).transpose(1, 2).flatten(2).to(torch.uint8)
    out[..., :page * D // 2] = at(code[..., 0::2] + 16 * code[..., 1::2])
    out[..., page * D // 2:] = at(s)
    return out.flatten()


def unpack(cache, Hk, D, page, scale):
    """64-bit values [slots, Hk, D] of a packed cache, without the rounding of the product with the tensor scale."""
    scale = torch.tensor(scale, dtype=torch.float32).double().item()
    pages = cache.view(-1, Hk, page * (D // 2 + D // 16))
    byte = pages[..., :page * D // 2].unflatten(-1, (page, -1)).long()
    values = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=cache.device)
    v = values[torch.stack([byte % 16, byte // 16], -1).flatten(-2)]
    table = torch.tensor(E4M3 + [math.nan] + [-v for v in E4M3] + [math.nan], dtype=torch.float64, device=cache.device)
    s = table[pages[..., page * D // 2:].unflatten(-1, (page, -1)).long()]
    return (v * s.repeat_interleave(16, -1) * scale).transpose(1, 2).flatten(0, 1)


def sample(x, temperature, top_k, top_p, min_p, u):
    """(token, logprob, margin) of one row of logits (64 bits); margin: how near, relative to the sum of weights, the
    row comes to another token."""
    x = torch.where(x.isnan(), -math.inf, x)
    order = torch.argsort(x, descending=True, stable=True)
    top = x[order[0]].item()
    if top == -math.inf:
        return -1, -math.inf, 1.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    w = torch.exp((x[order] - top) / temperature)
    w[x[order] == top] = 1.0
    w[x[order] == -math.inf] = 0.0
    margin = 1.0
    stays = torch.ones_like(w, dtype=torch.bool)
    if top_k > 0:
        stays[top_k:] = False
    if top_p < 1:
        left = torch.where(stays, w, 0.0)
        before = torch.nn.functional.pad(left.cumsum(0)[:-1], (1, 0))
        limit = max(top_p, 0.0) * left.sum()
        margin = min(margin, ((before - limit).abs() / left.sum())[1:].min().item() if len(w) > 1 else 1.0)
        stays &= before < limit
    if min_p > 0:
        stays &= w >= min_p
        margin = min(margin, (w[1:] - min_p).abs().min().item() if len(w) > 1 else 1.0)
    stays[0] = True
    kept = torch.zeros_like(w)
    kept[order] = torch.where(stays, w, 0.0)
    sums = kept.cumsum(0)
    total = sums[-1]
    limit = min(max(u, 0.0), 1 - 2.0 ** -24) * total
    margin = min(margin, ((sums - limit).abs() / total)[kept > 0].min().item())
    token = int((sums <= limit).sum())
    return token, (kept[token] / total).log().item(), margin
