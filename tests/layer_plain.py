"""Plain 64-bit forms of the attention half's operators, from their formulas, for the GPU tests.
They run on the tensors' device in float64 and share no code with the library."""
import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # unit roundoff of the 16-bit types


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """Normed and rotated heads of x[T, H, D], and per value the magnitude its rotation summed."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    size = y.abs()
    if cos_sin is None:
        return y, size
    rot = cos_sin.shape[1]
    cs = cos_sin.double()[positions.long()]
    z, size = y.clone(), size.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = cs[:, i, None], cs[:, rot // 2 + i, None]
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, size


def attention(Q, K_cache, V_cache, page, prefix_pages, prefix, pages, lens, starts, scale):
    """(O, lse, sum of softmax weights times |v|) of every row of Q[T, Hq, D], by its visible keys."""
    T, Hq, D = Q.shape
    G = Hq // K_cache.shape[1]
    O = torch.zeros(T, Hq, D, dtype=torch.float64, device=Q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=Q.device)
    S = torch.zeros_like(O)

    def slots(table, n):
        j = torch.arange(n, device=Q.device)
        return table.long()[j // page] * page + j % page

    for b in range(len(lens)):
        n, m = lens[b], starts[b + 1] - starts[b]
        for i in range(m):
            own = max(0, n - m + i + 1)
            at = torch.cat([slots(prefix_pages, prefix) if prefix else torch.empty(0, dtype=torch.long, device=Q.device),
                            slots(pages[b], own)])
            if not len(at):
                continue
            t = starts[b] + i
            k = K_cache[at].double().repeat_interleave(G, dim=1)
            v = V_cache[at].double().repeat_interleave(G, dim=1)
            z = torch.einsum("hd,khd->hk", Q[t].double(), k) * scale
            lse[t] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            O[t] = torch.einsum("hk,khd->hd", p, v)
            S[t] = torch.einsum("hk,khd->hd", p, v.abs())
    return O, lse, S


def lora(X, Y0, ids, adapters):
    """(Y, sum of |scale * b * a * x|) with adapters a list of (A, Bt, scale)."""
    Y, S = Y0.double().clone(), torch.zeros(Y0.shape, dtype=torch.float64, device=Y0.device)
    for i, a in enumerate(ids):
        if a < 0:
            continue
        A, Bt, scale = adapters[a]
        A, Bt, x = A.double(), Bt.double(), X[i].double()
        Y[i] += scale * ((A @ x) @ Bt)
        S[i] = abs(scale) * ((A.abs() @ x.abs()) @ Bt.abs())
    return Y, S
