"""Cases of the attention half of a layer of the verify pass: the operators between the quantized
projections (q, k, v and o, whose sizes the benchmark's configurations give: 40 query heads and
8 key/value heads of 128 on a width of 5120).

  norm_rope  the norm of every query and key head, the position rotation, and the write of keys and
             values to their cache slots, from the projections' results
  attn       attention of the rows of several streams over a prefix that all of them share and over
             each stream's own keys, both in pages of one cache
  lora       low-rank adapters of the rows' requests added to the result of a shared projection

``own`` False: plain torch operations in 32 bits.  ``own`` True: the library's calls.
"""
import math

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
TYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
SIZE = {BF16: 2, F16: 2, F32: 4}
EPS = 1e-6


# ------------------------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one row of one stream: the step between the projections and the cache where only latency counts
        dict(name="norm_rope 1 row", op="norm_rope", T=1, Hq=40, Hk=8, D=128, rot=128, interleaved=False,
             src=F32, dst=BF16, max_pos=32768),
        # a verify pass's 32 rows, from the projections' fp32 results
        dict(name="norm_rope verify 32 rows", op="norm_rope", T=32, Hq=40, Hk=8, D=128, rot=128, interleaved=False,
             src=F32, dst=BF16, max_pos=32768),
        # a prompt's rows at once, the largest call of the step
        dict(name="norm_rope 16384 rows", op="norm_rope", T=16384, Hq=40, Hk=8, D=128, rot=128, interleaved=False,
             src=F32, dst=BF16, max_pos=32768),
        # other head sizes and types: a partial rotation of neighbouring pairs, an odd row count
        dict(name="norm_rope 2311 rows partial", op="norm_rope", T=2311, Hq=24, Hk=3, D=64, rot=32, interleaved=True,
             src=BF16, dst=F16, max_pos=8192),
        # one stream decoding one token over its own short context: the smallest attention call
        dict(name="attn 1 stream", op="attn", B=1, rows_lo=1, rows_hi=1, prefix=0, len_lo=700, len_hi=700,
             Hq=40, Hk=8, D=128, page=16, dtype=BF16, lse=False),
        # sixteen streams decoding behind one long system prompt
        dict(name="attn 16 streams decode", op="attn", B=16, rows_lo=1, rows_hi=1, prefix=8192, len_lo=37, len_hi=1100,
             Hq=40, Hk=8, D=128, page=64, dtype=BF16, lse=False),
        # a verify pass: four streams of eight drafted rows behind a long shared prefix
        dict(name="attn 4 streams verify", op="attn", B=4, rows_lo=8, rows_hi=8, prefix=32768, len_lo=90, len_hi=500,
             Hq=40, Hk=8, D=128, page=64, dtype=BF16, lse=True),
        # ragged drafts, odd lengths, small heads, fp16
        dict(name="attn 29 streams ragged", op="attn", B=29, rows_lo=0, rows_hi=6, prefix=3001, len_lo=9, len_hi=777,
             Hq=24, Hk=3, D=64, page=32, dtype=F16, lse=True),
        # questions of many streams behind one long document: bound by the tensor cores
        dict(name="attn 64 streams 16 rows", op="attn", B=64, rows_lo=16, rows_hi=16, prefix=32768, len_lo=20,
             len_hi=1500, Hq=40, Hk=8, D=128, page=128, dtype=BF16, lse=False),
        # one row of one request on the three projections that share its activations
        dict(name="lora q,k,v 1 row", op="lora", M=1, adapters=4, rank_lo=16, rank_hi=16, none=0,
             N0=5120, N1=1024, N2=1024, K=5120),
        # requests without and with adapters of different ranks, an odd output width
        dict(name="lora 13 rows mixed ranks", op="lora", M=13, adapters=6, rank_lo=4, rank_hi=48, none=3,
             N0=1001, N1=0, N2=0, K=2304),
        # 32 requests with 32 adapters beside the widest projection of a layer
        dict(name="lora gate_up 32 adapters", op="lora", M=32, adapters=32, rank_lo=64, rank_hi=64, none=0,
             N0=34816, N1=0, N2=0, K=5120),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; the round ones are the listed cases'."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n % 1024 else n - 1


def draw(rng):
    op = rng.choice(["norm_rope", "attn", "attn", "lora"])
    if op == "norm_rope":
        D = rng.choice([64, 128])
        Hk = rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 12000), Hq=Hk * rng.choice([1, 2, 4, 5]), Hk=Hk, D=D,
                    rot=rng.choice([D, D // 2, D // 4]), interleaved=rng.random() < 0.5,
                    src=rng.choice([F32, F32, BF16]), dst=rng.choice([BF16, BF16, F16]), max_pos=32768)
    if op == "attn":
        while True:
            lo, hi = sorted((_log(rng, 16, 8000), _log(rng, 16, 8000)))
            rows = _log(rng, 1, 16)
            Hk = rng.randint(1, 8)
            c = dict(op=op, B=_log(rng, 1, 64), rows_lo=rng.randint(1, rows), rows_hi=rows,
                     prefix=rng.choice([0, _log(rng, 16, 40000), _log(rng, 16, 40000), _log(rng, 16, 40000)]),
                     len_lo=lo, len_hi=hi, Hq=Hk * rng.choice([1, 2, 3, 5, 7, 8]), Hk=Hk, D=rng.choice([64, 128, 128]),
                     page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice([BF16, BF16, F16]),
                     lse=rng.random() < 0.5)
            if c["Hq"] != 24 and work(c)["flops"] <= 4e11 and work(c)["bytes"] <= 1.5e9:
                return c
    M = _log(rng, 1, 32)
    lo, hi = sorted((_log(rng, 4, 128), _log(rng, 4, 128)))
    widths = [_log(rng, 256, 34816), rng.choice([0, 0, _log(rng, 256, 8192)])]
    return dict(op="lora", M=M, adapters=rng.randint(1, 32), rank_lo=lo, rank_hi=hi, none=rng.randint(0, M // 4),
                N0=widths[0], N1=widths[1], N2=0, K=rng.choice([512, 1280, 2304, 4352, 5120, 8960, 13056, 17408]))


def _spread(lo, hi, n, step):
    """n whole numbers of [lo, hi], the same ones for a case whatever the seed."""
    return [lo + int((hi - lo) * ((k * step) % 1.0) + 0.5) for k in range(n)]


def _shape(case):
    """Rows and own keys of each stream; a stream's own keys include its rows."""
    rows = _spread(case["rows_lo"], case["rows_hi"], case["B"], 0.7548776662)
    lens = _spread(case["len_lo"], case["len_hi"], case["B"], 0.6180339887)
    return rows, [max(m, n) for m, n in zip(rows, lens)]


def _lora_shape(case):
    """Rank of each adapter, adapter of each row (-1: none), and the widths of the projections."""
    ranks = _spread(case["rank_lo"], case["rank_hi"], case["adapters"], 0.6180339887)
    ids = [(5 * i + 1) % case["adapters"] for i in range(case["M"])]
    for i in range(case["none"]):
        ids[(3 * i + 1) % case["M"]] = -1
    return ranks, ids, [n for n in (case["N0"], case["N1"], case["N2"]) if n]


def work(case):
    if case["op"] == "norm_rope":
        T, Hq, Hk, D, rot = (case[k] for k in ("T", "Hq", "Hk", "D", "rot"))
        values = T * (Hq + 2 * Hk) * D
        return {"bytes": values * (SIZE[case["src"]] + SIZE[case["dst"]]) + T * rot * 4 + T * 12 + 8 * D,
                "flops": T * (Hq + Hk) * (4 * D + 3 * rot)}
    if case["op"] == "attn":
        Hq, Hk, D, P = case["Hq"], case["Hk"], case["D"], case["prefix"]
        rows, lens = _shape(case)
        keys = P + sum(n for m, n in zip(rows, lens) if m)
        seen = sum(m * P + m * (n - m) + m * (m + 1) // 2 for m, n in zip(rows, lens))
        return {"bytes": 4 * keys * Hk * D + 4 * sum(rows) * Hq * D + (4 * sum(rows) * Hq if case["lse"] else 0),
                "flops": 4 * D * Hq * seen}
    ranks, ids, widths = _lora_shape(case)
    M, K = case["M"], case["K"]
    used = sum(ranks[a] for a in set(ids) if a >= 0)
    per_row = sum(ranks[a] for a in ids if a >= 0)
    return {"bytes": sum(2 * used * (K + n) + 8 * M * n for n in widths) + 2 * M * K,
            "flops": sum(2 * per_row * (K + n) + M * n for n in widths)}


# ------------------------------------------------------------------------------------------
# Inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return {"norm_rope": _prepare_norm_rope, "attn": _prepare_attn, "lora": _prepare_lora}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, dtype=dtype, device="cuda")


def _cos_sin(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _prepare_norm_rope(case, g):
    T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
    src, dst = TYPES[case["src"]], TYPES[case["dst"]]
    n_slots = -(-(T + T // 8 + 64) // 64) * 64
    s = {"case": case,
         "Q": _randn(g, T, Hq, D).mul_(1.7).to(src), "K": _randn(g, T, Hk, D).mul_(0.6).to(src),
         "V": _randn(g, T, Hk, D).to(src),
         "q_weight": 1 + 0.2 * _randn(g, D), "k_weight": 1 + 0.2 * _randn(g, D),
         "cos_sin": _cos_sin(case["max_pos"], case["rot"]),
         "positions": torch.randint(0, case["max_pos"], (1,), generator=g, device="cuda").add(
             torch.arange(T, device="cuda")).remainder(case["max_pos"]).to(torch.int32),
         "slots": torch.randperm(n_slots // 16, generator=g, device="cuda")[:, None].mul(16).add(
             torch.arange(16, device="cuda")).reshape(-1)[:T].contiguous(),
         "Q_out": torch.empty(T, Hq, D, dtype=dst, device="cuda"),
         "K_cache": torch.zeros(n_slots, Hk, D, dtype=dst, device="cuda"),
         "V_cache": torch.zeros(n_slots, Hk, D, dtype=dst, device="cuda")}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        s["args"] = qmm.make_norm_rope(s["Q"], s["K"], s["V"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                       s["positions"], s["slots"], s["Q_out"], s["K_cache"], s["V_cache"],
                                       eps=EPS, interleaved=case["interleaved"])
    return s


def _prepare_attn(case, g):
    B, P, Hq, Hk, D, page = (case[k] for k in ("B", "prefix", "Hq", "Hk", "D", "page"))
    dtype = TYPES[case["dtype"]]
    rows, lens = _shape(case)
    per_stream = -(-max(lens) // page)
    n_prefix = -(-P // page)
    n_pages = n_prefix + sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, per_stream, dtype=torch.int32, device="cuda")
    at = n_prefix
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        at += k
    starts = [0]
    for m in rows:
        starts.append(starts[-1] + m)
    T = starts[-1]
    s = {"case": case, "T": T, "rows_max": max(rows), "len_max": max(lens),
         "Q": _randn(g, T, Hq, D).mul_(1.5).to(dtype),
         "K_cache": _randn(g, n_pages * page, Hk, D, dtype=dtype),
         "V_cache": _randn(g, n_pages * page, Hk, D, dtype=dtype),
         "prefix_pages": order[:n_prefix].contiguous(), "pages": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "row_starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "scale": D ** -0.5,
         "O": torch.empty(T, Hq, D, dtype=dtype, device="cuda"),
         "lse": torch.empty(T, Hq, device="cuda") if case["lse"] else None}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        s["args"] = qmm.make_attn(s["Q"], s["K_cache"], s["V_cache"], page, s["prefix_pages"], P, s["pages"],
                                  s["lens"], s["row_starts"], s["O"], scale=s["scale"], lse=s["lse"])
        s["workspace"] = torch.empty(qmm.attn_workspace_bytes(s["args"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_lora(case, g):
    M, K, n = case["M"], case["K"], case["adapters"]
    ranks, ids, widths = _lora_shape(case)
    r = max(ranks)
    bf16 = torch.bfloat16
    s = {"case": case, "X": _randn(g, M, K, dtype=bf16), "ids": torch.tensor(ids, dtype=torch.int32, device="cuda"),
         "ranks": torch.tensor(ranks, device="cuda"),
         "scales": 0.5 + torch.rand(n, generator=g, device="cuda"),
         "A": [_randn(g, n, r, K, dtype=bf16).mul_(K ** -0.5) for _ in widths],
         "Bt": [_randn(g, n, r, w, dtype=bf16).mul_(0.3) for w in widths],
         "Y0": [_randn(g, M, w) for w in widths],
         "Y": [torch.empty(M, w, device="cuda") for w in widths]}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        scales = s["scales"].tolist()
        s["tables"] = [qmm.make_lora_adapters([(A[a, :ranks[a]], Bt[a, :ranks[a]], scales[a]) for a in range(n)])
                       for A, Bt in zip(s["A"], s["Bt"])]
        s["entries"] = qmm.make_lora_entries([(t, s["X"], Y0, Y, w, K)
                                              for t, Y0, Y, w in zip(s["tables"], s["Y0"], s["Y"], widths)])
        s["workspace"] = torch.empty(qmm.lora_workspace_bytes(s["entries"], M, r), dtype=torch.uint8, device="cuda")
        s["rank_max"] = r
    return s


# ------------------------------------------------------------------------------------------
# One pass


def run(s):
    return {"norm_rope": _run_norm_rope, "attn": _run_attn, "lora": _run_lora}[s["case"]["op"]](s)


def _run_norm_rope(s):
    if own:
        from bit_quantized_skinny_gb300 import qmm
        qmm.norm_rope(s["args"])
    else:
        cs = s["cos_sin"][s["positions"].long()]
        s["Q_out"].copy_(_plain_head(s["Q"], s["q_weight"], cs, s["case"]))
        s["K_cache"][s["slots"]] = _plain_head(s["K"], s["k_weight"], cs, s["case"]).to(s["K_cache"].dtype)
        s["V_cache"][s["slots"]] = s["V"].to(s["V_cache"].dtype)
    return s["Q_out"], s["K_cache"], s["V_cache"]


def _plain_head(x, weight, cos_sin, case):
    """Norm and rotation of every head of x[T, H, D], in 32 bits."""
    rot = case["rot"]
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    c, s = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1)


def _run_attn(s):
    if own:
        from bit_quantized_skinny_gb300 import qmm
        qmm.attn_shared(s["args"], s["workspace"])
    else:
        o, lse = _plain_attn(s)
        s["O"].copy_(o)
        if s["lse"] is not None:
            s["lse"].copy_(lse)
    return (s["O"], s["lse"]) if s["lse"] is not None else s["O"]


def _plain_attn(s):
    """Scores of the prefix for all rows at once, of the own keys by stream (padded), one softmax over both."""
    case, T = s["case"], s["T"]
    B, P, Hq, Hk, D, page = (case[k] for k in ("B", "prefix", "Hq", "Hk", "D", "page"))
    G, dev = Hq // Hk, s["Q"].device
    q = s["Q"].float().reshape(T, Hk, G, D).transpose(0, 1) * s["scale"]               # Hk, T, G, D
    key = torch.arange(s["len_max"], device=dev)
    slots = s["pages"].long()[:, key // page] * page + key % page                       # B, L
    row = torch.arange(s["rows_max"], device=dev)
    starts, lens = s["row_starts"].long(), s["lens"].long()
    n_rows = starts[1:] - starts[:-1]
    rows = (starts[:-1, None] + row).clamp(max=T - 1)                                   # B, m
    valid = row < n_rows[:, None]
    seen = (key <= (lens - n_rows)[:, None, None] + row[:, None]) & valid[:, :, None]  # B, m, L
    held = (key < lens[:, None])[:, :, None, None]
    k_own = torch.where(held, s["K_cache"][slots].float(), 0.0).permute(0, 2, 3, 1)     # B, Hk, D, L
    v_own = torch.where(held, s["V_cache"][slots].float(), 0.0).transpose(1, 2)         # B, Hk, L, D
    q_own = q.transpose(0, 1)[rows].transpose(1, 2)                                     # B, Hk, m, G, D
    m_rows = s["rows_max"]
    s_own = (q_own.reshape(B, Hk, m_rows * G, D) @ k_own).reshape(B, Hk, m_rows, G, -1)
    s_own = s_own.masked_fill(~seen[:, None, :, None, :], -math.inf)
    b_of = torch.searchsorted(starts[1:], torch.arange(T, device=dev), right=True)
    i_of = torch.arange(T, device=dev) - starts[b_of]
    top = s_own.amax(-1).permute(0, 2, 1, 3)[b_of, i_of].transpose(0, 1)                # Hk, T, G
    if P:
        at = torch.arange(P, device=dev)
        slots = s["prefix_pages"].long()[at // page] * page + at % page
        s_pre = (q.reshape(Hk, T * G, D) @ s["K_cache"][slots].float().permute(1, 2, 0)).reshape(Hk, T, G, P)
        top = torch.maximum(top, s_pre.amax(-1))
    top = torch.where(torch.isinf(top), 0.0, top)
    top_own = top.transpose(0, 1)[rows].transpose(1, 2)                                 # B, Hk, m, G
    p_own = (s_own - top_own[..., None]).exp()
    o_own = (p_own.reshape(B, Hk, m_rows * G, -1) @ v_own).reshape(B, Hk, m_rows, G, D)
    total = p_own.sum(-1).transpose(1, 2)[b_of, i_of].transpose(0, 1)
    o = o_own.transpose(1, 2)[b_of, i_of].transpose(0, 1)                               # Hk, T, G, D
    if P:
        p_pre = (s_pre - top[..., None]).exp()
        total = total + p_pre.sum(-1)
        o = o + (p_pre.reshape(Hk, T * G, P) @ s["V_cache"][slots].float().transpose(0, 1)).reshape(Hk, T, G, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return (o.transpose(0, 1).reshape(T, Hq, D), (top + total.log()).transpose(0, 1).reshape(T, Hq))


def _run_lora(s):
    if own:
        from bit_quantized_skinny_gb300 import qmm
        qmm.run_lora(s["entries"], s["ids"], s["case"]["M"], s["rank_max"], s["workspace"])
        return s["Y"]
    ids = s["ids"].long().clamp(min=0)
    scale = torch.where(s["ids"] >= 0, s["scales"][ids], 0.0)
    rank = torch.arange(s["A"][0].shape[1], device=ids.device)
    keep = (rank < s["ranks"][ids][:, None]) & (s["ids"] >= 0)[:, None]
    x = s["X"].float()[:, :, None]
    return [_plain_adapter(x, A[ids], Bt[ids], keep, scale, Y0) for A, Bt, Y0 in zip(s["A"], s["Bt"], s["Y0"])]


def _plain_adapter(x, A, Bt, keep, scale, Y0):
    t = torch.where(keep, (A.float() @ x)[:, :, 0], 0.0) * scale[:, None]
    return Y0 + (t[:, None, :] @ Bt.float())[:, 0]


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm_rope": _exact_norm_rope, "attn": _exact_attn, "lora": _exact_lora}[case["op"]](s)


def _exact_norm_rope(s):
    case, out = s["case"], []
    rot = case["rot"]
    half = torch.arange(rot // 2, device="cuda")
    first, second = (2 * half, 2 * half + 1) if case["interleaved"] else (half, half + rot // 2)
    cs = s["cos_sin"].double()[s["positions"].long()].unsqueeze(1)
    for x, w in ((s["Q"], s["q_weight"]), (s["K"], s["k_weight"])):
        x = x.double()
        y = w.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS)
        z = y.clone()
        z[..., first] = y[..., first] * cs[..., :rot // 2] - y[..., second] * cs[..., rot // 2:]
        z[..., second] = y[..., first] * cs[..., rot // 2:] + y[..., second] * cs[..., :rot // 2]
        out.append(z)
    K = torch.zeros(s["K_cache"].shape, dtype=torch.float64, device="cuda")
    V = torch.zeros_like(K)
    K[s["slots"]], V[s["slots"]] = out[1], s["V"].double()
    return out[0], K, V


def _exact_attn(s):
    case = s["case"]
    P, Hq, Hk, D, page = (case[k] for k in ("prefix", "Hq", "Hk", "D", "page"))
    starts, lens = s["row_starts"].tolist(), s["lens"].tolist()
    O = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")

    def rows_of(cache, pages, n):
        flat = (pages.long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        return cache[flat].double()

    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        if r0 == r1:
            continue
        keys = torch.cat([rows_of(s["K_cache"], s["prefix_pages"], P), rows_of(s["K_cache"], s["pages"][b], n)])
        vals = torch.cat([rows_of(s["V_cache"], s["prefix_pages"], P), rows_of(s["V_cache"], s["pages"][b], n)])
        limit = P + n - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
        hidden = torch.arange(P + n, device="cuda")[None, :] > limit[:, None]
        for h in range(Hk):
            q = s["Q"][r0:r1, h * (Hq // Hk):(h + 1) * (Hq // Hk)].double()
            z = torch.einsum("rgd,kd->rgk", q, keys[:, h]) * s["scale"]
            z = z.masked_fill(hidden[:, None, :], -math.inf)
            here = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            lse[r0:r1, here] = torch.logsumexp(z, -1)
            O[r0:r1, here] = torch.einsum("rgk,kd->rgd", torch.softmax(z, -1), vals[:, h])
    return (O, lse) if s["lse"] is not None else O


def _exact_lora(s):
    ids, ranks = s["ids"].tolist(), s["ranks"].tolist()
    out = []
    for A, Bt, Y0 in zip(s["A"], s["Bt"], s["Y0"]):
        y = Y0.double().clone()
        for i, a in enumerate(ids):
            if a >= 0:
                t = A[a, :ranks[a]].double() @ s["X"][i].double()
                y[i] += s["scales"][a].double() * (t @ Bt[a, :ranks[a]].double())
        out.append(y)
    return out
