"""Cases of a verify pass whose context is held in 4 bits, and of its end: the operators beside the
attention half of a layer (40 query heads and 8 key/value heads of 128) and behind the lm_head (248320
logits a row), as the benchmark's configurations have them.

  append  norm and rotation of every query and key head, keys and values rounded to 4 bits on their way
          into the pages of a cache, and the cache read back as values
  attn    attention of the rows of several streams over a prefix that all of them share and over each
          stream's own keys, from that cache
  sample  the token of every row from its logits (temperature, top-k, top-p, min-p, given random numbers),
          and how many of each stream's drafted tokens stand

A cache holds, for each page and head, the page's codes (two E2M1 codes a byte, the lower index in the low
half), then its scales (an E4M3 value for 16 codes); a value is code * scale * (the tensor's scale).

``own`` False: plain torch operations.  ``own`` True: the library's calls.
"""
import math

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
TYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
SIZE = {BF16: 2, F16: 2, F32: 4}
EPS = 1e-6
K_SCALE, V_SCALE = 0.04, 0.055   # the tensors' scales: the largest value a cache holds is 2688 of them
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one row of one stream: the step between the projections and the cache where only latency counts
        dict(name="append 1 row", op="append", T=1, Hq=40, Hk=8, D=128, rot=128, interleaved=False, src=F32, dst=BF16,
             page=64, max_pos=32768),
        # other head sizes and types: a partial rotation of neighbouring pairs, an odd row count, small pages
        dict(name="append 2311 rows partial", op="append", T=2311, Hq=24, Hk=3, D=64, rot=32, interleaved=True, src=BF16,
             dst=F16, page=16, max_pos=8192),
        # a prompt's rows at once, the largest call of the step
        dict(name="append 16384 rows", op="append", T=16384, Hq=40, Hk=8, D=128, rot=128, interleaved=False, src=F32,
             dst=BF16, page=64, max_pos=32768),
        # one stream decoding one token over its own short context: the smallest attention call
        dict(name="attn 1 stream", op="attn", B=1, rows_lo=1, rows_hi=1, prefix=0, len_lo=700, len_hi=700, Hq=40, Hk=8,
             D=128, page=16, dtype=BF16, lse=False),
        # ragged drafts, odd lengths, small heads, fp16
        dict(name="attn 29 streams ragged", op="attn", B=29, rows_lo=0, rows_hi=6, prefix=3001, len_lo=9, len_hi=777,
             Hq=24, Hk=3, D=64, page=32, dtype=F16, lse=True),
        # a verify pass: four streams of eight drafted rows behind a very long shared document
        dict(name="attn 4 streams verify", op="attn", B=4, rows_lo=8, rows_hi=8, prefix=131072, len_lo=90, len_hi=500,
             Hq=40, Hk=8, D=128, page=64, dtype=BF16, lse=True),
        # streams that decode over long contexts of their own: what a cache in 4 bits is for
        dict(name="attn 24 streams long", op="attn", B=24, rows_lo=1, rows_hi=1, prefix=0, len_lo=19000, len_hi=41000,
             Hq=40, Hk=8, D=128, page=64, dtype=BF16, lse=False),
        # questions of many streams behind one long document: bound by the tensor cores
        dict(name="attn 64 streams 16 rows", op="attn", B=64, rows_lo=16, rows_hi=16, prefix=32768, len_lo=20,
             len_hi=1500, Hq=40, Hk=8, D=128, page=128, dtype=BF16, lse=False),
        # the token of one decoding stream
        dict(name="sample 1 row", op="sample", B=1, rows=1, V=248320, src=F32, params="nucleus"),
        # the rows of a mixed batch: greedy ones, top-k, min-p, flat and sharp ones; bf16 logits with many ties
        dict(name="sample 13 rows mixed", op="sample", B=5, rows=13, V=32003, src=BF16, params="mixed"),
        # a verify pass: four streams of eight drafted rows
        dict(name="sample 4 streams verify", op="sample", B=4, rows=32, V=248320, src=F32, params="nucleus"),
        # a large batch, every filter in use
        dict(name="sample 128 streams", op="sample", B=128, rows=128, V=248320, src=F32, params="mixed"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; the round ones are the listed cases'."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n % 1024 else n - 1


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sample"])
    if op == "append":
        D = rng.choice([64, 128, 128, 256])
        Hk = rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 12000 * 128 // D), Hq=Hk * rng.choice([1, 2, 4, 5]), Hk=Hk, D=D,
                    rot=rng.choice([D, D // 2, D // 4]), interleaved=rng.random() < 0.5,
                    src=rng.choice([F32, F32, BF16, F16]), dst=rng.choice([BF16, BF16, F16]),
                    page=rng.choice([16, 32, 64, 128, 256]), max_pos=32768)
    if op == "attn":
        while True:
            lo, hi = sorted((_log(rng, 16, 30000), _log(rng, 16, 30000)))
            rows = _log(rng, 1, 16)
            Hk = rng.randint(1, 8)
            c = dict(op=op, B=_log(rng, 1, 64), rows_lo=rng.randint(1, rows), rows_hi=rows,
                     prefix=rng.choice([0, _log(rng, 16, 120000), _log(rng, 16, 120000)]), len_lo=lo, len_hi=hi,
                     Hq=Hk * rng.choice([1, 2, 3, 5, 7, 8]), Hk=Hk, D=rng.choice([64, 128, 128]),
                     page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice([BF16, BF16, F16]),
                     lse=rng.random() < 0.5)
            if c["Hq"] != 24 and work(c)["flops"] <= 4e11 and work(c)["bytes"] <= 6e8:
                return c
    B = _log(rng, 1, 32)
    return dict(op=op, B=B, rows=B * rng.randint(1, 3) + rng.randint(0, 2), V=_log(rng, 900, 248000),
                src=rng.choice([F32, F32, BF16, F16]), params=rng.choice(["plain", "nucleus", "mixed", "mixed"]))


def _spread(lo, hi, n, step):
    """n whole numbers of [lo, hi], the same ones for a case whatever the seed."""
    return [lo + int((hi - lo) * ((k * step) % 1.0) + 0.5) for k in range(n)]


def _shape(case):
    """Rows and own keys of each stream; a stream's own keys include its rows."""
    rows = _spread(case["rows_lo"], case["rows_hi"], case["B"], 0.7548776662)
    lens = _spread(case["len_lo"], case["len_hi"], case["B"], 0.6180339887)
    return rows, [max(m, n) for m, n in zip(rows, lens)]


def _slots(case):
    return -(-(case["T"] + case["T"] // 8 + 64) // case["page"]) * case["page"]


def work(case):
    if case["op"] == "append":
        T, Hq, Hk, D, rot = (case[k] for k in ("T", "Hq", "Hk", "D", "rot"))
        packed = 2 * Hk * (D // 2 + D // 16)   # of one token's key and value
        read_back = _slots(case) * (packed + 2 * Hk * D * 2)
        return {"bytes": T * (Hq + 2 * Hk) * D * SIZE[case["src"]] + T * Hq * D * SIZE[case["dst"]] + T * packed + read_back +
                T * rot * 4 + T * 12 + 8 * D,
                "flops": T * (Hq + Hk) * (4 * D + 3 * rot) + 4 * T * Hk * D}
    if case["op"] == "attn":
        Hq, Hk, D, P = case["Hq"], case["Hk"], case["D"], case["prefix"]
        rows, lens = _shape(case)
        keys = P + sum(n for m, n in zip(rows, lens) if m)
        seen = sum(m * P + m * (n - m) + m * (m + 1) // 2 for m, n in zip(rows, lens))
        return {"bytes": 2 * keys * Hk * (D // 2 + D // 16) + 4 * sum(rows) * Hq * D +
                (4 * sum(rows) * Hq if case["lse"] else 0),
                "flops": 4 * D * Hq * seen}
    T, V = case["rows"], case["V"]
    return {"bytes": T * V * SIZE[case["src"]] + 40 * T, "flops": 4 * T * V}


# ------------------------------------------------------------------------------------------
# The 4-bit cache


def _quantise(y, scale):
    """Codes (uint8, one a value) and scales (E4M3) of the blocks of 16 along the last axis of fp32 y."""
    block = y.unflatten(-1, (-1, 16))
    r = (block.abs().amax(-1) / 6.0) / scale
    s = r.clamp(max=448.0).to(torch.float8_e4m3fn)
    S = (s.float() * scale)[..., None]
    a = torch.where(S > 0, block.abs() / S, 0.0)
    code = (a > 0.25).byte()
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if up else (a > border)   # a tie goes to the even code
    return (code | ((block < 0) & (code > 0)).byte() << 3).flatten(-2), s


def _values(code, s, scale):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    return ((table[code.int()].unflatten(-1, (-1, 16)) * s.float()[..., None]) * scale).flatten(-2)


def _pack(y, page, scale):
    """The packed cache of y[slots, Hk, D]."""
    n, Hk, D = y.shape
    code, s = _quantise(y, scale)
    two = (code[..., 0::2] | code[..., 1::2] << 4).view(n // page, page, Hk, D // 2).transpose(1, 2).reshape(n // page, Hk, -1)
    s = s.view(torch.uint8).view(n // page, page, Hk, D // 16).transpose(1, 2).reshape(n // page, Hk, -1)
    return torch.cat([two, s], -1).reshape(-1)


def _unpack(cache, Hk, D, page, scale):
    """fp32 values [slots, Hk, D] of a packed cache."""
    shape = (-1, Hk, page * (D // 2 + D // 16))
    two = cache.view(shape)[..., :page * D // 2].unflatten(-1, (page, -1))
    s = cache.view(torch.float8_e4m3fn).view(shape)[..., page * D // 2:].unflatten(-1, (page, -1))
    code = torch.stack([two & 15, two >> 4], -1).flatten(-2)
    return _values(code, s, scale).transpose(1, 2).reshape(-1, Hk, D)


# ------------------------------------------------------------------------------------------
# Inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6007 + 29)
    return {"append": _prepare_append, "attn": _prepare_attn, "sample": _prepare_sample}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, dtype=dtype, device="cuda")


def _cos_sin(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _prepare_append(case, g):
    T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
    src, dst = TYPES[case["src"]], TYPES[case["dst"]]
    n_slots = _slots(case)
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
         "K_values": torch.zeros(n_slots, Hk, D, dtype=dst, device="cuda"),
         "V_values": torch.zeros(n_slots, Hk, D, dtype=dst, device="cuda")}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        s["K_cache"], s["V_cache"] = (torch.zeros(qmm.kv_fp4_bytes(n_slots, Hk, D), dtype=torch.uint8, device="cuda")
                                      for _ in range(2))
        s["args"] = qmm.make_norm_rope_fp4(s["Q"], s["K"], s["V"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                           s["positions"], s["slots"], s["Q_out"], s["K_cache"], s["V_cache"],
                                           n_slots=n_slots, page_size=case["page"], k_scale=K_SCALE, v_scale=V_SCALE,
                                           eps=EPS, interleaved=case["interleaved"])
        s["read"] = qmm.make_kv_fp4_read(s["K_cache"], s["V_cache"], s["K_values"], s["V_values"],
                                         n_slots=n_slots, page_size=case["page"], k_scale=K_SCALE, v_scale=V_SCALE)
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
         "K_cache": _pack(_randn(g, n_pages * page, Hk, D), page, K_SCALE),
         "V_cache": _pack(_randn(g, n_pages * page, Hk, D), page, V_SCALE),
         "prefix_pages": order[:n_prefix].contiguous(), "pages": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "row_starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "scale": D ** -0.5,
         "O": torch.empty(T, Hq, D, dtype=dtype, device="cuda"),
         "lse": torch.empty(T, Hq, device="cuda") if case["lse"] else None}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        s["args"] = qmm.make_attn_fp4(s["Q"], s["K_cache"], s["V_cache"], Hk, page, s["prefix_pages"], P, s["pages"],
                                      s["lens"], s["row_starts"], s["O"], scale=s["scale"], k_scale=K_SCALE,
                                      v_scale=V_SCALE, lse=s["lse"])
        s["workspace"] = torch.empty(qmm.attn_fp4_workspace_bytes(s["args"]), dtype=torch.uint8, device="cuda")
    return s


# temperature, top_k, top_p, min_p of the rows, in turn
PARAMS = {"plain": [(1.0, 0, 1.0, 0.0), (0.8, 0, 1.0, 0.0), (1.3, 0, 1.0, 0.0)],
          "nucleus": [(0.7, 0, 0.9, 0.0), (1.0, 0, 0.95, 0.0), (0.6, 20, 0.95, 0.0)],
          "mixed": [(1.0, 50, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (0.8, 0, 0.95, 0.02), (1.0, 0, 1.0, 0.05), (1.5, 1000, 1.0, 0.0),
                    (1.0, 0, 0.5, 0.0), (0.3, 40, 0.8, 0.1)]}


def _prepare_sample(case, g):
    T, V, B = case["rows"], case["V"], case["B"]
    # most of a row's logits are a wide bell, a few stand out of it; some rows are sharper than others
    logits = _randn(g, T, V).mul_(1.0 + 1.5 * torch.rand(T, 1, generator=g, device="cuda"))
    few = torch.randint(0, V, (T, 24), generator=g, device="cuda")
    logits.scatter_add_(1, few, 9.0 * torch.rand(T, 24, generator=g, device="cuda"))
    table = PARAMS[case["params"]]
    column = lambda k, dtype: torch.tensor([table[(3 * t + 2) % len(table)][k] for t in range(T)], dtype=dtype, device="cuda")
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    logits = logits.to(TYPES[case["src"]])
    # a drafter's guesses: what was fed to a row is mostly the likeliest token of the row before it
    fed = logits.argmax(-1).roll(1).int()
    missed = torch.rand(T, generator=g, device="cuda") < 0.15
    fed = torch.where(missed, torch.randint(0, V, (T,), generator=g, device="cuda").int(), fed)
    s = {"case": case, "logits": logits, "temperature": column(0, torch.float32), "top_k": column(1, torch.int32),
         "top_p": column(2, torch.float32), "min_p": column(3, torch.float32),
         "uniform": torch.rand(T, generator=g, device="cuda"), "fed": fed,
         "row_starts": torch.tensor([T * b // B for b in range(B + 1)], dtype=torch.int32, device="cuda"),
         "rows_max": max(T * (b + 1) // B - T * b // B for b in range(B)),
         "tokens": i32(T), "logprobs": torch.empty(T, device="cuda"), "accepted": i32(B), "next": i32(B)}
    if own:
        from bit_quantized_skinny_gb300 import qmm
        s["args"] = qmm.make_sample(s["logits"], s["uniform"], s["tokens"], temperature=s["temperature"],
                                    top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], logprobs=s["logprobs"],
                                    fed=s["fed"], row_starts=s["row_starts"], accepted=s["accepted"], next=s["next"])
    return s


# ------------------------------------------------------------------------------------------
# One pass


def run(s):
    return {"append": _run_append, "attn": _run_attn, "sample": _run_sample}[s["case"]["op"]](s)


def _run_append(s):
    if own:
        from bit_quantized_skinny_gb300 import qmm
        qmm.norm_rope_fp4(s["args"])
        qmm.kv_fp4_read(s["read"])
    else:
        cs = s["cos_sin"][s["positions"].long()]
        s["Q_out"].copy_(_plain_head(s["Q"], s["q_weight"], cs, s["case"], torch.float32))
        # 64 bits for the keys: a value next to the border of two codes
        keys = _plain_head(s["K"], s["k_weight"], cs, s["case"], torch.float64).float()
        s["K_values"][s["slots"]] = _values(*_quantise(keys, K_SCALE), K_SCALE).to(s["K_values"].dtype)
        s["V_values"][s["slots"]] = _values(*_quantise(s["V"].float(), V_SCALE), V_SCALE).to(s["V_values"].dtype)
    return s["Q_out"], s["K_values"], s["V_values"]


def _plain_head(x, weight, cos_sin, case, dtype):
    """Norm and rotation of every head of x[T, H, D]."""
    rot = case["rot"]
    x, cos_sin = x.to(dtype), cos_sin.to(dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(dtype)
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
        qmm.attn_shared_fp4(s["args"], s["workspace"])
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
    K, V = _unpack(s["K_cache"], Hk, D, page, K_SCALE), _unpack(s["V_cache"], Hk, D, page, V_SCALE)
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
    k_own = torch.where(held, K[slots], 0.0).permute(0, 2, 3, 1)                        # B, Hk, D, L
    v_own = torch.where(held, V[slots], 0.0).transpose(1, 2)                            # B, Hk, L, D
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
        s_pre = (q.reshape(Hk, T * G, D) @ K[slots].permute(1, 2, 0)).reshape(Hk, T, G, P)
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
        o = o + (p_pre.reshape(Hk, T * G, P) @ V[slots].transpose(0, 1)).reshape(Hk, T, G, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return (o.transpose(0, 1).reshape(T, Hq, D), (top + total.log()).transpose(0, 1).reshape(T, Hq))


def _run_sample(s):
    if own:
        from bit_quantized_skinny_gb300 import qmm
        qmm.sample(s["args"])
    else:
        tokens, logprobs = _plain_sample(s)
        s["tokens"].copy_(tokens)
        s["logprobs"].copy_(logprobs)
        accepted, after = _plain_accept(s, tokens)
        s["accepted"].copy_(accepted)
        s["next"].copy_(after)
    return s["tokens"], s["logprobs"], s["accepted"], s["next"]


def _plain_sample(s):
    """Weights and their sums in 64 bits: a sum decides between neighbouring tokens."""
    T, V = s["logits"].shape
    x, order = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    greedy = s["temperature"] <= 0
    w = ((x - x[:, :1].double()) / torch.where(greedy, 1.0, s["temperature"]).double()[:, None]).exp()
    rank = torch.arange(V, device=x.device)
    k = torch.where(s["top_k"] > 0, s["top_k"], V)
    w = torch.where(rank < k[:, None], w, 0.0)
    before = torch.nn.functional.pad(w.cumsum(-1)[:, :-1], (1, 0))
    top_p = s["top_p"].double()[:, None]
    keep = ((before < top_p * w.sum(-1, keepdim=True)) | (top_p >= 1)) & (w >= s["min_p"].double()[:, None])
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))   # back in the order of tokens
    sums = w.cumsum(-1)
    token = (sums <= s["uniform"].double()[:, None] * sums[:, -1:]).sum(-1)
    token = torch.where(greedy, order[:, 0], token)
    logprob = (w.gather(1, token[:, None])[:, 0] / sums[:, -1]).log()
    return token.int(), torch.where(greedy, 0.0, logprob).float()


def _plain_accept(s, tokens):
    starts = s["row_starts"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(s["rows_max"], device=tokens.device)
    row = (starts[:-1, None] + i).clamp(max=tokens.numel() - 1)
    stands = (tokens[row] == s["fed"][(row + 1).clamp(max=tokens.numel() - 1)]) & (i < n[:, None] - 1)
    accepted = stands.int().cumprod(-1).sum(-1)
    after = tokens[(starts[:-1] + accepted).clamp(max=tokens.numel() - 1)]
    return accepted, torch.where(n > 0, after, -1)


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](s)


def _exact_codes(y, scale):
    """Values of the 4-bit form of y (fp32 values held in 64 bits); quotients and scales are fp32 by definition."""
    f32 = lambda t: t.float().double()
    scale = torch.tensor(scale, dtype=torch.float32).double().item()
    block = y.reshape(*y.shape[:-1], -1, 16)
    r = f32(f32(block.abs().max(-1).values / 6) / scale)
    step = torch.exp2((torch.frexp(r).exponent - 1).clamp(min=-6).double() - 3)
    s = torch.minimum(torch.round(r / step) * step, torch.full_like(r, 448.0))
    S = f32(s * scale).unsqueeze(-1)
    a = f32(block.abs() / torch.where(S > 0, S, torch.ones_like(S)))
    step = torch.exp2((torch.frexp(a).exponent - 1).clamp(min=0).double() - 1)
    a = torch.minimum(torch.round(a / step) * step, torch.full_like(a, 6.0))
    return (torch.sign(block) * a * (S > 0) * s.unsqueeze(-1) * scale).reshape(y.shape)


def _exact_append(s):
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
    K = torch.zeros(s["K_values"].shape, dtype=torch.float64, device="cuda")
    V = torch.zeros_like(K)
    K[s["slots"]] = _exact_codes(out[1].float().double(), K_SCALE)
    V[s["slots"]] = _exact_codes(s["V"].double(), V_SCALE)
    return out[0], K, V


def _exact_attn(s):
    case = s["case"]
    P, Hq, Hk, D, page = (case[k] for k in ("prefix", "Hq", "Hk", "D", "page"))
    starts, lens = s["row_starts"].tolist(), s["lens"].tolist()
    O = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    table = torch.tensor([(-1) ** (c >> 3) * ((c & 1) / 2 if c & 6 == 0 else (1 + (c & 1) / 2) * 2 ** ((c >> 1 & 3) - 1))
                          for c in range(16)], dtype=torch.float64, device="cuda")

    def head(cache, pages, n, h, scale):
        """The first n keys' (or values') head h of a page list: n x D."""
        part = cache.view(-1, Hk, page * D * 9 // 16)[pages.long()[:-(-n // page)], h]
        byte = part[:, :page * D // 2].reshape(-1, D // 2).long()
        v = torch.empty(byte.shape[0], D, dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = table[byte % 16], table[byte // 16]
        e = part[:, page * D // 2:].reshape(-1, D // 16).double()
        exponent, fraction = torch.floor(e / 8), e % 8
        e = torch.where(exponent == 0, fraction * 2.0 ** -9, (8 + fraction) * torch.exp2(exponent - 10))
        return (v * e.repeat_interleave(16, dim=1) * torch.tensor(scale, dtype=torch.float32).double().item())[:n]

    for h in range(Hk):
        here = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
        pre_k, pre_v = (head(s[n], s["prefix_pages"], P, h, c) for n, c in (("K_cache", K_SCALE), ("V_cache", V_SCALE)))
        for b, n in enumerate(lens):
            r0, r1 = starts[b], starts[b + 1]
            if r0 == r1:
                continue
            keys = torch.cat([pre_k, head(s["K_cache"], s["pages"][b], n, h, K_SCALE)])
            vals = torch.cat([pre_v, head(s["V_cache"], s["pages"][b], n, h, V_SCALE)])
            limit = P + n - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
            hidden = torch.arange(P + n, device="cuda")[None, :] > limit[:, None]
            z = torch.einsum("rgd,kd->rgk", s["Q"][r0:r1, here].double(), keys) * s["scale"]
            z = z.masked_fill(hidden[:, None, :], -math.inf)
            lse[r0:r1, here] = torch.logsumexp(z, -1)
            O[r0:r1, here] = torch.einsum("rgk,kd->rgd", torch.softmax(z, -1), vals)
    return (O, lse) if s["lse"] is not None else O


def _exact_sample(s):
    """The logprob of the token that the definition picks, row by row; tokens and lengths are whole numbers."""
    logprobs = []
    for t in range(s["case"]["rows"]):
        temperature, k, top_p, min_p, u = (s[n][t].item() for n in ("temperature", "top_k", "top_p", "min_p", "uniform"))
        if temperature <= 0:
            logprobs.append(0.0)
            continue
        x = s["logits"][t].double()
        order = torch.argsort(x, descending=True, stable=True)
        if k > 0:
            order = order[:k]
        p = torch.softmax(x[order] / temperature, 0)
        stays = p >= min_p * p[0]
        if top_p < 1:
            stays &= p.cumsum(0) - p < top_p
        stays[0] = True
        order, p = order[stays], p[stays]
        by_index = torch.argsort(order)
        p = p[by_index] / p.sum()
        at = int((p.cumsum(0) <= u).sum().clamp(max=p.numel() - 1))
        logprobs.append(p[at].log().item())
    return None, torch.tensor(logprobs, dtype=torch.float64), None, None
