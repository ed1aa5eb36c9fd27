"""The attention half of one layer of a verify pass, as a user of the library runs it:

    q, k, v = X Wq^T, X Wk^T, X Wv^T            one batched product launch (Q4K weights)
    q, k, v += the rows' adapters               run_lora, in place
    queries, cache <- norm and rotation         norm_rope, or norm_rope_fp4 into a 4-bit cache
    O = attention over the shared prefix and each stream's own keys     attn_shared, or attn_shared_fp4
    Y = O Wo^T + the rows' adapters             run, run_lora

Every buffer and argument block is made once; run() only enqueues, so a sequence of calls can be
captured into a CUDA graph (after one call on the capturing stream, which makes the products'
workspace of that stream).  What changes from pass to pass (X, positions, slots, kv_lens, row_starts, pages, adapter
ids) is device memory that the caller writes before run().
"""
from __future__ import annotations

import torch

from . import qmm


class AttentionHalf:
    def __init__(self, weights, width: int, Hq: int, Hk: int, D: int, rows: int, streams: int, K_cache, V_cache,
                 page_size: int, pages_per_stream: int, q_norm, k_norm, cos_sin, prefix_pages=None, prefix_len: int = 0,
                 adapters=None, rank_max: int = 0, kv_scales=None):
        """weights: {"q", "k", "v", "o"}: packed Q4K tensors (Hq*D x width, Hk*D x width twice, width x
        Hq*D); adapters: None, or {"q", "k", "v", "o"}: tables of qmm.make_lora_adapters(); kv_scales: None (a cache
        of 16-bit values), or the tensor scales of the keys and the values of a packed 4-bit cache."""
        dev = K_cache.device
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)
        self.rows, self.rank_max = rows, rank_max
        self.X = torch.zeros(rows, width, dtype=torch.bfloat16, device=dev)
        self.Y = f32(rows, width)
        self.positions, self.ids = i32(rows), i32(rows) - 1
        self.slots = torch.full((rows,), -1, dtype=torch.int64, device=dev)
        self.kv_lens, self.row_starts, self.pages = i32(streams), i32(streams + 1), i32(streams, pages_per_stream)
        shape = {"q": (Hq * D, width), "k": (Hk * D, width), "v": (Hk * D, width), "o": (width, Hq * D)}
        y = {n: f32(rows, shape[n][0]) for n in "qkv"}
        y["o"] = self.Y
        queries = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        O = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=dev)
        x = {"q": self.X, "k": self.X, "v": self.X, "o": O.view(rows, Hq * D)}
        self._o = (weights["o"], *shape["o"], x["o"], self.Y)
        self._qkv = qmm.make_entries([(weights[n], x[n], y[n], *shape[n]) for n in "qkv"])
        self._fp4 = kv_scales is not None
        heads = (y["q"].view(rows, Hq, D), y["k"].view(rows, Hk, D), y["v"].view(rows, Hk, D), q_norm, k_norm, cos_sin,
                 self.positions, self.slots, queries, K_cache, V_cache)
        keys = (queries, K_cache, V_cache, Hk, page_size) if self._fp4 else (queries, K_cache, V_cache, page_size)
        keys += (prefix_pages, prefix_len, self.pages, self.kv_lens, self.row_starts, O)
        if self._fp4:
            k_scale, v_scale = kv_scales
            self._attn = qmm.make_attn_fp4(*keys, scale=D ** -0.5, k_scale=k_scale, v_scale=v_scale)
            self._norm_rope = qmm.make_norm_rope_fp4(*heads, self._attn.base.n_slots, page_size, k_scale, v_scale)
        else:
            self._norm_rope = qmm.make_norm_rope(*heads)
            self._attn = qmm.make_attn(*keys, scale=D ** -0.5)
        self._lora = None
        if adapters is not None:
            entry = lambda n: (adapters[n], x[n], y[n], y[n], *shape[n])
            self._lora = [qmm.make_lora_entries([entry(n) for n in "qkv"]), qmm.make_lora_entries([entry("o")])]
        need = [(qmm.attn_fp4_workspace_bytes if self._fp4 else qmm.attn_workspace_bytes)(self._attn)]
        need += [qmm.lora_workspace_bytes(e, rows, rank_max) for e in self._lora or ()]
        self._workspace = torch.empty(max(need), dtype=torch.uint8, device=dev)   # one call at a time uses it
        self._keep = (weights, y, queries, O)

    def run(self, stream=None):
        """Y = attention half of X, enqueued on `stream` (default: torch's current one)."""
        qmm.run_batched(self._qkv, self.rows, stream=stream)
        if self._lora:
            qmm.run_lora(self._lora[0], self.ids, self.rows, self.rank_max, self._workspace, stream=stream)
        if self._fp4:
            qmm.norm_rope_fp4(self._norm_rope, stream=stream)
            qmm.attn_shared_fp4(self._attn, self._workspace, stream=stream)
        else:
            qmm.norm_rope(self._norm_rope, stream=stream)
            qmm.attn_shared(self._attn, self._workspace, stream=stream)
        W, N, K, X, Y = self._o
        qmm.run(W, N, K, X, Y, stream=stream)
        if self._lora:
            qmm.run_lora(self._lora[1], self.ids, self.rows, self.rank_max, self._workspace, stream=stream)
        return self.Y
