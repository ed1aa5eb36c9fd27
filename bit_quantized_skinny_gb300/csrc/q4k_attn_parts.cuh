// q4k_attn_parts.cuh — what the two attention kernels (over a cache of 16-bit values, and of 4-bit ones) share: the
// list of key tiles and its equal pieces, the walk along a piece, and the launch that joins a row's segments.
//
// Work.  A group is a block of rows that see the same keys, with one key/value head: for the prefix
// the rows of all streams, for own keys the rows of one stream; the G query heads of a key/value
// head are rows of the same block, so a key is read once for all of them.  The key tiles of all groups
// form one list, each group led by kLead units for what a segment costs besides its tiles, cut into
// equal pieces, one per CTA (one CTA an SM): every SM has the same work whatever the lengths, and the
// lengths stay on the device.  A piece holds one or several segments (runs of one group's key tiles).
// Each segment leaves its sums unnormalised in the workspace, with the running maximum and weight sum
// of each row, and attn_combine_kernel joins a row's segments in their order.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"

namespace q4k {
namespace {

constexpr int kRows = 128;           // rows of a row tile
constexpr int kMaxCtas = 152;
constexpr float kLn2 = 0.69314718055994530942f;

// One row's state beside its O: the maximum in units of log2, the weight sum, whether values were
// taken out of the block (nonzero), and, in the record of a group's first segment, the CTAs that hold
// the others: their number << 16 | the first of them.
struct RowStat {
  float top, sum;
  uint32_t odd, rest;
};

// What both kernels' launches take.
struct Common {
  qmm_attn_args a;
  float* o_rows;      // [2][T * Hq][D]: first segments, of the prefix and of own keys
  RowStat* s_rows;
  float* o_cta;       // [kMaxCtas][2 * kRows][D]: a CTA's first segment that begins inside a group
  RowStat* s_cta;
  int tokens;         // of a row tile
  int block;          // of a block of rows: one or two row tiles
  int n_pages, page_shift;
  uint32_t wait_polls, wait_ns;
  float k_scale, v_scale;   // of a 4-bit cache's tensors (1 for one of 16-bit values)
};

// Rows and own keys of a stream.
struct Stream {
  int t0, m, len;
};

// The piece of the list of key tiles that a CTA works on.
struct Piece {
  int64_t w0, w1, per;   // this CTA's units, units of a CTA
  int64_t scan[32];      // of the warps (a CTA has at most 32), beside what is written while some of them still read it
  int b, rb, h, rows;
  Stream s;           // stream b, if b >= 0
  int64_t unit;       // end of the CTA's units within that group
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Stream b, whatever the arrays hold.
__device__ __forceinline__ Stream stream_of(const qmm_attn_args& a, int b, bool* bad = nullptr) {
  const int r0 = a.row_starts[b], r1 = a.row_starts[b + 1], n = a.kv_lens[b];
  const int cap = (int)(a.pages_per_stream * a.page_size);
  Stream s;
  s.t0 = clampi(r0, 0, a.T);
  s.m = clampi(r1, s.t0, a.T) - s.t0;
  s.len = n < 0 || n > cap ? 0 : n;
  if (bad) *bad = r0 < 0 || r1 < r0 || r1 > a.T || (b == 0 && r0 != 0) || s.len != n;
  return s;
}
// Own keys that the rows of row block rb may see (by its last row), and the tiles they fill.
__device__ __forceinline__ int keys_of(const Stream& s, int rb, int block) {
  return clampi(s.len - s.m + min(s.m, (rb + 1) * block), 0, s.len);
}
template <int TILE>
__device__ __forceinline__ int tiles_of(int keys) { return (keys + TILE - 1) / TILE; }

// A run of key tiles of one group.
struct Seg {
  bool own;
  int h;            // key/value head
  int t0, rows;     // first row of the block, its rows (tokens)
  int keys;         // keys that its last row sees
  int first_keys;   // keys that its first row sees (below 0: rows further on see none either)
  int j0, j1;       // key tiles
  int rest;         // units of the group in the CTAs behind this one
  const int32_t* pages;
};

// Steps through a CTA's segments, the last one first; every role has its own.  (A piece usually ends with
// the beginning of a group and begins with the end of another: from the last one, the CTAs of the row
// blocks of a long prefix read its keys from the front at about the same time, and find them in L2.
// From the first one, each began elsewhere: 64 x 16 rows over 32768 keys read 1.9 GB from memory, not
// 0.48 GB.)
template <int TILE, int LEAD>
struct Walker {
  __device__ __forceinline__ static int units_of(int keys) { return keys > 0 ? tiles_of<TILE>(keys) + LEAD : 0; }
  int64_t left;
  int b, rb, h, j;   // group, end of what is left of it in units (-1: all)
  Stream s;
  int block, rows;   // rows of a block, rows in streams

  __device__ __forceinline__ void start(const Common& P, const Piece& m) {
    left = m.w1 - m.w0;
    b = m.b; rb = m.rb; h = m.h; j = (int)m.unit;
    block = P.block;
    rows = m.rows;
    s = m.s;
  }
  __device__ __forceinline__ bool next(const Common& P, Seg& g) {
    const qmm_attn_args& a = P.a;
    while (left > 0 && b >= -1) {
      if (rb < 0) {   // no group left of this stream
        if (--b < -1) return false;
        if (b >= 0) s = stream_of(a, b);
        rb = ((b >= 0 ? s.m : rows) + block - 1) / block - 1;
        h = a.Hk - 1;
        j = -1;
        continue;
      }
      g.own = b >= 0;
      g.t0 = rb * block;
      g.rows = min(block, (g.own ? s.m : rows) - g.t0);
      if (g.own) {
        g.keys = keys_of(s, rb, block);
        g.first_keys = s.len - s.m + g.t0 + 1;
        g.pages = a.pages + b * a.pages_per_stream;
        g.t0 += s.t0;
      } else {
        g.keys = g.first_keys = (int)a.prefix_len;
        g.pages = a.prefix_pages;
      }
      g.h = h;
      const int units = units_of(g.keys), end = j < 0 ? units : j;
      const int take = (int)min((int64_t)end, left);
      left -= take;
      g.j0 = max(0, end - take - LEAD);
      g.j1 = end - LEAD;
      g.rest = units - end;
      j = -1;
      if (--h < 0) {
        h = a.Hk - 1;
        --rb;
      }
      if (g.j1 > g.j0) return true;   // (else the piece holds only some of the group's lead)
    }
    return false;
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (TYPE == QMM_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Works out this CTA's piece; every thread of the CTA takes part, and the caller synchronises them before the piece is
// read.  Lengths and row starts that are out of range count as none and are reported.
template <int THREADS, int TILE, int LEAD>
__device__ __forceinline__ void deal(const Common& P, Piece& M, unsigned* status) {
  static_assert(THREADS % 32 == 0 && THREADS / 32 <= (int)(sizeof(M.scan) / sizeof(M.scan[0])), "an entry a warp");
  const qmm_attn_args& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = P.block;
  auto units = [](int keys) { return Walker<TILE, LEAD>::units_of(keys); };
  // the page tables towards L2 while the pieces are worked out: one 128-byte line a thread
  const int64_t line = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * 32;
  const int64_t n_pre = (a.prefix_len + a.page_size - 1) >> P.page_shift, n_own = a.B * a.pages_per_stream;
  if (line < n_pre) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.prefix_pages + line));
  if (line < n_own) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.pages + line));
  constexpr int kPer = (QMM_ATTN_MAX_STREAMS + THREADS - 1) / THREADS;
  Stream str[kPer];
  int64_t mine[kPer], sum = 0;
  bool wrong = false;
  const int rows = a.B > 0 ? clampi(a.row_starts[a.B], 0, a.T) : 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int b = threadIdx.x * kPer + q;
    mine[q] = 0;
    if (b < a.B) {
      bool bad;
      str[q] = stream_of(a, b, &bad);
      wrong |= bad;
      for (int rb = 0; rb * block < str[q].m; ++rb)
        mine[q] += (int64_t)a.Hk * units(keys_of(str[q], rb, block));
    }
    sum += mine[q];
  }
  if (wrong && blockIdx.x == 0) atomicOr(status, kErrIndex);
  int64_t upto = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) M.scan[warp] = upto;
  __syncthreads();
  int64_t before = upto - sum, own = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += M.scan[w];
    own += M.scan[w];
  }
  const int punits = units((int)a.prefix_len);
  const int64_t prefix = (int64_t)((rows + block - 1) / block) * a.Hk * punits;
  const int64_t W = prefix + own;
  // equal pieces: no CTA has more than ceil(W / CTAs), whichever way the remainder falls
  const int64_t per = W < (int64_t(1) << 31) ? (int64_t)(((uint32_t)W + gridDim.x - 1) / gridDim.x)
                                             : (W + gridDim.x - 1) / gridDim.x;
  const int64_t w0 = min(W, blockIdx.x * per), w1 = min(W, w0 + per);
  const int64_t last = w1 - 1;   // its group is the first one the CTA works on
  if (threadIdx.x == 0) {
    M.w0 = w0;
    M.w1 = w1;
    M.per = per;
    M.rows = rows;
    if (w0 < w1 && last < prefix) {
      const int64_t g = prefix < (int64_t(1) << 31) ? (int64_t)((uint32_t)last / (uint32_t)punits) : last / punits;
      M.b = -1;
      M.rb = (int)((uint32_t)g / (uint32_t)a.Hk);
      M.h = (int)((uint32_t)g - (uint32_t)M.rb * (uint32_t)a.Hk);
      M.unit = last - g * punits + 1;
    }
  }
  before += prefix;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int b = threadIdx.x * kPer + q;
    if (b < a.B && w0 < w1 && last >= before && last < before + mine[q]) {
      int64_t at = last - before;
      int rb = 0, h = 0, n = units(keys_of(str[q], 0, block));
      while (at >= (int64_t)a.Hk * n) { at -= (int64_t)a.Hk * n; n = units(keys_of(str[q], ++rb, block)); }
      while (at >= n) { at -= n; ++h; }
      M.s = str[q];
      M.b = b;
      M.rb = rb;
      M.h = h;
      M.unit = at + 1;
    }
    before += mine[q];
  }
}

// ------------------------------------------------------------------------------------------
// Joins a row's segments: SHARE warps per (row, head).  The segments of a group are the one that begins
// it (in the row's own record) and those of the CTAs whose piece begins inside it.
constexpr int kCombineWarps = 8;

// Column of the value at position p of a row's record: the epilogue keeps columns 8k + 2q, 8k + 2q + 1
// (k = 0..3) of each 32 together, as the 8 values of thread q of four.
__device__ __forceinline__ int column_of(int p) {
  return (p & ~31) + 8 * ((p & 7) >> 1) + 2 * ((p & 31) >> 3) + (p & 1);
}

template <int D, int TYPE, int SHARE, bool FP4>
__global__ void __launch_bounds__(32 * kCombineWarps) attn_combine_kernel(const __grid_constant__ Common P) {
  constexpr int kV = D / 32;   // values of a lane: positions kV * lane and on
  constexpr int kAhead = 8;    // records whose O a warp has in flight
  const qmm_attn_args& a = P.a;
  __shared__ int stream;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int head = (blockIdx.y * kCombineWarps + (threadIdx.x >> 5)) / SHARE, share = (threadIdx.x >> 5) % SHARE;
  if (threadIdx.x == 0) stream = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const Stream s = stream_of(a, b);
    if (t >= s.t0 && t < s.t0 + s.m) stream = b;   // one stream, if the starts do not decrease
  }
  __syncthreads();
  if (SHARE == 1 && head >= a.Hq) return;
  const int b = head < a.Hq ? stream : -1, G = a.Hq / a.Hk, block = P.block;
  Stream s{};
  bool has[2] = {b >= 0 && a.prefix_len > 0 && t < a.row_starts[a.B], false};   // key tiles of the prefix, of own keys
  if (b >= 0) {
    s = stream_of(a, b);
    has[1] = keys_of(s, (t - s.t0) / block, block) > 0;
  }
  const int64_t rec = (int64_t)t * a.Hq + head;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto load = [&](const float* p, float (&x)[kV]) {
    if constexpr (kV == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * lane);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p + 2 * lane);
      x[0] = v.x; x[1] = v.y;
    }
  };
  // a row that saw none of a segment's keys has no part in it
  auto saw = [](const RowStat& r) { return !(r.top == -INFINITY && r.sum == 0.0f); };
  RowStat st[2] = {{-INFINITY, 0.0f, 0u, 0u}, {-INFINITY, 0.0f, 0u, 0u}};
  float x[2][kV] = {};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (has[k]) {
      const int64_t at = k ? (int64_t)a.T * a.Hq + rec : rec;
      st[k] = P.s_rows[at];
      if (share == 0) load(P.o_rows + at * D, x[k]);
    }
  float top = share == 0 ? fmaxf(st[0].top, st[1].top) : -INFINITY, sum = 0.0f, o[kV] = {};
  uint32_t odd = st[0].odd | st[1].odd;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (share == 0 && saw(st[k])) {
      const float w = exp2_fast(st[k].top - top);
      sum = __fmaf_rn(st[k].sum, w, sum);
#pragma unroll
      for (int q = 0; q < kV; ++q) o[q] = __fmaf_rn(x[k][q], w, o[q]);
    }
  // the other segments of the two groups, one a lane
  const int n0 = min((int)(st[0].rest >> 16), kMaxCtas), all = n0 + min((int)(st[1].rest >> 16), kMaxCtas);
  const int part = (all + SHARE - 1) / SHARE, end = min(all, (share + 1) * part);   // this warp's of them
  int row[2] = {0, 0};   // of the tiles of each group's block
  if (all > 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int in = (k ? t - s.t0 : t) % block;
      row[k] = (in < P.tokens ? in * G : kRows + (in - P.tokens) * G) + head % G;
    }
  }
  constexpr int kFew = 3;
  if (SHARE == 1 && all > 0 && all <= kFew) {   // few of them, as a rule where rows are many: one after the other
    RowStat q[kFew];
    float y[kFew][kV];
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
      q[r] = RowStat{-INFINITY, 0.0f, 0u, 0u};
      if (r < all) {
        const bool own = r >= n0;
        const int cta = min((int)((own ? st[1].rest : st[0].rest) & 0xFFFFu) + (own ? r - n0 : r), kMaxCtas - 1);
        const int at = cta * 2 * kRows + (own ? row[1] : row[0]);
        q[r] = P.s_cta[at];
        load(P.o_cta + (int64_t)at * D, y[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
      if (!saw(q[r])) continue;
      const float best = fmaxf(top, q[r].top), f = exp2_fast(q[r].top - best);
      const float keep = top == -INFINITY && sum == 0.0f ? 0.0f : exp2_fast(top - best);
      sum = __fmaf_rn(sum, keep, q[r].sum * f);
      top = best;
      odd |= q[r].odd;
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] = __fmaf_rn(y[r][k], f, o[k] * keep);
    }
  } else if (share * part < end) {
    for (int r0 = share * part; r0 < end; r0 += 32) {
      const int r = r0 + lane;
      const bool own = r >= n0, live = r < end;
      const int cta = min((int)((own ? st[1].rest : st[0].rest) & 0xFFFFu) + (own ? r - n0 : r), kMaxCtas - 1);
      const int at = cta * 2 * kRows + (own ? row[1] : row[0]);
      RowStat q{-INFINITY, 0.0f, 0u, 0u};
      if (live) q = P.s_cta[at];
      // their O, some at a time, asked for before the statistics are there
      float best = top, keep = 1.0f, w = 0.0f;
#pragma unroll 1
      for (int j0 = 0; j0 < 32 && r0 + j0 < end; j0 += kAhead) {
        float y[kAhead][kV];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int from = __shfl_sync(0xffffffffu, at, j0 + j);
#pragma unroll
          for (int k = 0; k < kV; ++k) y[j][k] = 0.0f;
          if (r0 + j0 + j < end) load(P.o_cta + (int64_t)from * D, y[j]);
        }
        if (j0 == 0) {
          best = q.top;
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
          best = fmaxf(best, top);
          w = saw(q) ? exp2_fast(q.top - best) : 0.0f;
          float part = saw(q) ? q.sum * w : 0.0f;
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
          keep = top == -INFINITY && sum == 0.0f ? 0.0f : exp2_fast(top - best);
          sum = __fmaf_rn(sum, keep, part);
          top = best;
          odd |= __any_sync(0xffffffffu, q.odd != 0);
#pragma unroll
          for (int k = 0; k < kV; ++k) o[k] *= keep;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float f = __shfl_sync(0xffffffffu, w, j0 + j);
          if (f != 0.0f)   // (of a segment none of whose keys the row saw, O means nothing)
#pragma unroll
            for (int k = 0; k < kV; ++k) o[k] = __fmaf_rn(y[j][k], f, o[k]);
        }
      }
    }
  }
  if constexpr (SHARE > 1) {   // the warps of a row, joined by the first
    __shared__ float o_s[kCombineWarps][D];
    __shared__ float4 stat_s[kCombineWarps];
    const int w0 = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < kV; ++k) o_s[w0][kV * lane + k] = o[k];
    if (lane == 0) stat_s[w0] = make_float4(top, sum, __uint_as_float(odd), 0.0f);
    __syncthreads();
    if (share != 0 || head >= a.Hq) return;
    float best = top;
#pragma unroll
    for (int w = 1; w < SHARE; ++w) best = fmaxf(best, stat_s[w0 + w].x);
    const float keep = top == -INFINITY && sum == 0.0f ? 0.0f : exp2_fast(top - best);
    sum *= keep;
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] *= keep;
#pragma unroll
    for (int w = 1; w < SHARE; ++w) {
      const float4 q = stat_s[w0 + w];
      odd |= __float_as_uint(q.z);
      if (q.x == -INFINITY && q.y == 0.0f) continue;
      const float f = exp2_fast(q.x - best);
      sum = __fmaf_rn(q.y, f, sum);
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] = __fmaf_rn(o_s[w0 + w][kV * lane + k], f, o[k]);
    }
    top = best;
  }
  const float inv = sum == 0.0f ? 0.0f : (FP4 ? P.v_scale : 1.0f) / sum;
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = sum == 0.0f ? 0.0f : o[k] * inv;
  if (odd) {
    // infinities and NaN among the keys that only some rows of the block see: their sum
    float extra[kV] = {};
    const int sees = clampi(s.len - s.m + t - s.t0 + 1, 0, s.len);
    for (int j = max(0, s.len - s.m); j < sees; ++j) {
      const int page = a.pages[b * a.pages_per_stream + j / a.page_size];
      if (page < 0 || page >= a.n_slots / a.page_size) continue;
      if constexpr (FP4) {
        const uint8_t* scales = static_cast<const uint8_t*>(a.V_cache) + kv4::run_at(page, head / G, a.Hk, a.page_size, D) +
                                a.page_size * (D / 2) + (j % a.page_size) * (D / 16);
#pragma unroll
        for (int k = 0; k < kV; ++k)
          if ((scales[column_of(kV * lane + k) / kv4::kBlock] & 0x7Fu) == kv4::kScaleNaN) extra[k] = NAN;
        continue;
      }
      const int64_t at = (((int64_t)page * a.page_size + j % a.page_size) * a.Hk + head / G) * D;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const uint16_t raw = static_cast<const uint16_t*>(a.V_cache)[at + column_of(kV * lane + k)];
        const float v = TYPE == QMM_BF16 ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw));
        if (!(fabsf(v) < INFINITY)) extra[k] += v;
      }
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] += extra[k];
  }
  uint16_t* out = static_cast<uint16_t*>(a.O) + (int64_t)t * a.ldo + (int64_t)head * D;
#pragma unroll
  for (int k = 0; k < kV; k += 2)
    *reinterpret_cast<uint32_t*>(out + column_of(kV * lane + k)) = pack2<TYPE>(o[k], o[k + 1]);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + head] = sum == 0.0f ? -INFINITY : __fmaf_rn(top, kLn2, logf(sum));
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

struct Space {
  size_t o_rows, s_rows, o_cta, s_cta, total;
  explicit Space(const qmm_attn_args& a) {
    const size_t rows = 2 * (size_t)a.T * a.Hq, cta = (size_t)kMaxCtas * 2 * kRows;
    o_rows = 0;
    o_cta = o_rows + up(rows * a.D * sizeof(float));
    s_rows = o_cta + up(cta * a.D * sizeof(float));
    s_cta = s_rows + up(rows * sizeof(RowStat));
    total = s_cta + up(cta * sizeof(RowStat)) + 256;   // the base may be 16-byte aligned only
  }
};

// The launch that joins the segments, behind the attention's: it may be scheduled while that one finishes (programmatic
// dependent launch) and waits for it before it reads its records.
template <int D, int TYPE, bool FP4>
cudaError_t launch_combine(const Common& P, int sms, cudaStream_t stream) {
  const qmm_attn_args& a = P.a;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(a.T, (a.Hq + kCombineWarps - 1) / kCombineWarps);
  cfg.blockDim = dim3(32 * kCombineWarps);
  // Four warps share a row's records where all of their CTAs, three an SM, run at once; with more rows, one
  // warp a row.  The limit shows at any number of records.  Behind 32768 shared keys, some 19 records a row:
  // 800 rows 35.7 us (one warp a row 37.5), 960 rows 38.4 (37.8), 1280 rows 44.5 (43.7).  Behind 8192: 800 rows
  // 26.8 (27.0), 960 rows 31.4 (29.0).  640 rows of 8 streams' own 3000 to 6000 keys 15.0 (17.4).
  if ((int64_t)a.T * a.Hq * 4 <= 3 * kCombineWarps * (int64_t)sms) {
    cfg.gridDim.y = (a.Hq * 4 + kCombineWarps - 1) / kCombineWarps;
    return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, TYPE, 4, FP4>, P);
  }
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, TYPE, 1, FP4>, P);
}

// The common part of a call's parameters.
inline void fill(Common& P, const qmm_attn_args& a, int tokens, int block, void* workspace) {
  P.a = a;
  P.tokens = tokens;
  P.block = block;
  P.n_pages = (int)(a.n_slots / a.page_size);
  P.page_shift = 31 - __builtin_clz((unsigned)a.page_size);
  P.k_scale = P.v_scale = 1.0f;
  const Space sp(a);
  uint8_t* ws = reinterpret_cast<uint8_t*>(up(reinterpret_cast<uintptr_t>(workspace)));
  P.o_rows = reinterpret_cast<float*>(ws + sp.o_rows);
  P.o_cta = reinterpret_cast<float*>(ws + sp.o_cta);
  P.s_rows = reinterpret_cast<RowStat*>(ws + sp.s_rows);
  P.s_cta = reinterpret_cast<RowStat*>(ws + sp.s_cta);
  get_wait_limit(&P.wait_polls, &P.wait_ns);
}

}  // namespace
}  // namespace q4k
