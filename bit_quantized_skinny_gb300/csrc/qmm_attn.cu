// qmm_attn.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, both in pages of one cache (qmm_attn_shared).
//
// Work.  A group is a block of rows that see the same keys, with one key/value head: for the prefix
// the rows of all streams, for own keys the rows of one stream; the G query heads of a key/value
// head are rows of the same block, so a key is read once for all of them.  A row tile is 128 rows
// (128 / G tokens) and a block up to two tiles; a key tile is 128 keys.  The key tiles of all
// groups form one list, cut into equal pieces, one per CTA (one CTA an SM): every SM streams
// the same number of bytes whatever the lengths, and the lengths stay on the device.  A piece holds
// one or several segments (runs of one group's key tiles).  Each segment leaves its sums
// unnormalised in the workspace, with the running maximum and weight sum of each row, and
// attn_combine_kernel joins a row's segments in their order.
//
// One segment.  Two lanes of flash attention share the tensor cores: with more than one row tile
// each lane has a row tile and both read every key tile; with one, the lanes take the key tiles in
// turn and are joined at the segment's end.  Per lane and key tile:
//     S = Q K^T              tcgen05, both operands in shared memory (TMA, 128-byte swizzle)
//     p = 2^(c S - m)        a thread per row: S from tensor memory into registers, c = scale log2 e
//     O += p V               tcgen05, p (16 bits, rounded once) from tensor memory, V MN-major
// m is the maximum when it was last moved: it moves, and O is rescaled, only when the row's maximum
// grew by more than 8 (2^8 in a 16-bit p costs no precision), so O stays in tensor memory.
//
// Keys that a row may not see are set to -inf by position, so their K may hold anything.  Their p
// is 0, but 0 * NaN is not: value rows behind the last key are zeroed in shared memory, and so are
// non-finite values among the keys that only some rows of the block see (a draft's last keys);
// attn_combine_kernel then adds those back, from the cache, to the rows that see them.
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_tcgen05.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kTile = 128;           // rows of a row tile, keys of a key tile
constexpr int kMaxCtas = 152;
constexpr int kLaneWarps = 4;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kQWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr uint32_t kTmemCols = 512;   // S and p of the lanes at 128 L, O at 256 + 128 L
constexpr float kGrow = 8.0f;
constexpr uint32_t kWaitLimit = 1u << 17;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// One row's state beside its O: the maximum in units of log2, the weight sum, and whether values
// were taken out of the block (nonzero).
struct RowStat {
  float top, sum;
  uint32_t odd, unused;
};

struct Params {
  qmm_attn_args a;
  CUtensorMap mapQ, mapK, mapV;
  float* o_rows;      // [2][T * Hq][D]: first segments, of the prefix and of own keys
  RowStat* s_rows;
  float* o_cta;       // [kMaxCtas][2 * 128][D]: a CTA's first segment that begins inside a group
  RowStat* s_cta;
  int64_t* plan;      // [0] tiles, [1] CTAs with work, [2 + b] first own tile of stream b
  int tokens;         // of a row tile
  uint32_t wait_polls, wait_ns;
};

template <int D>
struct Smem {
  static constexpr int kHalf = kTile * 128;              // 128 rows of 64 values
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTileBytes;
  static constexpr int kStats = kKV + kStages * kTileBytes;   // (top, sum) of the two lanes' rows
  static constexpr int kMisc = kStats + 2 * kTile * 8;
  static constexpr int kTotal = kMisc + 1024;
};
static_assert(Smem<128>::kTotal <= 227 * 1024 && Smem<64>::kTotal <= 227 * 1024, "shared memory");

enum : int {   // barriers
  kBarFull = 0, kBarEmpty = 10, kBarQFull = 20, kBarQEmpty = 22, kBarS = 24, kBarP = 26, kBarO = 28, kBarJoin = 30,
  kBarDrain = 31, kBars = 32
};

struct Misc {
  uint64_t bars[kBars];
  int64_t total, prefix_tiles, w0, w1;
  int64_t scan[kThreads / 32];
  int b, rb, h;
  int64_t tile;       // first tile within its group
  uint32_t tmem;
  int abort;
  uint32_t odd[8];    // [s % 8]: s, if values were taken out in segment s (the lanes drift a few apart)
};
static_assert(sizeof(Misc) <= 1024, "misc");

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Rows and own keys of stream b, whatever the arrays hold.
struct Stream {
  int t0, m, len;
};
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
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// A run of key tiles of one group.
struct Seg {
  bool own;
  int h;            // key/value head
  int t0, rows;     // first row of the block, its rows (tokens)
  int keys;         // keys that its last row sees
  int first_keys;   // keys that its first row sees (below 0: rows further on see none either)
  int j0, j1;       // key tiles
  const int32_t* pages;
};

// Steps through a CTA's segments; every role has its own.
struct Walker {
  int64_t left;
  int b, rb, h, j;
  Stream s;
  int block;

  __device__ __forceinline__ void start(const Params& P, const Misc& m) {
    left = m.w1 - m.w0;
    b = m.b; rb = m.rb; h = m.h; j = (int)m.tile;
    block = 2 * P.tokens;
    if (b >= 0 && left > 0) s = stream_of(P.a, b);
  }
  __device__ __forceinline__ bool next(const Params& P, Seg& g) {
    const qmm_attn_args& a = P.a;
    while (left > 0) {
      int tiles;
      if (b < 0) {
        const int rows = a.B > 0 ? clampi(a.row_starts[a.B], 0, a.T) : 0;
        if (rb * (int64_t)block >= rows) { b = 0; rb = h = j = 0; s = stream_of(a, 0); continue; }
        g.own = false;
        g.t0 = rb * block;
        g.rows = min(block, rows - g.t0);
        g.keys = g.first_keys = (int)a.prefix_len;
        g.pages = a.prefix_pages;
      } else {
        if (rb * (int64_t)block >= s.m) {
          rb = h = j = 0;
          if (++b >= a.B) return false;
          s = stream_of(a, b);
          continue;
        }
        g.own = true;
        g.t0 = s.t0 + rb * block;
        g.rows = min(block, s.m - rb * block);
        g.keys = keys_of(s, rb, block);
        g.first_keys = s.len - s.m + rb * block + 1;
        g.pages = a.pages + b * a.pages_per_stream;
      }
      tiles = tiles_of(g.keys);
      if (j >= tiles) { j = 0; if (tiles == 0 || ++h == a.Hk) { h = 0; ++rb; } continue; }
      g.h = h;
      g.j0 = j;
      g.j1 = (int)min((int64_t)tiles, j + left);
      left -= g.j1 - g.j0;
      j = g.j1;
      return true;
    }
    return false;
  }
};

// Order of a segment's n key tiles in the ring: K0, then K1, V0, K2, V1, ...
__device__ __forceinline__ uint32_t pos_k(int i) { return i == 0 ? 0u : 2u * i - 1; }
__device__ __forceinline__ uint32_t pos_v(int i, int n) { return i == n - 1 ? 2u * n - 1 : 2u * i + 2; }

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

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

// Whether one of the two 16-bit values of w is an infinity or NaN (all exponent bits set).
template <int TYPE>
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  constexpr uint32_t kExp = TYPE == QMM_BF16 ? 0x7F807F80u : 0x7C007C00u;
  constexpr uint32_t kOne = TYPE == QMM_BF16 ? 0x00800080u : 0x04000400u;
  return (((w & kExp) + kOne) & 0x80008000u) != 0;
}
template <int TYPE>
__device__ __forceinline__ uint32_t without_odd(uint32_t w) {
  constexpr uint32_t kExp = TYPE == QMM_BF16 ? 0x7F80u : 0x7C00u;
  if ((w & kExp) == kExp) w &= 0xFFFF0000u;
  if ((w >> 16 & kExp) == kExp) w &= 0x0000FFFFu;
  return w;
}

__device__ __forceinline__ void store8(float* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using L = Smem<D>;
  constexpr int kS = L::kStages;
  const qmm_attn_args& a = P.a;
  Misc& M = *reinterpret_cast<Misc*>(smem + L::kMisc);
  volatile int* abort_flag = &M.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_addr(M.bars);
  auto bar = [&](int k) { return bars + 8u * k; };
  const int G = a.Hq / a.Hk, block = 2 * P.tokens;

  // ---- barriers, tensor memory, and this CTA's piece of the list of key tiles
  if (threadIdx.x == 0) {
    for (int k = 0; k < kS; ++k) { mbar_init(bar(kBarFull + k), 1); mbar_init(bar(kBarEmpty + k), 1); }
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(kBarQFull + k), 1);
      mbar_init(bar(kBarQEmpty + k), 1);
      mbar_init(bar(kBarS + k), 1);
      mbar_init(bar(kBarP + k), kLaneWarps);
      mbar_init(bar(kBarO + k), 1);
    }
    mbar_init(bar(kBarJoin), 2 * kLaneWarps);
    mbar_init(bar(kBarDrain), 1);
    M.abort = 0;
    for (int k = 0; k < 8; ++k) M.odd[k] = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_addr(&M.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  {
    constexpr int kPer = (QMM_ATTN_MAX_STREAMS + kThreads - 1) / kThreads;
    int64_t mine[kPer], sum = 0;
    bool wrong = false;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int b = threadIdx.x * kPer + q;
      mine[q] = 0;
      if (b < a.B) {
        bool bad;
        const Stream s = stream_of(a, b, &bad);
        wrong |= bad;
        for (int rb = 0; rb * (int64_t)block < s.m; ++rb) mine[q] += (int64_t)a.Hk * tiles_of(keys_of(s, rb, block));
      }
      sum += mine[q];
    }
    if (wrong && blockIdx.x == 0) atomicOr(&g_status, kErrIndex);
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += M.scan[w];
      own += M.scan[w];
    }
    const int ptiles = tiles_of((int)a.prefix_len);
    const int rows = a.B > 0 ? clampi(a.row_starts[a.B], 0, a.T) : 0;
    const int64_t prefix = (int64_t)((rows + block - 1) / block) * a.Hk * ptiles;
    const int64_t W = prefix + own, C = min((int64_t)gridDim.x, W);
    const int64_t w0 = C > 0 && blockIdx.x < C ? blockIdx.x * W / C : 0;
    const int64_t w1 = C > 0 && blockIdx.x < C ? (blockIdx.x + 1) * W / C : 0;
    if (threadIdx.x == 0) {
      M.w0 = w0;
      M.w1 = w1;
      if (w0 < prefix) {
        const int64_t g = w0 / ptiles;
        M.b = -1;
        M.rb = (int)(g / a.Hk);
        M.h = (int)(g % a.Hk);
        M.tile = w0 % ptiles;
      }
      if (blockIdx.x == 0) { P.plan[0] = W; P.plan[1] = C; }
    }
    before += prefix;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int b = threadIdx.x * kPer + q;
      if (b < a.B) {
        if (blockIdx.x == 0) P.plan[2 + b] = before;
        if (w0 >= before && w0 < before + mine[q]) {
          const Stream s = stream_of(a, b);
          int64_t at = w0 - before;
          int rb = 0, n = tiles_of(keys_of(s, 0, block));
          while (at >= (int64_t)a.Hk * n) { at -= (int64_t)a.Hk * n; n = tiles_of(keys_of(s, ++rb, block)); }
          M.b = b;
          M.rb = rb;
          M.h = (int)(at / n);
          M.tile = at % n;
        }
      }
      before += mine[q];
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = M.tmem;

  // A bounded wait for a phase of a barrier; false: this wait, or another one, gave up.
  auto wait = [&](int k, uint32_t parity) -> bool {
    if (mbar_try(bar(k), parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar(k), parity, P.wait_polls ? P.wait_polls : kWaitLimit, P.wait_ns ? P.wait_ns : kSuspendNs))
      return true;
    atomicOr(&g_status, kErrWaitTimeout);
    *abort_flag = 1;
    return false;
  };
  auto wait_w = [&](int k, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(k, parity)); };

  Walker walk;
  walk.start(P, M);
  Seg g;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ keys and values
    // A tile is one box per page (or 128 keys of a longer page) and half of 64 values; lane k copies
    // box k / halves of half k % halves.  Pages behind the last key are not read.
    constexpr int kHalves = D / 64;
    const int per_box = min(a.page_size, kTile);
    const uint32_t box_bytes = per_box * 128;
    const int64_t n_pages = a.n_slots / a.page_size;
    uint32_t pos = 0, filled = 0;   // stages ever filled
    bool ok = true;
    auto slot_of = [&](const Seg& s, int tile) -> int {   // first slot of this lane's box
      const int key = tile * kTile + lane / kHalves * per_box;
      if (lane >= kHalves * (kTile / per_box) || key >= s.keys) return -1;
      const int page = s.pages[key / a.page_size];
      if (page < 0 || page >= n_pages) {
        atomicOr(&g_status, kErrIndex);
        return (int)a.n_slots;   // outside the map: reads as zeros
      }
      return page * a.page_size + key % a.page_size;
    };
    auto copy = [&](const CUtensorMap* map, const Seg& s, int slot) {
      const uint32_t st = pos % kS, use = pos / kS;
      ++pos;
      ok = ok && (use == 0 || wait_w(kBarEmpty + st, (use - 1) & 1));
      if (!ok) return;
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, slot >= 0));
      if (lane == 0) mbar_arrive_expect_tx(bar(kBarFull + st), n * box_bytes);
      __syncwarp();
      filled = pos;
      const int half = lane % kHalves;
      if (slot >= 0)
        tma_3d(smem_addr(smem + L::kKV) + st * L::kTileBytes + half * L::kHalf + lane / kHalves * box_bytes, map,
               64 * half, s.h, slot, bar(kBarFull + st));
    };
    while (ok && walk.next(P, g)) {
      int slot = slot_of(g, g.j0);
      copy(&P.mapK, g, slot);
      for (int t = g.j0; ok && t < g.j1; ++t) {
        const int next = t + 1 < g.j1 ? slot_of(g, t + 1) : -1;
        if (t + 1 < g.j1) copy(&P.mapK, g, next);
        if (ok) copy(&P.mapV, g, slot);
        slot = next;
      }
    }
    // no copy of this CTA is in flight when it ends
    for (uint32_t k = filled > (uint32_t)kS ? filled - kS : 0; k < filled; ++k)
      mbar_wait(bar(kBarFull + k % kS), (k / kS) & 1, kWaitLimit);
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------------ query tiles
    if (elect_one()) {
      uint32_t pos = 0, filled = 0;
      bool ok = true;
      const uint32_t bytes = P.tokens * G * 128;
      while (ok && walk.next(P, g)) {
        const int n = g.rows > P.tokens ? 2 : 1;
        for (int k = 0; ok && k < n; ++k, ++pos) {
          const uint32_t st = pos & 1, use = pos >> 1;
          ok = use == 0 || wait(kBarQEmpty + st, (use - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kBarQFull + st), bytes * (D / 64));
          filled = pos + 1;
          for (int half = 0; half < D / 64; ++half)
            tma_3d(smem_addr(smem + L::kQ) + st * L::kTileBytes + half * L::kHalf, &P.mapQ, 64 * half, g.h * G,
                   g.t0 + k * P.tokens, bar(kBarQFull + st));
        }
      }
      for (uint32_t k = filled > 2 ? filled - 2 : 0; k < filled; ++k)
        mbar_wait(bar(kBarQFull + (k & 1)), (k >> 1) & 1, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ tensor cores
    if (elect_one()) {
      constexpr bool kBf16 = TYPE == QMM_BF16;
      constexpr uint32_t kIdS = tc::idesc_16_f32(128, kTile, kBf16, false);
      constexpr uint32_t kIdO = tc::idesc_16_f32(128, D, kBf16, true);
      const uint64_t dq = tc::smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_addr(smem + L::kKV), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(smem + L::kKV), L::kHalf, 1024);
      uint32_t pos = 0, qpos = 0;
      uint32_t done[2] = {0, 0};   // products p V issued for each lane
      bool ok = true;
      while (ok && walk.next(P, g)) {
        const int n = g.j1 - g.j0;
        const bool pair = g.rows > P.tokens;
        const int steps[2] = {pair ? n : (n + 1) / 2, pair ? n : n / 2};
        auto tile_of = [&](int l, int i) { return pair ? i : 2 * i + l; };
        auto scores = [&](int l, int i) {
          const uint32_t q = pair ? qpos + l : qpos;
          const int t = tile_of(l, i);
          const uint32_t kp = pos + pos_k(t), st = kp % kS;
          if (i == 0) ok = ok && wait(kBarQFull + (q & 1), (q >> 1) & 1);
          ok = ok && wait(kBarFull + st, (kp / kS) & 1);
          // the lane's p of the tile before sits where S goes: its product must have read it
          if (done[l] > 0) ok = ok && wait(kBarO + l, (done[l] - 1) & 1);
          if (!ok) return;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * L::kHalf + (k % 4) * 32;
            tc::mma_f16_ss(tmem + kTile * l, dq + (((q & 1) * L::kTileBytes + off) >> 4),
                           dk + ((st * L::kTileBytes + off) >> 4), kIdS, k > 0);
          }
          tc::commit(bar(kBarS + l));
          if (!pair || l == 1) tc::commit(bar(kBarEmpty + st));
          const bool last_q = i + 1 == steps[l] && (pair || t == n - 1);
          if (last_q) tc::commit(bar(kBarQEmpty + (q & 1)));
        };
        auto values = [&](int l, int i) {
          const int t = tile_of(l, i);
          const uint32_t vp = pos + pos_v(t, n), st = vp % kS;
          ok = ok && wait(kBarFull + st, (vp / kS) & 1) && wait(kBarP + l, done[l] & 1);
          if (!ok) return;
          tc::fence_after_sync();
          const int keys = min(kTile, g.keys - (g.j0 + t) * kTile);
          for (int k = 0; k * 16 < keys; ++k)
            tc::mma_f16_ts(tmem + 2 * kTile + kTile * l, tmem + kTile * l + 8 * k,
                           dv + ((st * L::kTileBytes + k * 2048) >> 4), kIdO, i > 0 || k > 0);
          tc::commit(bar(kBarO + l));
          ++done[l];
          if (!pair || l == 1) tc::commit(bar(kBarEmpty + st));
        };
        for (int l = 0; l < 2; ++l)
          if (ok && steps[l] > 0) scores(l, 0);
        for (int i = 0; ok && i < steps[0]; ++i)
          for (int l = 0; l < 2; ++l) {
            if (ok && i < steps[l]) values(l, i);
            if (ok && i + 1 < steps[l]) scores(l, i + 1);
          }
        pos += 2 * n;
        qpos += pair ? 2 : 1;
      }
      // no tensor-core operation of this CTA is in flight when it ends
      tc::commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax, one thread a row
    const int l = warp / kLaneWarps;                 // this warp's lane of flash attention
    const int row = (warp % kLaneWarps) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp % kLaneWarps) << 21;   // first TMEM lane << 16
    const uint32_t tS = tmem + lanes + kTile * l, tO = tmem + lanes + 2 * kTile;
    const float c = a.scale * kLog2e;
    float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
    uint32_t pos = 0, seen = 0, joins = 0, segs = 0;
    bool ok = true;
    while (ok && walk.next(P, g)) {
      const int n = g.j1 - g.j0;
      const bool pair = g.rows > P.tokens;
      const int steps = pair ? n : (n + 1 - l) / 2;
      const int tok0 = pair ? l * P.tokens : 0;                   // the lane's rows of the block
      const int live = min(P.tokens, g.rows - tok0) * G;          // rows of the tile in use
      const int tok = tok0 + row / G;
      const int sees = g.own ? clampi(g.first_keys + tok, 0, g.keys) : g.keys;
      const int clean_from = g.own ? clampi(g.first_keys + tok0, 0, g.keys) : g.keys;   // keys that not every row sees
      const bool idle = (warp % kLaneWarps) * 32 >= live;
      ++segs;
      float top = -INFINITY, sum = 0.0f;
      for (int i = 0; i < steps; ++i) {
        const int t = g.j0 + (pair ? i : 2 * i + l);
        ok = ok && wait_w(kBarS + l, seen & 1);
        if (!ok) break;
        ++seen;
        tc::fence_after_sync();
        const int base = t * kTile;
        if (!idle) {
          uint32_t s[128];
          tc::ld_wait_x128(tS, s);
          const int vis = sees - base;
          if (__any_sync(0xffffffffu, vis < kTile)) {
#pragma unroll
            for (int k = 0; k < kTile; ++k)
              if (k >= vis) s[k] = 0xFF800000u;   // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kTile; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(s[k]));
          const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const bool grew = now > top + kGrow || (top == -INFINITY && now > -INFINITY);
          if (i > 0 && __any_sync(0xffffffffu, grew)) {
            const float keep = grew ? exp2_fast(top - now) : 1.0f;
            sum *= keep;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32];
              tc::ld_wait_x32(tO + kTile * l + k, o);
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * keep);
              tc::st_x32(tO + kTile * l + k, o);
            }
          }
          if (grew) top = now;
          const float off = top == -INFINITY ? 0.0f : -top;
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < kTile; k += 2) {
            const float p0 = exp2_fast(__fmaf_rn(__uint_as_float(s[k]), c, off));
            const float p1 = exp2_fast(__fmaf_rn(__uint_as_float(s[k + 1]), c, off));
            part[k & 3] += p0;
            part[(k & 3) + 1] += p1;
            s[k / 2] = pack2<TYPE>(p0, p1);
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
          tc::st_x32(tS, s);
          tc::st_x32(tS + 32, s + 32);
          tc::wait_st();
        }
        // value rows that a weight of 0 must not meet
        const int upto = min(g.keys, base + kTile) - base;
        if (clean_from < base + kTile && (upto < kTile || g.own)) {
          const uint32_t vp = pos + pos_v(t - g.j0, n), st = vp % kS;
          ok = wait_w(kBarFull + st, (vp / kS) & 1);
          if (!ok) break;
          uint8_t* V = smem + L::kKV + st * L::kTileBytes;
          const int from = max(0, clean_from - base), end = (upto + 15) & ~15;
          for (int v = (warp % kLaneWarps) * 32 + lane; v < (end - from) * (D / 8); v += 32 * kLaneWarps) {
            const int r = from + v / (D / 8), piece = v % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(V + (piece / 8) * L::kHalf + r * 128 + (piece % 8) * 16);
            if (r >= upto) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              uint4 x = *at;
              if (odd_pair<TYPE>(x.x) || odd_pair<TYPE>(x.y) || odd_pair<TYPE>(x.z) || odd_pair<TYPE>(x.w)) {
                *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) = segs;
                __threadfence_block();
                x.x = without_odd<TYPE>(x.x);
                x.y = without_odd<TYPE>(x.y);
                x.z = without_odd<TYPE>(x.z);
                x.w = without_odd<TYPE>(x.w);
                *at = x;
              }
            }
          }
          fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + l));
      }
      pos += 2 * n;
      if (!ok) break;

      // ---- the segment's sums to the workspace
      if (steps > 0) ok = wait_w(kBarO + l, (seen - 1) & 1);
      if (!pair) {   // the other lane's state of the same rows
        stats[l * kTile + row] = make_float2(top, steps > 0 ? sum : -1.0f);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarJoin));
        ok = ok && wait_w(kBarJoin, joins++ & 1);
      }
      if (!ok) break;
      tc::fence_after_sync();
      const int64_t head = (int64_t)g.h * G + row % G;
      const bool mine = row < live;
      const bool inside = g.j0 > 0;   // not the first segment of its group: the CTA's own record
      int64_t rec = inside ? (int64_t)blockIdx.x * 2 * kTile + (pair ? l * kTile : 0) + row
                           : ((int64_t)(g.own ? a.T : 0) + g.t0 + tok) * a.Hq + head;
      float* out = (inside ? P.o_cta : P.o_rows) + rec * D;
      RowStat* stat = (inside ? P.s_cta : P.s_rows) + rec;
      const uint32_t odd = *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) == segs;
      if (pair) {
        if (!idle) {
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            tc::ld_wait_x32(tO + kTile * l + k, o);
            if (mine)
#pragma unroll
              for (int q = 0; q < 32; q += 8) store8(out + k + q, o + q);
          }
          if (mine) *stat = RowStat{top, sum, odd, 0u};
        }
      } else {
        const float2 s0 = stats[row], s1 = stats[kTile + row];
        const bool two = s1.y >= 0.0f || s1.y != s1.y;   // lane 1 had key tiles
        const float best = two ? fmaxf(s0.x, s1.x) : s0.x;
        const float f0 = s0.x == -INFINITY && s0.y == 0.0f ? 0.0f : exp2_fast(s0.x - best);
        const float f1 = !two || (s1.x == -INFINITY && s1.y == 0.0f) ? 0.0f : exp2_fast(s1.x - best);
        if (!idle) {
#pragma unroll 1
          for (int k = l * (D / 2); k < (l + 1) * (D / 2); k += 32) {   // half of O for each lane's warps
            uint32_t o[32];
            tc::ld_wait_x32(tO + k, o);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f0);
            if (two) {
              uint32_t o1[32];
              tc::ld_wait_x32(tO + kTile + k, o1);
#pragma unroll
              for (int q = 0; q < 32; ++q)
                o[q] = __float_as_uint(__fmaf_rn(__uint_as_float(o1[q]), f1, __uint_as_float(o[q])));
            }
            if (mine)
#pragma unroll
              for (int q = 0; q < 32; q += 8) store8(out + k + q, o + q);
          }
          if (mine && l == 0) *stat = RowStat{best, two ? __fmaf_rn(s1.y, f1, s0.y * f0) : s0.y * f0, odd, 0u};
        }
        // both lanes have read both sums before either lane's next product writes one
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarJoin));
        ok = wait_w(kBarJoin, joins++ & 1);
        tc::fence_after_sync();
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------------------
// Joins a row's segments: one warp per (row, head).  The segments of a group are the one that begins
// it (in the row's own record) and those of the CTAs whose piece begins inside it.
constexpr int kCombineWarps = 8;

template <int D, int TYPE>
__global__ void __launch_bounds__(32 * kCombineWarps) attn_combine_kernel(const __grid_constant__ Params P) {
  constexpr int kV = D / 32;
  const qmm_attn_args& a = P.a;
  __shared__ int stream;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int head = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
  if (threadIdx.x == 0) stream = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const Stream s = stream_of(a, b);
    if (t >= s.t0 && t < s.t0 + s.m) stream = b;   // one stream, if the starts do not decrease
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  if (head >= a.Hq) return;
  const int b = stream, G = a.Hq / a.Hk, block = 2 * P.tokens, h = head / G;
  const int64_t W = P.plan[0], C = P.plan[1];
  float o[kV] = {}, top = -INFINITY, sum = 0.0f;
  uint32_t odd = 0;

  auto add = [&](const float* rec_o, const RowStat& r) {
    if (r.top == -INFINITY && r.sum == 0.0f) return;   // the row saw none of the segment's keys
    const float best = fmaxf(top, r.top);
    const float f0 = top == -INFINITY && sum == 0.0f ? 0.0f : exp2_fast(top - best), f1 = exp2_fast(r.top - best);
    float x[kV];
    if constexpr (kV == 4) {
      const float4 v = *reinterpret_cast<const float4*>(rec_o + 4 * lane);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(rec_o + 2 * lane);
      x[0] = v.x; x[1] = v.y;
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] = __fmaf_rn(x[k], f1, o[k] * f0);
    sum = __fmaf_rn(r.sum, f1, sum * f0);
    top = best;
  };
  // the segments of the group whose first tile is `first` in the list and that has `tiles` tiles
  auto group = [&](int own, int64_t first, int tiles, int tok) {
    if (tiles == 0) return;
    const int64_t rec = ((int64_t)(own ? a.T : 0) + t) * a.Hq + head;
    const RowStat r = P.s_rows[rec];
    odd |= r.odd;
    add(P.o_rows + rec * D, r);
    const int row = (tok < P.tokens ? tok * G : kTile + (tok - P.tokens) * G) + head % G;
    for (int64_t cta = ((first + 1) * C + W - 1) / W; cta < C && cta * W / C < first + tiles; ++cta) {
      const int64_t at = cta * 2 * kTile + row;
      const RowStat q = P.s_cta[at];
      odd |= q.odd;
      add(P.o_cta + at * D, q);
    }
  };
  Stream s{};
  if (b >= 0) {
    s = stream_of(a, b);
    const int ptiles = tiles_of((int)a.prefix_len);
    group(0, ((int64_t)(t / block) * a.Hk + h) * ptiles, ptiles, t % block);
    const int rb = (t - s.t0) / block;
    int64_t first = P.plan[2 + b];
    for (int k = 0; k < rb; ++k) first += (int64_t)a.Hk * tiles_of(keys_of(s, k, block));
    const int tiles = tiles_of(keys_of(s, rb, block));
    group(1, first + (int64_t)h * tiles, tiles, (t - s.t0) % block);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = sum == 0.0f ? 0.0f : o[k] * inv;
  if (odd) {
    // infinities and NaN among the keys that only some rows of the block see: their sum
    float extra[kV] = {};
    const int sees = clampi(s.len - s.m + t - s.t0 + 1, 0, s.len);
    for (int j = max(0, s.len - s.m); j < sees; ++j) {
      const int page = a.pages[b * a.pages_per_stream + j / a.page_size];
      if (page < 0 || page >= a.n_slots / a.page_size) continue;
      const int64_t at = (((int64_t)page * a.page_size + j % a.page_size) * a.Hk + h) * D + kV * lane;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const uint16_t raw = static_cast<const uint16_t*>(a.V_cache)[at + k];
        const float v = TYPE == QMM_BF16 ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw));
        if (!(fabsf(v) < INFINITY)) extra[k] += v;
      }
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] += extra[k];
  }
  uint32_t w[kV / 2];
#pragma unroll
  for (int k = 0; k < kV / 2; ++k) w[k] = pack2<TYPE>(o[2 * k], o[2 * k + 1]);
  uint16_t* out = static_cast<uint16_t*>(a.O) + (int64_t)t * a.ldo + (int64_t)head * D + kV * lane;
  if constexpr (kV == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(out) = w[0];
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + head] = sum == 0.0f ? -INFINITY : __fmaf_rn(top, kLn2, logf(sum));
}

// ------------------------------------------------------------------------------------------

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

struct Space {
  size_t o_rows, s_rows, o_cta, s_cta, plan, total;
  explicit Space(const qmm_attn_args& a) {
    const size_t rows = 2 * (size_t)a.T * a.Hq, cta = (size_t)kMaxCtas * 2 * kTile;
    o_rows = 0;
    o_cta = o_rows + up(rows * a.D * sizeof(float));
    s_rows = o_cta + up(cta * a.D * sizeof(float));
    s_cta = s_rows + up(rows * sizeof(RowStat));
    plan = s_cta + up(cta * sizeof(RowStat));
    total = plan + up((2 + (size_t)a.B) * sizeof(int64_t)) + 256;   // the base may be 16-byte aligned only
  }
};

// A T x H x D (or slots x H x D) tensor of 16-bit values with `ld` values between its outer rows; boxes
// of 64 values, `heads` heads and `rows` rows, 128-byte swizzle.
bool tensor_map(CUtensorMap* m, const void* p, int D, int H, int64_t n, int64_t ld, int heads, int rows, int type) {
  const auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, type == QMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int TYPE>
cudaError_t set_smem_attr() {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(attn_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int D, int TYPE>
cudaError_t launch(const qmm_attn_args& a, void* workspace, cudaStream_t stream) {
  const int G = a.Hq / a.Hk;
  Params P;
  P.a = a;
  P.tokens = kTile / G;
  const Space sp(a);
  uint8_t* ws = reinterpret_cast<uint8_t*>(up(reinterpret_cast<uintptr_t>(workspace)));
  P.o_rows = reinterpret_cast<float*>(ws + sp.o_rows);
  P.o_cta = reinterpret_cast<float*>(ws + sp.o_cta);
  P.s_rows = reinterpret_cast<RowStat*>(ws + sp.s_rows);
  P.s_cta = reinterpret_cast<RowStat*>(ws + sp.s_cta);
  P.plan = reinterpret_cast<int64_t*>(ws + sp.plan);
  get_wait_limit(&P.wait_polls, &P.wait_ns);
  const int per_box = a.page_size < kTile ? a.page_size : kTile;
  if (!tensor_map(&P.mapQ, a.Q, D, a.Hq, a.T, a.ldq, G, P.tokens, TYPE) ||
      !tensor_map(&P.mapK, a.K_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE) ||
      !tensor_map(&P.mapV, a.V_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_attr<D, TYPE>();
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms < 1) return cudaErrorNoDevice;
  attn_kernel<D, TYPE><<<sms < kMaxCtas ? sms : kMaxCtas, kThreads, Smem<D>::kTotal, stream>>>(P);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.T, (a.Hq + kCombineWarps - 1) / kCombineWarps);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, TYPE>, P);
}

}  // namespace

size_t attn_workspace_bytes(const qmm_attn_args& a) { return Space(a).total; }

cudaError_t launch_attn(const qmm_attn_args& a, void* workspace, cudaStream_t stream) {
  if (a.D == 64)
    return a.type == QMM_BF16 ? launch<64, QMM_BF16>(a, workspace, stream) : launch<64, QMM_F16>(a, workspace, stream);
  return a.type == QMM_BF16 ? launch<128, QMM_BF16>(a, workspace, stream) : launch<128, QMM_F16>(a, workspace, stream);
}

cudaError_t read_and_clear_attn_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
