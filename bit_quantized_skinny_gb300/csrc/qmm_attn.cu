// qmm_attn.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, both in pages of one cache (qmm_attn_shared).
//
// Work.  A group is a block of rows that see the same keys, with one key/value head: for the prefix
// the rows of all streams, for own keys the rows of one stream; the G query heads of a key/value
// head are rows of the same block, so a key is read once for all of them.  A row tile is 128 rows
// (128 / G tokens) and a block up to two tiles; a key tile is 64 keys.  The key tiles of all groups
// form one list, each group led by kLead units for what a segment costs besides its tiles, cut into
// equal pieces, one per CTA (one CTA an SM): every SM has the same work whatever the lengths, and the
// lengths stay on the device.  A piece holds one or several segments (runs of one group's key tiles).
// Each segment leaves its sums unnormalised in the workspace, with the running maximum and weight sum
// of each row, and attn_combine_kernel joins a row's segments in their order.
//
// One segment.  Two lanes of flash attention take turns on the tensor cores: with more than one row
// tile each lane has a row tile and both read every key tile; with one, the lanes take the key tiles
// in turn and are joined at the segment's end.  Per lane and key tile:
//     S = Q K^T              tcgen05, both operands in shared memory (TMA, 128-byte swizzle)
//     p = 2^(c S - m)        a thread per row, S from tensor memory, c = scale log2 e
//     O += p V               tcgen05, p (16 bits, rounded once) from tensor memory, V MN-major
// A softmax frees S as soon as it has it in registers, and p has two places of its own, so the scores of
// the next item are formed during the softmax of this one: 64 keys a tile make room for that in
// tensor memory (2 lanes x (64 + 2 x 32 + 128 columns)).  The lanes take items (key tiles) in turn
// across segments, and a warp each issues their products.
// m is the maximum when it was last moved: it moves, and O is rescaled, only when the row's maximum
// grew by more than 8 (2^8 in a 16-bit p costs no precision), so O stays in tensor memory.
//
// Keys that a row may not see are set to -inf by position, so their K may hold anything.  Their p
// is 0, but 0 * NaN is not: value rows behind the last key are zeroed in shared memory, and so are
// non-finite values among the keys that only some rows of the block see (a draft's last keys);
// attn_combine_kernel then adds those back, from the cache, to the rows that see them.
//
// Measured (heads of 128, bf16, 40 query and 8 key/value heads; graph replays, the SM clock sampled at 2070
// MHz): 4 streams of 8 rows over 32768 shared keys 42 us, the keys and values at 5.8 TB/s while they stream,
// the rest the start, the pieces' sums through memory and the combine launch.  64 streams of 16 rows over the
// same keys 560 to 565 us, 1.25 PFLOP/s; 580 in runs so long that the power cap takes the clock to 1995 MHz.
// Its products take 354 us of that by their own rates (a score product of 64 keys 48 clocks where its
// arithmetic takes 32, Q being read from shared memory for each; a value product 64); without any softmax the
// kernel takes 496 us, and what holds it between the two has not been found.  A prompt of 4096 rows over
// its 8192 own keys 446 us, 1.16 PFLOP/s.  One row 10.8 us: start, first copies, combine, nothing but latency.
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_device.cuh"
#include "q4k_device_once.h"
#include "q4k_formats.cuh"
#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"
#include "q4k_tcgen05.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kRows = 128;           // rows of a row tile
constexpr int kTile = 64;            // keys of a key tile
constexpr int kLead = 4;             // units of a group besides its key tiles (2, 3, 6: 10, 6, 2 % slower for 16 streams)
constexpr int kMaxCtas = 152;
constexpr int kLaneWarps = 4;
constexpr int kLoadWarp = 8, kMmaWarp = 9 /* and 10 */, kQWarp = 11;
constexpr int kFirstDequantWarp = 12, kDequantWarps = 4;   // of a 4-bit cache
constexpr uint32_t kTmemCols = 512;   // lane L: S at 64 L, p at 128 + 64 L and 160 + 64 L, O at 256 + 128 L
constexpr float kGrow = 8.0f;
constexpr float kLift = 7.0f;        // fp16 weights lie at 2^kLift: at most 2^(kLift + kGrow), and normal down to 2^(-14 - kLift)
constexpr int kFactorTiles = 8;      // (the roles are a few tiles apart)
constexpr uint32_t kWaitLimit = 1u << 17;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// One row's state beside its O: the maximum in units of log2, the weight sum, whether values were
// taken out of the block (nonzero), and, in the record of a group's first segment, the CTAs that hold
// the others: their number << 16 | the first of them.
struct RowStat {
  float top, sum;
  uint32_t odd, rest;
};

struct Params {
  qmm_attn_args a;
  CUtensorMap mapQ, mapK, mapV;
  float* o_rows;      // [2][T * Hq][D]: first segments, of the prefix and of own keys
  RowStat* s_rows;
  float* o_cta;       // [kMaxCtas][2 * kRows][D]: a CTA's first segment that begins inside a group
  RowStat* s_cta;
  int tokens;         // of a row tile
  int n_pages, page_shift;
  uint32_t wait_polls, wait_ns;
  float k_scale, v_scale;   // of a 4-bit cache's tensors
};

template <int D, bool FP4>
struct Smem {
  static constexpr int kHalf = kTile * 128;              // 64 keys of 64 values
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQHalf = kRows * 128;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kStages = FP4 && D == 128 ? 3 : 5;   // of keys, and of values
  static constexpr int kPackBytes = kTile * kv4::slot_bytes(D);   // a tile as the 4-bit cache holds it
  static constexpr int kPacks = 12;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kQBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kPack = kV + kStages * kTileBytes;
  static constexpr int kStats = kPack + (FP4 ? kPacks * kPackBytes : 0);   // (top, sum) of the two lanes' rows
  static constexpr int kFactors = kStats + 2 * kRows * 8;      // of the rows of the last kFactorTiles query tiles
  static constexpr int kMisc = kFactors + (FP4 ? kFactorTiles * kRows * 4 : 0);
  static constexpr int kTotal = kMisc + 1024;
};
static_assert(Smem<128, false>::kTotal <= 227 * 1024 && Smem<128, true>::kTotal <= 227 * 1024 &&
              Smem<64, false>::kTotal <= 227 * 1024 && Smem<64, true>::kTotal <= 227 * 1024, "shared memory");

// Barriers.  A wait tells a phase from the one after it only, so a barrier is waited on by threads that
// see all of its phases, or that know the phase before to be over and the one after not begun: a stage of keys or values has a full barrier for each set of users (lane
// 0, lane 1, both), and a query tile is waited for and released by both lanes whoever uses it.
enum : int {
  kBarFullK = 0 /* 5 users + stage */, kBarFullV = 15, kBarEmptyK = 30, kBarEmptyV = 35, kBarQFull = 40, kBarQEmpty = 42,
  kBarS = 44, kBarFree = 46, kBarP = 48 /* 2 lane + item % 2 */, kBarO = 52, kBarEnd = 56, kBarJoin = 58, kBarDrain = 59,
  kBars16 = 61,                                    // of a cache of 16-bit values
  kBarPackFull = 61, kBarPackEmpty = 73, kBars = 85   // and of a 4-bit cache's tiles
};

// Rows and own keys of a stream.
struct Stream {
  int t0, m, len;
};

struct Misc {
  uint64_t bars[kBars];
  int64_t w0, w1, per;   // this CTA's units, units of a CTA
  int64_t scan[16];
  int b, rb, h, rows;
  Stream s;           // stream b, if b >= 0
  int64_t unit;       // end of the CTA's units within that group
  uint32_t tmem;
  int abort;
  uint32_t odd[8];    // [s % 8]: s, if values were taken out in segment s (the lanes drift a few apart)
};
static_assert(sizeof(Misc) <= 1024, "misc");

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
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? tiles + kLead : 0; }

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
struct Walker {
  int64_t left;
  int b, rb, h, j;   // group, end of what is left of it in units (-1: all)
  Stream s;
  int block, rows;   // rows of a block, rows in streams

  __device__ __forceinline__ void start(const Params& P, const Misc& m) {
    left = m.w1 - m.w0;
    b = m.b; rb = m.rb; h = m.h; j = (int)m.unit;
    block = 2 * P.tokens;
    rows = m.rows;
    s = m.s;
  }
  __device__ __forceinline__ bool next(const Params& P, Seg& g) {
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
      const int units = units_of(tiles_of(g.keys)), end = j < 0 ? units : j;
      const int take = (int)min((int64_t)end, left);
      left -= take;
      g.j0 = max(0, end - take - kLead);
      g.j1 = end - kLead;
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

// The wait for a phase that has not completed yet (out of line: the roles' loops stay short).
__device__ __noinline__ bool wait_slowly(uint32_t bar, uint32_t parity, uint32_t polls, uint32_t ns,
                                         volatile int* abort_flag) {
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity, polls, ns)) return true;
  atomicOr(&g_status, kErrWaitTimeout);
  *abort_flag = 1;
  return false;
}

template <bool FP4>
constexpr int kThreads = (FP4 ? kFirstDequantWarp + kDequantWarps : kFirstDequantWarp) * 32;

// Bulk copy global -> shared with the default L2 policy (a prefix's tiles are read by several CTAs).
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// One product of two fp16 pairs.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D, int TYPE, bool FP4>
__global__ void __launch_bounds__(kThreads<FP4>, 1) attn_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<D, FP4>;
  constexpr int kThreads = q4k::kThreads<FP4>;
  constexpr int kProduct = FP4 ? QMM_F16 : TYPE;   // the type of the products' operands
  constexpr uint32_t kS = L::kStages;
  const qmm_attn_args& a = P.a;
  Misc& M = *reinterpret_cast<Misc*>(smem + L::kMisc);
  volatile int* abort_flag = &M.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_addr(M.bars);
  auto bar = [&](int k) { return bars + 8u * k; };
  const int G = a.Hq / a.Hk, block = 2 * P.tokens;

  // ---- barriers, tensor memory, and this CTA's piece of the list of key tiles
  constexpr int kMyBars = FP4 ? kBars : kBars16;
  if (threadIdx.x < kMyBars) {
    const int k = threadIdx.x;
    const bool two = (k >= kBarEmptyK && k < kBarQFull) || (k >= kBarQEmpty && k < kBarS);
    const bool by_warps = FP4 && (k < kBarEmptyK || k >= kBarPackEmpty);   // dequantised, and read by that
    mbar_init(bar(k), by_warps ? kDequantWarps : two ? 2 : (k >= kBarFree && k < kBarO) ? kLaneWarps
                      : k == kBarJoin ? 2 * kLaneWarps : 1);
    fence_barrier_init();
  } else if (threadIdx.x == kMyBars) {
    M.abort = 0;
    for (int k = 0; k < 8; ++k) M.odd[k] = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_addr(&M.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  if (!FP4 && threadIdx.x < 3)
    asm volatile("prefetch.tensormap [%0];" :: "l"(threadIdx.x == 0 ? &P.mapK : threadIdx.x == 1 ? &P.mapV : &P.mapQ)
                 : "memory");
  // Launched early (behind a launch that allows it), this grid reads what was written before it from
  // here on; the combine launch, which reads the lengths before its own wait, may start from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  {
    // the page tables towards L2 while the pieces are worked out: one 128-byte line a thread
    const int64_t line = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 32;
    const int64_t n_pre = (a.prefix_len + a.page_size - 1) >> P.page_shift, n_own = a.B * a.pages_per_stream;
    if (line < n_pre) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.prefix_pages + line));
    if (line < n_own) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.pages + line));
    constexpr int kPer = (QMM_ATTN_MAX_STREAMS + kThreads - 1) / kThreads;
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
          mine[q] += (int64_t)a.Hk * units_of(tiles_of(keys_of(str[q], rb, block)));
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
    const int punits = units_of(tiles_of((int)a.prefix_len));
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
        int rb = 0, h = 0, n = units_of(tiles_of(keys_of(str[q], 0, block)));
        while (at >= (int64_t)a.Hk * n) { at -= (int64_t)a.Hk * n; n = units_of(tiles_of(keys_of(str[q], ++rb, block))); }
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
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = M.tmem;

  // A bounded wait for a phase of a barrier; false: this wait, or another one, gave up.  (A suspended try
  // from the start: polls take issue slots from the softmax; 32 of them first cost 14 %.)
  auto wait = [&](int k, uint32_t parity) -> bool {
    if (mbar_wait(bar(k), parity, 1, P.wait_ns ? P.wait_ns : kSuspendNs)) return true;
    return wait_slowly(bar(k), parity, P.wait_polls ? P.wait_polls : kWaitLimit, P.wait_ns ? P.wait_ns : kSuspendNs,
                       abort_flag);
  };
  auto wait_w = [&](int k, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(k, parity)); };

  Walker walk;
  walk.start(P, M);
  Seg g;
  // Segment by segment, the order in which keys and values are copied and dequantised: K0, K1, V0, K2, V1, ...
  // tile(values, t) of each; false ends it.
  [[maybe_unused]] auto in_order = [&](int n, auto&& tile) -> bool {
    for (int u = 0; u <= n; ++u) {
      if (u < n && !tile(std::false_type{}, u)) return false;
      if (u > 0 && !tile(std::true_type{}, u - 1)) return false;
    }
    return true;
  };

  if (FP4 && warp == kLoadWarp) {
    // ------------------------------------------------------------------ keys and values in 4 bits
    // A tile is a run of codes and one of scales per page (or of 64 keys of a longer page): lane 2k copies the
    // codes of run k, lane 2k + 1 its scales.  Pages behind the last key are not read.
    const int per_run = min(a.page_size, kTile);
    const int my_key = lane / 2 * per_run, my_bytes = lane % 2 ? D / 16 : D / 2;   // a slot
    const uint32_t dst = lane % 2 ? kTile * (D / 2) + my_key * (D / 16) : my_key * (D / 2);
    uint32_t filled = 0;
    bool ok = true;
    auto from = [&](const Seg& s, int tile) -> int64_t {   // offset of this lane's run in the caches, or -1
      const int key = tile * kTile + my_key;
      if (my_key >= kTile || key >= s.keys) return -1;
      int page = s.pages[key >> P.page_shift];
      if (page < 0 || page >= P.n_pages) {
        atomicOr(&g_status, kErrIndex);
        page = 0;   // (the rows that see it have unspecified values)
      }
      return kv4::run_at(page, s.h, a.Hk, a.page_size, D) + (lane % 2 ? a.page_size * (D / 2) : 0) +
             (key & (a.page_size - 1)) * my_bytes;
    };
    auto copy = [&](const void* cache, int64_t at) -> bool {
      const uint32_t st = filled % L::kPacks, use = filled / L::kPacks;
      ok = ok && (use == 0 || wait_w(kBarPackEmpty + st, (use - 1) & 1));
      if (!ok) return false;
      const uint32_t runs = __popc(__ballot_sync(0xffffffffu, at >= 0)) / 2;
      if (lane == 0) mbar_arrive_expect_tx(bar(kBarPackFull + st), runs * per_run * kv4::slot_bytes(D));
      __syncwarp();
      ++filled;
      if (at >= 0)
        bulk_copy(smem_addr(smem) + L::kPack + st * L::kPackBytes + dst, static_cast<const uint8_t*>(cache) + at,
                  per_run * my_bytes, bar(kBarPackFull + st));
      return true;
    };
    while (ok && walk.next(P, g)) {
      const int n = g.j1 - g.j0;
      // of the tile whose values come next, of the one whose keys come last, of the two behind it
      int64_t v_at = -1, k_last = -1, k_at = from(g, g.j0), k_next = n > 1 ? from(g, g.j0 + 1) : -1;
      in_order(n, [&](auto values, int t) {
        if constexpr (decltype(values)::value) return copy(a.V_cache, t + 1 < n ? v_at : k_last);
        v_at = k_last;   // (the values of a tile come behind the keys of the next, but for the last tile's)
        k_last = k_at;
        k_at = k_next;
        k_next = t + 2 < n ? from(g, g.j0 + t + 2) : -1;
        return copy(a.K_cache, k_last);
      });
    }
    // no copy of this CTA is in flight when it ends
    for (uint32_t k = filled > L::kPacks ? filled - L::kPacks : 0; k < filled; ++k)
      mbar_wait(bar(kBarPackFull + k % L::kPacks), (k / L::kPacks) & 1, kWaitLimit);
  } else if (FP4 && warp == kQWarp) {
    // ------------------------------------------------------------------ query tiles in fp16
    // A row of D/8 lanes.  A bf16 row is multiplied by the power of two that takes its largest value to
    // [2^14, 2^15): exact for what is not 2^-31 of that; the softmax multiplies its scores by the inverse.
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kAhead = 4;
    const float c = a.scale * P.k_scale * kLog2e;
    float* factors = reinterpret_cast<float*>(smem + L::kFactors);
    uint32_t pos = 0;
    bool ok = true;
    while (ok && walk.next(P, g)) {
      const int n = g.rows > P.tokens ? 2 : 1;
      for (int k = 0; ok && k < n; ++k, ++pos) {
        const uint32_t st = pos & 1, use = pos >> 1;
        ok = use == 0 || wait_w(kBarQEmpty + st, (use - 1) & 1);
        if (!ok) break;
        const int live = min(P.tokens, g.rows - k * P.tokens) * G;
        uint8_t* tile = smem + L::kQ + st * L::kQBytes;
        for (int r0 = 0; r0 < live; r0 += kAtOnce * kAhead) {
          uint4 q[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * kAtOnce + lane / kLanes;
            q[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < live) {
              const int tok = (int)((uint32_t)r / (uint32_t)G);
              q[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.Q) +
                                                     (g.t0 + k * P.tokens + tok) * a.ldq +
                                                     (int64_t)(g.h * G + r - tok * G) * D + 8 * (lane % kLanes));
            }
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * kAtOnce + lane / kLanes;
            uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            int up = 127;   // exponent field of the row's power of two
            if constexpr (TYPE == QMM_BF16) {
              uint32_t top = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
#pragma unroll
              for (int off = kLanes / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
              up = top == 0 || top >= 0x7F80u ? 127 : min(254, 268 - (int)(top >> 7));
              const float f = __uint_as_float((uint32_t)up << 23);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<QMM_F16>(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
            }
            if (r < live) {
              const int d = lane % kLanes;   // 16 bytes of the row
              *reinterpret_cast<uint4*>(tile + (d / 8) * L::kQHalf + r * 128 + ((d % 8) ^ (r & 7)) * 16) =
                  make_uint4(w[0], w[1], w[2], w[3]);
              if (d == 0) factors[(pos % kFactorTiles) * kRows + r] = scalbnf(c, 127 - up);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull + st));
      }
    }
  } else if (FP4 && warp >= kFirstDequantWarp) {
    // ------------------------------------------------------------------ 4 bits to fp16
    // A thread takes a block of 16 values: a code times its scale is exact in fp16 (two and four
    // significant bits).  Rows of values behind the last key are zeroed, and so are NaN blocks among the keys that
    // only some rows of the block see (a draft's last keys); attn_combine_kernel adds those back.  A step is the
    // keys of a tile and the values of the one before: one round of waits, loads, fence and arrivals for both (by
    // themselves each took as long, and the four warps, one a scheduler, have nobody to cover for them).
    constexpr int kBlocks = D / kv4::kBlock, kUnits = kTile * kBlocks / (32 * kDequantWarps);
    const int me = (warp - kFirstDequantWarp) * 32 + lane;
    uint32_t taken = 0, filled_k = 0, filled_v = 0, items = 0, segs = 0;
    bool ok = true;
    // (a phase that is over is the rule: the suspended wait costs 200 clocks even then)
    auto soon = [&](int k, uint32_t parity) { if (!mbar_try(bar(k), parity)) ok = wait(k, parity) && ok; };
    struct Units {
      uint2 code[kUnits];
      uint32_t scale[kUnits];
    };
    auto load = [&](uint32_t pack, Units& x) {
      const uint8_t* src = smem + L::kPack + pack * L::kPackBytes;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int unit = u * 32 * kDequantWarps + me;
        x.code[u] = *reinterpret_cast<const uint2*>(src + unit * 8);
        x.scale[u] = src[kTile * (D / 2) + unit];
      }
    };
    auto store = [&](uint8_t* dst, const Units& x, auto&& drop) {   // drop(key of the tile, scale): zeros instead
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int unit = u * 32 * kDequantWarps + me, key = unit / kBlocks, b = unit % kBlocks;
        const bool zero = drop(key, x.scale[u]);
        const uint32_t s = zero ? 0u : e4m3x2_pair(x.scale[u] * 0x101u);
        uint32_t lo[4], hi[4];
        e2m1x8_pairs(x.code[u].x, lo);
        e2m1x8_pairs(x.code[u].y, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = mul2(lo[e], s);
          hi[e] = mul2(hi[e], s);
        }
        uint8_t* row = dst + (b / 4) * L::kHalf + key * 128;
        // (the halves of a key in turn: eight neighbouring threads write to eight different 16-byte columns)
        const int c0 = 2 * (b % 4), turn = b / 4 & 1;
        const uint4 first = turn ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
        const uint4 other = turn ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(row + ((c0 + turn) ^ (key & 7)) * 16) = first;
        *reinterpret_cast<uint4*>(row + ((c0 + 1 - turn) ^ (key & 7)) * 16) = other;
      }
    };
    while (ok && walk.next(P, g)) {
      const int n = g.j1 - g.j0;
      const bool pair = g.rows > P.tokens;
      const int clean_from = g.own ? clampi(g.first_keys, 0, g.keys) : g.keys;
      ++segs;
      for (int t = 0; ok && t <= n; ++t) {   // the keys of tile t, the values of tile t - 1
        const bool keys = t < n, values = t > 0;
        const uint32_t pk = taken % L::kPacks, pv = (taken + keys) % L::kPacks;
        const uint32_t sk = filled_k % kS, sv = filled_v % kS;
        if (keys) {
          soon(kBarPackFull + pk, (taken / L::kPacks) & 1);
          if (filled_k >= kS) soon(kBarEmptyK + sk, (filled_k / kS - 1) & 1);
        }
        if (values) {
          soon(kBarPackFull + pv, ((taken + keys) / L::kPacks) & 1);
          if (filled_v >= kS) soon(kBarEmptyV + sv, (filled_v / kS - 1) & 1);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        Units k, v;
        if (keys) load(pk, k);
        if (values) load(pv, v);
        if (keys) store(smem + L::kK + sk * L::kTileBytes, k, [](int, uint32_t) { return false; });
        if (values) {
          const int base = (g.j0 + t - 1) * kTile;
          bool odd = false;
          if (base + kTile <= clean_from) {
            store(smem + L::kV + sv * L::kTileBytes, v, [](int, uint32_t) { return false; });
          } else {
            store(smem + L::kV + sv * L::kTileBytes, v, [&](int key, uint32_t scale) {
              const bool behind = base + key >= g.keys, nan = (scale & 0x7Fu) == kv4::kScaleNaN && base + key >= clean_from;
              odd |= nan && !behind;
              return behind || nan;
            });
            if (odd) *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) = segs;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (keys) {
            mbar_arrive(bar(kBarFullK + kS * (pair ? 2 : (items + t) & 1) + sk));
            mbar_arrive(bar(kBarPackEmpty + pk));
          }
          if (values) {
            mbar_arrive(bar(kBarFullV + kS * (pair ? 2 : (items + t - 1) & 1) + sv));
            mbar_arrive(bar(kBarPackEmpty + pv));
          }
        }
        taken += (keys ? 1 : 0) + (values ? 1 : 0);
        filled_k += keys;
        filled_v += values;
      }
      items += pair ? 2 * n : n;
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ keys and values
    // A tile is one box per page (or 64 keys of a longer page) and half of 64 values; lane k copies
    // box k / halves of half k % halves.  Pages behind the last key are not read.
    constexpr int kHalves = D / 64;
    const int per_box = min(a.page_size, kTile);
    const uint32_t box_bytes = per_box * 128;
    const int my_key = lane / kHalves * per_box;          // of the tile; behind it for lanes without a box
    struct Ring {
      uint32_t filled = 0;    // stages ever filled
      uint32_t parity = 0;    // bit kS * users + stage: of the next phase of its full barrier
      uint32_t users = 0;     // 2 bits a stage: of its last copy
    } rk, rv;
    uint32_t items = 0;
    bool ok = true;
    auto slot_of = [&](const Seg& s, int tile) -> int {   // first slot of this lane's box
      const int key = tile * kTile + my_key;
      if (my_key >= kTile || key >= s.keys) return -1;
      const int page = s.pages[key >> P.page_shift];
      if (page < 0 || page >= P.n_pages) {
        atomicOr(&g_status, kErrIndex);
        return (int)a.n_slots;   // outside the map: reads as zeros
      }
      return (page << P.page_shift) + (key & (a.page_size - 1));
    };
    auto copy = [&](const CUtensorMap* map, const Seg& s, int slot, uint32_t users, Ring& r, int full, int empty, int base) {
      const uint32_t st = r.filled % kS, use = r.filled / kS;
      ok = ok && (use == 0 || wait_w(empty + st, (use - 1) & 1));
      if (!ok) return;
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, slot >= 0)), at = kS * users + st;
      if (lane == 0) mbar_arrive_expect_tx(bar(full + at), n * box_bytes);
      __syncwarp();
      ++r.filled;
      r.parity ^= 1u << at;
      r.users = (r.users & ~(3u << 2 * st)) | users << 2 * st;
      const int half = lane % kHalves;
      if (slot >= 0)
        tma_3d(smem_addr(smem) + base + st * L::kTileBytes + half * L::kHalf + my_key * 128, map, 64 * half, s.h, slot,
               bar(full + at));
    };
    while (ok && walk.next(P, g)) {
      // K0, K1, K2, V0, K3, V1, ...: the order in which they are used
      const int n = g.j1 - g.j0;
      const bool pair = g.rows > P.tokens;
      auto users = [&](int t) -> uint32_t { return pair ? 2 : (items + t) & 1; };
      int slots[3] = {slot_of(g, g.j0), n > 1 ? slot_of(g, g.j0 + 1) : -1, n > 2 ? slot_of(g, g.j0 + 2) : -1};
      copy(&P.mapK, g, slots[0], users(0), rk, kBarFullK, kBarEmptyK, L::kK);
      if (n > 1) copy(&P.mapK, g, slots[1], users(1), rk, kBarFullK, kBarEmptyK, L::kK);
      for (int t = 0; ok && t < n; ++t) {
        const int next = t + 3 < n ? slot_of(g, g.j0 + t + 3) : -1;
        if (t + 2 < n) copy(&P.mapK, g, slots[2], users(t + 2), rk, kBarFullK, kBarEmptyK, L::kK);
        copy(&P.mapV, g, slots[0], users(t), rv, kBarFullV, kBarEmptyV, L::kV);
        slots[0] = slots[1];
        slots[1] = slots[2];
        slots[2] = next;
      }
      items += pair ? 2 * n : n;
    }
    // no copy of this CTA is in flight when it ends
    auto land = [&](const Ring& r, int full) {
      for (uint32_t st = 0; st < kS && st < r.filled; ++st) {
        const uint32_t at = kS * (r.users >> 2 * st & 3) + st;
        mbar_wait(bar(full + at), (r.parity >> at & 1) ^ 1, kWaitLimit);
      }
    };
    land(rk, kBarFullK);
    land(rv, kBarFullV);
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
            tma_3d(smem_addr(smem + L::kQ) + st * L::kQBytes + half * L::kQHalf, &P.mapQ, 64 * half, g.h * G,
                   g.t0 + k * P.tokens, bar(kBarQFull + st));
        }
      }
      for (uint32_t k = filled > 2 ? filled - 2 : 0; k < filled; ++k)
        mbar_wait(bar(kBarQFull + (k & 1)), (k >> 1) & 1, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ------------------------------------------------------------------ tensor cores
    // A warp for each lane, one elected thread of it: the lanes' waits and issue overlap each other's
    // products.  The scores of item j + 1 are issued ahead of the values of item j.  The empty barriers of keys and values count two arrivals, and the only user of a
    // tile makes both; those of query tiles count one of each lane.
    if (elect_one()) {
      constexpr bool kBf16 = kProduct == QMM_BF16;
      constexpr uint32_t kIdS = tc::idesc_16_f32(128, kTile, kBf16, false);
      constexpr uint32_t kIdO = tc::idesc_16_f32(128, D, kBf16, true);
      const uint64_t dq = tc::smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_addr(smem + L::kK), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(smem + L::kV), L::kHalf, 1024);
      const uint32_t l = warp - kMmaWarp;
      const uint32_t tS = tmem + kTile * l, tP = tmem + 2 * kTile + kTile * l, tO = tmem + 4 * kTile + kRows * l;
      const int barP = kBarP + 2 * l, barO = kBarO + 2 * l;
      struct Pass {
        Walker w;
        int left = 0;                  // the lane's items left of the segment
        bool pair = false, fresh = false;   // two row tiles; no item of the segment yet
        uint32_t users = 0;            // kS * users of the segment's tiles
        uint32_t step = 1;             // key tiles from item to item
        uint32_t st = 0, parity = 0;   // stage of the next item's key tile; of its full barriers' next phases
        uint32_t tiles = 0, items = 0, q = 0;   // key tiles, items and query tiles up to the segment's end
      } qk, pv;
      qk.w = pv.w = walk;
      bool ok = true;
      auto begin = [&](Pass& p) -> bool {   // the next segment that has items of this lane
        while (ok && p.w.next(P, g)) {
          const uint32_t n = g.j1 - g.j0;
          p.pair = g.rows > P.tokens;
          const uint32_t first = p.pair ? 0 : (p.items + l) & 1, at = p.tiles + first;
          p.step = p.pair ? 1 : 2;
          p.users = kS * (p.pair ? 2 : l);
          p.left = p.pair ? n : (n + 1 - first) / 2;
          p.st = at % kS;
          p.tiles += n;
          p.items += p.pair ? 2 * n : n;
          p.q += p.pair ? 2 : 1;
          p.fresh = true;
          if (p.left > 0) return true;
          if (&p == &qk) {   // no item: the segment's query tile passes by
            ok = wait(kBarQFull + ((p.q - 1) & 1), ((p.q - 1) >> 1) & 1);
            if (ok) mbar_arrive(bar(kBarQEmpty + ((p.q - 1) & 1)));
          }
        }
        return false;
      };
      auto full = [&](Pass& p, int k) -> bool {   // wait for the item's keys or values
        const uint32_t at = p.users + p.st;
        const bool yes = wait(k + at, p.parity >> at & 1);
        p.parity ^= 1u << at;
        return yes;
      };
      auto step = [&](Pass& p, int empty) {   // behind an item's products
        tc::commit(bar(empty + p.st));
        if (!p.pair) tc::commit(bar(empty + p.st));
        --p.left;
        p.fresh = false;
        p.st += p.step;
        if (p.st >= kS) p.st -= kS;
      };
      bool more = true;   // scores are left to issue
      auto scores = [&](int freed) {   // freed: the phase in which the softmax of the item before frees S, or -1
        if (qk.left == 0) more = more && begin(qk);
        if (!more || !ok) return;
        const uint32_t q = qk.q - (qk.pair ? 2 - l : 1), slot = q & 1;
        if (qk.fresh) {
          ok = wait(kBarQFull + ((qk.q - 1) & 1), ((qk.q - 1) >> 1) & 1);
          if (qk.pair) ok = ok && wait(kBarQFull + (qk.q & 1), ((qk.q - 2) >> 1) & 1);
        }
        ok = ok && full(qk, kBarFullK);
        if (freed >= 0) ok = ok && wait(kBarFree + l, freed);
        if (!ok) return;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 64; ++k)   // 64 values of the head: 4 MMAs, 32 bytes of each row further
          tc::mma_f16_ss_x4(tS, dq + ((slot * L::kQBytes + k * L::kQHalf) >> 4),
                            dk + ((qk.st * L::kTileBytes + k * L::kHalf) >> 4), 2, kIdS, k > 0);
        tc::commit(bar(kBarS + l));
        if (qk.left == 1) {
          tc::commit(bar(kBarQEmpty + slot));
          if (qk.pair) tc::commit(bar(kBarQEmpty + (slot ^ 1)));
        }
        step(qk, kBarEmptyK);
      };
      auto values = [&](auto b_, uint32_t parity) {
        constexpr int b = decltype(b_)::value;
        if (pv.left == 0 && !begin(pv)) return false;
        ok = full(pv, kBarFullV) && wait(barP + b, parity);
        if (!ok) return false;
        tc::fence_after_sync();
        tc::mma_f16_ts_x4(tO, tP + kTile / 2 * b, dv + ((pv.st * L::kTileBytes) >> 4), 128, kIdO,
                          !pv.fresh);   // 16 rows of V an MMA; the segment's first item begins O
        tc::commit(bar(barO + b));
        if (pv.left == 1) tc::commit(bar(kBarEnd + l));
        step(pv, kBarEmptyV);
        return true;
      };
      using S0 = std::integral_constant<int, 0>;
      using S1 = std::integral_constant<int, 1>;
      scores(-1);
      for (uint32_t r = 0; ok; ++r) {   // two items
        scores(0);
        if (!ok || !values(S0{}, r & 1)) break;
        scores(1);
        if (!ok || !values(S1{}, r & 1)) break;
      }
      // no tensor-core operation of this CTA is in flight when it ends
      tc::commit(bar(kBarDrain + l));
      mbar_wait(bar(kBarDrain + l), 0, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax, one thread a row
    const int l = warp / kLaneWarps;                 // this warp's lane of flash attention
    const int row = (warp % kLaneWarps) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp % kLaneWarps) << 21;   // first TMEM lane << 16
    const uint32_t tS = tmem + lanes + kTile * l, tP = tmem + lanes + 2 * kTile + kTile * l;
    const uint32_t tO = tmem + lanes + 4 * kTile;
    float c = a.scale * kLog2e;
    float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
    uint32_t parity = 0;   // of the next phases of the value stages' full barriers (single, both)
    uint32_t pos = 0, seen = 0, joins = 0, segs = 0, items = 0, ends = 0;
    [[maybe_unused]] uint32_t tiles_q = 0;   // query tiles before the segment's
    bool ok = true;
    while (ok && walk.next(P, g)) {
      const int n = g.j1 - g.j0;
      const bool pair = g.rows > P.tokens;
      const int first = pair ? 0 : (items + l) & 1;               // the lane's first key tile of the segment
      const bool has[2] = {pair || n > (int)(items & 1), pair || n > (int)((items + 1) & 1)};   // lanes with key tiles
      const int tok0 = pair ? l * P.tokens : 0;                   // the lane's rows of the block
      const int live = min(P.tokens, g.rows - tok0) * G;          // rows of the tile in use
      const int tok = tok0 + row / G;
      const int sees = g.own ? clampi(g.first_keys + tok, 0, g.keys) : g.keys;
      // Keys that not every row of the block sees.  The same ones for both lanes, also where each has a row
      // tile and they share the value tiles: whichever takes a value out first, the other one's product
      // follows its own pass over the same values, and what it may still write is what is there already.
      const int clean_from = g.own ? clampi(g.first_keys, 0, g.keys) : g.keys;
      const bool idle = (warp % kLaneWarps) * 32 >= live;
      ++segs;
      items += pair ? 2 * n : n;
      float top = -INFINITY, sum = 0.0f;
      uint32_t st = (pos + first) % kS;   // stage of the item's values
      for (int i = first; i < n; i += pair ? 1 : 2) {
        const int base = (g.j0 + i) * kTile;
        const int buf = seen & 1;   // which p of the lane
        const uint32_t at = pair ? kS + st : st;
        parity ^= 1u << at;
        ok = wait_w(kBarS + l, buf);   // (and with S the products of two items before, the last readers of this p)
        if constexpr (FP4) {   // (the product that made S waited for the query tile, and its rows' factors with it)
          if (ok && i == first)
            c = row < live ? reinterpret_cast<const float*>(smem + L::kFactors)[((tiles_q + (pair ? l : 0)) % kFactorTiles) * kRows + row]
                           : 0.0f;
        }
        // value rows that a weight of 0 must not meet
        const int upto = min(g.keys, base + kTile) - base;
        if (!FP4 && ok && clean_from < base + kTile && (upto < kTile || g.own)) {
          ok = wait_w(kBarFullV + kS * (pair ? 2 : l) + st, !(parity >> at & 1));
          if (!ok) break;
          uint8_t* V = smem + L::kV + st * L::kTileBytes;
          const int from = max(0, clean_from - base), end = (upto + 63) & ~63;
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
        if (!ok) break;
        tc::fence_after_sync();
        if (!idle) {
          uint32_t s[kTile];
          tc::ld_wait_x64(tS, s);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarFree + l));
          const int vis = sees - base;
          if (__any_sync(0xffffffffu, vis < kTile)) {
#pragma unroll
            for (int k = 0; k < kTile; ++k)
              if (k >= vis) s[k] = 0xFF800000u;   // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kTile; k += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1])));
          const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const bool grew = now > top + kGrow || (top == -INFINITY && now > -INFINITY);
          if (i > first && __any_sync(0xffffffffu, grew)) {
            // the item before is in O (the one before that is, with S)
            ok = wait_w(kBarO + 2 * l + (buf ^ 1), ((seen - 1) >> 1) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            const float keep = grew ? exp2_fast(top - now) : 1.0f;
            sum *= keep;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32];
              tc::ld_wait_x32(tO + kRows * l + k, o);
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * keep);
              tc::st_x32(tO + kRows * l + k, o);
            }
          }
          if (grew) top = now;
          const float off = top == -INFINITY ? 0.0f : FP4 ? kLift - top : -top;
          const uint64_t cc = f2pack(c, c), oo = f2pack(off, off);
          uint64_t part0 = 0, part1 = 0;   // sums of weights, two fp32 each
#pragma unroll
          for (int k = 0; k < kTile; k += 4) {
            const float2 x = f2unpack(fma2(f2pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, oo));
            const float2 y = f2unpack(fma2(f2pack(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), cc, oo));
            const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y), p2 = exp2_fast(y.x), p3 = exp2_fast(y.y);
            part0 = add2(part0, f2pack(p0, p1));
            part1 = add2(part1, f2pack(p2, p3));
            s[k / 2] = pack2<kProduct>(p0, p1);
            s[k / 2 + 1] = pack2<kProduct>(p2, p3);
          }
          tc::st_x32(tP + kTile / 2 * buf, s);
          const float2 u = f2unpack(part0), v = f2unpack(part1);
          sum += (u.x + u.y) + (v.x + v.y);
          tc::wait_st();
        } else if (lane == 0) {
          mbar_arrive(bar(kBarFree + l));
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + 2 * l + buf));
        ++seen;
        st += pair ? 1 : 2;
        if (st >= kS) st -= kS;
      }
      pos += n;   // value tiles before the next segment's
      tiles_q += pair ? 2 : 1;
      if (!ok) break;

      // ---- the segment's sums to the workspace
      const bool some = first < n;   // the lane had key tiles
      if (some) ok = wait_w(kBarEnd + l, ends++ & 1);
      if (!pair) {   // the other lane's state of the same rows
        stats[l * kRows + row] = make_float2(top, sum);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarJoin));
        ok = ok && wait_w(kBarJoin, joins++ & 1);
      }
      if (!ok) break;
      tc::fence_after_sync();
      const bool inside = g.j0 > 0;   // not the first segment of its group: the CTA's own record
      const uint32_t odd = *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) == segs;
      auto record = [&](int r) -> int64_t {   // of row r of the tile
        return inside ? (int64_t)blockIdx.x * 2 * kRows + (pair ? l * kRows : 0) + r
                      : ((int64_t)(g.own ? a.T : 0) + g.t0 + tok0 + r / G) * a.Hq + (int64_t)g.h * G + r % G;
      };
      float* out = inside ? P.o_cta : P.o_rows;
      if (row < live && (pair || l == 0)) {
        const uint32_t per = (uint32_t)min(M.per, (int64_t)0x7fffffff);
        const uint32_t others = g.rest > 0 ? ((uint32_t)g.rest + per - 1) / per : 0;
        RowStat st{top, sum, odd, others << 16 | (blockIdx.x + 1)};
        if (!pair) {
          const float2 s0 = stats[row], s1 = stats[kRows + row];
          st.top = fmaxf(s0.x, s1.x);
          st.sum = (!(s0.x == -INFINITY && s0.y == 0.0f) ? s0.y * exp2_fast(s0.x - st.top) : 0.0f) +
                   (!(s1.x == -INFINITY && s1.y == 0.0f) ? s1.y * exp2_fast(s1.x - st.top) : 0.0f);
        }
        if constexpr (FP4) st.top -= kLift;
        (inside ? P.s_cta : P.s_rows)[record(row)] = st;
      }
      // O: 16 rows x 32 columns at a time; the four threads of a row write 128 bytes of it.  A row's
      // values are kept in the order the load gives them (column_of).
      if (!idle) {
        const int c0 = pair ? 0 : l * (D / 2), c1 = pair ? D : c0 + D / 2;   // one tile: half of O for each lane's warps
#pragma unroll 1
        for (int hh = 0; hh < 2 && (warp % kLaneWarps) * 32 + 16 * hh < live; ++hh) {
          float f[2][2] = {{1.0f, 1.0f}, {1.0f, 1.0f}};   // [row][lane]
          float* dst[2];
          bool mine[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = (warp % kLaneWarps) * 32 + 16 * hh + 8 * k + lane / 4;
            mine[k] = r < live;
            dst[k] = out + record(r) * D + 8 * (lane & 3);
            if (!pair) {
              const float2 s0 = stats[r], s1 = stats[kRows + r];
              const float best = fmaxf(s0.x, s1.x);
              f[k][0] = s0.x == -INFINITY && s0.y == 0.0f ? 0.0f : exp2_fast(s0.x - best);
              f[k][1] = s1.x == -INFINITY && s1.y == 0.0f ? 0.0f : exp2_fast(s1.x - best);
            }
          }
#pragma unroll 1
          for (int k = c0; k < c1; k += 32) {
            const uint32_t at = tmem + lanes + ((uint32_t)hh << 20) + 4 * kTile + k;
            uint32_t o[16];
            if (pair) {
              tc::ld_wait_16x32(at + kRows * l, o);
            } else {
              if (has[0]) {
                tc::ld_wait_16x32(at, o);
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f[(q >> 1) & 1][0]);
              } else {
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = 0u;
              }
              if (has[1]) {
                uint32_t o1[16];
                tc::ld_wait_16x32(at + kRows, o1);
#pragma unroll
                for (int q = 0; q < 16; ++q)
                  o[q] = __float_as_uint(__fmaf_rn(__uint_as_float(o1[q]), f[(q >> 1) & 1][1], __uint_as_float(o[q])));
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t w[8] = {o[2 * q], o[2 * q + 1], o[2 * q + 4], o[2 * q + 5],
                                     o[2 * q + 8], o[2 * q + 9], o[2 * q + 12], o[2 * q + 13]};
              if (mine[q]) store8(dst[q] + k, w);
            }
          }
        }
      }
      if (!pair) {
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
// Joins a row's segments: SHARE warps per (row, head).  The segments of a group are the one that begins
// it (in the row's own record) and those of the CTAs whose piece begins inside it.
constexpr int kCombineWarps = 8;

// Column of the value at position p of a row's record: the epilogue keeps columns 8k + 2q, 8k + 2q + 1
// (k = 0..3) of each 32 together, as the 8 values of thread q of four.
__device__ __forceinline__ int column_of(int p) {
  return (p & ~31) + 8 * ((p & 7) >> 1) + 2 * ((p & 31) >> 3) + (p & 1);
}

template <int D, int TYPE, int SHARE, bool FP4>
__global__ void __launch_bounds__(32 * kCombineWarps) attn_combine_kernel(const __grid_constant__ Params P) {
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
  const int b = head < a.Hq ? stream : -1, G = a.Hq / a.Hk, block = 2 * P.tokens;
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

// ------------------------------------------------------------------------------------------

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

template <int D, int TYPE, bool FP4>
cudaError_t set_smem_attr() {
  static DeviceOnce once;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once.run(dev, cudaSuccess, [] {
    return cudaFuncSetAttribute(attn_kernel<D, TYPE, FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<D, FP4>::kTotal);
  });
}

template <int D, int TYPE, bool FP4>
cudaError_t launch(const qmm_attn_args& a, float k_scale, float v_scale, void* workspace, cudaStream_t stream) {
  const int G = a.Hq / a.Hk;
  Params P;
  P.a = a;
  P.k_scale = k_scale;
  P.v_scale = v_scale;
  P.tokens = kRows / G;
  P.n_pages = (int)(a.n_slots / a.page_size);
  P.page_shift = 31 - __builtin_clz((unsigned)a.page_size);
  const Space sp(a);
  uint8_t* ws = reinterpret_cast<uint8_t*>(up(reinterpret_cast<uintptr_t>(workspace)));
  P.o_rows = reinterpret_cast<float*>(ws + sp.o_rows);
  P.o_cta = reinterpret_cast<float*>(ws + sp.o_cta);
  P.s_rows = reinterpret_cast<RowStat*>(ws + sp.s_rows);
  P.s_cta = reinterpret_cast<RowStat*>(ws + sp.s_cta);
  get_wait_limit(&P.wait_polls, &P.wait_ns);
  const int per_box = a.page_size < kTile ? a.page_size : kTile;
  if (!FP4 && (!tensor_map(&P.mapQ, a.Q, D, a.Hq, a.T, a.ldq, G, P.tokens, TYPE) ||
      !tensor_map(&P.mapK, a.K_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE) ||
      !tensor_map(&P.mapV, a.V_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE)))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_attr<D, TYPE, FP4>();
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms < 1) return cudaErrorNoDevice;
  // Both launches may be scheduled while the one before them finishes (programmatic dependent launch);
  // each waits for it before it reads or writes memory.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms < kMaxCtas ? sms : kMaxCtas);
  cfg.blockDim = dim3(kThreads<FP4>);
  cfg.dynamicSmemBytes = Smem<D, FP4>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_kernel<D, TYPE, FP4>, P);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(a.T, (a.Hq + kCombineWarps - 1) / kCombineWarps);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.dynamicSmemBytes = 0;
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

template <bool FP4>
cudaError_t launch_any(const qmm_attn_args& a, float k_scale, float v_scale, void* workspace, cudaStream_t stream) {
  if (a.D == 64)
    return a.type == QMM_BF16 ? launch<64, QMM_BF16, FP4>(a, k_scale, v_scale, workspace, stream)
                              : launch<64, QMM_F16, FP4>(a, k_scale, v_scale, workspace, stream);
  return a.type == QMM_BF16 ? launch<128, QMM_BF16, FP4>(a, k_scale, v_scale, workspace, stream)
                            : launch<128, QMM_F16, FP4>(a, k_scale, v_scale, workspace, stream);
}

}  // namespace

size_t attn_workspace_bytes(const qmm_attn_args& a) { return Space(a).total; }

cudaError_t launch_attn(const qmm_attn_args& a, void* workspace, cudaStream_t stream) {
  return launch_any<false>(a, 1.0f, 1.0f, workspace, stream);
}

size_t attn_fp4_workspace_bytes(const qmm_attn_fp4_args& a) { return Space(a.base).total; }

cudaError_t launch_attn_fp4(const qmm_attn_fp4_args& a, void* workspace, cudaStream_t stream) {
  return launch_any<true>(a.base, a.k_scale, a.v_scale, workspace, stream);
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
