// qmm_attn_fp4.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, in pages of a 4-bit cache (qmm_attn_shared_fp4).
//
// Two forms, by the number of rows a key and of keys (expands() below): the kernel described here, and, with many rows or few
// keys, a launch that writes keys and values to the workspace in 16 bits and the 16-bit cache's kernel behind it.
//
// Work: equal pieces of the list of all key tiles, joined by a second launch (q4k_attn_parts.cuh).  A block is N / G
// tokens (at most N rows), a key tile 128 keys.
//
// A key is 72 bytes, and what an SM does for it is mostly to turn these into fp16 (a code times its scale
// is exact there).  So everything is laid out by the keys, with the rows as the narrow side of both products:
//     S^T = K Q^T        tcgen05, K (128 keys x D) from tensor memory, where four warps put it, a thread a key
//     p = 2^(c S + off)  a thread per key, S^T from tensor memory, c = scale k_scale log2 e over the row's power of two
//     O^T += V^T p^T     tcgen05, V and p^T (both MN-major) from shared memory; four more warps write V
//     l += p             the fp32 weights as they are before their rounding, added up over a warp's keys in the softmax
// so few rows cost little, the exponentials of a row are spread over 128 threads, and no 128-row tile of queries
// is read again for every tile.  Two groups of softmax warps have the key tiles in turn, with sums of their own that are
// joined at a segment's end: what a tile costs a group besides its rows (waits, votes, fences) is then paid once for all of them.
// off moves, and O^T is rescaled, only when a row's maximum grew by more than 8; weights are then at most 2^15, and
// fp16 holds those down to 2^-21 of the largest at full precision.  (l as a product of the rounded weights with ones took 201 us
// and 292 us in the calls below, but lse was off by up to 2^-12 where few keys have the weight, and by 2^-15 from the tensor cores' own
// rounding of long sums.)
//
// A role's work for a tile of 60 rows takes some 1300 to 1800 cycles (values to fp16 1400, keys 1300, the products' issue
// 1100 and 700, a group's softmax some 3400 for every other tile), a tile 2200: the roles wait for each other at most a third of
// the time, and each one's instructions wait for their own way to the warp more than for anything else (without the
// exponentials, without the conversions or with half the products a tile takes 4 to 10 % less, without the sums l 7 %).  Measured: 4 streams of 8 rows
// behind 131072 keys 213 us (three blocks of rows, 2.1 TB/s of packed keys in all); 24 streams of 19000 to 41000 keys of
// their own 287 us (2.9 TB/s).
//
// Keys that a row may not see are set to -inf by position, so their K may hold anything.  Value rows behind the last key
// are zeroed, and so are NaN blocks among the keys that only some rows of the block see (a draft's last keys);
// attn_combine_kernel adds those back, from the cache, to the rows that see them.
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_attn_parts.cuh"
#include "q4k_device.cuh"
#include "q4k_device_once.h"
#include "q4k_formats.cuh"
#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"
#include "q4k_tcgen05.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kTile = 128;           // keys of a key tile
// Units of a group besides its key tiles.  With 4, 6, 8, 10 and 12: 4 streams of 8 rows behind 131072 keys 259, 235, 213, 214 and 212 us,
// behind 60000 149, 130, 113, 115 and 115; 24 streams of 19000 to 41000 keys of their own 288, 288, 287, 288 and 289; 29 ragged ones
// behind 3001 28, 27, 29, 31 and 33.
constexpr int kLead = 8;
constexpr int kN = 64;               // rows of a block
constexpr int kHalf = kN / 2;        // rows up to which the products are half as wide
// warps: 0-3 and 4-7 softmax, 8 copies, 9 and 11 tensor cores, 10 queries, 12-15 keys and 16-19 values to fp16
constexpr int kLoadWarp = 8, kScoreWarp = 9, kQWarp = 10, kSumWarp = 11, kKeyWarp = 12, kValueWarp = 16;
constexpr int kThreads = 20 * 32, kGroupWarps = 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kKeyBufs = 3;          // of 64 values of a tile's keys, in tensor memory
constexpr int kScoreBufs = 4;        // two for each group
// Packed tiles in shared memory, of keys and of values in turn.  An even number, so that a role's next use of one follows its
// own last, and its wait takes no phase before that for it.
constexpr int kPacks = 8;
static_assert(kPacks % 2 == 0, "a pack is one role's");
// A row's weights of a tile are added up over four lanes by exchanges and over eight through shared memory, a run of rows behind
// the other for each of the eight (a step of 68 floats: no bank conflict either way).
constexpr int kPartsOf = 8, kPartStep = kN + 4;
constexpr int kFactorTiles = 8;      // (the softmax is a few query tiles behind)
constexpr float kGrow = 8.0f;
constexpr float kLift = 7.0f;        // log2 of the largest weight when off is set
constexpr uint32_t kWaitLimit = 1u << 17;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct Smem {
  static constexpr int kPackBytes = kTile * kv4::slot_bytes(D);
  static constexpr int kVHalf = kTile * 128;             // 128 keys of 64 values
  static constexpr int kVBytes = kTile * D * 2;
  static constexpr int kValueBufs = D == 128 ? 2 : 3;
  static constexpr int kQHalf = kN * 128;                // 64 values of N rows
  static constexpr int kQBytes = kN * D * 2;
  static constexpr int kPBytes = kTile * 128;            // 128 keys of 64 rows
  static constexpr int kV = 0;
  static constexpr int kQ = kV + kValueBufs * kVBytes;
  static constexpr int kP = kQ + 2 * kQBytes;
  static constexpr int kPack = kP + 2 * kPBytes;
  static constexpr int kFactors = kPack + kPacks * kPackBytes;   // of the rows of the last kFactorTiles query tiles
  static constexpr int kOff = kFactors + kFactorTiles * kN * 4;  // each softmax warp's copy of its group's rows' off
  static constexpr int kRed = kOff + 2 * kGroupWarps * kN * 4;   // the softmax warps' maxima of the rows
  static constexpr int kParts = kRed + 2 * kGroupWarps * kN * 4; // and the parts of a tile's sums
  static constexpr int kMisc = kParts + 2 * kGroupWarps * kPartsOf * kPartStep * 4;
  static constexpr int kTotal = kMisc + 1024;
};
static_assert(Smem<128>::kTotal <= 227 * 1024 && Smem<64>::kTotal <= 227 * 1024, "shared memory");

// Tensor memory: K at 0, then S^T (tile t's in t % kScoreBufs), and O^T of each group.
struct Tmem {
  static constexpr uint32_t kS = kKeyBufs * 32, kO = kS + kScoreBufs * kN;
  static_assert(kO + 2 * kN <= kTmemCols, "tensor memory");
};

// Barriers; a wait tells a phase from the one after it only, and every wait here is for the phase of a tile (or a segment)
// of whose successor on the same barrier the waiting role itself is a condition.
enum : int {
  kBarPackFull = 0, kBarPackEmpty = 10, kBarKeyFull = 20, kBarKeyEmpty = 24 /* 20 + and 24 + buffer */, kBarValueFull = 28, kBarValueEmpty = 31,
  kBarS = 34, kBarSFree = 38, kBarP = 42, kBarO = 44 /* products of a tile's values are done */, kBarQFull = 46,
  kBarQEmpty = 48, kBarOFree = 50, kBarDrain = 51 /* and 52 */, kBars = 53
};

struct Misc {
  uint64_t bars[kBars];
  Piece piece;
  uint32_t tmem;
  int abort;
  uint32_t odd[8];    // [s % 8]: s, if values were taken out in segment s
};
static_assert(sizeof(Misc) <= 1024, "misc");

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// One product of two fp16 pairs.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four chained MMAs with both operands in shared memory, their descriptors' steps apart (in 16-byte units).
__device__ __forceinline__ void mma_ss_x4(uint32_t d_taddr, uint64_t a, uint64_t a_step, uint64_t b, uint64_t b_step,
                                          uint32_t idesc, uint32_t accumulate_first) {
  asm volatile(
      "{\n .reg .pred p0, p1;\n setp.ne.b32 p0, %4, 0;\n setp.eq.b32 p1, %4, %4;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %6, %3, p1;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %8, %3, p1;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %9, %10, %3, p1;\n}"
      :: "r"(d_taddr), "l"(a), "l"(b), "r"(idesc), "r"(accumulate_first), "l"(a + a_step), "l"(b + b_step),
         "l"(a + 2 * a_step), "l"(b + 2 * b_step), "l"(a + 3 * a_step), "l"(b + 3 * b_step)
      : "memory");
}

// `threads` threads (a softmax group, or both) meet at barrier `id`: whether any of them says so.
__device__ __forceinline__ bool any_of(bool mine, int id, int threads) {
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(any) : "r"((uint32_t)mine), "r"(id), "r"(threads) : "memory");
  return any != 0;
}

// Four sums over four lanes each of sixteen values of every lane: lane l has those of values 4 (l / 8) and on, over the lanes that
// are l modulo 8.  (At each step a lane gives half of what it has to the one across and takes that one's other half.)
__device__ __forceinline__ float4 sum_over_four(float (&x)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8; n >= 4; n /= 2) {
    const bool upper = lane & 2 * n;
#pragma unroll
    for (int q = 0; q < n; ++q) {
      const float give = upper ? x[q] : x[q + n], keep = upper ? x[q + n] : x[q];
      x[q] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * n);
    }
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// The wait for a phase that has not completed yet (out of line: the roles' loops stay short).
__device__ __noinline__ bool wait_slowly(uint32_t bar, uint32_t parity, uint32_t polls, uint32_t ns,
                                         volatile int* abort_flag) {
  if (mbar_wait(bar, parity, 1, ns)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity, polls, ns)) return true;
  atomicOr(&g_status, kErrWaitTimeout);
  *abort_flag = 1;
  return false;
}

// The walk's next segment (out of line, and its state in memory: the roles' loops fit the instruction cache and
// their registers).
using Walk = Walker<kTile, kLead>;
__device__ __noinline__ bool next_of(Walk& walk, const Common& P, Seg& g) { return walk.next(P, g); }

// fp16 pairs of a block's eight bytes of codes and its scale (both halves), to h[AT] and on.
template <int AT, int N>
__device__ __forceinline__ void to_half(uint2 code, uint32_t s, uint32_t (&h)[N]) {
  uint32_t lo[4], hi[4];
  e2m1x8_pairs(code.x, lo);
  e2m1x8_pairs(code.y, hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[AT + e] = mul2(lo[e], s);
    h[AT + 4 + e] = mul2(hi[e], s);
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads, 1) attn_fp4_kernel(const __grid_constant__ Common P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<D>;
  using T = Tmem;
  constexpr uint32_t kVB = L::kValueBufs;
  const qmm_attn_args& a = P.a;
  Misc& M = *reinterpret_cast<Misc*>(smem + L::kMisc);
  volatile int* abort_flag = &M.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_addr(M.bars);
  auto bar = [&](int k) { return bars + 8u * k; };
  const int G = a.Hq / a.Hk;

  // ---- barriers, tensor memory, and this CTA's piece of the list of key tiles
  if (threadIdx.x < kBars) {
    const int k = threadIdx.x;
    const bool warps = (k >= kBarPackEmpty && k < kBarKeyEmpty) || (k >= kBarValueFull && k < kBarValueEmpty) ||
                       (k >= kBarSFree && k < kBarO);
    mbar_init(bar(k), k == kBarOFree ? 2 * kGroupWarps : warps ? kGroupWarps : 1);
    fence_barrier_init();
  } else if (threadIdx.x == kBars) {
    M.abort = 0;
    for (int k = 0; k < 8; ++k) M.odd[k] = 0;
  }
  if (warp == kScoreWarp) {
    tc::tmem_alloc(smem_addr(&M.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  // Launched early (behind a launch that allows it), this grid reads what was written before it from
  // here on; the combine launch, which reads the lengths before its own wait, may start from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  deal<kThreads, kTile, kLead>(P, M.piece, &g_status);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = M.tmem;
  // A bounded wait for a phase of a barrier; false: this wait, or another one, gave up.  (A phase that is over is the
  // rule, and a suspended wait takes 200 clocks to see it.)
  auto wait = [&](int k, uint32_t parity) -> bool {
    if (mbar_try(bar(k), parity)) return true;
    return wait_slowly(bar(k), parity, P.wait_polls ? P.wait_polls : kWaitLimit, P.wait_ns ? P.wait_ns : kSuspendNs,
                       abort_flag);
  };
  auto wait_w = [&](int k, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(k, parity)); };

  Walk walk;
  walk.start(P, M.piece);
  Seg g;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ packed tiles
    // A tile is a run of codes and one of scales per page (or of 128 keys of a longer page): lane 2k copies the
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
    auto copy = [&](const void* cache, int64_t at) {
      const uint32_t st = filled % kPacks, use = filled / kPacks;
      ok = ok && (use == 0 || wait_w(kBarPackEmpty + st, (use - 1) & 1));
      if (!ok) return;
      const uint32_t runs = __popc(__ballot_sync(0xffffffffu, at >= 0)) / 2;
      if (lane == 0) mbar_arrive_expect_tx(bar(kBarPackFull + st), runs * per_run * kv4::slot_bytes(D));
      __syncwarp();
      ++filled;
      if (at >= 0)
        bulk_copy(smem_addr(smem) + L::kPack + st * L::kPackBytes + dst, static_cast<const uint8_t*>(cache) + at,
                  per_run * my_bytes, bar(kBarPackFull + st));
    };
    while (ok && next_of(walk, P, g)) {
      int64_t at = from(g, g.j0), next = g.j0 + 1 < g.j1 ? from(g, g.j0 + 1) : -1;
      for (int j = g.j0; ok && j < g.j1; ++j) {
        const int64_t later = j + 2 < g.j1 ? from(g, j + 2) : -1;
        copy(a.K_cache, at);
        copy(a.V_cache, at);
        at = next;
        next = later;
      }
    }
    // no copy of this CTA is in flight when it ends
    for (uint32_t k = filled > kPacks ? filled - kPacks : 0; k < filled; ++k)
      mbar_wait(bar(kBarPackFull + k % kPacks), (k / kPacks) & 1, kWaitLimit);
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------------ query tiles in fp16
    // The rows come as they are, 16 bytes a lane, and bf16 ones are turned in place: a row is multiplied by the power of
    // two that takes its largest value to [2^14, 2^15), exact for what is not 2^-31 of that; the softmax
    // multiplies its scores by the inverse.  (All copies of a tile are in flight at once, and the code is short: it runs
    // once a segment, and instructions that come from afar cost more than they do.)
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    const float c = a.scale * P.k_scale * kLog2e;
    const int d = lane % kLanes;   // 16 bytes of a row
    uint32_t pos = 0;
    bool ok = true;
    for (; ok && next_of(walk, P, g); ++pos) {
      const uint32_t st = pos & 1, use = pos >> 1;
      ok = use == 0 || wait_w(kBarQEmpty + st, (use - 1) & 1);
      if (!ok) break;
      const int live = g.rows * G;
      const uint16_t* from = static_cast<const uint16_t*>(a.Q) + g.t0 * a.ldq + (int64_t)g.h * G * D + 8 * d;
      uint8_t* tile = smem + L::kQ + st * L::kQBytes + (d / 8) * L::kQHalf;
      float* factors = reinterpret_cast<float*>(smem + L::kFactors) + (pos % kFactorTiles) * kN;
      int tok = 0, head = lane / kLanes;   // of this lane's row
      while (head >= G) {
        head -= G;
        ++tok;
      }
#pragma unroll 1
      for (int r = lane / kLanes; r < live; r += kAtOnce) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :: "r"(smem_addr(tile) + r * 128 + ((d % 8) ^ (r & 7)) * 16), "l"(from + tok * a.ldq + head * D) : "memory");
        for (head += kAtOnce; head >= G; head -= G) ++tok;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll 1
      for (int r0 = 0; r0 < kN; r0 += kAtOnce) {
        const int r = r0 + lane / kLanes;
        int up = 127;   // exponent field of the row's power of two
        if (TYPE == QMM_BF16 && r0 < live) {
          uint4* at = reinterpret_cast<uint4*>(tile + r * 128 + ((d % 8) ^ (r & 7)) * 16);
          const uint4 q = *at;
          uint32_t w[4] = {q.x, q.y, q.z, q.w}, top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
#pragma unroll
          for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          up = top == 0 || top >= 0x7F80u ? 127 : min(254, 268 - (int)(top >> 7));
          const float f = __uint_as_float((uint32_t)up << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack2<QMM_F16>(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // (scores of rows behind the last one come to 0 or NaN: they never grow)
        if (d == 0) factors[r] = r < live ? scalbnf(c, 127 - up) : 0.0f;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQFull + st));
    }
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------------------ tensor cores, scores
    // (A warp for each product: issue waits for the tensor cores, and one warp's waits for its operands cost the other's
    // products nothing.)
    if (elect_one()) {
      constexpr uint32_t kIdBoth = tc::idesc_16_f32(128, kN, false, false), kIdHalf = tc::idesc_16_f32(128, kHalf, false, false);
      const uint64_t dq = tc::smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
      uint32_t tile = 0, unit = 0, segs = 0;
      bool ok = true;
      while (ok && next_of(walk, P, g)) {
        const uint32_t slot = segs & 1, id = g.rows * G > kHalf ? kIdBoth : kIdHalf;
        ok = wait(kBarQFull + slot, (segs >> 1) & 1);
        ++segs;
        for (int left = g.j1 - g.j0; ok && left > 0; --left, ++tile) {
          const uint32_t buf = tile % kScoreBufs;
          if (tile >= kScoreBufs) ok = wait(kBarSFree + buf, (tile / kScoreBufs - 1) & 1);
#pragma unroll 1
          for (uint32_t k = 0; ok && k < D / 64; ++k, ++unit) {   // 64 values of the head: 4 MMAs, 8 columns and 32 bytes of each row further
            const uint32_t kb = unit % kKeyBufs;
            ok = wait(kBarKeyFull + kb, (unit / kKeyBufs) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            tc::mma_f16_ts_x4(tmem + T::kS + kN * buf, tmem + 32 * kb, dq + ((slot * L::kQBytes + k * L::kQHalf) >> 4), 2, id, k > 0);
            tc::commit(bar(kBarKeyEmpty + kb));
          }
          if (!ok) break;
          tc::commit(bar(kBarS + buf));
          if (left == 1) tc::commit(bar(kBarQEmpty + slot));
        }
      }
      // no tensor-core operation of this CTA is in flight when it ends
      tc::commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == kSumWarp) {
    // ------------------------------------------------------------------ tensor cores, weighted sums
    if (elect_one()) {
      constexpr uint32_t kMnMajorA = 1u << 15, kMnMajorB = 1u << 16;   // V and p^T
      constexpr uint32_t kIdBoth = tc::idesc_16_f32(128, kN, false, false) | kMnMajorB;
      constexpr uint32_t kIdHalf = tc::idesc_16_f32(128, kHalf, false, false) | kMnMajorB;
      const uint64_t dp = tc::smem_desc_sw128(smem_addr(smem + L::kP), 16, 1024);
      // D = 64: O^T has 128 lanes all the same; the upper ones are products with other keys, and nobody reads them
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(smem + L::kV), D == 128 ? L::kVHalf : L::kVHalf / 2, 1024);
      uint32_t tile = 0, segs = 0;
      bool ok = true;
      while (ok && next_of(walk, P, g)) {
        const uint32_t id = g.rows * G > kHalf ? kIdBoth : kIdHalf;
        if (segs > 0) ok = wait(kBarOFree, (segs - 1) & 1);
        ++segs;
        const int n = g.j1 - g.j0;
        for (int i = 0; ok && i < n; ++i, ++tile) {
          const uint32_t vb = tile % kVB, buf = tile & 1;
          const bool fresh = i < 2;   // the first of its sums
          ok = wait(kBarValueFull + vb, (tile / kVB) & 1) && wait(kBarP + buf, (tile >> 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 2; ++k) {   // 64 keys: 4 MMAs of 16 rows of V and of p
            const uint32_t p = (buf * L::kPBytes + k * 64 * 128) >> 4;
            mma_ss_x4(tmem + T::kO + kN * buf, dv + ((vb * L::kVBytes + k * 64 * 128) >> 4), 128, dp + p, 128, id | kMnMajorA,
                      !fresh || k > 0);
          }
          tc::commit(bar(kBarO + buf));
          tc::commit(bar(kBarValueEmpty + vb));
        }
      }
      tc::commit(bar(kBarDrain + 1));
      mbar_wait(bar(kBarDrain + 1), 0, kWaitLimit);
    }
    __syncwarp();
  } else if (warp >= kKeyWarp && warp < kValueWarp) {
    // ------------------------------------------------------------------ keys to fp16, in tensor memory
    // A thread takes a key: D/2 bytes of codes, D/16 scales, D/2 columns of its lane.  (What lies behind the last key
    // is masked by position.)
    const int key = (warp - kKeyWarp) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp - kKeyWarp) << 21;   // first TMEM lane << 16
    uint32_t tile = 0, unit = 0;
    bool ok = true;
    while (ok && next_of(walk, P, g)) {
      const int j1 = g.j1;
      for (int j = g.j0; j < j1; ++j, ++tile) {
        const uint32_t from = 2 * tile % kPacks;
        ok = wait_w(kBarPackFull + from, (2 * tile / kPacks) & 1);
        const uint8_t* src = smem + L::kPack + from * L::kPackBytes;
#pragma unroll 1
        for (int half = 0; ok && half < D / 64; ++half, ++unit) {
          const uint32_t kb = unit % kKeyBufs;
          ok = unit < kKeyBufs || wait_w(kBarKeyEmpty + kb, (unit / kKeyBufs - 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {   // two blocks
            const uint4 code = *reinterpret_cast<const uint4*>(src + key * (D / 2) + 32 * half + 16 * q);
            const uint32_t two = *reinterpret_cast<const uint16_t*>(src + kTile * (D / 2) + key * (D / 16) + 4 * half + 2 * q);
            uint32_t h[16];
            to_half<0>(make_uint2(code.x, code.y), e4m3x2_pair(__byte_perm(two, 0, 0x00)), h);
            to_half<8>(make_uint2(code.z, code.w), e4m3x2_pair(__byte_perm(two, 0, 0x11)), h);
            tc::st_x16(tmem + lanes + 32 * kb + 16 * q, h);
          }
          tc::wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarKeyFull + kb));
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(kBarPackEmpty + from));
      }
    }
  } else if (warp >= kValueWarp) {
    // ------------------------------------------------------------------ values to fp16, in shared memory
    // A thread takes a block of 16 values at a time: of neighbouring threads four have the blocks of 64 values of one
    // key, so that eight write to eight different 16-byte columns.
    constexpr int kBlocks = D / kv4::kBlock, kUnits = kTile * kBlocks / (32 * kGroupWarps), kHalves = D / 64;
    const int me = (warp - kValueWarp) * 32 + lane;
    uint32_t tile = 0, segs = 0;
    bool ok = true;
    while (ok && next_of(walk, P, g)) {
      const int j1 = g.j1, keys = g.keys, clean_from = g.own ? clampi(g.first_keys, 0, keys) : keys;
      ++segs;
      for (int j = g.j0; j < j1; ++j, ++tile) {
        const uint32_t from = (2 * tile + 1) % kPacks, vb = tile % kVB;
        ok = wait(kBarPackFull + from, ((2 * tile + 1) / kPacks) & 1) &&
             (tile < kVB || wait(kBarValueEmpty + vb, (tile / kVB - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = smem + L::kPack + from * L::kPackBytes;
        uint8_t* dst = smem + L::kV + vb * L::kVBytes;
        const int base = j * kTile;
        // zeros behind the last key, and for the NaN blocks of keys that not every row sees
        const bool check = base + kTile > clean_from;
        bool odd = false;
#pragma unroll 1
        for (int u0 = 0; u0 < kUnits; u0 += 2) {
          uint2 code[2];
          uint32_t scale[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int u = u0 + e, key = u / kHalves * 32 + me / 4, block = u % kHalves * 4 + me % 4;
            code[e] = *reinterpret_cast<const uint2*>(src + key * (D / 2) + block * 8);
            scale[e] = src[kTile * (D / 2) + key * kBlocks + block];
            if (check) {
              const bool nan = (scale[e] & 0x7Fu) == kv4::kScaleNaN && base + key >= clean_from && base + key < keys;
              odd |= nan;
              if (nan || base + key >= keys) scale[e] = 0;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int u = u0 + e, key = u / kHalves * 32 + me / 4, c0 = 2 * (me % 4);
            uint32_t h[8];
            to_half<0>(code[e], e4m3x2_pair(scale[e] * 0x101u), h);
            uint8_t* row = dst + (u % kHalves) * L::kVHalf + key * 128;
            *reinterpret_cast<uint4*>(row + (c0 ^ (key & 7)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(row + ((c0 + 1) ^ (key & 7)) * 16) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        if (odd) *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) = segs;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarValueFull + vb));
          mbar_arrive(bar(kBarPackEmpty + from));
        }
      }
    }
  } else if (warp < 2 * kGroupWarps) {
    // ------------------------------------------------------------------ softmax, a thread per key
    const int grp = warp / kGroupWarps, wg = warp % kGroupWarps;
    const int mine = wg * 32 + lane;                  // key of the tile; value of O^T
    const uint32_t lanes = (uint32_t)wg << 21;        // first TMEM lane << 16
    float* off = reinterpret_cast<float*>(smem + L::kOff) + warp * kN;
    float* red = reinterpret_cast<float*>(smem + L::kRed) + grp * kGroupWarps * kN;
    float* parts = reinterpret_cast<float*>(smem + L::kParts) + warp * kPartsOf * kPartStep;
    auto any_here = [&](bool x) { return any_of(x, 1 + grp, 32 * kGroupWarps); };
    uint32_t tile = 0, segs = 0;
    bool ok = true;
    while (next_of(walk, P, g)) {
      const int rows = g.rows * G;
      const float* factors = reinterpret_cast<const float*>(smem + L::kFactors) + segs % kFactorTiles * kN;
      const int j1 = g.j1, n = g.j1 - g.j0, keys = g.keys, first_keys = g.first_keys;
      ++segs;
      off[lane] = off[kHalf + lane] = 0.0f;
      __syncwarp();
      float sum[2] = {0.0f, 0.0f};   // of the warp's weights of rows lane and kHalf + lane
      bool first = true, leave = false;   // leave: the whole group knows that a wait gave up
      for (int j = g.j0; j < j1; ++j, ++tile) {
        const uint32_t buf = tile & 1, phase = (tile >> 1) & 1, at = tile % kScoreBufs;
        if ((int)buf != grp) continue;
        const int key = j * kTile + mine;
        // the first row that sees this thread's key
        const int from = key >= keys ? kN : max(0, key - first_keys + 1) * G;
        const bool hidden = __any_sync(0xffffffffu, from > 0);
        ok = wait_w(kBarS + at, (tile / kScoreBufs) & 1) && ok;
        tc::fence_after_sync();
        if (tile >= 2) ok = wait_w(kBarO + buf, phase ^ 1) && ok;   // the last readers of this p
        // sixteen rows' scores in units of log2, plus off.  (The loops over them are not unrolled: five warps a scheduler
        // in as many loops are bound by the instructions' way to them before anything else.)
        auto scores = [&](int r, float (&x)[16]) {
          uint32_t s[16];
          tc::ld_wait_x16(tmem + lanes + T::kS + kN * at + r, s);
#pragma unroll
          for (int q = 0; q < 16; q += 4) {
            const float4 f = *reinterpret_cast<const float4*>(factors + r + q), o = *reinterpret_cast<const float4*>(off + r + q);
            const float2 u = f2unpack(fma2(f2pack(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), f2pack(f.x, f.y), f2pack(o.x, o.y)));
            const float2 v = f2unpack(fma2(f2pack(__uint_as_float(s[q + 2]), __uint_as_float(s[q + 3])), f2pack(f.z, f.w), f2pack(o.z, o.w)));
            x[q] = u.x;
            x[q + 1] = u.y;
            x[q + 2] = v.x;
            x[q + 3] = v.y;
          }
          if (hidden)
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (r + q < from) x[q] = -INFINITY;
        };
        uint8_t* p = smem + L::kP + buf * L::kPBytes + mine * 128;
        // the rows' weights to shared memory (those behind the last row do no harm); the largest exponent
        auto weights = [&]() -> float {
          float most = -INFINITY;
#pragma unroll 1
          for (int r = 0; r < rows; r += 16) {
            float x[16];
            scores(r, x);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[4];
#pragma unroll
              for (int q = 8 * h; q < 8 * h + 8; q += 2) {
                most = fmaxf(most, fmaxf(x[q], x[q + 1]));
                x[q] = exp2_fast(x[q]);
                x[q + 1] = exp2_fast(x[q + 1]);
                w[q / 2 - 4 * h] = pack2<QMM_F16>(x[q], x[q + 1]);
              }
              *reinterpret_cast<uint4*>(p + ((r / 8 + h) ^ (mine & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<float4*>(parts + lane % 8 * kPartStep + r + lane / 8 * 4) = sum_over_four(x);
          }
          return most;
        };
        for (bool set = first;; set = true) {   // twice, where off has to move before the weights hold
          if (set) {
            leave = any_here(!ok);
            if (leave) break;
            // the rows' maxima of this tile
#pragma unroll 1
            for (int r = 0; r < rows; r += 16) {
              float x[16], top = -INFINITY;
              scores(r, x);
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                const float v = x[q] == x[q] ? x[q] : -INFINITY;
                const uint32_t b = __float_as_uint(v), up = __reduce_max_sync(0xffffffffu, b & 0x80000000u ? ~b : b | 0x80000000u);
                if (lane == q) top = __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
              }
              if (lane < 16) red[wg * kN + r + lane] = top;
            }
            any_here(false);
            float keep[2] = {1.0f, 1.0f};   // of rows lane and kHalf + lane
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = kHalf * h + lane;
              if (r < rows) {
                const float top = fmaxf(fmaxf(red[r], red[kN + r]), fmaxf(red[2 * kN + r], red[3 * kN + r]));
                // a row that sees no key of the group's first tile sees none of its later ones
                const float was = off[r];
                const float now = top > -INFINITY && (first || top > kLift + kGrow) ? was - (top - kLift) : was;
                keep[h] = exp2_fast(now - was);
                off[r] = now;
                sum[h] *= keep[h];
              }
            }
            __syncwarp();
            if (!first) {   // O^T: the products of the group's tile before are in it
#pragma unroll 1
              for (int r0 = 0; r0 < rows; r0 += 8) {
                uint32_t o[8];
                tc::ld_wait_x8(tmem + lanes + T::kO + kN * grp + r0, o);
                const float of = r0 < kHalf ? keep[0] : keep[1];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                  o[r] = __float_as_uint(__uint_as_float(o[r]) * __shfl_sync(0xffffffffu, of, (r0 & (kHalf - 1)) + r));
                tc::st_x8(tmem + lanes + T::kO + kN * grp + r0, o);
              }
              tc::wait_st();
            }
          }
          const float most = weights();
          if (set || !any_here(most > kLift + kGrow || !ok)) break;
        }
        if (leave) break;
        first = false;
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarP + buf));
          mbar_arrive(bar(kBarSFree + at));
        }
        // (the parts were written ahead of the warp's last barrier, and are written again behind its next one)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (kHalf * h < rows) {
            const float* x = parts + kHalf * h + lane;
            float a[kPartsOf / 2];
#pragma unroll
            for (int q = 0; q < kPartsOf / 2; ++q) a[q] = x[2 * q * kPartStep] + x[(2 * q + 1) * kPartStep];
            sum[h] += (a[0] + a[1]) + (a[2] + a[3]);
          }
      }

      // ---- the segment's sums to the workspace
      // (the products of the group's last tile, and with them all before; of the other group's barrier this one could take a
      // phase for the one after it)
      const uint32_t last = tile - 1 - ((tile - 1 - grp) & 1);
      if (!leave && (n > 1 || last == tile - 1)) ok = wait_w(kBarO + grp, (last >> 1) & 1) && ok;
      red[wg * kN + lane] = sum[0];
      red[wg * kN + kHalf + lane] = sum[1];
      if (any_of(!ok || leave, 3, 64 * kGroupWarps)) break;
      tc::fence_after_sync();
      // Each group joins both groups' sums of half of the rows, from c0 on; lane r has row c0 + r: its sum, its exponent, what
      // the groups' sums count, and where its record lies.
      const int half = (rows + 15) / 16 * 8, c0 = grp * half, live = grp ? max(0, rows - half) : min(half, rows);
      const int row = min(c0 + lane, kN - 1);
      const uint32_t tO = tmem + lanes + T::kO + c0;
      auto sum_of = [&](int gr) -> float {
        const float* x = reinterpret_cast<const float*>(smem + L::kRed) + gr * kGroupWarps * kN + row;
        return (x[0] + x[kN]) + (x[2 * kN] + x[3 * kN]);
      };
      const float* offs = reinterpret_cast<const float*>(smem + L::kOff) + row;
      float f[2] = {0.0f, 0.0f}, all = 0.0f, top = -INFINITY;
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const bool has = n > 1 || (int)((tile - 1) & 1) == k;   // (a group without a tile has no sums)
        const float l = has ? sum_of(k) : 0.0f, t = -offs[k * kGroupWarps * kN];
        if (l != 0.0f) {   // (NaN counts)
          const float best = fmaxf(top, t), w = exp2_fast(t - best), was = exp2_fast(top - best);
          all = all * was + l * w;
          f[0] = k == 0 ? w : f[0] * was;
          f[1] = k == 0 ? 0.0f : w;
          top = best;
        }
      }
      const bool inside = g.j0 > 0;   // not the first segment of its group: the CTA's own record
      const int tok = (int)((uint32_t)row / (uint32_t)G);
      const int64_t record = inside ? (int64_t)blockIdx.x * 2 * kRows + row
                                    : ((int64_t)(g.own ? a.T : 0) + g.t0 + tok) * a.Hq + (int64_t)g.h * G + row - tok * G;
      if (wg == 0 && lane < live) {
        const uint32_t per = (uint32_t)min(M.piece.per, (int64_t)0x7fffffff);
        const uint32_t others = g.rest > 0 ? ((uint32_t)g.rest + per - 1) / per : 0;
        const uint32_t odd = *reinterpret_cast<volatile uint32_t*>(&M.odd[segs & 7]) == segs;
        (inside ? P.s_cta : P.s_rows)[record] = RowStat{top, all, odd, others << 16 | (blockIdx.x + 1)};
      }
      // O^T: this thread's value of every row, at the place where the combine launch looks for it (column_of)
      float* out = (inside ? P.o_cta : P.o_rows) + (mine & ~31) + 8 * (mine >> 1 & 3) + 2 * (mine >> 3 & 3) + (mine & 1);
#pragma unroll 1
      for (int r0 = 0; r0 < live; r0 += 8) {
        uint32_t o[8], o1[8];
        tc::ld_wait_x8(tO + r0, o);
        tc::ld_wait_x8(tO + kN + r0, o1);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int64_t at = __shfl_sync(0xffffffffu, record, r0 + r) * D;
          const float u = __shfl_sync(0xffffffffu, f[0], r0 + r), w = __shfl_sync(0xffffffffu, f[1], r0 + r);
          const float v = (u != 0.0f ? __uint_as_float(o[r]) * u : 0.0f) + (w != 0.0f ? __uint_as_float(o1[r]) * w : 0.0f);
          if (r0 + r < live && mine < D) out[at] = v;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOFree));
      any_of(false, 3, 64 * kGroupWarps);   // (off and red are written again behind this)
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kScoreWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D, int TYPE>
cudaError_t launch(const qmm_attn_fp4_args& f, void* workspace, cudaStream_t stream) {
  static DeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, cudaSuccess, [] {
    return cudaFuncSetAttribute(attn_fp4_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms < 1) return cudaErrorNoDevice;
  const int tokens = kN / (f.base.Hq / f.base.Hk);
  Common P;
  fill(P, f.base, tokens, tokens, workspace);
  P.k_scale = f.k_scale;
  P.v_scale = f.v_scale;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms < kMaxCtas ? sms : kMaxCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_fp4_kernel<D, TYPE>, P);
  if (e != cudaSuccess) return e;
  return launch_combine<D, TYPE, true>(P, sms, stream);
}

// ---- many rows a key, or few keys: keys and values to 16 bits once, and the 16-bit kernel

// The workspace behind the sums' one.
struct Expanded {
  int64_t n_pre, n_pages;   // pages of the prefix, and of all
  size_t ids, Q, factors, K, V, total;
  explicit Expanded(const qmm_attn_args& a) {
    n_pre = ((int64_t)a.prefix_len + a.page_size - 1) / a.page_size;
    n_pages = n_pre + (int64_t)a.B * a.pages_per_stream;
    const size_t rows = (size_t)a.T * a.Hq, values = (size_t)n_pages * a.page_size * a.Hk * a.D;
    ids = Space(a).total;
    Q = ids + up((size_t)n_pages * 4);
    factors = Q + up(a.type == QMM_BF16 ? rows * a.D * 2 : 0);
    K = factors + up(a.type == QMM_BF16 ? rows * 4 : 0);
    V = K + up(values * 2);
    total = V + up(values * 2) + 256;   // (all of it from a 256-byte boundary on)
  }
};

// A key costs the kernel above some 0.07 ns a head for each 64 rows that see it; to 16 bits (656 bytes read, written and read
// again, at HBM's rate) it costs 0.1 ns, and then 0.05 ns for each 128 rows in the 16-bit kernel.  So keys are expanded from
// kRowsExpanded rows a key on, on the average over the keys that the page lists have room for (the lengths are on the device),
// unless these are more than the workspace should hold.  Measured, 8 heads of 128 that 5 query heads share, 16 rows a stream
// behind 32768 keys: 160 rows a key 78 us either way; 320 rows 100 expanded, 124 not; 640 rows 128 and 213; 5120 rows
// (64 streams) 589 and 1547.  A prompt of 1000 rows over 8000 keys 153 and 381; 100 rows over them 40 and 65; 60 rows over
// 300 keys 18 and 26; 30 streams of 3 rows behind 30000 keys with 1000 of their own 142 and 174.
constexpr int64_t kRowsExpanded = 160;
constexpr int64_t kMostExpanded = int64_t(1) << 30;   // bytes
// Where all keys are few, the 16-bit kernel's shorter start is worth the launch ahead of it with any number of rows.  1 stream of 1
// row: 16 keys 11.4 us expanded, 14.8 not; 700 keys (2.9 MB) 15.9 and 16.4; 4000 (16 MB) 18.6 and 18.4; 8000 (33 MB) 23.8 and
// 19.5.  4 streams of 8 rows: 700 keys (11 MB) 18.2 and 23.5; 3000 (49 MB) 31.0 and 27.9.  29 ragged streams (18 MB) 23.9 and 29.4;
// 16 streams of 4 rows and 500 keys (33 MB) 27.7 and 26.4.
constexpr int64_t kFewExpanded = int64_t(24) << 20;   // bytes
double expanded_bytes(const qmm_attn_args& a) {
  return (a.prefix_len + (double)a.B * a.pages_per_stream * a.page_size) * a.Hk * a.D * 4;
}
bool expands(const qmm_attn_args& a) {
  const double own = (double)a.pages_per_stream * a.page_size, keys = a.prefix_len + a.B * own;
  const double rows = (double)a.T * (a.Hq / a.Hk) * (a.prefix_len + own);   // times keys
  const double bytes = expanded_bytes(a);
  return keys > 0 && (bytes <= (double)kFewExpanded || (rows >= kRowsExpanded * keys && bytes <= (double)kMostExpanded));
}

struct ExpandParams {
  qmm_attn_args a;
  float c;               // scale k_scale log2 e
  int64_t n_pre, page_ctas;
  int chunks, blocks;    // CTAs of a page's head, blocks of one
  int32_t* ids;
  __half *Q, *K, *V;
  float* factors;
};
// A CTA has a block of 16 values of a page's head a thread, keys and values, or two where keys are many.  64 streams of 16 rows
// behind 8000 keys 250 us with two, one, four and eight 261, 248, 246; 100 rows over 8000 keys 40.9, 39.9, 44.8, 49.0; 1 row over
// 2000 19.9 and with one 17.3.
constexpr int kExpandThreads = 128;
// Scores stay below 2^40, so a factor this small makes all weights 1, as a smaller one would; but 0 times the -inf of a masked
// key would be NaN.
constexpr float kLeastFactor = 0x1p-120f;

// A CTA for some blocks of 16 values of a page's head, keys and values, a thread a block at a time; behind these, for bf16, a warp for each row and head of
// the queries.
template <int D, int TYPE>
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ ExpandParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const qmm_attn_args& a = P.a;
  if (blockIdx.x >= P.page_ctas) {
    constexpr int kV = D / 32;
    const int64_t row = (int64_t)(blockIdx.x - P.page_ctas) * (kExpandThreads / 32) + (threadIdx.x >> 5);
    if (row >= (int64_t)a.T * a.Hq) return;
    const int lane = threadIdx.x & 31;
    const int64_t t = row / a.Hq;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.Q) + t * a.ldq + (row - t * a.Hq) * D) + lane * (kV / 2);
    uint32_t w[kV / 2], top = 0;
#pragma unroll
    for (int k = 0; k < kV / 2; ++k) {
      w[k] = q[k];
      top = max(top, max(w[k] & 0x7FFFu, w[k] >> 16 & 0x7FFFu));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // as in the kernel above: the power of two that takes the row's largest value to [2^14, 2^15)
    const int up = top == 0 || top >= 0x7F80u ? 127 : min(254, 268 - (int)(top >> 7));
    const float f = __uint_as_float((uint32_t)up << 23);
    uint32_t* out = reinterpret_cast<uint32_t*>(P.Q + row * D) + lane * (kV / 2);
#pragma unroll
    for (int k = 0; k < kV / 2; ++k)
      out[k] = pack2<QMM_F16>(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
    if (lane == 0) P.factors[row] = fmaxf(scalbnf(P.c, 127 - up), kLeastFactor);
    return;
  }
  constexpr int kBlocks = D / kv4::kBlock;
  const int64_t run_of = blockIdx.x / P.chunks, p = run_of / a.Hk;
  const int first = (int)(blockIdx.x - run_of * P.chunks) * P.blocks, h = (int)(run_of - p * a.Hk);
  if (h == 0 && first == 0 && threadIdx.x == 0) P.ids[p] = (int32_t)p;
  // (Of keys that no row sees, a stream's without rows or a prefix's without any stream's, not even the page is looked at.)
  int page, live;
  if (p < P.n_pre) {
    live = a.B > 0 && a.row_starts[a.B] > 0 ? (int)min((int64_t)a.page_size, a.prefix_len - p * a.page_size) : 0;
    page = live > 0 ? a.prefix_pages[p] : 0;
  } else {
    const int64_t own = p - P.n_pre;
    const int b = (int)(own / a.pages_per_stream);
    const Stream s = stream_of(a, b);
    live = s.m > 0 ? (int)min((int64_t)a.page_size, s.len - (own - (int64_t)b * a.pages_per_stream) * a.page_size) : 0;
    page = first < live * kBlocks ? a.pages[own] : 0;
  }
  const int end = min(live * kBlocks, first + P.blocks);
  if (first >= end) return;
  if (page < 0 || page >= a.n_slots / a.page_size) {
    if (threadIdx.x == 0) atomicOr(&g_status, kErrIndex);
    page = 0;   // (the rows that see it have unspecified values)
  }
  const int64_t from = kv4::run_at(page, h, a.Hk, a.page_size, D);
#pragma unroll 2
  for (int u = first + threadIdx.x; u < end; u += kExpandThreads) {
    const int slot = u / kBlocks, block = u % kBlocks;
    const int64_t to = ((p * a.page_size + slot) * a.Hk + h) * D + block * kv4::kBlock;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* run = static_cast<const uint8_t*>(k ? a.V_cache : a.K_cache) + from;
      const uint2 code = *reinterpret_cast<const uint2*>(run + (int64_t)u * 8);
      const uint32_t scale = run[a.page_size * (D / 2) + u];
      uint32_t w[8];
      to_half<0>(code, e4m3x2_pair(scale * 0x101u), w);
      uint4* out = reinterpret_cast<uint4*>((k ? P.V : P.K) + to);
      out[0] = make_uint4(w[0], w[1], w[2], w[3]);
      out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int D, int TYPE>
cudaError_t launch_expand(const qmm_attn_fp4_args& f, void* workspace, cudaStream_t stream) {
  const qmm_attn_args& a = f.base;
  const Expanded at(a);
  uint8_t* ws = static_cast<uint8_t*>(workspace) + (up(reinterpret_cast<uintptr_t>(workspace)) - reinterpret_cast<uintptr_t>(workspace));
  const int blocks = expanded_bytes(a) <= (double)kFewExpanded ? kExpandThreads : 2 * kExpandThreads;
  const int chunks = (a.page_size * (D / kv4::kBlock) + blocks - 1) / blocks;
  ExpandParams P{a, a.scale * f.k_scale * kLog2e, at.n_pre, at.n_pages * a.Hk * chunks, chunks, blocks,
                 reinterpret_cast<int32_t*>(ws + at.ids), reinterpret_cast<__half*>(ws + at.Q), reinterpret_cast<__half*>(ws + at.K),
                 reinterpret_cast<__half*>(ws + at.V), reinterpret_cast<float*>(ws + at.factors)};
  constexpr int kRowsOfCta = kExpandThreads / 32;
  const int64_t ctas = P.page_ctas + (TYPE == QMM_BF16 ? ((int64_t)a.T * a.Hq + kRowsOfCta - 1) / kRowsOfCta : 0);
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kExpandThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, expand_kernel<D, TYPE>, P);
  if (e != cudaSuccess) return e;
  qmm_attn_args view = a;
  view.type = QMM_F16;
  view.scale = fmaxf(a.scale * f.k_scale, kLeastFactor);
  view.K_cache = P.K;
  view.V_cache = P.V;
  view.n_slots = at.n_pages * a.page_size;
  view.prefix_pages = P.ids;
  view.pages = P.ids + at.n_pre;
  if (TYPE == QMM_BF16) {
    view.Q = P.Q;
    view.ldq = (int64_t)a.Hq * D;
  }
  int sms = 0;
  e = launch_attn_expanded(view, TYPE == QMM_BF16 ? P.factors : nullptr, workspace, &sms, stream);
  if (e != cudaSuccess) return e;
  Common C;
  const int tokens = kRows / (a.Hq / a.Hk);   // of that kernel's row tiles, two a block
  fill(C, a, tokens, 2 * tokens, workspace);
  C.v_scale = f.v_scale;
  return launch_combine<D, TYPE, true>(C, sms, stream);
}

template <int D, int TYPE>
cudaError_t launch_any(const qmm_attn_fp4_args& f, void* workspace, cudaStream_t stream) {
  return expands(f.base) ? launch_expand<D, TYPE>(f, workspace, stream) : launch<D, TYPE>(f, workspace, stream);
}

}  // namespace

size_t attn_fp4_workspace_bytes(const qmm_attn_fp4_args& f) {
  return expands(f.base) ? Expanded(f.base).total : Space(f.base).total;
}

cudaError_t launch_attn_fp4(const qmm_attn_fp4_args& f, void* workspace, cudaStream_t stream) {
  if (f.base.D == 64)
    return f.base.type == QMM_BF16 ? launch_any<64, QMM_BF16>(f, workspace, stream) : launch_any<64, QMM_F16>(f, workspace, stream);
  return f.base.type == QMM_BF16 ? launch_any<128, QMM_BF16>(f, workspace, stream) : launch_any<128, QMM_F16>(f, workspace, stream);
}

cudaError_t read_and_clear_attn_fp4_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
