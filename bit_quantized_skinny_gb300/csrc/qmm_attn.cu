// qmm_attn.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, both in pages of one cache (qmm_attn_shared).
//
// Work: equal pieces of the list of all key tiles, joined by a second launch (q4k_attn_parts.cuh).  A row tile is 128
// rows (128 / G tokens) and a block up to two tiles; a key tile is 64 keys.
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

#include "q4k_attn_parts.cuh"
#include "q4k_device.cuh"
#include "q4k_device_once.h"
#include "q4k_internal.h"
#include "q4k_tcgen05.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kTile = 64;            // keys of a key tile
constexpr int kLead = 4;             // units of a group besides its key tiles (2, 3, 6: 10, 6, 2 % slower for 16 streams)
constexpr int kLaneWarps = 4;
constexpr int kLoadWarp = 8, kMmaWarp = 9 /* and 10 */, kQWarp = 11;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;   // lane L: S at 64 L, p at 128 + 64 L and 160 + 64 L, O at 256 + 128 L
constexpr float kGrow = 8.0f;
constexpr uint32_t kWaitLimit = 1u << 17;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLift = 7.0f;        // (with kGrow, weights of at most 2^15)

struct Params : Common {
  CUtensorMap mapQ, mapK, mapV;
  const float* factors;   // EXPANDED: of each row and head, in place of scale log2 e; or NULL
};

template <int D>
struct Smem {
  static constexpr int kHalf = kTile * 128;              // 64 keys of 64 values
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQHalf = kRows * 128;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kStages = 5;                      // of keys, and of values
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kQBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kStats = kV + kStages * kTileBytes;   // (top, sum) of the two lanes' rows
  static constexpr int kMisc = kStats + 2 * kRows * 8;
  static constexpr int kTotal = kMisc + 1024;
};
static_assert(Smem<128>::kTotal <= 227 * 1024 && Smem<64>::kTotal <= 227 * 1024, "shared memory");

// Barriers.  A wait tells a phase from the one after it only, so a barrier is waited on by threads that
// see all of its phases, or that know the phase before to be over and the one after not begun: a stage of keys or values has a full barrier for each set of users (lane
// 0, lane 1, both), and a query tile is waited for and released by both lanes whoever uses it.
enum : int {
  kBarFullK = 0 /* 5 users + stage */, kBarFullV = 15, kBarEmptyK = 30, kBarEmptyV = 35, kBarQFull = 40, kBarQEmpty = 42,
  kBarS = 44, kBarFree = 46, kBarP = 48 /* 2 lane + item % 2 */, kBarO = 52, kBarEnd = 56, kBarJoin = 58, kBarDrain = 59,
  kBars = 61
};

struct Misc {
  uint64_t bars[kBars];
  Piece piece;
  uint32_t tmem;
  int abort;
  uint32_t odd[8];    // [s % 8]: s, if values were taken out in segment s (the lanes drift a few apart)
};
static_assert(sizeof(Misc) <= 1024, "misc");

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
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

// EXPANDED: keys and values are those of a 4-bit cache, which are few bits long, so p keeps more of its own than bf16
// has: it is fp16, and lifted by 2^kLift, so that a weight loses bits only below 2^-21 of the largest one.
template <int D, int TYPE, bool EXPANDED>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<D>;
  constexpr uint32_t kS = L::kStages;
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
    const bool two = (k >= kBarEmptyK && k < kBarQFull) || (k >= kBarQEmpty && k < kBarS);
    mbar_init(bar(k), two ? 2 : (k >= kBarFree && k < kBarO) ? kLaneWarps : k == kBarJoin ? 2 * kLaneWarps : 1);
    fence_barrier_init();
  } else if (threadIdx.x == kBars) {
    M.abort = 0;
    for (int k = 0; k < 8; ++k) M.odd[k] = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_addr(&M.tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  if (threadIdx.x < 3)
    asm volatile("prefetch.tensormap [%0];" :: "l"(threadIdx.x == 0 ? &P.mapK : threadIdx.x == 1 ? &P.mapV : &P.mapQ)
                 : "memory");
  // Launched early (behind a launch that allows it), this grid reads what was written before it from
  // here on; the combine launch, which reads the lengths before its own wait, may start from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  deal<kThreads, kTile, kLead>(P, M.piece, &g_status);
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

  Walker<kTile, kLead> walk;
  walk.start(P, M.piece);
  Seg g;

  if (warp == kLoadWarp) {
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
      constexpr bool kBf16 = TYPE == QMM_BF16;
      constexpr uint32_t kIdS = tc::idesc_16_f32(128, kTile, kBf16, false);
      constexpr uint32_t kIdO = tc::idesc_16_f32(128, D, kBf16, true);
      const uint64_t dq = tc::smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_addr(smem + L::kK), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(smem + L::kV), L::kHalf, 1024);
      const uint32_t l = warp - kMmaWarp;
      const uint32_t tS = tmem + kTile * l, tP = tmem + 2 * kTile + kTile * l, tO = tmem + 4 * kTile + kRows * l;
      const int barP = kBarP + 2 * l, barO = kBarO + 2 * l;
      struct Pass {
        Walker<kTile, kLead> w;
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
    bool ok = true;
    while (ok && walk.next(P, g)) {
      const int n = g.j1 - g.j0;
      const bool pair = g.rows > P.tokens;
      const int first = pair ? 0 : (items + l) & 1;               // the lane's first key tile of the segment
      const bool has[2] = {pair || n > (int)(items & 1), pair || n > (int)((items + 1) & 1)};   // lanes with key tiles
      const int tok0 = pair ? l * P.tokens : 0;                   // the lane's rows of the block
      const int live = min(P.tokens, g.rows - tok0) * G;          // rows of the tile in use
      const int tok = tok0 + row / G;
      if constexpr (EXPANDED)
        if (P.factors) c = row < live ? P.factors[(int64_t)(g.t0 + tok) * a.Hq + g.h * G + row % G] : 0.0f;
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
        // value rows that a weight of 0 must not meet
        const int upto = min(g.keys, base + kTile) - base;
        if (ok && clean_from < base + kTile && (upto < kTile || g.own)) {
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
          const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c - (EXPANDED ? kLift : 0.0f);
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
          const float off = top == -INFINITY ? 0.0f : -top;
          const uint64_t cc = f2pack(c, c), oo = f2pack(off, off);
          uint64_t part0 = 0, part1 = 0;   // sums of weights, two fp32 each
#pragma unroll
          for (int k = 0; k < kTile; k += 4) {
            const float2 x = f2unpack(fma2(f2pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, oo));
            const float2 y = f2unpack(fma2(f2pack(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), cc, oo));
            const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y), p2 = exp2_fast(y.x), p3 = exp2_fast(y.y);
            part0 = add2(part0, f2pack(p0, p1));
            part1 = add2(part1, f2pack(p2, p3));
            s[k / 2] = pack2<TYPE>(p0, p1);
            s[k / 2 + 1] = pack2<TYPE>(p2, p3);
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
        const uint32_t per = (uint32_t)min(M.piece.per, (int64_t)0x7fffffff);
        const uint32_t others = g.rest > 0 ? ((uint32_t)g.rest + per - 1) / per : 0;
        RowStat st{top, sum, odd, others << 16 | (blockIdx.x + 1)};
        if (!pair) {
          const float2 s0 = stats[row], s1 = stats[kRows + row];
          st.top = fmaxf(s0.x, s1.x);
          st.sum = (!(s0.x == -INFINITY && s0.y == 0.0f) ? s0.y * exp2_fast(s0.x - st.top) : 0.0f) +
                   (!(s1.x == -INFINITY && s1.y == 0.0f) ? s1.y * exp2_fast(s1.x - st.top) : 0.0f);
        }
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

template <int D, int TYPE, bool EXPANDED>
cudaError_t set_smem_attr() {
  static DeviceOnce once;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once.run(dev, cudaSuccess, [] {
    return cudaFuncSetAttribute(attn_kernel<D, TYPE, EXPANDED>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
  });
}

// The launch ahead of the combine's; *sms: what that one takes.
template <int D, int TYPE, bool EXPANDED>
cudaError_t launch_products(Params& P, int* sms_out, cudaStream_t stream) {
  const qmm_attn_args& a = P.a;
  const int G = a.Hq / a.Hk;
  const int per_box = a.page_size < kTile ? a.page_size : kTile;
  if (!tensor_map(&P.mapQ, a.Q, D, a.Hq, a.T, a.ldq, G, P.tokens, TYPE) ||
      !tensor_map(&P.mapK, a.K_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE) ||
      !tensor_map(&P.mapV, a.V_cache, D, a.Hk, a.n_slots, (int64_t)a.Hk * D, 1, per_box, TYPE))
    return cudaErrorInvalidValue;
  const cudaError_t e = set_smem_attr<D, TYPE, EXPANDED>();
  if (e != cudaSuccess) return e;
  const int sms = *sms_out = sm_count();
  if (sms < 1) return cudaErrorNoDevice;
  // Both launches may be scheduled while the one before them finishes (programmatic dependent launch);
  // each waits for it before it reads or writes memory.
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
  return cudaLaunchKernelEx(&cfg, attn_kernel<D, TYPE, EXPANDED>, P);
}

void fill_rows(Params& P, const qmm_attn_args& a, void* workspace) {
  const int tokens = kRows / (a.Hq / a.Hk);
  fill(P, a, tokens, 2 * tokens, workspace);
  P.factors = nullptr;
}

template <int D, int TYPE>
cudaError_t launch(const qmm_attn_args& a, void* workspace, cudaStream_t stream) {
  Params P;
  int sms = 0;
  fill_rows(P, a, workspace);
  const cudaError_t e = launch_products<D, TYPE, false>(P, &sms, stream);
  return e != cudaSuccess ? e : launch_combine<D, TYPE, false>(P, sms, stream);
}

template <int D>
cudaError_t launch_expanded(const qmm_attn_args& view, const float* factors, void* workspace, int* sms, cudaStream_t stream) {
  Params P;
  fill_rows(P, view, workspace);
  P.factors = factors;
  return launch_products<D, QMM_F16, true>(P, sms, stream);
}

}  // namespace

size_t attn_workspace_bytes(const qmm_attn_args& a) { return Space(a).total; }

cudaError_t launch_attn(const qmm_attn_args& a, void* workspace, cudaStream_t stream) {
  if (a.D == 64)
    return a.type == QMM_BF16 ? launch<64, QMM_BF16>(a, workspace, stream) : launch<64, QMM_F16>(a, workspace, stream);
  return a.type == QMM_BF16 ? launch<128, QMM_BF16>(a, workspace, stream) : launch<128, QMM_F16>(a, workspace, stream);
}

cudaError_t launch_attn_expanded(const qmm_attn_args& view, const float* factors, void* workspace, int* sms, cudaStream_t stream) {
  return view.D == 64 ? launch_expanded<64>(view, factors, workspace, sms, stream)
                      : launch_expanded<128>(view, factors, workspace, sms, stream);
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
