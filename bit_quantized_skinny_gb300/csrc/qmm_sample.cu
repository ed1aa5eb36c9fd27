// qmm_sample.cu — the token of every row from its logits, and how many drafted tokens stand (qmm_sample).
//
// Weights.  w = exp((x - max) / T) as an integer W = w 2^42, to a unit or two: two neighbouring tokens lie 2^-18 of the
// sum apart where 250000 share it, so fp32 weights would pick the wrong one in every hundredth row; integers
// also make every sum independent of its order.  t = (x - max) log2(e) / T is formed in two fp32 words
// (the difference and the product are exact but for 2^-45), split into -(n + j/1024) and a rest g of at most 2^-11, and
//     W = (2^42 2^(-j/1024) 2^g) >> n,     2^g - 1 = g ln2 + (g ln2)^2/2 + (g ln2)^3/6
// with 2^(42 - j/1024) from a table and the correction as a 32-bit integer.
//
// A row is read once, into the shared memory of a cluster's CTAs, and everything else is passes over it there.  What bounds
// a call: with few rows the barriers and exchanges between the cluster's CTAs, some 700 cycles each (1 row of 248320 18 us);
// with many, the rows' passes (128 rows: greedy ones 92 us, top_k 50 178, top_k 1000 293, min_p alone 151, top_p alone, the
// weights of all tokens twice, 526 and 671).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include "q4k_device_once.h"
#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kUnit = 42;              // a weight of 1 is 2^kUnit; QMM_SAMPLE_MAX_V of them stay below 2^62
constexpr int kSteps = 1024;           // of the table, for one octave
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
constexpr int kList = 1024;            // tokens of a CTA's list, and of the cluster's
static_assert(kList <= kBins / 2 && kList <= 2 * kThreads, "a list is sorted in the bins' place, two tokens a thread");
constexpr int kMaxCluster = 16, kMaxRun = ((QMM_SAMPLE_MAX_V / kMaxCluster + kThreads - 1) / kThreads) | 1;
static_assert(QMM_SAMPLE_MAX_V <= (1 << 19), "sums of weights");

using u64 = unsigned long long;

// 2^(42 - j/1024), j = 0 .. 1023: 2^(-1/1024) by ten integer square roots of 1/2, then its powers, with 62 bits
// behind the point (an error of 2^-52 at the end).
struct Table {
  u64 v[kSteps];
};
constexpr u64 isqrt(unsigned __int128 x) {
  unsigned __int128 lo = 0, hi = (unsigned __int128)1 << 63;
  while (hi - lo > 1) {
    const unsigned __int128 mid = (lo + hi) >> 1;
    if (mid * mid <= x) lo = mid; else hi = mid;
  }
  return (u64)lo;
}
constexpr Table make_table() {
  constexpr int kQ = 62;
  u64 r = u64(1) << (kQ - 1);
  for (int k = 0; k < 10; ++k) r = isqrt((unsigned __int128)r << kQ);
  Table t{};
  u64 at = u64(1) << kQ;
  for (int j = 0; j < kSteps; ++j) {
    t.v[j] = ((at >> (kQ - kUnit - 1)) + 1) >> 1;
    at = (u64)(((unsigned __int128)at * r + ((unsigned __int128)1 << (kQ - 1))) >> kQ);
  }
  return t;
}
__device__ constexpr Table kTable = make_table();

// log2(e) / T in two fp32 words: the rounded quotient, and what it leaves (a 64-bit division takes 4000 cycles).  Logits and
// temperature are taken in units of 2^64 where T is above that: their differences may leave fp32's range, and the quotient's words
// its precision, while a weight hangs on nothing of a logit below 2^-42 T.  In the same way in units of 2^-64 where T is below
// those (a logit that is infinite then differs from every other one by too many T's for a weight).
struct Slope {
  float hi, lo, unit;
};
__device__ __forceinline__ Slope slope_of(float temperature) {
  const float unit = temperature > 0x1p64f ? 0x1p-64f : temperature < 0x1p-64f ? 0x1p64f : 1.0f;
  temperature *= unit;
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746e-8f;   // log2(e)
  const float hi = __fdiv_rn(kHi, temperature);
  return Slope{hi, hi > 0.0f && hi < INFINITY ? __fdiv_rn(__fmaf_rn(-hi, temperature, kHi) + kLo, temperature) : 0.0f, unit};
}

// The weight of logit x (not NaN, not above top) as an integer.
__device__ __forceinline__ u64 weight(float x, float top, Slope c, const u64* table) {
  if (x == top) return u64(1) << kUnit;   // (also where both are infinite)
  x *= c.unit;
  top *= c.unit;
  const float d = x - top;                // two words: the rounded difference and what it lost
  const float b = d - x, lost = (x - (d - b)) + (-top - b);
  const float th = d * c.hi;
  if (!(th > -46.0f)) return 0;           // below half a unit (and any difference that is not finite)
  const float tl = __fmaf_rn(d, c.hi, -th) + __fmaf_rn(d, c.lo, lost * c.hi);
  const float kMagic = 12582912.0f;       // 1.5 * 2^23: added, a float of at most 2^22 has its integer in its low bits
  const float u = __fmaf_rn(th, -(float)kSteps, kMagic);
  const uint32_t k = __float_as_uint(u) - __float_as_uint(kMagic);
  const float gh = __fmaf_rn(u - kMagic, 1.0f / kSteps, th);
  // 2^g - 1 in units of 2^-42: the leading product exact in two words
  constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-09f;
  const float p = gh * kLn2Hi;
  const float low = __fmaf_rn(gh, kLn2Hi, -p) + __fmaf_rn(gh, kLn2Lo, tl * kLn2Hi) +
                    gh * gh * __fmaf_rn(gh, 0.0555041087f, 0.2402265070f);
  const float big = p * 0x1p42f, v = __fmaf_rn(big, 0x1p-9f, kMagic), vi = v - kMagic;
  const float rest = __fmaf_rn(vi, -0x1p9f, big) + low * 0x1p42f;
  const int grow = ((int)(__float_as_uint(v) - __float_as_uint(kMagic)) << 9) +
                   (int)(__float_as_uint(rest + kMagic) - __float_as_uint(kMagic));
  const u64 base = table[k & (kSteps - 1)];
  const int n = (int)(k / kSteps);
  const long long more = ((long long)(int)(base >> 12) * grow + (1 << 29)) >> 30;   // base * grow / 2^42
  return (base + more + ((u64(1) << n) >> 1)) >> n;   // (without rounding 250000 small weights would lose half a unit each)
}

// floor(f * n) of a finite fp32 f in [0, 1) and n below 2^63; exact: whether that is f * n itself.
__device__ __forceinline__ u64 fraction_of(float f, u64 n, bool* exact) {
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const u64 m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (int)(e ? e : 1u);   // f = m 2^-shift
  const u64 lo = m * n, hi = __umul64hi(m, n);
  u64 whole, rest;
  if (shift >= 128) {
    whole = 0;
    rest = lo | hi;
  } else if (shift >= 64) {
    whole = shift == 64 ? hi : hi >> (shift - 64);
    rest = lo | (shift == 64 ? 0 : hi << (128 - shift));
  } else {
    whole = lo >> shift | hi << (64 - shift);   // (24 <= shift)
    rest = lo << (64 - shift);
  }
  *exact = rest == 0;
  return whole;
}

template <int TYPE>
__device__ __forceinline__ float logit(const void* row, int i) {
  float x;
  if constexpr (TYPE == QMM_F32) x = static_cast<const float*>(row)[i];
  else if constexpr (TYPE == QMM_BF16) x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[i] << 16);
  else x = __half2float(__ushort_as_half(static_cast<const uint16_t*>(row)[i]));
  return x == x ? x + 0.0f : -INFINITY;   // (-0 and 0 are equal)
}
// Bits that order as the logits do.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The float of a key.
__device__ __forceinline__ float float_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); }

// Sum over the warp, in every lane (32 lanes of 16 bits fit into 32).
__device__ __forceinline__ u64 warp_sum(u64 v) {
  u64 sum = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) sum += (u64)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> (16 * q)) & 0xFFFFu) << (16 * q);
  return sum;
}
// Sum over the lanes up to this one.
__device__ __forceinline__ u64 warp_upto(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  return v;
}

constexpr int kWarps = kThreads / 32;

// A row lies in the shared memory of a cluster's CTAs, in order of the tokens: a CTA has a slice, a thread a run of it (an odd
// number of floats, so that a warp's runs lie in different banks).  Once a floor is known below which no token can
// stay, a CTA lists its tokens above it; where all lists are short, the first CTA takes them and ends the row alone.
struct Cta {
  u64 part[4];            // this CTA's part of a sum, a maximum or a scan over the cluster; used in turn
  uint32_t low[4];
  u64 scan[kWarps];
  uint32_t scan_low[kWarps];
  union {                 // of this CTA
    uint32_t count[kBins];
    u64 mass[kBins / 2];
  };
  union {                 // of the cluster
    uint32_t total[kBins];
    u64 mass_total[kBins / 2];
  };
  u64 found[2];           // what the thread that found it tells the others
  u64 table[kSteps];
  float list_x[2][kList];   // tokens above the floor, in order of their index
  int list_i[2][kList];
};

struct Keys {             // lo <= key <= hi
  uint32_t lo, hi;
};

// Sum over the threads of the CTA before this one, and over the CTA.  (Out of line, as weight_once() is: a sixth less code, the
// same times.)
struct Sums {
  u64 before, all;
};
__device__ __noinline__ Sums block_sums(u64* scan, u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 upto = warp_upto(v);
  __syncthreads();
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  const u64 of = lane < kWarps ? scan[lane] : 0;
  return Sums{upto - v + warp_sum(lane < warp ? of : 0), warp_sum(of)};
}
__device__ __noinline__ u64 weight_once(float x, float top, Slope c, const u64* table) { return weight(x, top, c, table); }

enum Raised { kDone, kSpread, kAlone };   // this CTA has nothing left to do; goes on with the others; has all tokens

struct Sampler {
  Cta& S;
  float* x;               // the slice
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int turn = 0;           // of part
  int run, first;         // tokens of a thread; index of its first one in the row, if they are a run of it
  const float* mine;
  const int* index = nullptr;   // of its tokens, if they are not
  uint32_t floor = 0;     // keys below it do not stay
  uint32_t own = 0;       // the key of this thread's largest token
  int lists = 0;          // made so far: the next one goes to the other place
  int listed = 0;         // alone: the tokens, their values and indices in list_x, list_i
  const float* all_x;
  const int* all_i;
  float top;
  Slope c;

  __device__ __forceinline__ int index_of(int j) const { return index ? index[j] : first + j; }
  // Every token of this thread above the floor: f(value, index).
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    if (own < floor) return;
#pragma unroll 2
    for (int j = 0; j < run; ++j) {
      const float v = mine[j];
      if (key_of(v) >= floor) f(v, index_of(j));
    }
  }
  __device__ __forceinline__ u64 weight_of(float v) const { return v == -INFINITY ? u64(0) : weight(v, top, c, S.table); }
  __device__ __forceinline__ u64 weight_of_one(float v) const { return v == -INFINITY ? u64(0) : weight_once(v, top, c, S.table); }

  __device__ __forceinline__ void sync() const {
    if (C > 1) cluster.sync();
    else __syncthreads();
  }
  // The parts of the cluster's CTAs, one a lane; they may be written again four calls later.
  __device__ __forceinline__ u64 exchange(u64 v) {
    const int lane = threadIdx.x & 31;
    if (C == 1) return lane == 0 ? v : 0;
    if (threadIdx.x == 0) S.part[turn] = v;
    cluster.sync();
    u64 got = 0;
    if (lane < C) got = *cluster.map_shared_rank(&S.part[turn], lane);
    turn = (turn + 1) & 3;
    return got;
  }
  __device__ __forceinline__ u64 cluster_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) S.scan[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < kWarps ? S.scan[threadIdx.x & 31] : 0;
    return warp_sum(exchange(warp_sum(v)));
  }
  // The largest key and the lowest index that has it, and the lowest of `low`.
  __device__ __forceinline__ void best_of(uint32_t& key, uint32_t& at, uint32_t& low) {
    auto within = [&]() {
      const uint32_t most = __reduce_max_sync(0xffffffffu, key);
      at = __reduce_min_sync(0xffffffffu, key == most ? at : 0xFFFFFFFFu);
      key = most;
      low = __reduce_min_sync(0xffffffffu, low);
    };
    const int lane = threadIdx.x & 31;
    auto have = [&](bool some, const u64* p, const uint32_t* l) {
      const u64 v = some ? *p : 0;
      key = (uint32_t)(v >> 32);
      at = some ? (uint32_t)v : 0xFFFFFFFFu;
      low = some ? *l : 0xFFFFFFFFu;
      within();
    };
    within();
    if (lane == 0) {
      S.scan[threadIdx.x >> 5] = (u64)key << 32 | at;
      S.scan_low[threadIdx.x >> 5] = low;
    }
    __syncthreads();
    have(lane < kWarps, &S.scan[lane % kWarps], &S.scan_low[lane % kWarps]);
    if (C == 1) return;
    if (threadIdx.x == 0) {
      S.part[turn] = (u64)key << 32 | at;
      S.low[turn] = low;
    }
    cluster.sync();
    have(lane < C, cluster.map_shared_rank(&S.part[turn], lane % C), cluster.map_shared_rank(&S.low[turn], lane % C));
    turn = (turn + 1) & 3;
  }
  // Sum over the threads of the CTA before this one; all: over the CTA.
  __device__ __forceinline__ u64 block_before(u64 v, u64* all) {
    const Sums sums = block_sums(S.scan, v);
    *all = sums.all;
    return sums.before;
  }
  // Sum over the threads of the cluster before this one; all: over the cluster.
  __device__ __forceinline__ u64 cluster_before(u64 v, u64* all) {
    u64 sum;
    const u64 before = block_before(v, &sum), parts = exchange(sum);
    *all = warp_sum(parts);
    return C == 1 ? before : before + warp_sum((threadIdx.x & 31) < rank ? parts : 0);
  }

  // Sums over the cluster's values that `in` takes, by bin(x), in `total` of every CTA: counts (N uint32_t, kBins of them) or
  // weights (N u64, kBins / 2).
  template <class N, class In, class Bin>
  __device__ __forceinline__ void histogram(In&& in, Bin&& bin) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) S.count[b] = 0;
    if constexpr (sizeof(N) == 4) {
      __syncthreads();
      each([&](float v, int i) {
        if (in(v, i)) atomicAdd(&S.count[bin(v)], 1u);
      });
    } else {
      // A weight in three parts of 14 bits, which 32 bits of a bin hold the sums of: shared memory adds these by itself, and
      // 64 bits by a loop of compares (13 rows of 32003 with top_p 41 us; in parts, with one pass of weights less, 28).
      constexpr int kHalfBins = kBins / 2;
      static_assert((int64_t)kMaxRun * kThreads < (1 << 17), "sums of parts");
      for (int b = threadIdx.x; b < kHalfBins; b += kThreads) S.total[b] = 0;
      __syncthreads();
      each([&](float v, int i) {
        if (!in(v, i)) return;
        const u64 w = weight_of(v);
        const int b = bin(v);
        if (const uint32_t part = (uint32_t)w & 0x3FFFu) atomicAdd(&S.count[b], part);
        if (const uint32_t part = (uint32_t)(w >> 14) & 0x3FFFu) atomicAdd(&S.count[kHalfBins + b], part);
        if (const uint32_t part = (uint32_t)(w >> 28)) atomicAdd(&S.total[b], part);
      });
      __syncthreads();
      u64 sum[kHalfBins / kThreads];
#pragma unroll
      for (int q = 0; q < kHalfBins / kThreads; ++q) {
        const int b = q * kThreads + threadIdx.x;
        sum[q] = S.count[b] + ((u64)S.count[kHalfBins + b] << 14) + ((u64)S.total[b] << 28);
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kHalfBins / kThreads; ++q) S.mass[q * kThreads + threadIdx.x] = sum[q];
    }
    join<N>();
  }
  // Counts of bin(v) of one value of each thread, in the same way.
  template <class Bin>
  __device__ __forceinline__ void histogram_of(float v, Bin&& bin) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) S.count[b] = 0;
    __syncthreads();
    atomicAdd(&S.count[bin(v)], 1u);
    join<uint32_t>();
  }
  // `total` of all CTAs from their `count`: each adds up its share of the bins and gives it to all.
  template <class N>
  __device__ __forceinline__ void join() {
    constexpr int kN = kBins * 4 / (int)sizeof(N);
    N* count = reinterpret_cast<N*>(S.count);
    N* total = reinterpret_cast<N*>(S.total);
    sync();
    const int bins = kN / C;
    for (int b = rank * bins + threadIdx.x; b < (rank + 1) * bins; b += kThreads) {
      N sum = 0;
      if (C == 1) {
        sum = count[b];
      } else {
#pragma unroll 8
        for (int r = 0; r < C; ++r) sum += *cluster.map_shared_rank(&count[b], r);
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&total[b], r) = sum;
      }
      if (C == 1) total[b] = sum;
    }
    sync();
  }
  // All weights, from the cluster's bins.
  __device__ __forceinline__ u64 mass_of_bins() {
    constexpr int kMine = kBins / 2 / kThreads;
    u64 sum = 0, all;
#pragma unroll
    for (int q = 0; q < kMine; ++q) sum += S.mass_total[kMine * threadIdx.x + q];
    block_before(sum, &all);
    return all;
  }
  // The first bin whose sums reach n >= 1, with those before it; false: all of them do not.
  template <class N>
  __device__ __forceinline__ bool find(u64 n, int* bin, u64* before) {
    constexpr int kMine = kBins * 4 / (int)sizeof(N) / kThreads;
    const N* total = reinterpret_cast<const N*>(S.total) + kMine * threadIdx.x;
    u64 sum = 0, all;
#pragma unroll
    for (int q = 0; q < kMine; ++q) sum += total[q];
    u64 at = block_before(sum, &all);
    *bin = 0;
    *before = 0;
    if (all < n) return false;
    if (at < n && at + sum >= n) {
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        const u64 m = total[q];
        if (at < n && at + m >= n) {
          S.found[0] = kMine * threadIdx.x + q;
          S.found[1] = at;
        }
        at += m;
      }
    }
    __syncthreads();
    *bin = (int)S.found[0];
    *before = S.found[1];
    __syncthreads();
    return true;
  }

  // The keys whose value `bin` (which does not rise with the key) puts into b1 .. b2: a warp for each end, 32 keys a step.
  template <class Bin>
  __device__ __forceinline__ Keys keys_of(int b1, int b2, Bin&& bin) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 2) {
      // the lowest key whose bin is at most b: the range's low end, and one above its high end
      const int b = warp ? b1 - 1 : b2;
      uint32_t lo = 0x007FFFFFu, hi = 0xFF800001u;   // of -infinity, behind infinity: hi has a bin that low
      while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32, key = lo + lane * step;   // lo, ..., lo + 31 steps
        const bool low = key >= hi || bin(float_of(min(key, 0xFF800000u))) <= b;
        const uint32_t some = __ballot_sync(0xffffffffu, low);
        const int at = some ? __ffs(some) - 1 : 32;   // the first of the 32 that is low enough
        hi = at < 32 ? min(hi, lo + at * step) : hi;
        if (at == 0) break;
        lo = lo + (at - 1) * step + 1;
      }
      if (lane == 0) S.found[warp] = warp ? (b < 0 ? 0xFF800000u : hi - 1) : hi;
    }
    __syncthreads();
    const Keys r{(uint32_t)S.found[0], (uint32_t)S.found[1]};
    __syncthreads();
    return r;
  }

  // The n2 entries of `mass` (a power of two, at most kBins / 2), the highest one first.
  __device__ __forceinline__ void sort(int n2) {
    u64* sorted = S.mass;
    const int tid = threadIdx.x;
    for (int size = 2; size <= n2; size *= 2) {
      for (int stride = size / 2; stride > 0; stride /= 2) {
        if (tid < n2 / 2) {
          const int i = 2 * stride * (tid / stride) + tid % stride;
          const u64 u = sorted[i], v = sorted[i + stride];
          if ((u < v) == ((i & size) == 0)) {
            sorted[i] = v;
            sorted[i + stride] = u;
          }
        }
        // (a warp keeps to its own 64 entries while the strides are at most 32)
        const int next = stride > 1 ? stride / 2 : size;
        if (stride > 32 || next > 32) __syncthreads();
        else __syncwarp();
      }
    }
    __syncthreads();
  }

  // Of the tokens that `in` takes, those with a key in r, the highest first and of equal ones the lowest index: the key and
  // the index of the one with which their sum reaches n (there is one).  The first CTA sorts them if they are few; more are
  // told apart by bins of 2^shift keys before, and ties on a key are counted.
  template <class N, class In>
  __device__ __forceinline__ void settle(Keys r, u64 n, In&& in, uint32_t* key_out, int* last) {
    constexpr int kBits = sizeof(N) == 4 ? kBinBits : kBinBits - 1;
    for (;;) {
      auto here = [&](float v, int i) { const uint32_t key = key_of(v); return key >= r.lo && key <= r.hi && in(v, i); };
      u64 mine_n = 0, all, found = 0;
      each([&](float v, int i) { mine_n += here(v, i); });
      const u64 before = cluster_before(mine_n, &all);
      if (all <= (u64)kList) {
        // keys and places from the end of the row to the first CTA
        u64 to = before;
        if (mine_n > 0)
          each([&](float v, int i) {
            if (!here(v, i)) return;
            u64* at = &S.mass[to++];
            *(C == 1 ? at : cluster.map_shared_rank(at, 0)) = (u64)key_of(v) << 32 | (0xFFFFFFFFu - (uint32_t)i);
          });
        sync();
        if (rank == 0) {
          int n2 = 2;
          while (n2 < (int)all) n2 *= 2;
          for (int e = (int)all + threadIdx.x; e < n2; e += kThreads) S.mass[e] = 0;
          __syncthreads();
          sort(n2);
          u64 w[2] = {0, 0}, sum;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int e = 2 * threadIdx.x + q;
            if (e < (int)all) w[q] = sizeof(N) == 4 ? u64(1) : weight_of_one(float_of((uint32_t)(S.mass[e] >> 32)));
          }
          const u64 at = block_before(w[0] + w[1], &sum);
          if (at < n && at + w[0] + w[1] >= n) S.found[0] = S.mass[2 * threadIdx.x + (at + w[0] < n)];
        }
        sync();
        const u64 one = C == 1 ? S.found[0] : *cluster.map_shared_rank(&S.found[0], 0);
        sync();
        *key_out = (uint32_t)(one >> 32);
        *last = (int)(0xFFFFFFFFu - (uint32_t)one);
        return;
      }
      if (r.lo == r.hi) {   // ties, in order of their index
        const u64 w = sizeof(N) == 4 ? u64(1) : max(weight_of_one(float_of(r.lo)), u64(1)), count = (n + w - 1) / w;
        u64 at = before;
        if (before < count && before + mine_n >= count)
          each([&](float v, int i) {
            if (here(v, i) && ++at == count) found = (u64)i + 1;
          });
        *key_out = r.lo;
        *last = (int)cluster_sum(found) - 1;
        return;
      }
      const int shift = max(0, 32 - __clz(r.hi - r.lo) - kBits);
      int b;
      u64 above;
      histogram<N>(here, [&](float v) { return (int)((r.hi - key_of(v)) >> shift); });
      find<N>(n, &b, &above);
      n -= above;
      r.hi -= (uint32_t)b << shift;
      r.lo = max(r.lo, r.hi - ((1u << shift) - 1));
    }
  }

  // Nothing below `lowest` stays, nor what `in` does not take: the CTA's other tokens into its list, and all lists to the
  // first CTA if they are short.
  template <class In>
  __device__ __forceinline__ Raised raise_floor(uint32_t lowest, In&& in) {
    floor = max(floor, lowest);
    u64 n = 0, all;
    each([&](float v, int i) { n += in(v, i); });
    const u64 at = block_before(n, &all);
    const bool fits = all <= (u64)kList;
    const int place = lists++ & 1;
    if (fits) {
      int to = (int)at;
      if (n > 0)
        each([&](float v, int i) {
          if (in(v, i)) {
            S.list_x[place][to] = v;
            S.list_i[place][to++] = i;
          }
        });
      run = ((int)all + kThreads - 1) / kThreads;
      const int from = min((int)all, (int)threadIdx.x * run);
      run = min(run, (int)all - from);
      mine = S.list_x[place] + from;
      index = S.list_i[place] + from;
      own = 0xFFFFFFFFu;
    }
    const u64 parts = exchange(fits ? all : u64(1) << 20), upto = warp_upto(parts);   // (the lists are written before it)
    const int sum = (int)__shfl_sync(0xffffffffu, upto, 31);
    if (sum > kList) {
      __syncthreads();
      return kSpread;
    }
    listed = sum;
    all_x = S.list_x[place];
    all_i = S.list_i[place];
    if (C == 1) {
      __syncthreads();
      return kAlone;
    }
    if (rank == 0) {   // a warp for each CTA's list
      float* xs = S.list_x[place ^ 1];
      int* is = S.list_i[place ^ 1];
      for (int r = threadIdx.x >> 5; r < C; r += kWarps) {
        const int to = (int)__shfl_sync(0xffffffffu, upto - parts, r), len = (int)__shfl_sync(0xffffffffu, parts, r);
        const float* from_x = cluster.map_shared_rank(S.list_x[place], r);
        const int* from_i = cluster.map_shared_rank(S.list_i[place], r);
        for (int j = threadIdx.x & 31; j < len; j += 32) {
          xs[to + j] = from_x[j];
          is[to + j] = from_i[j];
        }
      }
      all_x = xs;
      all_i = is;
    }
    cluster.sync();   // no CTA ends while another one reads its shared memory
    return rank == 0 ? kAlone : kDone;
  }
};

// log of total / 2^kUnit weights of 1, less w's: the logprob's terms in units of log2(e)^-1 are exact but for some 2^-34.
__device__ __forceinline__ float logprob_of(float v, float top, Slope c, u64 total, const u64* table) {
  // log2(total) = e + j / kSteps + log2(1 + r): the table's entry kSteps - j is 2^(j / kSteps) below one octave
  const int e = 63 - __clzll(total);
  const u64 m = e >= kUnit ? total >> (e - kUnit) : total << (kUnit - e);   // in [2^kUnit, 2^(kUnit + 1))
  const float log2m = log2f((float)m * 0x1p-42f);
  int j = min(kSteps - 1, max(0, (int)(log2m * kSteps)));
  const u64 base = j ? 2 * table[kSteps - j] : u64(1) << kUnit;
  const float r = (float)(long long)(m - base) / (float)base;
  const float rest = r * 1.44269504f * (1.0f - r * (0.5f - r * 0.333333333f));
  const float whole = (float)(e - kUnit) + (float)j * (1.0f / kSteps);        // exact
  float th = 0.0f, tl = 0.0f;
  if (v != top) {
    v *= c.unit;
    top *= c.unit;
    const float d = v - top, b = d - v, lost = (v - (d - b)) + (-top - b);
    th = d * c.hi;
    tl = __fmaf_rn(d, c.hi, -th) + __fmaf_rn(d, c.lo, lost * c.hi);
  }
  const float s = th - whole, b = s - th, err = (th - (s - b)) + (-whole - b);   // s + err = th - whole
  const float low = (tl - rest) + err, hi = s + low, lo = low - (hi - s);
  return __fmaf_rn(hi, 0.693147182464599609375f, __fmaf_rn(hi, -1.904654323148236017e-09f, lo * 0.693147182f));
}

// The rest of a row whose tokens are R's list: they are sorted, and everything else is two sums along them.  k: how many of
// them top_k leaves; all: the sum that top_p is a share of (0: of those k).
__device__ __forceinline__ void end_alone(const qmm_sample_args& a, Sampler& R, int t, int k, float p, float mp, u64 least, u64 all) {
  Cta& S = R.S;
  const int tid = threadIdx.x, n = R.listed;
  int n2 = 2;
  while (n2 < n) n2 *= 2;
  u64* sorted = S.mass;        // key, place from the end: the highest key first, of equal ones the lowest place
  u64* kept = S.mass_total;    // weights that stay, by place
  for (int e = tid; e < n2; e += kThreads)
    sorted[e] = e < n ? (u64)key_of(R.all_x[e]) << 32 | (0xFFFFFFFFu - (uint32_t)e) : 0;
  __syncthreads();
  R.sort(n2);
  u64 w[2] = {0, 0}, sum;
  int place[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = 2 * tid + q;
    place[q] = -1;
    if (e < n) {
      const u64 v = sorted[e];
      place[q] = (int)(0xFFFFFFFFu - (uint32_t)v);
      if (e < k) w[q] = R.weight_of_one(float_of((uint32_t)(v >> 32)));
    }
  }
  u64 at = R.block_before(w[0] + w[1], &sum);
  u64 target = ~u64(0);
  if (p < 1.0f) {
    bool exact;
    target = fraction_of(fmaxf(p, 0.0f), all ? all : sum, &exact);
    target = max(u64(1), target + !exact);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const bool stays = mp > 1.0f ? tid + q == 0 : at < target && w[q] >= least;
    if (place[q] >= 0) kept[place[q]] = stays ? w[q] : 0;
    at += w[q];
  }
  __syncthreads();
  const u64 k0 = 2 * tid < n ? kept[2 * tid] : 0, k1 = 2 * tid + 1 < n ? kept[2 * tid + 1] : 0;
  u64 total;
  const u64 before = R.block_before(k0 + k1, &total);
  bool exact;
  const u64 goal = fraction_of(fminf(fmaxf(a.uniform[t], 0.0f), 0x1.fffffep-1f), total, &exact);
  if (before <= goal && before + k0 + k1 > goal) {
    const int e = 2 * tid + (before + k0 <= goal);
    a.tokens[t] = R.all_i[e];
    if (a.logprobs) a.logprobs[t] = logprob_of(R.all_x[e], R.top, R.c, total, S.table);
  }
}

// A cluster per row.  The borders are found by sums over bins (of counts for top_k, of weights for top_p), first over the
// distance from the largest logit, then over the keys of the bin in which the border lies, until a bin is one key; ties
// on it go by index.  Before that, a floor leaves most of a vocabulary behind, and what is above it is as a rule
// few enough for one CTA to sort.
template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ qmm_sample_args a, int run, int vec) {
  extern __shared__ __align__(16) uint8_t smem[];
  Sampler R{*reinterpret_cast<Cta*>(smem), reinterpret_cast<float*>(smem + sizeof(Cta))};
  Cta& S = R.S;
  for (int j = threadIdx.x; j < kSteps; j += kThreads) S.table[j] = kTable.v[j];
  // launched early behind a launch that allows it: memory that it may be writing is read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x / R.C, V = a.V, slice = run * kThreads, begin = R.rank * slice;
  const int n = max(0, min(V - begin, slice));
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + t * a.ld * (TYPE == QMM_F32 ? 4 : 2);
  R.run = run;
  R.first = begin + (int)threadIdx.x * run;
  R.mine = R.x + (int)threadIdx.x * run;

  // the slice, its largest logit (the lowest index of equal ones)
  auto take = [&](float v) { return v == v ? v + 0.0f : -INFINITY; };   // (-0 and 0 are equal)
  constexpr int kPerVec = TYPE == QMM_F32 ? 4 : 8;
  const int whole = vec ? n / kPerVec * kPerVec : 0;
#pragma unroll 4
  for (int i = kPerVec * threadIdx.x; i < whole; i += kPerVec * kThreads) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + (int64_t)(begin + i) * (TYPE == QMM_F32 ? 4 : 2));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float v[kPerVec];
#pragma unroll
    for (int q = 0; q < kPerVec; ++q) {
      if constexpr (TYPE == QMM_F32) v[q] = take(__uint_as_float(u[q]));
      else if constexpr (TYPE == QMM_BF16) v[q] = take(__uint_as_float(q & 1 ? u[q / 2] & 0xFFFF0000u : u[q / 2] << 16));
      else v[q] = take(__half2float(__ushort_as_half((uint16_t)(u[q / 2] >> (16 * (q & 1))))));
    }
#pragma unroll
    for (int q = 0; q < kPerVec; q += 4)
      *reinterpret_cast<float4*>(&R.x[i + q]) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
  }
  for (int i = whole + threadIdx.x; i < n; i += kThreads) R.x[i] = take(logit<TYPE>(row, begin + i));
  for (int i = n + threadIdx.x; i < slice; i += kThreads) R.x[i] = -INFINITY;
  __syncthreads();
  float own = -INFINITY;   // this thread's largest, and where
  int where = 0;
#pragma unroll 4
  for (int j = 0; j < run; ++j) {
    const float v = R.mine[j];
    if (v > own) {
      own = v;
      where = j;
    }
  }
  R.own = key_of(own);
  uint32_t top_key = R.own, argmax = (uint32_t)(R.first + where), lowest = own > -INFINITY ? R.own : 0xFFFFFFFFu;
  R.best_of(top_key, argmax, lowest);
  const float top = float_of(top_key), temperature = a.temperature ? a.temperature[t] : 1.0f;
  R.top = top;
  if (top == -INFINITY || !(temperature > 0.0f)) {
    if (R.rank == 0 && threadIdx.x == 0) {
      a.tokens[t] = top == -INFINITY ? -1 : (int)argmax;
      if (a.logprobs) a.logprobs[t] = top == -INFINITY ? -INFINITY : 0.0f;
    }
    R.sync();   // no CTA ends while another one reads its shared memory
    return;
  }
  R.c = slope_of(temperature);
  const int k = a.top_k ? a.top_k[t] : 0;
  const float p = a.top_p ? a.top_p[t] : 1.0f, mp = a.min_p ? a.min_p[t] : 0.0f;
  const bool by_k = k > 0 && k < V, by_p = p < 1.0f;
  u64 least = 0;   // the least weight that min_p lets stay
  if (mp > 0.0f) {
    bool exact = true;
    least = mp < 1.0f ? fraction_of(mp, u64(1) << kUnit, &exact) + !exact : u64(1) << kUnit;
  }

  // bins over the distance from the top
  float per = 0.0f;
  auto bins_over = [&](float span) {
    per = kBins / span;
    if (!(span > 0.0f && per < INFINITY)) per = 0.0f;   // one bin
  };
  auto distance_bin = [&](float v) -> int {
    const float d = (top - v) * per;
    return d >= kBins - 1 ? kBins - 1 : (int)d;   // (NaN: an infinite top itself, bin 0)
  };
  auto half_bin = [&](float v) { return distance_bin(v) >> 1; };   // of weights
  // the lowest key that a token within d of the top can have
  // (the last term: where d has few bits)
  auto key_within = [&](float d) {
    return top < INFINITY ? key_of(top - d * (1.0f + 1e-5f) - fabsf(top) * 1e-6f - 0x1p-147f) : top_key;
  };
  // a key that no token of the distance bins up to b lies below; the last bin has all that lies further down.  (keys_of() takes
  // 3000 cycles more for the very key: 1 row 18.3 us, 18.8.)
  auto key_down_to = [&](int b) { return b >= kBins - 1 ? 0u : key_within((float)(b + 1) / per); };
  auto distance_to = [&](uint32_t key) { return top - float_of(max(key, 0x00800000u)); };   // of a finite key

  // what stays: keys above cut, and those on it up to the index last
  uint32_t cut = 0;
  int last = 0x7fffffff;
  auto in = [&](float v, int i) {
    const uint32_t key = key_of(v);
    return key > cut || (key == cut && i <= last);
  };
  auto everything = [](float, int) { return true; };

  if (by_k) {
    int b;
    u64 above;
    bins_over(distance_to(lowest));
    if (k <= kThreads * R.C) {
      // k threads have a token at or above the k-th largest of the threads' largest: nothing below it stays
      R.histogram_of(own, distance_bin);
      R.find<uint32_t>((u64)k, &b, &above);
      const Raised now = R.raise_floor(key_down_to(b), everything);
      if (now == kAlone) end_alone(a, R, t, k, p, mp, least, 0);
      if (now != kSpread) return;
      bins_over(distance_to(R.floor));
    }
    R.histogram<uint32_t>(everything, distance_bin);
    if (R.find<uint32_t>((u64)k, &b, &above)) {   // (an infinite top's floor may leave fewer: all of them stay)
      Keys r = R.keys_of(b, b, distance_bin);
      R.settle<uint32_t>(r, (u64)k - above, everything, &cut, &last);
    }
  }
  if (by_p) {
    // The top alone weighs 1, so tokens of less than (1 - top_p) / V cannot make up what may go: the border is within
    // `reach` of the top, and so are all bins but the last one, which has what lies further down too.
    const float reach = log2f((float)V / (1.0f - fmaxf(p, 0.0f))) * 1.001f / R.c.hi / R.c.unit;
    bins_over(fminf(reach, distance_to(R.floor)));
    R.histogram<u64>(in, half_bin);
    const u64 all = R.mass_of_bins();
    bool exact;
    u64 target = fraction_of(fmaxf(p, 0.0f), all, &exact);
    target = max(u64(1), target + !exact);
    int b;
    u64 above;
    R.find<u64>(target, &b, &above);
    Keys r = R.keys_of(2 * b, 2 * b + 1, distance_bin);
    r.hi = min(r.hi, top_key);
    const Raised now = R.raise_floor(max(cut, r.lo), in);
    if (now == kAlone) end_alone(a, R, t, R.listed, p, mp, least, all);
    if (now != kSpread) return;
    r.lo = max(r.lo, R.floor);
    uint32_t key;
    int index;
    R.settle<u64>(r, target - above, in, &key, &index);
    cut = key;
    last = index;
  } else if (mp > 0.0f && R.c.hi > 0.0f) {   // (a slope of 0: all weights are 1, and none is far enough down)
    // What stays weighs min_p less a weight's rounding at least; a millionth of it less again covers fp32's own in the distance,
    // which is 0 where min_p is 1.
    const float lightest = fmaxf(__fmaf_rn(fminf(mp, 1.0f), 1.0f - 0x1p-20f, -0x1p-40f), 0x1p-44f);
    const Raised now = R.raise_floor(max(cut, key_within(-log2f(lightest) / R.c.hi / R.c.unit)), in);
    if (now == kAlone) end_alone(a, R, t, R.listed, p, mp, least, 0);
    if (now != kSpread) return;
  }
  if (mp > 1.0f) {
    cut = top_key;
    last = (int)argmax;
  }

  // what stays, and the token
  u64 sure = 0;
  R.each([&](float v, int i) {
    if (!in(v, i)) return;
    const u64 w = R.weight_of(v);
    if (w >= least) sure += w;
  });
  u64 total;
  const u64 before = R.cluster_before(sure, &total);
  bool exact;
  const u64 goal = fraction_of(fminf(fmaxf(a.uniform[t], 0.0f), 0x1.fffffep-1f), total, &exact);
  const uint32_t who = __ballot_sync(0xffffffffu, before <= goal && before + sure > goal);
  if (who) {   // the warp goes through the tokens of its thread that has it
    const int lane = threadIdx.x & 31, from = __ffs(who) - 1;
    u64 at = __shfl_sync(0xffffffffu, before, from);
    const int off = __shfl_sync(0xffffffffu, (int)(R.mine - R.x), from) - (int)(R.mine - R.x);   // of its tokens from this thread's
    const int len = __shfl_sync(0xffffffffu, R.run, from), first = __shfl_sync(0xffffffffu, R.first, from);
    for (int j0 = 0; j0 < len; j0 += 32) {
      const bool here = j0 + lane < len;
      const float v = here ? R.mine[off + j0 + lane] : -INFINITY;
      const int i = !here ? 0 : R.index ? R.index[off + j0 + lane] : first + j0 + lane;
      u64 w = here && key_of(v) >= R.floor && in(v, i) ? R.weight_of_one(v) : 0;
      if (w < least) w = 0;
      const u64 upto = at + warp_upto(w);
      const uint32_t hit = __ballot_sync(0xffffffffu, upto > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          a.tokens[t] = i;
          if (a.logprobs) a.logprobs[t] = logprob_of(v, top, R.c, total, S.table);
        }
        break;
      }
      at = __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  R.sync();   // no CTA ends while another one reads its shared memory
}

// A thread per stream.
__global__ void __launch_bounds__(128) accept_kernel(const __grid_constant__ qmm_sample_args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.B) return;
  const int r0 = a.row_starts[b], r1 = a.row_starts[b + 1];
  int n = 0, next = -1;
  if (r0 < 0 || r1 < r0 || r1 > a.T) {
    atomicOr(&g_status, kErrIndex);
  } else if (r1 > r0) {
    while (r0 + n + 1 < r1 && a.tokens[r0 + n] == a.fed[r0 + n + 1]) ++n;
    next = a.tokens[r0 + n];
  }
  a.accepted[b] = n;
  a.next[b] = next;
}

// CTAs of a row.  A slice of at most 16384 floats leaves room for a second CTA on the SM, whose work covers this one's
// barriers; with few rows, as many CTAs as find an SM, down to slices of 1024.
int cluster_of(int T, int V, int sms) {
  int C = 1;
  while (C < kMaxCluster && (V + C - 1) / C > 16384) C *= 2;
  while (C < kMaxCluster && (int64_t)T * C * 2 <= sms && V / C >= 2048) C *= 2;
  return C;
}

template <int TYPE>
cudaError_t launch(const qmm_sample_args& a, cudaStream_t stream) {
  static DeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, cudaSuccess, [] {
    const cudaError_t f = cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return f != cudaSuccess ? f : cudaFuncSetAttribute(sample_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)(sizeof(Cta) + kMaxRun * kThreads * sizeof(float)));
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms < 1) return cudaErrorNoDevice;
  const int C = cluster_of(a.T, a.V, sms);
  const int run = ((a.V + C - 1) / C + kThreads - 1) / kThreads | 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.T * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Cta) + (size_t)run * kThreads * sizeof(float);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  // 16 bytes at a time where every row's slices begin on such a boundary (a slice is a multiple of 512 logits)
  const int64_t size = a.type == QMM_F32 ? 4 : 2;
  const int vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (a.T == 1 || a.ld * size % 16 == 0);
  return cudaLaunchKernelEx(&cfg, sample_kernel<TYPE>, a, run, vec);
}

}  // namespace

cudaError_t launch_sample(const qmm_sample_args& a, cudaStream_t stream) {
  if (a.T > 0) {
    const cudaError_t e = a.type == QMM_F32    ? launch<QMM_F32>(a, stream)
                          : a.type == QMM_BF16 ? launch<QMM_BF16>(a, stream)
                                               : launch<QMM_F16>(a, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.B == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.B + 127) / 128);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_kernel, a);
}

cudaError_t read_and_clear_sample_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
