// qmm_sample.cu — the token of every row from its logits, and how many drafted tokens stand (qmm_sample).
//
// Weights.  w = exp((x - max) / T) as an integer W = w 2^43, to a unit or two: two neighbouring tokens lie 2^-18 of the
// sum apart where 250000 share it, so fp32 weights would pick the wrong one in every hundredth row; integers
// also make every sum independent of its order.  t = (x - max) log2(e) / T is formed in two fp32 words
// (the difference and the product are exact but for 2^-45), split into -(n + j/2048) and a rest g of at most 2^-12, and
//     W = (2^43 2^(-j/2048) 2^g) >> n,     2^g - 1 = g ln2 + (g ln2)^2/2 + (g ln2)^3/6
// with 2^(43 - j/2048) from a table and the correction as a 32-bit integer.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kThreads = 1024;
constexpr int kUnit = 43;              // a weight of 1 is 2^kUnit; kMaxV of them stay below 2^62
constexpr int kSteps = 2048;           // of the table, for one octave
static_assert(QMM_SAMPLE_MAX_V <= (1 << 19), "sums of weights");

using u64 = unsigned long long;

// 2^(43 - j/2048), j = 0 .. 2047: 2^(-1/2048) by eleven integer square roots of 1/2, then its powers, with 62 bits
// behind the point (an error of 2^-51 at the end).
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
  for (int k = 0; k < 11; ++k) r = isqrt((unsigned __int128)r << kQ);
  Table t{};
  u64 at = u64(1) << kQ;
  for (int j = 0; j < kSteps; ++j) {
    t.v[j] = ((at >> (kQ - kUnit - 1)) + 1) >> 1;
    at = (u64)(((unsigned __int128)at * r + ((unsigned __int128)1 << (kQ - 1))) >> kQ);
  }
  return t;
}
__device__ constexpr Table kTable = make_table();

// log2(e) / T in two fp32 words.
struct Slope {
  float hi, lo;
};
__device__ __forceinline__ Slope slope_of(float temperature) {
  const double c = 1.4426950408889634074 / (double)temperature;
  const float hi = (float)c;
  return Slope{hi, hi < INFINITY ? (float)(c - (double)hi) : 0.0f};
}

// The weight of logit x (not NaN, not above top) as an integer.
__device__ __forceinline__ u64 weight(float x, float top, Slope c, const u64* table) {
  if (x == top) return u64(1) << kUnit;   // (also where both are infinite)
  const float d = x - top;                // two words: the rounded difference and what it lost
  const float b = d - x, lost = (x - (d - b)) + (-top - b);
  const float th = d * c.hi;
  if (!(th > -46.0f)) return 0;           // below half a unit (and any difference that is not finite)
  const float tl = __fmaf_rn(d, c.hi, -th) + __fmaf_rn(d, c.lo, lost * c.hi);
  const float kMagic = 12582912.0f;       // 1.5 * 2^23: added, a float of at most 2^22 has its integer in its low bits
  const float u = __fmaf_rn(th, -(float)kSteps, kMagic);
  const uint32_t k = __float_as_uint(u) - __float_as_uint(kMagic);
  const float gh = __fmaf_rn(u - kMagic, 1.0f / kSteps, th);
  // 2^g - 1 in units of 2^-43: the leading product exact in two words
  constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-09f;
  const float p = gh * kLn2Hi;
  const float low = __fmaf_rn(gh, kLn2Hi, -p) + __fmaf_rn(gh, kLn2Lo, tl * kLn2Hi) +
                    gh * gh * __fmaf_rn(gh, 0.0555041087f, 0.2402265070f);
  const float big = p * 0x1p43f, v = __fmaf_rn(big, 0x1p-9f, kMagic), vi = v - kMagic;
  const float rest = __fmaf_rn(vi, -0x1p9f, big) + low * 0x1p43f;
  const int grow = ((int)(__float_as_uint(v) - __float_as_uint(kMagic)) << 9) +
                   (int)(__float_as_uint(rest + kMagic) - __float_as_uint(kMagic));
  const u64 base = table[k & (kSteps - 1)];
  const int n = (int)(k / kSteps);
  const long long more = ((long long)(int)(base >> 13) * grow + (1 << 29)) >> 30;   // base * grow / 2^43
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

__device__ __forceinline__ u64 block_sum(u64 v, u64* space) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) space[threadIdx.x >> 5] = v;
  __syncthreads();
  v = space[threadIdx.x & 31];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Sum over the threads before this one.
__device__ __forceinline__ u64 block_before(u64 v, u64* space) {
  u64 upto = v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  __syncthreads();
  if (lane == 31) space[warp] = upto;
  __syncthreads();
  u64 before = upto - v;
  for (int w = 0; w < warp; ++w) before += space[w];
  return before;
}

// A CTA per row; each step of the two searches (for the top-k and the top-p border among the keys) is a pass.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ qmm_sample_args a) {
  __shared__ u64 space[32];
  __shared__ int found;
  const int t = blockIdx.x, V = a.V;
  const void* row = static_cast<const uint8_t*>(a.logits) + t * a.ld * (TYPE == QMM_F32 ? 4 : 2);
  const int per = (V + kThreads - 1) / kThreads, i0 = min(V, (int)threadIdx.x * per), i1 = min(V, i0 + per);
  // the largest logit and its lowest index
  u64 best = 0;
  for (int i = i0; i < i1; ++i) {
    const u64 v = (u64)key_of(logit<TYPE>(row, i)) << 32 | (0xFFFFFFFFu - (uint32_t)i);
    best = v > best ? v : best;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const u64 v = __shfl_xor_sync(0xffffffffu, best, off);
    best = v > best ? v : best;
  }
  if ((threadIdx.x & 31) == 0) space[threadIdx.x >> 5] = best;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  for (int w = 0; w < 32; ++w) best = space[w] > best ? space[w] : best;
  const int first = (int)(0xFFFFFFFFu - (uint32_t)best);
  const float top = logit<TYPE>(row, first), temperature = a.temperature ? a.temperature[t] : 1.0f;
  if (top == -INFINITY || !(temperature > 0.0f)) {
    if (threadIdx.x == 0) {
      a.tokens[t] = top == -INFINITY ? -1 : first;
      if (a.logprobs) a.logprobs[t] = top == -INFINITY ? -INFINITY : 0.0f;
    }
    return;
  }
  const Slope c = slope_of(temperature);
  auto W = [&](float x) { return x == -INFINITY ? u64(0) : weight(x, top, c, kTable.v); };

  // top_k: tokens above the key kk, and the first rk of those on it
  const int k = a.top_k ? a.top_k[t] : 0;
  uint32_t kk = 0;
  u64 rk = ~u64(0);
  if (k > 0 && k < V) {
    for (int bit = 31; bit >= 0; --bit) {
      u64 n = 0;
      for (int i = i0; i < i1; ++i) n += key_of(logit<TYPE>(row, i)) >= (kk | 1u << bit);
      if (block_sum(n, space) >= (u64)k) kk |= 1u << bit;
    }
    u64 n = 0;
    for (int i = i0; i < i1; ++i) n += key_of(logit<TYPE>(row, i)) > kk;
    rk = k - block_sum(n, space);
  }
  const float p = a.top_p ? a.top_p[t] : 1.0f;
  if (p < 1.0f) {
    // the sum of what top_k left, and what has to lie before the first token that goes
    u64 sum = 0, ties = 0;
    for (int i = i0; i < i1; ++i) {
      const float x = logit<TYPE>(row, i);
      if (key_of(x) > kk) sum += W(x);
      ties += key_of(x) == kk;
    }
    sum = block_sum(sum, space);
    ties = block_sum(ties, space);
    if (kk) sum += min(rk, ties) * W(__uint_as_float(kk & 0x80000000u ? kk & 0x7FFFFFFFu : ~kk));
    bool exact;
    u64 target = fraction_of(fmaxf(p, 0.0f), sum, &exact);
    target = max(u64(1), target + !exact);
    // the lowest key with less than that above it
    uint32_t kp = 0xFFFFFFFFu;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t lower = kp & ~(1u << bit);
      u64 above = 0;
      for (int i = i0; i < i1; ++i) {
        const float x = logit<TYPE>(row, i);
        if (key_of(x) > lower) above += W(x);
      }
      if (block_sum(above, space) < target) kp = lower;
    }
    if (kp >= kk) {
      u64 above = 0;
      for (int i = i0; i < i1; ++i) {
        const float x = logit<TYPE>(row, i);
        if (key_of(x) > kp) above += W(x);
      }
      above = block_sum(above, space);
      const u64 one = W(__uint_as_float(kp & 0x80000000u ? kp & 0x7FFFFFFFu : ~kp));
      const u64 rp = one ? (target - above + one - 1) / one : ~u64(0);
      rk = kp == kk ? min(rk, rp) : rp;
      kk = kp;
    }
  }
  u64 least = 0;
  const float mp = a.min_p ? a.min_p[t] : 0.0f;
  if (mp > 0.0f) {
    bool exact = true;
    least = mp < 1.0f ? fraction_of(mp, u64(1) << kUnit, &exact) + !exact : u64(1) << kUnit;
    if (mp > 1.0f) {
      kk = key_of(top);
      rk = 1;
    }
  }

  // what stays, and the token
  u64 ties = 0;
  for (int i = i0; i < i1; ++i) ties += key_of(logit<TYPE>(row, i)) == kk;
  const u64 ties_before = block_before(ties, space);
  auto stays = [&](float x, u64& tie) -> u64 {
    const uint32_t key = key_of(x);
    if (key < kk || (key == kk && tie++ >= rk)) return 0;
    const u64 w = W(x);
    return w >= least ? w : 0;
  };
  u64 sum = 0, tie = ties_before;
  for (int i = i0; i < i1; ++i) sum += stays(logit<TYPE>(row, i), tie);
  const u64 total = block_sum(sum, space), before = block_before(sum, space);
  bool exact;
  const float u = fminf(fmaxf(a.uniform[t], 0.0f), 0x1.fffffep-1f);
  const u64 target = fraction_of(u, total, &exact);
  if (before <= target && before + sum > target) {
    u64 at = before;
    tie = ties_before;
    for (int i = i0; i < i1; ++i) {
      const float x = logit<TYPE>(row, i);
      at += stays(x, tie);
      if (at > target) {
        a.tokens[t] = i;
        if (a.logprobs)
          a.logprobs[t] = (float)((x == top ? 0.0 : ((double)x - (double)top) / (double)temperature) -
                                  log((double)total * 0x1p-43));
        break;
      }
    }
  }
}

// A thread per stream.
__global__ void __launch_bounds__(128) accept_kernel(const __grid_constant__ qmm_sample_args a) {
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

}  // namespace

cudaError_t launch_sample(const qmm_sample_args& a, cudaStream_t stream) {
  if (a.T > 0) {
    if (a.type == QMM_F32) sample_kernel<QMM_F32><<<a.T, kThreads, 0, stream>>>(a);
    else if (a.type == QMM_BF16) sample_kernel<QMM_BF16><<<a.T, kThreads, 0, stream>>>(a);
    else sample_kernel<QMM_F16><<<a.T, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.B > 0) accept_kernel<<<(a.B + 127) / 128, 128, 0, stream>>>(a);
  return cudaGetLastError();
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
