// qmm_norm_rope.cu — from the q, k and v projections' results to the attention's operands
// (qmm_norm_rope): for every query and key head x of D values
//     y = x / sqrt(mean(x^2) + eps) * weight,   (a, b) -> (a c - b s, b c + a s) for its pairs,
// the values converted only; keys and values go to their cache slots.
//
// A head is one group of D/8 lanes, 8 neighbouring values a lane: the sum of squares is a
// butterfly over the group, and the partner of a value lies in the same lane (neighbouring pairs)
// or in the lane rot/16 away (halves).  A group takes several heads of its row, the next
// ones in flight while it works on these, the first ones while the row's position and slot arrive: the
// kernel is bound by the bytes it reads and writes (16384 rows of 40 + 16 heads of 128, fp32 to bf16:
// 104 us, 6.9 TB/s; without the loads ahead 144 us).
//
// Into a 4-bit cache (qmm_norm_rope_fp4) a block of 16 values is two neighbouring lanes, and the codes are
// those of the formulas in real numbers, rounded to fp32 where the definition says so: a code is a step of
// a third of the value, and it must not hang on the order of a sum.  The fp32 arithmetic knows its error;
// where a border of a code or of a scale lies within it (one head of some thousand), the head is computed
// again in 64 bits.  16384 rows of 40 + 16 heads of 128, fp32 to bf16 queries: 133 us, 460 MB, 3.5 TB/s; bound by the
// instructions of the two roundings (an interval's both ends are encoded) and, with few rows, by the one head in 64
// bits.  64 registers, so that an SM holds 16 CTAs: 129 us, 180 with 80.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kThreads = 64;

struct Params {
  qmm_norm_rope_args a;
  int parts;   // CTAs of one row
  int page_size, page_shift;   // of a 4-bit cache, and its tensors' scales
  float k_scale, v_scale;
};

// 8 values of in_type at p as fp32.  Plain loads throughout this kernel: it starts while the kernel ahead
// may still be writing these buffers, so they are not read-only for its lifetime, and only a load that
// is not taken for invariant stays behind the wait for that kernel.
template <int IN>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  if constexpr (IN == QMM_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 u = p[0], v = p[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (IN == QMM_BF16) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
  }
}

template <int OUT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&y)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (OUT == QMM_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest bits of |y| over a block: of two lanes' eight values each.  An infinity or NaN has more than
// any finite value.
__device__ __forceinline__ uint32_t block_top(const float (&y)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(y[k]) & 0x7FFFFFFFu);
  return max(top, __shfl_xor_sync(0xffffffffu, top, 1));
}

// Bit 0 of every nibble whose magnitude is 0.
__device__ __forceinline__ uint32_t zeros_of(uint32_t codes) { return ~(codes | codes >> 1 | codes >> 2) & 0x11111111u; }

// The codes and the scale of the lane's half of a block, by the definition: every quotient one fp32 rounding.
__device__ __forceinline__ void encode(const float (&y)[8], float tensor_scale, uint32_t& codes, uint32_t& scale) {
  const uint32_t top = block_top(y);
  scale = kv4::kScaleNaN;
  codes = 0;
  if (top >= 0x7F800000u) return;
  scale = kv4::e4m3_code(__fdiv_rn(__fdiv_rn(__uint_as_float(top), 6.0f), tensor_scale));
  const float S = kv4::e4m3_value(scale) * tensor_scale;
  if (!(S > 0.0f)) return;
  float t[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) t[k] = __fdiv_rn(y[k], S);
  codes = kv4::e2m1_codes(t);
  codes &= ~(zeros_of(codes) << 3);
}

// The same by one reciprocal, from values that are off by at most err; false: another code or scale is
// within reach, and encode() has to decide.  Relative, for the roundings of the quotients here and in encode(): a code's
// three (2^-24 each), a scale's seven.
__device__ __forceinline__ bool encode_fast(const float (&y)[8], const float (&err)[8], float tensor_scale,
                                            uint32_t& codes, uint32_t& scale) {
  constexpr float kCodeSlack = 0x1p-22f, kScaleSlack = 0x1p-21f;
  const uint32_t top = block_top(y);
  float worst = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) worst = fmaxf(worst, err[k]);
  worst = fmaxf(worst, __shfl_xor_sync(0xffffffffu, worst, 1));
  scale = kv4::kScaleNaN;
  codes = 0;
  if (top >= 0x7F800000u) return true;
  const float a = __uint_as_float(top), to = __frcp_rn(6.0f) * __frcp_rn(tensor_scale);
  scale = kv4::e4m3_code((a + worst) * to * (1.0f + kScaleSlack));
  bool sure = scale == kv4::e4m3_code(fmaxf(a - worst, 0.0f) * to * (1.0f - kScaleSlack));
  const float S = kv4::e4m3_value(scale) * tensor_scale, inv = __frcp_rn(S);
  if (!(S > 0.0f)) return sure;
  float lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = y[k] * inv, off = __fmaf_rn(fabsf(t), kCodeSlack, err[k] * inv);
    lo[k] = t - off;
    hi[k] = t + off;
  }
  codes = kv4::e2m1_codes(hi);
  codes &= ~(zeros_of(codes) << 3);   // 0 has no sign, so that the sign of a value that may be either is no border
  uint32_t other = kv4::e2m1_codes(lo);
  other &= ~(zeros_of(other) << 3);
  return sure && codes == other;
}

// m^(-1/2) to 2^-50: the fp32 one of m brought into [1, 4), and two steps of Newton's iteration, r += r (1 - m r^2) / 2.
__device__ __forceinline__ double inv_root(double m) {
  if (!(m > 0.0) || m > 1e300) return rsqrtf((float)m);   // 0, infinity and NaN (finite operands stay below 1e80)
  const int e = ((__double2hiint(m) >> 20) - 1023) & ~1;
  const double f = m * __hiloint2double((1023 - e) << 20, 0);
  double r = rsqrtf((float)f);
#pragma unroll
  for (int step = 0; step < 2; ++step) r = __fma_rn(r * 0.5, __fma_rn(-f * r, r, 1.0), r);
  return r * __hiloint2double((1023 - e / 2) << 20, 0);
}

// A key's head in some thousands comes here, and values that lie exactly between two codes, as they do where the tensor's
// scale is a short decimal.  (A 64-bit operation takes 16 cycles a warp: 2311 rows of 30 heads of 64 take 13.1 us,
// 8.7 with no key's head here, 21.5 when values went the 64 bits' way too.)
//
// The codes (x) and the scale (y) of the lane's eight values by the definition, a key's from 64 bits where `keys`: again from
// the operands, rounded to fp32 once.  Every lane of the warp takes part.  (Values go in and out by value: an array that a
// call has the address of would live in memory in the kernel's loop too.)
struct Eight {
  float x[8];
};
template <int D, int IN>
__device__ __noinline__ uint2 decide(const qmm_norm_rope_args& a, int64_t t, int h, int l, Eight in, bool keys,
                                     float tensor_scale) {
  if (keys) {
    constexpr int kLanes = D / 8;
    const bool is_k = h >= a.Hq && h < a.Hq + a.Hk, turns = 8 * l < a.rot;
    float x[8];
    load8<IN>(a.K, t * a.ldk + (int64_t)(is_k ? h - a.Hq : 0) * D + 8 * l, x);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = __fma_rn((double)x[k], (double)x[k], sum);
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const double r = inv_root(sum * (1.0 / D) + (double)a.eps);   // (off by less than 2^-50, as the products are)
    double y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (double)x[k] * (a.k_weight ? (double)a.k_weight[8 * l + k] : 1.0) * r;
    const int half = a.rot / 2, step = half / 8;
    const int from = (threadIdx.x & 31) + (8 * l < half ? step : (turns ? -step : 0));
    int64_t pos = turns ? a.positions[t] : 0;
    if (pos < 0 || pos >= a.max_pos) pos = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = 8 * l + k, pair = a.interleaved ? i / 2 : i < half ? i : i - half;   // of the value
      const bool second = a.interleaved ? i & 1 : i >= half;
      double other = __shfl_sync(0xffffffffu, y[k], from);
      if (a.interleaved) other = y[k ^ 1];
      double z = y[k];
      if (turns) {
        const double c = a.cos_sin[pos * a.rot + pair], s = a.cos_sin[pos * a.rot + half + pair];
        z = second ? z * c + other * s : z * c - other * s;
      }
      if (is_k) in.x[k] = (float)z;
    }
  }
  uint32_t codes, scale;
  encode(in.x, tensor_scale, codes, scale);
  return make_uint2(codes, scale);
}

// CTA (t, part): the heads part, part + groups * parts, ... of row t (queries, then keys, then
// values).
template <int D, int IN, int OUT, int AHEAD, bool FP4>
__global__ void __launch_bounds__(kThreads, AHEAD == 2 || FP4 ? 16 : 0) norm_rope_kernel(const __grid_constant__ Params P) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  // launched early behind a launch that allows it: memory is read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const qmm_norm_rope_args& a = P.a;
  const int64_t t = blockIdx.x / P.parts;
  const int part = blockIdx.x - (int)t * P.parts;
  const int l = threadIdx.x % kLanes;        // values 8 l .. 8 l + 7 of the head
  const int heads = a.Hq + (a.V ? 2 : 1) * a.Hk;
  const int mine = threadIdx.x / kLanes, stride = kGroups * P.parts;
  auto ask = [&](int h0, float (&x)[AHEAD][8]) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int h = h0 + u * stride + mine;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[u][k] = 0.0f;
      if (h < a.Hq) load8<IN>(a.Q, t * a.ldq + (int64_t)h * D + 8 * l, x[u]);
      else if (h < a.Hq + a.Hk) load8<IN>(a.K, t * a.ldk + (int64_t)(h - a.Hq) * D + 8 * l, x[u]);
      else if (h < heads) load8<IN>(a.V, t * a.ldv + (int64_t)(h - a.Hq - a.Hk) * D + 8 * l, x[u]);
    }
  };
  float next[AHEAD][8];
  ask(part * kGroups, next);
  int64_t slot = -1;
  if (a.Hk > 0) {
    slot = a.slots[t];
    if (slot >= a.n_slots) {
      atomicOr(&g_status, kErrIndex);
      slot = -1;
    }
  }
  // the lane's cosines and sines: of pairs 4l .. 4l+3, or of the 8 pairs its values belong to
  float c[8], s[8];
  const bool turns = 8 * l < a.rot;
  const int half = a.rot / 2;
  if (turns) {
    int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.max_pos) {
      atomicOr(&g_status, kErrIndex);
      pos = 0;
    }
    const float* row = a.cos_sin + pos * a.rot;
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[2 * k] = c[2 * k + 1] = row[4 * l + k];
        s[2 * k + 1] = row[half + 4 * l + k];
        s[2 * k] = -s[2 * k + 1];
      }
    } else {
      const bool second = 8 * l >= half;
      const int i = second ? 8 * l - half : 8 * l;
      load8<QMM_F32>(row, i, c);
      load8<QMM_F32>(row, half + i, s);
      if (!second)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = -s[k];
    }
  }
  for (int h0 = part * kGroups; h0 < heads; h0 += AHEAD * stride) {   // same trips for every lane
    float x[AHEAD][8];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[u][k] = next[u][k];
    ask(h0 + AHEAD * stride, next);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (h0 + u * stride >= heads) break;   // (the warp's heads all lie behind)
      const int h = h0 + u * stride + mine;
      const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
      float sum = 0.0f;
      if constexpr (FP4) {   // (three roundings, not eight: see err)
        float pair[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) pair[k] = __fmaf_rn(x[u][2 * k], x[u][2 * k], x[u][2 * k + 1] * x[u][2 * k + 1]);
        sum = (pair[0] + pair[1]) + (pair[2] + pair[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = __fmaf_rn(x[u][k], x[u][k], sum);
      }
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (is_q || is_k) {
        const float r = FP4 ? __frsqrt_rn(sum * (1.0f / D) + a.eps) : rsqrtf(sum * (1.0f / D) + a.eps);
        float g[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        const float* w = is_q ? a.q_weight : a.k_weight;
        if (w) load8<QMM_F32>(w, 8 * l, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = x[u][k] * r * g[k];
      }
      // partners: every lane takes part in the shuffles
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = x[u][k ^ 1];
      } else {
        const int step = half / 8;   // lanes between the halves
        const int from = (threadIdx.x & 31) + (8 * l < half ? step : (turns ? -step : 0));
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(0xffffffffu, x[u][k], from);
      }
      float err[8];   // of x, as the 4-bit codes have to know it
      if constexpr (FP4) {
        // in units of 2^-24, on the terms that are added: half of the mean's roundings (a square's, three and log2(D/8) sums', eps':
        // 10 at most), the root's, the two products', the rotation's two: 10; and the error's own roundings
#pragma unroll
        for (int k = 0; k < 8; ++k)
          err[k] = is_k ? 0x1.5p-21f * (turns ? __fmaf_rn(fabsf(x[u][k]), fabsf(c[k]), fabsf(y[k] * s[k])) : fabsf(x[u][k])) : 0.0f;
      }
      if (turns && (is_q || is_k))
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = __fmaf_rn(x[u][k], c[k], y[k] * s[k]);
      if constexpr (FP4) {
        if (is_q) store8<OUT>(a.Q_out, t * a.ldqo + (int64_t)h * D + 8 * l, x[u]);
        if (h0 + u * stride + kGroups > a.Hq) {   // some lane of the CTA holds a key or a value
          const float tensor_scale = is_k ? P.k_scale : P.v_scale;
          uint32_t codes, scale;
          const bool sure = encode_fast(x[u], err, tensor_scale, codes, scale);
          const bool mine_too = !is_q && h < heads;
          const bool in_range = !is_k || (sum < 1e38f && sum * (1.0f / D) + a.eps > 1e-30f);   // of the fp32 arithmetic
          if (__any_sync(0xffffffffu, mine_too && !(sure && in_range))) {
            Eight now;
#pragma unroll
            for (int k = 0; k < 8; ++k) now.x[k] = x[u][k];
            const uint2 by = decide<D, IN>(a, t, h, l, now, __any_sync(0xffffffffu, is_k && !(sure && in_range)), tensor_scale);
            codes = by.x;
            scale = by.y;
          }
          if (mine_too && slot >= 0) {
            const bool key = is_k;
            const int hh = key ? h - a.Hq : h - a.Hq - a.Hk, i = (int)(slot & (P.page_size - 1));
            uint8_t* run = static_cast<uint8_t*>(key ? a.K_cache : a.V_cache) +
                           kv4::run_at(slot >> P.page_shift, hh, a.Hk, P.page_size, D);
            *reinterpret_cast<uint32_t*>(run + i * (D / 2) + 4 * l) = codes;
            if ((l & 1) == 0) run[P.page_size * (D / 2) + i * (D / 16) + (l >> 1)] = (uint8_t)scale;
          }
        }
      } else if (is_q) store8<OUT>(a.Q_out, t * a.ldqo + (int64_t)h * D + 8 * l, x[u]);
      else if (slot >= 0 && is_k) store8<OUT>(a.K_cache, (slot * a.Hk + h - a.Hq) * D + 8 * l, x[u]);
      else if (slot >= 0 && h < heads) store8<OUT>(a.V_cache, (slot * a.Hk + h - a.Hq - a.Hk) * D + 8 * l, x[u]);
    }
  }
}

// A 4-bit cache's page and scales; page_size 0: a cache of 16-bit values.
struct Fp4 {
  int page_size = 0;
  float k_scale = 1.0f, v_scale = 1.0f;
};

template <int D, int IN, int OUT, int AHEAD, bool FP4>
cudaError_t launch_ahead(const qmm_norm_rope_args& a, const Fp4& f, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int heads = a.Hq + (a.V ? 2 : 1) * a.Hk;
  const int most = (heads + kGroups - 1) / kGroups;
  int parts = 1;
  while (parts < most && (int64_t)a.T * parts < 2048) ++parts;   // few rows: a CTA per few heads
  Params P{a, parts, f.page_size, f.page_size ? 31 - __builtin_clz((unsigned)f.page_size) : 0, f.k_scale, f.v_scale};
  if ((int64_t)a.T * parts > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.T * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, IN, OUT, AHEAD, FP4>, P);
}

// Two heads at a time for many fp32 rows, unless a group's last pair would stand half empty after few pairs:
// a row's heads take `steps` of a CTA's groups.  Heads of 128: 16384 rows of 56 heads (14 steps) 104 us, one at
// a time 114; 3000 rows 25.6 (28.0); 1024 rows 10.7 (10.2); 16384 rows of 8 heads (2) 29.2 (30.7).  Heads of 64:
// 24000 rows of 56 (7) 81 (87); 2049 rows of 24 (3) 5.1 (4.5), 16384 rows 33.0 (32.3).  Heads of 256: 4000
// rows of 10 (5) 15.4 (14.6).  Rows of 16 bits take one at a time (16384 rows of 56 heads of 128 117 us, two
// 124; 2311 rows of 30 heads of 64 5.8, 6.3): twice the instructions a byte, which fill half the issue slots,
// and the waits for loads between them (two would gain 5 to 7 % with 8 heads a row).
template <int D, int IN, int OUT>
cudaError_t launch(const qmm_norm_rope_args& a, const Fp4& f, cudaStream_t stream) {
  if (f.page_size) return launch_ahead<D, IN, OUT, 1, true>(a, f, stream);   // (a second head would not fit 64 registers)
  if constexpr (IN == QMM_F32) {
    constexpr int kGroups = kThreads / (D / 8);
    const int steps = (a.Hq + (a.V ? 2 : 1) * a.Hk + kGroups - 1) / kGroups;
    if (a.T > 2048 && (steps % 2 == 0 || steps >= 7)) return launch_ahead<D, IN, OUT, 2, false>(a, f, stream);
  }
  return launch_ahead<D, IN, OUT, 1, false>(a, f, stream);
}

template <int D, int IN>
cudaError_t launch_out(const qmm_norm_rope_args& a, const Fp4& f, cudaStream_t stream) {
  return a.out_type == QMM_BF16 ? launch<D, IN, QMM_BF16>(a, f, stream) : launch<D, IN, QMM_F16>(a, f, stream);
}

template <int D>
cudaError_t launch_in(const qmm_norm_rope_args& a, const Fp4& f, cudaStream_t stream) {
  if (a.in_type == QMM_F32) return launch_out<D, QMM_F32>(a, f, stream);
  if (a.in_type == QMM_BF16) return launch_out<D, QMM_BF16>(a, f, stream);
  return launch_out<D, QMM_F16>(a, f, stream);
}

cudaError_t launch_any(const qmm_norm_rope_args& a, const Fp4& f, cudaStream_t stream) {
  if (a.D == 64) return launch_in<64>(a, f, stream);
  if (a.D == 128) return launch_in<128>(a, f, stream);
  return launch_in<256>(a, f, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const qmm_norm_rope_args& a, cudaStream_t stream) { return launch_any(a, Fp4{}, stream); }

cudaError_t launch_norm_rope_fp4(const qmm_norm_rope_fp4_args& a, cudaStream_t stream) {
  return launch_any(a.base, Fp4{a.page_size, a.k_scale, a.v_scale}, stream);
}

cudaError_t read_and_clear_norm_rope_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
