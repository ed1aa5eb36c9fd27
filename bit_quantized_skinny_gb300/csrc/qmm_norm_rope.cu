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
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kThreads = 64;

struct Params {
  qmm_norm_rope_args a;
  int parts;   // CTAs of one row
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

// CTA (t, part): the heads part, part + groups * parts, ... of row t (queries, then keys, then
// values).
template <int D, int IN, int OUT, int AHEAD>
__global__ void __launch_bounds__(kThreads, AHEAD == 2 ? 16 : 0) norm_rope_kernel(const __grid_constant__ Params P) {
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
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __fmaf_rn(x[u][k], x[u][k], sum);
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (is_q || is_k) {
        const float r = rsqrtf(sum * (1.0f / D) + a.eps);
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
      if (turns && (is_q || is_k))
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = __fmaf_rn(x[u][k], c[k], y[k] * s[k]);
      if (is_q) store8<OUT>(a.Q_out, t * a.ldqo + (int64_t)h * D + 8 * l, x[u]);
      else if (slot >= 0 && is_k) store8<OUT>(a.K_cache, (slot * a.Hk + h - a.Hq) * D + 8 * l, x[u]);
      else if (slot >= 0 && h < heads) store8<OUT>(a.V_cache, (slot * a.Hk + h - a.Hq - a.Hk) * D + 8 * l, x[u]);
    }
  }
}

template <int D, int IN, int OUT, int AHEAD>
cudaError_t launch_ahead(const qmm_norm_rope_args& a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int heads = a.Hq + (a.V ? 2 : 1) * a.Hk;
  const int most = (heads + kGroups - 1) / kGroups;
  int parts = 1;
  while (parts < most && (int64_t)a.T * parts < 2048) ++parts;   // few rows: a CTA per few heads
  Params P{a, parts};
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
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, IN, OUT, AHEAD>, P);
}

// Two heads at a time for many fp32 rows, unless a group's last pair would stand half empty after few pairs:
// a row's heads take `steps` of a CTA's groups.  Heads of 128: 16384 rows of 56 heads (14 steps) 104 us, one at
// a time 114; 3000 rows 25.6 (28.0); 1024 rows 10.7 (10.2); 16384 rows of 8 heads (2) 29.2 (30.7).  Heads of 64:
// 24000 rows of 56 (7) 81 (87); 2049 rows of 24 (3) 5.1 (4.5), 16384 rows 33.0 (32.3).  Heads of 256: 4000
// rows of 10 (5) 15.4 (14.6).  Rows of 16 bits take one at a time (16384 rows of 56 heads of 128 117 us, two
// 124; 2311 rows of 30 heads of 64 5.8, 6.3): twice the instructions a byte, which fill half the issue slots,
// and the waits for loads between them (two would gain 5 to 7 % with 8 heads a row).
template <int D, int IN, int OUT>
cudaError_t launch(const qmm_norm_rope_args& a, cudaStream_t stream) {
  if constexpr (IN == QMM_F32) {
    constexpr int kGroups = kThreads / (D / 8);
    const int steps = (a.Hq + (a.V ? 2 : 1) * a.Hk + kGroups - 1) / kGroups;
    if (a.T > 2048 && (steps % 2 == 0 || steps >= 7)) return launch_ahead<D, IN, OUT, 2>(a, stream);
  }
  return launch_ahead<D, IN, OUT, 1>(a, stream);
}

template <int D, int IN>
cudaError_t launch_out(const qmm_norm_rope_args& a, cudaStream_t stream) {
  return a.out_type == QMM_BF16 ? launch<D, IN, QMM_BF16>(a, stream) : launch<D, IN, QMM_F16>(a, stream);
}

template <int D>
cudaError_t launch_in(const qmm_norm_rope_args& a, cudaStream_t stream) {
  if (a.in_type == QMM_F32) return launch_out<D, QMM_F32>(a, stream);
  if (a.in_type == QMM_BF16) return launch_out<D, QMM_BF16>(a, stream);
  return launch_out<D, QMM_F16>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const qmm_norm_rope_args& a, cudaStream_t stream) {
  if (a.D == 64) return launch_in<64>(a, stream);
  if (a.D == 128) return launch_in<128>(a, stream);
  return launch_in<256>(a, stream);
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
