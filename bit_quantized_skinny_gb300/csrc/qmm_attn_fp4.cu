// qmm_attn_fp4.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, in pages of a 4-bit cache (qmm_attn_shared_fp4).
//
// A CTA of four warps per row and head; a warp takes every fourth key, a lane D/32 neighbouring values of it,
// with a running maximum and sum of the softmax; the warps are joined at the end.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_device.cuh"
#include "q4k_formats.cuh"
#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kWarps = 4;

struct Params {
  qmm_attn_fp4_args f;
  int page_shift, n_pages;
};

template <int D, int TYPE>
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(const __grid_constant__ Params P) {
  constexpr int kV = D / 32;
  const qmm_attn_args& a = P.f.base;
  const int t = blockIdx.x, head = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = head / (a.Hq / a.Hk);
  __shared__ int stream_s;
  __shared__ float o_s[kWarps][D], top_s[kWarps], sum_s[kWarps];
  if (threadIdx.x == 0) stream_s = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int r0 = a.row_starts[b], r1 = a.row_starts[b + 1], n = a.kv_lens[b];
    if (r0 < 0 || r1 < r0 || r1 > a.T || (b == 0 && r0 != 0) || n < 0 || n > (int)(a.pages_per_stream * a.page_size))
      atomicOr(&g_status, kErrIndex);
    else if (t >= r0 && t < r1) stream_s = b;
  }
  __syncthreads();
  const int b = stream_s;
  float q[kV], o[kV] = {}, top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const uint16_t raw = static_cast<const uint16_t*>(a.Q)[t * a.ldq + (int64_t)head * D + kV * lane + k];
    q[k] = (TYPE == QMM_BF16 ? __uint_as_float((uint32_t)raw << 16) : __half2float(__ushort_as_half(raw))) *
           (a.scale * P.f.k_scale);
  }
  auto value = [&](const uint8_t* run, int i, int k) -> float {
    const int d = kV * lane + k;
    const uint32_t c = run[i * (D / 2) + d / 2] >> (4 * (d & 1)) & 15u;
    uint32_t p[4];
    e2m1x8_pairs(c, p);
    return __half2float(__ushort_as_half((uint16_t)p[0])) *
           kv4::e4m3_value(run[a.page_size * (D / 2) + i * (D / 16) + d / 16]);
  };
  auto keys = [&](const int32_t* pages, int n) {
    for (int j = warp; j < n; j += kWarps) {
      const int page = pages[j >> P.page_shift], i = j & (a.page_size - 1);
      if (page < 0 || page >= P.n_pages) {
        atomicOr(&g_status, kErrIndex);
        continue;
      }
      const int64_t run = kv4::run_at(page, h, a.Hk, a.page_size, D);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kV; ++k) s = __fmaf_rn(q[k], value(static_cast<const uint8_t*>(a.K_cache) + run, i, k), s);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float best = fmaxf(top, s), keep = top == -INFINITY ? 0.0f : expf(top - best), p = expf(s - best);
      sum = __fmaf_rn(sum, keep, p);
#pragma unroll
      for (int k = 0; k < kV; ++k)
        o[k] = __fmaf_rn(p, value(static_cast<const uint8_t*>(a.V_cache) + run, i, k), o[k] * keep);
      top = best;
    }
  };
  if (b >= 0) {
    keys(a.prefix_pages, (int)a.prefix_len);
    const int n = a.kv_lens[b], m = a.row_starts[b + 1] - a.row_starts[b];
    keys(a.pages + b * a.pages_per_stream, min(n, max(0, n - m + t - a.row_starts[b] + 1)));
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) o_s[warp][kV * lane + k] = o[k];
  if (lane == 0) {
    top_s[warp] = top;
    sum_s[warp] = sum;
  }
  __syncthreads();
  float best = -INFINITY, total = 0.0f;
  for (int w = 0; w < kWarps; ++w) best = fmaxf(best, top_s[w]);
  for (int w = 0; w < kWarps; ++w) total += sum_s[w] == 0.0f ? 0.0f : sum_s[w] * expf(top_s[w] - best);
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += sum_s[w] == 0.0f ? 0.0f : o_s[w][d] * expf(top_s[w] - best);
    x = total == 0.0f ? 0.0f : x / total * P.f.v_scale;
    uint16_t* out = static_cast<uint16_t*>(a.O) + t * a.ldo + (int64_t)head * D + d;
    *out = TYPE == QMM_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
  }
  if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * a.Hq + head] = total == 0.0f ? -INFINITY : best + logf(total);
}

template <int D, int TYPE>
cudaError_t launch(const qmm_attn_fp4_args& f, cudaStream_t stream) {
  const Params P{f, 31 - __builtin_clz((unsigned)f.base.page_size), (int)(f.base.n_slots / f.base.page_size)};
  attn_kernel<D, TYPE><<<dim3(f.base.T, f.base.Hq), 32 * kWarps, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

size_t attn_fp4_workspace_bytes(const qmm_attn_fp4_args&) { return 256; }

cudaError_t launch_attn_fp4(const qmm_attn_fp4_args& f, void*, cudaStream_t stream) {
  if (f.base.D == 64)
    return f.base.type == QMM_BF16 ? launch<64, QMM_BF16>(f, stream) : launch<64, QMM_F16>(f, stream);
  return f.base.type == QMM_BF16 ? launch<128, QMM_BF16>(f, stream) : launch<128, QMM_F16>(f, stream);
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
