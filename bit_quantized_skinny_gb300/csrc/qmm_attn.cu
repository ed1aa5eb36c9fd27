// qmm_attn.cu — attention of several streams' rows over a prefix that they share and over each
// stream's own keys, both in pages of one cache (qmm_attn_shared).
//
// One CTA per (row, head): its warps take the visible keys in turn, each with the running maximum
// and sum of an online softmax, and join them in shared memory.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kWarps = 8;

template <int TYPE>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (TYPE == QMM_BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(__ushort_as_half(v));
}

template <int TYPE>
__device__ __forceinline__ uint16_t from_f32(float v) {
  if constexpr (TYPE == QMM_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

template <int D, int TYPE>
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(const __grid_constant__ qmm_attn_args a) {
  constexpr int kV = D / 32;
  __shared__ float top_s[kWarps], sum_s[kWarps], acc_s[kWarps][D];
  const int t = blockIdx.x, h = blockIdx.y, hk = h / (a.Hq / a.Hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the row's stream and its keys
  int b = -1, own = 0;
  int last = 0;
  for (int k = 0; k <= a.B; ++k) {
    const int r = a.row_starts[k];
    if (r < last || r > a.T) atomicOr(&g_status, kErrIndex);
    if (k > 0 && b < 0 && last <= t && t < r) b = k - 1;
    last = r;
  }
  int64_t prefix = 0;
  if (b >= 0) {
    int len = a.kv_lens[b];
    if (len < 0 || len > a.pages_per_stream * a.page_size) { atomicOr(&g_status, kErrIndex); len = 0; }
    own = len - a.row_starts[b + 1] + t + 1;
    own = own < 0 ? 0 : (own > len ? len : own);
    prefix = a.prefix_len;
  }
  const uint16_t* q = static_cast<const uint16_t*>(a.Q) + t * a.ldq + (int64_t)h * D;
  float qv[kV], acc[kV] = {}, top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int c = 0; c < kV; ++c) qv[c] = to_f32<TYPE>(q[c * 32 + lane]) * a.scale;
  for (int64_t j = warp; j < prefix + own; j += kWarps) {
    const int64_t i = j < prefix ? j : j - prefix;
    const int32_t* list = j < prefix ? a.prefix_pages : a.pages + b * a.pages_per_stream;
    const int64_t page = list[i / a.page_size];
    if (page < 0 || page >= a.n_slots / a.page_size) { atomicOr(&g_status, kErrIndex); continue; }
    const int64_t at = ((page * a.page_size + i % a.page_size) * a.Hk + hk) * D;
    const uint16_t* k = static_cast<const uint16_t*>(a.K_cache) + at;
    const uint16_t* v = static_cast<const uint16_t*>(a.V_cache) + at;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kV; ++c) s = __fmaf_rn(qv[c], to_f32<TYPE>(k[c * 32 + lane]), s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float next = fmaxf(top, s);
    const float keep = expf(top - next), p = expf(s - next);
    top = next;
    sum = __fmaf_rn(sum, keep, p);
#pragma unroll
    for (int c = 0; c < kV; ++c) acc[c] = __fmaf_rn(acc[c], keep, p * to_f32<TYPE>(v[c * 32 + lane]));
  }
  if (lane == 0) { top_s[warp] = top; sum_s[warp] = sum; }
#pragma unroll
  for (int c = 0; c < kV; ++c) acc_s[warp][c * 32 + lane] = acc[c];
  __syncthreads();
  float all = -INFINITY, total = 0.0f;
  for (int w = 0; w < kWarps; ++w) all = fmaxf(all, top_s[w]);
  for (int w = 0; w < kWarps; ++w)
    if (sum_s[w] != 0.0f) total += sum_s[w] * expf(top_s[w] - all);
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float o = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (sum_s[w] != 0.0f) o = __fmaf_rn(acc_s[w][c], expf(top_s[w] - all), o);
    static_cast<uint16_t*>(a.O)[t * a.ldo + (int64_t)h * D + c] = from_f32<TYPE>(total != 0.0f ? o / total : 0.0f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * a.Hq + h] = total != 0.0f ? all + logf(total) : -INFINITY;
}

template <int D, int TYPE>
cudaError_t launch(const qmm_attn_args& a, cudaStream_t stream) {
  attn_kernel<D, TYPE><<<dim3(a.T, a.Hq), 32 * kWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(const qmm_attn_args&) { return 16; }

cudaError_t launch_attn(const qmm_attn_args& a, void*, cudaStream_t stream) {
  if (a.D == 64) return a.type == QMM_BF16 ? launch<64, QMM_BF16>(a, stream) : launch<64, QMM_F16>(a, stream);
  return a.type == QMM_BF16 ? launch<128, QMM_BF16>(a, stream) : launch<128, QMM_F16>(a, stream);
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
