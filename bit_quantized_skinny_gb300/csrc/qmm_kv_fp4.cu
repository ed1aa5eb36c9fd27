// qmm_kv_fp4.cu — slots of a 4-bit key/value cache as values (qmm_kv_fp4_read).
//
// A thread reads one block (8 bytes of codes and a scale) and writes its 16 values; eight neighbouring threads read
// one head's codes of a slot.  Bound by the bytes it writes (16384 slots of 8 heads of 128, keys and values to bf16: 18.7 us,
// 86 MB, of which L2 keeps much).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "q4k_formats.cuh"
#include "q4k_internal.h"
#include "q4k_kv_fp4.cuh"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kThreads = 256;

struct Params {
  qmm_kv_fp4_read_args a;
  int page_shift;
};

template <int OUT>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Params P) {
  // launched early behind a launch that allows it: memory is read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const qmm_kv_fp4_read_args& a = P.a;
  const int blocks = a.D / kv4::kBlock;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= a.n * a.Hk * blocks) return;
  const int64_t head_of = id / blocks;
  const int b = (int)(id - head_of * blocks);
  const int64_t row = head_of / a.Hk;
  const int h = (int)(head_of - row * a.Hk);
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    atomicOr(&g_status, kErrIndex);
    return;
  }
  const int i = (int)(slot & (a.page_size - 1));
  const int64_t run = kv4::run_at(slot >> P.page_shift, h, a.Hk, a.page_size, a.D);
  const uint8_t* cache = static_cast<const uint8_t*>(blockIdx.y ? a.V_cache : a.K_cache) + run;
  const uint2 w = *reinterpret_cast<const uint2*>(cache + i * (a.D / 2) + 8 * b);
  const float s = kv4::e4m3_value(cache[a.page_size * (a.D / 2) + i * blocks + b]);
  const float g = blockIdx.y ? a.v_scale : a.k_scale;
  float v[16];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t p[4];
    e2m1x8_pairs(k ? w.y : w.x, p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[q]));
      v[8 * k + 2 * q] = f.x * s * g;   // the first product is exact
      v[8 * k + 2 * q + 1] = f.y * s * g;
    }
  }
  void* out = blockIdx.y ? a.V_out : a.K_out;
  const int64_t at = head_of * a.D + 16 * b;
  if constexpr (OUT == QMM_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (OUT == QMM_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
        u[q] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
        u[q] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
    p[0] = make_uint4(u[0], u[1], u[2], u[3]);
    p[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

}  // namespace

cudaError_t launch_kv_fp4_read(const qmm_kv_fp4_read_args& a, cudaStream_t stream) {
  const Params P{a, 31 - __builtin_clz((unsigned)a.page_size)};
  const int64_t grid = (a.n * a.Hk * (a.D / kv4::kBlock) + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid, a.V_out ? 2 : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (a.out_type == QMM_F32) return cudaLaunchKernelEx(&cfg, read_kernel<QMM_F32>, P);
  if (a.out_type == QMM_BF16) return cudaLaunchKernelEx(&cfg, read_kernel<QMM_BF16>, P);
  return cudaLaunchKernelEx(&cfg, read_kernel<QMM_F16>, P);
}

cudaError_t read_and_clear_kv_fp4_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
