// qmm_lora.cu — low-rank adapters beside shared projections (qmm_run_lora):
//     Y[i] = Y0[i] + scale_a * B_a (A_a x_i),  a = ids[i].
//
// Two launches.  lora_shrink_kernel forms t_i = A_a x_i: one warp per (adapter in use, 4 ranks, a
// piece of K), partial sums of the pieces kept apart.  lora_expand_kernel sums the pieces and adds
// scale * t_i Bt_a to Y0: one CTA per (adapter in use, 256 columns), its warps sharing the ranks.
// An adapter is read once for all the rows that use it: the rows of one adapter are found by a warp
// match over the (at most 32) ids.
#include <cstdint>
#include <cuda_runtime.h>

#include "q4k_device.cuh"
#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kWarps = 8;
constexpr int kRanks = 4;        // ranks of one shrink warp
constexpr int kPiece = 1024;     // values of K of one shrink warp (a multiple of 256)
constexpr int kCols = 256;       // columns of one expand CTA, 8 a lane
constexpr int kRows = 4;         // rows of one adapter worked on together

struct Entry {
  const qmm_lora_adapter* adapters;
  const uint16_t* X;
  const float* Y0;
  float* Y;
  float* t;          // pieces x M x rank_max
  int64_t N, K;
  int n_adapters;
  int pieces;
  int first;         // first block of this entry in the expand grid's x
};
struct Params {
  Entry e[QMM_LORA_MAX_ENTRIES];
  const int32_t* ids;
  int count, M, rank_max;
};

// The rows of the g-th distinct adapter of the M ids (in order of first row) as a mask of rows; 0
// past the last.  All lanes of a warp call this; `id` comes back as that adapter's id.
__device__ __forceinline__ unsigned group_rows(const int32_t* ids, int M, int n_adapters, int g, int& id) {
  const int lane = threadIdx.x & 31;
  int mine = lane < M ? ids[lane] : -2;
  if (mine >= n_adapters || mine < -2 || (mine == -2 && lane < M)) {
    atomicOr(&g_status, kErrIndex);
    mine = -1;
  }
  const unsigned same = __match_any_sync(0xffffffffu, mine);
  const bool leader = lane < M && (same & ((1u << lane) - 1)) == 0;
  unsigned leaders = __ballot_sync(0xffffffffu, leader);
  if (g >= __popc(leaders)) return 0;
  for (int k = 0; k < g; ++k) leaders &= leaders - 1;
  const int at = __ffs(leaders) - 1;
  id = __shfl_sync(0xffffffffu, mine, at);
  return __shfl_sync(0xffffffffu, same, at);
}

// Adapter `id` of entry e; rank 0 for none, or for one whose rank or alignment is not allowed.
__device__ __forceinline__ qmm_lora_adapter adapter_of(const Entry& e, int id, int rank_max) {
  qmm_lora_adapter a{nullptr, nullptr, 0.0f, 0};
  if (id < 0) return a;
  a = e.adapters[id];
  if (a.rank < 0 || a.rank > rank_max || (a.rank > 0 && (!a.A || !a.Bt || (reinterpret_cast<uintptr_t>(a.A) & 15) ||
                                                         (reinterpret_cast<uintptr_t>(a.Bt) & 1)))) {
    atomicOr(&g_status, kErrIndex);
    a.rank = 0;
  }
  return a;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Grid (rank groups of kWarps * kRanks x pieces, adapters in use, entries).
__global__ void __launch_bounds__(32 * kWarps) lora_shrink_kernel(const __grid_constant__ Params P) {
  const Entry& e = P.e[blockIdx.z];
  const int piece = blockIdx.x % e.pieces;
  const int r0 = (blockIdx.x / e.pieces * kWarps + (threadIdx.x >> 5)) * kRanks;
  const int lane = threadIdx.x & 31;
  if (piece * (int64_t)kPiece >= e.K) return;
  int id = -1;
  unsigned rows = group_rows(P.ids, P.M, e.n_adapters, blockIdx.y, id);
  if (!rows || id < 0) return;
  const qmm_lora_adapter a = adapter_of(e, id, P.rank_max);
  if (r0 >= a.rank) return;
  const int64_t k0 = piece * (int64_t)kPiece;
  const int64_t k1 = k0 + kPiece < e.K ? k0 + kPiece : e.K;
  while (rows) {
    int row[kRows], n = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      row[j] = rows ? __ffs(rows) - 1 : row[0];
      if (rows) { rows &= rows - 1; ++n; }
    }
    float acc[kRows * kRanks] = {};
    for (int64_t k = k0 + 8 * lane; k < k1; k += 256) {
      float w[kRanks][8];
#pragma unroll
      for (int r = 0; r < kRanks; ++r) {
        const int rr = r0 + r < a.rank ? r0 + r : r0;
        unpack8(*reinterpret_cast<const uint4*>(a.A + rr * e.K + k), w[r]);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        if (j >= n) break;
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(e.X + row[j] * e.K + k), x);
#pragma unroll
        for (int r = 0; r < kRanks; ++r)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[j * kRanks + r] = __fmaf_rn(w[r][c], x[c], acc[j * kRanks + r]);
      }
    }
    butterfly_reduce<kRows * kRanks>(acc, lane);   // lane l: value l / (32 / values)
    constexpr int kPer = 32 / (kRows * kRanks);
    const int v = lane / kPer, j = v / kRanks, r = v % kRanks;
    int mine = row[0];
#pragma unroll
    for (int q = 0; q < kRows; ++q) mine = j == q ? row[q] : mine;
    if (lane % kPer == 0 && j < n && r0 + r < a.rank)
      e.t[((int64_t)piece * P.M + mine) * P.rank_max + r0 + r] = acc[0];
  }
}

// Grid (blocks of kCols columns over all entries, adapters in use).
__global__ void __launch_bounds__(32 * kWarps) lora_expand_kernel(const __grid_constant__ Params P) {
  __shared__ float ts[kRows][QMM_LORA_MAX_RANK];
  __shared__ float part[kWarps][kRows][kCols];
  int k = 0;
  while (k + 1 < P.count && (int)blockIdx.x >= P.e[k + 1].first) ++k;
  const Entry& e = P.e[k];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int id = -1;
  unsigned rows = group_rows(P.ids, P.M, e.n_adapters, blockIdx.y, id);
  if (!rows) return;
  const qmm_lora_adapter a = adapter_of(e, id, P.rank_max);
  const int64_t n0 = (int64_t)(blockIdx.x - e.first) * kCols;
  const int64_t n = n0 + 8 * lane;
  const bool wide = (reinterpret_cast<uintptr_t>(a.Bt) & 15) == 0 && e.N % 8 == 0;
  while (rows) {
    int row[kRows], m = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      row[j] = rows ? __ffs(rows) - 1 : row[0];
      if (rows) { rows &= rows - 1; ++m; }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < m * a.rank; v += blockDim.x) {
      const int j = v / a.rank, r = v % a.rank;
      int mine = row[0];
#pragma unroll
      for (int q = 0; q < kRows; ++q) mine = j == q ? row[q] : mine;
      float s = 0.0f;
      for (int p = 0; p < e.pieces; ++p) s += e.t[((int64_t)p * P.M + mine) * P.rank_max + r];
      ts[j][r] = s * a.scale;
    }
    __syncthreads();
    float acc[kRows][8] = {};
    for (int r = warp; r < a.rank; r += kWarps) {
      float b[8] = {};
      const uint16_t* src = a.Bt + (int64_t)r * e.N + n;
      if (wide && n < e.N) unpack8(*reinterpret_cast<const uint4*>(src), b);
      else
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (n + c < e.N) b[c] = __uint_as_float((uint32_t)src[c] << 16);
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (j < m)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[j][c] = __fmaf_rn(b[c], ts[j][r], acc[j][c]);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) part[warp][j][8 * lane + c] = acc[j][c];
    __syncthreads();
    for (int v = threadIdx.x; v < m * kCols; v += blockDim.x) {
      const int j = v / kCols, c = v % kCols;
      int mine = row[0];
#pragma unroll
      for (int q = 0; q < kRows; ++q) mine = j == q ? row[q] : mine;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += part[w][j][c];
      if (n0 + c < e.N) e.Y[mine * e.N + n0 + c] = e.Y0[mine * e.N + n0 + c] + s;
    }
  }
}

int pieces_of(int64_t K) { return (int)((K + kPiece - 1) / kPiece); }

size_t entry_floats(int64_t K, int M, int rank_max) { return ((size_t)pieces_of(K) * M * rank_max + 3) & ~(size_t)3; }

}  // namespace

size_t lora_workspace_bytes(const qmm_lora_entry* entries, int count, int M, int rank_max) {
  size_t n = 0;
  for (int k = 0; k < count; ++k) n += entry_floats(entries[k].K, M, rank_max);
  return n * sizeof(float);
}

cudaError_t launch_lora(const qmm_lora_entry* entries, int count, const int32_t* ids, int M, int rank_max,
                        void* workspace, cudaStream_t stream) {
  Params P{};
  P.ids = ids;
  P.count = count;
  P.M = M;
  P.rank_max = rank_max;
  float* t = static_cast<float*>(workspace);
  int64_t blocks = 0;
  int pieces = 0, groups = 1;
  for (int k = 0; k < count; ++k) {
    const qmm_lora_entry& e = entries[k];
    P.e[k] = Entry{e.adapters, e.X, e.Y0, e.Y, t, e.N, e.K, e.n_adapters, pieces_of(e.K), (int)blocks};
    t += entry_floats(e.K, M, rank_max);
    blocks += (e.N + kCols - 1) / kCols;
    pieces = pieces > P.e[k].pieces ? pieces : P.e[k].pieces;
    const int g = e.n_adapters < M ? e.n_adapters + 1 : M;   // adapters in use, and no adapter
    groups = groups > g ? groups : (g < M ? g : M);
  }
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const int rank_groups = (rank_max + kWarps * kRanks - 1) / (kWarps * kRanks);
  lora_shrink_kernel<<<dim3(pieces * rank_groups, groups, count), 32 * kWarps, 0, stream>>>(P);
  lora_expand_kernel<<<dim3((unsigned)blocks, groups), 32 * kWarps, 0, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t read_and_clear_lora_status(unsigned* out) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace q4k
