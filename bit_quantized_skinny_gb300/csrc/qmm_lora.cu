// qmm_lora.cu — low-rank adapters beside shared projections (qmm_run_lora):
//     Y[i] = Y0[i] + scale_a * B_a (A_a x_i),  a = ids[i].
//
// Two launches.  lora_shrink_kernel forms t_i = A_a x_i: one warp per (adapter in use, up to 4 of its
// rows, 4 ranks, run of pieces of K), the partial sums of the pieces of 512 values kept apart.
// lora_expand_kernel sums the pieces and adds scale * t_i Bt_a to Y0, 256 columns a warp, for up to 4 (2)
// rows of an adapter.  Both are bound by the adapters' bytes, which the rows of an item share (rows are
// matched to adapters by a warp match over the at most 32 ids); an adapter with more rows is read again
// from L2 by its next item, side by side: 32 rows of one adapter beside 34816 columns 20 us, one item
// after the other 41.  The expand launch starts while the shrink launch runs and has its first B values in
// flight before it waits for t.
//
// Measured: 32 rows of 32 adapters of rank 64 beside 34816 x 5120, 173 MB: 32.4 us, 5.3 TB/s over both
// launches; the same rows beside q, k and v (7168 columns of 5120, 94 MB) 28.4 us; one row beside q, k and
// v 4.4 us: two launches' chains of dependent loads.
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "q4k_device.cuh"
#include "q4k_internal.h"

namespace q4k {
namespace {

__device__ unsigned g_status;   // this file's kernels' status word

constexpr int kShrinkWarps = 4;
constexpr int kRanks = 4;        // ranks of one shrink warp
constexpr int kShrinkRows = 4;   // rows of one shrink warp (8 rows an adapter, K 17408: 13.0 us; 2: 15.0, 8: 16.4)
constexpr int kChunk = 512;      // values of K that a shrink warp holds at a time
constexpr int kPieces = 64;      // pieces of K at most
constexpr int kResident = 16;    // shrink warps an SM holds
constexpr int64_t kAhead = 16 << 20;   // bytes of B that the shrink launch asks into L2
constexpr int kCols = 256;       // columns of one expand warp, 8 a lane
// The two forms of the expand kernel.  kSplit: 8 warps share the ranks of one block of columns and join
// their sums in shared memory; up to 4 rows are worked on together.  kStream: a block of columns for
// each of 2 warps, up to 2 rows together, few enough registers that every warp of 32 adapters
// beside 34816 columns is resident at once (28.6 an SM; in CTAs of 8 warps the last ones waited for a
// second round: 45 us, not 37).
// In both, and on every boundary, a value is the sum of its ranks in shares (share_of), each share summed in
// order and the shares added up in order: its bits depend on K and the adapter's rank, not on
// the form, the batch, the table or where Bt lies.  (Two sums a value in kStream: 32 adapters beside 34816
// columns 32.4 us, one sum 32.0; shares of 4 instead of 8 ranks where a row of Bt is aligned: 32 of rank 32
// beside 5120 columns 12.8 us, 12.2.)
enum Form { kSplit, kStream };
__host__ __device__ constexpr int warps_of(Form f) { return f == kSplit ? 8 : 2; }
__host__ __device__ constexpr int rows_of(Form f) { return f == kSplit ? 4 : 2; }
__host__ __device__ constexpr int share_of(int rank) { return (rank + 31) / 32 * 4; }   // ranks of one of 8 sums
__host__ __device__ constexpr int step_of(Form f, bool wide) { return f == kSplit && wide ? 8 : 4; }   // ranks loaded together

struct Entry {
  const qmm_lora_adapter* adapters;
  const uint16_t* X;
  const float* Y0;
  float* Y;
  float* t;          // pieces x M x rank_max
  int64_t N, K;
  int n_adapters;
  int pieces, chunks;   // of K, and of a piece
  int first;         // first block of this entry in the expand grid's x
};
struct Params {
  Entry e[QMM_LORA_MAX_ENTRIES];
  const int32_t* ids;
  int count, M, rank_max;
  int rank_groups;   // of kRanks in rank_max
  int run;           // pieces of K of one shrink warp
};

// The work of item g: the rows of one adapter in use, R at most, as a mask; an adapter with more rows has
// several items (in the order of their first rows); 0 past the last.  All lanes of a warp call this; `id`
// comes back as the adapter's id, `groups` as the number of adapters in use, `nth` as the item's place
// among those of its adapter.
template <int R>
__device__ __forceinline__ unsigned item_rows(const int32_t* ids, int M, int n_adapters, int g, int& id, int& groups,
                                              int& nth) {
  const int lane = threadIdx.x & 31;
  int mine = lane < M ? ids[lane] : -2;
  if (mine >= n_adapters || mine < -2 || (mine == -2 && lane < M)) {
    atomicOr(&g_status, kErrIndex);
    mine = -1;
  }
  const unsigned same = __match_any_sync(0xffffffffu, mine);
  const int before = __popc(same & ((1u << lane) - 1));   // rows of the same adapter
  groups = __popc(__ballot_sync(0xffffffffu, lane < M && before == 0));
  unsigned firsts = __ballot_sync(0xffffffffu, lane < M && before % R == 0);
  if (g >= __popc(firsts)) return 0;
  for (int k = 0; k < g; ++k) firsts &= firsts - 1;
  const int at = __ffs(firsts) - 1;
  id = __shfl_sync(0xffffffffu, mine, at);
  nth = __shfl_sync(0xffffffffu, before / R, at);
  return __ballot_sync(0xffffffffu, mine == id && before / R == nth);
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

// A word that the shrink launch wrote, from L2.  volatile: behind the wait for that launch.
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Grid (rank groups x runs of pieces in units of kShrinkWarps, items, entries).
__global__ void __launch_bounds__(32 * kShrinkWarps, 4) lora_shrink_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Entry& e = P.e[blockIdx.z];
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kShrinkWarps + (threadIdx.x >> 5);
  const int run = unit / P.rank_groups, r0 = (unit - run * P.rank_groups) * kRanks;
  const int runs = (e.pieces + P.run - 1) / P.run;
  if (run >= runs) return;
  int id = -1, groups, nth;
  const unsigned all = item_rows<kShrinkRows>(P.ids, P.M, e.n_adapters, blockIdx.y, id, groups, nth);
  if (!all || id < 0) return;
  const qmm_lora_adapter a = adapter_of(e, id, P.rank_max);
  if (r0 >= a.rank) return;
  constexpr int kV = kChunk / 256;   // 16-byte loads of a lane in a chunk
  const int64_t end = min(e.K, (int64_t)(run + 1) * P.run * e.chunks * kChunk);
  int64_t k0 = (int64_t)run * P.run * e.chunks * kChunk;
  uint4 raw[kRanks][kV], x[kV];
  auto ask_a = [&](int64_t from, uint4 (&to)[kRanks][kV]) {
#pragma unroll
    for (int r = 0; r < kRanks; ++r)
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const bool in = r0 + r < a.rank && from + 256 * v < end;
        to[r][v] = in ? ldg_nc_v4(a.A + (r0 + r) * e.K + from + 256 * v + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  auto ask_x = [&](int row, int64_t from) {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      x[v] = from + 256 * v < end ? *reinterpret_cast<const uint4*>(e.X + row * e.K + from + 256 * v + 8 * lane)
                                  : make_uint4(0u, 0u, 0u, 0u);
  };
  const int first = __ffs(all) - 1;
  ask_a(k0, raw);
  ask_x(first, k0);
  if (nth == 0) {
    // The expand launch's first B towards L2, this warp's share of the adapter's (its units are the live
    // rank groups by the runs), so that memory is not idle while t is formed.
    const int live = (a.rank + kRanks - 1) / kRanks;
    const int64_t bytes = min((int64_t)a.rank * e.N * 2, kAhead / groups / P.count) & ~(int64_t)127;
    for (int64_t k = ((int64_t)run * live + r0 / kRanks) * 32 + lane; k < bytes / 128; k += 32 * (int64_t)live * runs)
      asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.Bt) + 128 * k));
  }
  int piece = run * P.run, part = 0;   // of the piece's chunks
  for (; k0 < end; k0 += kChunk) {
    uint4 next[kRanks][kV];   // the next chunk's A and a row's x are asked for while the ones before are worked on
    if (k0 + kChunk < end) ask_a(k0 + kChunk, next);
    for (unsigned rows = all; rows;) {
      const int row = __ffs(rows) - 1;
      rows &= rows - 1;
      uint4 now[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v) now[v] = x[v];
      if (rows) ask_x(__ffs(rows) - 1, k0);
      else if (k0 + kChunk < end) ask_x(first, k0 + kChunk);
      float acc[kRanks] = {};
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        float xs[8];
        unpack8(now[v], xs);
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
          float w[8];
          unpack8(raw[r][v], w);
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[r] = __fmaf_rn(w[c], xs[c], acc[r]);
        }
      }
      butterfly_reduce<kRanks>(acc, lane);   // lane l: rank l / 4
      const int r = r0 + lane / (32 / kRanks);
      if (lane % (32 / kRanks) == 0 && r < a.rank) {
        float* t = e.t + ((int64_t)piece * P.M + row) * P.rank_max + r;
        *t = part == 0 ? acc[0] : *t + acc[0];
      }
    }
    if (k0 + kChunk >= end) break;
    if (++part == e.chunks) {
      part = 0;
      ++piece;
    }
#pragma unroll
    for (int r = 0; r < kRanks; ++r)
#pragma unroll
      for (int v = 0; v < kV; ++v) raw[r][v] = next[r][v];
  }
}

// The 16 bytes at p (16-byte aligned), as far as they lie in [lo, hi); zeros for the rest.  (The first and
// the last of a matrix only: out of line.)
__device__ __noinline__ uint4 load_edge(const uint16_t* p, const uint16_t* lo, const uint16_t* hi) {
  uint32_t v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = p + c >= lo && p + c < hi ? p[c] : 0u;
  return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

__device__ __forceinline__ uint4 load_within(const uint16_t* p, const uint16_t* lo, const uint16_t* hi) {
  if (p >= lo && p + 8 <= hi) return __ldg(reinterpret_cast<const uint4*>(p));
  return load_edge(p, lo, hi);
}

// The 8 values that begin `skip` values (0..7) into a and go on in b.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int skip) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (skip & 4)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (skip & 2)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  if (skip & 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = w[k] >> 16 | w[k + 1] << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// STEP rows of Bt from rank r on, the lane's 8 columns n0 + 8 lane ..; zeros for ranks from r1 on.  (Columns
// behind N are never stored; what stands in their place is the next row's.)  WIDE: every row is 16-byte
// aligned; else a row's values are cut out of the two aligned words that hold them.
template <int STEP, bool WIDE>
__device__ __forceinline__ void load_b(const qmm_lora_adapter& a, int64_t N, int64_t n0, int r, int r1, int lane,
                                       uint4 (&b)[STEP]) {
#pragma unroll
  for (int q = 0; q < STEP; ++q) {
    b[q] = make_uint4(0u, 0u, 0u, 0u);
    if (r + q >= r1 || n0 + 8 * lane >= N) continue;
    const uint16_t* src = a.Bt + (int64_t)(r + q) * N + n0 + 8 * lane;
    if constexpr (WIDE) {
      b[q] = ldg_nc_v4(src);
    } else {
      const int skip = (int)(reinterpret_cast<uintptr_t>(src) & 15) / 2;   // the same for all lanes of a row
      const uint16_t* hi = a.Bt + (int64_t)a.rank * N;
      const uint4 u = load_within(src - skip, a.Bt, hi);
      b[q] = skip ? shifted(u, load_within(src - skip + 8, a.Bt, hi), skip) : u;
    }
  }
}

// acc[j][c] = sum over ranks [r0, r1) of ts[j][r] Bt[r][column c] for R rows: in one sum, or (SHARES) a sum
// for each `share` ranks and those added up in order.  `first` holds the first STEP ranks' values already.
template <int R, int STEP, bool WIDE, bool SHARES>
__device__ __forceinline__ void accumulate(const qmm_lora_adapter& a, int64_t N, int64_t n0, int r0, int r1, int share,
                                           int lane, const float (*ts)[QMM_LORA_MAX_RANK], const uint4 (&first)[STEP],
                                           float (&acc)[R][8]) {
  [[maybe_unused]] float total[R][8] = {};
  [[maybe_unused]] int left = share;
  uint4 b[STEP];
#pragma unroll
  for (int q = 0; q < STEP; ++q) b[q] = first[q];
#pragma unroll 1
  for (int r = r0; r < r1; r += STEP) {
    uint4 ahead[STEP];
    load_b<STEP, WIDE>(a, N, n0, r + STEP, r1, lane, ahead);
#pragma unroll
    for (int q = 0; q < STEP; ++q) {
      float x[8];
      unpack8(b[q], x);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float t = r + q < r1 ? ts[j][r + q] : 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = __fmaf_rn(x[c], t, acc[j][c]);
      }
    }
    if constexpr (SHARES) {
      left -= STEP;
      if (left == 0 || r + STEP >= r1) {
        left = share;
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            total[j][c] += acc[j][c];
            acc[j][c] = 0.0f;
          }
      }
    }
#pragma unroll
    for (int q = 0; q < STEP; ++q) b[q] = ahead[q];
  }
  if constexpr (SHARES)
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[j][c] = total[j][c];
}

// One CTA: one block (kSplit) or a block a warp (kStream) of columns for one item.
template <Form FORM, bool WIDE>
__device__ __forceinline__ void expand(const Params& P, const Entry& e, unsigned rows, const qmm_lora_adapter& a,
                                       int64_t block0, float (*ts)[QMM_LORA_MAX_RANK], float (*part)[rows_of(FORM)][kCols]) {
  constexpr bool SPLIT = FORM == kSplit;
  constexpr int kWarps = warps_of(FORM), kRows = rows_of(FORM), kStep = step_of(FORM, WIDE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n0 = SPLIT ? block0 : block0 + kCols * warp;
  const int share = share_of(a.rank);
  int r0 = 0, r1 = a.rank;
  if constexpr (SPLIT) {   // a share a warp
    r0 = min(a.rank, warp * share);
    r1 = min(a.rank, r0 + share);
  }
  uint4 first[kStep];
  load_b<kStep, WIDE>(a, e.N, n0, r0, r1, lane, first);
  const bool vec = e.N % 8 == 0 && ((reinterpret_cast<uintptr_t>(e.Y) | reinterpret_cast<uintptr_t>(e.Y0)) & 15) == 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto work = [&](auto r_) {   // R rows or fewer
    constexpr int R = decltype(r_)::value;
    int row[R], m = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      row[j] = rows ? __ffs(rows) - 1 : row[0];
      if (rows) { rows &= rows - 1; ++m; }
    }
    [[maybe_unused]] float ys[R];   // kSplit: Y0 of the thread's column, asked for ahead of the sums
    if constexpr (SPLIT)
#pragma unroll
      for (int j = 0; j < R; ++j)
        ys[j] = j < m && n0 + threadIdx.x < e.N ? e.Y0[row[j] * e.N + n0 + threadIdx.x] : 0.0f;
    for (int v = threadIdx.x; v < R * a.rank; v += 32 * kWarps) {
      const int j = v / a.rank, r = v - j * a.rank;
      int mine = row[0];
#pragma unroll
      for (int q = 1; q < R; ++q) mine = j == q ? row[q] : mine;
      float s = 0.0f;
      const float* t = e.t + (int64_t)mine * P.rank_max + r;
      constexpr int kTogether = 16;
      for (int p0 = 0; j < m && p0 < e.pieces; p0 += kTogether) {
        float x[kTogether];
#pragma unroll
        for (int p = 0; p < kTogether; ++p) x[p] = p0 + p < e.pieces ? ld_cg(t + (int64_t)(p0 + p) * P.M * P.rank_max) : 0.0f;
#pragma unroll
        for (int p = 0; p < kTogether; ++p) s += x[p];
      }
      ts[j][r] = s * a.scale;
    }
    __syncthreads();
    float acc[R][8] = {};
    float4 y0[2];   // one row: its Y0 is asked for ahead of the sums
    const bool early = R == 1 && !SPLIT && vec && n0 + 8 * lane < e.N;
    if (early) {
      y0[0] = *reinterpret_cast<const float4*>(e.Y0 + row[0] * e.N + n0 + 8 * lane);
      y0[1] = *reinterpret_cast<const float4*>(e.Y0 + row[0] * e.N + n0 + 8 * lane + 4);
    }
    accumulate<R, kStep, WIDE, !SPLIT>(a, e.N, n0, r0, r1, share, lane, ts, first, acc);
    if constexpr (SPLIT) {
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) part[warp][j][8 * lane + c] = acc[j][c];
      __syncthreads();
      static_assert(!SPLIT || kCols == 32 * kWarps, "a column a thread");
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[w][j][threadIdx.x];
        if (j < m && n0 + threadIdx.x < e.N) e.Y[row[j] * e.N + n0 + threadIdx.x] = ys[j] + s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (j >= m) break;
        const int64_t at = row[j] * e.N + n0;
        if (vec && n0 + 8 * lane < e.N) {
          const float4* src = reinterpret_cast<const float4*>(e.Y0 + at + 8 * lane);
          float4* y = reinterpret_cast<float4*>(e.Y + at + 8 * lane);
          const float4 u = early ? y0[0] : src[0], v = early ? y0[1] : src[1];
          y[0] = make_float4(u.x + acc[j][0], u.y + acc[j][1], u.z + acc[j][2], u.w + acc[j][3]);
          y[1] = make_float4(v.x + acc[j][4], v.y + acc[j][5], v.z + acc[j][6], v.w + acc[j][7]);
        } else if (!vec) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int col = 8 * lane + c;
            if (n0 + col < e.N) e.Y[at + col] = e.Y0[at + col] + acc[j][c];
          }
        }
      }
    }
  };
  if (__popc(rows) == 1) work(std::integral_constant<int, 1>{});
  else work(std::integral_constant<int, kRows>{});
}

// Grid (blocks of columns over all entries, items).
template <Form FORM>
__global__ void __launch_bounds__(32 * warps_of(FORM), FORM == kSplit ? 2 : 16) lora_expand_kernel(const __grid_constant__ Params P) {
  __shared__ float ts[rows_of(FORM)][QMM_LORA_MAX_RANK];
  __shared__ float part[FORM == kSplit ? warps_of(FORM) : 1][rows_of(FORM)][kCols];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int k = 0;
  while (k + 1 < P.count && (int)blockIdx.x >= P.e[k + 1].first) ++k;
  const Entry& e = P.e[k];
  int id = -1, groups, nth;
  const unsigned rows = item_rows<rows_of(FORM)>(P.ids, P.M, e.n_adapters, blockIdx.y, id, groups, nth);
  if (!rows) return;
  const qmm_lora_adapter a = adapter_of(e, id, P.rank_max);
  const int64_t n0 = (int64_t)(blockIdx.x - e.first) * (FORM == kSplit ? kCols : kCols * warps_of(FORM));
  if ((reinterpret_cast<uintptr_t>(a.Bt) & 15) == 0 && e.N % 8 == 0) expand<FORM, true>(P, e, rows, a, n0, ts, part);
  else expand<FORM, false>(P, e, rows, a, n0, ts, part);
}

int chunks_of(int64_t K) { return (int)((K + (int64_t)kChunk * kPieces - 1) / ((int64_t)kChunk * kPieces)); }
int pieces_of(int64_t K) {
  const int64_t piece = (int64_t)kChunk * chunks_of(K);
  return (int)((K + piece - 1) / piece);
}

size_t entry_floats(int64_t K, int M, int rank_max) { return ((size_t)pieces_of(K) * M * rank_max + 3) & ~(size_t)3; }

template <class F>
cudaError_t launch_early(F* kernel, dim3 grid, int warps, const Params& P, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P);
}

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
  P.rank_groups = (rank_max + kRanks - 1) / kRanks;
  // kStream where the blocks of columns alone make 16 warps an SM.  With 32 adapters of rank 64: 34816
  // columns (29 an SM) 32 us, kSplit 51; 7168 columns (6 an SM) 37 us, kSplit 28.
  int64_t warps = 0;
  int pieces = 0, groups = 1;   // groups: adapters in use at most, no adapter among them
  for (int k = 0; k < count; ++k) {
    const qmm_lora_entry& e = entries[k];
    const int g = e.n_adapters < M ? e.n_adapters + 1 : M;
    groups = groups > g ? groups : g;
    pieces = pieces > pieces_of(e.K) ? pieces : pieces_of(e.K);
    warps += (e.N + kCols - 1) / kCols * g;
  }
  const int64_t sms = sm_count();
  const bool split = warps < 16 * sms;
  const int64_t cols = split ? kCols : (int64_t)kCols * warps_of(kStream);
  float* t = static_cast<float*>(workspace);
  int64_t blocks = 0;
  for (int k = 0; k < count; ++k) {
    const qmm_lora_entry& e = entries[k];
    P.e[k] = Entry{e.adapters, e.X, e.Y0, e.Y, t, e.N, e.K, e.n_adapters, pieces_of(e.K), chunks_of(e.K), (int)blocks};
    t += entry_floats(e.K, M, rank_max);
    blocks += (e.N + cols - 1) / cols;
  }
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // A warp takes as many pieces as bring the launch into one round of resident warps, with the next
  // chunk's A in flight (16 adapters of rank 64, 7168 columns of 5120: 15.5 us; a piece a warp 18.7;
  // half or double the warps 21.3, 16.4).  Each piece keeps its own sum, so the result does not depend on this.
  const int64_t resident = kResident * sms;
  const int64_t each = (int64_t)P.rank_groups * groups * count;
  const int64_t fit = resident / each;   // runs
  P.run = fit >= pieces ? 1 : fit <= 1 ? pieces : (int)((pieces + fit - 1) / fit);
  const int runs = (pieces + P.run - 1) / P.run;
  // items of R rows at most: each of the groups has one, and one more for every R rows beside its first
  auto items = [&](int R) { return (unsigned)(groups + (M - groups) / R); };
  cudaError_t err = launch_early(lora_shrink_kernel,
                                 dim3((runs * P.rank_groups + kShrinkWarps - 1) / kShrinkWarps, items(kShrinkRows), count),
                                 kShrinkWarps, P, stream);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)blocks, items(split ? rows_of(kSplit) : rows_of(kStream)));
  return split ? launch_early(lora_expand_kernel<kSplit>, grid, warps_of(kSplit), P, stream)
               : launch_early(lora_expand_kernel<kStream>, grid, warps_of(kStream), P, stream);
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
