// q4k_kv_fp4.cuh — the 4-bit key/value cache: where a value lies, and how a block of 16 is rounded.
//
// A cache is n_slots / page_size pages; a page holds, for each key/value head, the codes of its slots
// (D/2 bytes each: value 2i in the low, 2i + 1 in the high half of byte i) and then their scales (D/16
// bytes each).  One head's keys of a page are one run of bytes, codes and scales: a tile of them is
// two bulk copies, whatever the number of heads.
#pragma once
#include <cstdint>

namespace q4k {
namespace kv4 {

constexpr int kBlock = 16;              // values that share a scale
constexpr uint32_t kScaleNaN = 0x7Fu;   // E4M3: a block that had an infinity or NaN reads as NaN

// Bytes of one slot's values of one head.
__host__ __device__ constexpr int slot_bytes(int D) { return D / 2 + D / 16; }

// Offset of the codes of (page, head, first slot); the scales follow page_size * D / 2 bytes behind.
__host__ __device__ __forceinline__ int64_t run_at(int64_t page, int head, int Hk, int page_size, int D) {
  return (page * Hk + head) * (int64_t)page_size * slot_bytes(D);
}

// E4M3 of a value that is not negative, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_code(float r) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(0.0f), "f"(r));
  return v & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t pair;
  const uint16_t c = (uint16_t)code;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"(c));
  return __half2float(__ushort_as_half((uint16_t)pair));
}

// E2M1 codes of eight values, to nearest even, at most 6, the first one lowest.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&t)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w) : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return w;
}

}  // namespace kv4
}  // namespace q4k
