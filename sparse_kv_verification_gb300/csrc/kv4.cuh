// A cache held in 4 bits: the layout of a record, and where a position's record
// lies.
//
// One record per (position, kv head), so that a gathered position is one piece
// of memory:
//   [D / 2]  codes of K, two channels to a byte, the lower one in the low bits
//   [D / 2]  codes of V
//   [D / 16] scales of K, e4m3, one per 16 channels;  [D / 16] those of V
//   zeros up to a multiple of 16 bytes
// A value is e2m1(code) * e4m3(scale) * 2^exp.  Records of 144 (D 128) and 80
// (D 64) bytes are 9 and 5 pieces of 16: eight records behind one another start
// in eight different bank groups of shared memory, as they lie.
#pragma once

#include "device_common.cuh"
#include "internal.h"

namespace dustin {

template <int D>
struct Rec {
  static constexpr int K = 0, V = D / 2, SK = D, SV = D + D / 16;
  static constexpr int BYTES = (D + D / 8 + 15) / 16 * 16;
  static constexpr int PIECES = BYTES / 16;
};

// Offset of position j of sequence bb, kv head h, in units of the strides of v (a
// KvView or a Kv4View); -1 if its page id lies outside the pool.
template <typename View>
__device__ __forceinline__ long long place_of(const View& v, int bb, int h, int j) {
  if (!v.page_table) return (long long)bb * v.sb + (long long)h * v.sh + (long long)j * v.sn;
  const int at = j / v.page_size;
  const int page = __ldg(v.page_table + (long long)bb * v.pages_per_seq + at);
  if (page < 0 || page >= v.num_pages) return -1;
  return (long long)page * v.sb + (long long)h * v.sh + (long long)(j - at * v.page_size) * v.sn;
}

// Two e2m1 codes (byte BYTE of w, the low nibble first) as f16x2: exact.
template <int BYTE>
__device__ __forceinline__ uint32_t e2m1_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (BYTE == 0)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}\n" : "=r"(r) : "r"(w));
  else if constexpr (BYTE == 1)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}\n" : "=r"(r) : "r"(w));
  else if constexpr (BYTE == 2)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}\n" : "=r"(r) : "r"(w));
  else
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, d;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
// Two e4m3 scales as f16x2: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace dustin
