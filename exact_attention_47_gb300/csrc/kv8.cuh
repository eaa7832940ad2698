// Layout of the 8-bit paged KV cache and the steps between its codes and
// numbers (shared by the append, the read-back and the attention over it).
//
// The cache is [num_blocks, Hkv, record] bytes: one record holds the 16 token
// slots of one KV head of one block, K and V together:
//   K codes   16 rows of D bytes          V codes   16 rows of D bytes
//   K scale, V scale (fp32), a word of flags (bit s: slot s's key has an element
//   that is no finite number; bit 16 + s: its value), 20 bytes of zeros
// A code is an e4m3 number (sign, 4 bits of exponent, 3 of fraction; at most
// 448) and stands for itself times the scale, a power of two: an 8-bit number
// with an exponent of its own gains nothing from the fraction of a scale, the
// values are then exact in bf16, and a block whose scale grows with a later
// token keeps its codes' fractions (but for those that become subnormal).
// The 32 bytes at the end keep every record on whole 32-byte sectors.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace attn47 {

constexpr int kKv8Slots = 16;
constexpr int kKv8Tail = 32;
constexpr int kKv8LeastExp = -64, kKv8MostExp = 64;   // of a scale

// Bytes of a record, in a form the host-side checks can use too.
inline constexpr size_t kv8_record_bytes_of(int d) { return static_cast<size_t>(2 * kKv8Slots) * d + kKv8Tail; }

template <int D>
struct Kv8Layout {
  static constexpr int kRow = D;                             // bytes of a row's codes
  static constexpr int kOffV = kKv8Slots * kRow;
  static constexpr int kOffTail = 2 * kOffV;
  static constexpr int kBytes = kOffTail + kKv8Tail;
  static_assert(kBytes == kv8_record_bytes_of(D), "record size");
  static_assert(kBytes % 16 == 0, "records are read in 16-byte pieces");
};

// Two e4m3 codes (the low 16 bits) as two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(codes));
  return r;
}
// The same of the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(codes));
  return r;
}
// Four numbers to the nearest e4m3 (half to even, at most 448 in size; NaN
// stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The scale (its bits) for values up to `most` (bits of a finite number >= 0):
// the smallest power of two under which that is at most 448 = 1.75 2^8.
__device__ __forceinline__ uint32_t kv8_scale_for(uint32_t most) {
  const int e = static_cast<int>(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, kKv8LeastExp), kKv8MostExp) + 127) << 23;
}
// 1 / scale.
__device__ __forceinline__ float kv8_inverse(uint32_t scale) { return __uint_as_float((254u << 23) - scale); }

}  // namespace attn47
