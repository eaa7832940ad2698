// Layout of the 4-bit paged KV cache and the warp steps that pack and unpack
// its rows (shared by the append, the read-back and the decode).
//
// The cache is [num_blocks, Hkv, record] bytes: one record holds the 16 token
// slots of one KV head of one block, K and V together, so that a decode
// fetches everything it needs of a (block, head) with one contiguous copy:
//   K codes   16 rows of D/2 bytes        V codes   16 rows of D/2 bytes
//   K params  16 rows of D/G words        V params  16 rows of D/G words
// A parameter word is (scale << 16) | min, both bf16, of one group of G
// consecutive elements; a value is code * scale + min.
//
// Inside a row the 4-bit codes are ordered so that a lane of the decode's
// warp MMAs finds all its codes of a row in one 16-byte (K) or 8-byte (V)
// load and gets operand registers from them with one mask each:
//   K: element e = 32 w + 8 i + 2 c + h is nibble i + 4 h of word
//      (D/32) c + w.  Lane c of a quad owns elements 2c, 2c+1 (mod 8), and
//      nibbles i, i + 4 of a word are the two halves of an operand register.
//   V: element e = r + 8 (8 w + p) is nibble p of word (D/64) r + w: the rows
//      r, r + 8, ... of V^T that lane group r owns.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace attn47 {

constexpr int kKv4Slots = 16;

// Bytes of a record, in a form the host-side checks can use too.
inline constexpr size_t kv4_record_bytes_of(int d, int group) {
  return static_cast<size_t>(2 * kKv4Slots) * (d / 2) + static_cast<size_t>(2 * kKv4Slots) * (d / group) * 4;
}

template <int D, int G>
struct Kv4Layout {
  static constexpr int kRow = D / 2;                         // bytes of a row's codes
  static constexpr int kGroups = D / G;
  static constexpr int kParRow = kGroups * 4;                // bytes of a row's parameters
  static constexpr int kOffV = kKv4Slots * kRow;
  static constexpr int kOffParK = 2 * kKv4Slots * kRow;
  static constexpr int kOffParV = kOffParK + kKv4Slots * kParRow;
  static constexpr int kBytes = kOffParV + kKv4Slots * kParRow;
  static_assert(kBytes == kv4_record_bytes_of(D, G), "record size");
  static_assert(kBytes % 128 == 0, "records are copied whole, 16-byte aligned");
};

// One step of a transposition of 4-bit cells over lanes: with lane bit `s`
// and cell blocks of `s` cells, swaps the off-diagonal blocks.
template <int S>
__device__ __forceinline__ uint32_t nibble_swap(uint32_t x, int lane) {
  constexpr uint32_t lo = S == 4 ? 0x0000ffffu : S == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;
  const uint32_t y = __shfl_xor_sync(0xffffffffu, x, S);
  return (lane & S) ? (x & ~lo) | ((y >> (4 * S)) & lo) : (x & lo) | ((y & lo) << (4 * S));
}

// K rows: lane j of the D/8 lanes of a row holds elements 8 j .. 8 j + 7 with
// element 2 c + h in nibble c + 4 h; afterwards it holds the row's word
// (D/32) (j % 4) + j / 4.  The steps are their own inverse.
__device__ __forceinline__ uint32_t kv4_k_transpose(uint32_t x, int lane) {
  x = nibble_swap<2>(x, lane);
  return nibble_swap<1>(x, lane);
}
template <int D>
__device__ __forceinline__ int kv4_k_word(int j) { return (D / 32) * (j & 3) + (j >> 2); }

// V rows: lane j holds elements 8 j .. 8 j + 7 in nibbles 0 .. 7; afterwards
// the row's word (D/64) (j % 8) + j / 8.  The steps are their own inverse.
__device__ __forceinline__ uint32_t kv4_v_transpose(uint32_t x, int lane) {
  x = nibble_swap<4>(x, lane);
  x = nibble_swap<2>(x, lane);
  return nibble_swap<1>(x, lane);
}
template <int D>
__device__ __forceinline__ int kv4_v_word(int j) { return (D / 64) * (j & 7) + (j >> 3); }

}  // namespace attn47
