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

// Rows between lanes and memory.  A row is held by D/16 lanes, 16 neighbouring
// elements each, as two words of eight 4-bit cells (the 8-element pieces 2 j
// and 2 j + 1 of lane j).  In memory, cell p of a word belongs to piece p of a
// block of pieces, so packing a row is a transposition of cells over pieces:
// piece bit by piece bit the off-diagonal blocks change places, bit 0 between
// the lane's two words, the others between lanes, where blocks of 8 and 16
// bits move with one byte permutation whose selector depends on the lane.
struct CellTranspose {
  uint32_t sel8, sel16;
  __device__ __forceinline__ explicit CellTranspose(int lane) {
    sel8 = (lane & 1) ? 0x3715u : 0x6240u;
    sel16 = (lane & 2) ? 0x3276u : 0x5410u;
  }
  __device__ __forceinline__ void bit0(uint32_t (&x)[2]) const {
    const uint32_t a = x[0], b = x[1];
    x[0] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
    x[1] = (b & 0xf0f0f0f0u) | ((a >> 4) & 0x0f0f0f0fu);
  }
  __device__ __forceinline__ uint32_t bit1(uint32_t x) const {
    return __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 1), sel8);
  }
  __device__ __forceinline__ uint32_t bit2(uint32_t x) const {
    return __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 2), sel16);
  }
  // Keys: cell c + 4 h of a piece's word is its element 2 c + h; afterwards
  // piece j's word is the row's word kv4_k_word(j).  Its own inverse.
  __device__ __forceinline__ void key(uint32_t (&x)[2]) const {
    bit0(x);
    x[0] = bit1(x[0]);
    x[1] = bit1(x[1]);
  }
  // Values: cell e is element e; afterwards piece j's word is the row's word
  // kv4_v_word(j).  Its own inverse.
  __device__ __forceinline__ void value(uint32_t (&x)[2]) const {
    bit0(x);
    x[0] = bit2(bit1(x[0]));
    x[1] = bit2(bit1(x[1]));
  }
};
template <int D>
__device__ __forceinline__ int kv4_k_word(int piece) { return (D / 32) * (piece & 3) + (piece >> 2); }
template <int D>
__device__ __forceinline__ int kv4_v_word(int piece) { return (D / 64) * (piece & 7) + (piece >> 3); }

}  // namespace attn47
