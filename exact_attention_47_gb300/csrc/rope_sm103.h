// Internal launcher interface of the rotary-position kernels: rotation of
// queries and keys, and the paged appends that rotate on the way (not part
// of the C-ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace attn47 {

// Rows of d bf16 values: head h of token n of batch b starts at
// data + b batch + n token + h head (in elements).
struct HeadRows {
  void* data = nullptr;
  long long batch = 0, token = 0, head = 0;
  int heads = 0;
};

struct RopeSpec {
  const float* inv_freq = nullptr;   // [rot / 2] fp32 (device)
  int rot = 0;                       // leading elements of a head that rotate (a multiple of 16)
  bool interleaved = false;          // pairs (2p, 2p + 1) instead of (p, p + rot / 2)
  bool inverse = false;              // rotate by the negative angle
  uint32_t pair_axis[4] = {0, 0, 0, 0};   // axis of pair p: bits 2p, 2p + 1
  const int* positions = nullptr;    // axis a, batch b, token n at a axis_stride + b batch_stride + n
  long long axis_stride = 0, batch_stride = 0;
};

struct RopeLaunch {
  RopeSpec spec;
  HeadRows q, k, q_out, k_out;       // k.heads == 0: queries only
  int B, N, d;
  int sms;
  cudaStream_t stream;
};

// New tokens appended to a paged cache: bf16 (k_cache, v_cache) or 4-bit
// records (kv_cache, group).  spec.positions == nullptr: rotate by the cache
// positions.
struct RopeAppendLaunch {
  RopeSpec spec;
  HeadRows q, k, v, q_out;           // q.heads == 0: keys and values only
  void* k_cache = nullptr;           // [num_blocks, Hkv, 16, d] bf16
  void* v_cache = nullptr;
  void* kv_cache = nullptr;          // [num_blocks, Hkv, record] bytes
  int group = 0;
  const int* block_table;            // [num_seqs, max_blocks]
  const int* seq_ids;                // [T]
  const int* positions;              // [T]
  int T, num_seqs, max_blocks, num_blocks, d;
  int sms;
  unsigned int* status;
  cudaStream_t stream;
};

struct Kv4ReadLaunch {
  const void* kv_cache;              // [num_blocks, Hkv, record] bytes
  const int* block_table;
  const int* seq_ids;
  const int* positions;
  void* k;                           // [T, Hkv, d] bf16
  void* v;
  int T, Hkv, d, group, num_seqs, max_blocks, num_blocks;
  int sms;
  unsigned int* status;
  cudaStream_t stream;
};

cudaError_t launch_rope_sm103(const RopeLaunch& a);
cudaError_t launch_rope_append_sm103(const RopeAppendLaunch& a);
cudaError_t launch_kv4_read_sm103(const Kv4ReadLaunch& a);

}  // namespace attn47
