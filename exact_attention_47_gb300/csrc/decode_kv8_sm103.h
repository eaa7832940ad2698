// Internal launcher interface of the decode over an 8-bit paged cache (not
// part of the C-ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace attn47 {

struct DecKv8Launch {
  const void* q;               // [S, Hq, N, d] bf16
  const CUtensorMap* records;  // the records' codes: bytes [num_blocks Hkv][d / 4 lines][128], a record to a box,
                               // 128-byte swizzle
  const void* kv_cache;        // [num_blocks, Hkv, record] bytes
  const int* block_table;      // [S, max_blocks] int32
  const int* seq_lens;         // [S] int32
  void* o;                     // [S, Hq, N, d] bf16
  float* lse;                  // [S, Hq, N] fp32 or nullptr
  void* workspace;
  int num_seqs, Hq, Hkv, N, d, max_blocks, num_blocks;
  int sms, device;
  int max_ctas;                // 0: one CTA per SM
  unsigned int epoch;          // tag of this call's arrival counters (never 0)
  int early_plan;              // >= 1: see attn_set_decode_early_plan
  float scale;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
};

// How many query rows of a KV head share a pass over its blocks, and in how many
// groups that takes all N Hq / Hkv of them.
struct Kv8Rows {
  int group, groups;
};
Kv8Rows decode_kv8_rows(int Hq, int Hkv, int N, int d);
// Bytes of workspace: two partial results of a group's rows and one counter for
// each CTA a launch can have.
size_t decode_kv8_workspace_bytes(int Hq, int Hkv, int N, int d);
cudaError_t launch_decode_kv8_sm103(const DecKv8Launch& a);

}  // namespace attn47
