// Internal launcher interface of the decode over a 4-bit paged cache (not
// part of the C-ABI).
#pragma once

#include <cuda_runtime.h>

namespace attn47 {

struct DecKv4Launch {
  const void* q;               // [S, Hq, d] bf16
  const void* kv_cache;        // [num_blocks, Hkv, record] bytes
  const int* block_table;      // [S, max_blocks] int32
  const int* seq_lens;         // [S] int32
  void* o;                     // [S, Hq, d] bf16
  float* lse;                  // [S, Hq] fp32 or nullptr
  void* workspace;
  int num_seqs, Hq, Hkv, d, group, max_blocks, num_blocks;
  int sms, device;
  int max_ctas;                // 0: one CTA per SM
  unsigned int epoch;          // tag of this call's arrival counters (never 0)
  int early_plan;              // >= 1: see attn_set_decode_early_plan
  float scale;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
};

// Bytes of workspace: two partial results of Hq / Hkv rows and one counter
// for each CTA a launch can have.
size_t decode_kv4_workspace_bytes(int Hq, int Hkv, int d);
cudaError_t launch_decode_kv4_sm103(const DecKv4Launch& a);

}  // namespace attn47
