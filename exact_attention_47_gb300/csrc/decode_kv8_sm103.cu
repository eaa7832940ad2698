// Attention of one query, or of a few, of each sequence over a paged KV cache
// held in 8 bits, for sm_103a.
//
// A value is an e4m3 code times the scale of its block, head and kind:
//   s_j = c scale_K (q . code_j),     o = sum over blocks scale_V (sum_j p_j code_j)
// so the codes, exact in fp16, are the operands of the warp MMAs (one conversion
// instruction for two of them), and a block's scales meet 16 x 8 scores and a
// block's sums, in fp32.  q enters in fp16 at a power of two of its head's own
// (its largest element in [2^14, 2^15): every bf16 element within 2^-31 of it
// stays exact); the numerators p are rounded to fp16's 11 bits, at 2^10 for the
// largest so far, so that those 2^-34 below it still count.
//
// The MMAs are 16 tokens x 8 rows (S^T = K q^T) and 16 elements x 8 rows (O^T = V^T
// P^T): the 16 slots of a block fill the MMA's rows, up to 8 query rows of a KV head
// its columns; two column tiles make 16, three (d = 64) 24.  P^T changes operand
// layout with movmatrix.  Which elements an MMA's columns of k are is free as long
// as both operands agree, and so is which token an MMA row is, so a lane takes
// neighbouring bytes: with r = lane / 4 and c = lane % 4, D/4 of two K rows (tokens
// of MMA rows r and r + 8) and D/8 of four V rows (those of MMA rows 2 c, 2 c + 1, 2
// c + 8, 2 c + 9), whose bytes are paired by token with byte permutations.
//
// The N queries of a sequence (draft tokens: its last N tokens) are rows like the
// heads that share a KV head, but for the keys they see: row i sees keys up to
// L - N + i.  More than 16 rows (d = 64: 24) go in several groups, each its own pass.
//
// Work split: see decode_split.cuh.  A warp streams the records of its blocks
// through a ring of its own in shared memory: the codes as one box of a tensor map
// over the records, 128-byte lines with TMA's 128-byte swizzle (16-byte piece p of
// line l at p ^ (l mod 8)), under which the loads above meet no bank twice; the
// scales as 16 bytes more.  (Copied by the lanes themselves, 16 bytes each of just
// what they use, 8 sequences of 30k .. 131k tokens took 79 us: a warp's scattered
// 16-byte copies cost the memory pipe 21 passes where the bytes make 4.)
//
// Measured (GB300, replayed graphs): 8 sequences of 30000 .. 131072 tokens, 16 heads
// over 2, d = 128 (346 MB) 64.3 us, 5.4 TB/s or 0.81 of a copy; 64 of 128 .. 4096, 12
// heads over 2 (70 MB) 19.2 us, of which 4 are dependent reads before the first block
// and 4 to 5 the merges at the end; 256 of 0 .. 2048, 64 heads over 4, d = 64 (139 MB)
// 40.8 us: two column tiles, 345 instructions a block (ends included) issued in 49 % of
// the cycles by the three warps that a scheduler's registers hold; one sequence of 100 tokens 6.4
// us, a chain of dependent steps.
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_kv8_sm103.h"
#include "decode_split.cuh"
#include "kv8.cuh"
#include "ptx.cuh"

namespace attn47 {
namespace {

// Lazy stabilisers (see attn_decode_paged): the running maximum moves only when a
// score exceeds it by more than kTau (log2 units).
constexpr float kTau = 4.f;
// A numerator is 2^kHigh for a score at the maximum, at most 2^(kHigh + kTau).
constexpr float kHigh = 10.f;

// NT: column tiles of 8 query rows (1 .. 3 with D = 64, 1 or 2 with D = 128).
template <int D, int NT>
struct DecKv8Cfg {
  using Rec = Kv8Layout<D>;
  static constexpr int kWarps = (D == 64 && NT <= 2) || NT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = D == 64 || NT == 2 ? 4 : 3;
  static constexpr int kBlocks = D == 64 || NT == 2 ? 2 : 1;      // taken at a time
  static constexpr int kStage = Rec::kOffTail;               // its scales are apart
  static constexpr int kRows = NT * 8;                       // rows of a piece
  static constexpr int kPitch = D + 4;                       // floats
  static constexpr int kPiece = kRows * kPitch * 4;
  // Per warp; its last piece takes the ring's place.
  static constexpr int kRing = kStages * kStage > kPiece ? kStages * kStage : (kPiece + 1023) / 1024 * 1024;
  static constexpr int kOffFirst = kWarps * kRing;           // first pieces, one per warp
  static constexpr int kOffTails = kOffFirst + kWarps * kPiece;         // [warp][kStages][16]
  static constexpr int kOffMl = kOffTails + kWarps * kStages * 16;      // (max, sum): [warp][2][kRows]
  static constexpr int kOffPlan = kOffMl + kWarps * 2 * kRows * 8;
  static constexpr int kOffSrc = kOffPlan + (3 * kPlan + 4) * 4;        // record numbers: [warp][2 batches of 32]
  static constexpr int kOffShared = (kOffSrc + kWarps * 64 * 4 + 15) / 16 * 16;
  static constexpr int kSmem = kOffShared + 3072 + 1024;     // + alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages < 32, "the next batch of records is there in time");
};
struct DecKv8Shared : SplitShared {
  uint64_t full[16][8];
};
static_assert(sizeof(DecKv8Shared) <= 3072, "shared control block");

struct DecKv8Params {
  const __nv_bfloat16* q;
  const uint8_t* kv_cache;
  const int* block_table;
  const int* seq_lens;
  __nv_bfloat16* o;
  float* lse;
  float* ws_o;                     // [2 kMaxCtas][group][D]
  float* ws_ml;                    // [2 kMaxCtas][group][2]
  unsigned long long* arrive;      // [kMaxCtas]
  int num_seqs, max_blocks, num_blocks;
  int Hq;                          // rows of a sequence: its heads times N
  int Hkv;                         // runs of a sequence: KV heads times groups of rows
  int kv_heads, rows, group, groups;   // rows of a KV head (Hq / Hkv N) in `groups` groups of up to `group`
  int N;
  unsigned int epoch;
  int early_plan;                  // plan before waiting for the preceding kernel
  float scale_log2;
  unsigned int* status;
  unsigned long long timeout_ns;
  __device__ __forceinline__ size_t row0(int b, int g) const {
    const int head = g / groups;
    return static_cast<size_t>(b) * Hq + static_cast<size_t>(head) * rows + static_cast<size_t>(g - head * groups) * group;
  }
  __device__ __forceinline__ int rows_of(int g) const { return min(group, rows - g % groups * group); }
};

template <int D>
struct DecKv8Costs {
  // What a merge across CTAs costs, in half blocks.  Teams against equal shares, where
  // 14 decides for teams and 7 does not (us; sequences x tokens, KV heads): 32 x 500 ..
  // 1000, 8, 16.1 and 16.7; 32 x 500 .. 1000, 2, 11.6 and 12.5; 24 instead of 12 with
  // d = 64 changes nothing.
  static constexpr int spare2 = D == 128 ? 14 : 12;
  // What a run costs beyond its blocks: a long share spends about 4 blocks' time on
  // one (its queries, its end).  A share is at least this and one more, though, so
  // with fewer blocks than shares it is 1.  Measured with 1, 3 and 4 (us): 256
  // sequences of up to 2048 tokens, 4 KV heads, d = 64, 46.6 42.2 40.6 (6: 40.6); 64 of
  // 128 .. 4096, 2 heads, d = 128, 19.8 19.4 19.4; with 1 and 4 always, 3 of 2000, 2
  // heads, d = 64, 9.3 11.0.
  __device__ __forceinline__ int run_cost(int total, int shares) const { return total <= shares ? 1 : 4; }
};

template <int N>
__device__ __forceinline__ void load_bytes(uint32_t address, uint32_t (&r)[N]) {
  static_assert(N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(address)
                 : "memory");
  else
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(address) : "memory");
}

// Where a lane's bytes lie in a stage.
template <int D>
struct LaneData {
  static constexpr int kVBytes = D / 8;          // of a V row
  uint32_t k[D / 64];                            // 16-byte pieces of MMA row r's K row; r + 8's lie k_next() on
  uint32_t v[2];                                 // V rows of MMA rows 2 c and 2 c + 1; 8 more, v_next() on
  int slot, slot_v;                              // slot of MMA row r (of r + 8: kNext more), of V row 2 c
  // D = 128: a line is a row, an MMA row is its slot.  A K load's 8 lanes at a time
  // are pieces 2 c + j of two neighbouring rows, a V load's are pieces r of rows
  // 2 c: all eight places each.  D = 64: a line is two rows; MMA rows 2 c, 2 c + 1,
  // 2 c + 8, 2 c + 9 are slots 4 c .. 4 c + 3, so that the V rows of a load lie in
  // every other line.
  static constexpr int kNext = D == 128 ? 8 : 2;
  __device__ __forceinline__ explicit LaneData(int lane) {
    const uint32_t r = static_cast<uint32_t>(lane) >> 2, c = static_cast<uint32_t>(lane) & 3u;
    if constexpr (D == 128) {
      slot = static_cast<int>(r);
      slot_v = static_cast<int>(2 * c);
#pragma unroll
      for (uint32_t j = 0; j < D / 64; ++j) k[j] = 128 * r + 16 * ((2 * c + j) ^ r);
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) v[i] = 16 * D + 128 * (2 * c + i) + 16 * (r ^ (2 * c + i));
    } else {
      slot = static_cast<int>(4 * (r >> 1) + (r & 1));
      slot_v = static_cast<int>(4 * c);
      const uint32_t line = 2 * (r >> 1);
      k[0] = 128 * line + 16 * ((4 * (r & 1) + c) ^ line);
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) v[i] = 16 * D + 128 * (2 * c) + 16 * ((4 * i + (r >> 1)) ^ (2 * c)) + 8 * (r & 1);
    }
  }
  // From MMA row r to r + 8: D = 128: 8 lines on, the same place; D = 64: the next
  // line, whose number ends in 1 instead of 0.
  __device__ __forceinline__ uint32_t k_next(int j) const { return D == 128 ? k[j] + 8 * 128 : (k[j] + 128) ^ 16u; }
  __device__ __forceinline__ uint32_t v_next(int i) const { return D == 128 ? v[i] + 8 * 128 : (v[i] + 128) ^ 16u; }
};

// Queries of one run as B operands, and what undoes their scaling.
template <int D, int NT>
struct QueryFrag {
  uint32_t b[NT][D / 16][2];       // elements D/4 c + 4 i + {0, 1}, {2, 3} of row lane / 4 for MMA i
  float back[NT][2];               // score factor of rows 2 c, 2 c + 1
  int behind[NT][2];               // how many of the sequence's last keys those rows do not see
};

template <int D, int NT>
struct QueryRaw {
  uint4 w[NT][D / 32];
  __device__ __forceinline__ void load(const DecKv8Params& p, int b, int g, int lane) {
    const int rows = p.rows_of(g);
    const __nv_bfloat16* first = p.q + p.row0(b, g) * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + (lane >> 2);
      const bool live = row < rows;
      const uint4* src = reinterpret_cast<const uint4*>(first + static_cast<size_t>(live ? row : 0) * D) +
                         D / 32 * (lane & 3);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) w[nt][j] = live ? src[j] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

template <int D, int NT>
__device__ __forceinline__ void make_queries(const DecKv8Params& p, const QueryRaw<D, NT>& all, int g, int lane,
                                             QueryFrag<D, NT>& f) {
  const int c = lane & 3;
  const int first = g % p.groups * p.group;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t raw[D / 16][2];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint4 x = all.w[nt][j];
      raw[2 * j][0] = x.x;
      raw[2 * j][1] = x.y;
      raw[2 * j + 1][0] = x.z;
      raw[2 * j + 1][1] = x.w;
    }
    uint32_t mx = 0;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      mx = __vmaxu2(mx, raw[s][0] & 0x7fff7fffu);
      mx = __vmaxu2(mx, raw[s][1] & 0x7fff7fffu);
    }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // Largest element in [2^(E-127), 2^(E-126)); times 2^(141-E) it is in
    // [2^14, 2^15).
    const int fe = min(268 - static_cast<int>(mx >> 7), 253);
    const float up = __uint_as_float(static_cast<uint32_t>(fe) << 23);
    const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - fe) << 23);
    f.back[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
    f.back[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f.b[nt][s][h] = pack_f16x2(__uint_as_float(raw[s][h] << 16) * up, __uint_as_float(raw[s][h] & 0xffff0000u) * up);
#pragma unroll
    for (int h = 0; h < 2; ++h) f.behind[nt][h] = p.N - 1 - (first + nt * 8 + 2 * c + h) % p.N;
  }
}

// Running state of one run: O^T tiles, stabilisers and sums, all in units of
// 2^stab per row.
template <int D, int NT>
struct RunState {
  float o[NT][D / 16][4];          // tile i: elements 2 i, 2 i + 1 of the lane's D/8, rows 2 c, 2 c + 1 each
  float stab[NT][2], l[NT][2];
  float limit[NT][2];              // score from which the stabiliser has to move

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      // (A block without visible tokens may come first: its numerators are then
      // ex2(-inf + 3e38) = 0.)
      stab[nt][0] = stab[nt][1] = -3e38f;
      limit[nt][0] = limit[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
  }

  // Moves the stabilisers for scores up to s; rare, and the same for the whole
  // warp.
  __device__ __forceinline__ void move(const float (&s)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = s[nt][h];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float top = __fadd_rd(stab[nt][h], kHigh);   // the running maximum
        // (To a multiple of 2^-10, so that adding whole numbers to a stabiliser,
        // here and for the LSE, rounds nothing.  Beyond 2^13 every fp32 number is one;
        // beyond 2^24 kHigh and kTau round themselves, so that a numerator is never more
        // than 2^(kHigh + kTau) and the stabiliser never creeps up.)
        const float most = mx > limit[nt][h] ? mx : top;
        const float to = __fsub_ru(fabsf(most) < 8192.f ? __fsub_rn(__fadd_rn(most, kGrid), kGrid) : most, kHigh);
        f[h] = to == stab[nt][h] ? 1.f : ex2(stab[nt][h] - to);
        stab[nt][h] = to;
        limit[nt][h] = __fadd_rd(to, kHigh + kTau);
        l[nt][h] *= f[h];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        o[nt][i][0] *= f[0];
        o[nt][i][1] *= f[1];
        o[nt][i][2] *= f[0];
        o[nt][i][3] *= f[1];
      }
    }
  }

  // Sums over the token rows of the warp.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], x);
  }

  // Element k of the lane's D/8 of row 2 c + h of tile nt.
  __device__ __forceinline__ float at(int nt, int k, int h) const { return o[nt][k >> 1][(k & 1) * 2 + h]; }
};

// NB blocks of a run, 16 slots each, in stages of the ring, their scales at
// `tail_at`; `valid` tokens from a block's first slot to the sequence's end (16 or
// more: all slots hold tokens; 0 or less: none, whatever the stage holds), in each
// block at least `least` of them seen by every row.
template <int D, int NT, int NB>
__device__ __forceinline__ void take_blocks(const LaneData<D>& at, const uint32_t (&stage)[NB],
                                            const uint32_t (&tail_at)[NB], const int (&valid)[NB], int least,
                                            const QueryFrag<D, NT>& q, RunState<D, NT>& st) {
  using Ld = LaneData<D>;

  // --- S^T: rows = slots, columns = query rows
  float s[NB][NT][4];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    float even[NT][4], odd[NT][4];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t a[4], b[4];
      load_bytes(stage[n] + at.k[j], a);
      load_bytes(stage[n] + at.k_next(j), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = e4m3x2_to_f16x2(a[i]), a1 = e4m3x2_to_f16x2(b[i]), a2 = e4m3x2_hi_to_f16x2(a[i]),
                       a3 = e4m3x2_hi_to_f16x2(b[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float (&acc)[4] = i & 1 ? odd[nt] : even[nt];
          if (j == 0 && i < 2)
            mma_16816_f16_first(acc, a0, a1, a2, a3, q.b[nt][4 * j + i][0], q.b[nt][4 * j + i][1]);
          else
            mma_16816_f16(acc, a0, a1, a2, a3, q.b[nt][4 * j + i][0], q.b[nt][4 * j + i][1]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][nt][i] = even[nt][i] + odd[nt][i];
  }

  float scale_v[NB];
  uint32_t flags[NB], any_flags = 0;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    uint32_t tail[4];
    load_bytes(tail_at[n], tail);
    const float scale_k = __uint_as_float(tail[0]);
    scale_v[n] = __uint_as_float(tail[1]);
    flags[n] = tail[2];
    any_flags |= tail[2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // (Finite, so that a score of 0 stays 0: queries of 2^78 beside keys of 2^64.)
      const float f0 = fminf(q.back[nt][0] * scale_k, 3.402823466e38f), f1 = fminf(q.back[nt][1] * scale_k, 3.402823466e38f);
      s[n][nt][0] *= f0;
      s[n][nt][1] *= f1;
      s[n][nt][2] *= f0;
      s[n][nt][3] *= f1;
    }
  }
  uint32_t v[NB][4][Ld::kVBytes / 4];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) load_bytes(stage[n] + (i < 2 ? at.v[i & 1] : at.v_next(i & 1)), v[n][i]);

  if (least < kBS || any_flags != 0) {           // (the same for the whole warp)
    // Slots that a row does not see have no score, those past the end no value;
    // a row that sees a flagged token has NaN for a score.
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint32_t bad = valid[n] > 0 ? flags[n] | (flags[n] >> 16) : 0u;
      if (valid[n] <= 0) scale_v[n] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = at.slot + (i >> 1) * Ld::kNext;
          if (slot >= valid[n] - q.behind[nt][i & 1])
            s[n][nt][i] = -INFINITY;
          else if ((bad >> slot) & 1u)
            s[n][nt][i] = __uint_as_float(0x7fc00000u);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = at.slot_v + (i & 1) + (i >> 1) * Ld::kNext;
        if (slot >= valid[n] || ((bad >> slot) & 1u)) {
#pragma unroll
          for (int w = 0; w < Ld::kVBytes / 4; ++w) v[n][i][w] = 0;
        }
      }
    }
  }

  float top[NT][2];
  bool move = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[nt][h] = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
#pragma unroll
      for (int n = 1; n < NB; ++n) top[nt][h] = fmax3(top[nt][h], s[n][nt][h], s[n][nt][2 + h]);
      move |= top[nt][h] > st.limit[nt][h];
    }
  if (__any_sync(0xffffffffu, move)) st.move(top);

  // --- numerators and O^T: rows = elements of V, columns = query rows
  uint32_t pw[NB][NT][2];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float p0 = ex2(s[n][nt][0] - st.stab[nt][0]), p1 = ex2(s[n][nt][1] - st.stab[nt][1]);
      const float p2 = ex2(s[n][nt][2] - st.stab[nt][0]), p3 = ex2(s[n][nt][3] - st.stab[nt][1]);
      st.l[nt][0] += p0 + p2;
      st.l[nt][1] += p1 + p3;
      pw[n][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
      pw[n][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
    }
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const uint64_t sv = f2_pack(scale_v[n], scale_v[n]);
#pragma unroll
    for (int w = 0; w < Ld::kVBytes / 4; ++w) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t sel = hf ? 0x7362u : 0x5140u;         // (token, next token) of two elements
        const uint32_t x = __byte_perm(v[n][0][w], v[n][1][w], sel), y = __byte_perm(v[n][2][w], v[n][3][w], sel);
        const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_hi_to_f16x2(x), a2 = e4m3x2_to_f16x2(y),
                       a3 = e4m3x2_hi_to_f16x2(y);
        const int i = 2 * w + hf;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4];
          mma_16816_f16_first(acc, a0, a1, a2, a3, pw[n][nt][0], pw[n][nt][1]);
          f2_unpack(f2_fma(f2_pack(acc[0], acc[1]), sv, f2_pack(st.o[nt][i][0], st.o[nt][i][1])), st.o[nt][i][0],
                    st.o[nt][i][1]);
          f2_unpack(f2_fma(f2_pack(acc[2], acc[3]), sv, f2_pack(st.o[nt][i][2], st.o[nt][i][3])), st.o[nt][i][2],
                    st.o[nt][i][3]);
        }
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(DecKv8Cfg<D, NT>::kThreads, 1)
    attn_decode_kv8_kernel(const __grid_constant__ CUtensorMap records, const __grid_constant__ DecKv8Params p) {
  using Cfg = DecKv8Cfg<D, NT>;
  using Rec = Kv8Layout<D>;
  constexpr int kWarps = Cfg::kWarps, kStages = Cfg::kStages, kRows = Cfg::kRows, NB = Cfg::kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  DecKv8Shared* sh = reinterpret_cast<DecKv8Shared*>(smem + Cfg::kOffShared);
  int* cost = reinterpret_cast<int*>(smem + Cfg::kOffPlan);             // [kPlan + 1]
  int* runs = cost + kPlan + 2;                                         // [kPlan + 1]
  int* seq_blocks = runs + kPlan + 2;                                   // [kPlan]
  float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffMl);           // [warp][2][kRows]
  auto first_piece = [&](int w) { return reinterpret_cast<float*>(smem + Cfg::kOffFirst + w * Cfg::kPiece); };
  auto last_piece = [&](int w) { return reinterpret_cast<float*>(smem + w * Cfg::kRing); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    sh->part_n[0] = sh->part_n[1] = 0;
    sh->abort = 0;
  }
  static_assert(kStages <= 8, "");
  if (lane < kStages) mbar_init(smem_addr(&sh->full[warp][lane]), 1);
  if (lane == kStages) mbar_init(smem_addr(&sh->ready[warp]), 1);
  fence_mbar_init();
  if (tid == 0) {
    prefetch_tmap(&records);
    prefetch_inputs<D>(p);
  }
  // With the early plan, seq_lens and the block table are read before the
  // preceding kernel has finished; the queries, the cache and everything that
  // is written come after the wait further down.
  if (!p.early_plan) pdl_wait_primary();

  const Plan plan = build_plan<kWarps>(p, sh, cost, runs, seq_blocks, DecKv8Costs<D>());
  __syncthreads();
  Share share = take_share<kWarps>(p, plan, sh);
  Walk& w = share.w;
  const int blocks = share.blocks;
  const WaitCtl wc{&sh->abort, p.status, p.timeout_ns};
  WarpMeta meta = {};

  if (blocks > 0) {
    w.left = blocks;
    // The first run's queries are on their way while the table is read.
    QueryRaw<D, NT> raw;
    if (!p.early_plan) raw.load(p, w.at.b, w.at.g, lane);
    // Lane j looks up block j of every batch of 32, two batches ahead, and
    // leaves its record's number for the issuing lane (-1: not in the pool).
    // Returns the batch's mask of blocks that have a record.
    Walk ahead = w;
    ahead.skip(p, plan, lane);
    int* src = reinterpret_cast<int*>(smem + Cfg::kOffSrc) + warp * 64;
    auto fetch = [&](int batch) {
      int rec = -1;
      if (ahead.left > 0) {
        const int ph = p.block_table[static_cast<size_t>(ahead.at.b) * p.max_blocks + ahead.at.blk];
        if (static_cast<unsigned>(ph) < static_cast<unsigned>(p.num_blocks))
          rec = ph * p.kv_heads + ahead.at.g / p.groups;
        else
          atomicOr(p.status, kDevBadBlock);      // outside the pool: that block is skipped
      }
      ahead.skip(p, plan, 32);
      src[(batch & 1) * 32 + lane] = rec;
      return __ballot_sync(0xffffffffu, rec >= 0);
    };
    const uint64_t policy = l2_policy_evict_first();
    unsigned present = fetch(0);
    if (p.early_plan) {
      pdl_wait_primary();
      raw.load(p, w.at.b, w.at.g, lane);
    }
    __syncwarp();
    const uint32_t ring_at = smem_addr(smem + warp * Cfg::kRing);
    const uint32_t tails = smem_addr(smem + Cfg::kOffTails) + warp * kStages * 16;
    const uint32_t bars = smem_addr(&sh->full[warp][0]);
    const LaneData<D> at(lane);
    // Block i of the share goes to stage i % kStages; blocks [0, taken + kStages)
    // are issued.  (One lane.)
    auto issue = [&](int i, int stage) {
      const int rec = src[i & 63];
      const uint32_t bar = bars + stage * 8;
      mbar_arrive_expect_tx(bar, rec >= 0 ? Cfg::kStage + 16 : 0);
      if (rec >= 0) {
        tma_load_3d_hint(ring_at + stage * Cfg::kStage, &records, bar, 0, 0, rec, policy);
        bulk_load_hint(tails + stage * 16, p.kv_cache + static_cast<size_t>(rec) * Rec::kBytes + Rec::kOffTail, 16, bar,
                       policy);
      }
    };
    if (lane < min(blocks, kStages)) issue(lane, lane);
    unsigned next_present = blocks > 32 ? fetch(1) : 0u;
    __syncwarp();
    announce_parts<kWarps>(p, plan, sh, share);

    QueryFrag<D, NT> q;
    RunState<D, NT> st;
    int taken = 0, stage = 0;
    uint32_t parity = 0;
    bool fail = false;
    while (w.left > 0 && !fail) {
      const int cnt = w.count();
      int valid = seq_len_of(p, w.at.b) - w.at.blk * kBS;       // tokens from this block on
      if (taken > 0) raw.load(p, w.at.b, w.at.g, lane);
      make_queries<D, NT>(p, raw, w.at.g, lane, q);
      st.reset();
      for (const int end = taken + cnt; taken < end;) {
        // Without a second block the first one's stage stands in, with no slot of
        // it alive.
        const bool two = NB == 2 && taken + 1 < end;
        const int next_stage = stage + 1 == kStages ? 0 : stage + 1;
        if (!wait_warp(bars + stage * 8, parity, wc) ||
            (two && !wait_warp(bars + next_stage * 8, next_stage == 0 ? parity ^ 1 : parity, wc))) {
          fail = true;
          break;
        }
        uint32_t rec_at[NB], tail_at[NB];
        int alive[NB];
        rec_at[0] = ring_at + stage * Cfg::kStage;
        tail_at[0] = tails + stage * 16;
        alive[0] = (present >> (taken & 31)) & 1u ? valid : 0;
        int least = alive[0];
        if constexpr (NB == 2) {
          rec_at[1] = two ? ring_at + next_stage * Cfg::kStage : rec_at[0];
          tail_at[1] = two ? tails + next_stage * 16 : tail_at[0];
          alive[1] = two && ((taken & 31) == 31 ? next_present & 1u : (present >> ((taken + 1) & 31)) & 1u) ? valid - kBS : 0;
          least = min(least, alive[1]);
        }
        take_blocks<D, NT, NB>(at, rec_at, tail_at, alive, least - (p.N - 1), q, st);
        __syncwarp();                            // every lane has read the stages
        const int n = two ? 2 : 1;
        if (lane < n && taken + lane + kStages < blocks) issue(taken + lane + kStages, lane ? next_stage : stage);
        valid -= n * kBS;
        if (((taken + n) ^ taken) & 32) {        // (what is issued is less than a batch ahead)
          present = next_present;
          next_present = ((taken + n) & ~31) + 32 < blocks ? fetch(((taken + n) >> 5) + 1) : 0u;
          __syncwarp();
        }
        taken += n;
        stage += n;
        if (stage >= kStages) {
          stage -= kStages;
          parity ^= 1;
        }
      }
      if (fail) break;
      st.finish();
      const bool has_start = w.at.blk == 0, has_end = w.at.blk + cnt == w.at.nblk;
      const int c = lane & 3, r = lane >> 2;
      bool whole = has_start && has_end;
      // A run that lies in two neighbouring warps' shares is finished by the
      // one that holds its start, from the piece that the other one, to which
      // it was the first thing to do, has left: with runs about as long as
      // shares that is most of them, and at the CTA's end they would queue.
      const int run0 = w.at.cost + plan.run_cost, run1 = run0 + w.at.nblk;
      const longlong2 reach = sh->reach[warp];
      const bool to_previous = has_end && !has_start && warp > 0 && run0 >= reach.x;
      if (has_start && !has_end && warp + 1 < kWarps && run1 <= reach.y) {
        if (!wait_warp(smem_addr(&sh->ready[warp + 1]), 0, wc)) {
          fail = true;
          break;
        }
        const float* from = first_piece(warp + 1) + r * (D / 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = nt * 8 + 2 * c + h;
            const float2 v = ml[(warp + 1) * 2 * kRows + row];
            const float to = fmaxf(st.stab[nt][h], v.x);
            const float f0 = ex2(st.stab[nt][h] - to), f1 = ex2(v.x - to);
            st.stab[nt][h] = to;
            st.l[nt][h] = st.l[nt][h] * f0 + v.y * f1;
#pragma unroll
            for (int k = 0; k < D / 8; k += 4) {
              const float4 x = *reinterpret_cast<const float4*>(from + row * Cfg::kPitch + k);
              float (&y0)[4] = st.o[nt][k / 2], (&y1)[4] = st.o[nt][k / 2 + 1];
              y0[h] = y0[h] * f0 + x.x * f1;
              y0[2 + h] = y0[2 + h] * f0 + x.y * f1;
              y1[h] = y1[h] * f0 + x.z * f1;
              y1[2 + h] = y1[2 + h] * f0 + x.w * f1;
            }
          }
        }
        whole = true;
      }
      if (whole) {
        const size_t h0 = p.row0(w.at.b, w.at.g);
        const int rows = p.rows_of(w.at.g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = nt * 8 + 2 * c + h;
            const float l = st.l[nt][h];
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (row < rows) {
              uint4* dst = reinterpret_cast<uint4*>(p.o + (h0 + row) * D + r * (D / 8));
#pragma unroll
              for (int k = 0; k < D / 8; k += 8) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[i] = pack_bf16x2(st.at(nt, k + 2 * i, h) * inv, st.at(nt, k + 2 * i + 1, h) * inv);
                dst[k / 8] = make_uint4(x[0], x[1], x[2], x[3]);
              }
              if (p.lse != nullptr && r == 0) p.lse[h0 + row] = l == 0.f ? -INFINITY : lse_of(st.stab[nt][h], l);
            }
          }
        }
      } else {
        // A piece: in the first-piece buffer if the run ends here, else in
        // this warp's ring, which has nothing more to take.
        const bool f = has_end;
        float* dst = (f ? first_piece(warp) : last_piece(warp)) + r * (D / 8);
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = nt * 8 + 2 * c + h;
#pragma unroll
            for (int k = 0; k < D / 8; k += 4)
              *reinterpret_cast<float4*>(dst + row * Cfg::kPitch + k) =
                  make_float4(st.at(nt, k, h), st.at(nt, k + 1, h), st.at(nt, k + 2, h), st.at(nt, k + 3, h));
            if (r == 0) ml[(warp * 2 + (f ? 0 : 1)) * kRows + row] = make_float2(st.stab[nt][h], st.l[nt][h]);
          }
        }
        if (to_previous) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh->ready[warp]));
        } else if (f) {
          meta.f_valid = 1;
          meta.fb = w.at.b;
          meta.fg = w.at.g;
        } else {
          meta.l_valid = 1;
          meta.l_start = has_start;
          meta.lb = w.at.b;
          meta.lg = w.at.g;
        }
      }
      w.next_run(p, plan, cnt);
    }
    if (fail) {
      // Copies in flight must land before the CTA may exit.
      for (int s = 0; s < kStages; ++s) {
        const int issued = min(blocks, taken + kStages);
        const int fills = issued / kStages + (s < issued % kStages ? 1 : 0);
        if (fills > 0) mbar_wait_warp_drain(bars + s * 8, static_cast<uint32_t>((fills - 1) & 1), wc);
      }
    }
  }
  if (p.early_plan) pdl_wait_primary();          // (warps without work)
  if (lane == 0) sh->meta[warp] = meta;
  write_empty_sequences<kWarps, D>(p, plan);
  merge_pieces<Cfg, D>(p, sh, ml, first_piece, last_piece);
}

template <int D, int NT>
cudaError_t launch_t(const DecKv8Launch& a, const Kv8Rows& rows) {
  using Cfg = DecKv8Cfg<D, NT>;
  auto kern = attn_decode_kv8_kernel<D, NT>;
  // The attribute belongs to the device's copy of the kernel: set once for each
  // (the host's time bounds a small decode).
  static std::atomic<unsigned long long> allowed{0};
  const unsigned long long bit = 1ull << a.device;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  DecKv8Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.N = a.N;
  p.Hq = a.Hq * a.N;
  p.kv_heads = a.Hkv;
  p.rows = a.Hq / a.Hkv * a.N;
  p.group = rows.group;
  p.groups = rows.groups;
  p.Hkv = a.Hkv * rows.groups;
  p.arrive = static_cast<unsigned long long*>(a.workspace);
  p.ws_o = reinterpret_cast<float*>(p.arrive + kMaxCtas);
  p.ws_ml = p.ws_o + static_cast<size_t>(2) * kMaxCtas * p.group * D;
  p.epoch = a.epoch;
  p.early_plan = a.early_plan;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  int ctas = a.sms < 1 ? 1 : a.sms > kMaxCtas ? kMaxCtas : a.sms;
  if (a.max_ctas > 0 && ctas > a.max_ctas) ctas = a.max_ctas;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(Cfg::kThreads), Cfg::kSmem, a.stream, *a.records, p);
}

}  // namespace

Kv8Rows decode_kv8_rows(int Hq, int Hkv, int N, int d) {
  // Two column tiles a pass; three with d = 64 where their fewer passes pay (one takes
  // 1.46 times as long: 16 sequences of 6000 tokens, 4 KV heads, 24 rows in one pass
  // 30.8 us, in two 32.8; 64 rows in three 57.3, in four 53.2; 32 rows in one pass of
  // four tiles 38.9, in two of two 32.8).  With d = 128 the accumulators of three do
  // not fit beside enough warps (24 rows of 32 sequences of 500 .. 6000 tokens, 2 KV
  // heads: two passes of 12 33.3 us, one of 24 35.9); one tile a pass, with 12 warps
  // instead of 8, is faster over few tokens (24 rows of 4 of 6000: 22.5 us in three
  // passes, 26.6 in two) and slower over many (16 of 6000, 8 KV heads, more than L2
  // holds: 117 and 86).
  const int rows = Hq / Hkv * N, by16 = (rows - 1) / 16 + 1, by24 = (rows - 1) / 24 + 1;
  const int groups = d == 64 && 1.46 * by24 < by16 ? by24 : by16;
  return Kv8Rows{(rows - 1) / groups + 1, groups};
}

size_t decode_kv8_workspace_bytes(int Hq, int Hkv, int N, int d) {
  return static_cast<size_t>(kMaxCtas) * sizeof(unsigned long long) +
         static_cast<size_t>(2) * kMaxCtas * decode_kv8_rows(Hq, Hkv, N, d).group * (static_cast<size_t>(d) + 2) * sizeof(float);
}

cudaError_t launch_decode_kv8_sm103(const DecKv8Launch& a) {
  const Kv8Rows rows = decode_kv8_rows(a.Hq, a.Hkv, a.N, a.d);
  const int tiles = (rows.group + 7) / 8;
  if (a.d == 128)
    return tiles == 1 ? launch_t<128, 1>(a, rows) : launch_t<128, 2>(a, rows);
  return tiles == 1 ? launch_t<64, 1>(a, rows) : tiles == 2 ? launch_t<64, 2>(a, rows) : launch_t<64, 3>(a, rows);
}

}  // namespace attn47
