// Single-token decode over a paged KV cache held in 4 bits, for sm_103a.
//
// With K[j] = code scale + min per group of elements (and V likewise), the
// scores and the output need no dequantised cache:
//   s_j = c q . K[j] = c sum_g (scale_jg (q_g . code_jg) + min_jg sum(q_g))
//   o   = sum_j p_j V[j]:  per group, sum_j (p_j scale_jg) code_j + sum_j p_j min_jg
// so the codes themselves are the operands of the warp MMAs and the
// parameters act on small accumulators.  A code in the low 10 bits of an fp16
// is the subnormal code 2^-24 (or 16 times that, four bits up), which the
// tensor core multiplies exactly: one mask per operand register is all the
// conversion there is.  The other operands are kept in fp16 at a power of
// two that loses nothing:
//   q    scaled per head so its largest element is in [2^14, 2^15): every
//        bf16 element within 2^-24 of it stays exact;
//   p scale  every group of V has a power of two that follows the largest of
//        its scales met so far, so that the products stay under 2^15 (they are
//        rounded to 11 bits: with bf16's 8 the error of O would show beside its
//        own rounding, and a second fp16 for the rest would double the output
//        MMAs).  A group's power is its own: a group of huge values, or of none
//        that are numbers, leaves the others and the softmax sums alone.
// The min terms of the scores are one more MMA (bf16, exact: sum(q_g) is split
// into three bf16 parts); those of the output are summed in fp32.
//
// The MMAs are 16 tokens x 8 heads (S^T = K q^T) and 16 elements x 8 heads
// (O^T += V^T P^T): the 16 slots of a block fill the rows and up to 8 query
// heads per KV head the columns, where 16-head rows would waste half for
// groups up to 8.  P^T changes operand layout with movmatrix.
//
// Work split: the blocks of all (sequence, KV head) runs in one flat order,
// cut into equal costs for every warp of a one-wave grid (a run costs a few
// blocks more than it has, for its queries and its end), or a team of a CTA's
// warps to each run where that is shorter.  A warp
// streams its blocks through a ring of its own in shared memory, one bulk copy
// per (block, head) record, and keeps its own running softmax, so nothing
// inside the CTA waits for anything else until the end.  A run that a warp
// holds whole is written by it; pieces of a run go to shared memory, are merged
// per CTA, and if the run reaches into other CTAs the merged part is published
// and the CTA that arrives last merges the parts.
//
// What bounds it (GB300, one column tile, d = 128): further blocks of long
// contexts stream at 6.1 TB/s (groups of 64; 6.0 with 32), near the rate of a
// copy; about 12 us of a call that fills the GPU are latency, three dependent
// reads before the first block (lengths, table, record: 4 us) and, at the end,
// the merge of a CTA's pieces, the arrival and the merge of published parts (4
// to 5 us, over 1 us for each trip to what another SM has written).  8 sequences
// of 30k .. 131k tokens (195 MB) take 45 us, 64 of 128 .. 4096 (44 MB) 18.0 us,
// one of 100 5.8 to 6.6 us.  With d = 64 (4.6 TB/s) and with two column tiles
// (3.3 at d = 64, 4.0 at d = 128) the arithmetic of a block takes longer than
// its bytes: its instructions wait on one another, at two to three warps a
// scheduler.  (A power of two to each V group instead of one for all costs 1 to
// 2%: 18.0 us instead of 17.6, 44.9 instead of 44.4.)
#include <atomic>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_kv4_sm103.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn47 {
namespace {

constexpr int kBS = kKv4Slots;
// CTAs a launch may have (one per SM); the workspace has room for this many.
constexpr int kMaxCtas = 256;
// Lazy stabilisers (see attn_decode_paged): the running maximum moves only
// when a score exceeds it by more than kTau (log2 units).
constexpr float kTau = 8.f;
// The weights p are softmax numerators times 2^-kLow: sums of p V then stay
// finite in fp32 for values up to 2^123.  With V scales brought under kFull the
// products p scale are under 2^15, which fp16 holds.
constexpr float kLow = 20.f;
constexpr float kFull = 0x1p27f;
constexpr float kGrid = 12288.f;   // 1.5 2^13: x + kGrid - kGrid is x to a multiple of 2^-10
// Entries of the plan's prefix sums (one per sequence up to this many, then
// one per several).
constexpr int kPlan = 1024;
constexpr float kLn2 = 0.6931471805599453f;

// NT: column tiles of 8 query heads (1 or 2).
template <int D, int G, int NT>
struct DecKv4Cfg {
  using Rec = Kv4Layout<D, G>;
  // 12 warps with 168 registers each, or 8 with 255 when two column tiles
  // double the accumulators.  (With one tile, d = 128, each further block of a
  // long context streams at 6.1 TB/s with 12 warps and 5.6 with 8; 16 spill,
  // and 10, uneven over the four schedulers, lose to 8.)
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  // A power of two.  (8 with d = 64, as many bytes as 4 with d = 128: 8
  // sequences of 20000 tokens, 2 KV heads, take 16.9 us instead of 14.6.)
  static constexpr int kStages = 4;
  static constexpr int kRows = NT * 8;                       // head rows of a piece
  static constexpr int kPitch = D + 4;                       // floats; conflict-free stores
  static constexpr int kPiece = kRows * kPitch * 4;
  static constexpr int kRing = kStages * Rec::kBytes;        // per warp
  static constexpr int kOffFirst = kWarps * kRing;           // first pieces, one per warp
  static constexpr int kOffMl = kOffFirst + kWarps * kPiece; // (max, sum): [warp][2][kRows]
  static constexpr int kOffPlan = kOffMl + kWarps * 2 * kRows * 8;
  static constexpr int kOffSrc = kOffPlan + (3 * kPlan + 4) * 4;        // record addresses: [warp][2 batches of 32]
  static constexpr int kOffShared = kOffSrc + kWarps * 64 * 8;
  static constexpr int kSmem = kOffShared + 2048 + 128;      // + alignment slack
  static_assert(kRing >= kPiece, "a warp's last piece reuses its ring");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct WarpMeta {
  int f_valid, l_valid, l_start;   // l_start: the last piece holds its run's block 0
  int fb, fg, lb, lg;              // runs of the two pieces
};

struct DecKv4Shared {
  uint64_t full[16][4];
  uint64_t ready[16];              // a warp's first piece is there for the warp before it
  WarpMeta meta[16];
  int4 scan[16];
  longlong2 reach[16];             // where the shares of the warps before and behind begin and end
  int part_cta0[2], part_n[2];     // parts of this CTA (see below): their run's first CTA and part count (0: none)
  int last[2];
  int abort;
};
static_assert(sizeof(DecKv4Shared) <= 2048, "shared control block");

struct DecKv4Params {
  const __nv_bfloat16* q;
  const uint8_t* kv_cache;
  const int* block_table;
  const int* seq_lens;
  __nv_bfloat16* o;
  float* lse;
  float* ws_o;                     // [2 kMaxCtas][group][D]
  float* ws_ml;                    // [2 kMaxCtas][group][2]
  unsigned long long* arrive;      // [kMaxCtas]
  int num_seqs, Hq, Hkv, group, max_blocks, num_blocks;
  unsigned int epoch;
  int early_plan;                  // plan before waiting for the preceding kernel
  float scale_log2;
  unsigned int* status;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ int kv4_seq_len(const DecKv4Params& p, int b) {
  const int L = p.seq_lens[b];
  return L < 0 ? 0 : min(L, p.max_blocks * kBS);
}

// Work in cost units: every run (sequence, KV head) is run_cost units followed
// by one per block, runs in order of (sequence, head).  cost[e] and runs[e]
// are the units and the runs before entry e, an entry being `per` sequences;
// blocks[e] the blocks of a head of sequence e (per == 1).
struct Plan {
  const int* cost;
  const int* runs;
  const int* blocks;
  int entries, per, total, total_blocks, total_runs, run_cost;
  int team;                        // warps that share a run (0: equal shares of all)
  __device__ __forceinline__ int seq_blocks(const DecKv4Params& p, int b) const {
    return per == 1 ? blocks[b] : (kv4_seq_len(p, b) + kBS - 1) / kBS;
  }
};

struct RunPos {
  int b, g, blk, nblk;
  int cost;                        // cost position where the run starts
};

// The run of cost unit x < total and the first block at or after it; returns
// the blocks before that one.  (One thread.)
__device__ __forceinline__ int locate(const DecKv4Params& p, const Plan& plan, int x, RunPos& at) {
  int e = 0;                                     // last entry that starts at or before x
  for (int step = 1 << (31 - __clz(plan.entries)); step > 0; step >>= 1)
    if (e + step < plan.entries && plan.cost[e + step] <= x) e += step;
  int start = plan.cost[e], runs = plan.runs[e];
  at.b = e * plan.per;
  at.nblk = plan.seq_blocks(p, at.b);
  for (int i = 1; i < plan.per; ++i) {           // several sequences to the entry: pass those before x
    const int c = at.nblk > 0 ? (at.nblk + plan.run_cost) * p.Hkv : 0;
    if (start + c > x) break;
    start += c;
    if (c > 0) runs += p.Hkv;
    at.nblk = plan.seq_blocks(p, ++at.b);
  }
  const int cost = at.nblk + plan.run_cost;
  at.g = (x - start) / cost;
  at.cost = start + at.g * cost;
  at.blk = max(0, x - at.cost - plan.run_cost);
  return at.cost - (runs + at.g) * plan.run_cost + at.blk;
}

// Run r < the number of runs, from its first block.
__device__ __forceinline__ void locate_run(const DecKv4Params& p, const Plan& plan, int r, RunPos& at) {
  int e = 0;                                     // last entry whose runs start at or before r
  for (int step = 1 << (31 - __clz(plan.entries)); step > 0; step >>= 1)
    if (e + step < plan.entries && plan.runs[e + step] <= r) e += step;
  int start = plan.runs[e];
  at.b = e * plan.per;
  at.nblk = plan.seq_blocks(p, at.b);
  for (int i = 1; i < plan.per; ++i) {
    const int c = at.nblk > 0 ? p.Hkv : 0;
    if (start + c > r) break;
    start += c;
    at.nblk = plan.seq_blocks(p, ++at.b);
  }
  at.g = r - start;
  at.blk = 0;
}

// Walk over the runs of a warp's share.
struct Walk {
  RunPos at;
  int left;                        // blocks of the share not yet passed
  __device__ __forceinline__ int count() const { return min(left, at.nblk - at.blk); }
  __device__ __forceinline__ void next_run(const DecKv4Params& p, const Plan& plan, int passed) {
    left -= passed;
    at.blk = 0;
    at.cost += at.nblk + plan.run_cost;
    if (++at.g == p.Hkv) {
      at.g = 0;
      do {
        ++at.b;
        at.nblk = (left > 0 && at.b < p.num_seqs) ? plan.seq_blocks(p, at.b) : 1;
      } while (left > 0 && at.nblk == 0);
    }
  }
  __device__ __forceinline__ void skip(const DecKv4Params& p, const Plan& plan, int k) {
    while (k > 0 && left > 0) {
      const int c = count();
      if (k < c) {
        at.blk += k;
        left -= k;
        k = 0;
      } else {
        next_run(p, plan, c);
        k -= c;
      }
    }
  }
};

// Arrivals at a run that is split over CTAs.  The counter holds a call's tag
// (never 0) in its high half and the arrivals in its low half.  Whatever it
// held, every CTA that has a part first sees to it that it carries this
// call's tag (only the first one there changes it), and adds its arrival much
// later; the last one leaves it at zero.  So the arrival itself is one add:
// with the tag settled on arrival, by compare and swap, the CTAs of a long run,
// which finish together, held each other up for 6 us.
__device__ __forceinline__ void ready_counter(unsigned long long* slot, unsigned int epoch) {
  unsigned long long cur = *reinterpret_cast<volatile unsigned long long*>(slot);
  while ((cur >> 32) != epoch) {                 // each failed swap is another CTA's success
    const unsigned long long prev = atomicCAS(slot, cur, static_cast<unsigned long long>(epoch) << 32);
    if (prev == cur) break;
    cur = prev;
  }
}
__device__ __forceinline__ bool count_ready(unsigned long long* slot, int nparts) {
  // Release and acquire: with a CTA barrier before and behind, the CTA's
  // stores are visible to whoever counts later, and its loads see theirs.
  unsigned long long before;
  asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(before) : "l"(slot), "l"(1ull) : "memory");
  const bool last = static_cast<int>(before & 0xffffffffu) + 1 >= nparts;
  if (last) atomicExch(slot, 0ull);
  return last;
}

// Loads of pieces, from shared memory or from what other CTAs have written
// (never through L1).
__device__ __forceinline__ float2 ld_shared_or_l2(const float2* p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_or_l2(const float4* p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Bounded wait of a whole warp; the loop that polls is kept out of line, so
// that the usual case costs one test and one vote.
__device__ __noinline__ bool wait_warp_slow(uint32_t bar, uint32_t parity, const WaitCtl w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return wait_warp_slow(bar, parity, w);
}

// fp16 operand registers of two of a word's four pairs: nibbles (0, 4) and
// (1, 5) of x, or (2, 6) and (3, 7) of x >> 8, as code 2^-24 and code 2^-20.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) { return x & 0x000f000fu; }
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) { return x & 0x00f000f0u; }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float word_scale(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float word_min(uint32_t w) { return __uint_as_float(w << 16); }

// (stab + log2(l)) ln 2, the whole part of the logarithm added to the
// stabiliser first (exactly): an LSE near 0 keeps its bits.
__device__ __forceinline__ float lse_of(float stab, float l) {
  const uint32_t bits = __float_as_uint(l);
  // (Infinities and NaN stay what they are.)
  const float part = bits >= 0x7f800000u ? l : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
  return ((stab + static_cast<float>(static_cast<int>(bits >> 23) - 127)) + __log2f(part)) * kLn2;
}

// N words from shared memory at address + OFFSET.
template <int N, int OFFSET>
__device__ __forceinline__ void load_words(uint32_t address, uint32_t (&r)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(address), "n"(OFFSET));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(r[0]), "=r"(r[1]) : "r"(address), "n"(OFFSET));
  else
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(r[0]) : "r"(address), "n"(OFFSET));
}

// Where a lane's data lies in every record, as shared addresses for a record
// at `ring`.
template <int D, int G>
struct LaneData {
  uint32_t k, par, par_min, v0, v1;
  int slot;
  // MMA row 2c + i (i < 2) and 8 + 2c + (i - 2) hold slot 4c + (i ^ (c & 1)):
  // a lane's four V slots are neighbours, and the exchange of pairs in odd
  // quads spreads its V loads over all banks.  So row r is `slot` and row
  // r + 8 is slot + 2.
  __device__ __forceinline__ LaneData(uint32_t ring, int lane) {
    using Rec = Kv4Layout<D, G>;
    const int r = lane >> 2, c = lane & 3;
    slot = 4 * (r >> 1) + ((r & 1) ^ ((r >> 1) & 1));
    k = ring + slot * Rec::kRow + c * (D / 8);
    par = ring + slot * Rec::kParRow;
    par_min = par + (c % (D / G)) * 4;
    v0 = ring + (4 * c + (c & 1)) * Rec::kRow + r * (D / 16);
    v1 = ring + (4 * c + 1 - (c & 1)) * Rec::kRow + r * (D / 16);
  }
};

// Queries of one (sequence, KV head) as B operands, and what undoes their
// scaling.
template <int D, int G, int NT>
struct QueryFrag {
  uint32_t b[NT][D / 16][2];       // second register: elements 8 up, divided by 16 (codes_hi)
  uint32_t sums[NT][2];            // sum(q_g) 2^-24 of group lane % 4 in three bf16 parts
  float back[NT][2];               // score factor of heads 2 (lane % 4), + 1
};

// The query rows as they are: element pairs 16 s + 2 c and 16 s + 8 + 2 c of
// head lane / 4 of a tile (c = lane % 4).
template <int D, int NT>
struct QueryRaw {
  uint32_t w[NT][D / 16][2];
  __device__ __forceinline__ void load(const DecKv4Params& p, int b, int g, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = nt * 8 + (lane >> 2);
      const bool live = head < p.group;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(g) * p.group + (live ? head : 0)) * D) + (lane & 3);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        w[nt][s][0] = live ? src[8 * s] : 0u;
        w[nt][s][1] = live ? src[8 * s + 4] : 0u;
      }
    }
  }
};

template <int D, int G, int NT>
__device__ __forceinline__ void make_queries(const DecKv4Params& p, const QueryRaw<D, NT>& all, int lane,
                                             QueryFrag<D, G, NT>& f) {
  constexpr int kGroups = D / G;
  const int c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t (&raw)[D / 16][2] = all.w[nt];
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
    // (Never 0, which the -inf of slots without a token would make NaN.)
    const float back = fmaxf(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * 0x1p24f, 0x1p-126f);
    f.back[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
    f.back[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
    float sum[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) sum[i] = 0.f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      f.b[nt][s][0] = pack_f16x2(word_min(raw[s][0]) * up, word_scale(raw[s][0]) * up);
      f.b[nt][s][1] = pack_f16x2(word_min(raw[s][1]) * up * 0.0625f, word_scale(raw[s][1]) * up * 0.0625f);
      // The sums are those of the rounded operands, so that the two terms of
      // a score belong to the same q.
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f.b[nt][s][0]));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f.b[nt][s][1]));
      sum[16 * s / G] += (x.x + x.y) + 16.f * (y.x + y.y);
    }
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
      if (c == i) mine = sum[i] * 0x1p-24f;
    }
    const float hi = __bfloat162float(__float2bfloat16_rn(mine));
    const float mid = __bfloat162float(__float2bfloat16_rn(mine - hi));
    f.sums[nt][0] = pack_bf16x2(hi, mid);
    f.sums[nt][1] = pack_bf16x2(mine - hi - mid, 0.f);
  }
}

// Running state of one run: O^T tiles, the min terms, stabilisers and sums,
// all in units of 2^stab per head.
template <int D, int G, int NT>
struct RunState {
  float o[NT][D / 16][4];          // rows r and r + 8 (the latter times 16), heads 2c, 2c + 1; times 2^-24 and room
  float mins[NT][D / G][2];        // sum of p min over this lane's tokens
  float stab[NT][2], l[NT][2];
  float limit[NT][2];              // raw score from which the stabiliser has to move
  // The power of two of a group of V by which its scales are multiplied for the
  // products p scale: it keeps the largest scale met so far under kFull.
  float room[D / G];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / G; ++i) mins[nt][i][0] = mins[nt][i][1] = 0.f;
      // (A block without tokens may come first: its weights are then
      // ex2(-inf + 1e30) = 0.)
      stab[nt][0] = stab[nt][1] = -1e30f;
      limit[nt][0] = limit[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < D / G; ++g) room[g] = 0x1p126f;
  }

  // Moves the stabilisers for raw scores up to s, and the groups' room for these
  // V parameter words; rare, and the same for the whole warp.
  template <int N>
  __device__ __forceinline__ void move(const float (&s)[NT][2], const float (&back)[NT][2],
                                       const uint32_t (&words)[N][2][D / G]) {
    float less[D / G];                             // what becomes of the products so far
#pragma unroll
    for (int g = 0; g < D / G; ++g) {
      uint32_t big = 0;
#pragma unroll
      for (int n = 0; n < N; ++n) big = max(big, max(words[n][0][g], words[n][1][g]));
      // Scales of exponent field E are below 2^(E - 126), 2^(151 - E) brings them
      // under a quarter of kFull, so that somewhat larger ones to come move nothing
      // (at most 2^126: scales under 2^-102 lose bits; one that is no number takes
      // its group to the end of the range, and spoils it anyway).
      const int E = static_cast<int>(__reduce_max_sync(0xffffffffu, big) >> 23);
      const int had = __float_as_int(room[g]), has = min(had, (278 - min(max(E, 25), 254)) << 23);
      room[g] = __int_as_float(has);
      less[g] = __int_as_float(max(has - had + (127 << 23), 0));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = s[nt][h] * back[nt][h];
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o_));
        const float top = stab[nt][h] - kLow;    // the running maximum
        // (To a multiple of 2^-10, so that adding whole numbers to a stabiliser,
        // here and for the LSE, rounds nothing.)
        const float to = __fsub_rn(__fadd_rn(mx > top + kTau ? mx : top, kGrid), kGrid) + kLow;
        f[h] = to == stab[nt][h] ? 1.f : ex2(stab[nt][h] - to);
        stab[nt][h] = to;
        limit[nt][h] = (to - kLow + kTau) / back[nt][h];
        l[nt][h] *= f[h];
#pragma unroll
        for (int g = 0; g < D / G; ++g) mins[nt][g][h] *= f[h];
      }
#pragma unroll
      for (int g = 0; g < D / G; ++g) {
        const float f0 = f[0] * less[g], f1 = f[1] * less[g];
#pragma unroll
        for (int i = g * (G / 16); i < (g + 1) * (G / 16); ++i) {
          o[nt][i][0] *= f0;
          o[nt][i][1] *= f1;
          o[nt][i][2] *= f0;
          o[nt][i][3] *= f1;
        }
      }
    }
  }

  // Sums over the token rows of the warp, and O in units of V.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) {
          l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], o_);
#pragma unroll
          for (int i = 0; i < D / G; ++i) mins[nt][i][h] += __shfl_xor_sync(0xffffffffu, mins[nt][i][h], o_);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // 2^24 / room, and a sixteenth of it.
        const float u = __int_as_float((278 << 23) - __float_as_int(room[16 * i / G])), u8 = u * 0x1p-4f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[nt][i][h] = fmaf(o[nt][i][h], u, mins[nt][16 * i / G][h]);
          o[nt][i][2 + h] = fmaf(o[nt][i][2 + h], u8, mins[nt][16 * i / G][h]);
        }
      }
    }
  }
};

// Two blocks of one run: 16 slots each, of which the first valid[i] (16 or
// more: all) hold tokens; their records rec[i] bytes into the ring.  Two at a
// time, because one block is a chain of dependent steps and a scheduler has
// only three warps to fill its gaps with.
template <int D, int G, int NT>
__device__ __forceinline__ void take_blocks(const LaneData<D, G>& at, const uint32_t (&rec)[2], const int (&valid)[2],
                                            const QueryFrag<D, G, NT>& q, RunState<D, G, NT>& st) {
  using Rec = Kv4Layout<D, G>;
  constexpr int kGroups = D / G, kKW = D / 32, kVW = D / 64;

  // --- S^T: rows = slots, columns = heads
  float s[2][NT][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    // The min terms: lane c of a quad brings group c (the others of its group
    // count meet zero operands).
    uint32_t lo[1], lo8[1];
    load_words<1, Rec::kOffParK>(at.par_min + rec[n], lo);
    load_words<1, Rec::kOffParK + 2 * Rec::kParRow>(at.par_min + rec[n], lo8);
    lo[0] = __byte_perm(lo[0], 0, 0x1010);
    lo8[0] = __byte_perm(lo8[0], 0, 0x1010);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mma_16816_bf16_first(s[n][nt], lo[0], lo8[0], lo[0], lo8[0], q.sums[nt][0], q.sums[nt][1]);
  }
  {
    uint32_t ka[2][kKW], kb[2][kKW], kpa[2][kGroups], kpb[2][kGroups];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      load_words<kKW, 0>(at.k + rec[n], ka[n]);
      load_words<kKW, 2 * Rec::kRow>(at.k + rec[n], kb[n]);
      load_words<kGroups, Rec::kOffParK>(at.par + rec[n], kpa[n]);
      load_words<kGroups, Rec::kOffParK + 2 * Rec::kParRow>(at.par + rec[n], kpb[n]);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float acc[2][NT][4];
#pragma unroll
      for (int ws = 0; ws < G / 32; ++ws) {
        const int w = g * (G / 32) + ws;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t xa = ka[n][w], xb = kb[n][w], ya = xa >> 8, yb = xb >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (ws == 0)
              mma_16816_f16_first(acc[n][nt], codes_lo(xa), codes_lo(xb), codes_hi(xa), codes_hi(xb), q.b[nt][2 * w][0],
                                  q.b[nt][2 * w][1]);
            else
              mma_16816_f16(acc[n][nt], codes_lo(xa), codes_lo(xb), codes_hi(xa), codes_hi(xb), q.b[nt][2 * w][0],
                            q.b[nt][2 * w][1]);
            mma_16816_f16(acc[n][nt], codes_lo(ya), codes_lo(yb), codes_hi(ya), codes_hi(yb), q.b[nt][2 * w + 1][0],
                          q.b[nt][2 * w + 1][1]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float sa = word_scale(kpa[n][g]), sb = word_scale(kpb[n][g]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f2_unpack(f2_fma(f2_pack(sa, sa), f2_pack(acc[n][nt][0], acc[n][nt][1]), f2_pack(s[n][nt][0], s[n][nt][1])),
                    s[n][nt][0], s[n][nt][1]);
          f2_unpack(f2_fma(f2_pack(sb, sb), f2_pack(acc[n][nt][2], acc[n][nt][3]), f2_pack(s[n][nt][2], s[n][nt][3])),
                    s[n][nt][2], s[n][nt][3]);
        }
      }
    }
  }

  uint32_t vp[2][2][kGroups];                    // of slots `slot` and slot + 2
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    load_words<kGroups, Rec::kOffParV>(at.par + rec[n], vp[n][0]);
    load_words<kGroups, Rec::kOffParV + 2 * Rec::kParRow>(at.par + rec[n], vp[n][1]);
  }
  uint32_t vw[2][4][kVW];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    load_words<kVW, Rec::kOffV>(at.v0 + rec[n], vw[n][0]);
    load_words<kVW, Rec::kOffV>(at.v1 + rec[n], vw[n][1]);
    load_words<kVW, Rec::kOffV + 2 * Rec::kRow>(at.v0 + rec[n], vw[n][2]);
    load_words<kVW, Rec::kOffV + 2 * Rec::kRow>(at.v1 + rec[n], vw[n][3]);
  }
  if (min(valid[0], valid[1]) < kBS) {
    // Slots past the end may hold anything: no score, no parameters.
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const bool dead = at.slot >= valid[n], dead8 = at.slot + 2 >= valid[n];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (dead) s[n][nt][0] = s[n][nt][1] = -INFINITY;
        if (dead8) s[n][nt][2] = s[n][nt][3] = -INFINITY;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (dead) vp[n][0][g] = 0;
        if (dead8) vp[n][1][g] = 0;
      }
    }
  }

  // Whether a scale times its group's room reaches kFull, in the bits of floats
  // (exponents add up).
  uint32_t big = 0;
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
    big = __viaddmax_u32(max(max(vp[0][0][g], vp[0][1][g]), max(vp[1][0][g], vp[1][1][g])), __float_as_uint(st.room[g]), big);
  bool move = big >= (__float_as_uint(kFull) + (127u << 23));
  float top[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[nt][h] = fmaxf(fmaxf(s[0][nt][h], s[0][nt][2 + h]), fmaxf(s[1][nt][h], s[1][nt][2 + h]));
      move |= top[nt][h] > st.limit[nt][h];
    }
  if (__any_sync(0xffffffffu, move)) st.move(top, q.back, vp);

  // --- weights and O^T: rows = elements of V, columns = heads
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint32_t pw[NT][kGroups][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint64_t back = f2_pack(q.back[nt][0], q.back[nt][1]), stab = f2_pack(-st.stab[nt][0], -st.stab[nt][1]);
      float p0, p1, p2, p3;
      f2_unpack(f2_fma(f2_pack(s[n][nt][0], s[n][nt][1]), back, stab), p0, p1);
      f2_unpack(f2_fma(f2_pack(s[n][nt][2], s[n][nt][3]), back, stab), p2, p3);
      const uint64_t pa = f2_pack(ex2(p0), ex2(p1)), pb = f2_pack(ex2(p2), ex2(p3));
      f2_unpack(f2_add(f2_pack(st.l[nt][0], st.l[nt][1]), f2_add(pa, pb)), st.l[nt][0], st.l[nt][1]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float sa = word_scale(vp[n][0][g]) * st.room[g], sb = word_scale(vp[n][1][g]) * st.room[g];
        const float ma = word_min(vp[n][0][g]), mb = word_min(vp[n][1][g]);
        f2_unpack(f2_fma(pa, f2_pack(ma, ma), f2_fma(pb, f2_pack(mb, mb), f2_pack(st.mins[nt][g][0], st.mins[nt][g][1]))),
                  st.mins[nt][g][0], st.mins[nt][g][1]);
        float w0, w1;
        f2_unpack(f2_mul(pa, f2_pack(sa, sa)), w0, w1);
        pw[nt][g][0] = movmatrix_trans(pack_f16x2(w0, w1));
        f2_unpack(f2_mul(pb, f2_pack(sb, sb)), w0, w1);
        pw[nt][g][1] = movmatrix_trans(pack_f16x2(w0, w1));
      }
    }
#pragma unroll
    for (int w = 0; w < kVW; ++w) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t sel = hf ? 0x7632u : 0x5410u;
        const uint32_t x = __byte_perm(vw[n][0][w], vw[n][1][w], sel), y = __byte_perm(vw[n][2][w], vw[n][3][w], sel);
        const uint32_t x8 = x >> 8, y8 = y >> 8;
        const int i = 4 * w + 2 * hf;            // tiles i and i + 1 of 16 elements
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816_f16(st.o[nt][i], codes_lo(x), codes_hi(x), codes_lo(y), codes_hi(y), pw[nt][16 * i / G][0],
                        pw[nt][16 * i / G][1]);
          mma_16816_f16(st.o[nt][i + 1], codes_lo(x8), codes_hi(x8), codes_lo(y8), codes_hi(y8),
                        pw[nt][16 * (i + 1) / G][0], pw[nt][16 * (i + 1) / G][1]);
        }
      }
    }
  }
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(DecKv4Cfg<D, G, NT>::kThreads, 1)
    attn_decode_kv4_kernel(const __grid_constant__ DecKv4Params p) {
  using Cfg = DecKv4Cfg<D, G, NT>;
  using Rec = Kv4Layout<D, G>;
  constexpr int kWarps = Cfg::kWarps, kThreads = Cfg::kThreads, kStages = Cfg::kStages, kRows = Cfg::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  DecKv4Shared* sh = reinterpret_cast<DecKv4Shared*>(smem + Cfg::kOffShared);
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
  static_assert(kStages <= 4, "");
  if (lane < kStages) mbar_init(smem_addr(&sh->full[warp][lane]), 1);
  if (lane == kStages) mbar_init(smem_addr(&sh->ready[warp]), 1);
  fence_mbar_init();
  if (tid == 0) {
    // What the plan and the first loads will read, into L2 while the work
    // before this kernel drains (hints only: nothing is read here).
    auto prefetch_share = [&](const void* base, size_t bytes) {
      const uintptr_t lo = (reinterpret_cast<uintptr_t>(base) + 15) & ~static_cast<uintptr_t>(15);
      const uintptr_t hi = (reinterpret_cast<uintptr_t>(base) + bytes) & ~static_cast<uintptr_t>(15);
      if (hi <= lo) return;
      const size_t share = ((hi - lo) / gridDim.x + 16) & ~static_cast<size_t>(15);
      const uintptr_t at = lo + share * blockIdx.x;
      // (At most 1 MB of each: with few CTAs a share may be far more than L2 is for.)
      if (at < hi)
        bulk_prefetch_l2(reinterpret_cast<const void*>(at),
                         static_cast<uint32_t>(min(min(share, static_cast<size_t>(hi - at)), size_t(1) << 20)));
    };
    prefetch_share(p.seq_lens, static_cast<size_t>(p.num_seqs) * 4);
    // (A wide table is mostly padding.)
    const size_t table = static_cast<size_t>(p.num_seqs) * p.max_blocks * 4;
    if (table <= (size_t(1) << 20)) prefetch_share(p.block_table, table);
    prefetch_share(p.q, static_cast<size_t>(p.num_seqs) * p.Hq * D * 2);
  }
  // With the early plan, seq_lens and the block table are read before the
  // preceding kernel has finished; the queries, the cache and everything that
  // is written come after the wait further down.
  if (!p.early_plan) pdl_wait_primary();

  // ------------------------------------------------------------------ plan
  Plan plan;
  plan.cost = cost;
  plan.runs = runs;
  plan.blocks = seq_blocks;
  plan.per = (p.num_seqs + kPlan - 1) / kPlan;
  plan.entries = (p.num_seqs + plan.per - 1) / plan.per;
  const int shares = static_cast<int>(gridDim.x) * kWarps;
  {
    // Thread t sums entries [t E, (t + 1) E); warp scan, then the warps' sums.
    constexpr int E = (kPlan + kThreads - 1) / kThreads;
    const int each = (plan.entries + kThreads - 1) / kThreads;          // <= E
    int ec[E], er[E], c = 0, r = 0, longest = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      ec[i] = c;
      er[i] = r;
      const int e = tid * each + i;
      if (i >= each || e >= plan.entries) continue;
      for (int b = e * plan.per; b < min(p.num_seqs, (e + 1) * plan.per); ++b) {
        const int L = p.seq_lens[b];
        bad |= L < 0 || L > p.max_blocks * kBS;
        const int blocks = ((L < 0 ? 0 : min(L, p.max_blocks * kBS)) + kBS - 1) / kBS;
        if (plan.per == 1) seq_blocks[b] = blocks;
        longest = max(longest, blocks);
        if (blocks > 0) {
          c += blocks * p.Hkv;
          r += p.Hkv;
        }
      }
    }
    if (bad && blockIdx.x == 0) atomicOr(p.status, kDevBadSeqLen);
    int cs = c, rs = r;
    longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int cy = __shfl_up_sync(0xffffffffu, cs, o), ry = __shfl_up_sync(0xffffffffu, rs, o);
      if (lane >= o) {
        cs += cy;
        rs += ry;
      }
    }
    if (lane == 31) sh->scan[warp] = make_int4(cs, rs, longest, 0);
    __syncthreads();
    int c0 = cs - c, r0 = rs - r, total = 0, total_runs = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int4 v = sh->scan[w];
      if (w < warp) {
        c0 += v.x;
        r0 += v.y;
      }
      total += v.x;
      total_runs += v.y;
      longest = max(longest, v.z);
    }
    plan.total_runs = total_runs;
    // Or a team of warps to each run: as many as there are for it, a CTA's
    // warps or a half, a third .. of them.  Then nothing has to be merged across
    // CTAs, which costs about as much as 3.5 blocks (6 with two column tiles,
    // whose merges cost more, or d = 64, whose blocks cost less): it is taken
    // where the longest run brings its team no more than that beyond an equal
    // share of all blocks.  Measured against equal shares (us; sequences x tokens,
    // KV heads): 4 x 100 .. 300, 2, 7.0 and 9.9; 32 x 400 .. 600, 2, 9.4 and 11.7;
    // 64 x 1500, 2, 13.7 and 16.1; 256 x 20 .. 90, 2, 9.1 and 12.0; 30 x 900 ..
    // 1000, 4 of 16 heads, 10.1 and 13.9; 256 x 1 .. 100, the same, 9.8 and 13.7;
    // and where the rule says no, 4 x 900, 2, 10.5 and 9.6.
    int team = 0;
#pragma unroll
    for (int k = kWarps; k >= 1; --k)
      if (kWarps % k == 0 && total_runs <= k * static_cast<int>(gridDim.x)) team = kWarps / k;
    constexpr int kSpare2 = NT == 1 && D == 128 ? 7 : 12;        // in half blocks
    if (static_cast<long long>(2 * longest - kSpare2 * team) * shares > 2LL * team * total) team = 0;
    plan.team = team;
    // What a run costs beyond its blocks.  A long share spends about 4 blocks'
    // time on a run (its queries, its end).  A share is at least run_cost + 1
    // blocks, though, a pass of two blocks takes a warp 0.9 us when it is alone,
    // and with few blocks most warps have none: then shares of one pass, and
    // between of two.  Measured with 1, 3 and 4 (us): one sequence of 100 tokens,
    // 2 KV heads, 6.8 6.9 7.7; 16 of 500, 9.9 12.7 12.8; 32 of 1000, 12.4 11.9
    // 13.0; 16 of up to 2000, 4 KV heads, 13.4 12.2 12.8; 256 of up to 2048, 45.6
    // 41.9 40.5.
    plan.run_cost = total <= shares ? 1 : total <= 8 * shares ? 3 : 4;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = tid * each + i;
      if (i >= each || e >= plan.entries) continue;
      cost[e] = c0 + ec[i] + (r0 + er[i]) * plan.run_cost;
      runs[e] = r0 + er[i];
    }
    plan.total = total + total_runs * plan.run_cost;
    plan.total_blocks = total;
  }
  __syncthreads();
  // Every share but the last of all holds at least one block (a share longer
  // than a run's start cost cannot lie inside it).
  int chunk = max(plan.run_cost + 1, (plan.total - 1) / shares + 1);
  Walk w;
  int place = static_cast<int>(blockIdx.x) * kWarps + warp;
  if (plan.team != 0) {
    place = warp % plan.team;
    const int run = static_cast<int>(blockIdx.x) + warp / plan.team * static_cast<int>(gridDim.x);
    w.at.nblk = 0;
    if (run < plan.total_runs) locate_run(p, plan, run, w.at);
    chunk = ((w.at.nblk + plan.team - 1) / plan.team + 1) & ~1;  // whole passes
  }
  const long long mine = static_cast<long long>(place) * chunk;
  // (Read back at a run's end: kept in registers, they cost the loop over the
  // blocks 1 to 2%.)
  if (lane == 0) sh->reach[warp] = make_longlong2(mine - chunk, mine + 2LL * chunk);

  const WaitCtl wc{&sh->abort, p.status, p.timeout_ns};
  WarpMeta meta = {};
  int blocks = 0;
  RunPos end;
  if (plan.team != 0) {
    end.blk = 0;
    w.at.cost = -plan.run_cost;                  // positions are those within the run
    w.at.blk = place * chunk;
    blocks = max(0, min(chunk, w.at.nblk - w.at.blk));
  } else {
    // Lane 0 finds where this warp's share begins, the other lanes where it
    // ends.
    RunPos at;
    at.b = at.g = at.blk = at.nblk = at.cost = 0;
    const long long x = mine + (lane > 0 ? chunk : 0);
    const int flat = x < plan.total ? locate(p, plan, static_cast<int>(x), at)
                                    : plan.total_blocks;
    const int from = __shfl_sync(0xffffffffu, flat, 0);
    blocks = __shfl_sync(0xffffffffu, flat, 1) - from;
    auto give = [&](int v, int& begin, int& finish) {
      begin = __shfl_sync(0xffffffffu, v, 0);
      finish = __shfl_sync(0xffffffffu, v, 1);
    };
    give(at.b, w.at.b, end.b);
    give(at.g, w.at.g, end.g);
    give(at.blk, w.at.blk, end.blk);
    give(at.nblk, w.at.nblk, end.nblk);
    give(at.cost, w.at.cost, end.cost);
  }

  if (blocks > 0) {
    uint8_t* ring = smem + warp * Cfg::kRing;
    w.left = blocks;
    // The first run's queries are on their way while the table is read.
    QueryRaw<D, NT> raw;
    if (!p.early_plan) raw.load(p, w.at.b, w.at.g, lane);
    // Lane j looks up block j of every batch of 32, two batches ahead, and
    // leaves its record's address for the issuing lane (0: not in the pool).
    // Returns the batch's mask of blocks that have a record.
    Walk ahead = w;
    ahead.skip(p, plan, lane);
    const uint8_t** src = reinterpret_cast<const uint8_t**>(smem + Cfg::kOffSrc) + warp * 64;
    auto fetch = [&](int batch) {
      const uint8_t* rec = nullptr;
      if (ahead.left > 0) {
        const int ph = p.block_table[static_cast<size_t>(ahead.at.b) * p.max_blocks + ahead.at.blk];
        if (static_cast<unsigned>(ph) < static_cast<unsigned>(p.num_blocks))
          rec = p.kv_cache + (static_cast<size_t>(ph) * p.Hkv + ahead.at.g) * Rec::kBytes;
        else
          atomicOr(p.status, kDevBadBlock);      // outside the pool: that block is skipped
      }
      ahead.skip(p, plan, 32);
      src[(batch & 1) * 32 + lane] = rec;
      return __ballot_sync(0xffffffffu, rec != nullptr);
    };
    const uint64_t policy = l2_policy_evict_first();
    unsigned present = fetch(0);
    if (p.early_plan) {
      pdl_wait_primary();
      raw.load(p, w.at.b, w.at.g, lane);
    }
    const uint32_t ring_at = smem_addr(ring), bars = smem_addr(&sh->full[warp][0]);
    // Block i of the share goes to stage i % kStages; blocks [0, taken +
    // kStages) are issued.  (One lane.)
    auto issue = [&](int i) {
      const uint8_t* from = src[i & 63];
      const uint32_t bar = bars + (i % kStages) * 8;
      mbar_arrive_expect_tx(bar, from != nullptr ? Rec::kBytes : 0);
      if (from != nullptr) bulk_load_hint(ring_at + (i % kStages) * Rec::kBytes, from, Rec::kBytes, bar, policy);
    };
    if (lane < min(blocks, kStages)) issue(lane);
    unsigned next_present = blocks > 32 ? fetch(1) : 0u;
    __syncwarp();
    const LaneData<D, G> at(ring_at, lane);

    // Runs that this CTA holds a part of: one that began before it and ends in
    // it (kind 0), one that goes on behind it (kind 1).  Their counters are
    // made ready now, long before they are counted on.
    if (lane == 0) {
      const long long cta_chunk = static_cast<long long>(chunk) * kWarps;
      auto take_part = [&](int kind, const RunPos& run) {
        const int first = run.cost + plan.run_cost;   // cost position of its block 0
        const int cta0 = static_cast<int>(first / cta_chunk), cta1 = static_cast<int>((first + run.nblk - 1) / cta_chunk);
        sh->part_cta0[kind] = cta0;
        sh->part_n[kind] = cta1 - cta0 + 1;
        ready_counter(p.arrive + cta0, p.epoch);
      };
      if (warp == 0 && w.at.blk > 0 && w.at.cost + plan.run_cost + w.at.nblk <= mine + cta_chunk) take_part(0, w.at);
      if (warp == kWarps - 1 && end.blk > 0) take_part(1, end);
    }

    QueryFrag<D, G, NT> q;
    RunState<D, G, NT> st;
    int taken = 0;
    bool fail = false;
    while (w.left > 0 && !fail) {
      const int cnt = w.count();
      int valid = kv4_seq_len(p, w.at.b) - w.at.blk * kBS;      // tokens from this block on
      if (taken > 0) raw.load(p, w.at.b, w.at.g, lane);
      make_queries<D, G, NT>(p, raw, lane, q);
      st.reset();
      for (const int end = taken + cnt; taken < end;) {
        const int stage = taken % kStages, stage1 = (taken + 1) % kStages;
        const bool two = taken + 1 < end;
        if (!wait_warp(bars + stage * 8, (taken / kStages) & 1, wc) ||
            (two && !wait_warp(bars + stage1 * 8, ((taken + 1) / kStages) & 1, wc))) {
          fail = true;
          break;
        }
        // Without a second block the first one's record stands in, with no
        // slot of it alive.
        const uint32_t rec0 = static_cast<uint32_t>(stage * Rec::kBytes);
        const uint32_t rec[2] = {rec0, two ? static_cast<uint32_t>(stage1 * Rec::kBytes) : rec0};
        const int alive[2] = {(present >> (taken & 31)) & 1u ? valid : 0,
                              two && ((taken & 31) == 31 ? next_present & 1u : (present >> ((taken + 1) & 31)) & 1u)
                                  ? valid - kBS : 0};
        take_blocks<D, G, NT>(at, rec, alive, q, st);
        __syncwarp();                            // every lane has read the stages
        const int n = two ? 2 : 1;
        if (lane < n && taken + lane + kStages < blocks) issue(taken + lane + kStages);
        valid -= n * kBS;
        if (((taken + n) ^ taken) & 32) {        // (the issuer is less than a batch ahead)
          present = next_present;
          next_present = ((taken + n) & ~31) + 32 < blocks ? fetch(((taken + n) >> 5) + 1) : 0u;
          __syncwarp();
        }
        taken += n;
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
        const float* src = first_piece(warp + 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 v = ml[(warp + 1) * 2 * kRows + nt * 8 + 2 * c + h];
            const float to = fmaxf(st.stab[nt][h], v.x);
            const float f0 = ex2(st.stab[nt][h] - to), f1 = ex2(v.x - to);
            st.stab[nt][h] = to;
            st.l[nt][h] = st.l[nt][h] * f0 + v.y * f1;
            const float* row = src + (nt * 8 + 2 * c + h) * Cfg::kPitch + r;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              st.o[nt][i][h] = st.o[nt][i][h] * f0 + row[16 * i] * f1;
              st.o[nt][i][2 + h] = st.o[nt][i][2 + h] * f0 + row[16 * i + 8] * f1;
            }
          }
        }
        whole = true;
      }
      if (whole) {
        const size_t h0 = static_cast<size_t>(w.at.b) * p.Hq + static_cast<size_t>(w.at.g) * p.group;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float i0 = st.l[nt][0] > 0.f ? 1.f / st.l[nt][0] : (st.l[nt][0] == 0.f ? 0.f : st.l[nt][0]);
          const float i1 = st.l[nt][1] > 0.f ? 1.f / st.l[nt][1] : (st.l[nt][1] == 0.f ? 0.f : st.l[nt][1]);
          const int head = nt * 8 + r;
          __nv_bfloat16* dst = p.o + (h0 + head) * D + 2 * c;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t t = movmatrix_trans(pack_bf16x2(st.o[nt][i][2 * k] * i0, st.o[nt][i][2 * k + 1] * i1));
              if (head < p.group) *reinterpret_cast<uint32_t*>(dst + 16 * i + 8 * k) = t;
            }
          }
          if (p.lse != nullptr && r == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int hd = nt * 8 + 2 * c + h;
              if (hd < p.group)
                p.lse[h0 + hd] = st.l[nt][h] == 0.f ? -INFINITY : lse_of(st.stab[nt][h], st.l[nt][h]);
            }
          }
        }
      } else {
        // A piece: in the first-piece buffer if the run ends here, else in
        // this warp's ring, which has nothing more to take.
        const bool f = has_end;
        float* dst = f ? first_piece(warp) : last_piece(warp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* row = dst + (nt * 8 + 2 * c + h) * Cfg::kPitch + r;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              row[16 * i] = st.o[nt][i][h];
              row[16 * i + 8] = st.o[nt][i][2 + h];
            }
            if (r == 0)
              ml[(warp * 2 + (f ? 0 : 1)) * kRows + nt * 8 + 2 * c + h] = make_float2(st.stab[nt][h], st.l[nt][h]);
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
  // Sequences without tokens: O = 0, LSE = -inf.
  for (int b = static_cast<int>(blockIdx.x) * kWarps + warp; b < p.num_seqs; b += shares) {
    if (plan.seq_blocks(p, b) != 0) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(b) * p.Hq * D);
    for (int i = lane; i < p.Hq * D / 2; i += 32) dst[i] = 0u;
    if (p.lse != nullptr)
      for (int h = lane; h < p.Hq; h += 32) p.lse[static_cast<size_t>(b) * p.Hq + h] = -INFINITY;
  }
  __syncthreads();
  pdl_launch_dependents();
  const bool parts_here[2] = {sh->part_n[0] > 0, sh->part_n[1] > 0};
  auto arrive = [&]() {                          // warps 0 and 1, one lane: one arrival per part
    if (lane == 0 && warp < 2 && parts_here[warp])
      sh->last[warp] = count_ready(p.arrive + sh->part_cta0[warp], sh->part_n[warp]);
  };
  if (sh->abort) {
    arrive();                                    // so that the counters are left at zero
    return;
  }

  // ------------------------------------------------- pieces of split runs
  // The pieces of a run lie in consecutive warps: last pieces, from the warp
  // that holds its start (or the CTA's first), up to the first piece of the
  // warp where it ends.  They are merged here; of a run that starts before
  // this CTA (kind 0) or goes on behind it (kind 1) that leaves one part,
  // which is published, and the CTA that arrives last at the run merges its
  // parts.  Both merges are the same loop, over jobs: the code is then fetched
  // once (cold, it took longer than its work).
  unsigned ends, starts;
  {
    const bool in = lane < kWarps;
    const WarpMeta& mt = sh->meta[in ? lane : 0];
    ends = __ballot_sync(0xffffffffu, in && mt.f_valid);
    starts = __ballot_sync(0xffffffffu, in && mt.l_valid && mt.l_start);
  }
  constexpr int W = D / 4;                       // lanes of a head's row, four columns each
  const int sub = lane / W, col = (lane % W) * 4;
  constexpr unsigned kGoesOn = 1u << 31;
  const int heads = (p.group + 32 / W - 1) & ~(32 / W - 1);
  unsigned todo = ends | (parts_here[1] ? kGoesOn : 0u);
  for (bool parts = false;; parts = true) {
    // The heads of all jobs in one row, 32 / W of them a step, over the warps.
    // (With the jobs one after another 64 sequences of 128 .. 4096 tokens took
    // 19.4 us instead of 17.5.)
    for (int hb = warp * (32 / W);; hb += kWarps * (32 / W)) {
      for (; todo != 0 && hb >= p.group; todo &= todo - 1) hb -= heads;
      if (todo == 0) break;
      const int bit = __ffs(todo) - 1;
      const int kind = bit == 31 ? 1 : 0;
      const int wi = kind ? kWarps - 1 : bit;
      const WarpMeta& mt = sh->meta[wi];
      const size_t h0 = static_cast<size_t>(kind ? mt.lb : mt.fb) * p.Hq + static_cast<size_t>(kind ? mt.lg : mt.fg) * p.group;
      // Piece x < n - 1 lies x steps from the first, piece n - 1 by itself.
      const float *o0, *o1;
      const float2 *m0, *m1;
      int n, o_step, m_step, pitch;
      bool whole = true;
      if (!parts) {
        const unsigned before = starts & (kind ? (2u << wi) - 1 : (1u << wi) - 1);
        const int lo = before ? 31 - __clz(before) : 0;
        whole = kind == 0 && before != 0;
        n = wi - lo + 1;
        o0 = last_piece(lo);
        o_step = Cfg::kRing / 4;
        o1 = kind ? last_piece(wi) : first_piece(wi);
        m0 = ml + (lo * 2 + 1) * kRows;
        m_step = 2 * kRows;
        m1 = ml + (wi * 2 + kind) * kRows;
        pitch = Cfg::kPitch;
      } else {
        // Part x is in CTA cta0 + x's slot 1, the run's end in slot 0.
        const int cta0 = sh->part_cta0[kind];
        n = sh->part_n[kind];
        const size_t s0 = (2 * static_cast<size_t>(cta0) + 1) * p.group, s1 = 2 * static_cast<size_t>(cta0 + n - 1) * p.group;
        o0 = p.ws_o + s0 * D;
        o1 = p.ws_o + s1 * D;
        o_step = 2 * p.group * D;
        m0 = reinterpret_cast<const float2*>(p.ws_ml) + s0;
        m1 = reinterpret_cast<const float2*>(p.ws_ml) + s1;
        m_step = 2 * p.group;
        pitch = D;
      }
      {
        const bool live = hb + sub < p.group;
        const int h = live ? hb + sub : hb;
        float M = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // 16 pieces at a time: their rows and their (stabiliser, sum) pairs are
        // all asked for before any is used (a part published by another CTA
        // takes over a microsecond to come), lane x of a row weighs piece x.
        for (int x0 = 0; x0 < n; x0 += 16) {
          const int m = min(16, n - x0);         // the same for all lanes
          float4 y[16];
#pragma unroll
          for (int q4 = 0; q4 < 16; q4 += 4) {
            if (q4 >= m) break;
#pragma unroll
            for (int i = q4; i < q4 + 4; ++i) {
              y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (i < m)
                y[i] = ld_shared_or_l2(reinterpret_cast<const float4*>(
                    (x0 + i == n - 1 ? o1 : o0 + static_cast<size_t>(x0 + i) * o_step) + h * pitch + col));
            }
          }
          const int x = x0 + lane % 16;
          float2 v = make_float2(-INFINITY, 0.f);
          if (x < n) v = ld_shared_or_l2(x == n - 1 ? m1 + h : m0 + x * m_step + h);
          float mx = v.x;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(M, mx);
          const float turn = ex2(M - mx);
          const float wt = x < n ? ex2(v.x - mx) : 0.f;
          float sum = wt * v.y;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          l = l * turn + sum;
          M = mx;
          acc.x *= turn;
          acc.y *= turn;
          acc.z *= turn;
          acc.w *= turn;
#pragma unroll
          for (int q4 = 0; q4 < 16; q4 += 4) {
            if (q4 >= m) break;
#pragma unroll
            for (int i = q4; i < q4 + 4; ++i) {
              const float w_i = __shfl_sync(0xffffffffu, wt, sub * W + i);
              acc.x += w_i * y[i].x;
              acc.y += w_i * y[i].y;
              acc.z += w_i * y[i].z;
              acc.w += w_i * y[i].w;
            }
          }
        }
        if (!live) continue;
        if (whole) {
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(p.o + (h0 + h) * D + col) = pk;
          if (col == 0 && p.lse != nullptr) p.lse[h0 + h] = l == 0.f ? -INFINITY : lse_of(M, l);
        } else {
          const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + kind) * p.group + h;
          *reinterpret_cast<float4*>(p.ws_o + slot * D + col) = acc;
          if (col == 0) *reinterpret_cast<float2*>(p.ws_ml + slot * 2) = make_float2(M, l);
        }
      }
    }
    if (parts || !(parts_here[0] || parts_here[1])) break;   // the same for the whole CTA
    __syncthreads();
    arrive();
    __syncthreads();
    // The run that ended here and began before this CTA is the first that ended.
    todo = (parts_here[0] && sh->last[0] ? ends & (0u - ends) : 0u) | (parts_here[1] && sh->last[1] ? kGoesOn : 0u);
  }
}

template <int D, int G, int NT>
cudaError_t launch_t(const DecKv4Launch& a) {
  using Cfg = DecKv4Cfg<D, G, NT>;
  auto kern = attn_decode_kv4_kernel<D, G, NT>;
  // The attribute belongs to the device's copy of the kernel: set once for each
  // (the host's time bounds a small decode).
  static std::atomic<unsigned long long> allowed{0};
  const unsigned long long bit = 1ull << a.device;
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  DecKv4Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.num_seqs = a.num_seqs;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.group = a.Hq / a.Hkv;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
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
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(Cfg::kThreads), Cfg::kSmem, a.stream, p);
}

template <int NT>
cudaError_t launch_nt(const DecKv4Launch& a) {
  if (a.d == 128) return a.group == 32 ? launch_t<128, 32, NT>(a) : launch_t<128, 64, NT>(a);
  return a.group == 32 ? launch_t<64, 32, NT>(a) : launch_t<64, 64, NT>(a);
}

}  // namespace

size_t decode_kv4_workspace_bytes(int Hq, int Hkv, int d) {
  return static_cast<size_t>(kMaxCtas) * sizeof(unsigned long long) +
         static_cast<size_t>(2) * kMaxCtas * (Hq / Hkv) * (static_cast<size_t>(d) + 2) * sizeof(float);
}

cudaError_t launch_decode_kv4_sm103(const DecKv4Launch& a) {
  return a.Hq / a.Hkv <= 8 ? launch_nt<1>(a) : launch_nt<2>(a);
}

}  // namespace attn47
