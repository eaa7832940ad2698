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
//   p scale  times ne, a power of two that follows the largest V scale met so
//        far (as the running maximum follows the scores) and puts it just
//        under 2^7; p <= 2^8, so weights stay under 2^15 and are rounded to
//        11 bits.
// The min terms of the scores are one more MMA (bf16, exact: sum(q_g) is split
// into three bf16 parts); those of the output are summed in fp32.
//
// The MMAs are 16 tokens x 8 heads (S^T = K q^T) and 16 elements x 8 heads
// (O^T += V^T P^T): the 16 slots of a block fill the rows and up to 8 query
// heads per KV head the columns, where 16-head rows would waste half for
// groups up to 8.  P^T changes operand layout with movmatrix.
//
// Work split: the blocks of all (sequence, KV head) runs in one flat order,
// cut into equal costs for every warp of a one-wave grid (a run costs
// kRunCost blocks more than its blocks, for its queries and its end).  A warp
// streams its blocks through a ring of its own in shared memory, one bulk copy
// per (block, head) record, and keeps its own running softmax, so nothing
// inside the CTA waits for anything else until the end.  A run that a warp
// holds whole is written by it; pieces of a run go to shared memory, are merged
// per CTA, and if the run reaches into other CTAs the merged part is published
// and the CTA that arrives last merges the parts.
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
constexpr int kRunCost = 4;
// Lazy stabilisers (see attn_decode_paged): the running maximum moves only
// when a score exceeds it by more than kTau (log2 units).
constexpr float kTau = 8.f;
constexpr int kSeqCache = 2048;
constexpr float kLn2 = 0.6931471805599453f;

// NT: column tiles of 8 query heads (1 or 2).
template <int D, int G, int NT>
struct DecKv4Cfg {
  using Rec = Kv4Layout<D, G>;
  // 12 warps with 168 registers each, or 8 with 255 when two column tiles
  // double the accumulators.
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRows = NT * 8;                       // head rows of a piece
  static constexpr int kPitch = D + 4;                       // floats; conflict-free stores
  static constexpr int kPiece = kRows * kPitch * 4;
  static constexpr int kRing = kStages * Rec::kBytes;        // per warp
  static constexpr int kOffFirst = kWarps * kRing;           // first pieces, one per warp
  static constexpr int kOffMl = kOffFirst + kWarps * kPiece; // (max, sum): [warp][2][kRows]
  static constexpr int kOffCache = kOffMl + kWarps * 2 * kRows * 8;
  static constexpr int kOffShared = kOffCache + kSeqCache * 4;
  static constexpr int kSmem = kOffShared + 2048 + 128;      // + alignment slack
  static_assert(kRing >= kPiece, "a warp's last piece reuses its ring");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct WarpMeta {
  int f_valid, l_valid, l_start;   // l_start: the last piece holds its run's block 0
  int fb, fg, lb, lg;              // runs of the two pieces
  int active;
  long long fcost, lcost;          // cost positions where those runs start
};

struct DecKv4Shared {
  uint64_t full[12][8];
  WarpMeta meta[12];
  long long total;                 // cost of all runs
  long long part_sum[12];
  int bad;
  int last;
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
  float scale_log2;
  unsigned int* status;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ int kv4_seq_len(const DecKv4Params& p, int b) {
  const int L = p.seq_lens[b];
  return L < 0 ? 0 : min(L, p.max_blocks * kBS);
}
__device__ __forceinline__ int kv4_seq_blocks(const DecKv4Params& p, const int* cache, int b) {
  return b < kSeqCache ? cache[b] : (kv4_seq_len(p, b) + kBS - 1) / kBS;
}

// Block position in the flat order of runs.
struct RunPos {
  int b, g, blk, nblk;
  long long cost;                  // cost position where the run starts
};

// The position of cost unit x (its run, and the first block at or after it),
// and the blocks before it.  One warp; all lanes get the result.
__device__ __forceinline__ void locate(const DecKv4Params& p, const int* cache, long long x, long long total,
                                       int lane, RunPos& at, long long& flat) {
  at.b = -1;
  flat = 0;
  long long cost = 0;
  if (x >= total) x = -1;          // the end: only the block count is wanted
  for (int base = 0; base < p.num_seqs; base += 32) {
    const int b = base + lane;
    const int blocks = b < p.num_seqs ? kv4_seq_blocks(p, cache, b) : 0;
    const long long f = static_cast<long long>(blocks) * p.Hkv;
    const long long c = blocks > 0 ? f + static_cast<long long>(kRunCost) * p.Hkv : 0;
    long long ci = c, fi = f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long cy = __shfl_up_sync(0xffffffffu, ci, o);
      const long long fy = __shfl_up_sync(0xffffffffu, fi, o);
      if (lane >= o) {
        ci += cy;
        fi += fy;
      }
    }
    const bool here = x >= 0 && c > 0 && cost + ci - c <= x && x < cost + ci;
    const unsigned hit = __ballot_sync(0xffffffffu, here);
    if (hit) {
      const int src = __ffs(hit) - 1;
      at.b = base + src;
      at.nblk = __shfl_sync(0xffffffffu, blocks, src);
      const long long start = cost + __shfl_sync(0xffffffffu, ci - c, src);
      const long long rel = x - start;
      const int per = at.nblk + kRunCost;
      at.g = static_cast<int>(rel / per);
      at.blk = max(0, static_cast<int>(rel - static_cast<long long>(at.g) * per) - kRunCost);
      at.cost = start + static_cast<long long>(at.g) * per;
      flat += __shfl_sync(0xffffffffu, fi - f, src) + static_cast<long long>(at.g) * at.nblk + at.blk;
      return;
    }
    cost += __shfl_sync(0xffffffffu, ci, 31);
    flat += __shfl_sync(0xffffffffu, fi, 31);
  }
}

// Walk over the runs of a warp's share.
struct Walk {
  RunPos at;
  long long left;                  // blocks of the share not yet passed
  const int* cache;
  __device__ int count() const { return static_cast<int>(min(left, static_cast<long long>(at.nblk - at.blk))); }
  __device__ void next_run(const DecKv4Params& p, int passed) {
    left -= passed;
    at.blk = 0;
    at.cost += at.nblk + kRunCost;
    if (++at.g == p.Hkv) {
      at.g = 0;
      do {
        ++at.b;
        at.nblk = (left > 0 && at.b < p.num_seqs) ? kv4_seq_blocks(p, cache, at.b) : 1;
      } while (left > 0 && at.nblk == 0);
    }
  }
  __device__ void skip(const DecKv4Params& p, int k) {
    while (k > 0 && left > 0) {
      const int c = count();
      if (k < c) {
        at.blk += k;
        left -= k;
        k = 0;
      } else {
        next_run(p, c);
        k -= c;
      }
    }
  }
};

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

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr));
}

// Queries of one (sequence, KV head) as B operands, and what undoes their
// scaling.
template <int D, int G, int NT>
struct QueryFrag {
  uint32_t b[NT][D / 16][2];       // second register: elements 8 up, divided by 16 (codes_hi)
  uint32_t sums[NT][2];            // sum(q_g) 2^-24 of group lane % 4 in three bf16 parts
  float back[NT][2];               // score factor of heads 2 (lane % 4), + 1
};

template <int D, int G, int NT>
__device__ __forceinline__ void load_queries(const DecKv4Params& p, int b, int g, int lane, QueryFrag<D, G, NT>& f) {
  constexpr int kGroups = D / G;
  const int c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = nt * 8 + (lane >> 2);
    const bool live = head < p.group;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        p.q + (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(g) * p.group + (live ? head : 0)) * D) + c;
    uint32_t raw[D / 16][2];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      raw[s][0] = live ? src[8 * s] : 0u;
      raw[s][1] = live ? src[8 * s + 4] : 0u;
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
    const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * 0x1p24f;
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

// Running state of one run: O^T tiles, the min terms, maxima and sums.
template <int D, int G, int NT>
struct RunState {
  float o[NT][D / 16][4];          // rows r and r + 8 (the latter times 16), heads 2c, 2c + 1
  float mins[NT][D / G][2];        // sum of p min over this lane's tokens
  float m[NT][2], l[NT][2];
  uint32_t cap;                    // largest parameter word the weights have room for
  float ne;                        // power of two on the weights

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / G; ++i) mins[nt][i][0] = mins[nt][i][1] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    cap = 0;
    ne = 1.f;
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
      const float inv = 1.f / ne;                // exact: a power of two
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[nt][i][h] = fmaf(o[nt][i][h] * 0x1p24f, inv, mins[nt][16 * i / G][h]);
          o[nt][i][2 + h] = fmaf(o[nt][i][2 + h] * 0x1p20f, inv, mins[nt][16 * i / G][h]);
        }
      }
    }
  }
};

// One block: 16 slots, of which the first `valid` hold tokens.
template <int D, int G, int NT>
__device__ __forceinline__ void take_block(uint32_t rec, int valid, int lane, const QueryFrag<D, G, NT>& q,
                                           RunState<D, G, NT>& st) {
  using Rec = Kv4Layout<D, G>;
  constexpr int kGroups = D / G, kKW = D / 32, kVW = D / 64;
  const int r = lane >> 2, c = lane & 3;
  // MMA row 2c + i (i < 2) and 8 + 2c + (i - 2) hold slot 4c + (i ^ (c & 1)):
  // a lane's four V slots are neighbours, and the exchange of pairs in odd
  // quads spreads its V loads over all banks.
  const int slot = 4 * (r >> 1) + ((r & 1) ^ ((r >> 1) & 1));   // row r; row r + 8 is slot + 2

  uint32_t ka[kKW], kb[kKW], kpa[kGroups], kpb[kGroups];
  lds_words<kKW>(rec + slot * Rec::kRow + c * (D / 8), ka);
  lds_words<kKW>(rec + (slot + 2) * Rec::kRow + c * (D / 8), kb);
  lds_words<kGroups>(rec + Rec::kOffParK + slot * Rec::kParRow, kpa);
  lds_words<kGroups>(rec + Rec::kOffParK + (slot + 2) * Rec::kParRow, kpb);
  uint32_t vw[4][kVW], vpa[kGroups], vpb[kGroups];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    lds_words<kVW>(rec + Rec::kOffV + (4 * c + (i ^ (c & 1))) * Rec::kRow + r * (D / 16), vw[i]);
  lds_words<kGroups>(rec + Rec::kOffParV + slot * Rec::kParRow, vpa);
  lds_words<kGroups>(rec + Rec::kOffParV + (slot + 2) * Rec::kParRow, vpb);

  // --- S^T: rows = slots, columns = heads
  float s[NT][4];
  {
    uint32_t mw = kpa[0], mw8 = kpb[0];          // this lane's group: lane % 4
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
      if (c == i) {
        mw = kpa[i];
        mw8 = kpb[i];
      }
    }
    const uint32_t lo = __byte_perm(mw, 0, 0x1010), lo8 = __byte_perm(mw8, 0, 0x1010);
    const uint32_t a[4] = {lo, lo8, lo, lo8};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      mma_16816(s[nt], a, q.sums[nt][0], q.sums[nt][1]);
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
    for (int ws = 0; ws < G / 32; ++ws) {
      const int w = g * (G / 32) + ws;
      const uint32_t xa = ka[w], xb = kb[w], ya = xa >> 8, yb = xb >> 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816_f16(acc[nt], codes_lo(xa), codes_lo(xb), codes_hi(xa), codes_hi(xb), q.b[nt][2 * w][0],
                      q.b[nt][2 * w][1]);
        mma_16816_f16(acc[nt], codes_lo(ya), codes_lo(yb), codes_hi(ya), codes_hi(yb), q.b[nt][2 * w + 1][0],
                      q.b[nt][2 * w + 1][1]);
      }
    }
    const float sa = word_scale(kpa[g]), sb = word_scale(kpb[g]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = fmaf(sa, acc[nt][0], s[nt][0]);
      s[nt][1] = fmaf(sa, acc[nt][1], s[nt][1]);
      s[nt][2] = fmaf(sb, acc[nt][2], s[nt][2]);
      s[nt][3] = fmaf(sb, acc[nt][3], s[nt][3]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] *= q.back[nt][e & 1];

  if (valid < kBS) {
    // Slots past the end may hold anything: no score, no parameters.
    const bool dead = slot >= valid, dead8 = slot + 2 >= valid;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (dead) s[nt][0] = s[nt][1] = -INFINITY;
      if (dead8) s[nt][2] = s[nt][3] = -INFINITY;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (dead) vpa[g] = 0;
      if (dead8) vpb[g] = 0;
    }
  }

  // --- stabilisers: rare, and the same for the whole warp
  uint32_t big = max(vpa[0], vpb[0]);
#pragma unroll
  for (int g = 1; g < kGroups; ++g) big = max(big, max(vpa[g], vpb[g]));
  bool move = big > st.cap;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    move |= fmaxf(s[nt][0], s[nt][2]) > st.m[nt][0] + kTau;
    move |= fmaxf(s[nt][1], s[nt][3]) > st.m[nt][1] + kTau;
  }
  if (__any_sync(0xffffffffu, move)) {
    big = __reduce_max_sync(0xffffffffu, big);
    float turn = 1.f;
    if (big > st.cap) {
      // Scales of this exponent are below 2^(E - 126): 2^(133 - E) brings
      // them under 2^7 (at most 2^100, so that p ne stays finite; scales
      // under 2^-93 then lose bits).
      const uint32_t E = min((big >> 23) & 0xffu, 254u);
      const float ne = __uint_as_float(min(260u - E, 227u) << 23);
      turn = st.cap ? ne / st.ne : 0.f;
      st.ne = ne;
      st.cap = ((E + 1) << 23) - 1;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(s[nt][h], s[nt][2 + h]);
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o_));
        const bool up = mx > st.m[nt][h] + kTau;
        const float mn = up ? mx : st.m[nt][h];
        f[h] = up ? ex2(st.m[nt][h] - mn) : 1.f;
        st.m[nt][h] = mn;
        st.l[nt][h] *= f[h];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) st.mins[nt][g][h] *= f[h];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        st.o[nt][i][0] *= f[0] * turn;
        st.o[nt][i][1] *= f[1] * turn;
        st.o[nt][i][2] *= f[0] * turn;
        st.o[nt][i][3] *= f[1] * turn;
      }
    }
  }

  // --- weights and O^T: rows = elements of V, columns = heads
  uint32_t pw[NT][kGroups][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float p0 = ex2(s[nt][0] - st.m[nt][0]), p1 = ex2(s[nt][1] - st.m[nt][1]);
    const float p2 = ex2(s[nt][2] - st.m[nt][0]), p3 = ex2(s[nt][3] - st.m[nt][1]);
    st.l[nt][0] += p0 + p2;
    st.l[nt][1] += p1 + p3;
    const float n0 = p0 * st.ne, n1 = p1 * st.ne, n2 = p2 * st.ne, n3 = p3 * st.ne;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float sa = word_scale(vpa[g]), sb = word_scale(vpb[g]);
      const float ma = word_min(vpa[g]), mb = word_min(vpb[g]);
      st.mins[nt][g][0] = fmaf(p0, ma, fmaf(p2, mb, st.mins[nt][g][0]));
      st.mins[nt][g][1] = fmaf(p1, ma, fmaf(p3, mb, st.mins[nt][g][1]));
      pw[nt][g][0] = movmatrix_trans(pack_f16x2(n0 * sa, n1 * sa));
      pw[nt][g][1] = movmatrix_trans(pack_f16x2(n2 * sb, n3 * sb));
    }
  }
#pragma unroll
  for (int w = 0; w < kVW; ++w) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t sel = hf ? 0x7632u : 0x5410u;
      const uint32_t x = __byte_perm(vw[0][w], vw[1][w], sel), y = __byte_perm(vw[2][w], vw[3][w], sel);
      const uint32_t x8 = x >> 8, y8 = y >> 8;
      const int i = 4 * w + 2 * hf;              // tiles i and i + 1 of 16 elements
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

template <int D, int G, int NT>
__global__ void __launch_bounds__(DecKv4Cfg<D, G, NT>::kThreads, 1)
    attn_decode_kv4_kernel(const __grid_constant__ DecKv4Params p) {
  using Cfg = DecKv4Cfg<D, G, NT>;
  using Rec = Kv4Layout<D, G>;
  constexpr int kWarps = Cfg::kWarps, kThreads = Cfg::kThreads, kStages = Cfg::kStages, kRows = Cfg::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  DecKv4Shared* sh = reinterpret_cast<DecKv4Shared*>(smem + Cfg::kOffShared);
  int* cache = reinterpret_cast<int*>(smem + Cfg::kOffCache);
  float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffMl);           // [warp][2][kRows]
  auto first_piece = [&](int w) { return reinterpret_cast<float*>(smem + Cfg::kOffFirst + w * Cfg::kPiece); };
  auto last_piece = [&](int w) { return reinterpret_cast<float*>(smem + w * Cfg::kRing); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    sh->bad = 0;
    sh->last = 0;
    sh->abort = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(smem_addr(&sh->full[w][s]), 1);
    fence_mbar_init();
  }
  pdl_wait_primary();

  // ------------------------------------------------------------------ plan
  {
    long long sum = 0;
    bool bad = false;
    for (int b = tid; b < p.num_seqs; b += kThreads) {
      const int L = p.seq_lens[b];
      bad |= L < 0 || L > p.max_blocks * kBS;
      const int blocks = ((L < 0 ? 0 : min(L, p.max_blocks * kBS)) + kBS - 1) / kBS;
      if (b < kSeqCache) cache[b] = blocks;
      if (blocks > 0) sum += static_cast<long long>(blocks + kRunCost) * p.Hkv;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sh->part_sum[warp] = sum;
    if (bad && blockIdx.x == 0) atomicOr(p.status, kDevBadSeqLen);
  }
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sh->part_sum[w];
  // Every share but the last of all holds at least one block (a share longer
  // than a run's start cost cannot lie inside it).
  const long long shares = static_cast<long long>(gridDim.x) * kWarps;
  const long long chunk = max(static_cast<long long>(kRunCost + 1), (total + shares - 1) / shares);
  const long long mine = (static_cast<long long>(blockIdx.x) * kWarps + warp) * chunk;

  const WaitCtl wc{&sh->abort, p.status, p.timeout_ns};
  WarpMeta meta = {};
  RunPos begin, end;
  long long flat0 = 0, flat1 = 0;
  begin.b = -1;
  if (mine < total) {
    locate(p, cache, mine, total, lane, begin, flat0);
    locate(p, cache, mine + chunk, total, lane, end, flat1);
  }
  const long long blocks = begin.b >= 0 ? flat1 - flat0 : 0;

  if (blocks > 0) {
    meta.active = 1;
    const uint32_t ring = smem_addr(smem + warp * Cfg::kRing);
    Walk w;
    w.at = begin;
    w.left = blocks;
    w.cache = cache;
    // Lane j translates block j of every batch of 32, two batches ahead.
    Walk ahead = w;
    ahead.skip(p, lane);
    auto fetch = [&](int& ph, int& g) {
      ph = -1;
      g = 0;
      if (ahead.left > 0) {
        g = ahead.at.g;
        ph = p.block_table[static_cast<size_t>(ahead.at.b) * p.max_blocks + ahead.at.blk];
      }
      ahead.skip(p, 32);
    };
    int ph0, g0, ph1, g1;
    fetch(ph0, g0);
    fetch(ph1, g1);
    const uint64_t policy = l2_policy_evict_first();
    unsigned present = 0;            // bit s: stage s holds a record (its table entry was in the pool)
    long long issued = 0;
    int stage_in = 0;
    auto issue = [&]() {
      const int src = static_cast<int>(issued & 31);
      bool ok = false;
      if (lane == src) {
        ok = static_cast<unsigned>(ph0) < static_cast<unsigned>(p.num_blocks);
        const uint32_t bar = smem_addr(&sh->full[warp][stage_in]);
        if (ok) {
          mbar_arrive_expect_tx(bar, Rec::kBytes);
          bulk_load_hint(ring + stage_in * Rec::kBytes,
                         p.kv_cache + (static_cast<size_t>(ph0) * p.Hkv + g0) * Rec::kBytes, Rec::kBytes, bar, policy);
        } else {
          atomicOr(p.status, kDevBadBlock);      // outside the pool: that block is skipped
          mbar_arrive(bar);
        }
      }
      const bool got = __any_sync(0xffffffffu, ok);
      present = (present & ~(1u << stage_in)) | (got ? 1u << stage_in : 0u);
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      if ((++issued & 31) == 0) {
        ph0 = ph1;
        g0 = g1;
        fetch(ph1, g1);
      }
    };
    for (int s = 0; s < kStages && issued < blocks; ++s) issue();

    QueryFrag<D, G, NT> q;
    RunState<D, G, NT> st;
    int stage = 0;
    uint32_t phase = 0;
    bool fail = false;
    while (w.left > 0 && !fail) {
      const int cnt = w.count();
      const int L = kv4_seq_len(p, w.at.b);
      load_queries<D, G, NT>(p, w.at.b, w.at.g, lane, q);
      st.reset();
      for (int i = 0; i < cnt; ++i) {
        if (!mbar_wait_warp(smem_addr(&sh->full[warp][stage]), phase, wc)) {
          fail = true;
          break;
        }
        if ((present >> stage) & 1u)
          take_block<D, G, NT>(ring + stage * Rec::kBytes, min(kBS, L - (w.at.blk + i) * kBS), lane, q, st);
        __syncwarp();                            // every lane has read the stage
        if (issued < blocks) issue();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (fail) break;
      st.finish();
      const bool has_start = w.at.blk == 0, has_end = w.at.blk + cnt == w.at.nblk;
      const int c = lane & 3, r = lane >> 2;
      if (has_start && has_end) {
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
                p.lse[h0 + hd] = st.l[nt][h] == 0.f ? -INFINITY : (st.m[nt][h] + __log2f(st.l[nt][h])) * kLn2;
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
              ml[(warp * 2 + (f ? 0 : 1)) * kRows + nt * 8 + 2 * c + h] = make_float2(st.m[nt][h], st.l[nt][h]);
          }
        }
        if (f) {
          meta.f_valid = 1;
          meta.fb = w.at.b;
          meta.fg = w.at.g;
          meta.fcost = w.at.cost;
        } else {
          meta.l_valid = 1;
          meta.l_start = has_start;
          meta.lb = w.at.b;
          meta.lg = w.at.g;
          meta.lcost = w.at.cost;
        }
      }
      w.next_run(p, cnt);
    }
    if (fail) {
      // Copies in flight must land before the CTA may exit.
      for (int s = 0; s < kStages; ++s) {
        const long long fills = issued / kStages + (s < issued % kStages ? 1 : 0);
        if (fills > 0) mbar_wait_warp_drain(smem_addr(&sh->full[warp][s]), static_cast<uint32_t>((fills - 1) & 1), wc);
      }
    }
  }
  if (lane == 0) sh->meta[warp] = meta;
  // Sequences without tokens: O = 0, LSE = -inf.
  for (long long b = static_cast<long long>(blockIdx.x) * kWarps + warp; b < p.num_seqs; b += shares) {
    if (kv4_seq_blocks(p, cache, static_cast<int>(b)) != 0) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(b) * p.Hq * D);
    for (int i = lane; i < p.Hq * D / 2; i += 32) dst[i] = 0u;
    if (p.lse != nullptr)
      for (int h = lane; h < p.Hq; h += 32) p.lse[static_cast<size_t>(b) * p.Hq + h] = -INFINITY;
  }
  __syncthreads();
  pdl_launch_dependents();
  if (sh->abort) return;

  // ------------------------------------------------- pieces of split runs
  // Pieces of one run lie in consecutive warps: last pieces, then one first
  // piece where the run ends.  A run that starts before this CTA or goes on
  // behind it becomes one part per CTA.
  const long long cta_chunk = chunk * kWarps;
  for (int wi = 0; wi < kWarps; ++wi) {
    const WarpMeta& mt = sh->meta[wi];
    const bool tail = mt.l_valid && (wi == kWarps - 1 || !sh->meta[wi + 1].active);
    for (int kind = 0; kind < 2; ++kind) {       // 0: a run that ends in warp wi; 1: the CTA's last run, going on
      if (kind == 0 ? !mt.f_valid : !tail) continue;
      int lo = wi;                               // first warp of the chain
      bool started = kind == 1 && mt.l_start;
      while (!started && lo > 0) {
        --lo;
        started = sh->meta[lo].l_start != 0;
      }
      const int rb = kind == 0 ? mt.fb : mt.lb, rg = kind == 0 ? mt.fg : mt.lg;
      const long long rcost = (kind == 0 ? mt.fcost : mt.lcost) + kRunCost;
      const bool whole = kind == 0 && started;
      const size_t h0 = static_cast<size_t>(rb) * p.Hq + static_cast<size_t>(rg) * p.group;
      const int ws_slot = 2 * static_cast<int>(blockIdx.x) + kind;
      auto piece_of = [&](int w) { return kind == 0 && w == wi ? first_piece(w) : last_piece(w); };
      auto ml_of = [&](int w) { return ml + (w * 2 + (kind == 0 && w == wi ? 0 : 1)) * kRows; };
      for (int item = tid; item < p.group * (D / 4); item += kThreads) {
        const int h = item / (D / 4), col = (item % (D / 4)) * 4;
        float M = -INFINITY;
        for (int w2 = lo; w2 <= wi; ++w2) M = fmaxf(M, ml_of(w2)[h].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        for (int w2 = lo; w2 <= wi; ++w2) {
          const float2 v = ml_of(w2)[h];
          const float wt = v.x == -INFINITY ? (v.y == 0.f ? 0.f : v.y) : ex2(v.x - M);
          const float4 x = *reinterpret_cast<const float4*>(piece_of(w2) + h * Cfg::kPitch + col);
          l += wt * v.y;
          acc.x += wt * x.x;
          acc.y += wt * x.y;
          acc.z += wt * x.z;
          acc.w += wt * x.w;
        }
        if (whole) {
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(p.o + (h0 + h) * D + col) = pk;
          if (col == 0 && p.lse != nullptr) p.lse[h0 + h] = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
        } else {
          *reinterpret_cast<float4*>(p.ws_o + (static_cast<size_t>(ws_slot) * p.group + h) * D + col) = acc;
          if (col == 0)
            *reinterpret_cast<float2*>(p.ws_ml + (static_cast<size_t>(ws_slot) * p.group + h) * 2) = make_float2(M, l);
        }
      }
      if (whole) continue;
      const int per_run = kv4_seq_blocks(p, cache, rb);
      const int cta0 = static_cast<int>(rcost / cta_chunk);
      const int cta1 = static_cast<int>((rcost + per_run - 1) / cta_chunk);
      const int nparts = cta1 - cta0 + 1;
      // Publish: every thread's part visible to the GPU, then one arrival.
      __threadfence();
      __syncthreads();
      if (tid == 0)
        sh->last = count_arrival(p.arrive + cta0, p.epoch, static_cast<int>(blockIdx.x) - cta0, nparts, p.status);
      __syncthreads();
      const bool last = sh->last != 0;
      if (last) {
        __threadfence();
        // Part x is in CTA x's slot 1, the run's end in slot 0.
        auto slot_of = [&](int x) { return static_cast<size_t>(2 * x + (x == cta1 ? 0 : 1)) * p.group; };
        for (int item = tid; item < p.group * (D / 4); item += kThreads) {
          const int h = item / (D / 4), col = (item % (D / 4)) * 4;
          float M = -INFINITY;
          for (int x = cta0; x <= cta1; ++x)
            M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot_of(x) + h).x);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float l = 0.f;
          for (int x = cta0; x <= cta1; ++x) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot_of(x) + h);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (slot_of(x) + h) * D + col));
            const float wt = v.x == -INFINITY ? (v.y == 0.f ? 0.f : v.y) : ex2(v.x - M);
            l += wt * v.y;
            acc.x += wt * y.x;
            acc.y += wt * y.y;
            acc.z += wt * y.z;
            acc.w += wt * y.w;
          }
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(p.o + (h0 + h) * D + col) = pk;
          if (col == 0 && p.lse != nullptr) p.lse[h0 + h] = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
        }
      }
      __syncthreads();                           // sh->last is free again
    }
  }
}

template <int D, int G, int NT>
cudaError_t launch_t(const DecKv4Launch& a) {
  using Cfg = DecKv4Cfg<D, G, NT>;
  auto kern = attn_decode_kv4_kernel<D, G, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
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
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  const int ctas = a.sms < 1 ? 1 : a.sms > kMaxCtas ? kMaxCtas : a.sms;
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
