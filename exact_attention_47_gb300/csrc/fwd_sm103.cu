// Exact attention forward (prefill) for sm_103a.
//
// softmax(scale * Q K^T + causal mask) V computed tile by tile with the
// running-max / running-sum softmax, so the N x N score matrix never leaves
// the SM ("Advanced attention mechanisms – II", sections "Flash Attention",
// "Tiling" steps 1-3, "Softmax stabiliser", "Incremental / online softmax";
// "Fast attention kernels and operator fusion accelerate AI models", section
// "FlashAttention-style attention and Paged Attention").
//
// One CTA owns a 256-row query block of one (batch, query head), split into
// two 128-row tiles A and B that share every K/V tile of the KV head:
//   warps 0-3   softmax of tile A, one thread per query row (= TMEM lane)
//   warps 4-7   softmax of tile B
//   warp 8      TMA producer: Q_A, Q_B once, then K_j / V_j into a stage ring
//   warp 9      MMA issuer (one thread) and owner of the TMEM allocation
//   warps 10-11 idle (they complete the third warpgroup for setmaxnreg);
//               in paged mode they gather the K and V tiles
// Tensor memory: S_A, S_B (128 fp32 columns each), O_A, O_B (d columns
// each; at d = 64 with contiguous K/V, d + 16, the extra columns holding the
// row sums of P that P V forms against a ones column beside V).  After
// reading S_X, the softmax writes P_X (bf16, two per column)
// over the first 64 columns of S_X and the MMA reads it from there (A
// operand in TMEM), so P never touches shared memory.  The tensor core runs
// ... PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) ... in issue order, so while one
// warpgroup computes exponentials the tensor core works on the other tile,
// and the completion of S_X(j+1) also proves PV_X(j) has finished, which
// makes O_X and the P_X columns safe to touch again.
// The whole MMA warp runs the issuing schedule and one elected lane issues,
// so descriptors and barrier addresses stay warp-uniform values.  The
// issuer tests the barriers of its next group while the last MMAs of the
// current group are being issued, and never re-tests a stage it already
// knows is full: no barrier round trip sits between two groups.
//
// The stabiliser m of a row ("Softmax stabiliser") is only moved when the
// tile maximum exceeds it by more than 2^8 (in the exp2 domain), so O and l
// are rescaled rarely; exponents stay <= 8, numerators <= 256, and the final
// O / l and LSE are the same function of the same stabiliser.
//
// Paged mode (chunked prefill over a paged KV cache; same page, same
// section: the cache lives in fixed-size blocks and every position goes
// through the block table): the N query rows of sequence b are its new
// tokens at positions ctx_b .. ctx_b + N - 1, and K/V come from the cache.
// A 128-key tile is eight 16-slot blocks of 16 x d contiguous values each.
// Warps 10 (K) and 11 (V), idle otherwise, gather them: the lanes look up
// the eight table entries, then copy each block with 16-byte cp.async
// (a warp instruction moves 512 contiguous bytes) straight into the
// 128-byte-swizzled tile layout the MMA descriptors read, wait for their
// copies, fence them into the async proxy and arrive on the stage's full
// barrier.  (Sixteen 16-row TMA boxes per tile took about a quarter longer
// per tile than this.)  Blocks past the sequence are written as zeros.
// Query row i may see keys 0 .. ctx_b + i: the causal mask at an offset, so
// it can fall across two key tiles.  A unit's cost grows with
// ctx_b + its query block's first row, so units are walked in decreasing
// order of that key (every CTA ranks the (sequence, query block) pairs the
// same way at start-up) instead of query block by query block.
//
// Paged mode over an 8-bit cache (kPagedKv8): the same, but the cache holds the
// new tokens already, sequence b's row i is the token at position seq_lens[b] -
// N + i (before position 0 it sees nothing: O = 0, LSE = -inf), and everything is
// fp16 in place of bf16: an e4m3 code is an fp16 number, and one conversion
// instruction makes two.  The scales, powers of two for each 16 keys, act where they
// cost least.  With S the product with the K codes, b a 16-key block, back the row's
// factor (below) and e_b = log2 of the V scale:
//   P'_j = 2^(S_j scale_Kb back + e_b - m),   O = sum P'_j code_j / l,
//   l = sum over blocks 2^-e_b sum P'_j
// so a block's scales are the two constants of the FMA before the exponential, and
// one more FMA for a block's sum.  P' is at most 2^16 (its sum over a tile is
// checked, a tile beyond is redone with m moved), 2^8 at the maximum; what rounds
// to zero in fp16 is 2^-32 of the largest contribution.  The rows of Q, which each
// softmax warpgroup loads for itself, are turned into fp16 in shared memory, each by
// a power of two of its own that brings its largest element to [2^14, 2^15).
// Warp 8 looks up the blocks and their scales, a tile ahead, and has the TMA bring
// their codes into a ring; warps 10 (K) and 11 (V) take two at a time from
// there, convert them and store them into the swizzled tile.  NaN codes are cleared
// where there can be any (a sequence's last block, flagged blocks); the look-up keeps
// the first position of a flagged token, and a row that sees that position gets NaN
// in the epilogue.  Rows whose sizes these exponents cannot hold are computed again
// behind the last unit (careful_rows).
// With fewer than 256 new tokens the rows of all query heads that share a KV head
// make one row of query blocks (row = head in the group times N + token), so that
// a 256-row unit is not mostly empty.
// A tile takes some 4500 cycles with d = 128 (4 sequences of up to 8192 keys, 2048 new
// tokens of 12 heads over 2: 225 us) where the tensor core is busy for 2850 of them
// and a softmax warp for 2100; the gather takes 2100 a tile and waits 1700 for codes,
// of which no more fit in flight.  Tried and slower: converting by shifts and masks
// (7 instructions for 4 codes instead of 4; a gather warp shares its scheduler with
// two softmax warps: 284 us and up), converting in place in the stage (300: a stage is
// held all the way from the copy to the MMA), copies issued by the gather warps
// themselves (291), a fourth warpgroup with two warps to an operand (300: the softmax
// has too few registers left).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fwd_sm103.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace attn47 {
namespace {

constexpr int kBM = 128;            // rows per query tile (= TMEM lanes)
constexpr int kBN = 128;            // keys per K/V tile
constexpr int kTiles = 2;           // query tiles per CTA
constexpr int kRowsPerCta = kBM * kTiles;
constexpr int kThreads = 384;       // 2 softmax warpgroups + 1 producer/MMA warpgroup
enum Source { kContiguous, kPagedBf16, kPagedKv8 };
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
// Launched at 168 registers a thread (384 x 168 = 64512); the softmax
// warpgroups then take 216 and the producer/MMA warpgroup keeps 72:
// 256 x 216 + 128 x 72 = 64512, and per sub-partition 216 + 216 + 72 = 504
// = 3 x 168, so the increase never waits for registers nobody frees.
// (8-bit cache: the gather spills at 72.  Timed with 216 + 72, 208 + 88 and 200 +
// 104: d = 128, 4 chunks of 2048 tokens, takes 263, 237 and 231 us; d = 64, 24
// left-padded chunks of 100, 22.9, 22.7 and 23.1.)
__host__ __device__ constexpr uint32_t regs_softmax(bool kv8, int d) { return !kv8 ? 216 : d == 128 ? 200 : 208; }
__host__ __device__ constexpr uint32_t regs_other(bool kv8, int d) { return !kv8 ? 72 : d == 128 ? 104 : 88; }
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTau = 8.0f;        // lazy-rescale threshold, log2 units
constexpr float kHigh8 = 8.0f;      // 8-bit cache: log2 of P' at the maximum
constexpr float kNoKeys = -1e30f;   // 8-bit cache: m before the row's first key

__host__ __device__ constexpr int sort_max_pairs(int source) { return source == kPagedKv8 ? 1024 : 2048; }
// 8-bit cache: raw blocks (K and V codes) in flight, taken in pairs; as many as there
// is room for (d = 64: 16 sequences of 6000 tokens took 125 us with 6, 108 with 14).
__host__ __device__ constexpr int raw_stages(int d) { return d == 128 ? 6 : 14; }
constexpr int kMaxRawStages = 14;
constexpr int kScaleTiles = 16;     // tiles whose scales are kept
constexpr int kAgain = 64;          // see FwdBarriers
constexpr int kWideExps = 72;       // see careful_rows

// SUMV (d = 64 with contiguous K/V): the row sums of P come from the tensor
// core.  Every V stage gets a second 64-column chunk, written once, whose
// first column is all ones, and P V runs with N = d + 16: columns d .. d+15
// of O_X then hold P times that column, the row sums of the bf16 P that P V
// uses, at no extra MMA instruction (three stages instead of four make room).
template <int D, bool SUMV = false, int SOURCE = kContiguous>
struct FwdLayout {
  static constexpr int kChunks = D / 64;                 // 128-byte swizzle atoms per row
  static constexpr int kStages = (D == 128) ? 2 : SUMV ? 3 : 4;
  static constexpr int kQTile = kBM * D * 2;
  static constexpr int kKV = kBN * D * 2;
  static constexpr int kQChunk = kBM * 128;              // one 64-column box of a Q tile
  static constexpr int kKVChunk = kBN * 128;
  static constexpr int kVStage = SUMV ? kKV + kKVChunk : kKV;   // V stage stride (+ the ones chunk)
  static constexpr int kNPV = SUMV ? D + 16 : D;         // N of the P V MMAs
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTiles * kQTile;
  static constexpr int kOffV = kOffK + kStages * kKV;
  static constexpr int kOffBar = kOffV + kStages * kVStage;
  static constexpr int kOffCtx = kOffBar + 1024;         // paged: ctx_b of each sequence
  static constexpr int kOffOrder = kOffCtx + 4 * 256;    // paged: (b << 16 | qblk) of each cost rank
  // 8-bit cache: (K scale times scale log2 e, log2 of V's, 1 / V's, whether the unit's V
  // scales as of this tile are kWideExps powers of two apart) of the 8 blocks of tile t
  // at t % kScaleTiles; a ring of raw blocks.
  static constexpr int kOffScales = kOffOrder + 4 * sort_max_pairs(SOURCE);
  static constexpr int kOffRaw = (kOffScales + kScaleTiles * 8 * 16 + 1023) / 1024 * 1024;
  static constexpr int kRawHalf = 16 * D;                     // a record's K or V codes
  static constexpr int kRaw = 2 * kRawHalf;
  static constexpr int kRawStages = raw_stages(D);
  static constexpr int kSmem = (SOURCE == kPagedKv8 ? kOffRaw + kRawStages * kRaw : kOffScales) + 1024;   // + alignment slack
  static constexpr uint32_t kColS0 = 0, kColS1 = 128;
  static constexpr uint32_t kColO0 = 256, kColO1 = SUMV ? 384 : 256 + D;
};

struct FwdBarriers {
  uint64_t q_full[2], q_empty[2];     // Q tile x of the current work unit / free again
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t o_free[2];                 // O_X read out by the epilogue of the previous unit
  uint64_t mma_final;
  // 8-bit cache: Q tile x is fp16; raw block s has come / has been read, and
  // what it is.
  uint64_t q_ready[2], raw_full[kMaxRawStages], raw_empty[kMaxRawStages];
  uint32_t tmem_base;
  int abort;
  int raw_kind[kMaxRawStages], raw_fills[kMaxRawStages];
  int q_loads[2];                     // copies of Q tile x asked for (its first thread's count)
  unsigned again[8][kAgain / 32];     // bands of softmax warp w with rows for careful_rows (the last one: and those behind)
  // The first position of a flagged token in unit u (of the CTA's), in its tiles so
  // far, at u % 16: the look-up is at most two tiles ahead of the gather, that kStages
  // ahead of the MMAs, and these a unit ahead of the epilogue (d = 64: 2 + 4 + 1 + 1),
  // which also bounds the scales' ring.
  int first_flagged[16];
};
enum RawKind { kRawNone, kRawCodes, kRawCareful, kRawEnd };   // none: zeros; careful: there may be NaN codes
static_assert(sizeof(FwdBarriers) <= 1024, "room in the layout");

struct FwdParams {
  void* o;
  float* lse;
  int N, Hq, Hkv, group, num_q_blocks, bh_total, num_units;
  float scale_log2;
  unsigned int* status;
  unsigned long long timeout_ns;
  // paged mode only
  const uint8_t* k_cache;   // [num_blocks, Hkv, 16, D] bf16
  const uint8_t* v_cache;
  const int* block_table;   // [B, max_blocks]
  const int* ctx_lens;      // [B] tokens cached before the N new ones
  int max_blocks, num_blocks;
  int max_ctx;              // max_blocks * 16 - N: largest valid ctx_lens entry
  // 8-bit cache: ctx_lens are the sequences' lengths, new tokens included; a
  // "query head" is a KV head's whole group where `rows` tokens are fewer than 256
  // (then N is group * rows, and row r is token r % rows).
  const uint8_t* kv_cache;
  int rows;
  bool packed;
  const __nv_bfloat16* q;   // [B, Hq, N, d]
};

// Cost ordering of the paged mode fits in shared memory up to these sizes
// (beyond them a second instantiation keeps the query-block-major order).
constexpr int kSortMaxSeqs = 256;

constexpr int kPageRows = 16;                        // token slots per cache block
constexpr int kPagesPerTile = kBN / kPageRows;
constexpr int kWarpGatherK = 10;                     // paged mode: K / V gather warps
constexpr int kWarpGatherV = 11;
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// Four e4m3 codes, those that are NaN as 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  const uint32_t nan = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;   // 1 in the byte of a 0x7f or 0xff
  return w & ~(nan * 0xffu);
}

// 8-bit cache: rows that the tiles cannot hold, one to a lane, key by key in fp32,
// each scale where its product is: the row's O and LSE, q at position qpos (-1: no
// such row). The tiles' numerators P' carry the V scales, 2^e.  One that is under
// 2^-126 is lost, and with it up to 2^(-126 - e) of l a key (moving m, up to 2^(-110 -
// e)), where l is at least 2^(8 - e') by the largest P'.  With all e within kWideExps
// of each other that is 2^-46 of l a key, beyond that with l of 2^-8 and more 2^-38 (e
// is at least -64); the other rows (their largest P' has an e' over 16) come here.  So
// do rows with scores beyond 2^26 log2 units, where m is a multiple of 8 and more and
// P' may leave fp16, and those whose O shows that it has done so (from 2^40 on, where
// rows not in use may be, they are NaN).  About 1000 instructions a key and 32 columns
// (4 sequences of 1000 tokens, 512 queries of 12 heads over 2, d = 128: 3.9 ms where
// the tiles take 40 us), out of line so that the tiles' loop stays as it is: sums of l
// of its own in that loop cost the chunks 3 to 6 %.
template <int D>
__device__ __noinline__ void careful_rows(const uint8_t* kv_cache, const int* table, int num_blocks, int Hkv, int kvh,
                                          float scale_log2, int qpos, const __nv_bfloat16* q, __nv_bfloat16* o,
                                          float* lse) {
  const int last = __reduce_max_sync(0xffffffffu, qpos);
  uint32_t qw[D / 2];                              // fp16, as in the tiles
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = qpos < 0 ? make_uint4(0u, 0u, 0u, 0u) : reinterpret_cast<const uint4*>(q)[i];
    qw[4 * i] = v.x;
    qw[4 * i + 1] = v.y;
    qw[4 * i + 2] = v.z;
    qw[4 * i + 3] = v.w;
    mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu),
                  __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  }
  const int fe = min(268 - static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7), 253);
  const float up = __uint_as_float(static_cast<uint32_t>(fe) << 23);
  const float back = __uint_as_float(static_cast<uint32_t>(254 - fe) << 23);
#pragma unroll
  for (int i = 0; i < D / 2; ++i)
    qw[i] = pack_f16x2(__uint_as_float(qw[i] << 16) * up, __uint_as_float(qw[i] & 0xffff0000u) * up);
  auto numbers = [](uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); };
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {             // 32 columns of O at a time
    float m = -INFINITY, l = 0.f, acc[32];
    bool spoilt = false;
#pragma unroll
    for (int c = 0; c < 32; ++c) acc[c] = 0.f;
#pragma unroll 1
    for (int blk = 0; blk <= last / kPageRows; ++blk) {
      const int phys = __ldg(table + blk);
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(num_blocks)) continue;
      const uint8_t* rec = kv_cache + (static_cast<size_t>(phys) * Hkv + kvh) * Kv8Layout<D>::kBytes;
      const uint4 tail = __ldg(reinterpret_cast<const uint4*>(rec + Kv8Layout<D>::kOffTail));
#pragma unroll 1
      for (int slot = 0; slot < kPageRows && blk * kPageRows + slot <= last; ++slot) {
        uint4 kw[D / 16], vw[2];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) kw[i] = __ldg(reinterpret_cast<const uint4*>(rec + slot * D) + i);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          vw[i] = __ldg(reinterpret_cast<const uint4*>(rec + Kv8Layout<D>::kOffV + slot * D + c0) + i);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t w[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 k0 = numbers(e4m3x2_to_f16x2(w[c])), k1 = numbers(e4m3x2_hi_to_f16x2(w[c]));
            const float2 q0 = numbers(qw[8 * i + 2 * c]), q1 = numbers(qw[8 * i + 2 * c + 1]);
            s[c] = fmaf(q0.x, k0.x, fmaf(q0.y, k0.y, fmaf(q1.x, k1.x, fmaf(q1.y, k1.y, s[c]))));
          }
        }
        // (0 stays 0.)
        const float x = ((s[0] + s[1]) + (s[2] + s[3])) * back * scale_log2 * __uint_as_float(tail.x);
        if (blk * kPageRows + slot > qpos) continue;
        spoilt |= (((tail.z | (tail.z >> 16)) >> slot) & 1u) != 0;
        const float to = fmaxf(m, x), turn = m == to ? 1.f : ex2(m - to);
        const float w0 = x == to ? 1.f : ex2(x - to);
        m = to;
        l = fmaf(l, turn, w0);
        const float wv = w0 * __uint_as_float(tail.y);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 v0 = numbers(e4m3x2_to_f16x2(w[c])), v1 = numbers(e4m3x2_hi_to_f16x2(w[c]));
            float* a = acc + 16 * i + 4 * c;
            a[0] = fmaf(a[0], turn, wv * v0.x);
            a[1] = fmaf(a[1], turn, wv * v0.y);
            a[2] = fmaf(a[2], turn, wv * v1.x);
            a[3] = fmaf(a[3], turn, wv * v1.y);
          }
        }
      }
    }
    if (qpos < 0) continue;
    spoilt |= fabsf(m) >= 0x1p40f && l != 0.f;     // (as in the epilogue)
    const float inv = spoilt ? __uint_as_float(0x7fc00000u) : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < 32; c += 8)
      reinterpret_cast<uint4*>(o + c0 + c)[0] =
          make_uint4(pack_bf16x2(acc[c] * inv, acc[c + 1] * inv), pack_bf16x2(acc[c + 2] * inv, acc[c + 3] * inv),
                     pack_bf16x2(acc[c + 4] * inv, acc[c + 5] * inv), pack_bf16x2(acc[c + 6] * inv, acc[c + 7] * inv));
    if (c0 == 0 && lse != nullptr) *lse = spoilt ? __uint_as_float(0x7fc00000u) : (m + __log2f(l)) * kLn2;
  }
}

template <int D, bool CAUSAL, int SOURCE, bool SORTED>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_sm103_kernel(const __grid_constant__ CUtensorMap tq,
                          const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const FwdParams p) {
  constexpr bool PAGED = SOURCE != kContiguous, KV8 = SOURCE == kPagedKv8;
  constexpr bool SUMV = D == 64 && !PAGED;
  using L = FwdLayout<D, SUMV, SOURCE>;
  extern __shared__ uint8_t smem_raw[];
  // Aligned through an integer round trip (the pointer becomes generic):
  // measured faster for this kernel than smem_align1024.
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FwdBarriers* bar = reinterpret_cast<FwdBarriers*>(smem + L::kOffBar);
  const uint32_t sQ = smem_addr(smem + L::kOffQ);
  const uint32_t sK = smem_addr(smem + L::kOffK);
  const uint32_t sV = smem_addr(smem + L::kOffV);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Persistent CTAs: work unit k (one 256-row query block of one (batch,
  // head)) in heaviest-first order (last query blocks first, for causal);
  // CTA c takes unit c of the first band of gridDim.x units, then walks the
  // bands in alternating directions so heavy and light units pair up.
  const int grid = static_cast<int>(gridDim.x);
  const int cta = static_cast<int>(blockIdx.x);
  auto unit_at = [&](int band) {
    return band * grid + ((band & 1) ? grid - 1 - cta : cta);
  };
  const int kv_total = (p.N + kBN - 1) / kBN;
  struct Unit {
    int qblk, zq, zkv, nA, nB;
    int pos0, b, kvh, nblk;                            // paged: ctx_b, sequence, KV head, blocks
  };
  const int* s_ctx = reinterpret_cast<const int*>(smem + L::kOffCtx);
  const int* s_order = reinterpret_cast<const int*>(smem + L::kOffOrder);
  auto unit_info = [&](int k) {
    Unit u;
    int bh;
    if constexpr (SORTED) {
      // Rank k / Hq of the (sequence, query block) pairs by decreasing cost;
      // the Hq heads of a pair are consecutive units (they share K/V tiles).
      const int r = k / p.Hq;
      const int e = s_order[r];
      u.qblk = e & 0xffff;
      bh = (e >> 16) * p.Hq + (k - r * p.Hq);
    } else {
      u.qblk = p.num_q_blocks - 1 - k / p.bh_total;
      bh = k % p.bh_total;
    }
    u.zq = bh;                                         // b * Hq + h
    u.b = bh / p.Hq;
    u.kvh = (bh % p.Hq) / p.group;
    u.zkv = u.b * p.Hkv + u.kvh;
    if constexpr (KV8) {
      const int len = min(max(__ldg(p.ctx_lens + u.b), 0), p.max_blocks * kPageRows);
      u.pos0 = len - p.rows;                           // (negative: rows that see nothing)
      // The last token among rows r0 .. r1 (packed: they may span heads).
      auto last = [&](int r0, int r1) {
        r1 = min(r1, p.N - 1);
        const int i0 = r0 % p.rows;
        return i0 + r1 - r0 >= p.rows ? p.rows - 1 : i0 + r1 - r0;
      };
      const int r0 = u.qblk * kRowsPerCta;
      const int lastA = last(r0, r0 + kBM - 1), lastB = r0 + kBM < p.N ? last(r0 + kBM, r0 + 2 * kBM - 1) : lastA;
      u.nA = max(u.pos0 + lastA, 0) / kBN + 1;
      u.nB = max(max(u.pos0 + lastB, 0) / kBN + 1, u.nA);
      u.nblk = (len + kPageRows - 1) / kPageRows;
    } else if constexpr (PAGED) {
      // A ctx_lens entry outside [0, max_ctx] was reported by the append
      // kernel; it is clamped here so every loop stays bounded.
      u.pos0 = min(max(__ldg(p.ctx_lens + u.b), 0), p.max_ctx);
      const int lastA = min(u.qblk * kRowsPerCta + kBM - 1, p.N - 1);
      const int lastB = min(u.qblk * kRowsPerCta + 2 * kBM - 1, p.N - 1);
      u.nA = (u.pos0 + lastA) / kBN + 1;               // tiles up to key pos0 + last row
      u.nB = (u.pos0 + lastB) / kBN + 1;
      u.nblk = min((u.pos0 + p.N + kPageRows - 1) / kPageRows, p.max_blocks);
    } else {
      u.pos0 = 0;
      u.nblk = 0;
      // K/V tiles each query tile needs; the diagonal tile of tile X is 2*qblk + X.
      u.nA = CAUSAL ? min(2 * u.qblk + 1, kv_total) : kv_total;
      u.nB = CAUSAL ? min(2 * u.qblk + 2, kv_total) : kv_total;
    }
    return u;
  };

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_addr(&bar->q_full[x]), 1);
      mbar_init(smem_addr(&bar->q_empty[x]), 1);
      mbar_init(smem_addr(&bar->o_free[x]), 4);
    }
    for (int s = 0; s < L::kStages; ++s) {
      // Paged: every lane of a gather warp arrives once its copies landed.
      mbar_init(smem_addr(&bar->k_full[s]), PAGED ? 32 : 1);
      mbar_init(smem_addr(&bar->v_full[s]), PAGED ? 32 : 1);
      mbar_init(smem_addr(&bar->k_empty[s]), 1);
      mbar_init(smem_addr(&bar->v_empty[s]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_addr(&bar->s_full[x]), 1);
      mbar_init(smem_addr(&bar->p_full[x]), 4);
      mbar_init(smem_addr(&bar->o_done[x]), 1);
    }
    mbar_init(smem_addr(&bar->mma_final), 1);
    if constexpr (KV8) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_addr(&bar->q_ready[x]), kBM);
        bar->q_loads[x] = 0;
      }
      for (int x = 0; x < 8 * kAgain / 32; ++x) (&bar->again[0][0])[x] = 0;
      for (int x = 0; x < L::kRawStages; ++x) {
        mbar_init(smem_addr(&bar->raw_full[x]), 1);
        mbar_init(smem_addr(&bar->raw_empty[x]), 2);
        bar->raw_fills[x] = 0;
      }
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&bar->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if constexpr (SUMV) {
    // The ones chunk of every V stage: in key row r, bf16 1.0 in its column
    // 0, whose 16-byte piece sits at piece 0 ^ (r mod 8) of the row's 128
    // bytes (the TMA's 128-byte swizzle); zeros elsewhere.
    for (int i = threadIdx.x; i < L::kStages * L::kKVChunk / 4; i += kThreads) {
      const int st = i / (L::kKVChunk / 4), k = i % (L::kKVChunk / 4);
      const int r = k / 32, w = k % 32;
      reinterpret_cast<uint32_t*>(smem + L::kOffV + st * L::kVStage + L::kKV)[k] =
          (w == (r & 7) * 4) ? 0x3F80u : 0u;
    }
    fence_proxy_async_smem();
  }
  // Launched as a programmatic dependent: the set-up above overlaps the end
  // of the kernel before this one in the stream; nothing in global memory
  // is read or written before that kernel has finished.
  pdl_wait_primary();
  if constexpr (KV8) {
    // (The append reports bad lengths for a bf16 cache; this call has none.)
    if (cta == 0) {
      bool bad = false;
      for (int b = threadIdx.x; b < p.bh_total / p.Hq; b += kThreads) {
        const int len = __ldg(p.ctx_lens + b);
        bad |= len < 0 || len > p.max_blocks * kPageRows;
      }
      if (bad) atomicOr(p.status, kDevBadSeqLen);
    }
  }
  if constexpr (SORTED) {
    {
      // Cost key of pair (b, qblk): ctx_b + 256 * qblk (the K/V tiles of the
      // unit grow with it).  Rank = pairs with a larger key, plus equal keys
      // of a smaller pair index; counted per sequence in closed form.
      const int S = p.bh_total / p.Hq;
      const int nq = p.num_q_blocks;
      int* ctx_w = reinterpret_cast<int*>(smem + L::kOffCtx);
      for (int b = threadIdx.x; b < S; b += kThreads)
        ctx_w[b] = min(max(__ldg(p.ctx_lens + b), 0), KV8 ? p.max_blocks * kPageRows : p.max_ctx);
      __syncthreads();
      int* order_w = reinterpret_cast<int*>(smem + L::kOffOrder);
      for (int i = threadIdx.x; i < S * nq; i += kThreads) {
        int rank = 0;
        if (KV8 && p.packed) {                     // all blocks of a sequence cost the same
          const int key = s_ctx[i / nq];
          for (int b = 0; b < S; ++b)
            if (s_ctx[b] > key || (s_ctx[b] == key && b < i / nq)) rank += nq;
          order_w[rank + i % nq] = ((i / nq) << 16) | (i % nq);
          continue;
        }
        const int key = s_ctx[i / nq] + kRowsPerCta * (i % nq);
        for (int b = 0; b < S; ++b) {
          const int dk = key - s_ctx[b];
          if (dk < 0) {
            rank += nq;                            // every block of b has a larger key
          } else {
            const int q0 = dk / kRowsPerCta;       // blocks above q0 have larger keys
            rank += max(nq - q0 - 1, 0);
            if (dk % kRowsPerCta == 0 && q0 < nq && b * nq + q0 < i) ++rank;
          }
        }
        order_w[rank] = ((i / nq) << 16) | (i % nq);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl wc{&bar->abort, p.status, p.timeout_ns};
  if (warp >= 8) {
  regs_decrease<regs_other(KV8, D)>();
  if (KV8 && warp == kWarpLoad) {
    // --------------------------------------- the blocks of the tiles, 8-bit records
    // Lane i < 8 looks up block i of a tile.  Table entries are read two tiles
    // ahead of their use here, scales one tile ahead.
    int band = 0, j = 0, left = 0, nblk = 0, kvh = 0;        // of the tile to read next
    const int* row = nullptr;
    auto open_unit = [&]() {
      const int k = unit_at(band);
      left = 0;
      if (k >= p.num_units) return;
      const Unit u = unit_info(k);
      left = u.nB;
      nblk = u.nblk;
      kvh = u.kvh;
      row = p.block_table + static_cast<size_t>(u.b) * p.max_blocks;
      j = 0;
    };
    open_unit();
    // A tile: the table entry of this lane's block and its KV head (-1: no such
    // block), then its record; its number in its unit (-1: there is no tile),
    // whether it is the last, and whether the block is the sequence's last.
    struct Tile {
      int entry, kvh, number;
      bool last, ends;
    };
    auto read_table = [&]() {
      Tile x;
      x.entry = -1;
      x.kvh = -1;
      x.number = left > 0 ? j : -1;
      x.last = left == 1;
      x.ends = false;
      if (left > 0) {
        const int lb = j * kPagesPerTile + lane;
        if (lane < kPagesPerTile && lb < nblk) {
          x.entry = __ldg(row + lb);
          x.kvh = kvh;
          x.ends = lb == nblk - 1;
        }
        ++j;
        if (--left == 0) {
          ++band;
          open_unit();
        }
      }
      return x;
    };
    // The record of the lane's block, -1 for none (read as zeros).
    auto record = [&](const Tile& x) {
      if (static_cast<unsigned>(x.entry) < static_cast<unsigned>(p.num_blocks)) return x.entry * p.Hkv + x.kvh;
      if (x.kvh >= 0) atomicOr(p.status, kDevBadBlock);
      return -1;
    };
    auto tail_of = [&](int rec) {                            // (K scale, V scale, flags)
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (rec >= 0)
        v = __ldg(reinterpret_cast<const uint4*>(p.kv_cache + static_cast<size_t>(rec) * Kv8Layout<D>::kBytes +
                                                 Kv8Layout<D>::kOffTail));
      return v;
    };
    Tile next = read_table();
    int now_rec = record(next), now_number = next.number;
    bool now_last = next.last, now_ends = next.ends;
    uint4 tail = tail_of(now_rec);
    next = read_table();
    int unit = 0, flagged = 0x7fffffff, n = 0;
    int least = 255, most = 0;                               // exponents of the unit's V scales so far
    bool ok = true;
    // Block number `at` into the ring.
    auto fill = [&](int at, int rec, int what) {
      const int s = at % L::kRawStages;
      const uint32_t full = smem_addr(&bar->raw_full[s]);
      if (!mbar_wait_sleep(smem_addr(&bar->raw_empty[s]), ((at / L::kRawStages) & 1) ^ 1, wc)) return false;
      reinterpret_cast<volatile int*>(bar->raw_kind)[s] = what;
      ++bar->raw_fills[s];
      mbar_arrive_expect_tx(full, rec >= 0 ? L::kRaw : 0);
      if (rec >= 0) tma_load_3d(smem_addr(smem + L::kOffRaw) + s * L::kRaw, &tk, full, 0, 0, rec);
      return true;
    };
    for (;; ++n) {
      const int next_rec = record(next), next_number = next.number;
      const bool next_last = next.last, next_ends = next.ends;
      const uint4 next_tail = tail_of(next_rec);
      // (d = 128, whose ring is short: 16 sequences of 6000 tokens, 64 queries of 4
      // heads each over 8 KV heads, 143 -> 131 us.)
      if (D == 128 && next_rec >= 0)
        bulk_prefetch_l2(p.kv_cache + static_cast<size_t>(next_rec) * Kv8Layout<D>::kBytes, L::kRaw);
      next = read_table();
      if (now_number < 0) break;
      // The unit's first flagged token so far: the lowest bit of its block's flags.
      // It is stored before the tile's blocks are on their way, so whoever has seen
      // this tile's products sees it, with query tile A already before the unit's end.
      const uint32_t bits = (tail.z | (tail.z >> 16)) & 0xffffu;
      if (__any_sync(0xffffffffu, bits != 0)) {
        const int at = bits != 0 ? (now_number * kPagesPerTile + lane) * kPageRows + __ffs(bits) - 1 : 0x7fffffff;
        flagged = min(flagged, __reduce_min_sync(0xffffffffu, at));
      }
      // (A block that nothing has been written to yet, all zeros, has values of zero by any
      // scale: the least there is.)
      const uint32_t scale_v = max(tail.y, static_cast<uint32_t>(127 + kKv8LeastExp) << 23);
      const int e = now_rec >= 0 ? static_cast<int>(scale_v >> 23) : -1;
      most = max(most, __reduce_max_sync(0xffffffffu, e));
      least = min(least, __reduce_min_sync(0xffffffffu, e < 0 ? 255 : e));
      if (lane == 0) reinterpret_cast<volatile int*>(bar->first_flagged)[unit & 15] = flagged;
      const bool wide = most - least >= kWideExps;
      if (now_last) {
        flagged = 0x7fffffff;
        least = 255;
        most = 0;
        ++unit;
      }
      if (lane < kPagesPerTile) {
        // (No block: a V scale whose logarithm leaves nothing of its keys' numerators.)
        reinterpret_cast<float4*>(smem + L::kOffScales)[n % kScaleTiles * 8 + lane] =
            make_float4(now_rec >= 0 ? __uint_as_float(tail.x) * p.scale_log2 : 1.f,
                        now_rec >= 0 ? static_cast<float>(e - 127) : -INFINITY,
                        now_rec >= 0 ? kv8_inverse(scale_v) : 1.f, wide ? 1.f : 0.f);
      }
      __syncwarp();                              // (lanes 0 and 1 release what all of them have stored)
      const int kind = now_rec < 0 ? kRawNone : now_ends || bits != 0 ? kRawCareful : kRawCodes;
      // Two blocks at a time.
      for (int first = 0; ok && first < kPagesPerTile; first += 2) {
        const int i = first + (lane & 1);
        const int rec = __shfl_sync(0xffffffffu, now_rec, i), what = __shfl_sync(0xffffffffu, kind, i);
        if (lane < 2) ok = fill(n * kPagesPerTile + i, rec, what);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      now_rec = next_rec;
      now_number = next_number;
      now_last = next_last;
      now_ends = next_ends;
      tail = next_tail;
    }
    // The end, for both gather warps; then the next kernel in the stream may set up.
    if (ok && lane < 2) ok = fill(n * kPagesPerTile + lane, -1, kRawEnd);
    ok = __all_sync(0xffffffffu, ok);
    pdl_launch_dependents();
    __syncwarp();
    if (!ok) {
      // Raw blocks in flight must land before the CTA may exit.
      for (int s = 0; s < L::kRawStages; ++s) {
        const int fills = bar->raw_fills[s];
        if (fills) mbar_wait_warp_drain(smem_addr(&bar->raw_full[s]), (fills - 1) & 1, wc);
      }
    }
  } else if (!KV8 && warp == kWarpLoad) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
      int kv_issued = 0, k_issued = 0, v_issued = 0, units = 0;
      bool ok = true;
      for (int band = 0; ok; ++band) {
        const int k = unit_at(band);
        if (k >= p.num_units) break;
        const Unit u = unit_info(k);
        // Q tile x of this unit, once the last S MMA of the previous unit has
        // read it.  Order: Q_A, K_0, Q_B, V_0, K_1, ...: the first S MMA of
        // the unit needs only Q_A and K_0, which can land while the previous
        // unit's last tile-B MMAs still read Q_B.
        auto load_q = [&](int x) {
          if (units > 0 && !(ok = mbar_wait(smem_addr(&bar->q_empty[x]), (units - 1) & 1, wc))) return;
          const uint32_t qf = smem_addr(&bar->q_full[x]);
          mbar_arrive_expect_tx(qf, L::kQTile);
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_3d(sQ + x * L::kQTile + c * L::kQChunk, &tq, qf, c * 64,
                        u.qblk * kRowsPerCta + x * kBM, u.zq);
        };
        load_q(0);
        if constexpr (PAGED) {                     // K/V come from the gather warps
          if (ok) load_q(1);
        }
        // K/V tiles: one stage ring for the whole CTA, across units.
        for (int j = 0; j < (PAGED ? 0 : u.nB) && ok; ++j) {
          const int g = kv_issued + j;
          const int st = g % L::kStages;
          const uint32_t ph = (g / L::kStages) & 1;
          auto load_kv = [&](uint32_t dst, const CUtensorMap* map, uint32_t full) {
            mbar_arrive_expect_tx(full, L::kKV);
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(dst + c * L::kKVChunk, map, full, c * 64, j * kBN, u.zkv);
          };
          if (!(ok = mbar_wait(smem_addr(&bar->k_empty[st]), ph ^ 1, wc))) break;
          load_kv(sK + st * L::kKV, &tk, smem_addr(&bar->k_full[st]));
          ++k_issued;
          if (j == 0) {
            load_q(1);
            if (!ok) break;
          }
          if (!(ok = mbar_wait(smem_addr(&bar->v_empty[st]), ph ^ 1, wc))) break;
          load_kv(sV + st * L::kVStage, &tv, smem_addr(&bar->v_full[st]));
          ++v_issued;
        }
        kv_issued += u.nB;
        ++units;
      }
      // Every load is issued: the next kernel in the stream may start
      // setting up on SMs this grid leaves (it waits for this grid to
      // finish before it touches memory).
      pdl_launch_dependents();
      // Every copy issued must have landed before the CTA may exit.
      if (units > 0)
        for (int x = 0; x < kTiles; ++x) mbar_wait(smem_addr(&bar->q_full[x]), (units - 1) & 1, wc, true);
      for (int st = 0; st < L::kStages; ++st) {
        const int nk = k_issued > st ? (k_issued - 1 - st) / L::kStages + 1 : 0;
        const int nv = v_issued > st ? (v_issued - 1 - st) / L::kStages + 1 : 0;
        if (nk) mbar_wait(smem_addr(&bar->k_full[st]), (nk - 1) & 1, wc, true);
        if (nv) mbar_wait(smem_addr(&bar->v_full[st]), (nv - 1) & 1, wc, true);
      }
    }
  } else if (warp == kWarpMma) {
    // --------------------------------------------------------- MMA issuer
    {
      constexpr uint32_t kFp16 = KV8 ? ~((1u << 7) | (1u << 10)) : ~0u;    // A and B formats: fp16 is 0
      constexpr uint32_t kIdescS = idesc_bf16_f32(kBM, kBN, false) & kFp16;
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, L::kNPV, true) & kFp16;
      constexpr int kSteps = D / 16;               // MMAs in an S group (K = d)
      constexpr int kPSteps = kBN / 16;            // MMAs in a PV group (K = keys)
      const uint32_t kF = smem_addr(&bar->k_full[0]);
      const uint32_t vF = smem_addr(&bar->v_full[0]);
      const uint32_t pF = smem_addr(&bar->p_full[0]);
      // K/V tile jj of the current unit is fill g0 + jj of the CTA's stage ring.
      int g0 = 0;
      auto kfull = [&](int jj) { return kF + 8u * ((g0 + jj) % L::kStages); };
      auto vfull = [&](int jj) { return vF + 8u * ((g0 + jj) % L::kStages); };
      auto ph = [&](int jj) { return static_cast<uint32_t>(((g0 + jj) / L::kStages) & 1); };
      // P_X(jj) of the current unit is completion pX0 + jj of p_full[X].
      int pa0 = 0, pb0 = 0;
      auto ppar = [&](int x, int jj) { return static_cast<uint32_t>(((x ? pb0 : pa0) + jj) & 1); };
      // A dependency that was probed ready is not waited on again.
      auto ensure = [&](uint32_t b, uint32_t parity, uint32_t probed) -> bool {
        return __all_sync(0xffffffffu, probed != 0u) || mbar_wait_warp(b, parity, wc);
      };
      // Next group's probes: issued before the last two MMAs of a group.
      uint32_t rA = 0, rB = 0;
      int probe_kind = 0, probe_x = 0, probe_j = 0;   // 1: PV (P, V)  2: S (K)
      auto do_probes = [&]() {
        if (probe_kind == 1) {
          rA = mbar_probe(pF + 8u * static_cast<uint32_t>(probe_x), ppar(probe_x, probe_j));
          rB = mbar_probe(vfull(probe_j), ph(probe_j));
        } else if (probe_kind == 2) {
          rA = mbar_probe(kfull(probe_j), ph(probe_j));
        }
      };
      auto group_s = [&](int x, int jj) {
        const int st = (g0 + jj) % L::kStages;
        const uint32_t qbase = sQ + x * L::kQTile;
        const uint32_t kbase = sK + st * L::kKV;
        const uint32_t dS = tmem + (x ? L::kColS1 : L::kColS0);
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          if (kk == kSteps - 2) do_probes();
          const uint64_t ad = sdesc_sw128(qbase + (kk >> 2) * L::kQChunk + (kk & 3) * 32, 16, 1024);
          const uint64_t bd = sdesc_sw128(kbase + (kk >> 2) * L::kKVChunk + (kk & 3) * 32, 16, 1024);
          umma_ss_warp(dS, ad, bd, kIdescS, kk > 0 ? 1u : 0u);
        }
        umma_commit_warp(smem_addr(&bar->s_full[x]));
      };
      auto group_pv = [&](int x, int jj) {
        const int st = (g0 + jj) % L::kStages;
        const uint32_t vbase = sV + st * L::kVStage;
        const uint32_t aP = tmem + (x ? L::kColS1 : L::kColS0);
        const uint32_t dO = tmem + (x ? L::kColO1 : L::kColO0);
#pragma unroll
        for (int kk = 0; kk < kPSteps; ++kk) {
          if (kk == kPSteps - 2) do_probes();
          // A = P from TMEM (8 columns = 16 keys per step), B = V (MN-major).
          const uint64_t bd = sdesc_sw128(vbase + kk * 2048, L::kKVChunk, 1024);
          umma_ts_warp(dO, aP + kk * 8, bd, kIdescPV, (jj > 0 || kk > 0) ? 1u : 0u);
        }
      };
      // Per unit (each group probes what the next one needs):
      //   S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) | ...
      // The first P V of a tile overwrites O_X, so it waits until the
      // epilogue of the previous unit has read O_X out; the last S group of
      // a tile releases its Q tile for the next unit's load.
      bool ok = true;
      int units = 0;
      for (int band = 0; ok; ++band) {
        const int k = unit_at(band);
        if (k >= p.num_units) break;
        const Unit u = unit_info(k);
        const int nA = u.nA, nB = u.nB;
        const uint32_t upar = static_cast<uint32_t>(units & 1);
        uint64_t* const q_there = KV8 ? bar->q_ready : bar->q_full;
        ok = mbar_wait_warp(smem_addr(&q_there[0]), upar, wc) &&
             mbar_wait_warp(kfull(0), ph(0), wc);
        if (ok) {
          tc_fence_after();
          probe_kind = 0;
          group_s(0, 0);
          if (nA == 1) umma_commit_warp(smem_addr(&bar->q_empty[0]));
          ok = mbar_wait_warp(smem_addr(&q_there[1]), upar, wc);
        }
        if (ok) {
          tc_fence_after();
          probe_kind = 1;                          // PV_A(0): P_A(0), V_0
          probe_x = 0;
          probe_j = 0;
          group_s(1, 0);
          if (nB == 1) umma_commit_warp(smem_addr(&bar->q_empty[1]));
          umma_commit_warp(smem_addr(&bar->k_empty[g0 % L::kStages]));
        }
        for (int j = 0; j < nB && ok; ++j) {
          const int st = (g0 + j) % L::kStages;
          if (j < nA) {
            // PV_A(j)
            if (!(ok = ensure(pF, ppar(0, j), rA) && ensure(vfull(j), ph(j), rB))) break;
            if (j == 0 && units > 0 && !(ok = mbar_wait_warp(smem_addr(&bar->o_free[0]), upar ^ 1, wc))) break;
            tc_fence_after();
            probe_kind = (j + 1 < nA) ? 2 : 0;     // S_A(j+1): K_{j+1}
            probe_j = j + 1;
            group_pv(0, j);
            if (j == nA - 1) umma_commit_warp(smem_addr(&bar->o_done[0]));
            if (j + 1 < nA) {
              // S_A(j+1)
              if (!(ok = ensure(kfull(j + 1), ph(j + 1), rA))) break;
              tc_fence_after();
              probe_kind = 1;                      // PV_B(j): P_B(j), V_j (known)
              probe_x = 1;
              probe_j = j;
              group_s(0, j + 1);
              if (j + 1 == nA - 1) umma_commit_warp(smem_addr(&bar->q_empty[0]));
              rB = 1;
            } else {
              rA = mbar_probe(pF + 8u, ppar(1, j));
              rB = 1;
            }
          } else {
            rA = mbar_probe(pF + 8u, ppar(1, j));
            rB = mbar_probe(vfull(j), ph(j));
          }
          // PV_B(j)
          if (!(ok = ensure(pF + 8u, ppar(1, j), rA) && ensure(vfull(j), ph(j), rB))) break;
          if (j == 0 && units > 0 && !(ok = mbar_wait_warp(smem_addr(&bar->o_free[1]), upar ^ 1, wc))) break;
          tc_fence_after();
          probe_kind = (j + 1 < nB && j + 1 >= nA) ? 2 : 0;   // S_B(j+1) needs K_{j+1} if S_A did not test it
          probe_j = j + 1;
          group_pv(1, j);
          umma_commit_warp(smem_addr(&bar->v_empty[st]));
          if (j == nB - 1) umma_commit_warp(smem_addr(&bar->o_done[1]));
          if (j + 1 < nB) {
            // S_B(j+1)
            if (j + 1 >= nA && !(ok = ensure(kfull(j + 1), ph(j + 1), rA))) break;
            tc_fence_after();
            probe_kind = (j + 1 < nA) ? 1 : 0;     // PV_A(j+1): P_A(j+1), V_{j+1}
            probe_x = 0;
            probe_j = j + 1;
            group_s(1, j + 1);
            if (j + 1 == nB - 1) umma_commit_warp(smem_addr(&bar->q_empty[1]));
            umma_commit_warp(smem_addr(&bar->k_empty[(g0 + j + 1) % L::kStages]));
          }
        }
        g0 += nB;
        pa0 += nA;
        pb0 += nB;
        ++units;
        probe_kind = 0;
        rA = rB = 0;
      }
      // All issued MMAs must retire before TMEM is released.
      umma_commit_warp(smem_addr(&bar->mma_final));
      __all_sync(0xffffffffu, mbar_wait(smem_addr(&bar->mma_final), 0, wc, true));
    }
  }
  if constexpr (KV8) {
    if (warp == kWarpGatherK || warp == kWarpGatherV) {
      // -------------------------------------- raw blocks into fp16 K / V tiles
      const int op = warp - kWarpGatherK;                      // 0: K, 1: V
      const uint32_t raw = smem_addr(smem + L::kOffRaw) + op * L::kRawHalf;
      const uint32_t full = smem_addr(&bar->raw_full[0]), empty = smem_addr(&bar->raw_empty[0]);
      const volatile int* kinds = bar->raw_kind;
      const uint32_t tile0 = op ? sV : sK;
      const uint32_t tile_full = smem_addr(op ? &bar->v_full[0] : &bar->k_full[0]);
      const uint32_t tile_empty = smem_addr(op ? &bar->v_empty[0] : &bar->k_empty[0]);
      constexpr int kPieces = 2 * (D / 64);                    // of 16 codes: rows r, r + 8, columns c (, c + 4)
      // 16 codes of a lane: those of 8 neighbouring lanes are the same columns of 8
      // rows, which the swizzles spread over all banks, here and in the tile.
      const int r = lane & 7, c = lane >> 3;
      const uint32_t raw_at = D == 128 ? 128 * r + 16 * (c ^ r) : 128 * (r >> 1) + 16 * ((4 * (r & 1) + c) ^ (r >> 1));
      // As fp16, 16-byte columns 2 c and 2 c + 1 of a 128-byte row.
      const uint32_t dst_at = 128 * r + 16 * ((2 * c) ^ r);
      auto raw_of = [&](int x) {
        if constexpr (D == 128) return (raw_at ^ (64u * (x & 1))) + 1024u * (x >> 1);
        return x ? (raw_at ^ 64u) + 512u : raw_at;             // (4 lines on)
      };
      auto dst_of = [&](int x) {
        return D == 128 ? dst_at + L::kKVChunk * (x & 1) + 1024u * (x >> 1) : dst_at + 1024u * x;
      };
      bool ok = true;
      int s = 0;                                               // raw stage and its barrier's phase
      uint32_t phase = 0;
      for (int g = 0; ok; ++g) {
        const int st = g % L::kStages;
        bool end = false;
#pragma unroll 1
        for (int i = 0; i < kPagesPerTile; i += 2) {
          if (!(ok = mbar_wait_warp(full + 8u * s, phase, wc))) break;
          if (!(ok = mbar_wait_warp(full + 8u * (s + 1), phase, wc))) break;
          const int kind[2] = {kinds[s], kinds[s + 1]};
          if (kind[0] == kRawEnd) {
            end = true;
            break;
          }
          uint4 w[2 * kPieces];
#pragma unroll
          for (int x = 0; x < 2 * kPieces; ++x) w[x] = ld_shared_v4(raw + (s + x / kPieces) * L::kRaw + raw_of(x % kPieces));
          if (i == 0 && !(ok = mbar_wait_warp(tile_empty + 8u * st, ((g / L::kStages) & 1) ^ 1, wc))) break;
          if (kind[0] != kRawCodes || kind[1] != kRawCodes) {  // (the same for the whole warp)
#pragma unroll
            for (int x = 0; x < 2 * kPieces; ++x)
              w[x] = kind[x / kPieces] == kRawNone
                         ? make_uint4(0u, 0u, 0u, 0u)
                         : make_uint4(without_nan(w[x].x), without_nan(w[x].y), without_nan(w[x].z), without_nan(w[x].w));
          }
          const uint32_t dst = tile0 + st * L::kKV + i * (kPageRows * 128);
#pragma unroll
          for (int x = 0; x < 2 * kPieces; ++x) {
            const uint32_t to = dst + x / kPieces * (kPageRows * 128);
            st_shared_v4(to + dst_of(x % kPieces), e4m3x2_to_f16x2(w[x].x), e4m3x2_hi_to_f16x2(w[x].x),
                         e4m3x2_to_f16x2(w[x].y), e4m3x2_hi_to_f16x2(w[x].y));
            st_shared_v4(to + (dst_of(x % kPieces) ^ 16u), e4m3x2_to_f16x2(w[x].z), e4m3x2_hi_to_f16x2(w[x].z),
                         e4m3x2_to_f16x2(w[x].w), e4m3x2_hi_to_f16x2(w[x].w));
          }
          __syncwarp();                                        // every lane has read the raw blocks
          if (lane < 2) mbar_arrive(empty + 8u * (s + lane));
          if ((s += 2) == L::kRawStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok || end) break;
        fence_proxy_async_smem();
        mbar_arrive(tile_full + 8u * st);
      }
    }
  } else if constexpr (PAGED) {
    if (warp == kWarpGatherK || warp == kWarpGatherV) {
      // ------------------------------------------------- paged K / V gather
      const bool is_v = warp == kWarpGatherV;
      const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
      const uint32_t s_base = is_v ? sV : sK;
      const uint32_t full0 = smem_addr(is_v ? &bar->v_full[0] : &bar->k_full[0]);
      const uint32_t empty0 = smem_addr(is_v ? &bar->v_empty[0] : &bar->k_empty[0]);
      constexpr int kRowPieces = D / 8;                        // 16-byte pieces of one key row
      constexpr int kPerLane = kPageRows * kRowPieces / 32;    // pieces of one block per lane
      const size_t slice_bytes = static_cast<size_t>(kPageRows) * D * 2;
      int g = 0;                                               // fill index of the stage ring
      bool ok = true;
      for (int band = 0; ok; ++band) {
        const int k = unit_at(band);
        if (k >= p.num_units) break;
        const Unit u = unit_info(k);
        const int* row = p.block_table + static_cast<size_t>(u.b) * p.max_blocks;
        for (int j = 0; j < u.nB; ++j, ++g) {
          // Lane i < 8 translates block i of the tile (before the wait, so the
          // lookup overlaps it); p.num_blocks stands for "no block": zeros.
          int e = p.num_blocks;
          const int lb = j * kPagesPerTile + lane;
          if (lane < kPagesPerTile && lb < u.nblk) {
            e = __ldg(row + lb);
            if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.num_blocks)) {
              atomicOr(p.status, kDevBadBlock);                // reported, read as zeros
              e = p.num_blocks;
            }
          }
          const int st = g % L::kStages;
          if (!(ok = mbar_wait_warp(empty0 + 8u * st, ((g / L::kStages) & 1) ^ 1, wc))) break;
          const uint32_t dst0 = s_base + st * L::kKV;
#pragma unroll 1
          for (int i = 0; i < kPagesPerTile; ++i) {
            const int phys = __shfl_sync(0xffffffffu, e, i);
            const bool valid = phys < p.num_blocks;
            const uint8_t* src0 = cache + (static_cast<size_t>(valid ? phys : 0) * p.Hkv + u.kvh) * slice_bytes;
#pragma unroll
            for (int t = 0; t < kPerLane; ++t) {
              const int piece = t * 32 + lane;                 // consecutive lanes: consecutive 16 B
              const int slot = piece / kRowPieces;
              const int col = piece % kRowPieces;
              // 128-byte swizzle: 16-byte column (col & 7) of row r sits at (col & 7) ^ (r & 7).
              const uint32_t dst = dst0 + (col >> 3) * L::kKVChunk + (i * kPageRows + slot) * 128 +
                                   ((static_cast<uint32_t>((col & 7) ^ (slot & 7))) << 4);
              cp_async16(dst, src0 + piece * 16, valid ? 16u : 0u);
            }
          }
          cp_async_wait_all();
          fence_proxy_async_smem();
          mbar_arrive(full0 + 8u * st);
        }
      }
    }
  }
    // Each role ends on the same named barrier, so the register-split
    // branches never merge back; then the MMA warp frees the TMEM.
    tc_fence_before();
    named_barrier_sync(1, kThreads);
    if (warp == kWarpMma) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
  } else {
    regs_increase<regs_softmax(KV8, D)>();
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;                       // query tile of this warpgroup
    const int quarter = warp & 3;                  // TMEM lane quarter of this warp
    const int row = quarter * 32 + lane;           // row within the tile = TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t colS = x ? L::kColS1 : L::kColS0;
    const uint32_t colO = x ? L::kColO1 : L::kColO0;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int sx0 = 0;                                   // S_X tiles consumed in earlier units
    int kv0 = 0;                                   // K/V tiles of earlier units
    // 8-bit cache: each softmax warpgroup loads its Q tile (its first thread, as soon
    // as the last S of the unit before is there), and each thread turns its row into
    // fp16 in place.
    const uint32_t q_tile = sQ + x * L::kQTile, q_full = smem_addr(&bar->q_full[x]);
    auto load_q = [&](int band) {
      const int k = unit_at(band);
      if (quarter != 0 || lane != 0 || k >= p.num_units) return;
      const Unit u = unit_info(k);
      ++bar->q_loads[x];
      mbar_arrive_expect_tx(q_full, L::kQTile);
      for (int c = 0; c < L::kChunks; ++c)
        tma_load_3d(q_tile + c * L::kQChunk, &tq, q_full, c * 64, u.qblk * kRowsPerCta + x * kBM, u.zq);
    };
    // Returns what undoes the row's scaling.
    auto turn_q = [&]() {
      auto piece = [&](int i) { return q_tile + (i >> 3) * L::kQChunk + row * 128 + (((i & 7) ^ (row & 7)) << 4); };
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = ld_shared_v4(piece(i));
        mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu),
                      __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      }
      mx = max(mx & 0xffffu, mx >> 16);
      // Largest element in [2^(E-127), 2^(E-126)); times 2^(141-E) it is in
      // [2^14, 2^15).
      const int fe = min(268 - static_cast<int>(mx >> 7), 253);
      const float up = __uint_as_float(static_cast<uint32_t>(fe) << 23);
      auto turn = [&](uint32_t w) {
        return pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
      };
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = ld_shared_v4(piece(i));
        st_shared_v4(piece(i), turn(v.x), turn(v.y), turn(v.z), turn(v.w));
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_addr(&bar->q_ready[x]));
      return __uint_as_float(static_cast<uint32_t>(254 - fe) << 23);
    };
    if constexpr (KV8) load_q(0);
    int units = 0;
    for (int band = 0; ok; ++band) {
    const int k = unit_at(band);
    if (k >= p.num_units) break;
    const Unit u = unit_info(k);
    const int qrow = u.qblk * kRowsPerCta + x * kBM + row;
    const int n_kv = x ? u.nB : u.nA;
    const int diag = 2 * u.qblk + x;               // causal: the tile holding key == row
    // Paged: position of this row's token, and the lowest of the tile's rows'.
    const int qpos = u.pos0 + (KV8 ? qrow % p.rows : qrow);
    const int first = u.qblk * kRowsPerCta + x * kBM;
    const int qpos_first = u.pos0 + (!KV8 || !p.packed ? first : first % p.rows + kBM <= p.rows ? first % p.rows : 0);
    const int zq = u.zq;
    float m = 0.f;                                 // stabiliser in use (exp2 domain)
    float l = 0.f;                                 // denominator relative to m (fp32 terms)
    float lr = 0.f;                                // same, bf16-rounded terms
    float back = 1.f;                              // 8-bit cache: the factor of this row of Q
    if constexpr (KV8) {
      if (!mbar_wait_warp(q_full, units & 1, wc)) {
        ok = false;
        break;
      }
      back = turn_q();
    }

    for (int j = 0; j < n_kv; ++j) {
      if (!mbar_wait_warp(smem_addr(&bar->s_full[x]), static_cast<uint32_t>(sx0 + j) & 1u, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if constexpr (KV8) {
        if (j == n_kv - 1) load_q(band + 1);       // (Q has been read for the last time)
      }
      uint32_t r0[32], r1[32], r2[32], r3[32];
      ATTN47_TMEM_LD32(tl + colS + 0, r0);
      ATTN47_TMEM_LD32(tl + colS + 32, r1);
      ATTN47_TMEM_LD32(tl + colS + 64, r2);
      ATTN47_TMEM_LD32(tl + colS + 96, r3);
      ATTN47_TMEM_LD_WAIT(r0);
      ATTN47_TMEM_LD_WAIT(r1);
      ATTN47_TMEM_LD_WAIT(r2);
      ATTN47_TMEM_LD_WAIT(r3);

      float s[128];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        s[c] = __uint_as_float(r0[c]);
        s[32 + c] = __uint_as_float(r1[c]);
        s[64 + c] = __uint_as_float(r2[c]);
        s[96 + c] = __uint_as_float(r3[c]);
      }
      const int kbase = j * kBN;
      const bool need_mask = PAGED ? (kbase + kBN - 1 > qpos_first)
                                   : CAUSAL ? (j == diag) : (kbase + kBN > p.N);
      if (need_mask) {
#pragma unroll
        for (int c = 0; c < 128; ++c) {
          const int key = kbase + c;
          const bool masked = PAGED ? (key > qpos) : CAUSAL ? (key > qrow) : (key >= p.N);
          s[c] = masked ? -INFINITY : s[c];
        }
      }
      // 8-bit cache: a block's scales (see kOffScales) and its scores' factor
      // (never 0, which the -inf of masked keys would make NaN).
      auto scales = [&](int blk) {
        return reinterpret_cast<const float4*>(smem + L::kOffScales)[(kv0 + j) % kScaleTiles * 8 + blk];
      };
      auto factor = [&](const float4& w) { return fmaxf(w.x * back, 1e-37f); };
      // Row maximum: a depth-5 tree of three-input maxima.  (8-bit cache: of the
      // exponents of P'.)
      auto row_max = [&]() {
        if constexpr (KV8) {
          float mx = -INFINITY;
#pragma unroll
          for (int blk = 0; blk < 8; ++blk) {
            const float* y = s + 16 * blk;
            const float a = fmax3(fmax3(y[0], y[1], y[2]), fmax3(y[3], y[4], y[5]), fmax3(y[6], y[7], y[8]));
            const float b = fmax3(fmax3(y[9], y[10], y[11]), fmax3(y[12], y[13], y[14]), y[15]);
            const float4 w = scales(blk);
            mx = fmaxf(mx, fmaf(fmaxf(a, b), factor(w), w.y));
          }
          return mx;
        }
        float t[43], u[15];
#pragma unroll
        for (int i = 0; i < 42; ++i) t[i] = fmax3(s[3 * i], s[3 * i + 1], s[3 * i + 2]);
        t[42] = fmaxf(s[126], s[127]);
#pragma unroll
        for (int i = 0; i < 14; ++i) u[i] = fmax3(t[3 * i], t[3 * i + 1], t[3 * i + 2]);
        u[14] = t[42];
        return fmaxf(fmax3(fmax3(u[0], u[1], u[2]), fmax3(u[3], u[4], u[5]), fmax3(u[6], u[7], u[8])),
                     fmax3(fmax3(u[9], u[10], u[11]), u[12], fmaxf(u[13], u[14])));
      };
      // Numerators p = 2^(s * scale * log2 e - m), two lanes per instruction
      // for the scale and the sums.  Two denominators: `lr` sums the
      // bf16-rounded numerators that P V uses, so O / lr weights every value
      // row by exactly the factor it got (with SUMV the tensor core forms
      // this sum in column d of O_X and the loop leaves it out); `l` sums the
      // fp32 numerators and gives the LSE.  P_X goes over the first 64
      // columns of S_X (keys 2c, 2c+1 in column c), the first half while the
      // second is computed.
      float lt, lrt;                               // this tile's two sums (8-bit cache: lrt is that of P')
      auto numerators = [&]() {
        if constexpr (KV8) {
          lt = lrt = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int blk = 0; blk < 4; ++blk) {
              const float4 w = scales(half * 4 + blk);
              const float a = factor(w), b = w.y - m;
              const uint64_t sc2 = f2_pack(a, a), add2 = f2_pack(b, b);
              uint64_t acc[2] = {0, 0};
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const int i = half * 64 + blk * 16 + 2 * c;
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(s[i], s[i + 1]), sc2, add2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                acc[c & 1] = f2_add(acc[c & 1], f2_pack(p0, p1));
                pk[blk * 8 + c] = pack_f16x2(p0, p1);
              }
              float e0, e1;
              f2_unpack(f2_add(acc[0], acc[1]), e0, e1);
              const float sum = e0 + e1;
              lrt += sum;
              lt = fmaf(sum, w.z, lt);
            }
            ATTN47_TMEM_ST32(tl + colS + half * 32, pk);
          }
          return;
        }
        const uint64_t sc2 = f2_pack(sl2, sl2);
        const uint64_t nm2 = f2_pack(-m, -m);
        uint64_t accE[4] = {0, 0, 0, 0};
        float accR[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int e = half * 64 + 2 * c;
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), sc2, nm2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            const uint32_t w = pack_bf16x2(p0, p1);
            accE[c & 3] = f2_add(accE[c & 3], f2_pack(p0, p1));
            if constexpr (!SUMV) {
              accR[(c & 1) * 2] = add_bf16lo_f32(w, accR[(c & 1) * 2]);
              accR[(c & 1) * 2 + 1] = add_bf16hi_f32(w, accR[(c & 1) * 2 + 1]);
            }
            pk[c] = w;
          }
          ATTN47_TMEM_ST32(tl + colS + half * 32, pk);
        }
        float e0, e1;
        f2_unpack(f2_add(f2_add(accE[0], accE[1]), f2_add(accE[2], accE[3])), e0, e1);
        lt = e0 + e1;
        lrt = (accR[0] + accR[1]) + (accR[2] + accR[3]);
      };
      // Moves the stabiliser to the tile's maximum where that exceeds it by
      // more than kTau, rescaling the sums and O_X (which holds PV_X(0..j-1),
      // complete since S_X(j) completed after it).
      auto restabilise = [&](float mt) {
        const bool need = mt > m + (KV8 ? 0.f : kTau);
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mt : m;
          const float alpha = ex2(m - m_new);
          l *= alpha;
          lr *= alpha;
          m = m_new;
          const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
          for (int c0 = 0; c0 < (SUMV ? D + 32 : D); c0 += 32) {   // SUMV: the row sums too
            uint32_t o[32];
            ATTN47_TMEM_LD32(tl + colO + c0, o);
            ATTN47_TMEM_LD_WAIT(o);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float lo, hi;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1])), a2),
                        lo, hi);
              o[2 * c] = __float_as_uint(lo);
              o[2 * c + 1] = __float_as_uint(hi);
            }
            ATTN47_TMEM_ST32(tl + colO + c0, o);
          }
        }
      };
      // The stabiliser only has to keep the numerators finite (fp32 and
      // bf16 reach 2^127), so after the first tile the tile's maximum is not
      // formed up front: the numerators are computed with the current m, and
      // only a tile whose fp32 sum exceeds 2^100 (or is not finite) is redone
      // with the stabiliser moved to its maximum.  Same function, same
      // rounding.  One call site, so the unrolled loop is emitted once.
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (j == 0 || pass == 1) {                 // the tile's maximum is needed
          const float mt = KV8 ? row_max() - kHigh8 : row_max() * sl2;
          if (j == 0)
            m = (mt == -INFINITY) ? (KV8 ? kNoKeys : 0.f) : mt;   // (8-bit cache: keys may come in a later tile)
          else
            restabilise(mt);
        }
        numerators();
        if (j == 0 || pass == 1) break;
        const bool big = !(KV8 ? lrt <= 65504.f : lt <= 0x1p100f);   // (P' has to fit in fp16)
        if (!__any_sync(0xffffffffu, big)) break;
      }
      l += lt;
      lr += lrt;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bar->p_full[x]));
    }

    // ------------------------------------------------------------ epilogue
    ok = __all_sync(0xffffffffu, ok);
    if (ok && mbar_wait_warp(smem_addr(&bar->o_done[x]), static_cast<uint32_t>(units & 1), wc)) {
      tc_fence_after();
      float lsum = KV8 ? l : lr;
      if constexpr (SUMV) {
        uint32_t rs[32];
        ATTN47_TMEM_LD32(tl + colO + D, rs);
        ATTN47_TMEM_LD_WAIT(rs);
        lsum = __uint_as_float(rs[0]);
      }
      float inv_l = 1.f / lsum;
      bool spoilt = false;
      if constexpr (KV8) {
        // (The look-up stored this, as of this query tile's last K/V tile at least,
        // before that tile's blocks were on their way; later ones are seen by no row.)
        spoilt = qpos >= reinterpret_cast<const volatile int*>(bar->first_flagged)[units & 15];
        // Scores that mean nothing any more: what lies in rows that are not in use, too.
        spoilt |= fabsf(m) >= 0x1p40f && m != kNoKeys;
        if (lsum == 0.f) inv_l = 0.f;              // a row that sees nothing
        if (spoilt) inv_l = __uint_as_float(0x7fc00000u);
      }
      bool again = false;
      if constexpr (KV8) {
        // (As of the query tile's last K/V tile: whatever the look-up has met since.)
        const float4* last = reinterpret_cast<const float4*>(smem + L::kOffScales) + (kv0 + n_kv - 1) % kScaleTiles * 8;
        again = (l < 0x1p-8f && last->w != 0.f) || (fabsf(m) >= 0x1p26f && m != kNoKeys);
      }
      const bool in_range = qrow < p.N;
      __nv_bfloat16* orow =
          reinterpret_cast<__nv_bfloat16*>(p.o) + (static_cast<size_t>(zq) * p.N + qrow) * D;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        ATTN47_TMEM_LD32(tl + colO + c0, o);
        ATTN47_TMEM_LD_WAIT(o);
        if constexpr (KV8) again |= !(fabsf(__uint_as_float(o[0])) <= 3.402823466e38f);
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c)
          w[c] = pack_bf16x2(__uint_as_float(o[2 * c]) * inv_l, __uint_as_float(o[2 * c + 1]) * inv_l);
        if (in_range) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dst[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
      }
      if (in_range && p.lse != nullptr)
        p.lse[static_cast<size_t>(zq) * p.N + qrow] =
            KV8 && spoilt ? __uint_as_float(0x7fc00000u) : (m + __log2f(l)) * kLn2;
      if constexpr (KV8) {
        // (A query that is not finite itself has back = 2^114, and NaN.)
        again = again && qpos >= 0 && in_range && !spoilt && back < 0x1p114f;
        if (__any_sync(0xffffffffu, again) && lane == 0) {
          const int at = min(band, kAgain - 1);
          bar->again[warp][at / 32] |= 1u << (at % 32);
        }
      }
      // O_X has been read out: the next unit's first P V may overwrite it.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bar->o_free[x]));
    } else {
      ok = false;
    }
    sx0 += n_kv;
    kv0 += u.nB;
    ++units;
    }
    if constexpr (KV8) {
      __syncwarp();
      for (int w = 0; w < kAgain / 32 && ok; ++w)
        for (unsigned todo = bar->again[warp][w]; todo != 0; todo &= todo - 1) {
          const int first = 32 * w + __ffs(todo) - 1;
          for (int band = first; unit_at(band) < p.num_units && (band == first || first == kAgain - 1); ++band) {
            const Unit u = unit_info(unit_at(band));
            const int qrow = u.qblk * kRowsPerCta + x * kBM + row;
            const size_t at = static_cast<size_t>(u.zq) * p.N + qrow;
            const int qpos = qrow < p.N ? max(u.pos0 + qrow % p.rows, -1) : -1;
            careful_rows<D>(p.kv_cache, p.block_table + static_cast<size_t>(u.b) * p.max_blocks, p.num_blocks, p.Hkv, u.kvh,
                            p.scale_log2, qpos, p.q + at * D, static_cast<__nv_bfloat16*>(p.o) + at * D,
                            p.lse != nullptr ? p.lse + at : nullptr);
          }
        }
      // After a wait that ran out: the last copy of Q (this unit's, or already the
      // next one's) must land before the CTA may exit.
      if (!ok && quarter == 0 && lane == 0) {
        const int loads = bar->q_loads[x];
        if (loads > 0) mbar_wait(q_full, (loads - 1) & 1, wc, true);
      }
    }
    tc_fence_before();
    named_barrier_sync(1, kThreads);
  }
}

template <int D, bool CAUSAL, int SOURCE, bool SORTED = false>
cudaError_t launch_t(const FwdLaunch& a) {
  constexpr bool PAGED = SOURCE != kContiguous;
  using L = FwdLayout<D, D == 64 && !PAGED, SOURCE>;
  static_assert(L::kSmem <= 227 * 1024, "shared memory");
  auto kern = attn_fwd_sm103_kernel<D, CAUSAL, SOURCE, SORTED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  FwdParams p;
  p.o = a.o;
  p.lse = a.lse;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.group = a.Hq / a.Hkv;
  p.num_q_blocks = (a.N + kRowsPerCta - 1) / kRowsPerCta;
  p.bh_total = a.B * a.Hq;
  p.num_units = p.num_q_blocks * p.bh_total;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.max_ctx = PAGED ? a.max_blocks * kPageRows - a.N : 0;
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.rows = a.rows;
  p.packed = a.rows != a.N;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  // Persistent: one CTA per SM (shared memory allows one), each walking units.
  const unsigned grid = static_cast<unsigned>(min(p.num_units, a.sms > 0 ? a.sms : 1));
  return launch_pdl(kern, dim3(grid), dim3(kThreads), L::kSmem, a.stream, *a.tq, *a.tk, *a.tv, p);
}

}  // namespace

int fwd_box_rows() { return kBM; }

cudaError_t launch_fwd_sm103(const FwdLaunch& a) {
  if (a.paged) {
    const long long pairs = static_cast<long long>(a.B) * ((a.N + kRowsPerCta - 1) / kRowsPerCta);
    const bool sorted = a.B <= kSortMaxSeqs && pairs <= sort_max_pairs(a.kv_cache != nullptr ? kPagedKv8 : kPagedBf16);
    if (a.kv_cache != nullptr) {
      if (a.d == 128) return sorted ? launch_t<128, true, kPagedKv8, true>(a) : launch_t<128, true, kPagedKv8>(a);
      return sorted ? launch_t<64, true, kPagedKv8, true>(a) : launch_t<64, true, kPagedKv8>(a);
    }
    if (a.d == 128) return sorted ? launch_t<128, true, kPagedBf16, true>(a) : launch_t<128, true, kPagedBf16>(a);
    return sorted ? launch_t<64, true, kPagedBf16, true>(a) : launch_t<64, true, kPagedBf16>(a);
  }
  if (a.d == 128) return a.causal ? launch_t<128, true, kContiguous>(a) : launch_t<128, false, kContiguous>(a);
  return a.causal ? launch_t<64, true, kContiguous>(a) : launch_t<64, false, kContiguous>(a);
}

}  // namespace attn47
