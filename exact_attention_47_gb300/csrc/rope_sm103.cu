// Rotary positions for sm_103a: rotation of queries and keys (and of their
// gradients), the same rotation on the way into a paged cache (bf16 or 4
// bits), and the read-back of 4-bit rows.
//
// Pair p of a head's rotating part turns by the angle a = pos f_p, pos the
// token's position on pair p's axis and f_p its frequency:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a);
// the backward pass is the same map with -a.  cos and sin need a mod 2 pi,
// which fp32 loses at far positions (2^-24 of a million radians is 0.06).
// Here f_p / (2 pi) is a 64-bit binary fraction of a turn and the position
// multiplies it modulo 2^64: whole turns fall off the top exactly, and the
// error is under 2^-33 turns at any 31-bit position (|f_p| <= 1; it grows
// with |f_p| above that).
//
// All of it is data movement with a little arithmetic: a row (one head of
// one token) is held by d/16 lanes, both members of eight pairs each, so a
// warp moves 1 KB a step and keeps several loads in flight.  A warp takes one
// token's rows (all of them when there are many tokens, a slice when there are
// few), so the angles of a token are formed once for all its heads, each by one
// lane of the warp.
//
// Measured (GB300, replayed graphs): 4 x 4096 tokens of 12 + 2 heads, d = 128
// (118 MB) 22.1 us, 5.3 TB/s or 0.79 of a copy; 5001 tokens of 16 + 16 heads, d
// = 64, three axes (41 MB) 10.3 us; an append of 7 ragged chunks (68 MB) 14.5
// us.  About 3 us of each are the launch and its first trip to memory; the rest
// is at the copy rate.  The 4-bit append of 14600 tokens of 16 + 4 heads (158
// MB) takes 37 us: 1640 warp instructions a token, most of them for the
// quantiser, issued in 57% of the cycles (a warp waits for its rows and then
// works through them, in turn).
// Copying rows ahead into a ring in shared memory, over the ends of tokens and
// with equal shares for all warps, was slower (22.4 us instead of 21.5, 17.6
// instead of 14.4): enough loads are in flight already, and each step then waits
// for two more trips inside the SM.  The 4-bit append and its read-back take
// 47 us together; 4-bit rows loaded before the queries are done cost 2 us more,
// and a fourth CTA a SM with its 64 registers gains 0.7 us here and loses 0.25 of
// 5.6 in a decode step.  Equal shares of steps instead of whole tokens change
// nothing (21.5, 10.2, 14.5 and 47.3 us).
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "ptx.cuh"
#include "rope_sm103.h"

namespace attn47 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = kKv4Slots;
enum Mode { kRotate, kAppend, kAppendKv4 };
// Resident CTAs per SM (the register budget follows), and so the size of the
// persistent grids: one CTA more than fits would be a second wave.
constexpr int ctas_per_sm(int mode) { return mode == kAppendKv4 ? 3 : 4; }
constexpr int kReadCtas = 6;

// Rows by strides: those within a batch in units of 8 elements and 32 bits,
// so that a row's address takes one multiplication.
template <class T>
struct Rows {
  T* data;
  long long batch;
  int token, head;
  __device__ __forceinline__ T* of(int b, int t) const {
    return data + b * batch + static_cast<long long>(t) * token * 8;
  }
  static __device__ __forceinline__ T* row(T* token_rows, int r, int head) {
    return token_rows + static_cast<long long>(r) * head * 8;
  }
};
using RowPtr = Rows<const __nv_bfloat16>;
using OutPtr = Rows<__nv_bfloat16>;

struct RopeParams {
  RowPtr q, k, v;
  OutPtr q_out, k_out;
  const float* inv_freq;
  const int* rope_pos;               // nullptr: the cache positions (append)
  long long axis_stride, batch_stride;
  uint32_t pair_axis[4];
  int rot, inverse;
  int Hq, Hk, rows;                  // rows of a token: Hq + Hk (+ Hk values when appending)
  int N;                             // tokens per batch (rotation)
  int parts, rows_per_part;
  long long tasks;                   // tokens * parts
  // append
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  uint8_t* kv_cache;
  const int* block_table;
  const int* seq_ids;
  const int* positions;
  int num_seqs, max_blocks, num_blocks;
  unsigned int* status;
};

// f / (2 pi) mod 1 as a 64-bit fraction (0 for non-finite f, with `bad` set).
__device__ __forceinline__ uint64_t turn_fraction(float f, bool& bad) {
  constexpr uint64_t kInvTwoPi = 2935890503282001226ull;   // round(2^64 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 0xffu);
  bad = ex == 255;
  if (bad) return 0;
  // |f| = m 2^e exactly; f / (2 pi) 2^64 = m kInvTwoPi 2^e, an up to 88-bit
  // product shifted into place.
  const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int e = (ex ? ex : 1) - 150;
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  uint64_t t;
  if (e >= 0)
    t = e < 64 ? lo << e : 0;
  else if (e > -64)
    t = (lo >> -e) | (hi << (64 + e));
  else
    t = e > -128 ? hi >> (-e - 64) : 0;
  return (bits >> 31) ? 0 - t : t;
}

// Sine and cosine of the position's turn, correctly rounded but for one in 200:
// of a key that is quantised, the last bit may decide the code.  The turn less
// whole quarters is at most an eighth; there both are their Taylor series, the
// leading terms in pairs of floats (error-free sums and products, Dekker).
__device__ __forceinline__ void turn_sincos(int pos, uint64_t frac, float& s, float& c) {
  const int64_t t = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * frac);
  const int quarter = static_cast<int>((static_cast<uint64_t>(t) + (1ull << 61)) >> 62);
  const int64_t rem = static_cast<int64_t>(static_cast<uint64_t>(t) - (static_cast<uint64_t>(quarter) << 62));
  // The angle pi (rh + rl), as th + tl.
  constexpr float kPi = 3.14159274101257324f, kPiLow = -8.74227800037e-8f;
  const float rh = static_cast<float>(static_cast<int>(rem >> 40)) * 0x1p-23f;
  const float rl = static_cast<float>(static_cast<int>((rem >> 16) & 0xffffff)) * 0x1p-47f;
  const float a = __fmul_rn(rh, kPi);
  const float b = __fadd_rn(fmaf(rh, kPi, -a), fmaf(rh, kPiLow, __fmul_rn(rl, kPi)));
  const float th = __fadd_rn(a, b), tl = __fsub_rn(b, __fsub_rn(th, a));
  const float zh = __fmul_rn(th, th), zl = fmaf(2.f * th, tl, fmaf(th, th, -zh));
  // cos = 1 - z / 2 + z^2 (1 / 24 - ..)
  const float even = fmaf(fmaf(fmaf(zh, 2.08767570e-9f, -2.75573192e-7f), zh, 2.48015873e-5f), zh, -1.38888889e-3f);
  const float half = 0.5f * zh, ch = __fsub_rn(1.f, half);
  const float cl = __fadd_rn(__fsub_rn(__fsub_rn(1.f, ch), half),
                             fmaf(__fmul_rn(zh, zh), fmaf(even, zh, 4.16666667e-2f), -0.5f * zl));
  const float cosine = __fadd_rn(ch, cl);
  // sin = theta + theta z (-1 / 6 + z (1 / 120 - ..))
  constexpr float kSixth = -0.166666671633720398f, kSixthLow = 4.96705373e-9f;
  const float odd = fmaf(fmaf(fmaf(zh, -2.50521084e-8f, 2.75573192e-6f), zh, -1.98412698e-4f), zh, 8.33333333e-3f);
  const float zq = __fmul_rn(zh, odd), ph = __fadd_rn(kSixth, zq);
  const float pl = __fadd_rn(__fsub_rn(zq, __fsub_rn(ph, kSixth)), kSixthLow);
  const float uh = __fmul_rn(zh, ph), ul = fmaf(zh, pl, fmaf(zl, ph, fmaf(zh, ph, -uh)));
  const float vh = __fmul_rn(th, uh), vl = fmaf(th, ul, fmaf(tl, uh, fmaf(th, uh, -vh)));
  const float sh = __fadd_rn(th, vh), sl = __fsub_rn(vh, __fsub_rn(sh, th));
  const float sine = __fadd_rn(sh, __fadd_rn(sl, __fadd_rn(tl, vl)));
  s = (quarter & 1) ? cosine : sine;
  c = (quarter & 1) ? sine : cosine;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void unpack8(const uint4& x, float (&y)[8]) {
  y[0] = bf_lo(x.x); y[1] = bf_hi(x.x);
  y[2] = bf_lo(x.y); y[3] = bf_hi(x.y);
  y[4] = bf_lo(x.z); y[5] = bf_hi(x.z);
  y[6] = bf_lo(x.w); y[7] = bf_hi(x.w);
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}
// NaN-propagating extremes, of two and (sm_100+) of three.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 1.5 2^23: x + kRound is x rounded to a whole number (half to even), whose
// value lies in the low bits of the sum.
constexpr float kRound = 12582912.f;
constexpr uint32_t kRoundBits = 0x4b400000u;

// 4-bit codes of this lane's 16 elements, as kRoundBits + code, and the
// parameter word of their group (the G/16 lanes of a group agree on it).  low =
// bf16(min), scale = bf16((max - low) (1 / 15)), code = (x - low) / scale rounded
// to even, clamped.  A scale below the smallest normal number counts as 0 (a
// constant group: every value reads back as low); a group whose range is not
// finite gets NaN parameters, so that it reads back as NaN.
template <int G>
__device__ __forceinline__ uint32_t quantise16(const float (&y)[2][8], uint32_t (&code)[2][8]) {
  float lo = y[0][0], hi = lo;
#pragma unroll
  for (int e = 1; e < 15; e += 2) {
    const float a = y[e / 8][e % 8], b = y[(e + 1) / 8][(e + 1) % 8];
    lo = min_nan(lo, a, b);
    hi = max_nan(hi, a, b);
  }
  lo = min_nan(lo, y[1][7]);
  hi = max_nan(hi, y[1][7]);
#pragma unroll
  for (int o = 1; o < G / 16; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t low_bits = pack_bf16x2(lo, 0.f) & 0xffffu;
  lo = __uint_as_float(low_bits << 16);
  const float range = hi - lo;
  const bool finite = fabsf(range) <= 3.402823466e38f;
  uint32_t scale_bits = pack_bf16x2(0.f, __fmul_rn(fmaxf(range, 0.f), 1.f / 15.f)) & 0xffff0000u;
  if (scale_bits < 0x00800000u || !finite) scale_bits = 0;
  const float scale = __uint_as_float(scale_bits);
  // code = t / scale (t the clamped distance from low) rounded to even: the
  // product with an approximate reciprocal, then one step with the remainder,
  // which one fma gives exactly (Markstein's correction of a quotient), so that a
  // half-way quotient is met exactly.  Of a thousand bf16 values a few lie
  // exactly there.
  float inv = 0.f;
  if (scale_bits) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  const float top = 15.f * scale;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = fminf(fmaxf(y[i][e] - lo, 0.f), top);
      const float near = t * inv;
      code[i][e] = __float_as_uint(fmaf(fmaf(-near, scale, t), inv, near) + kRound);
    }
  return finite ? scale_bits | low_bits : 0x7fc07fc0u;
}

// The codes in one word, code ORDER(n) in nibble n: the copies of kRoundBits
// add up to a constant.
template <bool KEY>
__device__ __forceinline__ uint32_t pack_codes(const uint32_t (&code)[8]) {
  uint32_t w = 0, extra = 0;
#pragma unroll
  for (int n = 7; n >= 0; --n) {
    const int e = KEY ? 2 * (n & 3) + (n >> 2) : n;
    w = w * 16u + code[e];
    extra = extra * 16u + kRoundBits;
  }
  return w - extra;
}

// Turn fractions and axes of the pairs, formed once per CTA, and the cosines
// and sines of the token a warp is at.
struct RopeShared {
  uint64_t frac[64];
  uint32_t axis[64];               // bit 2: not finite
  alignas(16) float2 cs[kWarps][64];   // read two at a time
};
static_assert(alignof(RopeShared) == 16, "16-byte loads of the angles");

__device__ __forceinline__ void load_pairs(const RopeParams& p, RopeShared& sh) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
    bool bad;
    sh.frac[i] = turn_fraction(p.inv_freq[i], bad);
    const uint32_t w = i < 32 ? (i < 16 ? p.pair_axis[0] : p.pair_axis[1]) : (i < 48 ? p.pair_axis[2] : p.pair_axis[3]);
    sh.axis[i] = ((w >> (2 * (i & 15))) & 3u) | (bad ? 4u : 0u);
  }
}

// Cosines and sines of a token's pairs: each lane forms its share of the (at
// most 64) angles and leaves them in `buf` for the warp.  (Every lane forming
// those of its own elements cost four times the arithmetic, and 13 us of the
// rotation of 4 x 4096 tokens of 14 heads.)  `position(axis)` gives the token's
// position.
template <class Position>
__device__ __forceinline__ void form_angles(const RopeParams& p, const RopeShared& sh, float2* buf, int lane,
                                            Position position) {
  __syncwarp();
  for (int i = lane; i < p.rot / 2; i += 32) {
    const uint32_t ax = sh.axis[i];
    float s, c;
    turn_sincos(position(static_cast<int>(ax & 3u)), sh.frac[i], s, c);
    if (ax & 4u) s = c = __uint_as_float(0x7fc00000u);
    buf[i] = make_float2(c, p.inverse ? -s : s);
  }
  __syncwarp();
}

// A row held by D/16 lanes, two 16-byte pieces each, both members of 8 pairs
// (elements e0 .. e0 + 7 and e1 .. e1 + 7), so a rotation stays in the lane;
// past the rotating part, 16 neighbouring elements.
template <bool IL>
struct PairLanes {
  int e0, e1;
  bool turns;
  float cs[8], sn[8];

  __device__ __forceinline__ PairLanes(int rot, int slot) {
    turns = 16 * slot < rot;
    e0 = (IL || !turns) ? 16 * slot : 8 * slot;
    e1 = (IL || !turns) ? e0 + 8 : e0 + rot / 2;
  }
  __device__ __forceinline__ void load_angles(const float2* buf, int slot) {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 v = *reinterpret_cast<const float4*>(buf + 8 * slot + i);
      cs[i] = v.x;
      sn[i] = v.y;
      cs[i + 1] = v.z;
      sn[i + 1] = v.w;
    }
  }
  __device__ __forceinline__ void turn(uint4& x0, uint4& x1) const {
    if (!turns) return;
    float a[8], b[8];
    unpack8(x0, a);
    unpack8(x1, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // Interleaved, x0 holds pairs 0 .. 3 and x1 pairs 4 .. 7.
      float& u = IL ? (i < 4 ? a[(2 * i) % 8] : b[(2 * i) % 8]) : a[i];
      float& v = IL ? (i < 4 ? a[(2 * i) % 8 + 1] : b[(2 * i) % 8 + 1]) : b[i];
      const float first = u * cs[i] - v * sn[i];
      v = v * cs[i] + u * sn[i];
      u = first;
    }
    x0 = pack8(a);
    x1 = pack8(b);
  }
};

// Elements 8 piece .. 8 piece + 7 of a row, turned; `other` holds those that
// they pair with (split pairs).  Products and sums are rounded one by one, as
// the formula reads: codes then agree with those of the fp32 formula.
template <bool IL>
__device__ __forceinline__ void turn_piece(const uint4& x, const uint4& other, const float2* angles, int rot,
                                           int piece, float (&y)[8]) {
  unpack8(x, y);
  if (8 * piece >= rot) return;
  if constexpr (IL) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = angles[4 * piece + e];
      const float a = y[2 * e], b = y[2 * e + 1];
      y[2 * e] = __fsub_rn(__fmul_rn(a, v.x), __fmul_rn(b, v.y));
      y[2 * e + 1] = __fadd_rn(__fmul_rn(b, v.x), __fmul_rn(a, v.y));
    }
  } else {
    const bool second = 16 * piece >= rot;
    const float2* cs = angles + 8 * piece - (second ? rot / 2 : 0);
    float z[8];
    unpack8(other, z);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 v = *reinterpret_cast<const float4*>(cs + e);
      // The first member of a pair takes -sin times the second.
      y[e] = __fadd_rn(__fmul_rn(y[e], v.x), __fmul_rn(second ? z[e] : -z[e], v.y));
      y[e + 1] = __fadd_rn(__fmul_rn(y[e + 1], v.z), __fmul_rn(second ? z[e + 1] : -z[e + 1], v.w));
    }
  }
}

// Tasks are (token, slice of its rows), one warp each.  Rows of a token:
// queries, keys, values.
template <int D, int MODE, int G, bool IL>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(MODE)) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kSlotLanes = D / 16;             // lanes of a row held in pairs
  constexpr int kRows = 32 / kSlotLanes;
  constexpr int kFlight = 2;                     // steps whose loads are in flight together
  __shared__ RopeShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = lane % kSlotLanes, sub = lane / kSlotLanes;

  pdl_wait_primary();
  pdl_launch_dependents();
  load_pairs(p, sh);
  __syncthreads();
  PairLanes<IL> pl(p.rot, slot);
  float2* angles = sh.cs[warp];
  const CellTranspose transpose(lane);

  const int tasks = static_cast<int>(p.tasks), stride = gridDim.x * kWarps;
  int task = blockIdx.x * kWarps + warp;
  // Where the next task's token goes is read while this one's rows come.
  int next_seq = 0, next_pos = 0, next_phys = 0;
  auto token = [&](int task_) {
    const int t_ = p.parts == 1 ? task_ : task_ / p.parts;
    next_seq = p.seq_ids[t_];
    next_pos = p.positions[t_];
  };
  auto entry = [&]() {
    if (next_seq >= 0 && next_seq < p.num_seqs && next_pos >= 0 && next_pos < p.max_blocks * kSlots)
      next_phys = p.block_table[static_cast<size_t>(next_seq) * p.max_blocks + next_pos / kSlots];
  };
  if (MODE != kRotate && task < tasks) {
    token(task);
    entry();
  }
  for (; task < tasks; task += stride) {
    const int t = p.parts == 1 ? task : task / p.parts;
    const int row0 = (task - t * p.parts) * p.rows_per_part;
    const int row1 = min(p.rows, row0 + p.rows_per_part);

    const int batch = MODE == kRotate ? t / p.N : 0;
    const int tok = t - batch * p.N;
    const int seq = next_seq, cache_pos = next_pos, phys = next_phys;
    if (MODE != kRotate) {
      if (task + stride < tasks) token(task + stride);
      unsigned err = 0;
      if (seq >= p.num_seqs) err = kDevBadSeqId;
      else if (cache_pos < 0 || cache_pos >= p.max_blocks * kSlots) err = kDevBadSeqLen;
      else if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) err = kDevBadBlock;
      if (seq < 0 || err) {                      // a row of padding; nothing of a bad token is written
        if (seq >= 0 && lane == 0) atomicOr(p.status, err);
        if (task + stride < tasks) entry();
        continue;
      }
    }
    const int cache_slot = cache_pos % kSlots;

    // Rows held in pairs: all of them, or with a 4-bit cache the queries.
    const int end = MODE == kAppendKv4 ? min(row1, p.Hq) : row1;
    const __nv_bfloat16 *qs = p.q.of(batch, tok), *ks = p.k.of(batch, tok), *vs = p.v.of(batch, tok);
    __nv_bfloat16 *qd = p.q_out.of(batch, tok), *kd = p.k_out.of(batch, tok);
    uint4 x0[kFlight], x1[kFlight];
    auto load = [&](int base) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r = base + u * kRows + sub;
        x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= end) continue;
        const bool value = MODE == kAppend && r >= p.Hq + p.Hk;
        const __nv_bfloat16* src = r < p.Hq ? RowPtr::row(qs, r, p.q.head)
                                   : value  ? RowPtr::row(vs, r - p.Hq - p.Hk, p.v.head)
                                            : RowPtr::row(ks, r - p.Hq, p.k.head);
        x0[u] = *reinterpret_cast<const uint4*>(src + (value ? 16 * slot : pl.e0));
        x1[u] = *reinterpret_cast<const uint4*>(src + (value ? 16 * slot + 8 : pl.e1));
      }
    };
    if (row0 < end) load(row0);
    if (MODE != kRotate && task + stride < tasks) entry();
    if (row0 < p.Hq + p.Hk) {
      const int* pos = p.rope_pos + batch * p.batch_stride + tok;
      const bool own = MODE != kRotate && p.rope_pos == nullptr;
      form_angles(p, sh, angles, lane, [&](int axis) { return own ? cache_pos : pos[axis * p.axis_stride]; });
      if (row0 < end) pl.load_angles(angles, slot);
    }
    for (int base = row0; base < end;) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r = base + u * kRows + sub;
        if (r >= end) continue;
        const bool value = MODE == kAppend && r >= p.Hq + p.Hk;
        if (!value) pl.turn(x0[u], x1[u]);
        __nv_bfloat16* dst;
        if (r < p.Hq) {
          dst = OutPtr::row(qd, r, p.q_out.head);
        } else if (MODE == kRotate) {
          dst = OutPtr::row(kd, r - p.Hq, p.k_out.head);
        } else {
          const int h = value ? r - p.Hq - p.Hk : r - p.Hq;
          dst = (value ? p.v_cache : p.k_cache) + ((static_cast<size_t>(phys) * p.Hk + h) * kSlots + cache_slot) * D;
        }
        *reinterpret_cast<uint4*>(dst + (value ? 16 * slot : pl.e0)) = x0[u];
        *reinterpret_cast<uint4*>(dst + (value ? 16 * slot + 8 : pl.e1)) = x1[u];
      }
      base += kFlight * kRows;
      if (base < end) load(base);
    }

    if constexpr (MODE == kAppendKv4) {
      // Keys and values for a 4-bit cache: rows of 16 neighbouring elements a
      // lane, as the groups lie; what they pair with is loaded as well (from
      // L1).
      using Lt = Kv4Layout<D, G>;
      if (row1 <= p.Hq) continue;
      const int k0 = max(row0 - p.Hq, 0), k1 = row1 - p.Hq;   // keys, then values
      const int shift = 16 * slot < p.rot / 2 ? p.rot / 2 : -p.rot / 2;         // of piece 2 slot
      const int shift1 = 16 * slot + 8 < p.rot / 2 ? p.rot / 2 : -p.rot / 2;    // of piece 2 slot + 1
      for (int base = k0; base < k1; base += kRows) {
        const int r = base + sub;
        const bool value = r >= p.Hk;
        uint4 x[2], z[2];
        x[0] = x[1] = z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < k1) {
          const __nv_bfloat16* src = (value ? RowPtr::row(vs, r - p.Hk, p.v.head) : RowPtr::row(ks, r, p.k.head)) + 16 * slot;
          x[0] = *reinterpret_cast<const uint4*>(src);
          x[1] = *reinterpret_cast<const uint4*>(src + 8);
          if (!IL && !value) {
            if (16 * slot < p.rot) z[0] = *reinterpret_cast<const uint4*>(src + shift);
            if (16 * slot + 8 < p.rot) z[1] = *reinterpret_cast<const uint4*>(src + 8 + shift1);
          }
        }
        float y[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (value)
            unpack8(x[i], y[i]);
          else
            turn_piece<IL>(x[i], z[i], angles, p.rot, 2 * slot + i, y[i]);
        }
        uint32_t code[2][8], w[2] = {0u, 0u};
        const uint32_t par = quantise16<G>(y, code);
        if (base < p.Hk) {                       // some row of this step is a key
          w[0] = pack_codes<true>(code[0]);
          w[1] = pack_codes<true>(code[1]);
          transpose.key(w);
        }
        if (base + kRows > p.Hk) {               // some row of this step is a value
          uint32_t wv[2] = {pack_codes<false>(code[0]), pack_codes<false>(code[1])};
          transpose.value(wv);
          if (value) {
            w[0] = wv[0];
            w[1] = wv[1];
          }
        }
        if (r < k1) {
          uint8_t* rec = p.kv_cache + (static_cast<size_t>(phys) * p.Hk + (value ? r - p.Hk : r)) * Lt::kBytes;
          uint32_t* row = reinterpret_cast<uint32_t*>(rec + (value ? Lt::kOffV : 0) + cache_slot * Lt::kRow);
#pragma unroll
          for (int i = 0; i < 2; ++i) row[value ? kv4_v_word<D>(2 * slot + i) : kv4_k_word<D>(2 * slot + i)] = w[i];
          if (slot % (G / 16) == 0)
            reinterpret_cast<uint32_t*>(rec + (value ? Lt::kOffParV : Lt::kOffParK) +
                                        cache_slot * Lt::kParRow)[slot / (G / 16)] = par;
        }
      }
    }
  }
}

// Rows of cached tokens back to bf16: value = code * scale + min, rounded
// once.  Rows of a token: its keys, then its values.  Measured: 15500 tokens of
// 4 KV heads, d = 128 (10 MB read, 32 MB written) 10.7 us, 3.9 TB/s; 2.1 us for
// 1570 of 2, d = 64.  3 us are the launch and three dependent reads (sequence,
// table, record); then the ALU pipe is half busy undoing the cells.
struct Kv4ReadParams {
  const uint8_t* kv_cache;
  const int* block_table;
  const int* seq_ids;
  const int* positions;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int Hkv, num_seqs, max_blocks, num_blocks;
  int parts, rows_per_part;
  long long tasks;
  unsigned int* status;
};

template <int D, int G>
__global__ void __launch_bounds__(kThreads, kReadCtas) kv4_read_kernel(const Kv4ReadParams p) {
  using Lt = Kv4Layout<D, G>;
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kFlight = 2;
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int rows = 2 * p.Hkv;
  const CellTranspose transpose(lane);

  pdl_wait_primary();
  pdl_launch_dependents();

  const int tasks = static_cast<int>(p.tasks), stride = gridDim.x * kWarps;
  int task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (task >= tasks) return;
  // The next task's token and table entry are read while this one's rows come
  // (10.7 us instead of 11.1 for the 15500 tokens).
  auto token = [&](int task_, int& seq_, int& pos_) {
    const int t_ = p.parts == 1 ? task_ : task_ / p.parts;
    seq_ = p.seq_ids[t_];
    pos_ = p.positions[t_];
  };
  auto entry = [&](int seq_, int pos_) {
    return seq_ >= 0 && seq_ < p.num_seqs && pos_ >= 0 && pos_ < p.max_blocks * kSlots
               ? p.block_table[static_cast<size_t>(seq_) * p.max_blocks + pos_ / kSlots] : 0;
  };
  int seq, pos, phys;
  token(task, seq, pos);
  phys = entry(seq, pos);
  for (int next; task < tasks; task = next) {
    next = task + stride;
    const int t = p.parts == 1 ? task : task / p.parts;
    const int row0 = (task - t * p.parts) * p.rows_per_part;
    const int row1 = min(rows, row0 + p.rows_per_part);
    const int my_seq = seq, my_pos = pos, my_phys = phys;
    if (next < tasks) token(next, seq, pos);
    unsigned err = 0;
    if (my_seq >= p.num_seqs) err = kDevBadSeqId;
    else if (my_pos < 0 || my_pos >= p.max_blocks * kSlots) err = kDevBadSeqLen;
    else if (static_cast<unsigned>(my_phys) >= static_cast<unsigned>(p.num_blocks)) err = kDevBadBlock;
    if (my_seq < 0 || err) {
      if (my_seq >= 0 && lane == 0) atomicOr(p.status, err);
      if (next < tasks) phys = entry(seq, pos);
      continue;
    }
    const int slot = my_pos % kSlots;
    const uint8_t* recs = p.kv_cache + static_cast<size_t>(my_phys) * p.Hkv * Lt::kBytes;
    for (int base = row0; base < row1; base += kFlight * kRows) {
      uint32_t w[kFlight][2], par[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r = base + u * kRows + sub;
        w[u][0] = w[u][1] = par[u] = 0;
        if (r < row1) {
          const bool value = r >= p.Hkv;
          const uint8_t* rec = recs + static_cast<size_t>(value ? r - p.Hkv : r) * Lt::kBytes;
          const uint32_t* row = reinterpret_cast<const uint32_t*>(rec + (value ? Lt::kOffV : 0) + slot * Lt::kRow);
#pragma unroll
          for (int i = 0; i < 2; ++i) w[u][i] = row[value ? kv4_v_word<D>(2 * j + i) : kv4_k_word<D>(2 * j + i)];
          par[u] = reinterpret_cast<const uint32_t*>(rec + (value ? Lt::kOffParV : Lt::kOffParK) +
                                                     slot * Lt::kParRow)[j / (G / 16)];
        }
      }
      if (base == row0 && next < tasks) phys = entry(seq, pos);
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r0 = base + u * kRows, r = r0 + sub;
        if (r0 >= row1) break;                   // the same for all lanes
        const bool value = r >= p.Hkv;
        uint32_t wk[2] = {w[u][0], w[u][1]}, wv[2] = {w[u][0], w[u][1]};
        if (r0 < p.Hkv) transpose.key(wk);
        if (r0 + kRows > p.Hkv) transpose.value(wv);
        const float scale = bf_hi(par[u]), low = bf_lo(par[u]);
        uint4 out[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // Cell n as a float: 2^23 + code, less 2^23.
          const uint32_t x = value ? wv[i] : wk[i];
          const uint32_t even = x & 0x0f0f0f0fu, odd = (x >> 4) & 0x0f0f0f0fu;
          float n[8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            n[2 * c] = fmaf(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440u + c)) - 8388608.f, scale, low);
            n[2 * c + 1] = fmaf(__uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440u + c)) - 8388608.f, scale, low);
          }
          // Element e of a value is cell e, element 2 c + h of a key cell c + 4 h.
          const uint32_t k0 = pack_bf16x2(n[0], n[4]), k1 = pack_bf16x2(n[1], n[5]), k2 = pack_bf16x2(n[2], n[6]),
                         k3 = pack_bf16x2(n[3], n[7]);
          out[i] = value ? pack8(n) : make_uint4(k0, k1, k2, k3);
        }
        if (r < row1) {
          uint4* dst = reinterpret_cast<uint4*>(
              (value ? p.v : p.k) + (static_cast<size_t>(t) * p.Hkv + (value ? r - p.Hkv : r)) * D + 16 * j);
          dst[0] = out[0];
          dst[1] = out[1];
        }
      }
    }
  }
}

// Slices of a token's `rows` rows such that `tokens` of them fill the GPU:
// one warp per token once there are enough tokens, else as many slices as
// that takes, down to one warp step each.
struct Split {
  int parts, rows_per_part;
  unsigned grid;
};
Split split_rows(long long tokens, int rows, int rows_per_step, int sms, int resident) {
  const long long want = static_cast<long long>(sms) * 16;
  const int most = (rows + rows_per_step - 1) / rows_per_step;
  long long parts = (want + tokens - 1) / tokens;
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  Split s;
  const int steps = (most + static_cast<int>(parts) - 1) / static_cast<int>(parts);
  s.rows_per_part = steps * rows_per_step;
  s.parts = (rows + s.rows_per_part - 1) / s.rows_per_part;
  const long long ctas = (tokens * s.parts + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(sms) * resident;
  s.grid = static_cast<unsigned>(ctas < cap ? ctas : cap);
  return s;
}

RowPtr in_rows(const HeadRows& h) {
  return RowPtr{static_cast<const __nv_bfloat16*>(h.data), h.batch, static_cast<int>(h.token / 8), static_cast<int>(h.head / 8)};
}
OutPtr out_rows(const HeadRows& h) {
  return OutPtr{static_cast<__nv_bfloat16*>(h.data), h.batch, static_cast<int>(h.token / 8), static_cast<int>(h.head / 8)};
}

void fill_spec(RopeParams& p, const RopeSpec& s) {
  p.inv_freq = s.inv_freq;
  p.rope_pos = s.positions;
  p.axis_stride = s.axis_stride;
  p.batch_stride = s.batch_stride;
  for (int i = 0; i < 4; ++i) p.pair_axis[i] = s.pair_axis[i];
  p.rot = s.rot;
  p.inverse = s.inverse ? 1 : 0;
}

template <int D, int MODE, int G>
cudaError_t launch_t(RopeParams& p, long long tokens, bool interleaved, int sms, cudaStream_t stream) {
  const Split s = split_rows(tokens, p.rows, 32 / (D / 16), sms, ctas_per_sm(MODE));
  p.parts = s.parts;
  p.rows_per_part = s.rows_per_part;
  p.tasks = tokens * s.parts;
  auto kern = interleaved ? rope_kernel<D, MODE, G, true> : rope_kernel<D, MODE, G, false>;
  return launch_pdl(kern, dim3(s.grid), dim3(kThreads), 0, stream, p);
}

template <int D, int G>
cudaError_t launch_read_t(Kv4ReadParams& p, long long tokens, int sms, cudaStream_t stream) {
  const Split s = split_rows(tokens, 2 * p.Hkv, 32 / (D / 16), sms, kReadCtas);
  p.parts = s.parts;
  p.rows_per_part = s.rows_per_part;
  p.tasks = tokens * s.parts;
  return launch_pdl(kv4_read_kernel<D, G>, dim3(s.grid), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_sm103(const RopeLaunch& a) {
  RopeParams p = {};
  fill_spec(p, a.spec);
  p.q = in_rows(a.q);
  p.k = in_rows(a.k);
  p.q_out = out_rows(a.q_out);
  p.k_out = out_rows(a.k_out);
  p.Hq = a.q.heads;
  p.Hk = a.k.heads;
  p.rows = p.Hq + p.Hk;
  p.N = a.N;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  if (a.d == 128) return launch_t<128, kRotate, 0>(p, tokens, a.spec.interleaved, a.sms, a.stream);
  return launch_t<64, kRotate, 0>(p, tokens, a.spec.interleaved, a.sms, a.stream);
}

cudaError_t launch_rope_append_sm103(const RopeAppendLaunch& a) {
  RopeParams p = {};
  fill_spec(p, a.spec);
  p.q = in_rows(a.q);
  p.k = in_rows(a.k);
  p.v = in_rows(a.v);
  p.q_out = out_rows(a.q_out);
  p.Hq = a.q.heads;
  p.Hk = a.k.heads;
  p.rows = p.Hq + 2 * p.Hk;
  p.N = 1;
  p.k_cache = static_cast<__nv_bfloat16*>(a.k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(a.v_cache);
  p.kv_cache = static_cast<uint8_t*>(a.kv_cache);
  p.block_table = a.block_table;
  p.seq_ids = a.seq_ids;
  p.positions = a.positions;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.status = a.status;
  const bool il = a.spec.interleaved;
  if (a.kv_cache == nullptr) {
    if (a.d == 128) return launch_t<128, kAppend, 0>(p, a.T, il, a.sms, a.stream);
    return launch_t<64, kAppend, 0>(p, a.T, il, a.sms, a.stream);
  }
  if (a.d == 128)
    return a.group == 32 ? launch_t<128, kAppendKv4, 32>(p, a.T, il, a.sms, a.stream)
                         : launch_t<128, kAppendKv4, 64>(p, a.T, il, a.sms, a.stream);
  return a.group == 32 ? launch_t<64, kAppendKv4, 32>(p, a.T, il, a.sms, a.stream)
                       : launch_t<64, kAppendKv4, 64>(p, a.T, il, a.sms, a.stream);
}

cudaError_t launch_kv4_read_sm103(const Kv4ReadLaunch& a) {
  Kv4ReadParams p;
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.block_table = a.block_table;
  p.seq_ids = a.seq_ids;
  p.positions = a.positions;
  p.k = static_cast<__nv_bfloat16*>(a.k);
  p.v = static_cast<__nv_bfloat16*>(a.v);
  p.Hkv = a.Hkv;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.status = a.status;
  if (a.d == 128)
    return a.group == 32 ? launch_read_t<128, 32>(p, a.T, a.sms, a.stream)
                         : launch_read_t<128, 64>(p, a.T, a.sms, a.stream);
  return a.group == 32 ? launch_read_t<64, 32>(p, a.T, a.sms, a.stream)
                       : launch_read_t<64, 64>(p, a.T, a.sms, a.stream);
}

}  // namespace attn47
