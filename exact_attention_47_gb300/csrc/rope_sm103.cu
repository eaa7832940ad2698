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
// one token) is held by d/8 lanes, one 16-byte piece each, so a warp moves
// 512 bytes a step and keeps several loads in flight; the partner elements of
// a half-split pair come from another lane by shuffle.  A warp takes one
// token's rows (all of them when there are many tokens, a slice when there are
// few), so the angles of a token are formed once for all its heads, each by one
// lane of the warp.
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

struct RowPtr {
  const __nv_bfloat16* data;
  long long batch, token, head;
};
struct OutPtr {
  __nv_bfloat16* data;
  long long batch, token, head;
};

struct RopeParams {
  RowPtr q, k, v;
  OutPtr q_out, k_out;
  const float* inv_freq;
  const int* rope_pos;               // nullptr: the cache positions (append)
  long long axis_stride, batch_stride;
  uint32_t pair_axis[4];
  int rot, axes, inverse;
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

__device__ __forceinline__ void turn_sincos(int pos, uint64_t frac, float& s, float& c) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * frac;
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
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

// 4-bit codes of this lane's 8 elements and the parameter word of their
// group (the G/8 lanes of a group agree on it).  low = bf16(min), scale =
// bf16((max - low) / 15), code = (x - low) / scale rounded to even, clamped.
// A scale below the smallest normal number counts as 0 (a constant group:
// every value reads back as low); a group whose range is not finite gets NaN
// parameters, so that it reads back as NaN.
template <int G>
__device__ __forceinline__ uint32_t quantise8(const float (&y)[8], int (&code)[8]) {
  float lo = y[0], hi = y[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = min_nan(lo, y[e]);
    hi = max_nan(hi, y[e]);
  }
#pragma unroll
  for (int o = 1; o < G / 8; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t low_bits = pack_bf16x2(lo, 0.f) & 0xffffu;
  lo = __uint_as_float(low_bits << 16);
  const float range = hi - lo;
  const bool finite = fabsf(range) <= 3.402823466e38f;
  uint32_t scale_bits = pack_bf16x2(0.f, __fdiv_rn(fmaxf(range, 0.f), 15.f)) & 0xffff0000u;
  if (scale_bits < 0x00800000u) scale_bits = 0;
  if (!finite) scale_bits = 0;
  const float scale = __uint_as_float(scale_bits);
  const float inv = scale_bits ? __frcp_rn(scale) : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = y[e] - lo;
    // t inv is within 2e-6 of the quotient (which is at most 15.1): only next
    // to a half-way point can its rounding differ from the quotient's, and
    // there the division decides.  (Dividing always costs a third more.)
    float u = t * inv;
    if (fabsf(u - floorf(u) - 0.5f) < 1e-5f) u = __fdiv_rn(t, scale);
    code[e] = __float2int_rn(fminf(fmaxf(u, 0.f), 15.f));
  }
  return finite ? scale_bits | low_bits : 0x7fc07fc0u;
}

// Turn fractions and axes of the pairs, formed once per CTA, and the cosines
// and sines of the token a warp is at.
struct RopeShared {
  uint64_t frac[64];
  uint32_t axis[64];               // bit 2: not finite
  float2 cs[kWarps][64];
};

__device__ __forceinline__ void load_pairs(const RopeParams& p, RopeShared& sh) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
    bool bad;
    sh.frac[i] = turn_fraction(p.inv_freq[i], bad);
    const uint32_t w = i < 32 ? (i < 16 ? p.pair_axis[0] : p.pair_axis[1]) : (i < 48 ? p.pair_axis[2] : p.pair_axis[3]);
    sh.axis[i] = ((w >> (2 * (i & 15))) & 3u) | (bad ? 4u : 0u);
  }
}

// What a lane does to the 8 elements it holds of a row: it takes part in
// pairs `pair0` up, whose other members (of split pairs) lane `partner` holds.
template <bool IL>
struct LaneTurn {
  static constexpr int kPairs = IL ? 4 : 8;
  bool turns, second;
  int pair0, partner;
  float cs[kPairs], sn[kPairs];

  __device__ __forceinline__ LaneTurn(int rot, int j, int lane) {
    turns = 8 * j < rot;
    second = !IL && 16 * j >= rot;
    pair0 = IL ? 4 * j : second ? 8 * j - rot / 2 : 8 * j;
    partner = (!IL && turns) ? lane + (second ? -rot / 16 : rot / 16) : lane;
  }
  // Cosines and sines of a token's pairs: each lane forms its share of the
  // (at most 64) angles and the warp exchanges them through `buf` (every lane
  // forming those of its own elements cost 4 times the arithmetic: 41 us
  // instead of 26 for the rotation of 4 x 4096 tokens of 14 heads).
  // `position(axis)` gives the token's position.
  template <class Position>
  __device__ __forceinline__ void angles(const RopeParams& p, const RopeShared& sh, float2* buf, int lane,
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
    if (turns) {
#pragma unroll
      for (int e = 0; e < kPairs; e += 2) {
        const float4 v = *reinterpret_cast<const float4*>(buf + pair0 + e);
        cs[e] = v.x;
        sn[e] = v.y;
        cs[e + 1] = v.z;
        sn[e + 1] = v.w;
      }
      if (!IL && !second) {                      // the first member of a split pair takes -sin times the second
#pragma unroll
        for (int e = 0; e < kPairs; ++e) sn[e] = -sn[e];
      }
    }
  }
  // y = the 8 elements of x, turned (all lanes take part; `rotate` false: as
  // they are).
  __device__ __forceinline__ void apply(const uint4& x, float (&y)[8], bool rotate) const {
    unpack8(x, y);
    if constexpr (IL) {
      if (turns && rotate) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = y[2 * e], b = y[2 * e + 1];
          y[2 * e] = a * cs[e] - b * sn[e];
          y[2 * e + 1] = b * cs[e] + a * sn[e];
        }
      }
    } else {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, x.x, partner);
      o.y = __shfl_sync(0xffffffffu, x.y, partner);
      o.z = __shfl_sync(0xffffffffu, x.z, partner);
      o.w = __shfl_sync(0xffffffffu, x.w, partner);
      if (turns && rotate) {
        float z[8];
        unpack8(o, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * cs[e] + z[e] * sn[e];
      }
    }
  }
};

// Rows [r0, r1) of `src` (one token's heads `step` elements apart), turned,
// to the same rows of `dst`.  All lanes of a warp; kFlight steps of loads are
// in flight together.
template <int D, int kFlight, bool IL>
__device__ __forceinline__ void turn_rows(const LaneTurn<IL>& turn, const __nv_bfloat16* src, long long src_step,
                                          __nv_bfloat16* dst, long long dst_step, int r0, int r1, int j, int sub) {
  constexpr int kRows = 256 / D;
  src += 8 * j;
  dst += 8 * j;
  for (int base = r0; base < r1; base += kFlight * kRows) {
    uint4 x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int r = base + u * kRows + sub;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < r1) x[u] = *reinterpret_cast<const uint4*>(src + r * src_step);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (base + u * kRows >= r1) break;         // the same for all lanes
      const int r = base + u * kRows + sub;
      float y[8];
      turn.apply(x[u], y, true);
      if (r < r1) *reinterpret_cast<uint4*>(dst + r * dst_step) = turn.turns ? pack8(y) : x[u];
    }
  }
}

// Tasks are (token, slice of its rows), one warp each.
template <int D, int MODE, int G, bool IL>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;           // lanes of a row
  constexpr int kRows = 32 / kLanes;      // rows of a warp step
  __shared__ RopeShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % kLanes, sub = lane / kLanes;

  pdl_wait_primary();
  pdl_launch_dependents();
  load_pairs(p, sh);
  __syncthreads();
  LaneTurn<IL> turn(p.rot, j, lane);

  const int tasks = static_cast<int>(p.tasks), stride = gridDim.x * kWarps;
  for (int task = blockIdx.x * kWarps + warp; task < tasks; task += stride) {
    const int t = task / p.parts;
    const int row0 = (task - t * p.parts) * p.rows_per_part;
    const int row1 = min(p.rows, row0 + p.rows_per_part);

    long long batch = 0, tok = t;
    if (MODE == kRotate) {
      const int b = t / p.N;
      batch = b;
      tok = t - b * p.N;
    }
    int cache_pos = 0, phys = 0;
    if (MODE != kRotate) {
      const int seq = p.seq_ids[t];
      cache_pos = p.positions[t];
      if (seq < 0) continue;                     // a row of padding
      unsigned err = 0;
      if (seq >= p.num_seqs) err = kDevBadSeqId;
      else if (cache_pos < 0 || cache_pos >= p.max_blocks * kSlots) err = kDevBadSeqLen;
      else {
        phys = p.block_table[static_cast<size_t>(seq) * p.max_blocks + cache_pos / kSlots];
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) err = kDevBadBlock;
      }
      if (err) {                                 // nothing of this token is written
        if (lane == 0) atomicOr(p.status, err);
        continue;
      }
    }

    if (row0 < p.Hq + p.Hk) {
      const int* pos = p.rope_pos + batch * p.batch_stride + tok;
      const bool own = MODE != kRotate && p.rope_pos == nullptr;
      turn.angles(p, sh, sh.cs[warp], lane,
                  [&](int axis) { return own ? cache_pos : pos[axis * p.axis_stride]; });
    }
    if (row0 < p.Hq)
      turn_rows<D, 4, IL>(turn, p.q.data + batch * p.q.batch + tok * p.q.token, p.q.head,
                          p.q_out.data + batch * p.q_out.batch + tok * p.q_out.token, p.q_out.head, row0,
                          min(row1, p.Hq), j, sub);
    if (row1 <= p.Hq) continue;
    const int k0 = max(row0 - p.Hq, 0), k1 = row1 - p.Hq;   // keys, then values
    if constexpr (MODE == kRotate) {
      turn_rows<D, 4, IL>(turn, p.k.data + batch * p.k.batch + tok * p.k.token, p.k.head,
                          p.k_out.data + batch * p.k_out.batch + tok * p.k_out.token, p.k_out.head, k0, k1, j, sub);
    } else {
      constexpr int kFlight = 2;
      const __nv_bfloat16* ks = p.k.data + tok * p.k.token + 8 * j;
      const __nv_bfloat16* vs = p.v.data + tok * p.v.token + 8 * j;
      const int slot = cache_pos % kSlots;
      for (int base = k0; base < k1; base += kFlight * kRows) {
        uint4 x[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          const int r = base + u * kRows + sub;
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < k1)
            x[u] = *reinterpret_cast<const uint4*>(r < p.Hk ? ks + r * p.k.head : vs + (r - p.Hk) * p.v.head);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          if (base + u * kRows >= k1) break;     // the same for all lanes
          const int r = base + u * kRows + sub;
          const bool value = r >= p.Hk;
          const int h = value ? r - p.Hk : r;
          float y[8];
          turn.apply(x[u], y, !value);
          if constexpr (MODE == kAppend) {
            __nv_bfloat16* dst = (value ? p.v_cache : p.k_cache) +
                                 ((static_cast<size_t>(phys) * p.Hk + h) * kSlots + slot) * D + 8 * j;
            if (r < k1) *reinterpret_cast<uint4*>(dst) = (turn.turns && !value) ? pack8(y) : x[u];
          } else {
            using Lt = Kv4Layout<D, G>;
            int code[8];
            const uint32_t par = quantise8<G>(y, code);
            uint32_t wk = 0, wv = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              wk |= static_cast<uint32_t>(code[e]) << (4 * ((e >> 1) + 4 * (e & 1)));
              wv |= static_cast<uint32_t>(code[e]) << (4 * e);
            }
            wk = kv4_k_transpose(wk, lane);
            wv = kv4_v_transpose(wv, lane);
            if (r < k1) {
              uint8_t* rec = p.kv_cache + (static_cast<size_t>(phys) * p.Hk + h) * Lt::kBytes;
              uint32_t* row = reinterpret_cast<uint32_t*>(rec + (value ? Lt::kOffV : 0) + slot * Lt::kRow);
              row[value ? kv4_v_word<D>(j) : kv4_k_word<D>(j)] = value ? wv : wk;
              if (j % (G / 8) == 0)
                reinterpret_cast<uint32_t*>(rec + (value ? Lt::kOffParV : Lt::kOffParK) +
                                            slot * Lt::kParRow)[j / (G / 8)] = par;
            }
          }
        }
      }
    }
  }
}

// Rows of cached tokens back to bf16: value = code * scale + min, rounded
// once.  Row 2 h of a token is head h's key, row 2 h + 1 its value.
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
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4ReadParams p) {
  using Lt = Kv4Layout<D, G>;
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kFlight = 4;
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int rows = 2 * p.Hkv;

  pdl_wait_primary();
  pdl_launch_dependents();

  const long long stride = static_cast<long long>(gridDim.x) * kWarps;
  for (long long task = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); task < p.tasks;
       task += stride) {
    const long long t = task / p.parts;
    const int row0 = static_cast<int>(task - t * p.parts) * p.rows_per_part;
    const int row1 = min(rows, row0 + p.rows_per_part);
    const int seq = p.seq_ids[t], pos = p.positions[t];
    if (seq < 0) continue;
    unsigned err = 0;
    int phys = 0;
    if (seq >= p.num_seqs) err = kDevBadSeqId;
    else if (pos < 0 || pos >= p.max_blocks * kSlots) err = kDevBadSeqLen;
    else {
      phys = p.block_table[static_cast<size_t>(seq) * p.max_blocks + pos / kSlots];
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) err = kDevBadBlock;
    }
    if (err) {
      if (lane == 0) atomicOr(p.status, err);
      continue;
    }
    const int slot = pos % kSlots;
    for (int base = row0; base < row1; base += kFlight * kRows) {
      uint32_t w[kFlight], par[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r = base + u * kRows + sub;
        w[u] = par[u] = 0;
        if (r < row1) {
          const uint8_t* rec = p.kv_cache + (static_cast<size_t>(phys) * p.Hkv + (r >> 1)) * Lt::kBytes;
          const bool value = r & 1;
          w[u] = reinterpret_cast<const uint32_t*>(rec + (value ? Lt::kOffV : 0) + slot * Lt::kRow)[
              value ? kv4_v_word<D>(j) : kv4_k_word<D>(j)];
          par[u] = reinterpret_cast<const uint32_t*>(rec + (value ? Lt::kOffParV : Lt::kOffParK) +
                                                     slot * Lt::kParRow)[j / (G / 8)];
        }
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int r0 = base + u * kRows;
        if (r0 >= row1) break;                   // the same for all lanes
        const int r = r0 + sub;
        const uint32_t ck = kv4_k_transpose(w[u], lane), cv = kv4_v_transpose(w[u], lane);
        const float scale = bf_hi(par[u]), low = bf_lo(par[u]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t code = (r & 1) ? cv >> (4 * e) : ck >> (4 * ((e >> 1) + 4 * (e & 1)));
          y[e] = fmaf(static_cast<float>(code & 15u), scale, low);
        }
        if (r < row1) {
          __nv_bfloat16* dst = (r & 1) ? p.v : p.k;
          *reinterpret_cast<uint4*>(dst + (static_cast<size_t>(t) * p.Hkv + (r >> 1)) * D + 8 * j) = pack8(y);
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
Split split_rows(long long tokens, int rows, int rows_per_step, int sms) {
  const long long want = static_cast<long long>(sms) * 16;
  const int most = (rows + rows_per_step - 1) / rows_per_step;
  long long parts = (want + tokens - 1) / tokens;
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  Split s;
  const int steps = (most + static_cast<int>(parts) - 1) / static_cast<int>(parts);
  s.rows_per_part = steps * rows_per_step;
  s.parts = (rows + s.rows_per_part - 1) / s.rows_per_part;
  const long long ctas = (tokens * s.parts + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(sms) * 4;
  s.grid = static_cast<unsigned>(ctas < cap ? ctas : cap);
  return s;
}

RowPtr in_rows(const HeadRows& h) {
  return RowPtr{static_cast<const __nv_bfloat16*>(h.data), h.batch, h.token, h.head};
}
OutPtr out_rows(const HeadRows& h) {
  return OutPtr{static_cast<__nv_bfloat16*>(h.data), h.batch, h.token, h.head};
}

void fill_spec(RopeParams& p, const RopeSpec& s) {
  p.inv_freq = s.inv_freq;
  p.rope_pos = s.positions;
  p.axis_stride = s.axis_stride;
  p.batch_stride = s.batch_stride;
  for (int i = 0; i < 4; ++i) p.pair_axis[i] = s.pair_axis[i];
  p.rot = s.rot;
  p.axes = s.axes;
  p.inverse = s.inverse ? 1 : 0;
}

template <int D, int MODE, int G>
cudaError_t launch_t(RopeParams& p, long long tokens, bool interleaved, int sms, cudaStream_t stream) {
  const Split s = split_rows(tokens, p.rows, 32 / (D / 8), sms);
  p.parts = s.parts;
  p.rows_per_part = s.rows_per_part;
  p.tasks = tokens * s.parts;
  auto kern = interleaved ? rope_kernel<D, MODE, G, true> : rope_kernel<D, MODE, G, false>;
  return launch_pdl(kern, dim3(s.grid), dim3(kThreads), 0, stream, p);
}

template <int D, int G>
cudaError_t launch_read_t(Kv4ReadParams& p, long long tokens, int sms, cudaStream_t stream) {
  const Split s = split_rows(tokens, 2 * p.Hkv, 32 / (D / 8), sms);
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
