// What the decodes over quantised paged caches (4 and 8 bits) share: the split
// of the work over the warps of a one-wave grid, and the merge of the runs that
// it cuts.
//
// The blocks of all (sequence, KV head) runs lie in one flat order, cut into
// equal costs for every warp (a run costs a few blocks more than it has, for its
// queries and its end), or a team of a CTA's warps to each run where that is
// shorter.  A run that a warp holds whole is written by it; pieces of a run go to
// shared memory, are merged per CTA, and if the run reaches into other CTAs the
// merged part is published and the CTA that arrives last merges the parts.
//
// P is a kernel's parameters: seq_lens, num_seqs, max_blocks, Hkv (runs of a
// sequence), group (rows of a run), Hq (rows of a sequence), o, lse, ws_o, ws_ml,
// arrive, epoch, status, and row0(b, g) and rows_of(g), the first row of a run and
// how many of its rows there are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace attn47 {
namespace {

constexpr int kBS = 16;            // token slots of a block
// CTAs a launch may have (one per SM); the workspace has room for this many.
constexpr int kMaxCtas = 256;
// Entries of the plan's prefix sums (one per sequence up to this many, then
// one per several).
constexpr int kPlan = 1024;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrid = 12288.f;   // 1.5 2^13: x + kGrid - kGrid is x to a multiple of 2^-10

struct WarpMeta {
  int f_valid, l_valid, l_start;   // l_start: the last piece holds its run's block 0
  int fb, fg, lb, lg;              // runs of the two pieces
};

struct SplitShared {
  uint64_t ready[16];              // a warp's first piece is there for the warp before it
  WarpMeta meta[16];
  int4 scan[16];
  longlong2 reach[16];             // where the shares of the warps before and behind begin and end
  int part_cta0[2], part_n[2];     // parts of this CTA (see below): their run's first CTA and part count (0: none)
  int last[2];
  int abort;
};

template <class P>
__device__ __forceinline__ int seq_len_of(const P& p, int b) {
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
  template <class P>
  __device__ __forceinline__ int seq_blocks(const P& p, int b) const {
    return per == 1 ? blocks[b] : (seq_len_of(p, b) + kBS - 1) / kBS;
  }
};

struct RunPos {
  int b, g, blk, nblk;
  int cost;                        // cost position where the run starts
};

// The run of cost unit x < total and the first block at or after it; returns
// the blocks before that one.  (One thread.)
template <class P>
__device__ __forceinline__ int locate(const P& p, const Plan& plan, int x, RunPos& at) {
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
template <class P>
__device__ __forceinline__ void locate_run(const P& p, const Plan& plan, int r, RunPos& at) {
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
  template <class P>
  __device__ __forceinline__ void next_run(const P& p, const Plan& plan, int passed) {
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
  template <class P>
  __device__ __forceinline__ void skip(const P& p, const Plan& plan, int k) {
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

// (stab + log2(l)) ln 2, the whole part of the logarithm added to the
// stabiliser first (exactly): an LSE near 0 keeps its bits.
__device__ __forceinline__ float lse_of(float stab, float l) {
  const uint32_t bits = __float_as_uint(l);
  // (Infinities and NaN stay what they are.)
  const float part = bits >= 0x7f800000u ? l : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
  return ((stab + static_cast<float>(static_cast<int>(bits >> 23) - 127)) + __log2f(part)) * kLn2;
}

// What the plan and the first loads will read, into L2 while the work
// before this kernel drains (hints only: nothing is read here).  (One thread.)
template <int D, class P>
__device__ __forceinline__ void prefetch_inputs(const P& p) {
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

// The plan of a launch: the prefix sums go to cost, runs and seq_blocks (a CTA
// barrier has to follow).  costs.spare2: half blocks that a merge across CTAs is
// worth; costs.run_cost(blocks, shares): what a run costs beyond its blocks.
template <int kWarps, class P, class Costs>
__device__ __forceinline__ Plan build_plan(const P& p, SplitShared* sh, int* cost, int* runs, int* seq_blocks,
                                           const Costs& costs) {
  constexpr int kThreads = kWarps * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    // CTAs: it is taken where the longest run brings its team no more than
    // spare2 / 2 blocks beyond an equal share of all blocks.
    int team = 0;
#pragma unroll
    for (int k = kWarps; k >= 1; --k)
      if (kWarps % k == 0 && total_runs <= k * static_cast<int>(gridDim.x)) team = kWarps / k;
    if (static_cast<long long>(2 * longest - costs.spare2 * team) * shares > 2LL * team * total) team = 0;
    plan.team = team;
    plan.run_cost = costs.run_cost(total, shares);
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
  return plan;
}

// A warp's share: `blocks` blocks from w.at on, to before `end`.
struct Share {
  Walk w;
  RunPos end;
  int blocks, chunk;
  long long mine;                  // cost position where it begins
};

template <int kWarps, class P>
__device__ __forceinline__ Share take_share(const P& p, const Plan& plan, SplitShared* sh) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int shares = static_cast<int>(gridDim.x) * kWarps;
  Share s;
  Walk& w = s.w;
  RunPos& end = s.end;
  // Every share but the last of all holds at least one block (a share longer
  // than a run's start cost cannot lie inside it).
  int chunk = max(plan.run_cost + 1, (plan.total - 1) / shares + 1);
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

  int blocks = 0;
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
  s.blocks = blocks;
  s.chunk = chunk;
  s.mine = mine;
  return s;
}

// Runs that this CTA holds a part of: one that began before it and ends in
// it (kind 0), one that goes on behind it (kind 1).  Their counters are
// made ready now, long before they are counted on.  (Warps with a share.)
template <int kWarps, class P>
__device__ __forceinline__ void announce_parts(const P& p, const Plan& plan, SplitShared* sh, const Share& s) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    const long long cta_chunk = static_cast<long long>(s.chunk) * kWarps;
    auto take_part = [&](int kind, const RunPos& run) {
      const int first = run.cost + plan.run_cost;   // cost position of its block 0
      const int cta0 = static_cast<int>(first / cta_chunk), cta1 = static_cast<int>((first + run.nblk - 1) / cta_chunk);
      sh->part_cta0[kind] = cta0;
      sh->part_n[kind] = cta1 - cta0 + 1;
      ready_counter(p.arrive + cta0, p.epoch);
    };
    if (warp == 0 && s.w.at.blk > 0 && s.w.at.cost + plan.run_cost + s.w.at.nblk <= s.mine + cta_chunk) take_part(0, s.w.at);
    if (warp == kWarps - 1 && s.end.blk > 0) take_part(1, s.end);
  }
}

// Sequences without tokens: O = 0, LSE = -inf.
template <int kWarps, int D, class P>
__device__ __forceinline__ void write_empty_sequences(const P& p, const Plan& plan) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int shares = static_cast<int>(gridDim.x) * kWarps;
  for (int b = static_cast<int>(blockIdx.x) * kWarps + warp; b < p.num_seqs; b += shares) {
    if (plan.seq_blocks(p, b) != 0) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(b) * p.Hq * D);
    for (int i = lane; i < p.Hq * D / 2; i += 32) dst[i] = 0u;
    if (p.lse != nullptr)
      for (int h = lane; h < p.Hq; h += 32) p.lse[static_cast<size_t>(b) * p.Hq + h] = -INFINITY;
  }
}

// The end of a CTA: its warps' pieces merged, the parts of runs that other CTAs
// share published, and merged where this CTA is the last to arrive.  The pieces'
// rows are kPitch floats apart.
template <class Cfg, int D, class P, class First, class Last>
__device__ __forceinline__ void merge_pieces(const P& p, SplitShared* sh, float2* ml, First first_piece,
                                             Last last_piece) {
  constexpr int kWarps = Cfg::kWarps, kRows = Cfg::kRows;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
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
      const int run_g = kind ? mt.lg : mt.fg;
      const size_t h0 = p.row0(kind ? mt.lb : mt.fb, run_g);
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
          if (h >= p.rows_of(run_g)) continue;
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

}  // namespace
}  // namespace attn47
