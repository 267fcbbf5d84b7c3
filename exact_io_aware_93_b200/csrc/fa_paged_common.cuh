// fa_paged_common.cuh -- attention over a paged cache: the work list, page loads, query scaling
// and the join, shared by the kernels for few rows (fa_paged_few_kernel.cuh) and for tiles of 128
// rows (fa_paged_kernel.cuh).
//
// Rows.  The G = H / H_kv query heads of a key/value head and a sequence's new tokens form the
// rows r = i * G + g, so the cache is read once for all of them.  A TILE holds TQ tokens (one TMA
// box of G heads x TQ tokens).  A UNIT is a pair of consecutive tiles of one (sequence, key/value
// head), or one tile when a sequence has no more.
//
// Work list.  A unit visits T = hi - lo tiles of 128 keys, those that some row of it sees
// (causal: up to its last token; window: from its first token's first key).  The key tiles of
// all units are laid end to end (sequence, key/value head, unit), each as long as it takes
// (Cfg::kPairCost, kSplitCost, and kUnitCost once per unit: its epilogue), and CTA c of the persistent grid takes the tiles that start in
// [c L, (c+1) L), L = total / grid: every SM gets the same work whatever the mix of chunks,
// single tokens and lengths.  A CTA's run falls into SEGMENTS, each inside one unit; a segment
// that is not a whole unit leaves a partial result (O normalised, log-sums) that
// fa_paged_merge_kernel joins.  The lengths are read on the device, so a captured graph replays
// as they grow.  One warp walks the list and writes each segment into a small ring in shared
// memory that the CTA's other warps follow.
//
// Pages.  A key tile is 128 / page boxes (or a part of one page), each fetched by its own lane
// of the loading warp; page numbers are read 32 at a time, one window ahead.  Pages that no row
// of the unit sees are not fetched, and value rows outside the unit's keys are zeroed in shared
// memory: stale slots, and pages a sliding window has left behind, may hold anything.
#pragma once

#include <type_traits>

#include "fa_cache_kernels.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

// fp16 weights are 2^(x - m + 7): the largest, 2^kTau over the reference maximum m, still fits below
// 65504, and the smallest, 2^-24, is 2^-31 of the reference weight, so that a hundred thousand keys of
// little weight each keep their sum.  bf16 has the range without it.
template <Elem W>
constexpr float kWeightShift = W == Elem::kF16 ? 7.0f : 0.0f;

// Bounded waits, smaller than mbar_wait: these kernels have many and their code has to stay in
// the instruction cache.  A wait that runs out (2 s) leaves its site in the CTA's abort flag,
// which ends every other wait; the flag is reported once, when the CTA ends (pg_report).
struct PgWait {
  volatile int* abort_flag;
  int site;
};
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// One warp waits for up to a barrier per lane (null: none) together: barriers that are ready cost
// one round trip to shared memory, not one each.
__device__ __forceinline__ bool pg_wait_lanes(uint64_t* bar, uint32_t parity, const PgWait& w) {
  const uint32_t a = smem_u32(bar);
  bool done = bar == nullptr;
  uint32_t t0 = 0;
  for (uint32_t spins = 0;; ++spins) {
    if (!done) done = mbar_test(a, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if (spins % 64 != 63) continue;  // the timer is slow to read
    const uint32_t now = globaltimer_lo();
    if (spins == 63) t0 = now;
    bool stop = *w.abort_flag != 0;
    if (now - t0 > static_cast<uint32_t>(FA_WAIT_TIMEOUT_NS)) {
      if (!stop) *w.abort_flag = w.site;
      stop = true;
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
}
__device__ __forceinline__ bool pg_wait(uint64_t* bar, uint32_t parity, const PgWait& w) {
  return pg_wait_lanes(bar, parity, w);
}
// At the end of a CTA, after its last barrier: one thread.
__device__ __forceinline__ void pg_report(const int* abort_flag, int* status) {
  if (*abort_flag != 0) {
    atomicCAS(status, 0, 6 /* FA_ERR_TIMEOUT */);
    atomicCAS(status + 1, 0, *abort_flag);
  }
}

// A unit computed by several CTAs, from the one that began it: what the join needs.
struct PgSplit {
  int parts;  // CTAs; 0: none
  int kvh;
  int q0;     // first token
  int ntok;
};

struct PgArgs {
  const int* cu;          // [B + 1]
  const int* seqlens;     // [B]
  const int* table;       // [B, max_pages]
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const float* q_scale;   // e4m3 pages: [T, H] factors of the scaled queries
  void* out;              // [T, H, D]
  float* lse;             // [H, T]
  PgSplit* splits;        // of each CTA: the unit that it began and did not finish
  float* part_lse;        // [slots * kSubs, kRows, 2]
  float* part_o;          // [slots * kSubs, kRows, D]
  int n_lo, n_hi;         // sequences with more than n_lo and up to n_hi new tokens are computed
  int B, T, H, H_kv, max_q, TQ, max_pages, page, page_shift, P, window, causal;
  float scale_log2;
  long long slots;        // 2 per CTA
  int behind;             // launched behind the few-rows kernel of the same call
  int* status;
};

// ---------------------------------------------------------------- the work list
struct PgSeq {
  int q0, n, len, units;
};
__device__ __forceinline__ PgSeq pg_seq(const PgArgs& a, int b) {
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.seqlens + b);
  PgSeq s;
  const bool in = c0 >= 0 && c0 <= a.T && c1 > c0;
  s.q0 = in ? c0 : 0;
  s.n = in ? min(min(c1 - c0, a.max_q), a.T - c0) : 0;
  if (s.n <= a.n_lo || s.n > a.n_hi) s.n = 0;
  s.len = min(max(len, 0), a.max_pages * a.page);
  s.units = s.n <= 2 * a.TQ ? s.n > 0 : ((s.n + a.TQ - 1) / a.TQ + 1) / 2;
  return s;
}
__device__ __forceinline__ bool pg_seq_ok(const PgArgs& a, int b) {
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.seqlens + b);
  return c0 >= 0 && c1 >= c0 && c1 <= a.T && c1 - c0 <= a.max_q && len >= 0 && len <= a.max_pages * a.page;
}

// The first key that the window leaves a token at position `pos` (negative: before the sequence's first).
__device__ __forceinline__ int pg_first_key(const PgArgs& a, int pos) {
  return a.window >= 0 && pos > a.window ? pos - a.window : 0;
}

// Keys [lo, hi) that the tokens at positions p0 .. p1 of a sequence of `len` keys see, and the
// key tiles that hold them.
struct PgKeys {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ PgKeys pg_keys(const PgArgs& a, int len, int p0, int p1) {
  PgKeys k;
  k.hi = a.causal ? min(p1 + 1, len) : len;
  k.lo = pg_first_key(a, p0);
  if (k.hi <= k.lo) k.hi = k.lo = 0;
  k.t0 = k.lo >> 7;
  k.t1 = (k.hi + 127) >> 7;
  return k;
}

__device__ __forceinline__ PgKeys pg_unit_keys(const PgArgs& a, const PgSeq& s, int u) {
  const int tok0 = u * 2 * a.TQ;
  const int ntok = min(2 * a.TQ, s.n - tok0);
  const int p0 = s.len - s.n + tok0;
  return pg_keys(a, s.len, p0, p0 + ntok - 1);
}

__device__ __forceinline__ bool pg_is_pair(const PgArgs& a, const PgSeq& s, int u) {
  return s.n - u * 2 * a.TQ > a.TQ;
}

// Cost of a unit: its end (kUnitCost, which lies before its first tile in the list), then its tiles.
template <typename Cfg>
__device__ __forceinline__ int pg_unit_cost(const PgArgs& a, const PgSeq& s, int u) {
  const PgKeys k = pg_unit_keys(a, s, u);
  const int tiles = k.t1 - k.t0;
  return tiles > 0 ? Cfg::kUnitCost + tiles * (pg_is_pair(a, s, u) ? Cfg::kPairCost : Cfg::kSplitCost) : 0;
}

// Cost of a sequence's units for one key/value head.
template <typename Cfg>
__device__ __forceinline__ int pg_seq_cost(const PgArgs& a, const PgSeq& s) {
  int w = 0;
  for (int u = 0; u < s.units; ++u) w += pg_unit_cost<Cfg>(a, s, u);
  return w;
}

// This CTA's slice [t0, t1) of the work and the unit that t0 falls into, which starts at `start`.
struct PgPlan {
  int t0, t1, per, b, kvh, u, start;
};

// One warp; CTA 0's also checks the lengths and offsets.
template <typename Cfg>
__device__ __forceinline__ void pg_plan(const PgArgs& a, int lane, PgPlan* out) {
  constexpr unsigned kFull = 0xffffffffu;
  int total = 0, acc = 0;
  PgPlan p{0, 0, 0, 0, 0, 0, 0};
  // first the total, then the sequence that the slice starts in; up to 32 sequences are read once
  PgSeq s{0, 0, 0, 0};
  int w = 0;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      if (round == 0 || a.B > 32) {
        s = PgSeq{0, 0, 0, 0};
        if (b < a.B) {
          s = pg_seq(a, b);
          if (round == 0 && blockIdx.x == 0 && !pg_seq_ok(a, b)) plan_fail(a.status, 43);
        }
        w = pg_seq_cost<Cfg>(a, s);
      }
      int incl = w * a.H_kv;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      incl += acc;
      const int excl = incl - w * a.H_kv;
      if (round == 1 && excl <= p.t0 && p.t0 < incl) {  // one lane
        p.b = b;
        p.kvh = (p.t0 - excl) / w;
        p.start = excl + p.kvh * w;
        while (true) {
          const int c = pg_unit_cost<Cfg>(a, s, p.u);
          if (p.t0 < p.start + c) break;
          p.start += c;
          ++p.u;
        }
        *out = p;
      }
      acc = __shfl_sync(kFull, incl, 31);
      if (round == 1 && acc > p.t0) return;
    }
    if (round == 0) {
      total = acc;
      acc = 0;
      // at least a tile's cost, so that no CTA inside a unit's span is left without one of its tiles
      p.per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), Cfg::kPairCost);
      p.t0 = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(blockIdx.x) * p.per));
      p.t1 = min(total - p.t0, p.per) + p.t0;
      p.start = p.t0;
      if (lane == 0) *out = p;  // the answer when there is nothing to do
      if (p.t0 >= p.t1) return;
      p.start = 0;
      __syncwarp();
    }
  }
}

// Key tiles [lo, hi).
struct PgRange {
  int lo, hi;
};

// A run of nt key tiles from tile kt0 of one unit; nt = 0 ends a CTA's list.
struct PgSeg {
  int b, kvh;
  int q0;        // the unit's first token
  int pos0;      // its position
  int ntok;      // tokens of the unit
  int len;
  PgKeys keys;   // what the unit sees
  int kt0, nt;
  int pair;      // two tiles
  int whole;     // the run is the whole unit
  int slot;      // of a partial result: 0 when the unit started in an earlier CTA, else 1
  PgRange tile[2];  // pair: the key tiles of the run that each tile visits
};

// Walks this CTA's slice segment by segment (the schedule's warp, every lane alike).  Each lane holds one
// of 32 sequences: those that are not this kernel's, a mixed batch's single tokens between two chunks, are
// stepped over 32 at a time (2048 of them between chunks of 500 tokens: 1106 us one at a time, 778 so, 753
// with both chunks in front).
template <typename Cfg>
struct PgWalk {
  int t0, t1, per, b, kvh, u, start;
  PgSeq s;
  PgSeq mine;     // of sequence b - b % 32 + lane
  PgSplit split;  // of the last segment
  __device__ __forceinline__ PgWalk(const PgArgs& a, const PgPlan& p)
      : t0(p.t0), t1(p.t1), per(p.per), b(p.b), kvh(p.kvh), u(p.u), start(p.start), split{0, 0, 0, 0} {
    fetch(a, b & ~31);
    take(b & 31);
  }
  __device__ __forceinline__ void fetch(const PgArgs& a, int b0) {
    const int i = b0 + static_cast<int>(threadIdx.x & 31);
    mine = PgSeq{0, 0, 0, 0};
    if (i < a.B) mine = pg_seq(a, i);
  }
  __device__ __forceinline__ void take(int from) {
    constexpr unsigned kFull = 0xffffffffu;
    s.q0 = __shfl_sync(kFull, mine.q0, from);
    s.n = __shfl_sync(kFull, mine.n, from);
    s.len = __shfl_sync(kFull, mine.len, from);
    s.units = __shfl_sync(kFull, mine.units, from);
  }
  // The next sequence with units.
  __device__ __forceinline__ bool next_seq(const PgArgs& a) {
    unsigned left = __ballot_sync(0xffffffffu, mine.units > 0) & (0xfffffffeu << (b & 31));
    b &= ~31;
    while (left == 0) {
      b += 32;
      if (b >= a.B) return false;
      fetch(a, b);
      left = __ballot_sync(0xffffffffu, mine.units > 0);
    }
    b += __ffs(left) - 1;
    take(b & 31);
    return true;
  }
  __device__ __forceinline__ bool next(const PgArgs& a, PgSeg& g) {
    while (start < t1) {
      if (u >= s.units) {
        u = 0;
        if (++kvh >= a.H_kv) {
          kvh = 0;
          if (!next_seq(a)) return false;
        }
        continue;
      }
      const PgKeys k = pg_unit_keys(a, s, u);
      const bool pair = pg_is_pair(a, s, u);
      const int cost = pair ? Cfg::kPairCost : Cfg::kSplitCost;
      const int T = k.t1 - k.t0;
      // the tiles that start in [t0, t1)
      const int begin = start + Cfg::kUnitCost;
      const int first = t0 > begin ? (t0 - begin + cost - 1) / cost : 0;
      const int last = t1 > begin ? min(T, (t1 - begin + cost - 1) / cost) : 0;
      const int tok0 = u * 2 * a.TQ;
      if (T > 0) start = begin + T * cost;
      ++u;
      if (first >= last) continue;
      g.b = b;
      g.kvh = kvh;
      g.q0 = s.q0 + tok0;
      g.pos0 = s.len - s.n + tok0;
      g.ntok = min(2 * a.TQ, s.n - tok0);
      g.len = s.len;
      g.keys = k;
      g.kt0 = k.t0 + first;
      g.nt = last - first;
      g.pair = pair;
      g.whole = first == 0 && last == T;
      g.slot = first == 0;
      if (first == 0 && last < T)
        split = PgSplit{(begin + (T - 1) * cost) / per - static_cast<int>(blockIdx.x) + 1, kvh, g.q0, g.ntok};
      for (int i = 0; i < 2; ++i) {
        const int tok = i * a.TQ;
        const int n = min(a.TQ, g.ntok - tok);
        PgRange r{0, 0};
        if (n > 0) {
          const PgKeys kt = pg_keys(a, g.len, g.pos0 + tok, g.pos0 + tok + n - 1);
          r = PgRange{max(kt.t0, g.kt0), min(kt.t1, g.kt0 + g.nt)};
          if (r.hi < r.lo) r.hi = r.lo;
        }
        g.tile[i] = r;
      }
      return true;
    }
    return false;
  }
};

// The key tiles of a segment in the order the MMA warp consumes them.  pair: K_j, V_j; split:
// K_0, .., K_{Ahead-1}, V_0, K_Ahead, V_1, ..  f(is_value, tile) returns false to stop.
template <int Ahead, typename F>
__device__ __forceinline__ bool pg_loads(const PgSeg& g, F f) {
  if (g.pair) {
    for (int t = 0; t < g.nt; ++t)
      if (!f(false, g.kt0 + t) || !f(true, g.kt0 + t)) return false;
    return true;
  }
  for (int t = 0; t < Ahead && t < g.nt; ++t)
    if (!f(false, g.kt0 + t)) return false;
  for (int t = 0; t < g.nt; ++t)
    if (!f(true, g.kt0 + t) || (t + Ahead < g.nt && !f(false, g.kt0 + t + Ahead))) return false;
  return true;
}

// Page numbers of one sequence as the loading warp needs them: windows of 32 table entries, the
// even and the odd one held (keys run a few tiles ahead of values), one read ahead.
struct PgPages {
  int even, odd, ahead, at;
  __device__ __forceinline__ int entry(const PgArgs& a, int b, int win, int lane) const {
    const long long i = static_cast<long long>(win) * 32 + lane;
    return i < a.max_pages ? __ldg(a.table + static_cast<long long>(b) * a.max_pages + i) : -1;
  }
  __device__ __forceinline__ void start(const PgArgs& a, const PgSeg& g, int lane) {
    at = (((g.kt0 << 7) >> a.page_shift) >> 5) - 1;
    ahead = entry(a, g.b, at + 1, lane);
  }
  // Page number of tile j's page p0 + k (p0 its first), per lane.
  __device__ __forceinline__ int get(const PgArgs& a, const PgSeg& g, int p0, int k, int lane) {
    if ((p0 >> 5) > at) {
      at = p0 >> 5;
      if (at & 1) odd = ahead; else even = ahead;
      ahead = entry(a, g.b, at + 1, lane);
    }
    return __shfl_sync(0xffffffffu, (p0 >> 5) & 1 ? odd : even, (p0 + k) & 31);
  }
};

// Issues the boxes of key tile j that hold a key of the unit (whole warp; the slot is free).  With
// `scales` also the tile's scale bytes, keys' and then values': every lane's arrive on their own
// barrier.
template <int kRowBytes, int kChunks>
__device__ __forceinline__ void pg_load_tile(const PgArgs& a, const PgSeg& g, PgPages& pages, const CUtensorMap* map,
                                             int j, uint8_t* dst, uint64_t* full, int lane, uint8_t* scales = nullptr,
                                             uint64_t* scales_full = nullptr) {
  const int bs = min(7, a.page_shift);      // box: 1 << bs keys
  const int p0 = (j << 7) >> a.page_shift;  // the tile's first page
  const int k0 = max(g.keys.lo - (j << 7), 0) >> bs;
  const int k1 = (min(g.keys.hi - (j << 7), 128) + (1 << bs) - 1) >> bs;
  const int k = k0 + lane / kChunks, c = lane % kChunks;
  const int id = pages.get(a, g, p0, k, lane);
  if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(((k1 - k0) << bs) * kRowBytes * kChunks));
  __syncwarp();
  if (k < k1) {
    const int row = (j << 7) & (a.page - 1) & ~((1 << bs) - 1);  // inside a page of 256
    const bool good = id >= 0 && id < a.P;
    if (!good) plan_fail(a.status, 44);
    // a bad page number reads as zeros: a coordinate past the pool
    if (FA_IN_BOUNDS(row + (1 << bs) <= a.page && p0 + k < a.max_pages && (k << bs) < 128, a.status, 502))
      tma_load_3d(dst + c * 128 * kRowBytes + (k << bs) * kRowBytes, map, full, c * 64, row,
                  good ? id * a.H_kv + g.kvh : a.P * a.H_kv);
  }
  if (scales) {
    // four keys per lane, which lie in one page; keys that the unit does not see are left out
    const int key = (j << 7) + lane * 4;
    const int pg = pages.get(a, g, p0, (lane * 4) >> a.page_shift, lane);
    const bool seen = key + 3 >= g.keys.lo && key < g.keys.hi, good = pg >= 0 && pg < a.P;
    if (seen && good) {
      const int64_t at = (static_cast<int64_t>(pg) * a.H_kv + g.kvh) * a.page + (key & (a.page - 1));
      if (FA_IN_BOUNDS(at >= 0 && at + 4 <= static_cast<int64_t>(a.P) * a.H_kv * a.page, a.status, 513)) {
        cp_async4(scales + lane * 4, a.k_scales + at);
        cp_async4(scales + 128 + lane * 4, a.v_scales + at);
      }
    }
    if (seen && !good) {  // the zeros of a bad page number have scale 1; a plain arrival publishes plain stores
      *reinterpret_cast<uint32_t*>(scales + lane * 4) = 0x7f7f7f7fu;
      *reinterpret_cast<uint32_t*>(scales + 128 + lane * 4) = 0x7f7f7f7fu;
      mbar_arrive(scales_full);
    } else {
      cp_async_arrive(scales_full);
    }
  }
  __syncwarp();
}

// A loading warp's copies in flight: the ring slots it filled last and their phases.  After an
// abort it waits (bounded) for them before the CTA exits.
struct PgInFlight {
  uint32_t slots = 0, phases = 0;
  __device__ __forceinline__ void add(int slot, uint32_t phase) {
    slots |= 1u << slot;
    phases = (phases & ~(1u << slot)) | (phase << slot);
  }
  __device__ __forceinline__ void drain(uint64_t* full, int* status) const {
    for (uint32_t left = slots; left; left &= left - 1) {
      const int slot = __ffs(left) - 1;
      mbar_wait_drain(full + slot, (phases >> slot) & 1, status);
    }
  }
};

// The scale bytes of a lane's four keys of every tile of a segment in turn, fetched four tiles
// ahead: a fetch is two dependent reads of global memory.
struct PgScaleStream {
  uint32_t k[4], v[4], nk[4], nv[4];
  // the bytes of the lane's four keys of tile j; 2^0 for keys the unit does not see
  __device__ __forceinline__ static void fetch(const PgArgs& a, const PgSeg& g, int j, int lane, uint32_t& kw,
                                               uint32_t& vw) {
    kw = vw = 0x7f7f7f7fu;
    const int key = (j << 7) + lane * 4;
    if (key + 3 < g.keys.lo || key >= g.keys.hi) return;
    const int pg = key >> a.page_shift;
    const int id = pg < a.max_pages ? __ldg(a.table + static_cast<int64_t>(g.b) * a.max_pages + pg) : -1;
    if (id < 0 || id >= a.P) return;
    const int64_t at = (static_cast<int64_t>(id) * a.H_kv + g.kvh) * a.page + (key & (a.page - 1));
    if (!FA_IN_BOUNDS(at >= 0 && at + 4 <= static_cast<int64_t>(a.P) * a.H_kv * a.page, a.status, 511)) return;
    kw = __ldg(reinterpret_cast<const uint32_t*>(a.k_scales + at));
    vw = __ldg(reinterpret_cast<const uint32_t*>(a.v_scales + at));
  }
  // f(tile, key bytes, value bytes) for every tile; returns false to stop.
  template <typename F>
  __device__ __forceinline__ bool run(const PgArgs& a, const PgSeg& g, int lane, F f) {
    const int jend = g.kt0 + g.nt;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (g.kt0 + x < jend) fetch(a, g, g.kt0 + x, lane, nk[x], nv[x]);
    for (int j0 = g.kt0; j0 < jend; j0 += 4) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        k[x] = nk[x];
        v[x] = nv[x];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (j0 + 4 + x < jend) fetch(a, g, j0 + 4 + x, lane, nk[x], nv[x]);
#pragma unroll 1
      for (int x = 0; x < 4 && j0 + x < jend; ++x) {
        const uint32_t kw = x == 0 ? k[0] : (x == 1 ? k[1] : (x == 2 ? k[2] : k[3]));
        const uint32_t vw = x == 0 ? v[0] : (x == 1 ? v[1] : (x == 2 ? v[2] : v[3]));
        if (!f(j0 + x, kw, vw)) return false;
      }
    }
    return true;
  }
};

// The largest exponent of a tile's scale bytes (NaN apart) over the keys the unit sees, or -1000.
__device__ __forceinline__ int pg_top(const PgSeg& g, int j, int lane, uint32_t w) {
  int top = -1000;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int key = (j << 7) + lane * 4 + x;
    const int b = (w >> (8 * x)) & 255;
    if (key >= g.keys.lo && key < g.keys.hi && b != 255) top = max(top, b - 127);
  }
  return __reduce_max_sync(0xffffffffu, top);
}

// The factor 2^(byte - 127 - e) of a scale byte as fp32 and as fp16 bits; NaN for 255, and zero
// for what lies far below 2^e.
__device__ __forceinline__ float pg_factor(int byte, int e) {
  const int d = byte - 127 - e;
  return byte == 255 ? __uint_as_float(0x7fc00000u) : (d < -126 ? 0.f : __int_as_float((127 + d) << 23));
}
__device__ __forceinline__ uint32_t pg_factor16(int byte, int e) {
  const int d = min(byte - 127 - e, 0);
  return byte == 255 ? 0x7e00u : (d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : (d >= -24 ? 1u << (24 + d) : 0u));
}

// Sets value rows [z0, z1) of a tile to zero (one warp).  kRowBytes per chunk, kChunks chunks.
template <int kRowBytes, int kChunks>
__device__ __forceinline__ void pg_zero_rows(uint8_t* tile, int z0, int z1, int lane) {
  constexpr int kUnits = kRowBytes / 16;
  for (int u = lane; u < (z1 - z0) * kUnits * kChunks; u += 32) {
    const int c = u % kChunks, x = u / kChunks;
    *reinterpret_cast<uint4*>(tile + c * 128 * kRowBytes + z0 * kRowBytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ bool pg_cleans(const PgSeg& g, int j) {
  return g.keys.lo > j << 7 || g.keys.hi < (j + 1) << 7;
}

// Value rows of tile j that the unit does not see are zeroed: zero weights times stale infinities
// would not be zero (one warp, after the tile has landed).
template <int kRowBytes, int kChunks>
__device__ __forceinline__ void pg_clean(const PgSeg& g, int j, uint8_t* tile, int lane) {
  const int z0 = max(g.keys.lo - (j << 7), 0), z1 = min(g.keys.hi - (j << 7), 128);
  if (z0 > 0 || z1 < 128) {
    pg_zero_rows<kRowBytes, kChunks>(tile, 0, z0, lane);
    pg_zero_rows<kRowBytes, kChunks>(tile, z1, 128, lane);
    fence_proxy_async_smem();
    __syncwarp();
  }
}

// ---------------------------------------------------------------- queries for e4m3 pages
// Every query row is scaled by a power of two, 2^e the smallest with max|row| <= 448 * 2^e, and
//   kPieces   cut into that many e4m3 pieces, each the rounding of what the ones before it left:
//             two hold a bf16, three an fp16, exactly, down to 2^-18 of the row's largest
//   kHalf     written as fp16: exact for both types, down to 2^-33 of the row's largest
// Piece i of (token, head) lies at pieces[((i T + token) H + head) D], fp16 rows likewise at half; factors
// 2^e at q_scale[token H + head].  D / 16 lanes per row.
template <int D, Elem E, int kPieces, bool kHalf>
__global__ void __launch_bounds__(256) fa_paged_scale_q_kernel(const void* q, int64_t token_stride, int64_t head_stride,
                                                               uint8_t* pieces, uint8_t* half, float* q_scale, int T,
                                                               int H, int* status) {
  constexpr int L = D / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before it may still run
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / L;
  const int item = threadIdx.x % L;
  const bool live = row < static_cast<int64_t>(T) * H;
  const int64_t token = row / H;
  const int h = static_cast<int>(row - token * H);
  float f[16];
  float amax = 0.f;
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const typename ElemOps<E>::T*>(q) +
                                                      token * token_stride + h * head_stride + item * 16);
    const uint4 x0 = __ldg(src), x1 = __ldg(src + 1);
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = ElemOps<E>::unpack(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (fabsf(f[i]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(f[i]));
      else f[i] = __uint_as_float(0x7fc00000u);
    }
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = e4m3_exponent<Elem::kBf16>(amax);
  const float inv = __int_as_float((127 - e) << 23);
  if (!live || !FA_IN_BOUNDS(token < T && h < H && item * 16 + 16 <= D, status, 510)) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= inv;
  if constexpr (kHalf) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = pack_f16x2(f[2 * i], f[2 * i + 1]);
    uint4* dst = reinterpret_cast<uint4*>(half + (row * D + item * 16) * 2);
    dst[0] = make_uint4(c[0], c[1], c[2], c[3]);
    dst[1] = make_uint4(c[4], c[5], c[6], c[7]);
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = pack_e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      const float2 a = e4m3x2_to_float2(c[i]), b = e4m3x2_to_float2(c[i] >> 16);
      f[4 * i] -= a.x;
      f[4 * i + 1] -= a.y;
      f[4 * i + 2] -= b.x;
      f[4 * i + 3] -= b.y;
    }
    *reinterpret_cast<uint4*>(pieces + ((static_cast<int64_t>(p) * T + token) * H + h) * D + item * 16) =
        make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (item == 0) q_scale[row] = __int_as_float((127 + e) << 23);
}

// ---------------------------------------------------------------- joining the partial results
// Per row: LSE = log sum_s exp(lse_s) and O = sum_s exp(lr_s - LR) O_s with LR = log sum_s
// exp(lr_s), the convex combination one CTA would have formed.  Blocks (c, y) with c < `ctas` take
// the unit that CTA c began and did not finish; further blocks c = ctas + b give the rows of
// sequence b's units without keys O = 0, LSE = -inf.  All other rows were written by their CTA.  A mixed
// batch is joined by one launch, y below `many_y` the tiles' part, the others the few rows'.
//
// A warp takes 32 / L rows at a time: L lanes form the weights of a row's next L partial results,
// then all 32 lanes share each row's columns.  Tiles of 128 leave many rows of two or three partial
// results: L = 16 has two rows' loads in flight per chain of dependent loads (L = 8 / 16 / 32: a call
// with 2048 tokens at 32K 1042 / 1044 / 1098 us, one of 24 sequences of 30 rows 70.5 / 68.0 / 66.6).
// Few rows leave up to a hundred partial results: L = 32, and W warps share a row's.
template <int D, Elem E, typename Cfg, int L, int W, int kThreads>
__device__ __forceinline__ void pg_merge(const PgArgs& a, int ctas, int by, int ny, float (*acc_sh)[D]) {
  using T = typename ElemOps<E>::T;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int V = D / 32;       // columns per lane
  constexpr int R = 32 / L;       // rows per warp
  constexpr int kRowsAtOnce = kThreads / 32 / W * R;
  static_assert(W == 1 || (R == 1 && kThreads == 32 * W), "warps that share a row are a block");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = a.H / a.H_kv;
  if (static_cast<int>(blockIdx.x) >= ctas) {
    const int b = static_cast<int>(blockIdx.x) - ctas;
    const PgSeq s = pg_seq(a, b);
    // a token at a position >= 0 sees itself
    if (by > 0 || (s.len > 0 && (!a.causal || s.len >= s.n))) return;
    for (int u = 0; u < s.units; ++u) {
      const PgKeys k = pg_unit_keys(a, s, u);
      if (k.t1 > k.t0) continue;
      const int tok0 = u * 2 * a.TQ;
      const int rows = min(2 * a.TQ, s.n - tok0) * a.H;  // all key/value heads'
      for (int row = warp; row < rows; row += kThreads / 32) {
        const int64_t token = static_cast<int64_t>(s.q0) + tok0 + row / a.H;
        const int h = row % a.H;
        if (!FA_IN_BOUNDS(token >= 0 && token < a.T, a.status, 507)) continue;
        for (int c = lane; c < D; c += 32) static_cast<T*>(a.out)[(token * a.H + h) * D + c] = ElemOps<E>::one(0.f);
        if (lane == 0) a.lse[static_cast<int64_t>(h) * a.T + token] = -INFINITY;
      }
    }
    return;
  }
  const PgSplit sp = a.splits[blockIdx.x];
  const int rows = G * sp.ntok;
  if (sp.parts == 0) return;
  const int share = W > 1 ? warp : 0;
  // where a row lies in each partial result, and partial result i: the beginning is in its CTA's
  // second slot
  auto in_part = [&](int row) -> int {
    const int tile = row / (G * a.TQ);
    return tile * Cfg::kRows + row - tile * G * a.TQ;
  };
  auto part = [&](int i) -> int64_t {
    return static_cast<int64_t>(2 * (static_cast<int>(blockIdx.x) + i) + (i == 0)) * (Cfg::kSubs * Cfg::kRows);
  };
  for (int row0 = by * kRowsAtOnce + (W > 1 ? 0 : warp * R); row0 < rows; row0 += ny * kRowsAtOnce) {
    // this lane's row and partial results sl, sl + L, ..; behind the last row the last again, not stored
    const int mine_at = in_part(min(row0 + lane / L, rows - 1)), sl = lane % L;
    const float* po[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      po[r] = a.part_o + static_cast<int64_t>(__shfl_sync(kFull, mine_at, r * L)) * D + lane * V;
    float mx_l = -INFINITY, mx_r = -INFINITY, s_l = 0.f, s_r = 0.f;
    float2 mine = make_float2(-INFINITY, -INFINITY);  // of the lane's last partial result
    for (int i = sl; i < sp.parts; i += L) {
      const int64_t x = part(i) + mine_at;
      if (!FA_IN_BOUNDS(x >= 0 && x < a.slots * Cfg::kSubs * Cfg::kRows, a.status, 508)) continue;
      mine = *reinterpret_cast<const float2*>(a.part_lse + x * 2);
      mx_l = fmaxf(mx_l, mine.x);
      mx_r = fmaxf(mx_r, mine.y);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      mx_l = fmaxf(mx_l, __shfl_xor_sync(kFull, mx_l, o));
      mx_r = fmaxf(mx_r, __shfl_xor_sync(kFull, mx_r, o));
    }
    if (mx_l == -INFINITY) mx_l = 0.f;  // no key, or NaN only: the sums decide
    if (mx_r == -INFINITY) mx_r = 0.f;
    for (int i = sl; i < sp.parts; i += L) {
      if (sp.parts > L) mine = *reinterpret_cast<const float2*>(a.part_lse + (part(i) + mine_at) * 2);
      s_l += expf(mine.x - mx_l);
      s_r += expf(mine.y - mx_r);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      s_l += __shfl_xor_sync(kFull, s_l, o);
      s_r += __shfl_xor_sync(kFull, s_r, o);
    }
    float acc[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int x = 0; x < V; ++x) acc[r][x] = 0.f;
    const float inv = s_r == 0.f ? 0.f : 1.0f / s_r;
    for (int base = share * L; base < sp.parts; base += L * W) {
      // a partial result without keys was not written and is not read
      float wl = 0.f;
      if (base + sl < sp.parts) {
        const float v = sp.parts > L ? a.part_lse[(part(base + sl) + mine_at) * 2 + 1] : mine.y;
        wl = v == -INFINITY ? 0.f : expf(v - mx_r) * inv;
      }
      const int cnt = min(L, sp.parts - base);
#pragma unroll(R > 1 ? 1 : 4)
      for (int t = 0; t < cnt; ++t) {
        const int64_t from = part(base + t) * D;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float wgt = __shfl_sync(kFull, wl, r * L + t);
          if (wgt == 0.f) continue;
          if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(po[r] + from);
            acc[r][0] = fmaf(wgt, v.x, acc[r][0]);
            acc[r][1] = fmaf(wgt, v.y, acc[r][1]);
            acc[r][2] = fmaf(wgt, v.z, acc[r][2]);
            acc[r][3] = fmaf(wgt, v.w, acc[r][3]);
          } else {
            const float2 v = *reinterpret_cast<const float2*>(po[r] + from);
            acc[r][0] = fmaf(wgt, v.x, acc[r][0]);
            acc[r][1] = fmaf(wgt, v.y, acc[r][1]);
          }
        }
      }
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int x = 0; x < V; ++x) acc_sh[warp][lane * V + x] = acc[0][x];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int x = 0; x < V; ++x) {
          acc[0][x] = 0.f;
#pragma unroll
          for (int y = 0; y < W; ++y) acc[0][x] += acc_sh[y][lane * V + x];
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= rows) break;
      const int iq = (row0 + r) / G, h = sp.kvh * G + row0 + r - iq * G;
      const int64_t token = static_cast<int64_t>(sp.q0) + iq;
      if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H, a.status, 509)) {
        T* orow = static_cast<T*>(a.out) + (token * a.H + h) * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<uint2*>(orow) =
              make_uint2(ElemOps<E>::pack(acc[r][0], acc[r][1]), ElemOps<E>::pack(acc[r][2], acc[r][3]));
        else
          *reinterpret_cast<uint32_t*>(orow) = ElemOps<E>::pack(acc[r][0], acc[r][1]);
        if (lane == r * L) a.lse[static_cast<int64_t>(h) * a.T + token] = s_l == 0.f ? -INFINITY : mx_l + logf(s_l);
      }
    }
  }
}

// FewCfg, ManyCfg: the kernels of the call, void for one that it does not take.
template <int D, Elem E, typename FewCfg, typename ManyCfg, int kThreads>
__global__ void __launch_bounds__(kThreads) fa_paged_merge_kernel(const PgArgs few, const PgArgs many, int ctas, int many_y) {
  constexpr int W = kThreads / 32;
  __shared__ float acc_sh[W][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results are there
  const int y = static_cast<int>(blockIdx.y);
  if constexpr (!std::is_void_v<ManyCfg>) {
    if (y < many_y) {
      pg_merge<D, E, ManyCfg, 16, 1, kThreads>(many, ctas, y, many_y, nullptr);
      return;
    }
  }
  if constexpr (!std::is_void_v<FewCfg>)
    pg_merge<D, E, FewCfg, 32, W, kThreads>(few, ctas, y - many_y, static_cast<int>(gridDim.y) - many_y, acc_sh);
}

}  // namespace fa
