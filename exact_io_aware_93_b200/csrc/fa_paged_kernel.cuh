// fa_paged_kernel.cuh -- exact attention of the new tokens of every sequence of a ragged batch
// against that sequence's pages, for sm_100a.  One token (decoding), a few (drafted tokens) or
// a chunk of a prompt, mixed in one call.
//
// Rows.  The G = H / H_kv query heads of a key/value head and the new tokens form the rows
// r = i * G + g, so the cache is read once for all of them.  A TILE holds TQ = floor(128 / G)
// tokens (one TMA box of G heads x TQ tokens; rows past G * TQ are zero).  A UNIT is a pair of
// consecutive tiles of one (sequence, key/value head), or one tile when a sequence has no more.
//
// Work list.  A unit visits T = hi - lo tiles of 128 keys, those that some row of it sees
// (causal: up to its last token; window: from its first token's first key).  The key tiles of
// all units are laid end to end (sequence, key/value head, unit), each as long as it takes
// (PgCfg::kPairCost, kSplitCost), and CTA c of the persistent grid takes the tiles that start in
// [c L, (c+1) L), L = total / grid: every SM gets the same work whatever the mix of chunks,
// single tokens and lengths.  A CTA's run falls into SEGMENTS, each inside one unit; a segment
// that is not a whole unit leaves a partial result (O normalised, log-sums) that
// fa_paged_merge_kernel joins.  The lengths are read on the device, so a captured graph replays
// as they grow.
//
// Two ways through a segment, chosen per unit:
//   pair    two tiles: softmax group g owns tile g and both share one stream of K/V tiles, in
//           the order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1) of the forward kernel.
//   split   one tile: group g takes the segment's key tiles g, g + 2, ..: two independent
//           online softmaxes over disjoint keys, joined through shared memory at its end.
// Few rows (G * max_q <= 32, every unit split) use tiles that hold COPIES of the rows: copy c of
// R takes keys [c 128/R, (c+1) 128/R) of every tile, so a softmax warp handles 32 or 64 keys of a
// tile instead of 128 (see fa_decode_kernel.cuh).
//
// Pages.  A key tile is 128 / page boxes (or a part of one page), each fetched by its own lane
// of the producer warp; page numbers are read 32 at a time, one window ahead.  Pages that no row
// of the unit sees are not fetched, and value rows outside the unit's keys are zeroed in shared
// memory: stale slots, and pages a sliding window has left behind, may hold anything.
//
// e4m3 pages.  The tensor core takes the codes as they are (kind::f8f6f4): a tile moves half the
// bytes and K is never converted.  What is not e4m3 is cut into pieces that are, and the products
// of the pieces are summed:
//   Q   fa_paged_split_kernel writes q = 2^eq (q1 + q2), q1 the e4m3 rounding of q / 2^eq and q2
//       that of the rest: exact for bf16, 8 significant bits of an fp16's 11 (down to 2^-18 of
//       the row's largest).  A third piece would cost half as many products again for bits that
//       the cache's own 4-bit significands bury.
//   P   with few rows: the weight, an fp16 value rounded to 9 bits, is the sum of three e5m2
//       pieces (e5m2 is the upper byte of an fp16): relative error 2^-9 down to 2^-23 of the
//       largest weight.  e5m2 and not e4m3 for its range: a long tail of small weights beside a
//       large one keeps its mass.
//   V   with tiles of 128 rows the pieces would cost the softmax warps more than its exponentials,
//       so there a fourth warpgroup turns V's codes into fp16 tiles, code * 2^(ev - E) (exact),
//       and P is one fp16 operand for both element types.
// The scales: S_j is multiplied by 2^ek_j, and P or V by 2^(ev_j - E), E the segment's largest
// value exponent so far (O is rescaled when it grows).  Warps 10 and 11 fetch the scale bytes and
// expand them into small rings.  (Converting K and V of every tile to 16 bits bounded the kernel:
// 2116 cycles a tile and a bf16 result, where fetching one takes 700.)
//   Up to 8 rows  each row takes 4 of a warp's lanes, 8 apart: the rows of the pieces q1 and q2
//       give partial scores that a shuffle adds, and each lane stores one piece of P: 4 + 4
//       products of 64 cycles per tile instead of 8 + 12.
//
// Warp roles (384 threads, 512 with e4m3 pages and tiles of 128 rows): warps 0-3 and 4-7 the
// softmax groups, warp 8 the schedule and the TMA loads, warp 9 the MMA issuer, warps 10-11 the
// scales, warps 12-15 the conversion of V.  Warp 8 writes each segment into a small ring that all
// others follow.
// Tensor memory: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 [256+D,256+2D); P overwrites S.
#pragma once

#include "fa_cache_kernels.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

constexpr uint32_t kPagedLaunchRegs = 168;      // 16-bit pages, tiles of 128 rows
constexpr uint32_t kPagedLaunchRegsConv = 128;  // e4m3 pages, tiles of 128 rows
constexpr int kPPieces = 3;                     // e5m2 pieces of a weight
constexpr float kPShift = 7.0f;                 // weights cut into pieces are 2^(x - m + 7) <= 2^15

// R = 0: tiles of 128 rows, both ways; R = 2, 4: one tile of 64 rows holding R copies of up to 32
// or 16 rows; R = 8 (e4m3 pages): 128 rows holding 4 copies of up to 8 rows, 4 lanes each.
template <int D, Elem E, bool Q8, int R>
struct PgCfg {
  static constexpr bool kGeneral = R == 0;
  static constexpr bool kConv = Q8 && kGeneral;       // V as fp16 tiles
  static constexpr int kSlots = R == 8 ? 4 : 1;       // lanes of a row
  static constexpr int kCopies = kGeneral ? 1 : (R == 8 ? 4 : R);
  static constexpr int kM = (kGeneral || R == 8) ? 128 : 64;
  static constexpr int kRows = kM / kCopies / kSlots; // rows of a partial result
  static constexpr int kSubs = kGeneral ? 2 : 1;      // partial results per segment
  static constexpr int kStageCols = kGeneral ? 16 : 32;  // columns joined at a time
  static constexpr int kStageRows = kGeneral ? 128 : 2 * kCopies * kRows;
  static constexpr int kThreads = kConv ? 512 : 384;
  // setmaxnreg, tiles of 128 rows only: 2 x 128 x 200 + 128 x 104 of 384 x 168, and with the
  // conversion warps 128 x (2 x 184 + 72 + 72) of 512 x 128
  static constexpr uint32_t kLaunch = kConv ? kPagedLaunchRegsConv : kPagedLaunchRegs;
  static constexpr uint32_t kRegsSoftmax = kConv ? 184 : 200;
  static constexpr uint32_t kRegsOther = kConv ? 72 : 104;
  static_assert(2 * kRegsSoftmax + (kConv ? 2 : 1) * kRegsOther <= kLaunch * (kThreads / 128), "register split");
  // time of a key tile, in the work list's units: of a pair, and of a single tile
  static constexpr int kPairCost = kConv ? 5 : 3;
  static constexpr int kSplitCost = 2;
  // a row in shared memory: 128-byte chunks of 64 16-bit elements, or D codes (D = 64 in the
  // 64-byte swizzle)
  static constexpr int kRowBytes = Q8 ? D : 128;
  static constexpr int kChunks = Q8 ? 1 : D / 64;
  static constexpr int kChunkBytes = 128 * kRowBytes;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kQParts = Q8 ? (R == 8 ? 1 : 2) : D / 64;  // pieces, or chunks
  static constexpr int kQPartBytes = kM * kRowBytes;
  static constexpr int kQBytes = kQParts * kQPartBytes;
  static constexpr int kScale = 128 / D;              // slots scale with the tile
  // the ring of K and V tiles, or of K tiles beside V's codes and fp16 tiles
  static constexpr int kStages = (kConv ? 2 : (Q8 ? 8 : 4)) * kScale;
  static constexpr int kVRaw = kConv ? 2 * kScale : 1;
  static constexpr int kV16 = kConv ? 2 * kScale : 1;
  static constexpr int kV16Bytes = kConv ? 128 * D * 2 : 16;
  static constexpr int kScaleRing = 4;
  static constexpr int kSegRing = 4;
  static constexpr int kSegReaders = 9 + (Q8 ? 2 : 0) + (kConv ? 4 : 0);  // warps
  static constexpr int kPArrive = kGeneral ? 128 : 4;
  static constexpr uint32_t kOCol = 256;
  static constexpr uint32_t kTmemCols = 512;
};

struct PgArgs {
  const int* cu;          // [B + 1]
  const int* seqlens;     // [B]
  const int* table;       // [B, max_pages]
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const float* q_scale;   // e4m3 pages: [T, H] factors of the query pieces
  void* out;              // [T, H, D]
  float* lse;             // [H, T]
  int* meta;              // total, L, unit prefix [B + 1], key-tile prefix [B + 1]
  float* part_lse;        // [slots * kSubs, kRows, 2]
  float* part_o;          // [slots * kSubs, kRows, D]
  int B, T, H, H_kv, max_q, TQ, max_pages, page, page_shift, P, window, causal;
  float scale_log2;
  long long slots;        // 2 per CTA
  int* status;
};

// ---------------------------------------------------------------- the work list
struct PgSeq {
  int q0, n, len, units;
};
__device__ __forceinline__ PgSeq pg_seq(const PgArgs& a, int b) {
  const long long c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  PgSeq s;
  const bool in = c0 >= 0 && c0 <= a.T && c1 > c0;
  s.q0 = in ? static_cast<int>(c0) : 0;
  s.n = in ? static_cast<int>(min(min(c1 - c0, static_cast<long long>(a.max_q)), a.T - c0)) : 0;
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  s.len = static_cast<int>(min(max(static_cast<long long>(__ldg(a.seqlens + b)), 0ll), cap));
  s.units = ((s.n + a.TQ - 1) / a.TQ + 1) / 2;
  return s;
}
__device__ __forceinline__ bool pg_seq_ok(const PgArgs& a, int b) {
  const long long c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  const long long len = __ldg(a.seqlens + b);
  return c0 >= 0 && c1 >= c0 && c1 <= a.T && c1 - c0 <= a.max_q && len >= 0 &&
         len <= static_cast<long long>(a.max_pages) * a.page;
}

// Keys [lo, hi) that the tokens at positions p0 .. p1 of a sequence of `len` keys see, and the
// key tiles that hold them.
struct PgKeys {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ PgKeys pg_keys(const PgArgs& a, int len, int p0, int p1) {
  PgKeys k;
  k.hi = a.causal ? min(p1 + 1, len) : len;
  k.lo = a.window >= 0 ? max(0, p0 - a.window) : 0;
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

// Cost of a sequence's units for one key/value head.
template <typename Cfg>
__device__ __forceinline__ int pg_seq_cost(const PgArgs& a, const PgSeq& s) {
  int w = 0;
  for (int u = 0; u < s.units; ++u) {
    const PgKeys k = pg_unit_keys(a, s, u);
    w += (k.t1 - k.t0) * (pg_is_pair(a, s, u) ? Cfg::kPairCost : Cfg::kSplitCost);
  }
  return w;
}

// This CTA's slice [t0, t1) of the work and the unit that t0 falls into, which starts at `start`.
struct PgPlan {
  int t0, t1, b, kvh, u, start;
};

// One warp.  With `write` it also stores the prefixes for the merge kernel and checks the
// lengths and offsets.
template <typename Cfg>
__device__ __forceinline__ void pg_plan(const PgArgs& a, int lane, PgPlan* out, bool write) {
  constexpr unsigned kFull = 0xffffffffu;
  int total = 0;
  PgSeq s{0, 0, 0, 0};
  int w = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    s = PgSeq{0, 0, 0, 0};
    if (b < a.B) s = pg_seq(a, b);
    w = pg_seq_cost<Cfg>(a, s);
    total += static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(w * a.H_kv)));
  }
  const int grid = static_cast<int>(gridDim.x);
  // at least a tile's cost, so that no CTA inside a unit's span is left without one of its tiles
  const int per = max((total + grid - 1) / grid, Cfg::kPairCost);
  const int t0 = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(blockIdx.x) * per));
  const int t1 = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(t0) + per));
  bool found = t0 >= t1;
  if (found && lane == 0) *out = PgPlan{t0, t0, 0, 0, 0, t0};
  int acc = 0, uacc = 0;
  for (int b0 = 0; b0 < a.B && (!found || write); b0 += 32) {
    const int b = b0 + lane;
    if (a.B > 32) {  // up to 32 sequences are still at hand
      s = PgSeq{0, 0, 0, 0};
      if (b < a.B) s = pg_seq(a, b);
      w = pg_seq_cost<Cfg>(a, s);
    }
    if (write && b < a.B && !pg_seq_ok(a, b)) plan_fail(a.status, 43);
    int incl = w * a.H_kv, uincl = s.units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o), y = __shfl_up_sync(kFull, uincl, o);
      if (lane >= o) {
        incl += x;
        uincl += y;
      }
    }
    incl += acc;
    uincl += uacc;
    const int excl = incl - w * a.H_kv;
    if (write && b < a.B) {
      a.meta[2 + b + 1] = uincl;
      a.meta[2 + a.B + 1 + b + 1] = incl;
    }
    if (!found && b < a.B && excl <= t0 && t0 < incl) {  // one lane
      const int kvh = (t0 - excl) / w;
      int start = excl + kvh * w, u = 0;
      while (true) {
        const PgKeys k = pg_unit_keys(a, s, u);
        const int c = (k.t1 - k.t0) * (pg_is_pair(a, s, u) ? Cfg::kPairCost : Cfg::kSplitCost);
        if (t0 < start + c) break;
        start += c;
        ++u;
      }
      *out = PgPlan{t0, t1, b, kvh, u, start};
    }
    found = found || (t0 < __shfl_sync(kFull, incl, 31));
    acc = __shfl_sync(kFull, incl, 31);
    uacc = __shfl_sync(kFull, uincl, 31);
  }
  if (write && lane == 0) {
    a.meta[0] = total;
    a.meta[1] = per;
    a.meta[2] = 0;
    a.meta[2 + a.B + 1] = 0;
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

// Walks this CTA's slice segment by segment (the schedule's warp, every lane alike).
template <typename Cfg>
struct PgWalk {
  int t0, t1, b, kvh, u, start;
  PgSeq s;
  __device__ __forceinline__ PgWalk(const PgArgs& a, const PgPlan& p)
      : t0(p.t0), t1(p.t1), b(p.b), kvh(p.kvh), u(p.u), start(p.start), s(pg_seq(a, p.b)) {}
  __device__ __forceinline__ bool next(const PgArgs& a, PgSeg& g) {
    while (start < t1) {
      if (u >= s.units) {
        u = 0;
        if (s.units == 0 || ++kvh >= a.H_kv) {
          kvh = 0;
          if (++b >= a.B) return false;
          s = pg_seq(a, b);
        }
        continue;
      }
      const PgKeys k = pg_unit_keys(a, s, u);
      const bool pair = pg_is_pair(a, s, u);
      const int cost = pair ? Cfg::kPairCost : Cfg::kSplitCost;
      const int T = k.t1 - k.t0;
      // the tiles that start in [t0, t1)
      const int first = t0 > start ? (t0 - start + cost - 1) / cost : 0;
      const int last = min(T, (t1 - start + cost - 1) / cost);
      const int tok0 = u * 2 * a.TQ;
      start += T * cost;
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
// K_0, K_1, V_0, K_2, V_1, ..  f(is_value, tile) returns false to stop.
template <typename F>
__device__ __forceinline__ bool pg_loads(const PgSeg& g, F f) {
  if (g.pair) {
    for (int t = 0; t < g.nt; ++t)
      if (!f(false, g.kt0 + t) || !f(true, g.kt0 + t)) return false;
    return true;
  }
  if (!f(false, g.kt0) || (g.nt > 1 && !f(false, g.kt0 + 1))) return false;
  for (int t = 0; t < g.nt; ++t)
    if (!f(true, g.kt0 + t) || (t + 2 < g.nt && !f(false, g.kt0 + t + 2))) return false;
  return true;
}

// ---------------------------------------------------------------- e4m3 pages
// The two pieces of every query row: piece i of (token, head) at pieces[((i T + token) H + head) D],
// factors q_scale[token H + head].  L = D / 16 lanes per row.
template <int D, Elem E>
__global__ void __launch_bounds__(256) fa_paged_split_kernel(const void* q, int64_t token_stride, int64_t head_stride,
                                                             uint8_t* pieces, float* q_scale, int T, int H,
                                                             int* status) {
  constexpr int L = D / 16;
  constexpr int kPieces = 2;
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
  // the bf16 rule of the cache for both types: e4m3's largest is 448, 2^e <= 2^119
  const int e = e4m3_exponent<Elem::kBf16>(amax);
  const float inv = __int_as_float((127 - e) << 23);
  if (!live || !FA_IN_BOUNDS(token < T && h < H && item * 16 + 16 <= D, status, 510)) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= inv;
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

// Four weights (an fp16 pair of pairs) to the three words of their e5m2 pieces.  The fp16 values
// are rounded to 9 significant bits; the upper byte of an fp16 is its e5m2 truncation, and each
// remainder is exact in fp16.
__device__ __forceinline__ void split_e5m2(uint32_t a, uint32_t b, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  a += 0x00020002u;
  b += 0x00020002u;
  p0 = __byte_perm(a, b, 0x7531);
  uint32_t ra, rb;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(a & 0xff00ff00u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rb) : "r"(b), "r"(b & 0xff00ff00u));
  p1 = __byte_perm(ra, rb, 0x7531);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(ra), "r"(ra & 0xff00ff00u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(rb), "r"(rb & 0xff00ff00u));
  p2 = __byte_perm(a, b, 0x7531);
}

// Weights of one score row of NC keys, 2^(s * c - m), times the value factors vs[] (shared
// memory), as e5m2 pieces p[piece], four keys per word; l gets the fp32 sum of the weights.
template <int NC>
__device__ __forceinline__ void softmax_row_f8(const uint32_t (&s)[NC], const float* vs,
                                               uint32_t (&p)[kPPieces][NC / 4], float c, float m, float& l) {
  const float2 c2 = make_float2(c, c), nm2 = make_float2(-m, -m);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < NC / 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(vs)[i];
    const float2 x = ffma2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), c2, nm2);
    const float2 y = ffma2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), c2, nm2);
    const float2 e0 = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    const float2 e1 = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    sum[0] = fadd2(sum[0], e0);
    sum[1] = fadd2(sum[1], e1);
    const float2 w0 = fmul2(e0, make_float2(f.x, f.y)), w1 = fmul2(e1, make_float2(f.z, f.w));
    split_e5m2(pack_f16x2(w0.x, w0.y), pack_f16x2(w1.x, w1.y), p[0][i], p[1][i], p[2][i]);
  }
  l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The factor 2^(byte - 127 - e) of a value's scale byte as fp32 and as fp16 bits; NaN for 255.
__device__ __forceinline__ float pg_factor(int byte, int e) {
  const int d = byte - 127 - e;  // <= 0 unless NaN; far below the largest is zero
  return byte == 255 ? __uint_as_float(0x7fc00000u) : (d < -126 ? 0.f : __int_as_float((127 + d) << 23));
}
__device__ __forceinline__ uint32_t pg_factor16(int byte, int e) {
  const int d = byte - 127 - e;
  return byte == 255 ? 0x7e00u : (d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : (d >= -24 ? 1u << (24 + d) : 0u));
}

// Sixteen codes times an fp16 factor (twice in f), in order.
__device__ __forceinline__ void pg_convert16(const uint4& c, uint32_t f, uint32_t (&o)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 x, y;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, lo;\n\tcvt.rn.f16x2.e4m3x2 y, hi;\n\t"
        "mul.rn.f16x2 %0, x, %3;\n\tmul.rn.f16x2 %1, y, %3;\n\t}"
        : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
        : "r"(w[i]), "r"(f));
}

// Scale factors of one key tile: of the scores, and of the weights (or, for V's conversion, fp16
// factors of the rows) relative to 2^e.
struct PgScales {
  float ks[128];
  float vs[128];
  int e;
  int pad[3];
};
struct PgVScales {
  uint32_t f[128];
};

// ---------------------------------------------------------------- the kernel
template <int D, Elem E, bool Q8, int R>
struct __align__(1024) PgSmem {
  using Cfg = PgCfg<D, E, Q8, R>;
  uint8_t q[2][Cfg::kQBytes];
  uint8_t kv[Cfg::kStages][Cfg::kTileBytes];
  uint8_t v16[Cfg::kV16][Cfg::kConv ? Cfg::kV16Bytes : 16];
  uint8_t vraw[Cfg::kVRaw][Cfg::kConv ? Cfg::kTileBytes : 16];
  alignas(16) float stage[2][Cfg::kStageRows * Cfg::kStageCols];  // a split segment's columns being joined
  PgScales scales[2][Q8 ? Cfg::kScaleRing : 1];       // of each softmax group's tiles
  PgVScales vscales[Cfg::kConv ? Cfg::kScaleRing : 1];
  float3 stat[2 * Cfg::kCopies][Cfg::kRows];          // m, l, lr of a split segment's copies
  PgSeg segs[Cfg::kSegRing];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t kv_full[Cfg::kStages];
  uint64_t kv_empty[Cfg::kStages];
  uint64_t vraw_full[Cfg::kVRaw];
  uint64_t vraw_empty[Cfg::kVRaw];
  uint64_t v16_full[Cfg::kV16];
  uint64_t v16_empty[Cfg::kV16];
  uint64_t sc_full[2][Cfg::kScaleRing];
  uint64_t sc_empty[2][Cfg::kScaleRing];
  uint64_t vsc_full[Cfg::kScaleRing];
  uint64_t vsc_empty[Cfg::kScaleRing];
  uint64_t seg_full[Cfg::kSegRing];
  uint64_t seg_empty[Cfg::kSegRing];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_done[2];
  uint64_t groups;  // both softmax groups, at the end of a split segment
  uint64_t mma_drain;
  PgPlan plan;
  uint32_t tmem_base;
  int abort_flag;
};

// Sets value rows [z0, z1) of a tile to zero (one warp).  kRowBytes per chunk, kChunks chunks.
template <int kRowBytes, int kChunks>
__device__ __forceinline__ void pg_zero_rows(uint8_t* tile, int z0, int z1, int lane) {
  constexpr int kUnits = kRowBytes / 16;
  for (int u = lane; u < (z1 - z0) * kUnits * kChunks; u += 32) {
    const int c = u % kChunks, x = u / kChunks;
    *reinterpret_cast<uint4*>(tile + c * 128 * kRowBytes + z0 * kRowBytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D, Elem E, bool Q8, int R>
__global__ void __launch_bounds__(PgCfg<D, E, Q8, R>::kThreads, 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PgArgs a) {
  using Cfg = PgCfg<D, E, Q8, R>;
  constexpr int NS = Cfg::kStages;
  constexpr int NSC = Cfg::kScaleRing;
  constexpr int NSEG = Cfg::kSegRing;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  PgSmem<D, E, Q8, R>& sm = *reinterpret_cast<PgSmem<D, E, Q8, R>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                                    ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = a.H / a.H_kv;
  int* status = a.status;

  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], Cfg::kPArrive);
      mbar_init(&sm.o_done[i], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    if constexpr (Q8) {
      for (int s = 0; s < NSC; ++s) {
        for (int i = 0; i < 2; ++i) {
          mbar_init(&sm.sc_full[i][s], 1);
          mbar_init(&sm.sc_empty[i][s], 4);
        }
        mbar_init(&sm.vsc_full[s], 1);
        mbar_init(&sm.vsc_empty[s], 4);
      }
    }
    if constexpr (Cfg::kConv) {
      for (int s = 0; s < Cfg::kVRaw; ++s) {
        mbar_init(&sm.vraw_full[s], 1);
        mbar_init(&sm.vraw_empty[s], 4);
      }
      for (int s = 0; s < Cfg::kV16; ++s) {
        mbar_init(&sm.v16_full[s], 4);
        mbar_init(&sm.v16_empty[s], 1);
      }
    }
    for (int s = 0; s < NSEG; ++s) {
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], Cfg::kSegReaders);
    }
    mbar_init(&sm.groups, 8);
    mbar_init(&sm.mma_drain, 1);
    fence_mbar_init();
  }
  // rows of a query tile that hold no query are never loaded
  for (uint32_t i = threadIdx.x; i < 2u * Cfg::kQBytes / 16; i += Cfg::kThreads)
    reinterpret_cast<uint4*>(sm.q[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, Cfg::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    pg_plan<Cfg>(a, lane, &sm.plan, blockIdx.x == 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;

  // Readers of the segment ring: the next segment, or null at the end or after an abort; a
  // reader gives the one it holds back first.
  uint32_t nseg = 0;
  auto next_seg = [&](const WaitCtx& wc) -> const PgSeg* {
    if (nseg > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_empty[(nseg - 1) % NSEG]);
    }
    const int i = nseg % NSEG;
    if (!__all_sync(kFull, mbar_wait(&sm.seg_full[i], (nseg / NSEG) & 1, wc))) return nullptr;
    ++nseg;
    return sm.segs[i].nt > 0 ? &sm.segs[i] : nullptr;
  };

  // Each warpgroup's setmaxnreg sits at the top of the branch holding all of its code.
  if (warp >= 8 && warp < 12) {
    if constexpr (Cfg::kGeneral) regs_set<Cfg::kLaunch, Cfg::kRegsOther>();
    if (warp == 8) {
      // ---------------------------------------------------------- schedule and TMA loads
      const WaitCtx wc{&sm.abort_flag, status, 31};
      PgWalk<Cfg> w(a, sm.plan);
      PgSeg g;
      uint32_t it = 0, itv = 0, qcnt[2] = {0, 0};
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait(bar, parity, wc)); };
      auto load_q = [&](int slot, int tok) -> bool {
        if (!wait_all(&sm.q_empty[slot], (qcnt[slot] & 1) ^ 1)) return false;
        // a box per copy and chunk or piece; with four lanes a row, the pieces go to the row
        // blocks of a copy in turn
        constexpr int kBoxes = Cfg::kCopies * (Cfg::kSlots > 1 ? Cfg::kSlots : Cfg::kQParts);
        if (lane == 0)
          mbar_arrive_expect_tx(&sm.q_full[slot], static_cast<uint32_t>(kBoxes * Cfg::kRowBytes * G * a.TQ));
        __syncwarp();
        if (lane < kBoxes) {
          const int cp = lane % Cfg::kCopies, x = lane / Cfg::kCopies;
          const int part = Cfg::kSlots > 1 ? 0 : x;
          const int row = (cp * Cfg::kSlots + (Cfg::kSlots > 1 ? x : 0)) * Cfg::kRows;
          const int piece = Cfg::kSlots > 1 ? x & 1 : x;
          if (FA_IN_BOUNDS(tok >= 0 && tok < a.T && g.kvh < a.H_kv && G * a.TQ <= Cfg::kRows, status, 501))
            tma_load_4d(sm.q[slot] + part * Cfg::kQPartBytes + row * Cfg::kRowBytes, &tm_q, &sm.q_full[slot],
                        Q8 ? 0 : part * 64, 0, g.kvh, Q8 ? piece * a.T + tok : tok);
        }
        __syncwarp();
        ++qcnt[slot];
        return true;
      };
      const int box = min(128, a.page);  // keys per box
      // page numbers of windows of 32 table entries: the even and the odd one held, one ahead
      int id_even = -1, id_odd = -1, ahead = -1, window_at = -1;
      auto entry = [&](int win) {
        const long long i = static_cast<long long>(win) * 32 + lane;
        return i < a.max_pages ? __ldg(a.table + static_cast<long long>(g.b) * a.max_pages + i) : -1;
      };
      while (ok) {
        const int i = nseg % NSEG;
        const bool more = w.next(a, g);
        if (more) ahead = entry(((g.kt0 << 7) >> a.page_shift) >> 5);
        ok = wait_all(&sm.seg_empty[i], ((nseg / NSEG) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          if (!more) g.nt = 0;
          sm.segs[i] = g;
          mbar_arrive(&sm.seg_full[i]);
        }
        ++nseg;
        if (!more) break;
        if (Cfg::kGeneral && g.pair) {
          for (int x = 0; x < 2 && ok; ++x)
            if (g.tile[x].hi > g.tile[x].lo) ok = load_q(x, g.q0 + x * a.TQ);
        } else {
          ok = load_q(Cfg::kGeneral ? 0 : ((nseg - 1) & 1), g.q0);
        }
        if (!ok) break;
        window_at = (((g.kt0 << 7) >> a.page_shift) >> 5) - 1;
        ok = pg_loads(g, [&](bool isv, int j) -> bool {
          const int p0 = (j << 7) >> a.page_shift;  // the tile's first page
          if ((p0 >> 5) > window_at) {              // keys run at most two tiles ahead of values
            window_at = p0 >> 5;
            if (window_at & 1) id_odd = ahead; else id_even = ahead;
            ahead = entry(window_at + 1);
          }
          // the boxes that hold a key of the unit
          const int k0 = max(g.keys.lo - (j << 7), 0) / box;
          const int k1 = (min(g.keys.hi - (j << 7), 128) + box - 1) / box;
          const bool raw = Cfg::kConv && isv;
          const int n = raw ? Cfg::kVRaw : NS;
          uint32_t& cnt = raw ? itv : it;
          const int slot = cnt % n;
          uint64_t* full = raw ? &sm.vraw_full[slot] : &sm.kv_full[slot];
          if (!wait_all(raw ? &sm.vraw_empty[slot] : &sm.kv_empty[slot], ((cnt / n) & 1) ^ 1)) return false;
          if (lane == 0)
            mbar_arrive_expect_tx(full, static_cast<uint32_t>((k1 - k0) * box * Cfg::kRowBytes * Cfg::kChunks));
          __syncwarp();
          const int k = k0 + lane / Cfg::kChunks, c = lane % Cfg::kChunks;
          const int held = (p0 >> 5) & 1 ? id_odd : id_even;
          const int id = __shfl_sync(kFull, held, (p0 + k) & 31);
          if (k < k1) {
            const int row = (j << 7) & (a.page - 1) & ~(box - 1);  // inside a page of 256
            const bool good = id >= 0 && id < a.P;
            if (!good) plan_fail(status, 44);
            uint8_t* dst = raw ? sm.vraw[slot] : sm.kv[slot];
            // a bad page number reads as zeros: a coordinate past the pool
            if (FA_IN_BOUNDS(row + box <= a.page && p0 + k < a.max_pages && k * box < 128, status, 502))
              tma_load_3d(dst + c * Cfg::kChunkBytes + k * box * Cfg::kRowBytes, isv ? &tm_v : &tm_k, full, c * 64, row,
                          good ? id * a.H_kv + g.kvh : a.P * a.H_kv);
          }
          __syncwarp();
          ++cnt;
          return true;
        });
      }
      if (!ok && lane == 0) {
        // Unwinding: wait (bounded) for the copies still in flight before the CTA exits.
        for (uint32_t idx = (it > static_cast<uint32_t>(NS) ? it - NS : 0); idx < it; ++idx)
          mbar_wait_drain(&sm.kv_full[idx % NS], (idx / NS) & 1, status);
        constexpr uint32_t NV = Cfg::kVRaw;
        for (uint32_t idx = (itv > NV ? itv - NV : 0); idx < itv; ++idx)
          mbar_wait_drain(&sm.vraw_full[idx % NV], (idx / NV) & 1, status);
        for (int i = 0; i < 2; ++i)
          if (qcnt[i] > 0) mbar_wait_drain(&sm.q_full[i], (qcnt[i] - 1) & 1, status);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer (whole warp)
      const WaitCtx wc{&sm.abort_flag, status, 32};
      // Q, K K-major; P in TMEM, V MN-major
      constexpr uint32_t idesc_s =
          Q8 ? idesc_kind_f8(Cfg::kM, kBN, 0, 0, 0) : idesc_kind_f16(Cfg::kM, kBN, 0, 0, ElemOps<E>::kMmaType);
      constexpr bool kPieces = Q8 && !Cfg::kConv;  // P as e5m2 pieces, V as codes
      constexpr uint32_t idesc_o = kPieces ? idesc_kind_f8(Cfg::kM, D, 0, 1, 1)
                                           : idesc_kind_f16(Cfg::kM, D, 0, 1, Cfg::kConv ? 0 : ElemOps<E>::kMmaType);
      constexpr uint32_t kGroup = 8 * Cfg::kRowBytes;  // 8-row groups
      auto desc = [](const void* p, uint32_t lbo, uint32_t sbo) {
        return Cfg::kRowBytes == 64 ? sdesc_sw64(smem_u32(p), lbo, sbo) : sdesc_sw128(smem_u32(p), lbo, sbo);
      };
      const uint64_t dq[2] = {desc(sm.q[0], 16, kGroup), desc(sm.q[1], 16, kGroup)};
      const uint64_t dk0 = desc(sm.kv[0], 16, kGroup);
      const uint64_t dv0 = Cfg::kConv ? sdesc_sw128(smem_u32(sm.v16[0]), 128 * 128, 1024)
                                      : desc(sm.kv[0], Cfg::kChunkBytes, kGroup);
      constexpr int kVBytes = Cfg::kConv ? Cfg::kV16Bytes : Cfg::kTileBytes;
      auto issue_s = [&](int i, int qs, int slot) {
        const uint64_t dk = dk0 + static_cast<uint64_t>((slot * Cfg::kTileBytes) >> 4);
        const uint64_t dqi = qs ? dq[1] : dq[0];
        if constexpr (Q8) {
#pragma unroll
          for (int p = 0; p < Cfg::kQParts; ++p)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_ss_f8_w(tbase + i * 128, dqi + ((p * Cfg::kQPartBytes + kk * 32) >> 4), dk + ((kk * 32) >> 4),
                           idesc_s, p + kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss_w(tbase + i * 128, dqi + (((kk / 4) * Cfg::kQPartBytes + (kk % 4) * 32) >> 4),
                      dk + (((kk / 4) * Cfg::kChunkBytes + (kk % 4) * 32) >> 4), idesc_s, kk > 0);
        }
      };
      auto issue_pv = [&](int i, int slot, uint32_t acc) {
        const uint64_t dv = dv0 + static_cast<uint64_t>((slot * kVBytes) >> 4);
        const uint32_t tO = tbase + Cfg::kOCol + i * D, tP = tbase + i * 128;
        if constexpr (kPieces) {
#pragma unroll
          for (int p = 0; p < (Cfg::kSlots > 1 ? 1 : kPPieces); ++p)
#pragma unroll
            for (int kk = 0; kk < kBN / 32; ++kk)
              umma_ts_f8_w(tO, tP + p * 32 + kk * 8, dv + ((kk * 32 * Cfg::kRowBytes) >> 4), idesc_o,
                           (p + kk > 0) || acc);
        } else {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            umma_ts_w(tO, tP + kk * 8, dv + ((kk * 16 * 128) >> 4), idesc_o, (kk > 0) || acc);
        }
      };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait(bar, parity, wc)); };
      uint32_t it = 0, itv = 0, qcnt[2] = {0, 0}, pcnt[2] = {0, 0};
      bool ok = true;
      int slot = 0;
      auto take_k = [&]() -> bool {
        slot = it % NS;
        const bool r = wait_all(&sm.kv_full[slot], (it / NS) & 1);
        ++it;
        return r;
      };
      auto take_v = [&]() -> bool {
        if constexpr (!Cfg::kConv) return take_k();
        slot = itv % Cfg::kV16;
        const bool r = wait_all(&sm.v16_full[slot], (itv / Cfg::kV16) & 1);
        ++itv;
        return r;
      };
      auto free_v = [&](int sv) { umma_commit_w(Cfg::kConv ? &sm.v16_empty[sv] : &sm.kv_empty[sv]); };
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        const int kt0 = g.kt0, nt = g.nt;
        // value rows of tile j that the unit does not see are zeroed: zero weights times stale
        // infinities would not be zero (the conversion does it for its fp16 tiles)
        auto clean = [&](int sv, int j) {
          if constexpr (!Cfg::kConv) {
            const int z0 = max(g.keys.lo - (j << 7), 0), z1 = min(g.keys.hi - (j << 7), 128);
            if (z0 > 0 || z1 < 128) {
              pg_zero_rows<Cfg::kRowBytes, Cfg::kChunks>(sm.kv[sv], 0, z0, lane);
              pg_zero_rows<Cfg::kRowBytes, Cfg::kChunks>(sm.kv[sv], z1, 128, lane);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
        };
        if (Cfg::kGeneral && g.pair) {
          const PgRange rg[2] = {g.tile[0], g.tile[1]};
          const int jhi = kt0 + nt;
          auto in = [&](int i, int j) { return j >= rg[i].lo && j < rg[i].hi; };
          for (int i = 0; i < 2 && ok; ++i)
            if (rg[i].hi > rg[i].lo) ok = wait_all(&sm.q_full[i], qcnt[i] & 1);
          if (!ok) break;
          ok = take_k();
          if (!ok) break;
          tc_fence_after();
          for (int i = 0; i < 2; ++i) {
            if (!in(i, kt0)) continue;
            issue_s(i, i, slot);
            umma_commit_w(&sm.s_full[i]);
            if (rg[i].hi == kt0 + 1) umma_commit_w(&sm.q_empty[i]);
          }
          umma_commit_w(&sm.kv_empty[slot]);
          for (int j = kt0; j < jhi && ok; ++j) {
            ok = take_v();
            if (!ok) break;
            const int sv = slot;
            clean(sv, j);
            int skn = -1;
            if (j + 1 < jhi) {
              ok = take_k();
              if (!ok) break;
              skn = slot;
            }
            for (int i = 0; i < 2 && ok; ++i) {
              if (in(i, j)) {
                ok = wait_all(&sm.p_full[i], pcnt[i] & 1);
                if (!ok) break;
                ++pcnt[i];
                tc_fence_after();
                issue_pv(i, sv, j > rg[i].lo);
                if (j + 1 == rg[i].hi) umma_commit_w(&sm.o_done[i]);
              }
              if (in(i, j + 1)) {
                issue_s(i, i, skn);
                umma_commit_w(&sm.s_full[i]);
                if (j + 2 == rg[i].hi) umma_commit_w(&sm.q_empty[i]);
              }
            }
            if (!ok) break;
            free_v(sv);
            if (skn >= 0) umma_commit_w(&sm.kv_empty[skn]);
          }
          for (int i = 0; i < 2; ++i)
            if (rg[i].hi > rg[i].lo) ++qcnt[i];
        } else {
          const int qs = Cfg::kGeneral ? 0 : ((nseg - 1) & 1);
          ok = wait_all(&sm.q_full[qs], qcnt[qs] & 1);
          if (!ok) break;
          ++qcnt[qs];
          tc_fence_after();
          for (int t = 0; t < 2 && t < nt && ok; ++t) {
            ok = take_k();
            if (!ok) break;
            tc_fence_after();
            issue_s(t, qs, slot);
            umma_commit_w(&sm.s_full[t]);
            umma_commit_w(&sm.kv_empty[slot]);
            if (t == nt - 1) umma_commit_w(&sm.q_empty[qs]);
          }
          for (int t = 0; t < nt && ok; ++t) {
            const int i = t & 1;
            ok = take_v();
            if (!ok) break;
            clean(slot, kt0 + t);
            ok = wait_all(&sm.p_full[i], (i ? pcnt[1] : pcnt[0]) & 1);
            if (!ok) break;
            if (i) ++pcnt[1]; else ++pcnt[0];
            tc_fence_after();
            issue_pv(i, slot, t >= 2);
            free_v(slot);
            if (t + 2 >= nt) umma_commit_w(&sm.o_done[i]);
            if (t + 2 < nt) {
              ok = take_k();
              if (!ok) break;
              tc_fence_after();
              issue_s(i, qs, slot);
              umma_commit_w(&sm.s_full[i]);
              umma_commit_w(&sm.kv_empty[slot]);
              if (t + 2 == nt - 1) umma_commit_w(&sm.q_empty[qs]);
            }
          }
        }
      }
      // Wait for every MMA issued to finish before the columns are freed.
      umma_commit_w(&sm.mma_drain);
      mbar_wait_drain(&sm.mma_drain, 0, status);
      __syncwarp();
    } else if constexpr (Q8) {
      // ---------------------------------------------------------- scales
      // Split segments, and pieces: warp 10 + g serves group g.  With V's conversion warp 10
      // serves both groups and warp 11 the conversion, and both follow every tile, so that they
      // agree on the exponent.
      const WaitCtx wc{&sm.abort_flag, status, 35};
      const int me = warp - 10;
      uint32_t cnt[2] = {0, 0};
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        // the scale bytes of the lane's four keys of tile j; 2^0 for keys the unit does not see
        auto fetch = [&](int j, uint32_t& kw, uint32_t& vw) {
          kw = vw = 0x7f7f7f7fu;
          const int key = (j << 7) + lane * 4;
          if (key + 3 < g.keys.lo || key >= g.keys.hi) return;
          const int pg = key >> a.page_shift;
          const int id = pg < a.max_pages ? __ldg(a.table + static_cast<int64_t>(g.b) * a.max_pages + pg) : -1;
          if (id < 0 || id >= a.P) return;
          const int64_t at = (static_cast<int64_t>(id) * a.H_kv + g.kvh) * a.page + (key & (a.page - 1));
          if (!FA_IN_BOUNDS(at >= 0 && at + 4 <= static_cast<int64_t>(a.P) * a.H_kv * a.page, status, 511)) return;
          if (!Cfg::kConv || me == 0) kw = __ldg(reinterpret_cast<const uint32_t*>(a.k_scales + at));
          vw = __ldg(reinterpret_cast<const uint32_t*>(a.v_scales + at));
        };
        const int jend = g.kt0 + g.nt;
        const int dj = Cfg::kConv ? 1 : 2;
        int e = -1000;
        uint32_t kw = 0, vw = 0, kn = 0, vn = 0;
        int j = g.kt0 + (Cfg::kConv ? 0 : me);
        if (j < jend) fetch(j, kw, vw);
        for (; j < jend && ok; j += dj) {
          if (j + dj < jend) fetch(j + dj, kn, vn);  // in flight over this tile
          const int key = (j << 7) + lane * 4;
          int top = -1000;
          bool in[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int b = (vw >> (8 * x)) & 255;
            in[x] = key + x >= g.keys.lo && key + x < g.keys.hi;
            if (in[x] && b != 255) top = max(top, b - 127);
          }
          e = max(e, __reduce_max_sync(kFull, top));
          if (e == -1000) e = 0;  // every scale NaN
          if (Cfg::kConv && me == 1) {
            const int slot = cnt[0] % NSC;
            ok = __all_sync(kFull, mbar_wait(&sm.vsc_empty[slot], ((cnt[0] / NSC) & 1) ^ 1, wc));
            if (!ok) break;
            ++cnt[0];
            uint32_t f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = pg_factor16((vw >> (8 * x)) & 255, e) * 0x10001u;
            *reinterpret_cast<uint4*>(sm.vscales[slot].f + lane * 4) = make_uint4(f[0], f[1], f[2], f[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.vsc_full[slot]);
          } else {
            float k4[4], v4[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              k4[x] = in[x] ? e8m0_to_float((kw >> (8 * x)) & 255) : 0.f;
              v4[x] = in[x] ? pg_factor((vw >> (8 * x)) & 255, e) : 0.f;
            }
#pragma unroll
            for (int grp = 0; grp < 2; ++grp) {
              const bool mine = !Cfg::kConv ? grp == me
                                            : (g.pair ? j >= g.tile[grp].lo && j < g.tile[grp].hi
                                                      : ((j - g.kt0) & 1) == grp);
              if (!mine) continue;
              const int slot = cnt[grp] % NSC;
              ok = __all_sync(kFull, mbar_wait(&sm.sc_empty[grp][slot], ((cnt[grp] / NSC) & 1) ^ 1, wc));
              if (!ok) break;
              ++cnt[grp];
              PgScales& sc = sm.scales[grp][slot];
              *reinterpret_cast<float4*>(sc.ks + lane * 4) = make_float4(k4[0], k4[1], k4[2], k4[3]);
              if constexpr (!Cfg::kConv)
                *reinterpret_cast<float4*>(sc.vs + lane * 4) = make_float4(v4[0], v4[1], v4[2], v4[3]);
              if (lane == 0) sc.e = e;
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.sc_full[grp][slot]);
            }
          }
          kw = kn;
          vw = vn;
        }
      }
    }
  } else if (Cfg::kConv && warp >= 12) {
    // ------------------------------------------------------------ V's codes to fp16 tiles
    if constexpr (Cfg::kConv) {
      regs_set<Cfg::kLaunch, Cfg::kRegsOther>();
      const WaitCtx wc{&sm.abort_flag, status, 36};
      constexpr int L = D / 16;          // threads per row
      constexpr int kStep = 128 / L;     // rows per pass
      constexpr int U = 4;
      const int tid = threadIdx.x - 384;
      const int item = tid % L, r0 = tid / L;
      // codes lie in the swizzle of their row; the thread's two 16-byte units of the fp16 row are
      // 2 (item % 4) and the next of chunk item / 4, the upper chunk's threads storing the odd one
      // first, so that a row's threads cover all banks.  Rows a multiple of 8 apart share both
      // swizzles.
      static_assert(kStep % 8 == 0, "one swizzle for all of a thread's rows");
      const int in_unit = D == 128 ? item ^ (r0 & 7) : item ^ ((r0 >> 1) & 3);
      const int odd = (item >> 2) & 1;
      const int first = ((item & 3) * 2 + odd) ^ (r0 & 7), second = ((item & 3) * 2 + 1 - odd) ^ (r0 & 7);
      uint32_t it = 0;
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        const int jend = g.kt0 + g.nt;
        for (int j = g.kt0; j < jend; ++j) {
          const int rs = it % Cfg::kVRaw, vs = it % Cfg::kV16, ss = it % NSC;
          ok = __all_sync(kFull, mbar_wait(&sm.vsc_full[ss], (it / NSC) & 1, wc)) &&
               __all_sync(kFull, mbar_wait(&sm.vraw_full[rs], (it / Cfg::kVRaw) & 1, wc)) &&
               __all_sync(kFull, mbar_wait(&sm.v16_empty[vs], ((it / Cfg::kV16) & 1) ^ 1, wc));
          if (!ok) break;
          ++it;
          const int z0 = max(g.keys.lo - (j << 7), 0), z1 = min(g.keys.hi - (j << 7), 128);
          uint8_t* dst = sm.v16[vs] + (item >> 2) * 128 * 128;
#pragma unroll 1
          for (int base = r0; base < 128; base += U * kStep) {
            uint4 c[U];
            uint32_t f[U], o[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              c[u] = *reinterpret_cast<const uint4*>(sm.vraw[rs] + (base + u * kStep) * D + in_unit * 16);
              f[u] = sm.vscales[ss].f[base + u * kStep];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) pg_convert16(c[u], f[u], o[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint8_t* p = dst + (base + u * kStep) * 128;
              const uint4 lo = make_uint4(o[u][0], o[u][1], o[u][2], o[u][3]);
              const uint4 hi = make_uint4(o[u][4], o[u][5], o[u][6], o[u][7]);
              *reinterpret_cast<uint4*>(p + (first << 4)) = odd ? hi : lo;
              *reinterpret_cast<uint4*>(p + (second << 4)) = odd ? lo : hi;
            }
          }
          if (z0 > 0 || z1 < 128) {
            for (int row = r0; row < 128; row += kStep)
              if (row < z0 || row >= z1) {
                *reinterpret_cast<uint4*>(dst + row * 128 + (first << 4)) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(dst + row * 128 + (second << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.v16_full[vs]);
            mbar_arrive(&sm.vraw_empty[rs]);
            mbar_arrive(&sm.vsc_empty[ss]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    if constexpr (Cfg::kGeneral) regs_set<Cfg::kLaunch, Cfg::kRegsSoftmax>();
    constexpr bool kPieces = Q8 && !Cfg::kConv;
    constexpr int NC = 128 / Cfg::kCopies;         // keys of a tile this warp handles
    constexpr int kQuarter = Cfg::kM / 4;          // accumulator rows per 32-lane quarter
    constexpr int kWarpsPerCopy = 4 / Cfg::kCopies;
    const int grp = warp >> 2;
    const int wq = warp & 3;
    const int cp = wq / kWarpsPerCopy;
    const int col0 = cp * NC;
    // row within the copy; with M = 64, lanes 16-31 of a quarter hold no rows
    const int wrow0 = Cfg::kSlots > 1 ? 0 : (wq % kWarpsPerCopy) * kQuarter;  // the warp's first row
    const int rc = Cfg::kSlots > 1 ? lane % Cfg::kRows : (lane < kQuarter ? wrow0 + lane : 1 << 20);
    const bool writer = Cfg::kSlots == 1 || lane < Cfg::kRows;  // of a row's lanes
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + grp * 128 + lane_off;
    const uint32_t tO = tbase + Cfg::kOCol + grp * D + lane_off;
    const WaitCtx wc{&sm.abort_flag, status, 33 + grp};
    uint32_t scnt = 0, ocnt = 0, gcnt = 0;  // scnt also counts the group's scale entries
    bool ok = true;
    while (ok) {
      const PgSeg* gp = next_seg(wc);
      if (gp == nullptr) break;
      const PgSeg& g = *gp;
      // this group's tile and its key tiles j0, j0 + dj, .. below j1
      const bool pair = Cfg::kGeneral && g.pair;
      const int tok = pair ? grp * a.TQ : 0;
      const int M = G * min(a.TQ, g.ntok - tok);
      const int j0 = pair ? g.tile[grp].lo : g.kt0 + grp;
      const int j1 = pair ? g.tile[grp].hi : g.kt0 + g.nt;
      const int dj = pair ? 1 : 2;
      const bool any = j0 < j1;
      const bool rows_here = wrow0 < M;  // a warp without rows only keeps the barriers
      int vis_hi, vis_lo, all_hi, all_lo;
      // log2 units per score; with e4m3 pages the row's query factor, and the exponent of O
      float c_row = a.scale_log2;
      int e_ref = 0;
      {
        const int iq = rc < M ? rc / G : 0;
        const int qpos = g.pos0 + tok + iq;
        vis_hi = rc < M ? (a.causal ? min(qpos, g.len - 1) : g.len - 1) : -1;
        vis_lo = a.window >= 0 ? qpos - a.window : 0;
        // every row of the tile sees the keys from all_lo to all_hi
        all_hi = a.causal ? g.pos0 + tok : g.len - 1;
        all_lo = a.window >= 0 ? g.pos0 + tok + M / G - 1 - a.window : 0;
        if constexpr (Q8) {
          if (rc < M && FA_IN_BOUNDS(g.q0 + tok + iq < a.T, status, 512))
            c_row *= __ldg(a.q_scale + (static_cast<int64_t>(g.q0) + tok + iq) * a.H + g.kvh * G + rc - iq * G);
        }
      }
      float m_ref = -INFINITY, l = 0.f, lr = 0.f;
      for (int j = j0; j < j1; j += dj) {
        const int ss = scnt % NSC;
        if constexpr (Q8) {
          ok = __all_sync(kFull, mbar_wait(&sm.sc_full[grp][ss], (scnt / NSC) & 1, wc));
          if (!ok) break;
        }
        ok = __all_sync(kFull, mbar_wait(&sm.s_full[grp], scnt & 1, wc));
        if (!ok) break;
        ++scnt;
        tc_fence_after();
        if (rows_here) {
          const int k0 = (j << 7) + col0;
          uint32_t s[NC];
#pragma unroll
          for (int c = 0; c < NC; c += 32) tmem_ld32(tS + col0 + c, s + c);
          tmem_wait_ld();
          if constexpr (Cfg::kSlots > 1) {
            // the scores of the pieces q1 and q2 lie 8 lanes apart
#pragma unroll
            for (int c = 0; c < NC; ++c)
              s[c] = __float_as_uint(__uint_as_float(s[c]) +
                                     __uint_as_float(__shfl_xor_sync(kFull, s[c], Cfg::kRows)));
          }
          if constexpr (Q8) {
            const float4* ks = reinterpret_cast<const float4*>(sm.scales[grp][ss].ks + col0);
#pragma unroll
            for (int c = 0; c < NC / 4; ++c) {
              const float4 f = ks[c];
              const float2 x = fmul2(make_float2(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])),
                                     make_float2(f.x, f.y));
              const float2 y = fmul2(make_float2(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])),
                                     make_float2(f.z, f.w));
              s[4 * c] = __float_as_uint(x.x);
              s[4 * c + 1] = __float_as_uint(x.y);
              s[4 * c + 2] = __float_as_uint(y.x);
              s[4 * c + 3] = __float_as_uint(y.y);
            }
          }
          if (k0 + NC - 1 > all_hi || k0 < all_lo) {
            const int lim = vis_hi - k0, first = vis_lo - k0;
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (c > lim || c < first) s[c] = __float_as_uint(-INFINITY);
          }
          float mx8[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 8]));
#pragma unroll
          for (int c = 16; c < NC; c += 16)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              mx8[x] = fmax3(mx8[x], __uint_as_float(s[c + x]), __uint_as_float(s[c + 8 + x]));
          const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                 fmaxf(mx8[6], mx8[7]));
          const float m_new = mx * c_row;
          const bool raise = m_new > m_ref + kTau;
          bool grown = false;  // the value exponent grew: O is held in units of 2^e_ref
          float alpha = raise ? ex2_approx(m_ref - m_new) : 1.0f;
          if (raise) {
            l *= alpha;
            lr *= alpha;
            m_ref = m_new;
          }
          if constexpr (Q8) {
            const int e = sm.scales[grp][ss].e;
            grown = j > j0 && e > e_ref;
            if (grown) alpha = e - e_ref > 126 ? 0.f : alpha * __int_as_float((127 + e_ref - e) << 23);
            e_ref = e;
          }
          if (__any_sync(kFull, raise) || grown) {
            if (j > j0) {
              // the commit that signalled this S covers the group's previous P.V
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                tmem_st32(tO + c, o);
              }
              tmem_wait_st();
            }
          }
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          // P for all 128 keys: this copy's columns, zeros for the other copies' keys
          uint32_t zero[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) zero[x] = 0u;
          if constexpr (kPieces) {
            uint32_t p[kPPieces][NC / 4];
            softmax_row_f8<NC>(s, sm.scales[grp][ss].vs + col0, p, c_row, m_use - kPShift, l);
            if constexpr (Cfg::kSlots > 1) {
              // each of a row's lanes stores one piece, the fourth zeros
              const int slot = lane / Cfg::kRows;
#pragma unroll
              for (int x = 0; x < NC / 4; ++x)
                p[0][x] = slot == 0 ? p[0][x] : (slot == 1 ? p[1][x] : (slot == 2 ? p[2][x] : 0u));
            }
            constexpr int n = Cfg::kSlots > 1 ? 1 : kPPieces;
#pragma unroll
            for (int y = 0; y < n; ++y)
#pragma unroll
              for (int x = 0; x < NC / 4; x += 8) tmem_st8(tS + y * 32 + col0 / 4 + x, p[y] + x);
            if constexpr (Cfg::kCopies > 1) {
#pragma unroll
              for (int c = 0; c < n * 32; c += 8)
                if ((c & 31) < col0 / 4 || (c & 31) >= col0 / 4 + NC / 4) tmem_st8(tS + c, zero);
            }
          } else {
            uint32_t p[NC / 2];
            softmax_row<Cfg::kConv ? Elem::kF16 : E, NC>(s, p, c_row, m_use, l, lr);
#pragma unroll
            for (int x = 0; x < NC / 2; x += 16) tmem_st16(tS + col0 / 2 + x, p + x);
            if constexpr (Cfg::kCopies > 1) {
#pragma unroll
              for (int c = 0; c < 64; c += 16)
                if (c < col0 / 2 || c >= col0 / 2 + NC / 2) tmem_st16(tS + c, zero);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        if constexpr (Cfg::kPArrive == 4) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[grp]);
        } else {
          mbar_arrive(&sm.p_full[grp]);
        }
        if constexpr (Q8) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sc_empty[grp][ss]);
        }
      }
      if (!ok) break;
      float unit = 1.0f;  // of O
      if constexpr (Q8) unit = e8m0_to_float(static_cast<uint32_t>(e_ref + 127));
      if constexpr (kPieces) {
        // the pieces' weights carry 2^7, and fp32 sums normalise them
        m_ref -= kPShift;
        lr = l;
      }
      if (any) {
        ok = __all_sync(kFull, mbar_wait(&sm.o_done[grp], ocnt & 1, wc));
        if (!ok) break;
        ++ocnt;
        tc_fence_after();
      }
      const bool real = rc < M && writer;
      // a segment that is not a whole unit leaves a partial result
      const int64_t part0 =
          ((static_cast<int64_t>(blockIdx.x) * 2 + g.slot) * Cfg::kSubs + (pair ? grp : 0)) * Cfg::kRows;
      auto put = [&](int row, int c, const auto& v) {  // columns c .. of a row of the tile
        constexpr int n = sizeof(v) / sizeof(float);
        const int i = row / G;
        const int64_t token = static_cast<int64_t>(g.q0) + tok + i;
        const int h = g.kvh * G + row - i * G;
        if (g.whole) {
          if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H && c + n <= D, status, 503)) {
            typename ElemOps<E>::T* dst =
                static_cast<typename ElemOps<E>::T*>(a.out) + (token * a.H + h) * D + c;
            if constexpr (n % 8 == 0) {
#pragma unroll
              for (int x = 0; x < n / 8; ++x)
                reinterpret_cast<uint4*>(dst)[x] = make_uint4(
                    ElemOps<E>::pack(v[8 * x], v[8 * x + 1]), ElemOps<E>::pack(v[8 * x + 2], v[8 * x + 3]),
                    ElemOps<E>::pack(v[8 * x + 4], v[8 * x + 5]), ElemOps<E>::pack(v[8 * x + 6], v[8 * x + 7]));
            } else {
#pragma unroll
              for (int x = 0; x < n / 2; ++x)
                reinterpret_cast<uint32_t*>(dst)[x] = ElemOps<E>::pack(v[2 * x], v[2 * x + 1]);
            }
          }
        } else if (FA_IN_BOUNDS(part0 + row < a.slots * Cfg::kSubs * Cfg::kRows && row < Cfg::kRows && c + n <= D, status,
                                504)) {
          float* dst = a.part_o + (part0 + row) * D + c;
          if constexpr (n % 4 == 0) {
#pragma unroll
            for (int x = 0; x < n / 4; ++x)
              reinterpret_cast<float4*>(dst)[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
          } else {
            *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[1]);
          }
        }
      };
      auto put_lse = [&](float m, float ls, float lrs) {
        const float lse_l = ls == 0.f ? -INFINITY : (m + lg2_approx(ls)) * kLn2;
        const float lse_r = lrs == 0.f ? -INFINITY : (m + lg2_approx(lrs)) * kLn2;
        const int iq = rc / G;
        const int64_t token = static_cast<int64_t>(g.q0) + tok + iq;
        const int h = g.kvh * G + rc - iq * G;
        if (g.whole) {
          if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H, status, 505))
            a.lse[static_cast<int64_t>(h) * a.T + token] = lse_l;
        } else if (FA_IN_BOUNDS(part0 + rc < a.slots * Cfg::kSubs * Cfg::kRows, status, 506)) {
          *reinterpret_cast<float2*>(a.part_lse + (part0 + rc) * 2) = make_float2(lse_l, lse_r);
        }
      };
      if (pair) {
        // O normalised by the sum of the rounded weights, and the log-sums of both
        const float inv = lr == 0.f ? 0.f : unit / lr;
        if (rows_here) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (any) {
              tmem_ld32(tO + c, o);
              tmem_wait_ld();
            }
            float v[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = lr == 0.f ? 0.f : __uint_as_float(o[x]) * inv;
            if (real) put(rc, c, v);
          }
          if (real) put_lse(m_ref, l, lr);
        }
      } else {
        // Join the copies: weights 2^(m_k - max m) / sum of lr, the rows summed through shared
        // memory a few columns at a time in two buffers, so that one barrier per step suffices
        auto sync_groups = [&]() -> bool {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.groups);
          const bool r = __all_sync(kFull, mbar_wait(&sm.groups, gcnt & 1, wc));
          ++gcnt;
          return r;
        };
        constexpr int SC = Cfg::kStageCols;
        constexpr int kUnits = SC / 4;  // 16-byte units of a staged row; unit u sits at u ^ key(row)
        auto key = [](int r) { return (kUnits == 8 ? r : r >> 1) & (kUnits - 1); };
        const int me = grp * Cfg::kCopies + cp;
        if (real) sm.stat[me][rc] = make_float3(m_ref, l, lr);
        ok = sync_groups();
        if (!ok) break;
        float mm = -INFINITY, ls = 0.f, lrs = 0.f, wgt = 0.f;
        if (rc < M) {
#pragma unroll
          for (int k = 0; k < 2 * Cfg::kCopies; ++k) mm = fmaxf(mm, sm.stat[k][rc].x);
          const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int k = 0; k < 2 * Cfg::kCopies; ++k) {
            const float3 st = sm.stat[k][rc];
            const float e = ex2_approx(st.x - ref);
            ls += e * st.y;
            lrs += e * st.z;
          }
          wgt = (lr == 0.f || lrs == 0.f) ? 0.f : ex2_approx(m_ref - ref) * unit / lrs;
          if (me == 0 && writer) put_lse(ref, ls, lrs);
        }
#pragma unroll 1
        for (int c = 0; c < D; c += SC) {
          float* stage = sm.stage[(c / SC) & 1];
          const int srow = Cfg::kGeneral ? rc : me * Cfg::kRows + rc;
          uint32_t o[SC];
          float v[SC];
          if (any && rows_here) {
#pragma unroll
            for (int x = 0; x < SC; x += 16) tmem_ld16(tO + c + x, o + x);
            tmem_wait_ld();
          }
#pragma unroll
          for (int x = 0; x < SC; ++x) {
            v[x] = lr == 0.f ? 0.f : __uint_as_float(o[x]) * wgt;
            if constexpr (Cfg::kSlots > 1) {  // the products of a row's pieces
              v[x] += __shfl_xor_sync(kFull, v[x], 8);
              v[x] += __shfl_xor_sync(kFull, v[x], 16);
            }
          }
          if (real && (!Cfg::kGeneral || grp == 1)) {
#pragma unroll
            for (int x = 0; x < kUnits; ++x)
              *reinterpret_cast<float4*>(stage + srow * SC + ((x ^ key(srow)) << 2)) =
                  make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
          }
          ok = sync_groups();
          if (!ok) break;
          if constexpr (Cfg::kGeneral) {
            if (grp == 0 && real) {
#pragma unroll
              for (int x = 0; x < kUnits; ++x) {
                const float4 y = *reinterpret_cast<const float4*>(stage + rc * SC + ((x ^ key(rc)) << 2));
                v[4 * x] += y.x;
                v[4 * x + 1] += y.y;
                v[4 * x + 2] += y.z;
                v[4 * x + 3] += y.w;
              }
              put(rc, c, v);
            }
          } else {
            // two columns of a row per thread
            const int col = (threadIdx.x % (SC / 2)) * 2;  // warps 0-7
            for (int row = threadIdx.x / (SC / 2); row < M; row += 256 / (SC / 2)) {
              float sum[2] = {0.f, 0.f};
#pragma unroll
              for (int k = 0; k < 2 * Cfg::kCopies; ++k) {
                const int sr = k * Cfg::kRows + row;
                const float2 y =
                    *reinterpret_cast<const float2*>(stage + sr * SC + (((col >> 2) ^ key(sr)) << 2) + (col & 3));
                sum[0] += y.x;
                sum[1] += y.y;
              }
              put(row, c + col, sum);
            }
          }
        }
        if (!ok) break;
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, Cfg::kTmemCols);
  }
}

// ---------------------------------------------------------------- joining the partial results
// Per row: LSE = log sum_s exp(lse_s) and O = sum_s exp(lr_s - LR) O_s with LR = log sum_s
// exp(lr_s), the convex combination one CTA would have formed.  Units that one CTA computed
// were written by it; rows of units without keys get O = 0, LSE = -inf.  Block (unit,
// key/value head, part) of four warps; W warps share a row's partial results.
template <int D, Elem E, bool Q8, int R, int W>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const PgArgs a) {
  using T = typename ElemOps<E>::T;
  using Cfg = PgCfg<D, E, Q8, R>;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int V = D / 32;  // columns per lane
  __shared__ float acc_sh[W > 1 ? W : 1][D];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = a.H / a.H_kv;
  const int kvh = blockIdx.y;
  const int unit = blockIdx.x;
  const int b = find_seq(a.meta + 2, a.B, unit, lane);
  if (b >= a.B) return;
  const PgSeq s = pg_seq(a, b);
  const int u = unit - a.meta[2 + b];
  const int tok0 = u * 2 * a.TQ;
  const int ntok = min(2 * a.TQ, s.n - tok0);
  const PgKeys k = pg_unit_keys(a, s, u);
  const int T_u = k.t1 - k.t0;
  const int* costs = a.meta + 2 + a.B + 1;
  int start = costs[b] + kvh * ((costs[b + 1] - costs[b]) / a.H_kv);
  int before = 0;  // the sequence's units before this one are pairs
  for (int x = lane; x < u; x += 32) {
    const PgKeys kx = pg_unit_keys(a, s, x);
    before += (kx.t1 - kx.t0) * Cfg::kPairCost;
  }
  start += static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(before)));
  const int per = a.meta[1];
  const int cf = start / per;
  const int cost = pg_is_pair(a, s, u) ? Cfg::kPairCost : Cfg::kSplitCost;
  const int cl = T_u > 0 ? (start + (T_u - 1) * cost) / per : cf;
  if (T_u > 0 && cf == cl) return;  // written by its CTA
  const int parts = T_u > 0 ? cl - cf + 1 : 0;
  const int rows = G * ntok;
  for (int row = blockIdx.z * (4 / W) + warp / W; row < rows; row += gridDim.z * (4 / W)) {
    const int tile = row / (G * a.TQ);
    const int rc = row - tile * G * a.TQ;
    const int iq = row / G, h = kvh * G + (row - iq * G);
    const int64_t token = static_cast<int64_t>(s.q0) + tok0 + iq;
    // index of partial result i of this row
    auto at = [&](int i) -> int64_t {
      const int slot = 2 * (cf + i) + (i == 0);
      return (static_cast<int64_t>(slot) * Cfg::kSubs + tile) * Cfg::kRows + rc;
    };
    float mx_l = -INFINITY, mx_r = -INFINITY, s_l = 0.f, s_r = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const int64_t x = at(i);
      if (!FA_IN_BOUNDS(x >= 0 && x < a.slots * Cfg::kSubs * Cfg::kRows, a.status, 507)) continue;
      const float2 v = *reinterpret_cast<const float2*>(a.part_lse + x * 2);
      mx_l = fmaxf(mx_l, v.x);
      mx_r = fmaxf(mx_r, v.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx_l = fmaxf(mx_l, __shfl_xor_sync(kFull, mx_l, o));
      mx_r = fmaxf(mx_r, __shfl_xor_sync(kFull, mx_r, o));
    }
    if (mx_l == -INFINITY) mx_l = 0.f;  // no key, or NaN only: the sums decide
    if (mx_r == -INFINITY) mx_r = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const int64_t x = at(i);
      if (!FA_IN_BOUNDS(x >= 0 && x < a.slots * Cfg::kSubs * Cfg::kRows, a.status, 508)) continue;
      const float2 v = *reinterpret_cast<const float2*>(a.part_lse + x * 2);
      s_l += expf(v.x - mx_l);
      s_r += expf(v.y - mx_r);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s_l += __shfl_xor_sync(kFull, s_l, o);
      s_r += __shfl_xor_sync(kFull, s_r, o);
    }
    float acc[V];
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = 0.f;
    const float inv = s_r == 0.f ? 0.f : 1.0f / s_r;
    // 32 partial results at a time: a lane forms one weight, then the warp sums the rows with
    // the weights broadcast; a partial result without keys was not written and is not read
    for (int base = (W > 1 ? warp * 32 : 0); base < parts; base += 32 * W) {
      float wl = 0.f;
      int64_t x = 0;
      if (base + lane < parts) {
        x = at(base + lane);
        const float v = a.part_lse[x * 2 + 1];
        wl = v == -INFINITY ? 0.f : expf(v - mx_r) * inv;
      }
      const int cnt = min(32, parts - base);
#pragma unroll 4
      for (int t = 0; t < cnt; ++t) {
        const float wgt = __shfl_sync(kFull, wl, t);
        const int64_t xt = __shfl_sync(kFull, x, t);
        if (wgt == 0.f) continue;
        const float* po = a.part_o + xt * D + lane * V;
        if constexpr (V == 4) {
          const float4 v = *reinterpret_cast<const float4*>(po);
          acc[0] = fmaf(wgt, v.x, acc[0]);
          acc[1] = fmaf(wgt, v.y, acc[1]);
          acc[2] = fmaf(wgt, v.z, acc[2]);
          acc[3] = fmaf(wgt, v.w, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(po);
          acc[0] = fmaf(wgt, v.x, acc[0]);
          acc[1] = fmaf(wgt, v.y, acc[1]);
        }
      }
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int x = 0; x < V; ++x) acc_sh[warp][lane * V + x] = acc[x];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int x = 0; x < V; ++x) {
          acc[x] = 0.f;
#pragma unroll
          for (int y = 0; y < W; ++y) acc[x] += acc_sh[y][lane * V + x];
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H, a.status, 509)) {
      T* orow = static_cast<T*>(a.out) + (token * a.H + h) * D + lane * V;
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(orow) =
            make_uint2(ElemOps<E>::pack(acc[0], acc[1]), ElemOps<E>::pack(acc[2], acc[3]));
      else
        *reinterpret_cast<uint32_t*>(orow) = ElemOps<E>::pack(acc[0], acc[1]);
      if (lane == 0) a.lse[static_cast<int64_t>(h) * a.T + token] = s_l == 0.f ? -INFINITY : mx_l + logf(s_l);
    }
  }
}

}  // namespace fa
