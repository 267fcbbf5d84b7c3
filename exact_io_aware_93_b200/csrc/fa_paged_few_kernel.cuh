// fa_paged_few_kernel.cuh -- exact attention over a paged cache for few query rows per key/value
// head (up to 16: single tokens, drafted tokens), for sm_100a.  The work list, the page loads and
// the join of partial results are in fa_paged_common.cuh.
//
// The cache is a stream: nothing but its bytes should cost time, so the KEYS take the 128 rows of
// the tensor core's tile and the few query rows its narrow side:
//   S^T = K Q^T    M = 128 keys, N = the rows, both operands as they lie in shared memory
//   O^T += V^T P^T M = d, N = the rows, V read MN-major
// A product then moves its 128-row operand once (32 cycles of shared memory) and the narrow side
// is nearly free: 16 products of 32 cycles per tile (8 with e4m3 pages) where rows-first tiles
// need 16 of 64.  A softmax thread owns one KEY of a tile and all rows, so a tile costs it as many
// exponentials as there are rows, the sums stay in registers until the segment ends, and the
// narrow score tiles leave tensor memory for four of them in flight.
//
// The two softmax groups take alternate key tiles, each with its own accumulator.  A group's
// rows share one reference maximum per row over its 128 threads: per tile each warp posts whether
// one of its scores exceeds the reference by a threshold; only then do the four warps exchange maxima and
// rescale O^T.  Weights P^T go to shared memory as the next product's B operand.
//
// e4m3 pages.  The codes are operands as they are (kind::f8f6f4): a tile moves half the bytes and
// nothing is converted.
//   Q   e4m3 pieces per row (fa_paged_scale_q_kernel), two of a bf16 and three of an fp16 row, as
//       rows r, RW + r, .. of the tile: the score columns are added by the key's thread
//   P   the weight, an fp16 value, is the sum of e5m2 pieces (e5m2 is the upper byte of an fp16):
//       three hold the 9 bits that it is rounded to, one more than bf16, and four all 11, for fp16
//       outputs.  e5m2 and not e4m3 for its range: a long tail of small weights beside a large one
//       keeps its mass.  The pieces are rows of P^T, their products columns of O^T, added at the end.
//   scales  a key's 2^ek and 2^(ev - E) are one number each for its thread; E is the largest
//       value exponent of the group's tiles so far (O^T is rescaled when it grows).  The bytes
//       come with the K tile, into a ring of their own that the softmax groups free.
// (The rows-first form of this kernel took 187 us for 16 sequences of 16-32K tokens; it waited for
// its softmax and its products in turn.)
//
// Bound by device memory: 16 sequences of 16-32K tokens, 32 heads sharing 8, d 128, one new token each:
// 230 us over 16-bit pages (6.5 TB/s), 132 us over e4m3 pages (5.7 TB/s).  Pages of 16 e4m3 slots are boxes
// of 2 KB and stream at three quarters of that.  What does not grow with the cache, 17 us: launch and plan
// 3, the first tile 4, a segment's end 2.5, the join 5.
//
// Warp roles (384 threads): warps 0-3 and 4-7 the softmax groups, warp 8 the schedule and the loads
// of Q and K, warp 10 those of V (one warp for both took 700 cycles a load and bounded the kernel),
// warp 9 the MMA issuer, warp 11 idle.
#pragma once

#include "fa_paged_common.cuh"
#include "fa_paged_launch.h"

namespace fa {

// Over e4m3 pages a score may exceed its row's reference maximum m by 2^2 (16-bit pages: kTau, 2^8)
// before m is raised, and weights are 2^(x - m + 13) <= 2^15: they are cut off at e5m2's 2^-16,
// 2^-29 of the reference weight, far below what a long tail of small weights adds up to.  The weight
// carries its key's value scale, 2^(ev - E): a row that far below the largest is cut off that much earlier.
constexpr float kTauCodes = 2.0f;
constexpr float kCodesShift = 13.0f;

template <int D, Elem E, bool Q8, int RW>
struct PfCfg {
  static constexpr int kQPieces = paged_q_pieces(E == Elem::kF16);  // e4m3 pieces of a query
  static constexpr int kPPieces = E == Elem::kF16 ? 4 : 3;  // e5m2 pieces of a weight
  static constexpr int kRows = RW;      // rows of a tile and of a partial result
  static constexpr int kSubs = 1;
  static constexpr int kPairCost = 2;   // units are single tiles
  static constexpr int kSplitCost = 2;
  // the end of a unit, as long as 2 key tiles of 16-bit pages and 4 of e4m3 (without: 24 sequences of
  // 512 tokens 20.5 us, with 16.9; e4m3 24.8 and 21.6)
  static constexpr int kUnitCost = Q8 ? 8 : 4;
  static constexpr int kThreads = 384;
  static constexpr int kAhead = 3;      // key tiles whose scores run ahead of their values
  static constexpr int kSBufs = 4;
  // a row in shared memory: 128-byte chunks of 64 16-bit elements, or D codes (D = 64 in the
  // 64-byte swizzle)
  static constexpr int kRowBytes = Q8 ? D : 128;
  static constexpr int kChunks = Q8 ? 1 : D / 64;
  static constexpr int kChunkBytes = 128 * kRowBytes;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  // N of the products: rows, or all pieces of each, in whole 16s
  static constexpr int kNS = ((Q8 ? kQPieces : 1) * RW + 15) / 16 * 16;
  static constexpr int kNO = ((Q8 ? kPPieces : 1) * RW + 15) / 16 * 16;
  static constexpr int kQPartBytes = kNS * kRowBytes;
  static constexpr int kQBytes = kChunks * kQPartBytes;
  static constexpr int kPChunks = Q8 ? 1 : 2;         // 128 keys of a row in 128-byte chunks
  static constexpr int kPChunkBytes = kNO * 128;
  static constexpr int kPBytes = kPChunks * kPChunkBytes;
  static constexpr int kStages = (Q8 ? (RW == 16 && E == Elem::kF16 ? 11 : 12) : 6) * (128 / D);
  static constexpr int kScaleRing = 8;  // key tiles
  static constexpr int kSegRing = 4;
  static constexpr int kSegReaders = 10;  // warps
  static constexpr uint32_t kOCol = kSBufs * kNS;
  static constexpr uint32_t kCols = kOCol + 2 * kNO;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
  static_assert(kCols <= 512 && RW % 8 == 0, "tensor memory");
};

template <int D, Elem E, bool Q8, int RW>
struct __align__(1024) PfSmem {
  using Cfg = PfCfg<D, E, Q8, RW>;
  uint8_t kv[Cfg::kStages][Cfg::kTileBytes];
  uint8_t q[2][Cfg::kQBytes];
  uint8_t p[2][Cfg::kPBytes];               // each group's P^T
  alignas(16) float part[RW][D];            // group 1's O on its way to group 0
  alignas(16) uint8_t scales[Q8 ? Cfg::kScaleRing : 1][2][128];  // a key tile's, of keys and values
  float2 sums[2][4][RW];                    // l, lr of each group's warps
  float ref[2][RW];                         // each group's reference maxima
  float weight[2][RW];                      // of each group's O in the result
  float top[2][4][RW];                      // maxima of a group's warps, when one is raised
  alignas(16) int flag[2][2][4];            // by tiles' parity, of a group's warps: does one want to
                                            // raise a maximum (bit 0), and its largest value exponent
  PgSeg segs[Cfg::kSegRing];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t kv_full[Cfg::kStages];
  uint64_t kv_empty[Cfg::kStages];
  uint64_t sc_full[Cfg::kScaleRing];
  uint64_t sc_empty[Cfg::kScaleRing];
  uint64_t seg_full[Cfg::kSegRing];
  uint64_t seg_empty[Cfg::kSegRing];
  uint64_t s_full[Cfg::kSBufs];
  uint64_t p_full[2];
  uint64_t p_empty[2];  // the group's last product is complete
  uint64_t group[2];    // a group's warps
  uint64_t groups;      // both groups
  uint64_t mma_drain;
  PgPlan plan;
  uint32_t tmem_base;
  int abort_flag;
};

// Columns of tensor memory, N a multiple of 8.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t t, uint32_t (&r)[N]) {
  if constexpr (N % 32 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(t + c, r + c);
  } else if constexpr (N % 16 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 16) tmem_ld16(t + c, r + c);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8) tmem_ld8(t + c, r + c);
  }
}

// Largest value over the warp (NaN apart or not: either leaves the row NaN).
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x);
  const int m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
  return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

template <int D, Elem E, bool Q8, int RW>
__global__ void __launch_bounds__(384, 1)
    fa_paged_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PgArgs a) {
  using Cfg = PfCfg<D, E, Q8, RW>;
  using T = typename ElemOps<E>::T;
  constexpr int NS = Cfg::kStages;
  constexpr int NSC = Cfg::kScaleRing;
  constexpr int NSEG = Cfg::kSegRing;
  constexpr int NB = Cfg::kSBufs;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr float kRaise = Q8 ? kTauCodes : kTau;
  constexpr float kPShift = Q8 ? kCodesShift : kWeightShift<E>;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset and not through an integer: the compiler keeps seeing shared memory
  PfSmem<D, E, Q8, RW>& sm = *reinterpret_cast<PfSmem<D, E, Q8, RW>*>(smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = a.H / a.H_kv;
  int* status = a.status;

  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.p_empty[i], 1);
      mbar_init(&sm.group[i], 4);
    }
    for (int s = 0; s < NSC; ++s) {
      mbar_init(&sm.sc_full[s], 32);
      mbar_init(&sm.sc_empty[s], 4);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(&sm.s_full[s], 1);
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
  // Launched while the kernel before it may still run: what that one writes is read from here on.
  // (e4m3 pages: it is the scaling of the queries, which has waited for the kernel before it and
  // writes nothing that the plan reads.)
  if constexpr (!Q8) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    pg_plan<Cfg>(a, lane, &sm.plan);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  if constexpr (Q8) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Readers of the segment ring: the next segment, or null at the end or after an abort; a
  // reader gives the one it holds back first.
  uint32_t nseg = 0;
  auto next_seg = [&](const PgWait& wc) -> const PgSeg* {
    if (nseg > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_empty[(nseg - 1) % NSEG]);
    }
    const int i = nseg % NSEG;
    if (!pg_wait(&sm.seg_full[i], (nseg / NSEG) & 1, wc)) return nullptr;
    ++nseg;
    return sm.segs[i].nt > 0 ? &sm.segs[i] : nullptr;
  };

  if (warp == 8) {
    // ------------------------------------------------------------ schedule and TMA loads
    const PgWait wc{&sm.abort_flag, 31};
    PgWalk<Cfg> w(a, sm.plan);
    PgSeg g;
    PgPages pages{};
    PgInFlight flight;
    uint32_t it = 0, tiles = 0, qcnt[2] = {0, 0};
    bool ok = true;
    while (ok) {
      const int i = nseg % NSEG;
      const bool more = w.next(a, g);
      if (more) pages.start(a, g, lane);
      ok = pg_wait(&sm.seg_empty[i], ((nseg / NSEG) & 1) ^ 1, wc);
      if (!ok) break;
      if (lane == 0) {
        if (!more) g.nt = 0;
        sm.segs[i] = g;
        mbar_arrive(&sm.seg_full[i]);
      }
      const int qs = nseg & 1;
      ++nseg;
      if (!more) break;
      ok = pg_wait(&sm.q_empty[qs], (qcnt[qs] & 1) ^ 1, wc);
      if (!ok) break;
      // a box of G heads x TQ tokens per chunk, or per piece
      constexpr int kBoxes = Q8 ? Cfg::kQPieces : Cfg::kChunks;
      if (lane == 0)
        mbar_arrive_expect_tx(&sm.q_full[qs], static_cast<uint32_t>(kBoxes * Cfg::kRowBytes * G * a.TQ));
      __syncwarp();
      if (lane < kBoxes &&
          FA_IN_BOUNDS(g.q0 >= 0 && g.q0 < a.T && g.kvh < a.H_kv && G * a.TQ <= RW, status, 520))
        tma_load_4d(sm.q[qs] + lane * (Q8 ? RW * Cfg::kRowBytes : Cfg::kQPartBytes), &tm_q, &sm.q_full[qs],
                    Q8 ? 0 : lane * 64, 0, g.kvh, Q8 ? lane * a.T + g.q0 : g.q0);
      __syncwarp();
      ++qcnt[qs];
      ok = pg_loads<Cfg::kAhead>(g, [&](bool isv, int j) -> bool {
        const int slot = it % NS;
        const uint32_t phase = (it / NS) & 1;
        ++it;
        if (isv) return true;
        const int ss = tiles % NSC;
        const uint32_t sphase = (tiles / NSC) & 1;
        if (!pg_wait_lanes(lane == 0 ? &sm.kv_empty[slot] : (Q8 && lane == 1 ? &sm.sc_empty[ss] : nullptr),
                           (lane == 0 ? phase : sphase) ^ 1, wc))
          return false;
        ++tiles;
        flight.add(slot, phase);
        if constexpr (Q8) {
          pg_load_tile<Cfg::kRowBytes, 1>(a, g, pages, &tm_k, j, sm.kv[slot], &sm.kv_full[slot], lane, sm.scales[ss][0],
                                          &sm.sc_full[ss]);
        } else {
          pg_load_tile<Cfg::kRowBytes, Cfg::kChunks>(a, g, pages, &tm_k, j, sm.kv[slot], &sm.kv_full[slot], lane);
        }
        return true;
      });
    }
    if (lane == 0 && FA_IN_BOUNDS(static_cast<int>(blockIdx.x) * 2 < a.slots, status, 526)) a.splits[blockIdx.x] = w.split;
    if (!ok && lane == 0) {
      flight.drain(sm.kv_full, status);
      for (int i = 0; i < 2; ++i)
        if (qcnt[i] > 0) mbar_wait_drain(&sm.q_full[i], (qcnt[i] - 1) & 1, status);
    }
    if constexpr (Q8) cp_async_wait_all();
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ loads of V
    const PgWait wc{&sm.abort_flag, 37};
    PgPages pages{};
    PgInFlight flight;
    uint32_t it = 0;
    bool ok = true;
    while (ok) {
      const PgSeg* gp = next_seg(wc);
      if (gp == nullptr) break;
      pages.start(a, *gp, lane);
      ok = pg_loads<Cfg::kAhead>(*gp, [&](bool isv, int j) -> bool {
        const int slot = it % NS;
        const uint32_t phase = (it / NS) & 1;
        ++it;
        if (!isv) return true;
        if (!pg_wait(&sm.kv_empty[slot], phase ^ 1, wc)) return false;
        flight.add(slot, phase);
        pg_load_tile<Cfg::kRowBytes, Cfg::kChunks>(a, *gp, pages, &tm_v, j, sm.kv[slot], &sm.kv_full[slot], lane);
        return true;
      });
    }
    if (sm.abort_flag != 0 && lane == 0) flight.drain(sm.kv_full, status);
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (whole warp)
    const PgWait wc{&sm.abort_flag, 32};
    // K, Q K-major; V MN-major, P K-major
    constexpr uint32_t idesc_s =
        Q8 ? idesc_kind_f8(128, Cfg::kNS, 0, 0, 0) : idesc_kind_f16(128, Cfg::kNS, 0, 0, ElemOps<E>::kMmaType);
    constexpr uint32_t idesc_o =
        Q8 ? idesc_kind_f8(D, Cfg::kNO, 1, 0, 1) : idesc_kind_f16(D, Cfg::kNO, 1, 0, ElemOps<E>::kMmaType);
    constexpr uint32_t kGroup = 8 * Cfg::kRowBytes;  // 8-row groups
    auto desc = [](const void* p, uint32_t lbo, uint32_t sbo) {
      return Cfg::kRowBytes == 64 ? sdesc_sw64(smem_u32(p), lbo, sbo) : sdesc_sw128(smem_u32(p), lbo, sbo);
    };
    const uint64_t dq0 = desc(sm.q[0], 16, kGroup);
    const uint64_t dp0 = sdesc_sw128(smem_u32(sm.p[0]), 16, 1024);
    const uint64_t dk0 = desc(sm.kv[0], 16, kGroup);
    const uint64_t dv0 = desc(sm.kv[0], Cfg::kChunkBytes, kGroup);
    auto issue_s = [&](int buf, int qs, int slot) {
      const uint64_t dk = dk0 + static_cast<uint64_t>((slot * Cfg::kTileBytes) >> 4);
      const uint64_t dq = dq0 + static_cast<uint64_t>((qs * Cfg::kQBytes) >> 4);
      const uint32_t tS = tbase + buf * Cfg::kNS;
      if constexpr (Q8) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          umma_ss_f8_w(tS, dk + ((kk * 32) >> 4), dq + ((kk * 32) >> 4), idesc_s, kk > 0);
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_w(tS, dk + (((kk / 4) * Cfg::kChunkBytes + (kk % 4) * 32) >> 4),
                    dq + (((kk / 4) * Cfg::kQPartBytes + (kk % 4) * 32) >> 4), idesc_s, kk > 0);
      }
    };
    auto issue_pv = [&](int grp, int slot, uint32_t acc) {
      const uint64_t dv = dv0 + static_cast<uint64_t>((slot * Cfg::kTileBytes) >> 4);
      const uint64_t dp = dp0 + static_cast<uint64_t>((grp * Cfg::kPBytes) >> 4);
      const uint32_t tO = tbase + Cfg::kOCol + grp * Cfg::kNO;
      if constexpr (Q8) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss_f8_w(tO, dv + ((kk * 32 * Cfg::kRowBytes) >> 4), dp + ((kk * 32) >> 4), idesc_o, (kk > 0) || acc);
      } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss_w(tO, dv + ((kk * 16 * 128) >> 4), dp + (((kk / 4) * Cfg::kPChunkBytes + (kk % 4) * 32) >> 4), idesc_o,
                    (kk > 0) || acc);
      }
    };
    uint32_t it = 0, qcnt = 0, scnt = 0, pcnt[2] = {0, 0};
    bool ok = true;
    while (ok) {
      const PgSeg* gp = next_seg(wc);
      if (gp == nullptr) break;
      const PgSeg& g = *gp;
      const int nt = g.nt, kt0 = g.kt0;
      const int qs = (nseg - 1) & 1;
      // Step n issues the products of tile n - kAhead with its weights and the scores of tile n.
      // A score buffer was last read for the tile four before, whose weights (posted after the
      // read) have been waited for by then.
      for (int n = 0; n < nt + Cfg::kAhead; ++n) {
        const int t = n - Cfg::kAhead;
        const bool pv = t >= 0, sc = n < nt;
        const int grp = t & 1;
        const uint32_t p = grp ? pcnt[1] : pcnt[0];
        const uint32_t itk = it + pv;
        // the ring's order is V_t, K_n
        if (pv && pg_cleans(g, kt0 + t)) {
          ok = pg_wait(&sm.kv_full[it % NS], (it / NS) & 1, wc);
          if (!ok) break;
          pg_clean<Cfg::kRowBytes, Cfg::kChunks>(g, kt0 + t, sm.kv[it % NS], lane);
        }
        uint64_t* bar = nullptr;
        uint32_t parity = 0;
        if (lane == 0 && pv) bar = &sm.kv_full[it % NS], parity = (it / NS) & 1;
        if (lane == 1 && pv) bar = &sm.p_full[grp], parity = p & 1;
        if (lane == 2 && sc) bar = &sm.kv_full[itk % NS], parity = (itk / NS) & 1;
        if (lane == 3 && n == 0) bar = &sm.q_full[qs], parity = (qcnt >> 1) & 1;
        ok = pg_wait_lanes(bar, parity, wc);
        if (!ok) break;
        tc_fence_after();
        if (pv) {
          if (grp) ++pcnt[1]; else ++pcnt[0];
          const int slot = it % NS;
          ++it;
          issue_pv(grp, slot, t >= 2);
          umma_commit_w(&sm.p_empty[grp]);
          umma_commit_w(&sm.kv_empty[slot]);
        }
        if (sc) {
          const int slot = it % NS;
          ++it;
          const int buf = scnt % NB;
          ++scnt;
          issue_s(buf, qs, slot);
          umma_commit_w(&sm.s_full[buf]);
          umma_commit_w(&sm.kv_empty[slot]);
          if (n == nt - 1) umma_commit_w(&sm.q_empty[qs]);
        }
      }
      ++qcnt;
    }
    // Wait for every MMA issued to finish before the columns are freed.
    umma_commit_w(&sm.mma_drain);
    mbar_wait_drain(&sm.mma_drain, 0, status);
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax groups
    const int grp = warp >> 2;
    const int wq = warp & 3;
    const int me = wq * 32 + lane;  // this thread's key of a tile
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tO = tbase + Cfg::kOCol + grp * Cfg::kNO + lane_off;
    const PgWait wc{&sm.abort_flag, 33 + grp};
    uint8_t* const prow = sm.p[grp];
    uint32_t tiles = 0, mine = 0, gcnt = 0, xcnt = 0;  // score tiles, the group's, barriers passed
    bool ok = true;
    auto sync4 = [&]() -> bool {  // the group's warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.group[grp]);
      const bool r = pg_wait(&sm.group[grp], gcnt & 1, wc);
      ++gcnt;
      return r;
    };
    auto sync8 = [&]() -> bool {  // both groups
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.groups);
      const bool r = pg_wait(&sm.groups, xcnt & 1, wc);
      ++xcnt;
      return r;
    };
    while (ok) {
      const PgSeg* gp = next_seg(wc);
      if (gp == nullptr) break;
      const PgSeg& g = *gp;
      const int M = G * g.ntok;
      const int nt = g.nt, kt0 = g.kt0;
      // every row sees the keys from all_lo to all_hi
      const int all_hi = a.causal ? g.pos0 : g.len - 1;
      const int all_lo = pg_first_key(a, g.pos0 + g.ntok - 1);
      float ref[RW], l[RW], lr[RW], c_row[Q8 ? RW : 1];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        ref[r] = -INFINITY;
        l[r] = lr[r] = 0.f;
      }
      if constexpr (Q8) {
        // log2 units per score: the scale and the row's query factor
        int i = 0, h = 0;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          c_row[r] = a.scale_log2;
          if (r < M && FA_IN_BOUNDS(g.q0 + i < a.T && h < G, status, 521))
            c_row[r] *= __ldg(a.q_scale + (static_cast<int64_t>(g.q0) + i) * a.H + g.kvh * G + h);
          if (++h == G) h = 0, ++i;
        }
      }
      int e_ref = 0;
      bool first = true;
      for (int t = grp; t < nt; t += 2) {
        const uint32_t tile = tiles + t;
        const int buf = tile % NB, ss = tile % NSC;
        // the scores, the scales, and the group's previous products: P^T may then be overwritten and
        // O^T rescaled
        ok = pg_wait_lanes(lane == 0   ? &sm.s_full[buf]
                           : lane == 1 ? &sm.p_empty[grp]
                           : Q8 && lane == 2 ? &sm.sc_full[ss]
                                             : nullptr,
                           lane == 0 ? (tile / NB) & 1 : (lane == 1 ? (mine & 1) ^ 1 : (tile / NSC) & 1), wc);
        if (!ok) break;
        tc_fence_after();
        float kf = 1.f;
        int vb = 0, e = -127;  // the key's value scale byte, the largest exponent of the warp's keys
        if constexpr (Q8) {
          kf = e8m0_to_float(sm.scales[ss][0][me]);
          vb = sm.scales[ss][1][me];
          const int key = ((kt0 + t) << 7) + me;
          const bool in = key >= g.keys.lo && key < g.keys.hi;  // stale bytes may be anything
          if (!in) vb = 127;
          e = __reduce_max_sync(kFull, in && vb != 255 ? vb - 127 : -127);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sc_empty[ss]);
        }
        float x[RW];  // scores in log2 units
        {
          uint32_t s[Q8 ? Cfg::kQPieces * RW : RW];
          tmem_ld_cols(tbase + buf * Cfg::kNS + lane_off, s);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            if constexpr (Q8) {
              float sum = __uint_as_float(s[r]) + __uint_as_float(s[RW + r]);
              if constexpr (Cfg::kQPieces == 3) sum += __uint_as_float(s[2 * RW + r]);
              x[r] = sum * kf * c_row[r];
            } else {
              x[r] = __uint_as_float(s[r]) * a.scale_log2;
            }
          }
        }
        const int k0 = (kt0 + t) << 7;
        if (k0 + 127 > all_hi || k0 < all_lo) {
          const int key = k0 + me;
          int i = 0, h = 0;
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const int pos = g.pos0 + i;
            const int hi = a.causal ? min(pos, g.len - 1) : g.len - 1;
            const int lo = pg_first_key(a, pos);
            if (key > hi || key < lo) x[r] = -INFINITY;
            if (++h == G) h = 0, ++i;
          }
        }
        bool raise = false;
#pragma unroll
        for (int r = 0; r < RW; ++r) raise = raise || (r < M && x[r] > ref[r] + kRaise);
        const bool any = __any_sync(kFull, raise);
        if (lane == 0) sm.flag[grp][mine & 1][wq] = e * 2 + any;
        ok = sync4();
        if (!ok) break;
        const int4 flags = *reinterpret_cast<const int4*>(sm.flag[grp][mine & 1]);
        bool raised = (flags.x | flags.y | flags.z | flags.w) & 1, grown = false;
        if constexpr (Q8) {
          e = max(max(flags.x, flags.y), max(flags.z, flags.w)) >> 1;
          if (!first) e = max(e, e_ref);
          grown = !first && e > e_ref;
          raised = raised || grown;
        }
        if (raised) {
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float m = warp_max(x[r]);
            if (lane == 0) sm.top[grp][wq][r] = m;
          }
          ok = sync4();
          if (!ok) break;
          const float shrink = (grown && e - e_ref <= 126) ? __int_as_float((127 + e_ref - e) << 23) : (grown ? 0.f : 1.f);
          float alpha[RW];
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float m = fmaxf(fmaxf(sm.top[grp][0][r], sm.top[grp][1][r]),
                                  fmaxf(sm.top[grp][2][r], sm.top[grp][3][r]));
            const bool up = m > ref[r] + kRaise;
            alpha[r] = up ? ex2_approx(ref[r] - m) : 1.f;
            l[r] *= alpha[r];
            lr[r] *= alpha[r];
            if (up) ref[r] = m;
            alpha[r] *= shrink;
          }
          if (!first) {
#pragma unroll
            for (int c = 0; c < (Q8 ? Cfg::kPPieces * RW : RW); c += 8) {
              uint32_t o[8];
              tmem_ld8(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha[(c + y) % RW]);
              tmem_st8(tO + c, o);
            }
            tmem_wait_st();
          }
        }
        e_ref = e;
        const float vf = Q8 ? pg_factor(vb, e) : 1.f;
        // weights, and their place in P^T: row r, this thread's key
        if constexpr (Q8) {
          const uint32_t at = me & 15;
          const uint32_t unit = me >> 4;
#pragma unroll
          for (int r = 0; r < RW; r += 2) {
            float w[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float p = ex2_approx(x[r + y] - (ref[r + y] == -INFINITY ? 0.f : ref[r + y]) + kPShift);
              l[r + y] += p;
              w[y] = p * vf;
              // Three pieces hold 9 significant bits: rounded to the nearest, here, since l sums the
              // weights before it (the pieces of an fp16 as they fall cut it off, by 3.2e-4 in the mean,
              // up to 2.6e-3).  w + 2^15 w rounds at 2^-8 of w's power of two, and what is left of it
              // without 2^15 w is exact.
              if constexpr (Cfg::kPPieces == 3) w[y] = fmaf(w[y], -32768.f, fmaf(w[y], 32768.f, w[y]));
            }
            // fp16: its upper byte is the e5m2 truncation, and each remainder is exact in fp16
            uint32_t v = pack_f16x2(w[0], w[1]);
#pragma unroll
            for (int piece = 0; piece < Cfg::kPPieces; ++piece) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
                prow[(piece * RW + r + y) * 128 + ((unit ^ ((r + y) & 7)) << 4) + at] =
                    static_cast<uint8_t>(v >> (8 + 16 * y));
              if (piece + 1 < Cfg::kPPieces)
                asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(v & 0xff00ff00u));
            }
          }
        } else {
          const uint32_t base = (me >> 6) * Cfg::kPChunkBytes + (me & 7) * 2;
          const uint32_t unit = (me >> 3) & 7;
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float p = ex2_approx(x[r] - (ref[r] == -INFINITY ? 0.f : ref[r]) + kPShift);
            const T v = ElemOps<E>::one(p);
            l[r] += p;
            // bf16: the rounded weights normalise O, as in softmax_row
            lr[r] += E == Elem::kBf16 ? static_cast<float>(v) : p;
            *reinterpret_cast<T*>(prow + base + r * 128 + ((unit ^ (r & 7)) << 4)) = v;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[grp]);
        ++mine;
        first = false;
      }
      tiles += nt;
      if (!ok) break;
      // Sums over the group's keys, then both groups' weights of each row
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        if constexpr (Q8) lr[r] = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          l[r] += __shfl_xor_sync(kFull, l[r], o);
          if constexpr (!Q8) lr[r] += __shfl_xor_sync(kFull, lr[r], o);
        }
        if constexpr (Q8) lr[r] = l[r];
        if (lane == 0) sm.sums[grp][wq][r] = make_float2(l[r], lr[r]);
        if (wq == 0 && lane == 0) sm.ref[grp][r] = ref[r] - kPShift;
      }
      // the group's last product (none: passes at once)
      ok = pg_wait(&sm.p_empty[grp], (mine & 1) ^ 1, wc);
      if (!ok) break;
      tc_fence_after();
      if (Q8 && wq == 0 && lane == 0) sm.top[grp][0][0] = e8m0_to_float(static_cast<uint32_t>(e_ref + 127));
      ok = sync8();
      if (!ok) break;
      const int64_t part0 = (static_cast<int64_t>(blockIdx.x) * 2 + g.slot) * Cfg::kRows;
      if (grp == 0 && me < M) {
        float2 sum[2];
        float m[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          sum[y] = make_float2(0.f, 0.f);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            sum[y].x += sm.sums[y][z][me].x;
            sum[y].y += sm.sums[y][z][me].y;
          }
          m[y] = sm.ref[y][me];
        }
        const float mm = fmaxf(m[0], m[1]);
        const float top = mm == -INFINITY ? 0.f : mm;
        const float e0 = ex2_approx(m[0] - top), e1 = ex2_approx(m[1] - top);
        const float ls = e0 * sum[0].x + e1 * sum[1].x, lrs = e0 * sum[0].y + e1 * sum[1].y;
        sm.weight[0][me] = sum[0].y == 0.f || lrs == 0.f ? 0.f : e0 * (Q8 ? sm.top[0][0][0] : 1.f) / lrs;
        sm.weight[1][me] = sum[1].y == 0.f || lrs == 0.f ? 0.f : e1 * (Q8 ? sm.top[1][0][0] : 1.f) / lrs;
        const float lse_l = ls == 0.f ? -INFINITY : (top + lg2_approx(ls)) * kLn2;
        const float lse_r = lrs == 0.f ? -INFINITY : (top + lg2_approx(lrs)) * kLn2;
        const int i = me / G;
        const int64_t token = static_cast<int64_t>(g.q0) + i;
        const int h = g.kvh * G + me - i * G;
        if (g.whole) {
          if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H, status, 522))
            a.lse[static_cast<int64_t>(h) * a.T + token] = lse_l;
        } else if (FA_IN_BOUNDS(part0 + me < a.slots * Cfg::kRows, status, 523)) {
          *reinterpret_cast<float2*>(a.part_lse + (part0 + me) * 2) = make_float2(lse_l, lse_r);
        }
      }
      ok = sync8();
      if (!ok) break;
      // O^T: a thread holds one column of the rows, of the group's own keys (a group without tiles
      // has weight 0 and unwritten columns)
      const int d = D == 128 ? me : wq * 16 + lane;
      const bool has = !first;
      const bool live = D == 128 || lane < 16;
      auto rows8 = [&](int r0, float (&v)[8]) {
#pragma unroll
        for (int y = 0; y < 8; ++y) v[y] = 0.f;
        if (has) {
#pragma unroll
          for (int piece = 0; piece < (Q8 ? Cfg::kPPieces : 1); ++piece) {
            uint32_t o[8];
            tmem_ld8(tO + piece * RW + r0, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 8; ++y) v[y] += __uint_as_float(o[y]);
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float w = r0 + y < M ? sm.weight[grp][r0 + y] : 0.f;
            v[y] = w == 0.f ? 0.f : v[y] * w;
          }
        }
      };
      if (grp == 1) {
#pragma unroll 1
        for (int r0 = 0; r0 < M; r0 += 8) {
          float v[8];
          rows8(r0, v);
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (live) sm.part[r0 + y][d] = v[y];
        }
      }
      ok = sync8();
      if (!ok) break;
      if (grp == 0) {
#pragma unroll 1
        for (int r0 = 0; r0 < M; r0 += 8) {
          float v[8];
          rows8(r0, v);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = r0 + y;
            if (!live || r >= M) continue;
            const float o = v[y] + sm.part[r][d];
            const int i = r / G;
            const int64_t token = static_cast<int64_t>(g.q0) + i;
            const int h = g.kvh * G + r - i * G;
            if (g.whole) {
              if (FA_IN_BOUNDS(token >= 0 && token < a.T && h < a.H && d < D, status, 524))
                static_cast<T*>(a.out)[(token * a.H + h) * D + d] = ElemOps<E>::one(o);
            } else if (FA_IN_BOUNDS(part0 + r < a.slots * Cfg::kRows && d < D, status, 525)) {
              a.part_o[(part0 + r) * D + d] = o;
            }
          }
        }
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
  if (threadIdx.x == 0) pg_report(&sm.abort_flag, status);
}

}  // namespace fa
