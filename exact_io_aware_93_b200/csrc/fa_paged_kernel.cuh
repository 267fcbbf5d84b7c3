// fa_paged_kernel.cuh -- exact attention over a paged cache with tiles of 128 query rows, for
// sm_100a: chunks of a prompt, and sequences with too many rows for fa_paged_few_kernel.cuh.  The
// work list, the page loads and the join of partial results are in fa_paged_common.cuh.
//
// TQ = floor(128 / G) tokens fill a tile (rows past G * TQ are zero).  Two ways through a segment:
//   pair    two tiles: softmax group g owns tile g and both share one stream of K/V tiles, in
//           the order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1) of the forward kernel.
//   split   one tile: group g takes the segment's key tiles g, g + 2, ..: two independent
//           online softmaxes over disjoint keys, joined through shared memory at its end.
//
// e4m3 pages.  Codes land in a ring of their own and a fourth warpgroup turns them into fp16
// tiles, for queries that are fp16 too (scaled by a power of two per row, fa_paged_scale_q_kernel)
// and whatever the outputs' type.  Row j of a tile becomes code * 2^(e_j - E): E is the tile's
// largest exponent for K (the softmax multiplies the scores by 2^E) and the segment's largest so
// far for V (O is rescaled when it grows), so the fp16 products are exact but for rows 2^-15
// below the largest.  fp16 and not the queries' type: e4m3 to fp16 is one conversion per pair of
// codes, to bf16 it took 10 integer operations per four codes and 2116 cycles per tile.  (Feeding
// the codes to the tensor core as they are, with two e4m3 pieces per query and per-key scales
// applied to the scores by the softmax, was no faster: 32 factors a row and tile read from shared
// memory beside operands that already saturate it.)
//
// Warp roles (384 threads, 512 with e4m3 pages): warps 0-3 and 4-7 the softmax groups, warp 8 the
// schedule and the loads of Q and K, warp 10 those of V, warp 9 the MMA issuer, warp 11 the scales,
// warps 12-15 the conversion.
//
// Bound by the chain scores, softmax, weights, products of a tile, as the forward kernel: 2048 new tokens
// at 32K, 32 heads sharing 8, d 128, 16-bit pages 1.15 to 1.19 ms under the power cap (895 to 925 TFLOP/s),
// 1016 us (1048) in a short run; there, with 2 key/value heads, whose pages stay in L2, 1109 TFLOP/s, and
// over e4m3 pages 1217 us (875), bound by the conversion and the three converted tiles that fit.
//
// Tensor memory: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 [256+D,256+2D); P
// overwrites the second half of S.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

constexpr uint32_t kPagedLaunchRegs = 168;      // 16-bit pages
constexpr uint32_t kPagedLaunchRegsConv = 128;  // e4m3 pages

template <int D, Elem E, bool Q8>
struct PgCfg {
  static constexpr int kRows = 128;                   // rows of a partial result
  static constexpr int kSubs = 2;                     // partial results per segment
  static constexpr int kStageCols = 16;               // columns joined at a time
  static constexpr int kStageBufs = Q8 ? 1 : 2;
  static constexpr int kThreads = Q8 ? 512 : 384;
  // setmaxnreg: 2 x 128 x 200 + 128 x 104 of 384 x 168, and with the conversion warps
  // 128 x (2 x 184 + 72 + 72) of 512 x 128
  static constexpr uint32_t kLaunch = Q8 ? kPagedLaunchRegsConv : kPagedLaunchRegs;
  static constexpr uint32_t kRegsSoftmax = Q8 ? 184 : 200;
  static constexpr uint32_t kRegsOther = Q8 ? 72 : 104;
  static_assert(2 * kRegsSoftmax + (Q8 ? 2 : 1) * kRegsOther <= kLaunch * (kThreads / 128), "register split");
  // time of a key tile, in the work list's units: of a pair, and of a single tile
  static constexpr int kPairCost = 3;
  static constexpr int kSplitCost = 2;
  // the end of a unit, 5.5 us.  (Without it CTAs of several short units ended 18 us after the mean: 24
  // sequences of 700 to 16384 tokens, 5 new ones each, window 4096, 64.6 us; 4 / 6 / 8 / 12: 56.3 / 52.6 /
  // 51.6 / 51.3.)
  static constexpr int kUnitCost = 8;
  static constexpr int kChunks = D / 64;              // 128-byte chunks of a 16-bit row
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kScale = 128 / D;              // slots scale with the tile
  static constexpr int kStages = (Q8 ? 3 : 4) * kScale;
  static constexpr int kRaw = Q8 ? 3 * kScale : 1;
  static constexpr int kRawBytes = Q8 ? 128 * D : 16;
  static constexpr int kScaleRing = 4;
  static constexpr int kSegRing = 4;
  static constexpr int kSegReaders = Q8 ? 15 : 10;    // warps
  static constexpr uint32_t kOCol = 256;
  static constexpr uint32_t kTmemCols = 512;
};

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

// Of a key tile: the factor of its scores, and the exponent of O from it on.
struct PgTileScale {
  float k;
  int e;
};

template <int D, Elem E, bool Q8>
struct __align__(1024) PgSmem {
  using Cfg = PgCfg<D, E, Q8>;
  uint8_t q[2][Cfg::kTileBytes];
  uint8_t kv[Cfg::kStages][Cfg::kTileBytes];
  uint8_t raw[Cfg::kRaw][Cfg::kRawBytes];
  alignas(16) float stage[Cfg::kStageBufs][128 * Cfg::kStageCols];  // a split segment's columns being joined
  alignas(16) uint32_t factors[Q8 ? Cfg::kScaleRing : 1][2][128];   // of K's and V's rows: fp16, twice
  PgTileScale scales[2][Cfg::kScaleRing];                           // of each softmax group's tiles
  float3 stat[2][128];                                              // m, l, lr of a split segment's groups
  PgSeg segs[Cfg::kSegRing];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t kv_full[Cfg::kStages];
  uint64_t kv_empty[Cfg::kStages];
  uint64_t raw_full[Cfg::kRaw];
  uint64_t raw_empty[Cfg::kRaw];
  uint64_t sc_full[2][Cfg::kScaleRing];
  uint64_t sc_empty[2][Cfg::kScaleRing];
  uint64_t fac_full[Cfg::kScaleRing];
  uint64_t fac_empty[Cfg::kScaleRing];
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

template <int D, Elem E, bool Q8>
__global__ void __launch_bounds__(PgCfg<D, E, Q8>::kThreads, 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PgArgs a) {
  using Cfg = PgCfg<D, E, Q8>;
  constexpr int NS = Cfg::kStages;
  constexpr int NSC = Cfg::kScaleRing;
  constexpr int NSEG = Cfg::kSegRing;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr float kShift = kWeightShift<Q8 ? Elem::kF16 : E>;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset and not through an integer: the compiler keeps seeing shared memory
  PgSmem<D, E, Q8>& sm = *reinterpret_cast<PgSmem<D, E, Q8>*>(smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u);
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
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_done[i], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.kv_full[s], Q8 ? 4 : 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    if constexpr (Q8) {
      for (int s = 0; s < NSC; ++s) {
        for (int i = 0; i < 2; ++i) {
          mbar_init(&sm.sc_full[i][s], 1);
          mbar_init(&sm.sc_empty[i][s], 4);
        }
        mbar_init(&sm.fac_full[s], 1);
        mbar_init(&sm.fac_empty[s], 4);
      }
      for (int s = 0; s < Cfg::kRaw; ++s) {
        mbar_init(&sm.raw_full[s], 1);
        mbar_init(&sm.raw_empty[s], 4);
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
  for (uint32_t i = threadIdx.x; i < 2u * Cfg::kTileBytes / 16; i += Cfg::kThreads)
    reinterpret_cast<uint4*>(sm.q[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, Cfg::kTmemCols);
    tmem_relinquish();
  }
  // Launched while the kernel before it may still run: what that one writes is read from here on.
  // (e4m3 pages: it is the scaling of the queries, which has waited for the kernel before it and
  // writes nothing that the plan reads.)  Behind the few-rows kernel (a mixed batch), which has waited
  // before it let this one start, nothing is left to wait for: its end is waited for at this one's.
  if constexpr (!Q8)
    if (!a.behind) asm volatile("griddepcontrol.wait;" ::: "memory");
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
  if constexpr (Q8)
    if (!a.behind) asm volatile("griddepcontrol.wait;" ::: "memory");
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

  // Each warpgroup's setmaxnreg sits at the top of the branch holding all of its code.
  if (warp >= 8 && warp < 12) {
    regs_set<Cfg::kLaunch, Cfg::kRegsOther>();
    if (warp == 8) {
      // ---------------------------------------------------------- schedule and TMA loads
      const PgWait wc{&sm.abort_flag, 31};
      PgWalk<Cfg> w(a, sm.plan);
      PgSeg g;
      PgPages pages{};
      PgInFlight flight;
      uint32_t it = 0, qcnt[2] = {0, 0};
      bool ok = true;
      auto load_q = [&](int slot, int tok) -> bool {
        if (!pg_wait(&sm.q_empty[slot], (qcnt[slot] & 1) ^ 1, wc)) return false;
        if (lane == 0)
          mbar_arrive_expect_tx(&sm.q_full[slot], static_cast<uint32_t>(Cfg::kChunks * 128 * G * a.TQ));
        __syncwarp();
        if (lane < Cfg::kChunks &&
            FA_IN_BOUNDS(tok >= 0 && tok < a.T && g.kvh < a.H_kv && G * a.TQ <= Cfg::kRows, status, 501))
          tma_load_4d(sm.q[slot] + lane * Cfg::kChunkBytes, &tm_q, &sm.q_full[slot], lane * 64, 0, g.kvh, tok);
        __syncwarp();
        ++qcnt[slot];
        return true;
      };
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
        ++nseg;
        if (!more) break;
        if (g.pair) {
          for (int x = 0; x < 2 && ok; ++x)
            if (g.tile[x].hi > g.tile[x].lo) ok = load_q(x, g.q0 + x * a.TQ);
        } else {
          ok = load_q(0, g.q0);
        }
        if (!ok) break;
        ok = pg_loads<2>(g, [&](bool isv, int j) -> bool {
          constexpr int N = Q8 ? Cfg::kRaw : NS;
          const int slot = it % N;
          const uint32_t phase = (it / N) & 1;
          ++it;
          if (isv) return true;
          if (!pg_wait(Q8 ? &sm.raw_empty[slot] : &sm.kv_empty[slot], phase ^ 1, wc)) return false;
          flight.add(slot, phase);
          if constexpr (Q8)
            pg_load_tile<D, 1>(a, g, pages, &tm_k, j, sm.raw[slot], &sm.raw_full[slot], lane);
          else
            pg_load_tile<128, Cfg::kChunks>(a, g, pages, &tm_k, j, sm.kv[slot], &sm.kv_full[slot], lane);
          return true;
        });
      }
      if (lane == 0 && FA_IN_BOUNDS(static_cast<int>(blockIdx.x) * 2 < a.slots, status, 514)) a.splits[blockIdx.x] = w.split;
      if (!ok && lane == 0) {
        flight.drain(Q8 ? sm.raw_full : sm.kv_full, status);
        for (int i = 0; i < 2; ++i)
          if (qcnt[i] > 0) mbar_wait_drain(&sm.q_full[i], (qcnt[i] - 1) & 1, status);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---------------------------------------------------------- loads of V
      const PgWait wc{&sm.abort_flag, 37};
      PgPages pages{};
      PgInFlight flight;
      uint32_t it = 0;
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        pages.start(a, *gp, lane);
        ok = pg_loads<2>(*gp, [&](bool isv, int j) -> bool {
          constexpr int N = Q8 ? Cfg::kRaw : NS;
          const int slot = it % N;
          const uint32_t phase = (it / N) & 1;
          ++it;
          if (!isv) return true;
          if (!pg_wait(Q8 ? &sm.raw_empty[slot] : &sm.kv_empty[slot], phase ^ 1, wc)) return false;
          flight.add(slot, phase);
          if constexpr (Q8)
            pg_load_tile<D, 1>(a, *gp, pages, &tm_v, j, sm.raw[slot], &sm.raw_full[slot], lane);
          else
            pg_load_tile<128, Cfg::kChunks>(a, *gp, pages, &tm_v, j, sm.kv[slot], &sm.kv_full[slot], lane);
          return true;
        });
      }
      if (sm.abort_flag != 0 && lane == 0) flight.drain(Q8 ? sm.raw_full : sm.kv_full, status);
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer (whole warp)
      const PgWait wc{&sm.abort_flag, 32};
      // Q, K K-major; P in TMEM, V MN-major
      constexpr uint32_t kType = Q8 ? 0 : ElemOps<E>::kMmaType;  // e4m3 pages: all operands fp16
      constexpr uint32_t idesc_s = idesc_kind_f16(128, kBN, 0, 0, kType);
      constexpr uint32_t idesc_o = idesc_kind_f16(128, D, 0, 1, kType);
      const uint64_t dq[2] = {sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), sdesc_sw128(smem_u32(sm.q[1]), 16, 1024)};
      const uint64_t dk0 = sdesc_sw128(smem_u32(sm.kv[0]), 16, 1024);
      const uint64_t dv0 = sdesc_sw128(smem_u32(sm.kv[0]), Cfg::kChunkBytes, 1024);
      auto issue_s = [&](int i, int qs, int slot) {
        const uint64_t dk = dk0 + static_cast<uint64_t>((slot * Cfg::kTileBytes) >> 4);
        const uint64_t dqi = qs ? dq[1] : dq[0];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * Cfg::kChunkBytes + (kk % 4) * 32) >> 4;
          umma_ss_w(tbase + i * 128, dqi + off, dk + off, idesc_s, kk > 0);
        }
      };
      auto issue_pv = [&](int i, int slot, uint32_t acc) {
        const uint64_t dv = dv0 + static_cast<uint64_t>((slot * Cfg::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          umma_ts_w(tbase + Cfg::kOCol + i * D, tbase + i * 128 + 64 + kk * 8, dv + ((kk * 16 * 128) >> 4), idesc_o,
                    (kk > 0) || acc);
      };
      uint32_t it = 0, qcnt[2] = {0, 0}, pcnt[2] = {0, 0};
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        const bool pair = g.pair;
        const int kt0 = g.kt0, kend = g.kt0 + g.nt;
        const PgRange rg0 = pair ? g.tile[0] : PgRange{kt0, kend}, rg1 = pair ? g.tile[1] : rg0;
        if (pair) {
          uint64_t* q = lane == 0 && rg0.hi > rg0.lo ? &sm.q_full[0] : (lane == 1 && rg1.hi > rg1.lo ? &sm.q_full[1] : nullptr);
          ok = pg_wait_lanes(q, (lane ? qcnt[1] : qcnt[0]) & 1, wc);
        } else {
          ok = pg_wait(&sm.q_full[0], qcnt[0] & 1, wc);
        }
        if (!ok) break;
        if (pair) {
          // per key tile: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1); the first round has scores only
          for (int j = kt0 - 1; j < kend; ++j) {
            const bool v = j >= kt0, k = j + 1 < kend;
            const uint32_t itk = it + v;
            const int sv = it % NS, sk = itk % NS;
            if (!Q8 && v && pg_cleans(g, j)) {
              ok = pg_wait(&sm.kv_full[sv], (it / NS) & 1, wc);
              if (!ok) break;
              pg_clean<128, Cfg::kChunks>(g, j, sm.kv[sv], lane);
            }
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const PgRange r = i ? rg1 : rg0;
              const bool pv = j >= r.lo && j < r.hi, sc = j + 1 >= r.lo && j + 1 < r.hi;
              // with a ring of three converted tiles K_{j+1} is not there before V_{j-1}'s slot is
              // free: there it is waited for after the products
              uint64_t* bar = nullptr;
              uint32_t parity = 0;
              if (lane == 0 && pv) bar = &sm.p_full[i], parity = (i ? pcnt[1] : pcnt[0]) & 1;
              if (lane == 1 && i == 0 && v) bar = &sm.kv_full[sv], parity = (it / NS) & 1;
              if (lane == 2 && i == 0 && k && !Q8) bar = &sm.kv_full[sk], parity = (itk / NS) & 1;
              ok = pg_wait_lanes(bar, parity, wc);
              if (!ok) break;
              tc_fence_after();
              if (pv) {
                if (i) ++pcnt[1]; else ++pcnt[0];
                issue_pv(i, sv, j > r.lo);
                if (j + 1 == r.hi) umma_commit_w(&sm.o_done[i]);
              }
              if (i == 1 && v) umma_commit_w(&sm.kv_empty[sv]);
              if (Q8 && i == 0 && k) {
                ok = pg_wait(&sm.kv_full[sk], (itk / NS) & 1, wc);
                if (!ok) break;
                tc_fence_after();
              }
              if (sc) {
                issue_s(i, i, sk);
                umma_commit_w(&sm.s_full[i]);
                if (j + 2 == r.hi) umma_commit_w(&sm.q_empty[i]);
              }
            }
            if (!ok) break;
            if (k) umma_commit_w(&sm.kv_empty[sk]);
            it += v + k;
          }
        } else {
          // PV_i(j), S_i(j+2), the groups in turn; the first two rounds have scores only
          for (int j = kt0 - 2; j < kend; ++j) {
            const int i = (j - kt0) & 1;
            const bool v = j >= kt0, k = j + 2 < kend;
            const uint32_t itk = it + v;
            const int sv = it % NS, sk = itk % NS;
            if (!Q8 && v && pg_cleans(g, j)) {
              ok = pg_wait(&sm.kv_full[sv], (it / NS) & 1, wc);
              if (!ok) break;
              pg_clean<128, Cfg::kChunks>(g, j, sm.kv[sv], lane);
            }
            uint64_t* bar = nullptr;
            uint32_t parity = 0;
            if (lane == 0 && v) bar = &sm.p_full[i], parity = (i ? pcnt[1] : pcnt[0]) & 1;
            if (lane == 1 && v) bar = &sm.kv_full[sv], parity = (it / NS) & 1;
            if (lane == 2 && k && !(Q8 && v)) bar = &sm.kv_full[sk], parity = (itk / NS) & 1;
            ok = pg_wait_lanes(bar, parity, wc);
            if (!ok) break;
            tc_fence_after();
            if (v) {
              if (i) ++pcnt[1]; else ++pcnt[0];
              issue_pv(i, sv, j - 2 >= kt0);
              umma_commit_w(&sm.kv_empty[sv]);
              if (j + 2 >= kend) umma_commit_w(&sm.o_done[i]);
            }
            if (k) {
              if (Q8 && v) {
                ok = pg_wait(&sm.kv_full[sk], (itk / NS) & 1, wc);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(i, 0, sk);
              umma_commit_w(&sm.s_full[i]);
              umma_commit_w(&sm.kv_empty[sk]);
              if (j + 3 == kend) umma_commit_w(&sm.q_empty[0]);
            }
            it += v + k;
          }
        }
        if (!ok) break;
        if (rg0.hi > rg0.lo) ++qcnt[0];
        if (pair && rg1.hi > rg1.lo) ++qcnt[1];
      }
      // Wait for every MMA issued to finish before the columns are freed.
      umma_commit_w(&sm.mma_drain);
      mbar_wait_drain(&sm.mma_drain, 0, status);
      __syncwarp();
    } else if constexpr (Q8) {
      // ---------------------------------------------------------- scales
      const PgWait wc{&sm.abort_flag, 35};
      PgScaleStream stream;
      uint32_t tiles = 0, cnt[2] = {0, 0};
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        int e = -127;
        ok = stream.run(a, g, lane, [&](int j, uint32_t kw, uint32_t vw) -> bool {
          const int top = max(pg_top(g, j, lane, kw), -127);
          e = max(e, pg_top(g, j, lane, vw));
          // the conversion's factors of the tile's rows
          const int fs = tiles % NSC;
          if (!pg_wait(&sm.fac_empty[fs], ((tiles / NSC) & 1) ^ 1, wc)) return false;
          ++tiles;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t w = kv ? vw : kw;
            uint32_t f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = pg_factor16((w >> (8 * x)) & 255, kv ? e : top) * 0x10001u;
            *reinterpret_cast<uint4*>(sm.factors[fs][kv] + lane * 4) = make_uint4(f[0], f[1], f[2], f[3]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.fac_full[fs]);
          // each softmax group's exponents of its tiles
#pragma unroll 1
          for (int grp = 0; grp < 2; ++grp) {
            if (!(g.pair ? j >= g.tile[grp].lo && j < g.tile[grp].hi : ((j - g.kt0) & 1) == grp)) continue;
            const uint32_t c = grp ? cnt[1] : cnt[0];
            const int slot = c % NSC;
            if (!pg_wait(&sm.sc_empty[grp][slot], ((c / NSC) & 1) ^ 1, wc)) return false;
            if (grp) ++cnt[1]; else ++cnt[0];
            if (lane == 0) {
              sm.scales[grp][slot] = PgTileScale{e8m0_to_float(static_cast<uint32_t>(top + 127)), e};
              mbar_arrive(&sm.sc_full[grp][slot]);
            }
            __syncwarp();
          }
          return true;
        });
      }
    }
  } else if (Q8 && warp >= 12) {
    // ------------------------------------------------------------ codes to fp16 tiles
    if constexpr (Q8) {
      regs_set<Cfg::kLaunch, Cfg::kRegsOther>();
      const PgWait wc{&sm.abort_flag, 36};
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
      uint32_t it = 0, tiles = 0;
      bool ok = true;
      while (ok) {
        const PgSeg* gp = next_seg(wc);
        if (gp == nullptr) break;
        const PgSeg& g = *gp;
        ok = pg_loads<2>(g, [&](bool isv, int j) -> bool {
          const int rs = it % Cfg::kRaw, ks = it % NS;
          const uint32_t tile = tiles + (j - g.kt0);
          const int fs = tile % NSC;
          if (!pg_wait_lanes(lane == 0   ? &sm.fac_full[fs]
                             : lane == 1 ? &sm.raw_full[rs]
                             : lane == 2 ? &sm.kv_empty[ks]
                                         : nullptr,
                             lane == 0 ? (tile / NSC) & 1 : (lane == 1 ? (it / Cfg::kRaw) & 1 : ((it / NS) & 1) ^ 1), wc))
            return false;
          ++it;
          uint8_t* dst = sm.kv[ks] + (item >> 2) * Cfg::kChunkBytes;
#pragma unroll 1
          for (int base = r0; base < 128; base += U * kStep) {
            uint4 c[U];
            uint32_t f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              c[u] = *reinterpret_cast<const uint4*>(sm.raw[rs] + (base + u * kStep) * D + in_unit * 16);
              f[u] = sm.factors[fs][isv][base + u * kStep];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint32_t o[8];
              pg_convert16(c[u], f[u], o);
              uint8_t* p = dst + (base + u * kStep) * 128;
              const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]);
              const uint4 hi = make_uint4(o[4], o[5], o[6], o[7]);
              *reinterpret_cast<uint4*>(p + (first << 4)) = odd ? hi : lo;
              *reinterpret_cast<uint4*>(p + (second << 4)) = odd ? lo : hi;
            }
          }
          if (isv) {  // as pg_clean
            const int z0 = max(g.keys.lo - (j << 7), 0), z1 = min(g.keys.hi - (j << 7), 128);
            if (z0 > 0 || z1 < 128) {
              for (int row = r0; row < 128; row += kStep)
                if (row < z0 || row >= z1) {
                  *reinterpret_cast<uint4*>(dst + row * 128 + (first << 4)) = make_uint4(0u, 0u, 0u, 0u);
                  *reinterpret_cast<uint4*>(dst + row * 128 + (second << 4)) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.kv_full[ks]);
            mbar_arrive(&sm.raw_empty[rs]);
            if (isv) mbar_arrive(&sm.fac_empty[fs]);  // K_j came before
          }
          return true;
        });
        tiles += g.nt;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    regs_set<Cfg::kLaunch, Cfg::kRegsSoftmax>();
    const int grp = warp >> 2;
    const int wq = warp & 3;
    const int wrow0 = wq * 32;      // the warp's first row
    const int rc = wrow0 + lane;    // this thread's row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + grp * 128 + lane_off;
    const uint32_t tO = tbase + Cfg::kOCol + grp * D + lane_off;
    const PgWait wc{&sm.abort_flag, 33 + grp};
    uint32_t scnt = 0, ocnt = 0, gcnt = 0;  // scnt also counts the group's scale entries
    bool ok = true;
    while (ok) {
      const PgSeg* gp = next_seg(wc);
      if (gp == nullptr) break;
      const PgSeg& g = *gp;
      // this group's tile and its key tiles j0, j0 + dj, .. below j1
      const bool pair = g.pair;
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
        vis_lo = pg_first_key(a, qpos);
        // every row of the tile sees the keys from all_lo to all_hi
        all_hi = a.causal ? g.pos0 + tok : g.len - 1;
        all_lo = pg_first_key(a, g.pos0 + tok + M / G - 1);
        if constexpr (Q8) {
          if (rc < M && FA_IN_BOUNDS(g.q0 + tok + iq < a.T, status, 512))
            c_row *= __ldg(a.q_scale + (static_cast<int64_t>(g.q0) + tok + iq) * a.H + g.kvh * G + rc - iq * G);
        }
      }
      float m_ref = -INFINITY, l = 0.f, lr = 0.f;
      for (int j = j0; j < j1; j += dj) {
        const int ss = scnt % NSC;
        ok = pg_wait_lanes(lane == 0 ? &sm.s_full[grp] : (Q8 && lane == 1 ? &sm.sc_full[grp][ss] : nullptr),
                           lane == 0 ? scnt & 1 : (scnt / NSC) & 1, wc);
        if (!ok) break;
        ++scnt;
        tc_fence_after();
        if (rows_here) {
          const int k0 = j << 7;
          float c_tile = c_row;
          if constexpr (Q8) c_tile *= sm.scales[grp][ss].k;
          const bool masked = k0 + kBN - 1 > all_hi || k0 < all_lo;
          // Raises the reference maximum and brings O to it; `e`: with e4m3 pages the exponent of O from here
          // on (O is held in units of 2^e_ref).  The subtrahend of the weights' exponents.
          auto reference = [&](float m_new, int e) -> float {
            const bool raise = m_new > m_ref + kTau;
            bool grown = false;
            float alpha = raise ? ex2_approx(m_ref - m_new) : 1.0f;
            if (raise) {
              l *= alpha;
              lr *= alpha;
              m_ref = m_new;
            }
            if constexpr (Q8) {
              grown = j > j0 && e > e_ref;
              if (grown) alpha = e - e_ref > 126 ? 0.f : alpha * __int_as_float((127 + e_ref - e) << 23);
              e_ref = e;
            }
            if ((__any_sync(kFull, raise) || grown) && j > j0) {
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
            return (m_ref == -INFINITY ? 0.f : m_ref) - kShift;
          };
          // the largest of n scores
          auto largest = [&](const auto& s) -> float {
            constexpr int n = sizeof(s) / 4;
            float mx8[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 8]));
#pragma unroll
            for (int c = 16; c < n; c += 16)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mx8[x] = fmax3(mx8[x], __uint_as_float(s[c + x]), __uint_as_float(s[c + 8 + x]));
            return fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
          };
          auto mask = [&](auto& s, int base) {
            constexpr int n = sizeof(s) / 4;
            const int lim = vis_hi - k0 - base, first = vis_lo - k0 - base;
#pragma unroll
            for (int c = 0; c < n; ++c)
              if (c > lim || c < first) s[c] = __float_as_uint(-INFINITY);
          };
          if constexpr (!Q8) {
            // the whole row in registers
            uint32_t s[kBN], p[kBN / 2];
#pragma unroll
            for (int c = 0; c < kBN; c += 32) tmem_ld32(tS + c, s + c);
            tmem_wait_ld();
            if (masked) mask(s, 0);
            const float m_use = reference(largest(s) * c_tile, 0);
            softmax_row<E, kBN>(s, p, c_tile, m_use, l, lr);
            tmem_st32(tS + 64, p);
            tmem_st32(tS + 96, p + 32);
          } else {
            // A row is taken in halves, first for its maximum and then for its weights, in one rolled loop:
            // the roles' code together has to stay in the instruction cache (unrolled, with the conversion
            // beside it, every warp ran two to three times slower).  P lies over the second half of S,
            // which is read last before it is overwritten.
            float mx = -INFINITY, m_use = 0.f;
#pragma unroll 1
            for (int pass = 0; pass < 4; ++pass) {
              const int half = pass == 1 || pass == 2;
              uint32_t s[64];
              tmem_ld32(tS + half * 64, s);
              tmem_ld32(tS + half * 64 + 32, s + 32);
              tmem_wait_ld();
              if (masked) mask(s, half * 64);
              if (pass < 2) {
                mx = fmaxf(mx, largest(s));
                if (pass == 1) m_use = reference(mx * c_tile, sm.scales[grp][ss].e);
              } else {
                uint32_t p[32];
                softmax_row<Elem::kF16, 64>(s, p, c_tile, m_use, l, lr);
                tmem_st32(tS + 64 + half * 32, p);
              }
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&sm.p_full[grp]);
        if constexpr (Q8) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sc_empty[grp][ss]);
        }
      }
      if (!ok) break;
      float unit = 1.0f;  // of O
      if constexpr (Q8) unit = e8m0_to_float(static_cast<uint32_t>(e_ref + 127));
      if (any) {
        ok = pg_wait(&sm.o_done[grp], ocnt & 1, wc);
        if (!ok) break;
        ++ocnt;
        tc_fence_after();
      }
      const bool real = rc < M;
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
#pragma unroll
            for (int x = 0; x < n / 8; ++x)
              reinterpret_cast<uint4*>(dst)[x] = make_uint4(
                  ElemOps<E>::pack(v[8 * x], v[8 * x + 1]), ElemOps<E>::pack(v[8 * x + 2], v[8 * x + 3]),
                  ElemOps<E>::pack(v[8 * x + 4], v[8 * x + 5]), ElemOps<E>::pack(v[8 * x + 6], v[8 * x + 7]));
          }
        } else if (FA_IN_BOUNDS(part0 + row < a.slots * Cfg::kSubs * Cfg::kRows && row < Cfg::kRows && c + n <= D, status,
                                504)) {
          float* dst = a.part_o + (part0 + row) * D + c;
#pragma unroll
          for (int x = 0; x < n / 4; ++x)
            reinterpret_cast<float4*>(dst)[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
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
      // Weight of this group's O: a tile's own (pair: normalised by the sum of the rounded weights),
      // or its share of the two groups' (split: 2^(m_k - max m) / sum of lr, group 1's columns handed
      // over through shared memory).
      auto sync_groups = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.groups);
        const bool r = pg_wait(&sm.groups, gcnt & 1, wc);
        ++gcnt;
        return r;
      };
      constexpr int SC = Cfg::kStageCols;
      constexpr int kUnits = SC / 4;  // 16-byte units of a staged row; unit u sits at u ^ key(row)
      auto key = [](int r) { return (r >> 1) & (kUnits - 1); };
      if (!pair) {
        if (real) sm.stat[grp][rc] = make_float3(m_ref - kShift, l, lr);
        ok = sync_groups();
        if (!ok) break;
      }
      float mm = m_ref - kShift, ls = l, lrs = lr, wgt = 1.f;
      if (!pair && real) {
        const float3 st = sm.stat[grp ^ 1][rc];
        mm = fmaxf(m_ref - kShift, st.x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        const float mine = ex2_approx(m_ref - kShift - ref), other = ex2_approx(st.x - ref);
        // the same order in both groups
        ls = grp == 0 ? mine * l + other * st.y : other * st.y + mine * l;
        lrs = grp == 0 ? mine * lr + other * st.z : other * st.z + mine * lr;
        wgt = mine;
      }
      wgt = lr == 0.f || lrs == 0.f ? 0.f : wgt * unit / lrs;
      if (real && (pair || grp == 0)) put_lse(mm, ls, lrs);
#pragma unroll 1
      for (int c = 0; c < D; c += SC) {
        float* stage = sm.stage[(c / SC) % Cfg::kStageBufs];
        uint32_t o[SC];
        float v[SC];
        if (any && rows_here) {
          tmem_ld16(tO + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < SC; ++x) v[x] = wgt == 0.f ? 0.f : __uint_as_float(o[x]) * wgt;
        if (!pair) {
          if (real && grp == 1) {
#pragma unroll
            for (int x = 0; x < kUnits; ++x)
              *reinterpret_cast<float4*>(stage + rc * SC + ((x ^ key(rc)) << 2)) =
                  make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
          }
          ok = sync_groups();
          if (!ok) break;
          if (real && grp == 0) {
#pragma unroll
            for (int x = 0; x < kUnits; ++x) {
              const float4 y = *reinterpret_cast<const float4*>(stage + rc * SC + ((x ^ key(rc)) << 2));
              v[4 * x] += y.x;
              v[4 * x + 1] += y.y;
              v[4 * x + 2] += y.z;
              v[4 * x + 3] += y.w;
            }
          }
        }
        if (real && (pair || grp == 0)) put(rc, c, v);
        if (!pair && Cfg::kStageBufs == 1) {  // with two buffers the next barrier says that one is free
          ok = sync_groups();
          if (!ok) break;
        }
      }
      if (!ok) break;
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
  // the join waits for this kernel and reads both kernels' partial results
  if (a.behind) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace fa
