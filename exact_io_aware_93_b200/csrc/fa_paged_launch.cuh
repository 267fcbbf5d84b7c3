// fa_paged_launch.cuh -- the launches of one (element type, page type) of paged attention.
#pragma once

#include <type_traits>

#include "fa_paged_few_kernel.cuh"
#include "fa_paged_kernel.cuh"
#include "fa_paged_launch.h"
#include "tma_host.h"

namespace fa {

// Launch; with `early` the blocks may start while the kernel before them in the stream ends, and wait
// for it themselves (griddepcontrol.wait): about 1 us less between two kernels.
template <typename... P, typename... Args>
bool launch_after(bool early, void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

// One pass: the kernel for the sequences with n_lo < n <= n_hi new tokens, tiles of TQ tokens,
// and the join of its partial results.  RW: rows of the few-rows kernel, 0 for tiles of 128.
template <int D, Elem E, bool Q8, int RW>
fa_status launch_paged(DeviceInfo& di, const PagedCall& c, int n_lo, int n_hi) {
  constexpr bool kFew = RW > 0;
  using Cfg = std::conditional_t<kFew, PfCfg<D, E, Q8, kFew ? RW : 8>, PgCfg<D, E, Q8>>;
  using Smem = std::conditional_t<kFew, PfSmem<D, E, Q8, kFew ? RW : 8>, PgSmem<D, E, Q8>>;
  static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of one CTA");
  const fa_paged_problem& p = c.p;
  auto kern = [] {
    if constexpr (kFew) return fa_paged_few_kernel<D, E, Q8, RW>;
    else return fa_paged_kernel<D, E, Q8>;
  }();
  constexpr int kPieces = kFew ? paged_q_pieces(E == Elem::kF16) : 0;
  const int smem = static_cast<int>(sizeof(Smem)) + 1024;
  const int G = p.H / p.H_kv;
  const int TQ = kFew ? n_hi : 128 / G;
  const MapElem me = E == Elem::kF16 ? MapElem::kF16 : MapElem::kBf16;
  const MapElem pe = Q8 ? MapElem::kE4M3 : me;
  const long long planes = static_cast<long long>(p.P) * p.H_kv;
  const int box = p.page < 128 ? p.page : 128;
  const int grid = di.sm_count;
  const PagedLayout L = paged_layout(p, grid);
  const PagedLayout::Pass& ps = kFew ? L.few : L.many;
  uint8_t* w = static_cast<uint8_t*>(c.workspace);
  CUtensorMap mq, mk, mv;
  const bool q_ok =
      !Q8 ? make_ragged_q_map(&mq, c.q, p.T, p.H_kv, G, D, p.q_stride[0], p.q_stride[1], TQ, me)
      // the e4m3 pieces, one batch of tokens after the other, or the fp16 queries
      : kFew ? make_ragged_q_map(&mq, w + ps.q, static_cast<long long>(kPieces) * p.T, p.H_kv, G, D, static_cast<long long>(p.H) * D, D, TQ,
                                 MapElem::kE4M3)
             : make_ragged_q_map(&mq, w + ps.q, p.T, p.H_kv, G, D, static_cast<long long>(p.H) * D, D, TQ,
                                 MapElem::kF16);
  if (!q_ok || !make_pages_map(&mk, c.k_pages, planes, p.page, D, box, pe) ||
      !make_pages_map(&mv, c.v_pages, planes, p.page, D, box, pe))
    return FA_ERR_LAUNCH;
  PgArgs a{};
  a.cu = c.cu;
  a.seqlens = c.seqlens;
  a.table = c.page_table;
  a.k_scales = static_cast<const uint8_t*>(c.k_scales);
  a.v_scales = static_cast<const uint8_t*>(c.v_scales);
  a.q_scale = reinterpret_cast<const float*>(w + L.q_scale);
  a.out = c.o;
  a.lse = c.lse;
  a.splits = reinterpret_cast<PgSplit*>(w + ps.splits);
  a.part_lse = reinterpret_cast<float*>(w + ps.part_lse);
  a.part_o = reinterpret_cast<float*>(w + ps.part_o);
  a.n_lo = n_lo;
  a.n_hi = n_hi;
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.H_kv = p.H_kv;
  a.max_q = p.max_q;
  a.TQ = TQ;
  a.max_pages = p.max_pages;
  a.page = p.page;
  for (a.page_shift = 0; (1 << a.page_shift) < p.page;) ++a.page_shift;
  a.P = p.P;
  a.window = p.window;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.slots = 2ll * grid;
  a.status = di.status;
  if constexpr (Q8) {
    const long long threads = static_cast<long long>(p.T) * p.H * (D / 16);
    fa_paged_scale_q_kernel<D, E, kPieces><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, c.stream>>>(
        c.q, p.q_stride[0], p.q_stride[1], w + ps.q, reinterpret_cast<float*>(w + L.q_scale), p.T, p.H, di.status);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  }
  if (!launch_after(Q8, kern, dim3(grid), Cfg::kThreads, smem, c.stream, mq, mk, mv, a)) return FA_ERR_LAUNCH;
  // few rows: a block of four warps per row; otherwise eight blocks of eight warps, two rows each
  bool ok;
  if constexpr (kFew)
    ok = launch_after(true, fa_paged_merge_kernel<D, E, Cfg, 32, 4, 128>, dim3(grid + p.B, G * TQ), 128, 0, c.stream, a, grid);
  else
    ok = launch_after(true, fa_paged_merge_kernel<D, E, Cfg, 16, 1, 256>, dim3(grid + p.B, 8), 256, 0, c.stream, a, grid);
  return ok ? FA_OK : FA_ERR_LAUNCH;
}

// Kernel attributes of one instantiation, before anything is enqueued.
template <int D, Elem E, bool Q8, int RW>
bool paged_ready(DeviceInfo& di) {
  return once_per_device(di.paged_attr[E == Elem::kF16][Q8][D == 128][RW / 8 < 4 ? RW / 8 : 3], [&] {
    if constexpr (RW > 0)
      return cudaFuncSetAttribute(fa_paged_few_kernel<D, E, Q8, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(sizeof(PfSmem<D, E, Q8, RW>)) + 1024) == cudaSuccess;
    else
      return launch_regs_ok(fa_paged_kernel<D, E, Q8>, PgCfg<D, E, Q8>::kLaunch) &&
             cudaFuncSetAttribute(fa_paged_kernel<D, E, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(sizeof(PgSmem<D, E, Q8>)) + 1024) == cudaSuccess;
  });
}

template <Elem E, bool Q8, int D>
fa_status paged_call_d(DeviceInfo& di, const PagedCall& c) {
  const PagedKernels s = paged_kernels(c.p);
  constexpr int kMost = paged_most_rows(Q8, E == Elem::kF16);
  if (!(s.rows != 8 || paged_ready<D, E, Q8, 8>(di)) || !(s.rows != 16 || paged_ready<D, E, Q8, 16>(di)) ||
      !(s.rows != 32 || paged_ready<D, E, Q8, kMost>(di)) || !(!s.many || paged_ready<D, E, Q8, 0>(di)))
    return FA_ERR_LAUNCH;
  fa_status st = FA_OK;
  if (s.rows == 8) st = launch_paged<D, E, Q8, 8>(di, c, 0, s.few_q);
  if (s.rows == 16) st = launch_paged<D, E, Q8, 16>(di, c, 0, s.few_q);
  if (s.rows == 32) st = launch_paged<D, E, Q8, kMost>(di, c, 0, s.few_q);
  if (st == FA_OK && s.many) st = launch_paged<D, E, Q8, 0>(di, c, s.few_q, c.p.max_q);
  return st;
}

template <Elem E, bool Q8>
fa_status paged_call(DeviceInfo& di, const PagedCall& c) {
  return c.p.d == 128 ? paged_call_d<E, Q8, 128>(di, c) : paged_call_d<E, Q8, 64>(di, c);
}

}  // namespace fa
