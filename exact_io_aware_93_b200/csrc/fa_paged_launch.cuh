// fa_paged_launch.cuh -- the launch of one (element type, page type) of paged attention.
#pragma once

#include "fa_paged_kernel.cuh"
#include "fa_paged_launch.h"
#include "tma_host.h"

#include <type_traits>

namespace fa {

template <int D, Elem E, bool Q8, int R>
fa_status launch_paged(DeviceInfo& di, const PagedCall& c) {
  using Cfg = PgCfg<D, E, Q8, R>;
  const fa_paged_problem& p = c.p;
  auto kern = fa_paged_kernel<D, E, Q8, R>;
  const int smem = static_cast<int>(sizeof(PgSmem<D, E, Q8, R>)) + 1024;
  static_assert(sizeof(PgSmem<D, E, Q8, R>) + 1024 <= 232448, "shared memory of one CTA");
  if (!once_per_device(di.paged_attr[E == Elem::kF16][Q8][D == 128][R == 8 ? 3 : R / 2], [&] {
        return (!Cfg::kGeneral || launch_regs_ok(kern, Cfg::kLaunch)) &&
               cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
      }))
    return FA_ERR_LAUNCH;
  const int G = p.H / p.H_kv;
  const int TQ = paged_tile_tokens(p);
  const MapElem me = E == Elem::kF16 ? MapElem::kF16 : MapElem::kBf16;
  const MapElem pe = Q8 ? MapElem::kE4M3 : me;
  const long long planes = static_cast<long long>(p.P) * p.H_kv;
  const int box = p.page < 128 ? p.page : 128;
  const int grid = di.sm_count;
  const PagedLayout L = paged_layout(p, grid);
  uint8_t* w = static_cast<uint8_t*>(c.workspace);
  CUtensorMap mq, mk, mv;
  // e4m3 pages: the query pieces, one batch of tokens after the other
  if (!(Q8 ? make_ragged_q_map(&mq, w + L.pieces, 2ll * p.T, p.H_kv, G, D,
                               static_cast<long long>(p.H) * D, D, TQ, MapElem::kE4M3)
           : make_ragged_q_map(&mq, c.q, p.T, p.H_kv, G, D, p.q_stride[0], p.q_stride[1], TQ, me)) ||
      !make_pages_map(&mk, c.k_pages, planes, p.page, D, box, pe) ||
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
  a.meta = reinterpret_cast<int*>(w + L.meta);
  a.part_lse = reinterpret_cast<float*>(w + L.part_lse);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
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
  a.slots = L.slots;
  a.status = di.status;
  if constexpr (Q8) {
    const long long threads = static_cast<long long>(p.T) * p.H * (D / 16);
    fa_paged_split_kernel<D, E><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, c.stream>>>(
        c.q, p.q_stride[0], p.q_stride[1], w + L.pieces, reinterpret_cast<float*>(w + L.q_scale), p.T, p.H, di.status);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  }
  kern<<<grid, Cfg::kThreads, smem, c.stream>>>(mq, mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  // few rows: a block per row, its four warps sharing the partial results; otherwise a warp per
  // row and blocks of up to 32 rows
  const unsigned units = static_cast<unsigned>(paged_units(p));
  const int rows = G * (p.max_q < 2 * TQ ? p.max_q : 2 * TQ);
  if constexpr (Cfg::kGeneral)
    fa_paged_merge_kernel<D, E, Q8, R, 1><<<dim3(units, p.H_kv, (rows + 31) / 32), 128, 0, c.stream>>>(a);
  else
    fa_paged_merge_kernel<D, E, Q8, R, 4><<<dim3(units, p.H_kv, rows), 128, 0, c.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <Elem E, bool Q8>
fa_status paged_call(DeviceInfo& di, const PagedCall& c) {
  const auto go = [&](auto d) -> fa_status {
    constexpr int D = decltype(d)::value;
    switch (paged_copies(c.p)) {
      case 8:
        if constexpr (Q8) return launch_paged<D, E, Q8, 8>(di, c);
        return FA_ERR_LAUNCH;
      case 4: return launch_paged<D, E, Q8, 4>(di, c);
      case 2: return launch_paged<D, E, Q8, 2>(di, c);
      default: return launch_paged<D, E, Q8, 0>(di, c);
    }
  };
  return c.p.d == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

}  // namespace fa
