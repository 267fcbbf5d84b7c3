// fa_paged_launch.cuh -- the launches of one (element type, page type) of paged attention.
#pragma once

#include <type_traits>

#include "fa_paged_few_kernel.cuh"
#include "fa_paged_kernel.cuh"
#include "fa_paged_launch.h"
#include "tma_host.h"

namespace fa {

// Launch whose blocks may start while the kernel before them in the stream ends; they wait for it
// themselves (griddepcontrol.wait): about 1 us less between two kernels.
template <typename... P, typename... Args>
bool launch_after(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

// A kernel of a call: the sequences with n_lo < n <= n_hi new tokens, tiles of TQ tokens.  RW: rows of the
// few-rows kernel, 0 for tiles of 128.
template <int D, Elem E, bool Q8, int RW>
struct PagedPass {
  static constexpr bool kFew = RW > 0;
  using Cfg = std::conditional_t<kFew, PfCfg<D, E, Q8, kFew ? RW : 8>, PgCfg<D, E, Q8>>;
  using Smem = std::conditional_t<kFew, PfSmem<D, E, Q8, kFew ? RW : 8>, PgSmem<D, E, Q8>>;
  static constexpr int kSmem = static_cast<int>(sizeof(Smem)) + 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  CUtensorMap mq, mk, mv;
  PgArgs a{};

  bool prepare(DeviceInfo& di, const PagedCall& c, const PagedLayout& L, int n_lo, int n_hi) {
    const fa_paged_problem& p = c.p;
    const int G = p.H / p.H_kv;
    const int TQ = kFew ? n_hi : 128 / G;
    const MapElem me = E == Elem::kF16 ? MapElem::kF16 : MapElem::kBf16;
    const MapElem pe = Q8 ? MapElem::kE4M3 : me;
    const long long planes = static_cast<long long>(p.P) * p.H_kv, hd = static_cast<long long>(p.H) * D;
    const int box = p.page < 128 ? p.page : 128;
    const PagedLayout::Pass& ps = kFew ? L.few : L.many;
    uint8_t* w = static_cast<uint8_t*>(c.workspace);
    // e4m3 pages: the queries' pieces, one batch of tokens after the other, or their fp16 form
    const bool q_ok = !Q8 ? make_ragged_q_map(&mq, c.q, p.T, p.H_kv, G, D, p.q_stride[0], p.q_stride[1], TQ, me)
                      : kFew ? make_ragged_q_map(&mq, w + ps.q, static_cast<long long>(paged_q_pieces(E == Elem::kF16)) * p.T,
                                                 p.H_kv, G, D, hd, D, TQ, MapElem::kE4M3)
                             : make_ragged_q_map(&mq, w + ps.q, p.T, p.H_kv, G, D, hd, D, TQ, MapElem::kF16);
    if (!q_ok || !make_pages_map(&mk, c.k_pages, planes, p.page, D, box, pe) ||
        !make_pages_map(&mv, c.v_pages, planes, p.page, D, box, pe))
      return false;
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
    a.slots = 2ll * di.sm_count;
    a.behind = !kFew && n_lo > 0;
    a.status = di.status;
    return true;
  }
  bool launch(DeviceInfo& di, const PagedCall& c) const {
    auto kern = [] {
      if constexpr (kFew) return fa_paged_few_kernel<D, E, Q8, RW>;
      else return fa_paged_kernel<D, E, Q8>;
    }();
    return launch_after(kern, dim3(di.sm_count), Cfg::kThreads, kSmem, c.stream, mq, mk, mv, a);
  }
};

// The kernels of a call, in this order: the scaling of the queries (e4m3 pages), few rows, tiles of 128,
// and one join of both's partial results.  Each may start while the one before it ends.  (The tiles'
// kernel fills the SMs that the few-rows kernel leaves; one after the other, each with its own scaling
// and join: 259 us for 1001 new tokens beside 16 single ones over e4m3 pages.)
template <int D, Elem E, bool Q8, int RW, bool kMany>
fa_status launch_paged(DeviceInfo& di, const PagedCall& c, int few_q) {
  constexpr bool kFew = RW > 0;
  using Few = PagedPass<D, E, Q8, kFew ? RW : 8>;
  using Many = PagedPass<D, E, Q8, 0>;
  const fa_paged_problem& p = c.p;
  const PagedLayout L = paged_layout(p, di.sm_count);
  uint8_t* w = static_cast<uint8_t*>(c.workspace);
  Few few;
  Many many;
  // what can fail comes before the first launch
  if constexpr (kFew)
    if (!few.prepare(di, c, L, 0, few_q)) return FA_ERR_LAUNCH;
  if constexpr (kMany)
    if (!many.prepare(di, c, L, kFew ? few_q : 0, p.max_q)) return FA_ERR_LAUNCH;
  if constexpr (Q8) {
    const long long threads = static_cast<long long>(p.T) * p.H * (D / 16);
    if (!launch_after(fa_paged_scale_q_kernel<D, E, kFew ? paged_q_pieces(E == Elem::kF16) : 0, kMany>,
                      dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, c.stream, c.q, p.q_stride[0],
                      p.q_stride[1], w + L.few.q, w + L.many.q, reinterpret_cast<float*>(w + L.q_scale), p.T, p.H, di.status))
      return FA_ERR_LAUNCH;
  }
  if constexpr (kFew)
    if (!few.launch(di, c)) return FA_ERR_LAUNCH;
  if constexpr (kMany)
    if (!many.launch(di, c)) return FA_ERR_LAUNCH;
  // few rows: a block of four (beside tiles: eight) warps per row; tiles: eight blocks of eight warps, two
  // rows each
  constexpr int kThreads = kMany ? 256 : 128, kManyY = kMany ? 8 : 0;
  using FewCfg = std::conditional_t<kFew, typename Few::Cfg, void>;
  using ManyCfg = std::conditional_t<kMany, typename Many::Cfg, void>;
  const int rows = kFew ? p.H / p.H_kv * few_q : 0;
  return launch_after(fa_paged_merge_kernel<D, E, FewCfg, ManyCfg, kThreads>, dim3(di.sm_count + p.B, kManyY + rows),
                      kThreads, 0, c.stream, few.a, many.a, di.sm_count, kManyY)
             ? FA_OK
             : FA_ERR_LAUNCH;
}

// Kernel attributes of one instantiation, before anything is enqueued.
template <int D, Elem E, bool Q8, int RW>
bool paged_ready(DeviceInfo& di) {
  return once_per_device(di.paged_attr[E == Elem::kF16][Q8][D == 128][RW / 8], [&] {
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
  if (!(s.rows != 8 || paged_ready<D, E, Q8, 8>(di)) || !(s.rows != 16 || paged_ready<D, E, Q8, 16>(di)) ||
      !(!s.many || paged_ready<D, E, Q8, 0>(di)))
    return FA_ERR_LAUNCH;
  if (s.rows == 0) return launch_paged<D, E, Q8, 0, true>(di, c, 0);
  if (s.rows == 8)
    return s.many ? launch_paged<D, E, Q8, 8, true>(di, c, s.few_q) : launch_paged<D, E, Q8, 8, false>(di, c, s.few_q);
  return s.many ? launch_paged<D, E, Q8, 16, true>(di, c, s.few_q) : launch_paged<D, E, Q8, 16, false>(di, c, s.few_q);
}

template <Elem E, bool Q8>
fa_status paged_call(DeviceInfo& di, const PagedCall& c) {
  return c.p.d == 128 ? paged_call_d<E, Q8, 128>(di, c) : paged_call_d<E, Q8, 64>(di, c);
}

}  // namespace fa
