// fa_cache.cu -- the C ABI of rotary positions and the paged key/value cache: argument
// validation and launches of fa_cache_kernels.cuh.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_cache_kernels.cuh"
#include "fa_host.h"

namespace {

using fa::aligned;
using fa::Elem;

bool is_16bit(int dtype) { return dtype == FA_DTYPE_BF16 || dtype == FA_DTYPE_F16; }

template <Elem E>
void launch_rope(const fa::RopeArgs& a, bool interleaved, bool vec, dim3 grid, size_t smem, cudaStream_t s) {
  if (vec)
    interleaved ? fa::fa_rope_kernel<E, true><<<grid, fa::kRopeThreads, smem, s>>>(a)
                : fa::fa_rope_kernel<E, false><<<grid, fa::kRopeThreads, smem, s>>>(a);
  else
    interleaved ? fa::fa_rope_any_kernel<E, true><<<grid, fa::kRopeThreads, smem, s>>>(a)
                : fa::fa_rope_any_kernel<E, false><<<grid, fa::kRopeThreads, smem, s>>>(a);
}

fa_status check_cache(const fa_cache_problem& p) {
  if (p.B < 1 || p.T < 1 || p.H_kv < 1 || p.P < 1 || p.max_pages < 1) return FA_ERR_INVALID_ARG;
  if (p.quant != 0 && p.quant != 1) return FA_ERR_INVALID_ARG;
  if (p.d != 64 && p.d != 128) return FA_ERR_UNSUPPORTED;
  if (p.page != 16 && p.page != 32 && p.page != 64 && p.page != 128 && p.page != 256) return FA_ERR_UNSUPPORTED;
  if (!is_16bit(p.dtype)) return FA_ERR_UNSUPPORTED;
  if (p.H_kv > (1 << 20)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The common fields, all but the tensors of the call.
fa::CacheArgs cache_args(const fa_cache_problem& p, const void* k_pages, const void* v_pages, const void* k_scales,
                         const void* v_scales, const int* table, const int* seqlens, const int* cu, int* status) {
  fa::CacheArgs a{};
  a.k_pages = const_cast<void*>(k_pages);
  a.v_pages = const_cast<void*>(v_pages);
  a.k_scales = static_cast<uint8_t*>(const_cast<void*>(k_scales));
  a.v_scales = static_cast<uint8_t*>(const_cast<void*>(v_scales));
  a.table = table;
  a.seqlens = seqlens;
  a.cu = cu;
  a.B = p.B;
  a.T = p.T;
  a.H_kv = p.H_kv;
  a.max_pages = p.max_pages;
  a.page = p.page;
  a.P = p.P;
  a.status = status;
  return a;
}

// A warp takes as many rows, up to 8, as fill the 2048 elements that its four passes have in flight,
// fewer while that leaves an SM less than 16 warps: what comes before its first load of the cache
// (sequence, length, page number) is a chain of four loads.  1 / 2 / 4 / 8 rows:
// 8K appended and 45K gathered rows of 640 elements, e4m3 pages: 37.7 / 29.0 / 28.1 / 32.2 us; 32K and
// 32K of 2048 elements: 91.2 / 93.0 / 97.6 / 101.3 us; 64 and 64: 9.2 / 12.2 / 18.4 / 30.1 us.
unsigned cache_blocks(fa::CacheArgs* a, int d, int sms) {
  a->lg = 0;
  while (a->lg < 3 && (2ll * a->H_kv * d) << a->lg < 2048 && a->T >> (a->lg + 1) >= 16 * sms) ++a->lg;
  const unsigned warps = (static_cast<unsigned>(a->T) + (1u << a->lg) - 1) >> a->lg;
  return (warps + 3) / 4;
}

template <Elem E, int D>
void launch_append(const fa::CacheArgs& a, bool quant, unsigned blocks, cudaStream_t s) {
  quant ? fa::fa_cache_append_kernel<E, D, true><<<blocks, 128, 0, s>>>(a)
        : fa::fa_cache_append_kernel<E, D, false><<<blocks, 128, 0, s>>>(a);
}

template <Elem E, int D>
void launch_gather(const fa::CacheArgs& a, bool quant, unsigned blocks, cudaStream_t s) {
  quant ? fa::fa_cache_gather_kernel<E, D, true><<<blocks, 128, 0, s>>>(a)
        : fa::fa_cache_gather_kernel<E, D, false><<<blocks, 128, 0, s>>>(a);
}

}  // namespace

extern "C" {

fa_status fa_rope(const fa_rope_problem* problem, const void* q, const void* k, void* q_out, void* k_out,
                  const void* positions, const double* inv_freq, void* stream) {
  if (!problem || !q || !q_out || !positions || !inv_freq) return FA_ERR_INVALID_ARG;
  const fa_rope_problem p = *problem;
  if (p.B < 1 || p.N < 1 || p.H < 1 || p.H_k < 0 || p.H > (1 << 20) || p.H_k > (1 << 20)) return FA_ERR_INVALID_ARG;
  if ((p.H_k > 0) != (k != nullptr) || (p.H_k > 0) != (k_out != nullptr)) return FA_ERR_INVALID_ARG;
  if (p.d < 2 || p.d > 1024 || p.rotary_dim < 2 || p.rotary_dim > p.d || p.rotary_dim % 2 != 0)
    return FA_ERR_INVALID_ARG;
  if ((p.interleaved != 0 && p.interleaved != 1) || (p.inverse != 0 && p.inverse != 1) ||
      (p.pos64 != 0 && p.pos64 != 1) || !isfinite(p.factor))
    return FA_ERR_INVALID_ARG;
  if (!is_16bit(p.dtype)) return FA_ERR_UNSUPPORTED;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(q_out, 2) || !aligned(k_out, 2) ||
      !aligned(positions, p.pos64 ? 8 : 4) || !aligned(inv_freq, 8))
    return FA_ERR_ALIGNMENT;
  fa::RopeArgs a{};
  bool vec = p.d % 16 == 0 && p.rotary_dim % 16 == 0 && aligned(q, 16) && aligned(k, 16) && aligned(q_out, 16) &&
             aligned(k_out, 16);
  for (int i = 0; i < 3; ++i) {
    a.xs[0][i] = p.q_stride[i];
    a.xs[1][i] = p.k_stride[i];
    a.ys[0][i] = p.q_out_stride[i];
    a.ys[1][i] = p.k_out_stride[i];
    vec = vec && p.q_stride[i] % 8 == 0 && p.q_out_stride[i] % 8 == 0;
    if (p.H_k > 0) vec = vec && p.k_stride[i] % 8 == 0 && p.k_out_stride[i] % 8 == 0;
  }
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k_out;
  a.pos = positions;
  a.ps[0] = p.pos_stride[0];
  a.ps[1] = p.pos_stride[1];
  a.inv_freq = inv_freq;
  a.pos64 = p.pos64;
  a.B = p.B;
  a.N = p.N;
  a.H = p.H;
  a.Hk = p.H_k;
  a.d = p.d;
  a.rd = p.rotary_dim;
  a.factor = p.factor;
  a.sign = p.inverse ? -1.0f : 1.0f;
  fa::DeviceInfo* di = nullptr;
  const fa_status st = fa::current_device(&di);
  if (st != FA_OK) return st;
  a.status = di->status;
  // A block takes all heads of as many tokens, up to 16, as give each of its threads four items
  // (what it has in flight at a time), so that one row of cosines serves every head; fewer while
  // that leaves less than four blocks per SM, and of a single token a part of its heads when there
  // are not two per SM.
  // (5 heads of 128 x 16384 tokens, 4 / 16 tokens a block: 22.9 / 16.6 us; 32 heads, 4 / 8: 96.8 / 112.7.)
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const int heads = p.H + p.H_k;
  const long long want = 2ll * di->sm_count;
  const long long items = static_cast<long long>(heads) * (p.d >= 16 ? p.d / 16 : 1);
  int tpb = 1;
  while (tpb < 16 && tpb * items < 4 * fa::kRopeThreads && 2 * tpb * p.rotary_dim <= 8192 && tokens >= 4 * tpb * want)
    tpb *= 2;
  a.tokens_per_block = tpb;
  const long long bx = (tokens + a.tokens_per_block - 1) / a.tokens_per_block;
  long long by = bx >= want ? 1 : (want + bx - 1) / bx;
  by = by > heads ? heads : by;
  if (bx > INT_MAX || heads / by > (1 << 16)) return FA_ERR_INVALID_ARG;
  a.heads_per_block = static_cast<int>((heads + by - 1) / by);
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>((heads + a.heads_per_block - 1) / a.heads_per_block));
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * p.rotary_dim * sizeof(float);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dtype == FA_DTYPE_F16)
    launch_rope<Elem::kF16>(a, p.interleaved, vec, grid, smem, s);
  else
    launch_rope<Elem::kBf16>(a, p.interleaved, vec, grid, smem, s);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_cache_append(const fa_cache_problem* problem, const void* k, const void* v, void* k_pages, void* v_pages,
                          void* k_scales, void* v_scales, const int* page_table, const int* seqlens, const int* cu,
                          void* stream) {
  if (!problem || !k || !v || !k_pages || !v_pages || !page_table || !seqlens || !cu) return FA_ERR_INVALID_ARG;
  const fa_cache_problem p = *problem;
  fa_status st = check_cache(p);
  if (st != FA_OK) return st;
  if (p.quant && (!k_scales || !v_scales)) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(page_table, 4) || !aligned(seqlens, 4) || !aligned(cu, 4))
    return FA_ERR_ALIGNMENT;
  for (int i = 0; i < 2; ++i)
    if (p.k_stride[i] % 8 != 0 || p.v_stride[i] % 8 != 0) return FA_ERR_ALIGNMENT;
  fa::DeviceInfo* di = nullptr;
  st = fa::current_device(&di);
  if (st != FA_OK) return st;
  fa::CacheArgs a = cache_args(p, k_pages, v_pages, k_scales, v_scales, page_table, seqlens, cu, di->status);
  a.k = k;
  a.v = v;
  for (int i = 0; i < 2; ++i) {
    a.ks[i] = p.k_stride[i];
    a.vs[i] = p.v_stride[i];
  }
  const unsigned blocks = cache_blocks(&a, p.d, di->sm_count);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dtype == FA_DTYPE_F16)
    p.d == 128 ? launch_append<Elem::kF16, 128>(a, p.quant, blocks, s)
               : launch_append<Elem::kF16, 64>(a, p.quant, blocks, s);
  else
    p.d == 128 ? launch_append<Elem::kBf16, 128>(a, p.quant, blocks, s)
               : launch_append<Elem::kBf16, 64>(a, p.quant, blocks, s);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

fa_status fa_cache_gather(const fa_cache_problem* problem, const void* k_pages, const void* v_pages,
                          const void* k_scales, const void* v_scales, const int* page_table, const int* seqlens,
                          const int* cu, const int* starts, void* k_out, void* v_out, void* stream) {
  if (!problem || !k_pages || !v_pages || !page_table || !seqlens || !cu || !k_out || !v_out)
    return FA_ERR_INVALID_ARG;
  const fa_cache_problem p = *problem;
  fa_status st = check_cache(p);
  if (st != FA_OK) return st;
  if (p.quant && (!k_scales || !v_scales)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(page_table, 4) || !aligned(seqlens, 4) || !aligned(cu, 4) || !aligned(starts, 4))
    return FA_ERR_ALIGNMENT;
  fa::DeviceInfo* di = nullptr;
  st = fa::current_device(&di);
  if (st != FA_OK) return st;
  fa::CacheArgs a = cache_args(p, k_pages, v_pages, k_scales, v_scales, page_table, seqlens, cu, di->status);
  a.k_out = k_out;
  a.v_out = v_out;
  a.starts = starts;
  const unsigned blocks = cache_blocks(&a, p.d, di->sm_count);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dtype == FA_DTYPE_F16)
    p.d == 128 ? launch_gather<Elem::kF16, 128>(a, p.quant, blocks, s)
               : launch_gather<Elem::kF16, 64>(a, p.quant, blocks, s);
  else
    p.d == 128 ? launch_gather<Elem::kBf16, 128>(a, p.quant, blocks, s)
               : launch_gather<Elem::kBf16, 64>(a, p.quant, blocks, s);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
