// fa_paged.cu -- the C ABI of attention over a paged cache: argument validation and dispatch.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "fa_paged_launch.h"

namespace {

using fa::aligned;

fa_status check_paged(const fa_paged_problem& p) {
  if (p.B < 1 || p.T < 1 || p.H < 1 || p.H_kv < 1 || p.max_q < 1 || p.P < 1 || p.max_pages < 1)
    return FA_ERR_INVALID_ARG;
  if (p.H_kv > p.H || p.H % p.H_kv != 0) return FA_ERR_INVALID_ARG;
  if (!(p.scale > 0.0f) || !isfinite(p.scale)) return FA_ERR_INVALID_ARG;
  if (p.causal != 0 && p.causal != 1) return FA_ERR_INVALID_ARG;
  if (p.quant != 0 && p.quant != 1) return FA_ERR_INVALID_ARG;
  if (p.window < -1 || (p.window >= 0 && p.causal != 1)) return FA_ERR_INVALID_ARG;
  if (p.d != 64 && p.d != 128) return FA_ERR_UNSUPPORTED;
  if (p.page != 16 && p.page != 32 && p.page != 64 && p.page != 128 && p.page != 256) return FA_ERR_UNSUPPORTED;
  if (p.dtype != FA_DTYPE_BF16 && p.dtype != FA_DTYPE_F16) return FA_ERR_UNSUPPORTED;
  if (p.H / p.H_kv > 128) return FA_ERR_UNSUPPORTED;
  // key-tile counts, planes, positions and grid extents stay in range
  const long long cap = static_cast<long long>(p.max_pages) * p.page;
  const long long planes = static_cast<long long>(p.P) * p.H_kv;
  if (cap > INT_MAX - 1024 || planes >= INT_MAX || p.H_kv > 65535 || p.T > INT_MAX / 4) return FA_ERR_INVALID_ARG;
  // the work list is counted in 32 bits, up to 3 units of cost per key tile and 8 per unit
  const int tq = 128 / (p.H / p.H_kv);
  const long double cost = fa::paged_units(p, p.max_q, tq) * (3.0L * ((cap + 127) / 128) + 8.0L) * p.H_kv;
  if (cost > static_cast<long double>(INT_MAX / 2)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// A chunk longer than the batch has no more rows than the batch.
fa_paged_problem clamped(fa_paged_problem p) {
  if (p.T > 0 && p.max_q > p.T) p.max_q = p.T;
  return p;
}

}  // namespace

extern "C" {

size_t fa_paged_workspace_size(const fa_paged_problem* problem) {
  if (!problem) return 0;
  const fa_paged_problem p = clamped(*problem);
  if (check_paged(p) != FA_OK) return 0;
  fa::DeviceInfo* di = nullptr;
  if (fa::current_device(&di) != FA_OK) return 0;
  return fa::paged_layout(p, di->sm_count).total;
}

fa_status fa_paged(const fa_paged_problem* problem, const void* q, const void* k_pages, const void* v_pages,
                   const void* k_scales, const void* v_scales, const int* page_table, const int* seqlens,
                   const int* cu_q, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!problem || !q || !k_pages || !v_pages || !page_table || !seqlens || !cu_q || !o || !lse)
    return FA_ERR_INVALID_ARG;
  fa::PagedCall c{clamped(*problem), q,    k_pages, v_pages, k_scales,  v_scales,
                  page_table,        seqlens, cu_q, o,       lse,       workspace,
                  static_cast<cudaStream_t>(stream)};
  const fa_paged_problem& p = c.p;
  fa_status st = check_paged(p);
  if (st != FA_OK) return st;
  if (p.quant && (!k_scales || !v_scales)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(page_table, 4) || !aligned(seqlens, 4) || !aligned(cu_q, 4))
    return FA_ERR_ALIGNMENT;
  if (p.quant && (!aligned(k_scales, 16) || !aligned(v_scales, 16))) return FA_ERR_ALIGNMENT;
  // the tensor map of q: strides of whole 16-byte units below 2^40 bytes
  for (int i = 0; i < 2; ++i) {
    if (p.q_stride[i] < 0 || p.q_stride[i] > (1ll << 31)) return FA_ERR_INVALID_ARG;
    if (p.q_stride[i] % 8 != 0) return FA_ERR_ALIGNMENT;
  }
  fa::DeviceInfo* di = nullptr;
  st = fa::current_device(&di);
  if (st != FA_OK) return st;
  if (workspace == nullptr || workspace_bytes < fa::paged_layout(p, di->sm_count).total) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  if (p.dtype == FA_DTYPE_F16) return p.quant ? fa::paged_f16_e4m3(*di, c) : fa::paged_f16(*di, c);
  return p.quant ? fa::paged_bf16_e4m3(*di, c) : fa::paged_bf16(*di, c);
}

}  // extern "C"
