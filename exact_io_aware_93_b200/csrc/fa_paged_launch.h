// fa_paged_launch.h -- launches of the paged attention kernels.  Each (element type, page type)
// is instantiated in a source of its own, so that they compile side by side.
#pragma once

#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_host.h"

namespace fa {

struct PagedCall {
  fa_paged_problem p;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const void* k_scales;
  const void* v_scales;
  const int* page_table;
  const int* seqlens;
  const int* cu;
  void* o;
  float* lse;
  void* workspace;
  cudaStream_t stream;
};

// The kernel's variant (PgCfg's R) by the rows that one key/value head contributes at most: 4
// copies of up to 16 rows in a tile, 2 of up to 32, otherwise 0 for tiles of 128 rows; with e4m3
// pages 8 for 4 copies of up to 8 rows of four lanes each.
inline int paged_copies(const fa_paged_problem& p) {
  const long long rows = static_cast<long long>(p.H / p.H_kv) * p.max_q;
  if (p.quant && rows <= 8) return 8;
  return rows <= 16 ? 4 : (rows <= 32 ? 2 : 0);
}
inline int paged_tile_tokens(const fa_paged_problem& p) {
  return paged_copies(p) ? p.max_q : 128 / (p.H / p.H_kv);
}
// At most this many units (pairs of tiles) per key/value head: each sequence's last may be short.
inline long long paged_units(const fa_paged_problem& p) {
  const long long tokens = 2ll * paged_tile_tokens(p);
  const long long each = static_cast<long long>(p.B) * ((p.max_q + tokens - 1) / tokens);
  const long long all = p.T / tokens + p.B;
  return each < all ? each : all;
}

// Workspace regions: the plan (total, tiles per CTA, unit and key-tile prefixes), then the
// partial log-sums [rows, 2] and the partial outputs [rows, d]; a CTA leaves at most two
// partial segments of 256 rows (8, 16 or 32 where a tile holds copies).  With e4m3 pages also the
// query pieces (2 bytes per element) and a factor per query row.
struct PagedLayout {
  size_t meta, part_lse, part_o, pieces, q_scale, total;
  long long slots;
};
inline PagedLayout paged_layout(const fa_paged_problem& p, int grid) {
  const auto round256 = [](size_t x) { return (x + 255) / 256 * 256; };
  const int R = paged_copies(p);
  const size_t rows = 2 * static_cast<size_t>(grid) * (R == 0 ? 256 : (R == 8 ? 8 : 64 / R));
  PagedLayout L;
  L.slots = 2ll * grid;
  L.meta = 0;
  L.part_lse = round256((2 + 2 * (static_cast<size_t>(p.B) + 1)) * 4);
  L.part_o = L.part_lse + round256(rows * 2 * 4);
  L.pieces = L.part_o + round256(rows * static_cast<size_t>(p.d) * 4);
  const size_t q_rows = p.quant ? static_cast<size_t>(p.T) * p.H : 0;
  L.q_scale = L.pieces + round256(q_rows * p.d * 2);
  L.total = L.q_scale + q_rows * 4;
  return L;
}

fa_status paged_bf16(DeviceInfo& di, const PagedCall& c);
fa_status paged_bf16_e4m3(DeviceInfo& di, const PagedCall& c);
fa_status paged_f16(DeviceInfo& di, const PagedCall& c);
fa_status paged_f16_e4m3(DeviceInfo& di, const PagedCall& c);

}  // namespace fa
