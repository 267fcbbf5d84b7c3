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

// With e4m3 pages, the e4m3 pieces of a query in the few-rows kernel: all bits of a bf16 (8), or of
// an fp16 (11), four to a piece.
constexpr int paged_q_pieces(bool f16) { return f16 ? 3 : 2; }
// Most rows of a key/value head in the few-rows kernel.  (20 rows, tiles of 128 against an instance for
// 32 rows: 16-bit pages, 16 sequences of 16-32K tokens, 262 / 270 us; e4m3 pages, 24 of 4096, 84 / 112 us,
// 24 of 16384, 210 / 231 us.)
constexpr int kPagedMostRows = 16;

// Which kernels a call takes.  A key/value head's rows, (H / H_kv) * n for n new tokens, choose
// per sequence: up to `rows` of them the few-rows kernel (n <= few_q), more the tiles of 128.
//   all sequences few (max_q says so): that kernel alone, at the smaller of 8 and 16 rows
//   all sequences max_q tokens long (T = B max_q): the tiles alone
//   a mixture: both, one behind the other, single tokens in the first at the smaller size
struct PagedKernels {
  int rows;   // 8, 16, or 0: the few-rows kernel is not used
  int few_q;  // its most tokens per sequence
  bool many;
};
inline PagedKernels paged_kernels(const fa_paged_problem& p) {
  const int G = p.H / p.H_kv;
  const long long rows = static_cast<long long>(G) * p.max_q;
  if (rows <= kPagedMostRows) return {rows <= 8 ? 8 : 16, p.max_q, false};
  if (G > kPagedMostRows || static_cast<long long>(p.B) * p.max_q == p.T) return {0, 0, true};
  const int r = G <= 8 ? 8 : 16;
  return {r, r / G, true};
}
// At most this many units (pairs of tiles of TQ tokens) per key/value head among sequences of up
// to n tokens: each sequence's last may be short.
inline long long paged_units(const fa_paged_problem& p, int n, int TQ) {
  const long long tokens = 2ll * TQ;
  const long long each = static_cast<long long>(p.B) * ((n + tokens - 1) / tokens);
  const long long all = p.T / tokens + p.B;
  return each < all ? each : all;
}

// Workspace regions of each kernel used: the units that CTAs share (16 bytes per CTA), the partial
// log-sums [rows, 2] and outputs [rows, d] (a CTA leaves at most two partial segments, of `rows` or
// 256 rows), and with e4m3 pages the queries' pieces (2 or 3 bytes per element) or fp16 form; then a
// factor per query row.
struct PagedLayout {
  struct Pass {
    size_t splits, part_lse, part_o, q;
  };
  Pass few, many;
  size_t q_scale, total;
};
inline PagedLayout paged_layout(const fa_paged_problem& p, int grid) {
  const auto round256 = [](size_t x) { return (x + 255) / 256 * 256; };
  const PagedKernels s = paged_kernels(p);
  const size_t q_rows = p.quant ? static_cast<size_t>(p.T) * p.H : 0;
  PagedLayout L{};
  size_t at = 0;
  const auto pass = [&](PagedLayout::Pass& x, size_t rows, int q_bytes) {
    rows *= 2 * static_cast<size_t>(grid);
    x.splits = at;
    x.part_lse = x.splits + round256(static_cast<size_t>(grid) * 16);
    x.part_o = x.part_lse + round256(rows * 2 * 4);
    x.q = x.part_o + round256(rows * static_cast<size_t>(p.d) * 4);
    at = x.q + round256(q_rows * p.d * q_bytes);
  };
  if (s.rows) pass(L.few, s.rows, paged_q_pieces(p.dtype == FA_DTYPE_F16));
  if (s.many) pass(L.many, 256, 2);
  L.q_scale = at;
  L.total = at + q_rows * 4;
  return L;
}

fa_status paged_bf16(DeviceInfo& di, const PagedCall& c);
fa_status paged_bf16_e4m3(DeviceInfo& di, const PagedCall& c);
fa_status paged_f16(DeviceInfo& di, const PagedCall& c);
fa_status paged_f16_e4m3(DeviceInfo& di, const PagedCall& c);

}  // namespace fa
