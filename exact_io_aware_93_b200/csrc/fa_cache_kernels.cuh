// fa_cache_kernels.cuh -- what a step does to queries, keys and values around attention:
// rotary positions, the write of new keys and values into a paged cache, and the read of a
// range of positions back out of it.  All three move each byte once and compute little, so
// device memory bounds them from a few thousand tokens on and latency below.
//
// Paged cache.  A pool of P pages holds [P, H_kv, page, d]; position p of sequence b lies in
// page table[b][p / page] at slot p % page.  Heads come before slots, so one head's page is
// one run of page * d elements: the attention kernel fetches it as one box.  An e4m3 pool
// holds codes, and a scale 2^e per (page, head, slot) as its exponent byte e + 127.
#pragma once

#include "sm100_ptx.cuh"

namespace fa {

// A length, offset or page number read on the device was out of range: recorded once in the
// status word (FA_ERR_PLAN) with its site; the caller skips the access.
__device__ __noinline__ inline void plan_fail(int* status, int site) {
  atomicCAS(status, 0, 9 /* FA_ERR_PLAN */);
  atomicCAS(status + 1, 0, site);
}

// ---------------------------------------------------------------- rotary positions
// The pair (a, b) with frequency f at position p becomes (a c - b s, b c + a s) with
// c = factor * cos(p f), s = factor * sin(p f); the gradient is the transpose, s negated.
// Pair j of a head is (x[j], x[j + R/2]) or, interleaved, (x[2j], x[2j + 1]); columns from R
// on are copied.  The angle is formed in 64 bits and reduced to a fraction of a turn before
// it is rounded to 32: at position 131072 a 32-bit product would be off by up to 2^-8 rad.
struct RopeArgs {
  const void* x[2];     // q and k
  void* y[2];
  int64_t xs[2][3];     // element strides: batch, token, head
  int64_t ys[2][3];
  const void* pos;      // int32 or int64 positions
  int64_t ps[2];        // position strides: batch, token
  const double* inv_freq;
  int pos64;
  int B, N, H, Hk;      // heads of q; heads of k (0: no k)
  int d, rd;
  float factor, sign;   // sign -1: the inverse rotation
  int tokens_per_block, heads_per_block;
  int* status;
};

constexpr int kRopeThreads = 256;
constexpr double kInv2Pi = 0.15915494309189535;     // 1 / (2 pi) to 53 bits, and the rest
constexpr double kInv2PiLo = -9.839338337591243e-18;

// Batch row and place in it of token `add` after (b, n).
struct RopeToken {
  int b;
  unsigned n;
  __device__ __forceinline__ RopeToken(const RopeArgs& a, int b0, int n0, int add)
      : b(b0), n(static_cast<unsigned>(n0) + add) {
    if (n >= static_cast<unsigned>(a.N)) {
      b += static_cast<int>(n / a.N);
      n %= a.N;
    }
  }
};

// cos and sin of every pair of the block's tokens, (b, n) the first: tab[0][token][j], tab[1][token][j].
__device__ __forceinline__ void rope_table(const RopeArgs& a, int b, int n, int nt, float* tab) {
  const int half = a.rd >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tk = i / half;
    const int j = i - tk * half;
    const RopeToken t(a, b, n, tk);
    const int64_t at = t.b * a.ps[0] + t.n * a.ps[1];
    const double p = a.pos64 ? static_cast<double>(static_cast<const long long*>(a.pos)[at])
                             : static_cast<double>(static_cast<const int*>(a.pos)[at]);
    // p * f / (2 pi) modulo 1 with the roundings of both products carried along: at p = 2^31
    // a plain fp64 product is already 2^-22 rad off
    const double f = a.inv_freq[j];
    const double w = f * kInv2Pi;
    const double w_lo = fma(f, kInv2Pi, -w) + f * kInv2PiLo;
    const double hi = p * w;
    const double turns = (hi - rint(hi)) + (fma(p, w, -hi) + p * w_lo);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns), &s, &c);
    tab[i] = c * a.factor;
    tab[nt * half + i] = s * a.factor * a.sign;
  }
}

// The rotated pair; the contraction is spelled out so that every path gives the same bits.
__device__ __forceinline__ float2 rope_pair(float x0, float x1, float c, float s) {
  return make_float2(fmaf(x0, c, -__fmul_rn(x1, s)), fmaf(x1, c, __fmul_rn(x0, s)));
}

// The rows (token, head) of a block in order, `step` apart: a thread divides once and then adds,
// since two divisions per row, 64 bits wide for the batch, took as many instructions as the rotation.
struct RopeRow {
  int b, n;   // the block's first token: batch row and place in it
  int tk, h;  // this row's token, from that one on, and head among the block's
  int dt, dh; // what a step adds
  __device__ __forceinline__ RopeRow(const RopeArgs& a, int64_t t0, int nh, int row, int step)
      : b(a.B == 1 ? 0 : static_cast<int>(t0 / a.N)), n(static_cast<int>(t0 - static_cast<int64_t>(b) * a.N)), tk(row / nh),
        h(row - tk * nh), dt(step / nh), dh(step - dt * nh) {}
  __device__ __forceinline__ void next(int nh) {
    tk += dt;
    h += dh;
    if (h >= nh) {
      h -= nh;
      ++tk;
    }
  }
  // Element offset of head `head` of all (q's, then k's); w says which.
  __device__ __forceinline__ int64_t offset(const RopeArgs& a, const int64_t (&st)[2][3], int head, int w) const {
    const RopeToken t(a, b, n, tk);
    return t.b * st[w][0] + t.n * st[w][1] + (head - (w ? a.H : 0)) * st[w][2];
  }
};

// 16384 tokens of 32 heads of 128 rotated, 268 MB moved: 45.3 us (5.9 TB/s); plain instead of evict-first
// loads and stores: 47.
//
// Rows of whole 16-element items (R and d multiples of 16, 16-byte aligned rows): a thread
// owns one item of a head for several rows, 32 bytes in and out per row, and issues four
// rows' loads before it needs the first.  The block's cos/sin are computed once per token and
// serve all its heads.
template <Elem E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4) fa_rope_kernel(const RopeArgs a) {
  using T = typename ElemOps<E>::T;
  extern __shared__ __align__(16) float tab[];
  constexpr int U = 4;
  const int half = a.rd >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t left = static_cast<int64_t>(a.B) * a.N - t0;
  const int nt = left < a.tokens_per_block ? static_cast<int>(left) : a.tokens_per_block;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.heads_per_block, a.H + a.Hk - h0);
  const int items = a.d >> 4;
  const int rows = nt * nh;
  const int item = threadIdx.x % items;
  const int step = kRopeThreads / items;  // rows per pass
  const int r0 = threadIdx.x / items;
  const bool turned = item * 16 < a.rd;
  // the item's two 8-element vectors
  const int c0 = (turned && !INTERLEAVED) ? item * 8 : item * 16;
  const int c1 = (turned && !INTERLEAVED) ? half + item * 8 : item * 16 + 8;
  uint4 v0[U], v1[U];
  RopeRow in(a, t0, nh, r0, step), out = in;
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 < step && base + u * step < rows) {
        const int w = h0 + in.h >= a.H;
        const T* x = static_cast<const T*>(a.x[w]) + in.offset(a, a.xs, h0 + in.h, w);
        if (FA_IN_BOUNDS(t0 + in.tk < static_cast<int64_t>(a.B) * a.N && c1 + 8 <= a.d, a.status, 401)) {
          v0[u] = __ldcs(reinterpret_cast<const uint4*>(x + c0));  // coherent: y may be x
          v1[u] = __ldcs(reinterpret_cast<const uint4*>(x + c1));
        }
        in.next(nh);
      }
    }
  };
  load(r0);  // in flight while the table is computed
  rope_table(a, in.b, in.n, nt, tab);
  __syncthreads();
  for (int base = r0; r0 < step && base < rows; base += U * step) {
    if (base != r0) load(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * step >= rows) break;
      const int tk = out.tk;
      uint32_t* p0 = &v0[u].x;
      uint32_t* p1 = &v1[u].x;
      if (turned) {
        float c[8], s[8];
        const float4* tc = reinterpret_cast<const float4*>(tab + tk * half + item * 8);
        const float4* ts = reinterpret_cast<const float4*>(tab + nt * half + tk * half + item * 8);
        *reinterpret_cast<float4*>(c) = tc[0];
        *reinterpret_cast<float4*>(c + 4) = tc[1];
        *reinterpret_cast<float4*>(s) = ts[0];
        *reinterpret_cast<float4*>(s + 4) = ts[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e0 = ElemOps<E>::unpack(p0[i]);
          const float2 e1 = ElemOps<E>::unpack(p1[i]);
          if (INTERLEAVED) {  // a word is a pair
            const float2 y0 = rope_pair(e0.x, e0.y, c[i], s[i]);
            const float2 y1 = rope_pair(e1.x, e1.y, c[i + 4], s[i + 4]);
            p0[i] = ElemOps<E>::pack(y0.x, y0.y);
            p1[i] = ElemOps<E>::pack(y1.x, y1.y);
          } else {            // a word of each vector holds two pairs' halves
            const float2 y0 = rope_pair(e0.x, e1.x, c[2 * i], s[2 * i]);
            const float2 y1 = rope_pair(e0.y, e1.y, c[2 * i + 1], s[2 * i + 1]);
            p0[i] = ElemOps<E>::pack(y0.x, y1.x);
            p1[i] = ElemOps<E>::pack(y0.y, y1.y);
          }
        }
      }
      const int w = h0 + out.h >= a.H;
      T* y = static_cast<T*>(a.y[w]) + out.offset(a, a.ys, h0 + out.h, w);
      if (FA_IN_BOUNDS(t0 + tk < static_cast<int64_t>(a.B) * a.N && c1 + 8 <= a.d, a.status, 402)) {
        __stcs(reinterpret_cast<uint4*>(y + c0), v0[u]);
        __stcs(reinterpret_cast<uint4*>(y + c1), v1[u]);
      }
      out.next(nh);
    }
  }
}

// Any even R <= d and any alignment: a thread per pair (or copied column), 2-byte accesses.  16384 tokens
// of 32 heads of 80 columns, 20 turned: 238 us, 0.71 TB/s (interleaved 222); with 32 turned, which the
// kernel above takes, 38 us.  Bound by its two divisions and two 2-byte accesses per pair.
template <Elem E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_any_kernel(const RopeArgs a) {
  using T = typename ElemOps<E>::T;
  extern __shared__ __align__(16) float tab[];
  const int half = a.rd >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_block;
  const int64_t left = static_cast<int64_t>(a.B) * a.N - t0;
  const int nt = left < a.tokens_per_block ? static_cast<int>(left) : a.tokens_per_block;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.heads_per_block, a.H + a.Hk - h0);
  RopeRow at(a, t0, nh, 0, 1);
  rope_table(a, at.b, at.n, nt, tab);
  __syncthreads();
  const int per = a.d - half;  // pairs, then copied columns
  const int rows = nt * nh;
  for (int i = threadIdx.x; i < rows * per; i += kRopeThreads) {
    const int row = i / per;
    const int e = i - row * per;
    const int tk = row / nh;
    const int head = h0 + row - tk * nh, w = head >= a.H;
    at.tk = tk;
    const T* x = static_cast<const T*>(a.x[w]) + at.offset(a, a.xs, head, w);
    T* y = static_cast<T*>(a.y[w]) + at.offset(a, a.ys, head, w);
    if (!FA_IN_BOUNDS(t0 + tk < static_cast<int64_t>(a.B) * a.N && half + e < a.d, a.status, 403)) continue;
    if (e >= half) {
      y[half + e] = x[half + e];
    } else {
      const int i0 = INTERLEAVED ? 2 * e : e;
      const int i1 = INTERLEAVED ? 2 * e + 1 : half + e;
      const float c = tab[tk * half + e], s = tab[nt * half + tk * half + e];
      const float2 r = rope_pair(static_cast<float>(x[i0]), static_cast<float>(x[i1]), c, s);
      y[i0] = ElemOps<E>::one(r.x);
      y[i1] = ElemOps<E>::one(r.y);
    }
  }
}

// ---------------------------------------------------------------- paged cache
struct CacheArgs {
  const void* k;          // append: new keys / values [T, H_kv, d] (strided); gather: null
  const void* v;
  int64_t ks[2], vs[2];   // element strides: token, head
  void* k_pages;          // [P, H_kv, page, d]
  void* v_pages;
  uint8_t* k_scales;      // [P, H_kv, page] exponent bytes, or null
  uint8_t* v_scales;
  void* k_out;            // gather: [T, H_kv, d]
  void* v_out;
  const int* table;       // [B, max_pages]
  const int* seqlens;     // [B]
  const int* cu;          // [B + 1] offsets of the batch's rows
  const int* starts;      // gather: first position of each sequence, or null (0)
  int B, T, H_kv, max_pages, page, P;
  int lg;                 // log2 of a warp's rows
  int* status;
};

// The sequence of row t: how many of cu[1..B] are <= t, found by the whole warp 32 offsets at
// a time (one round of loads up to 32 sequences, two up to 1024).
__device__ __forceinline__ int find_seq(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = (lane + 1) * step;  // 1-based index of this lane's last candidate
    const unsigned hit = __ballot_sync(0xffffffffu, at <= n && __ldg(cu + lo + at) <= t);
    const int full = __popc(hit);
    lo += full * step;
    n = min(step - 1, n - full * step);
  }
  return lo;
}

// The sequence of row t + lane, `first` being row t's.
__device__ __forceinline__ int find_seq_from(const int* cu, int B, int first, int t) {
  int lo = first, hi = B;  // cu[lo] <= t < cu[hi + 1], if hi < B
  while (lo < hi && __ldg(cu + lo + 1) <= t) {
    const int mid = lo + 1 + (hi - lo - 1) / 2;
    if (__ldg(cu + mid) <= t) {
      lo = mid;
    } else {
      hi = mid - 1;
      ++lo;
    }
  }
  return lo;
}

// Where position `pos` of sequence b lies: the row index (page * H_kv) * slots + slot of head
// 0, or -1 (recorded) for a position or page number out of range.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& a, int b, int64_t pos, int site) {
  int64_t at = -1;
  if (pos >= 0 && pos < static_cast<int64_t>(a.max_pages) * a.page) {
    const int pg = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + pos / a.page);
    if (pg >= 0 && pg < a.P) at = (static_cast<int64_t>(pg) * a.H_kv) * a.page + pos % a.page;
  }
  if (at < 0) plan_fail(a.status, site);
  return at;
}

__device__ __forceinline__ float e8m0_to_float(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : (b == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23));
}

// Two e4m3 codes (low 16 bits) to floats.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t u) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo;\n\t.reg .b16 hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(u));
  return unpack_f16x2(h);
}

// The exponent e of a row's scale: the smallest power of two with amax <= 448 * 2^e, clamped
// to what the 16-bit type needs (2^-15 makes e4m3's smallest step fp16's own, 448 * 2^8 holds
// every fp16; bf16 likewise over its range).  A power of two costs e4m3 nothing, since its
// steps are relative, and it makes code * 2^e exact in bf16 and fp16: a reader of the cache
// rounds nothing.
template <Elem E>
__device__ __forceinline__ int e4m3_exponent(float amax) {
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);  // 448 = 1.75 * 2^8
  return E == Elem::kF16 ? min(max(e, -15), 8) : min(max(e, -126), 119);
}

// 32768 tokens of 8 heads of 128, 16-bit pages, 268 MB moved by each: append and gather 45 us (6.0 TB/s).
// (Evict-first loads and stores, or loads alone: 1 to 2 us slower.)
//
// Appends rows of the new keys and values at their positions: the last position of a sequence is
// seqlens[b] - 1.  A warp takes 2^lg rows (a lane finds where one lies) and its lanes 16 elements of
// a head each, the rows of one head side by side: their slots, and the scales, are neighbours in a
// page.  The first four passes' elements are loaded before the positions are known.
template <Elem E, int D, bool Q8>
__global__ void __launch_bounds__(128) fa_cache_append_kernel(const CacheArgs a) {
  using T = typename ElemOps<E>::T;
  constexpr int L = D / 16;    // lanes per row
  constexpr int RW = 32 / L;   // rows per pass
  constexpr int U = 4;
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)) << a.lg;
  if (t0 >= a.T) return;
  const int nt = static_cast<int>(min(static_cast<int64_t>(1) << a.lg, a.T - t0));
  const int item = lane % L;
  const int rows = (2 * a.H_kv) << a.lg;  // the keys' heads, then the values', each of all tokens
  uint4 x0[U], x1[U];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * RW, tk = row & ((1 << a.lg) - 1), r = row >> a.lg;
      if (row < rows && tk < nt) {
        const bool isv = r >= a.H_kv;
        const T* src = static_cast<const T*>(isv ? a.v : a.k) + (t0 + tk) * (isv ? a.vs[0] : a.ks[0]) +
                       (isv ? r - a.H_kv : r) * (isv ? a.vs[1] : a.ks[1]) + item * 16;
        x0[u] = __ldg(reinterpret_cast<const uint4*>(src));
        x1[u] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      }
    }
  };
  load(lane / L);
  const int first = find_seq(a.cu, a.B, static_cast<int>(t0), lane);
  int64_t mine = -1;  // of row t0 + lane
  if (lane < nt) {
    const int t = static_cast<int>(t0) + lane;
    const int b = find_seq_from(a.cu, a.B, first, t);
    if (b < a.B) {  // else behind the last sequence
      const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
      const int64_t pos = static_cast<int64_t>(__ldg(a.seqlens + b)) - (static_cast<int64_t>(c1) - c0) + (t - c0);
      if (t >= c0) mine = cache_row(a, b, pos, 41);
    }
  }
  if (__all_sync(kFull, mine < 0)) return;
  for (int base = 0; base < rows; base += U * RW) {
    if (base != 0) load(base + lane / L);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * RW >= rows) break;  // the same for the whole warp: all lanes shuffle
      const int idx = base + u * RW + lane / L;
      const int tk = idx & ((1 << a.lg) - 1), r = idx >> a.lg;
      const bool isv = r >= a.H_kv;
      const int64_t at = __shfl_sync(kFull, mine, tk);
      const bool live = idx < rows && at >= 0;
      const int64_t row = at + static_cast<int64_t>(isv ? r - a.H_kv : r) * a.page;
      const bool in = live && FA_IN_BOUNDS(row >= 0 && row < static_cast<int64_t>(a.P) * a.H_kv * a.page, a.status, 404);
      if constexpr (!Q8) {
        if (in) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(isv ? a.v_pages : a.k_pages) + row * D + item * 16);
          dst[0] = x0[u];
          dst[1] = x1[u];
        }
      } else {
        float f[16];
        const uint32_t* w0 = &x0[u].x;
        const uint32_t* w1 = &x1[u].x;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = ElemOps<E>::unpack(live ? w0[i] : 0u), q = ElemOps<E>::unpack(live ? w1[i] : 0u);
          f[2 * i] = p.x;
          f[2 * i + 1] = p.y;
          f[8 + 2 * i] = q.x;
          f[9 + 2 * i] = q.y;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool fin = fabsf(f[i]) <= 3.402823466e38f;
          if (fin) amax = fmaxf(amax, fabsf(f[i]));
          else f[i] = __uint_as_float(0x7fc00000u);  // infinities and NaN become e4m3's NaN
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = e4m3_exponent<E>(amax);
        const float inv = __int_as_float((127 - e) << 23);
        if (E == Elem::kF16 && e == 8) {  // 256 * 2^8 would be read back as infinity: 240 is the last code that fits
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = fabsf(f[i]) > 240.f * 256.f ? copysignf(240.f * 256.f, f[i]) : f[i];
        }
        if (in) {
          uint4 c;
          c.x = pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
          c.y = pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
          c.z = pack_e4m3x4(f[8] * inv, f[9] * inv, f[10] * inv, f[11] * inv);
          c.w = pack_e4m3x4(f[12] * inv, f[13] * inv, f[14] * inv, f[15] * inv);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(isv ? a.v_pages : a.k_pages) + row * D + item * 16) = c;
          if (item == 0) (isv ? a.v_scales : a.k_scales)[row] = static_cast<uint8_t>(e + 127);
        }
      }
    }
  }
}

// Reads rows of a ragged batch back from the cache: row cu[b] + i is position starts[b] + i of
// sequence b.  Rows whose position is at or past the sequence's length, and rows behind the last
// sequence, are left as they were.  Warps and lanes as in the append.
template <Elem E, int D, bool Q8>
__global__ void __launch_bounds__(128) fa_cache_gather_kernel(const CacheArgs a) {
  using T = typename ElemOps<E>::T;
  constexpr int L = D / 16;
  constexpr int RW = 32 / L;
  constexpr int U = 4;
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)) << a.lg;
  if (t0 >= a.T) return;
  const int first = find_seq(a.cu, a.B, static_cast<int>(t0), lane);
  int64_t mine = -1;
  if (lane < 1 << a.lg && t0 + lane < a.T) {
    const int t = static_cast<int>(t0) + lane;
    const int b = find_seq_from(a.cu, a.B, first, t);
    if (b < a.B) {
      const int c0 = __ldg(a.cu + b);
      const int64_t pos = (a.starts ? static_cast<int64_t>(__ldg(a.starts + b)) : 0) + (t - c0);
      if (t >= c0 && pos < __ldg(a.seqlens + b)) mine = cache_row(a, b, pos, 42);
    }
  }
  if (__all_sync(kFull, mine < 0)) return;
  const int item = lane % L;
  const int rows = (2 * a.H_kv) << a.lg;
  for (int base = 0; base < rows; base += U * RW) {
    uint4 x0[U], x1[U];
    uint32_t sc[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int idx = base + u * RW + lane / L;
      const int r = idx >> a.lg;
      const int64_t at = __shfl_sync(kFull, mine, idx & ((1 << a.lg) - 1));
      const bool isv = r >= a.H_kv;
      const int64_t row = at + static_cast<int64_t>(isv ? r - a.H_kv : r) * a.page;
      live[u] = idx < rows && at >= 0 &&
                FA_IN_BOUNDS(row >= 0 && row < static_cast<int64_t>(a.P) * a.H_kv * a.page, a.status, 405);
      if (!live[u]) continue;
      if constexpr (Q8) {
        x0[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(isv ? a.v_pages : a.k_pages) +
                                                     row * D + item * 16));
        sc[u] = __ldg((isv ? a.v_scales : a.k_scales) + row);
      } else {
        const uint4* src =
            reinterpret_cast<const uint4*>(static_cast<const T*>(isv ? a.v_pages : a.k_pages) + row * D + item * 16);
        x0[u] = __ldg(src);
        x1[u] = __ldg(src + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      const int idx = base + u * RW + lane / L;
      const int r = idx >> a.lg;
      const int64_t t = t0 + (idx & ((1 << a.lg) - 1));
      const bool isv = r >= a.H_kv;
      if constexpr (Q8) {
        const float f = e8m0_to_float(sc[u]);
        const uint32_t w[4] = {x0[u].x, x0[u].y, x0[u].z, x0[u].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = e4m3x2_to_float2(w[i]), q = e4m3x2_to_float2(w[i] >> 16);
          o[2 * i] = ElemOps<E>::pack(p.x * f, p.y * f);
          o[2 * i + 1] = ElemOps<E>::pack(q.x * f, q.y * f);
        }
        x0[u] = make_uint4(o[0], o[1], o[2], o[3]);
        x1[u] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      T* dst = static_cast<T*>(isv ? a.v_out : a.k_out) + (t * a.H_kv + (isv ? r - a.H_kv : r)) * D + item * 16;
      if (FA_IN_BOUNDS(t < a.T && item * 16 + 16 <= D, a.status, 406)) {
        reinterpret_cast<uint4*>(dst)[0] = x0[u];
        reinterpret_cast<uint4*>(dst)[1] = x1[u];
      }
    }
  }
}

}  // namespace fa
