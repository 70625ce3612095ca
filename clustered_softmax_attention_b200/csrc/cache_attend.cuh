// What the two forms of attention over the 4-bit cache share: the line of work and its stretches,
// small device pieces, and the join of partial sums.
#pragma once

#include <algorithm>

#include <cuda_fp16.h>

#include "cache.cuh"

namespace muse {

constexpr int kMaxCtas = 592;   // 148 SMs x 4: the bound of the partials in the workspace
constexpr int kTcRows = 128;    // rows of a block of the form for many rows
constexpr int kTcMaxCtas = 160; // its CTAs: one an SM
struct AttendArgs {
  muse_rows Q, O;
  float *lse;
  const int32_t *lens, *counts;
  int B, H, M, G;      // G = H / Hkv
  int nrb;             // row blocks of a head's G * M rows, 2^block_log2 rows each
  int block_log2;
  int min_tiles;       // a CTA takes at least so many tiles
  int tile_log2;       // tokens of a tile: 32, or 128
  int item_tiles;      // kItemTiles, in such tiles
  int cluster;         // CTAs of an item, or 0: stretches of the line
  float scale;
  float *part;         // [2 kMaxCtas][rows of a block][Dv]
  float *part_ml;      // [2 kMaxCtas][rows of a block][2]
  int2 *ends;          // [items]: slot of an item's first part, CTA of its last
};

// New rows, and tokens that the last of them may see, of sequence b.
__device__ __forceinline__ int seq_rows(const AttendArgs &a, int b) {
  if (!a.counts) return a.M;
  return min(max(a.counts[b], 0), a.M);
}
__device__ __forceinline__ int seq_len(const AttendArgs &a, const CacheView &v, int b) {
  const int64_t cap = (int64_t)v.max_pages << v.page_log2;
  return (int)min((int64_t)max(a.lens[b], 0), cap);
}
// Lengths and counts outside their range: those tokens and rows are left out.
__device__ __forceinline__ void check_lengths(const AttendArgs &a, const CacheView &v, int b,
                                              int *status) {
  if ((a.counts && seq_rows(a, b) != a.counts[b]) || seq_len(a, v, b) != a.lens[b])
    report(status, MUSE_ERR_DEVICE);
}
__device__ __forceinline__ int seq_tiles(const AttendArgs &a, const CacheView &v, int b) {
  return seq_rows(a, b) ? (seq_len(a, v, b) + (1 << a.tile_log2) - 1) >> a.tile_log2 : 0;
}

// Beginning and ending an item (its queries, joining its sums) takes a CTA as long as kItemTiles
// tiles: so many places on the line come before each item's tiles.  With 8, 12, 16, 20 and 28, us behind
// a flushed L2 (they repeat within 2): 48 sequences of up to 8192 tokens, 8 heads, 109 99 93 91 91; 64 of up
// to 4096 with 16 rows a head, 130 112 103 103 105; 200 of up to 2048, 136 128 120 118 122; 2 of 65536, 16
// heads, 97 95 93 93 93; float32 rows, the first batch, 122 116 118 116 120.  With 64 rows a head, whose
// tiles take six times as long, fewer would do: 24 of up to 4096 144 151 155 161 169, float32 of up to
// 2048 155 162 171 179 198.  Where a stretch is shorter than this, CTAs fall between the items.
constexpr int kItemTiles = 20;
// Row blocks of sequence b: a padded batch has sequences with fewer rows than M.
__device__ __forceinline__ int seq_blocks(const AttendArgs &a, int b) {
  return (a.G * seq_rows(a, b) + (1 << a.block_log2) - 1) >> a.block_log2;
}
__device__ __forceinline__ int64_t seq_units(const AttendArgs &a, const CacheView &v, int b) {
  const int nt = seq_tiles(a, v, b);
  return nt ? (int64_t)(nt + a.item_tiles) * v.Hkv * seq_blocks(a, b) : 0;
}

// The length of the line.  Each thread sums a run of sequences; run[t] is where thread t's ends.
template <int kThreads>
__device__ __forceinline__ int64_t line_total(const AttendArgs &a, const CacheView &v, int64_t *run) {
  const int tid = threadIdx.x, per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int64_t s = 0;
  for (int b = b0; b < b1; ++b) s += seq_units(a, v, b);
  // inclusive scan over the threads
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) run[kThreads + warp] = s;
  __syncthreads();
  int64_t add = 0;
  for (int w = 0; w < warp; ++w) add += run[kThreads + w];
  run[tid] = s + add;
  __syncthreads();
  return run[kThreads - 1];
}
// The sequence in which position x lies, and the position of its first item.
template <int kThreads>
__device__ __forceinline__ void line_find(const AttendArgs &a, const CacheView &v,
                                          const int64_t *run, int64_t x, int &b, int64_t &first) {
  int lo = 0, hi = kThreads - 1;  // the first thread whose run ends behind x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (run[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  const int per = (a.B + kThreads - 1) / kThreads;
  b = lo * per;
  first = lo ? run[lo - 1] : 0;
  while (b < a.B - 1) {
    const int64_t n = seq_units(a, v, b);
    if (first + n > x) break;
    first += n;
    ++b;
  }
}
// A CTA's walk along the line, from x to x1, and the part of one item that it has come to.
struct Walk {
  int64_t x, x1, first;  // first: position of sequence b's first item
  int b;
};
struct Span {
  int b, hk, rb, t0, t1, nt, len, rows;
  int parts_in;  // CTAs, from this one on, that the item's tiles lie in (where t0 is 0)
};
static __device__ __noinline__ bool next_span(const AttendArgs &a, const CacheView &v, Walk &w, Span &s,
                                       int64_t per) {
  while (w.x < w.x1) {
    int64_t units = seq_units(a, v, w.b);
    while (w.x >= w.first + units) {
      w.first += units;
      units = seq_units(a, v, ++w.b);
    }
    const int nt = seq_tiles(a, v, w.b);
    const int64_t in = w.x - w.first;
    const uint32_t one = (uint32_t)(nt + a.item_tiles);
    const int item = in >> 32 ? (int)(in / one) : (int)((uint32_t)in / one);
    const int64_t start = w.first + (int64_t)item * one + a.item_tiles;  // of its tiles
    s.b = w.b;
    const int blocks = seq_blocks(a, w.b);
    s.hk = item / blocks;
    s.rb = item - s.hk * blocks;
    s.nt = nt;
    s.t0 = (int)max((int64_t)0, w.x - start);
    s.t1 = (int)max((int64_t)0, min((int64_t)nt, w.x1 - start));
    s.len = seq_len(a, v, w.b);
    s.rows = seq_rows(a, w.b);
    const int64_t left = w.x1 - start;  // tiles of the item up to this stretch's end
    const uint32_t per32 = (uint32_t)min(per, (int64_t)0x7fffffff);
    s.parts_in = left >= nt ? 1 : 1 + (int)(((uint32_t)(nt - left) + per32 - 1) / per32);
    w.x = left >= nt ? start + nt : w.x1;
    if (s.t0 < s.t1) return true;
  }
  return false;
}

// Places of a CTA's stretch, and where this one's begins; false when there is nothing left for it.
template <int kThreads>
__device__ __forceinline__ bool line_start(const AttendArgs &a, const CacheView &v, int64_t *run,
                                           Walk &w, int64_t &per) {
  const int64_t total = line_total<kThreads>(a, v, run);
  const int64_t up = total + gridDim.x - 1;
  per = max((int64_t)a.min_tiles, up >> 32 ? up / gridDim.x : (int64_t)((uint32_t)up / gridDim.x));
  w.x = blockIdx.x * per;
  w.x1 = min(total, w.x + per);
  if (w.x >= w.x1) return false;
  line_find<kThreads>(a, v, run, w.x, w.b, w.first);
  return true;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  return bits(__floats2half2_rn(lo, hi));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A weight is 2^(x r - m) with x r rounded, as it was when the reference m was taken: by the unrounded
// product a logit of 2^28 would be off by up to 16, and its weight past what float16 holds.  m, 9 below a
// logit, is rounded upwards.  The tcgen05 form, which has 128 weights a row and tile, rounds product and
// difference once as long as its references are below kFar, where that is off by 2^-4 at most.
constexpr float kFar = 0x1p20f;
// (x & mask) | with in one operation (written out, it becomes two).
template <uint32_t kMask>
__device__ __forceinline__ uint32_t picked(uint32_t x, uint32_t with) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "n"(kMask), "r"(with));
  return y;
}
// Four pairs of codes of a word (nibbles n and n + 4) as float16: 1024 + u, or 1024 + 16 u,
// without its offset.  Small integers under the exponent of a power of two, whose mantissa they become, is
// a published way of unpacking 4-bit weights (Y. J. Kim et al., 2022).
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&c)[4]) {
  const uint32_t y = x >> 8;
  const __half2 less = __half2half2(__ushort_as_half(0xE408));     // -1032
  const __half2 part = __half2half2(__ushort_as_half(0x2C00));     // 1/16
  const __half2 less16 = __half2half2(__ushort_as_half(0xD480));   // -72
  constexpr uint32_t k1024 = 0x64006400u;
  uint32_t t[4] = {picked<0x000f000fu>(x, k1024), picked<0x00f000f0u>(x, k1024),
                   picked<0x000f000fu>(y, k1024), picked<0x00f000f0u>(y, k1024)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&t[i]);
    c[i] = bits(i & 1 ? __hfma2(h, part, less16) : __hadd2(h, less));
  }
}
__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// Four channels of a row: sums y over weights of sum z at reference `at`.
template <typename T>
__device__ __forceinline__ void finish_row(const AttendArgs &a, int b, int h, int m, int c,
                                           const float (&y)[4], float z, float at) {
  const float inv = z == 0.f ? 0.f : 1.f / z;  // a row that sees nothing is zero
  T *dst = (T *)a.O.p + b * a.O.sb + h * a.O.sh + m * a.O.sn + c;
  if (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(dst) = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
  } else {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(bits(__floats2bfloat162_rn(y[0] * inv, y[1] * inv)),
                                                 bits(__floats2bfloat162_rn(y[2] * inv, y[3] * inv)));
  }
  if (c == 0 && a.lse)
    a.lse[((int64_t)b * a.H + h) * a.M + m] =
        z == 0.f ? -CUDART_INF_F : (at + log2f(z)) * 0.693147181f;
}

// Rows of items that lie in several stretches (or in none: nothing to see).  One CTA per row, its
// parts read by four warps in turn and joined in a fixed order.  It takes as long as the loads that
// wait for one another: the ends, then references and sums together.  Four sums a thread are asked
// for ahead, in the 40 registers of which 12 CTAs fit an SM (eight sums take 56 registers, 9 CTAs an
// SM, and 1536 rows two waves).  References first and sums after them took 2 us longer with 2
// heads x 512 rows over 16384 tokens, 1 us with 2 x 16 rows over 65536.
template <typename T, int Dv, int kRows>
__global__ void __launch_bounds__(128, 12) attend_join(const __grid_constant__ AttendArgs a,
                                                   const __grid_constant__ CacheView v, int *status) {
  constexpr int kThreads = 128, kGroups = kThreads / (Dv / 4), kAhead = 4;
  constexpr int kCtas = kRows == kTcRows ? kTcMaxCtas : kMaxCtas;
  constexpr int kMine = (kCtas + kThreads - 1) / kThreads;  // references of a thread
  __shared__ float s_w[kCtas], s_red[8];
  __shared__ float4 s_y[kGroups][Dv / 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int m = gr / a.G, h = hk * a.G + (gr - m * a.G);
  const int rb = gr / kRows, row = gr - rb * kRows;
  dependents_may_launch();
  wait_for_earlier();
  int2 ends = a.ends[((int64_t)b * v.Hkv + hk) * a.nrb + rb];  // not written where there is nothing
  const int rows = seq_rows(a, b);
  if (gr == 0 && hk == 0 && tid == 0) check_lengths(a, v, b, status);
  const int nt = seq_tiles(a, v, b);
  if (m >= rows) return;
  if (!nt) ends = make_int2(0, -1);
  const int c0 = ends.x >> 1, n = ends.y - c0 + 1;
  if (n == 1) return;  // finished by its only CTA
  // a wait that gave up leaves an item without its ends: nothing is read by them
  if (nt && ((unsigned)c0 >= (unsigned)kCtas || (unsigned)ends.y >= (unsigned)kCtas || n < 1)) {
    if (tid == 0) report(status, MUSE_ERR_DEVICE);
    return;
  }
  // a part that begins its stretch is in the even slot: all but, perhaps, the first
  auto slot_of = [&](int k) { return k ? 2 * (int64_t)(c0 + k) : (int64_t)ends.x; };
  const int grp = tid / (Dv / 4), c4 = tid - grp * (Dv / 4);
  auto part = [&](int k) {
    return reinterpret_cast<const float4 *>(a.part + (slot_of(k) * kRows + row) * Dv)[c4];
  };
  float2 ml[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int k = tid + i * kThreads;
    ml[i] = make_float2(-CUDART_INF_F, 0.f);
    if (k < n) ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + (slot_of(k) * kRows + row) * 2);
  }
  float4 first[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    first[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp + i * kGroups < n) first[i] = part(grp + i * kGroups);
  }
  float ref = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < kMine; ++i) ref = fmaxf(ref, ml[i].x);
  ref = warp_max(ref);
  if (lane == 0) s_red[warp] = ref;
  __syncthreads();
  ref = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  const float at = ref == -CUDART_INF_F ? 0.f : ref;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int k = tid + i * kThreads;
    const float w = ex2(ml[i].x - at);
    if (k < n) s_w[k] = w;
    z = fmaf(w, ml[i].y, z);
  }
  z = warp_sum(z);
  if (lane == 0) s_red[4 + warp] = z;
  __syncthreads();
  z = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](float f, const float4 &o) {
    y[0] = fmaf(f, o.x, y[0]);
    y[1] = fmaf(f, o.y, y[1]);
    y[2] = fmaf(f, o.z, y[2]);
    y[3] = fmaf(f, o.w, y[3]);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (grp + i * kGroups < n) add(s_w[grp + i * kGroups], first[i]);
#pragma unroll 8
  for (int k = grp + kAhead * kGroups; k < n; k += kGroups) add(s_w[k], part(k));
  s_y[grp][c4] = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) add(1.f, s_y[k][c4]);
  finish_row<T>(a, b, h, m, 4 * c4, y, z, at);
}

// The form for more than 64 bfloat16 rows of a cache head (cache_attend_tc.cu), in blocks of 128.
// Beginning and ending an item, in its tiles of 128 tokens.  With 0, 3, 6, 8, 11 and 16, us behind a
// flushed L2: 2 x 2 heads of 16384 tokens, 512 rows each, 92 86 81 79 83 83; 48 sequences of 128 to 8000
// tokens, 4 heads of 128 rows, 273 251 228 228 228 233; 24 of 0 to 8191, 8 heads, 300 250 225 225 222 239;
// but 8 heads of 1024 tokens, 512 rows each, 44 46 48 50 50 52 (stretches shorter than this).
constexpr int kTcItemTiles = 8;
template <int D, int Dv>
cudaError_t launch_attend_tc(AttendArgs a, const CacheView &v, int *status, cudaStream_t st);

}  // namespace muse
