// Causal attention of a sequence's newest rows over its 4-bit cache.
//
// The rows of one cache head (the H / Hkv query heads of every new token) are the columns of a
// 16 x 8 matrix-instruction tile and tokens, then value channels, its rows, so that eight rows
// or fewer (a token of grouped heads) fill it.  Keys and values enter as their integer codes,
// dequantised in registers to signed float16 (exact, two codes a register):
//   S^T = sum_w kstep[t][w] (sum_{c in group w} code_tc q_c),    p = 2^(S rf - m),
//   O^T = sum_t code_tc (p_t vstep[t][w]),
// so a step multiplies a sum (keys) or a weight (values), never a code.  The layout of a tile is
// such that 16 bytes a lane are operands as they lie; only the weights are turned over between
// the two products, eight by eight (movmatrix).
//
// Work is split evenly whatever the lengths: the 32-token tiles of all (sequence, head, row
// block) items form one line, and every CTA takes a stretch of it.  An item that lies in one
// stretch is finished there; the others leave float32 partial sums (at most two a CTA), which
// attend_join adds in the order of the CTAs: results do not depend on timing.  Where no sequence
// can be long, a cluster of CTAs takes an item instead and joins its sums through distributed
// shared memory: one launch.
//
// What bounds it, bfloat16 rows of 128 + 128 channels: up to 8 rows a cache head a further 32-token
// tile costs the card 1.03 ns (4.5 TB/s of codes); it is the instructions that turn codes and weights
// into operands (746 a tile; ALU 39 %, tensor pipe 29 %, issue slots about half used), not DRAM (44 %).
// Two sequences of 65536 tokens, 16 heads: 87 us, 3.5 TB/s, 53 % of a copy's rate, of which 68 are tiles
// and 19 are not: setting up, the first tile's way, 6 us of joining.  A tile with 16, 32 and 64 rows:
// 1.6, 3.3 and 6.4 ns: codes are dequantised by every warp for its 16 rows.
#include <algorithm>
#include <atomic>

#include "cache_attend.cuh"

namespace muse {
namespace {

constexpr int kWarps = 4;
constexpr int kCluster = 8;      // CTAs of a cluster that takes an item
// Clusters take tables of up to so many 32-token tiles a token slice (a sequence's CTAs are fixed
// beforehand, so a ragged batch waits for its longest).  In stretches and here, us behind a flushed
// L2: 8 heads of 4000 tokens 21 and 16; 4 x 8 of 8000 30 and 27, ragged or not; 4 x 8 of 16000 40 and 39,
// ragged 36 and 37.  Float32 rows, whose tiles take three times as long: 9 heads of 4000 tokens 19 and 16,
// of 8000 24 and 22, of 16000 28 and 33.  More CTAs than fit at once: 7 x 8 heads of 8000 tokens 38 and
// 48; only short tables then (of 1000: 24 and 25).  It goes by the table, whose width the host knows: a
// sequence of 1000 tokens in a table of 65536 takes 17 us in stretches, in one of its own size 14.
template <typename T>
constexpr int kClusterTiles = sizeof(T) == 4 ? 32 : 64;
constexpr int kClusterTilesTwice = 16;
// ------------------------------------------------------------------ small device pieces

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 cluster_ld4(const float *p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(at)
               : "memory");
  return x;
}
template <int N>
__device__ __forceinline__ void slice_sync(int slice) {  // the N warps of a token slice
  if (N == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "n"(32 * N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values turned over: lane (g, q) gives row g, columns 2 q and 2 q + 1,
// and takes column g, rows 2 q and 2 q + 1.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The same pairs as bfloat16 (128 + u without its offset).
__device__ __forceinline__ void codes_bf16(uint32_t x, uint32_t (&c)[4]) {
  const __nv_bfloat162 less = __bfloat162bfloat162(__ushort_as_bfloat16(0xC308));  // -136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = picked<0x000f000fu>(x >> (4 * i), 0x43004300u);
    c[i] = bits(__hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&t), less));
  }
}
// Group w of two packed steps.
template <int N>
__device__ __forceinline__ float step_of(const uint32_t (&s)[N], int w) {
  return w & 1 ? hi_f(s[w >> 1]) : lo_f(s[w >> 1]);
}

// Words of eight tokens: K words of token 8 i + g for the groups, V words of tokens 8 i + 2 q and
// 8 i + 2 q + 1 for the halves.
template <int D>
__device__ __forceinline__ void words(const uint8_t *codes, int i, int lane, uint32_t (&w)[D / 32]) {
  const uint4 *p = reinterpret_cast<const uint4 *>(codes);
  if (D == 128) {
    const uint4 x = p[i * 32 + lane];
    w[0] = x.x;
    w[1] = x.y;
    w[D / 32 - 2] = x.z;
    w[D / 32 - 1] = x.w;
  } else {
    const uint2 x = reinterpret_cast<const uint2 *>(p + (i >> 1) * 32 + lane)[i & 1];
    w[0] = x.x;
    w[1] = x.y;
  }
}
// Steps of token t, two groups a register.
template <int D>
__device__ __forceinline__ void steps(const uint8_t *p, int t, uint32_t (&s)[D / 64]) {
  if (D == 128) {
    const uint2 x = reinterpret_cast<const uint2 *>(p)[t];
    s[0] = x.x;
    s[D / 64 - 1] = x.y;
  } else {
    s[0] = reinterpret_cast<const uint32_t *>(p)[t];
  }
}
// Both tokens' words of a value group: a half word of each, four channels.
template <int Dv>
__device__ __forceinline__ uint32_t value_pair(const uint32_t (&x)[Dv / 32], int grp) {
  return __byte_perm(Dv == 128 ? x[grp >> 1] : x[0], Dv == 128 ? x[Dv / 64 + (grp >> 1)] : x[1],
                     grp & 1 ? 0x7632 : 0x5410);
}

// O^T of 8 NB rows times unit[group]: row 8 nb + 2 q + e, channel 16 j + 8 h + g at
// [nb][j][2 h + e].
template <int Dv, int NB>
struct Acc {
  float o[NB][Dv / 16][4];
};
// Logits, then weights, of the tile: [nb][i][e] = row 8 nb + 2 q + e, token 8 i + g.
template <int NB>
struct Tok {
  float p[NB][4][2];
};
// Which tokens of a tile the rows do not see (left = see - the tile's first token).
template <int NB>
struct Hide {
  bool edge;
  int left[NB][2];
  __device__ __forceinline__ bool at(int nb, int t, int e) const { return edge && t >= left[nb][e]; }
};

// O += (p vstep) code; ds: the steps as float16 in the accumulators' unit, in [2^-7, 2), two groups
// a register.  p vstep is the sum of two float16: the rounded product of p's upper piece, and what that
// rounding cut off together with p's lower piece: 21 bits, and never coarser than 2^-23 of the unit, where
// a weight at the reference is 2^9.  In one piece (11 bits, rounded twice) results differed from float32
// arithmetic's by a bfloat16 step in one element of thirty (1e-3 in norm, 5e-5 in two pieces).  8 x 8
// heads of 32768 tokens, 128 + 128 channels, one piece and two: 8 rows 88 and 96 us, 64 rows 363 and 452.
template <int Dv, int NB>
__device__ __forceinline__ void values_f16(Acc<Dv, NB> &acc, const uint8_t *codes,
                                           const uint32_t (&ds)[4][Dv / 64], const Tok<NB> &tk,
                                           int lane) {
  __half2 p[NB][4], rest[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[nb][i] = __floats2half2_rn(tk.p[nb][i][0], tk.p[nb][i][1]);
      rest[nb][i] = __floats2half2_rn(tk.p[nb][i][0] - __low2float(p[nb][i]),
                                      tk.p[nb][i][1] - __high2float(p[nb][i]));
    }
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint32_t x[2][Dv / 32];
    words<Dv>(codes, 2 * kk, lane, x[0]);
    words<Dv>(codes, 2 * kk + 1, lane, x[1]);
#pragma unroll
    for (int grp = 0; grp < Dv / 32; ++grp) {
      // nibbles n and n + 4 of a pair are channel 8 n + g of the group, of both tokens
      uint32_t c[2][4];
      codes_f16(value_pair<Dv>(x[0], grp), c[0]);
      codes_f16(value_pair<Dv>(x[1], grp), c[1]);
      const uint32_t a0[4] = {c[0][0], c[0][1], c[1][0], c[1][1]};
      const uint32_t a1[4] = {c[0][2], c[0][3], c[1][2], c[1][3]};
      __half2 f[2];
#pragma unroll
      for (int ii = 0; ii < 2; ++ii) {
        const __half2 x2 = *reinterpret_cast<const __half2 *>(&ds[2 * kk + ii][grp >> 1]);
        f[ii] = grp & 1 ? __high2half2(x2) : __low2half2(x2);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {
          const int i = 2 * kk + ii;
          const __half2 w = __hmul2(p[nb][i], f[ii]);
          // what the product's rounding cut off (exact), and the rest of the weight
          lo[ii] = turned(bits(__hfma2(rest[nb][i], f[ii], __hfma2(p[nb][i], f[ii], __hneg2(w)))));
          hi[ii] = turned(bits(w));
        }
        mma_f16(acc.o[nb][2 * grp], a0, hi[0], hi[1]);
        mma_f16(acc.o[nb][2 * grp + 1], a1, hi[0], hi[1]);
        mma_f16(acc.o[nb][2 * grp], a0, lo[0], lo[1]);
        mma_f16(acc.o[nb][2 * grp + 1], a1, lo[0], lo[1]);
      }
    }
  }
}

// The same with p vstep in three bfloat16 pieces (24 bits): any range.  The sum over the tile's 32
// tokens is formed apart and added once.
template <int Dv, int NB>
__device__ __forceinline__ void values_wide(Acc<Dv, NB> &acc, const uint8_t *codes,
                                            const uint8_t *vstep, const Tok<NB> &tk,
                                            const float (&unit)[Dv / 32], const Hide<NB> &hide,
                                            int lane) {
  const int g = lane >> 2;
#pragma unroll
  for (int grp = 0; grp < Dv / 32; ++grp) {
    float t[NB][2][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 8; ++e) t[nb][e >> 2][e & 3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t c[2][4];
      float f[2];
#pragma unroll
      for (int ii = 0; ii < 2; ++ii) {
        uint32_t x[Dv / 32], s[Dv / 64];
        words<Dv>(codes, 2 * kk + ii, lane, x);
        codes_bf16(value_pair<Dv>(x, grp), c[ii]);
        steps<Dv>(vstep, 8 * (2 * kk + ii) + g, s);
        f[ii] = step_of(s, grp) * unit[grp];
      }
      const uint32_t a0[4] = {c[0][0], c[0][1], c[1][0], c[1][1]};
      const uint32_t a1[4] = {c[0][2], c[0][3], c[1][2], c[1][3]};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float w[2][2];
#pragma unroll
        for (int ii = 0; ii < 2; ++ii)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * kk + ii;
            w[ii][e] = hide.at(nb, 8 * i + g, e) ? 0.f : tk.p[nb][i][e] * f[ii];
          }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t b[2];
#pragma unroll
          for (int ii = 0; ii < 2; ++ii) {
            b[ii] = bits(__floats2bfloat162_rn(w[ii][0], w[ii][1]));
            w[ii][0] -= lo_f(b[ii]);
            w[ii][1] -= hi_f(b[ii]);
            b[ii] = turned(b[ii]);
          }
          mma_bf16(t[nb][0], a0, b[0], b[1]);
          mma_bf16(t[nb][1], a1, b[0], b[1]);
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        acc.o[nb][2 * grp + (e >> 2)][e & 3] += t[nb][e >> 2][e & 3];
  }
}

// One CTA: RT row tiles of 8 NB x kWarps / RT token slices.
template <typename T, int D, int Dv, int NB, int RT>
struct Shape {
  static constexpr int kSlices = kWarps / RT;
  static constexpr int kTileRows = 8 * NB;
  static constexpr int kRows = kTileRows * RT;
  static constexpr int kStages = RT == 1 ? 3 : 4;            // tiles under way of a token slice
  static constexpr int kRing = kSlices * kStages * TileShape<D, Dv>::kBytes;
  static constexpr int kSumRow = Dv + 4;                     // so that lanes store to other banks
  static constexpr int kSum = kWarps * 8 * kSumRow * 4;      // eight rows of every warp
  static constexpr int kSmem = kRing + kSum;
  static constexpr bool kClusters = kRows * kSumRow * 4 <= kRing;  // an item's rows, over the ring
  static constexpr int kLoads = sizeof(T) / 2;               // 16-byte loads of eight channels
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;      // float16 pieces of a query
};

template <typename T, int D, int Dv, int NB, int RT>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 4 || (NB == 2 && Dv == 128) ? 2 : 3)
attend(const __grid_constant__ AttendArgs a, const __grid_constant__ CacheView v, int *status) {
  using S = TileShape<D, Dv>;
  using C = Shape<T, D, Dv, NB, RT>;
  constexpr int NGk = D / 32, NG = Dv / 32, TS = C::kSlices, kThreads = 32 * kWarps;
  constexpr int QP = C::kParts, kStages = C::kStages;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t run[kThreads + kWarps];
  __shared__ float s_ml[TS][RT * 8][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int rt = warp % RT, ts = warp / RT;

  // ---- what this CTA does: a stretch of the line, or its part of its cluster's item
  Walk walk;
  Span sp;
  int64_t per = 1;
  dependents_may_launch();
  wait_for_earlier();
  if (C::kClusters && a.cluster) {
    const int rank = blockIdx.x % a.cluster, item = blockIdx.x / a.cluster;
    sp.b = item / (v.Hkv * a.nrb);
    sp.hk = item / a.nrb % v.Hkv;
    sp.rb = item % a.nrb;
    sp.nt = sp.rb < seq_blocks(a, sp.b) ? seq_tiles(a, v, sp.b) : 0;
    sp.t0 = sp.nt * rank / a.cluster;
    sp.t1 = sp.nt * (rank + 1) / a.cluster;
    sp.len = seq_len(a, v, sp.b);
    sp.rows = seq_rows(a, sp.b);
    walk.x = walk.x1 = 0;
    if (rank == 0 && sp.hk == 0 && sp.rb == 0 && tid == 0) check_lengths(a, v, sp.b, status);
  } else {
    if (!line_start<kThreads>(a, v, run, walk, per)) return;
    if (!next_span(a, v, walk, sp, per)) return;
  }

  uint8_t *ring = smem + ts * kStages * S::kBytes;
  float *sum = reinterpret_cast<float *>(smem + C::kRing);
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  const int slice_tid = rt * 32 + lane;

  // ---- the slice's tiles t0 + ts, + TS, ... of one span after the other: kStages - 1 of them are
  // under way, across spans too
  Walk ahead = walk;
  int f_tile = sp.t0 + ts, f_end = sp.t1;
  uint32_t there = 0;  // bit 0: the tile to be used next is there (its page is in the cache)
  uint32_t into = 0, used = 0;
  const uint8_t *src = nullptr;
  // a head's tiles of page 0, the sequence's pages, and from page to page in units of 128 bytes
  const int per_log2 = v.page_log2 - 5, per_mask = (1 << per_log2) - 1;
  const uint32_t page_units = ((uint32_t)v.Hkv * (S::kBytes / 128)) << per_log2;
  const uint8_t *f_head;
  const int32_t *f_pages;
  auto begin = [&](const Span &to) {
    f_head = v.tiles + (((int64_t)to.hk * S::kBytes) << per_log2);
    f_pages = v.table + (int64_t)to.b * v.max_pages;
    f_tile = to.t0 + ts;
    f_end = to.t1;
  };
  begin(sp);
  auto place = [&]() {  // where the next tile lies, asked for a step before it is fetched
    while (f_tile >= f_end) {
      Span n;
      if (!next_span(a, v, ahead, n, per)) return;
      begin(n);
    }
    const uint32_t pg = (uint32_t)f_pages[f_tile >> per_log2];
    src = pg < (uint32_t)v.pages
              ? f_head + ((uint64_t)pg * page_units << 7) + (uint32_t)((f_tile & per_mask) * S::kBytes)
              : nullptr;
  };
  auto fetch = [&]() {
    if (f_tile < f_end) {
      if (src) {
#pragma unroll
        for (int i = 0; i < S::kBytes / 16; i += 32 * RT)
          if (S::kBytes / 16 % (32 * RT) == 0 || i + slice_tid < S::kBytes / 16)
            cp16(ring_s + into + (i + slice_tid) * 16, src + (i + slice_tid) * 16);
        there |= 1u << (kStages - 1);
      } else if (slice_tid == 0) {
        report(status, MUSE_ERR_DEVICE);
      }
      into = into == (kStages - 1) * S::kBytes ? 0 : into + S::kBytes;
      f_tile += TS;
      place();
    }
    cp_commit();
  };
  place();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    fetch();
    there >>= 1;
  }

  // this lane's part of row 8 nb + g: channels 32 w + 8 q + (0..7)
  uint4 raw[NB][NGk * C::kLoads];
  auto load_rows = [&](const Span &to) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = to.rb * C::kRows + rt * C::kTileRows + 8 * nb + g;
      const int m = row / a.G, h = to.hk * a.G + (row - m * a.G);
      const T *from = (const T *)a.Q.p + to.b * a.Q.sb + h * a.Q.sh + m * a.Q.sn + 8 * q;
#pragma unroll
      for (int i = 0; i < NGk * C::kLoads; ++i)
        raw[nb][i] = m < to.rows ? reinterpret_cast<const uint4 *>(
                                       from + 32 * (i / C::kLoads))[i % C::kLoads]
                                 : make_uint4(0, 0, 0, 0);
    }
  };
  load_rows(sp);

  for (int spans = 0;; ++spans) {
    const int n_it = max(0, (sp.t1 - sp.t0 - ts + TS - 1) / TS);

    // ---- queries as float16 pieces, a power of two a row
    uint32_t qb[QP][NB][D / 16][2];
    float rf[NB][2];     // rows 2 q + e from here on
    int see[NB][2], see_all = 0x7fffffff;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t top = 0;  // the largest magnitude's bits: an infinity or a NaN is above all others
#pragma unroll
      for (int i = 0; i < NGk * C::kLoads; ++i) {
        const uint32_t x[4] = {raw[nb][i].x, raw[nb][i].y, raw[nb][i].z, raw[nb][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top = sizeof(T) == 4 ? max(top, x[k] & 0x7fffffffu) : __vmaxu2(top, x[k] & 0x7fff7fffu);
      }
      if (sizeof(T) == 2) top = max(top << 16, top & 0xffff0000u);
      top = max(top, __shfl_xor_sync(kAll, top, 1));
      top = max(top, __shfl_xor_sync(kAll, top, 2));
      const bool bad = top >= 0x7f800000u;
      // q 2^-e with its largest in [2^14, 2^15): float16 keeps bfloat16 values exactly down to
      // 2^-31 of the largest, float32 ones to 22 bits in two pieces.  A row with an infinity or a
      // NaN is NaN.
      const int e = min(max((int)(top >> 23) - 127 - 14, -114), 113);
      const float mul = bad ? CUDART_NAN_F : a.scale < 0.f ? -ldexpf(1.f, -e) : ldexpf(1.f, -e);
      // logits in units of log 2; above zero, so that what is hidden stays -infinity
      const float rfg = fmaxf(ldexpf(fabsf(a.scale) * 1.44269504f, e), 1e-45f);
      const int row0 = sp.rb * C::kRows + rt * C::kTileRows + 8 * nb;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rf[nb][k] = __shfl_sync(kAll, rfg, (2 * q + k) * 4);
        const int m = (row0 + 2 * q + k) / a.G;
        // a place without a row sees all, so that it masks nothing for its tile (it is not written)
        see[nb][k] = m < sp.rows ? min(max(sp.len - sp.rows + m + 1, 0), sp.len) : sp.len;
        see_all = min(see_all, see[nb][k]);
      }
#pragma unroll
      for (int w = 0; w < NGk; ++w) {
        float u[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const uint4 x = raw[nb][w * C::kLoads + (sizeof(T) == 4 ? n >> 2 : 0)];
          const int k = sizeof(T) == 4 ? n & 3 : n >> 1;
          const uint32_t y = k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
          u[n] = (sizeof(T) == 4 ? __uint_as_float(y) : n & 1 ? hi_f(y) : lo_f(y)) * mul;
        }
        // the two halves of a register of codes are nibbles n and n + 4
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const __half2 hi = __floats2half2_rn(u[n], u[n + 4]);
          qb[0][nb][2 * w + (n >> 1)][n & 1] = bits(hi);
          if (QP == 2)
            qb[QP - 1][nb][2 * w + (n >> 1)][n & 1] =
                pack_f16((u[n] - __low2float(hi)) * 2048.f, (u[n + 4] - __high2float(hi)) * 2048.f);
        }
      }
    }
    // tokens that every row of the warp's tile sees
    see_all = min(see_all, __shfl_xor_sync(kAll, see_all, 1));
    see_all = min(see_all, __shfl_xor_sync(kAll, see_all, 2));

    Acc<Dv, NB> acc;
    float mx[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < Dv / 4; ++e) acc.o[nb][e >> 2][e & 3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nb][e] = -CUDART_INF_F;
        l[nb][e] = 0.f;
      }
    }
    // the accumulators of value group w hold O * unit[w], a power of two; shift: what takes two
    // groups' steps, as bits, to that unit
    uint32_t shift[NG / 2], open = (1u << NG) - 1;  // open: groups that have no unit yet
    float unit[NG];
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      unit[w] = 1.f;
      shift[w >> 1] = 0;
    }

    int tok = (sp.t0 + ts) * kTile - TS * kTile;
    for (int it = 0; it < n_it; ++it) {
      const uint8_t *tile = ring + used;
      used = used == (kStages - 1) * S::kBytes ? 0 : used + S::kBytes;
      tok += TS * kTile;
      cp_wait<kStages - 2>();
      slice_sync<RT>(ts);
      fetch();
      const bool here = there & 1u;
      there >>= 1;
      if (__builtin_expect(!here, 0)) continue;

      // ---- logits
      Tok<NB> tk;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t w[2][NGk], ks[2][NGk / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          words<D>(tile + S::kK, 2 * mt + h, lane, w[h]);
          steps<D>(tile + S::kKStep, 16 * mt + 8 * h + g, ks[h]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) tk.p[nb][2 * mt + h][0] = tk.p[nb][2 * mt + h][1] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < NGk; ++c) {
          uint32_t k[2][4];
          codes_f16(w[0][c], k[0]);
          codes_f16(w[1][c], k[1]);
          const uint32_t a0[4] = {k[0][0], k[1][0], k[0][1], k[1][1]};
          const uint32_t a1[4] = {k[0][2], k[1][2], k[0][3], k[1][3]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(d, a0, qb[0][nb][2 * c][0], qb[0][nb][2 * c][1]);
            mma_f16(d, a1, qb[0][nb][2 * c + 1][0], qb[0][nb][2 * c + 1][1]);
            if (QP == 2) {
              float d2[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d2, a0, qb[QP - 1][nb][2 * c][0], qb[QP - 1][nb][2 * c][1]);
              mma_f16(d2, a1, qb[QP - 1][nb][2 * c + 1][0], qb[QP - 1][nb][2 * c + 1][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) d[e] = fmaf(d2[e], 1.f / 2048.f, d[e]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = step_of(ks[h], c);
              float(&p)[2] = tk.p[nb][2 * mt + h];
              p[0] = fmaf(d[2 * h], f, p[0]);
              p[1] = fmaf(d[2 * h + 1], f, p[1]);
            }
          }
        }
      }
      Hide<NB> hide;
      hide.edge = tok + kTile > see_all;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) hide.left[nb][e] = see[nb][e] - tok;
      if (__builtin_expect(hide.edge, 0)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (hide.at(nb, 8 * i + g, e)) tk.p[nb][i][e] = -CUDART_INF_F;
      }
      // ---- softmax: weights are 2^9 at the reference, which moves when one would pass 2^14
      float top[NB][2];
      bool move = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float(&p)[4][2] = tk.p[nb];
          top[nb][e] = fmaxf(fmaxf(p[0][e], p[1][e]), fmaxf(p[2][e], p[3][e]));
          move |= __fmul_rn(top[nb][e], rf[nb][e]) - mx[nb][e] > 14.f;
        }
      if (__builtin_expect(__any_sync(kAll, move), 0)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = top[nb][e];
            y = fmaxf(y, __shfl_xor_sync(kAll, y, 4));
            y = fmaxf(y, __shfl_xor_sync(kAll, y, 8));
            y = fmaxf(y, __shfl_xor_sync(kAll, y, 16));
            const float now = fmaxf(mx[nb][e], __fsub_ru(__fmul_rn(y, rf[nb][e]), 9.f));
            const float fix = now == -CUDART_INF_F ? 1.f : ex2(mx[nb][e] - now);
            mx[nb][e] = now;
            l[nb][e] *= fix;
#pragma unroll
            for (int j = 0; j < Dv / 16; ++j) {
              acc.o[nb][j][e] *= fix;
              acc.o[nb][j][2 + e] *= fix;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            tk.p[nb][i][e] = ex2(__fmul_rn(tk.p[nb][i][e], rf[nb][e]) - mx[nb][e]);
      if (__builtin_expect(hide.edge, 0)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (hide.at(nb, 8 * i + g, e)) tk.p[nb][i][e] = 0.f;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          l[nb][e] += (tk.p[nb][0][e] + tk.p[nb][1][e]) + (tk.p[nb][2][e] + tk.p[nb][3][e]);

      // ---- value steps in the unit of the accumulators, which a group's first tile that is not all
      // zeros sets (before it the sums are zero, and any unit is right): its largest step comes to
      // [2^-3, 2^-2)
      uint32_t ds[4][NG / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) steps<Dv>(tile + S::kVStep, 8 * i + g, ds[i]);
      if (__builtin_expect(open != 0, 0)) {
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          uint32_t big = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)  // NaN is negative here, and left out
            if (tok + 8 * i + g < sp.len) big = __vmaxs2(big, ds[i][w]);
          big = __vmaxs2(big, __shfl_xor_sync(kAll, big, 4));
          big = __vmaxs2(big, __shfl_xor_sync(kAll, big, 8));
          big = __vmaxs2(big, __shfl_xor_sync(kAll, big, 16));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!((big >> (16 * k)) & 0xffffu) || !((open >> (2 * w + k)) & 1)) continue;
            open &= ~(1u << (2 * w + k));
            const int ex = min(max((int)((big >> (16 * k + 7)) & 255u) - 127, -40), 60);
            unit[2 * w + k] = ldexpf(1.f, -3 - ex);
            // with float16's exponent: 112 less than bfloat16's
            shift[w] += (uint32_t)((-3 - ex - 112) * 128) << (16 * k);
          }
        }
      }
      if (sizeof(T) == 4) {
        values_wide<Dv, NB>(acc, tile + S::kV, tile + S::kVStep, tk, unit, hide, lane);
      } else {
        // A step in [2^-7, 2) of the unit (exponent field 8..15 of a float16; with bfloat16's 7
        // bits below it, so one shift is left) is exact, p at most 2^14, and their product below
        // 2^15.  A tile with another step (a jump of the values' size, a zero, a NaN) goes the wide
        // way.
        uint32_t off_range = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < NG / 2; ++w) {
            ds[i][w] += shift[w];
            off_range |= ds[i][w] ^ 0x04000400u;
            ds[i][w] <<= 3;
          }
        if (__builtin_expect(__any_sync(kAll, off_range & 0xfc00fc00u), 0))
          values_wide<Dv, NB>(acc, tile + S::kV, tile + S::kVStep, tk, unit, hide, lane);
        else
          values_f16<Dv, NB>(acc, tile + S::kV, ds, tk, lane);
      }
    }
    // ---- the next span's queries are asked for, then the slices' sums joined, eight rows of
    // every warp at a time
    const int b = sp.b, hk = sp.hk, rb = sp.rb, rows = sp.rows;
    const bool whole = sp.t0 == 0 && sp.t1 == sp.nt && !(C::kClusters && a.cluster);
    const int slot = 2 * blockIdx.x + (spans ? 1 : 0);
    if (sp.t0 == 0 && tid == 0 && !(C::kClusters && a.cluster))
      a.ends[((int64_t)b * v.Hkv + hk) * a.nrb + rb] = make_int2(slot, blockIdx.x + sp.parts_in - 1);
    const bool more = next_span(a, v, walk, sp, per);
    if (more) load_rows(sp);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __syncthreads();  // the last sums have been read
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(kAll, y, 4);
        y += __shfl_xor_sync(kAll, y, 8);
        y += __shfl_xor_sync(kAll, y, 16);
        const int row = rt * 8 + 2 * q + e;
        if (g == 0) {
          s_ml[ts][row][0] = mx[nb][e];
          s_ml[ts][row][1] = y;
        }
        float *to = sum + (ts * RT * 8 + row) * C::kSumRow + g;
#pragma unroll
        for (int j = 0; j < Dv / 16; ++j) {
          const float back = 1.f / unit[j >> 1];
          to[16 * j] = acc.o[nb][j][e] * back;
          to[16 * j + 8] = acc.o[nb][j][2 + e] * back;
        }
      }
      __syncthreads();
      for (int i = tid; i < RT * 8 * (Dv / 4); i += kThreads) {
        const int r8 = i / (Dv / 4), c = (i - r8 * (Dv / 4)) * 4;
        const int row = r8 / 8 * C::kTileRows + 8 * nb + r8 % 8;  // of the CTA
        const int gr = rb * C::kRows + row;
        const int m = gr / a.G, h = hk * a.G + (gr - m * a.G);
        float ref = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < TS; ++k) ref = fmaxf(ref, s_ml[k][r8][0]);
        const float at = ref == -CUDART_INF_F ? 0.f : ref;
        float z = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < TS; ++k) {
          const float f = ex2(s_ml[k][r8][0] - at);
          const float4 o =
              *reinterpret_cast<const float4 *>(sum + (k * RT * 8 + r8) * C::kSumRow + c);
          z = fmaf(f, s_ml[k][r8][1], z);
          y[0] = fmaf(f, o.x, y[0]);
          y[1] = fmaf(f, o.y, y[1]);
          y[2] = fmaf(f, o.z, y[2]);
          y[3] = fmaf(f, o.w, y[3]);
        }
        if (whole) {
          if (m < rows) finish_row<T>(a, b, h, m, c, y, z, at);
        } else if (C::kClusters && a.cluster) {
          float *to = reinterpret_cast<float *>(smem) + row * C::kSumRow;
          *reinterpret_cast<float4 *>(to + c) = make_float4(y[0], y[1], y[2], y[3]);
          if (c == 0) *reinterpret_cast<float4 *>(to + Dv) = make_float4(ref, z, 0.f, 0.f);
        } else if (m < rows) {
          const int64_t at_row = (int64_t)slot * C::kRows + row;
          *reinterpret_cast<float4 *>(a.part + at_row * Dv + c) = make_float4(y[0], y[1], y[2], y[3]);
          if (c == 0)
            *reinterpret_cast<float2 *>(a.part_ml + at_row * 2) = make_float2(ref, z);
        }
      }
    }
    if (C::kClusters && a.cluster) {
      // a row's sums of all CTAs of the cluster, the rows dealt out among them
      cluster_sync();
      const float *rows_at = reinterpret_cast<const float *>(smem);
      for (int i = tid + kThreads * (blockIdx.x % a.cluster); i < C::kRows * (Dv / 4);
           i += kThreads * a.cluster) {
        const int row = i / (Dv / 4), c = (i - row * (Dv / 4)) * 4;
        const int gr = rb * C::kRows + row;
        const int m = gr / a.G, h = hk * a.G + (gr - m * a.G);
        if (m >= rows) continue;
        float ref = -CUDART_INF_F, z = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < a.cluster; ++k)
          ref = fmaxf(ref, cluster_ld4(rows_at + row * C::kSumRow + Dv, k).x);
        const float at = ref == -CUDART_INF_F ? 0.f : ref;
        for (int k = 0; k < a.cluster; ++k) {
          const float4 ml = cluster_ld4(rows_at + row * C::kSumRow + Dv, k);
          const float4 o = cluster_ld4(rows_at + row * C::kSumRow + c, k);
          const float f = ex2(ml.x - at);
          z = fmaf(f, ml.y, z);
          y[0] = fmaf(f, o.x, y[0]);
          y[1] = fmaf(f, o.y, y[1]);
          y[2] = fmaf(f, o.z, y[2]);
          y[3] = fmaf(f, o.w, y[3]);
        }
        finish_row<T>(a, b, h, m, c, y, z, at);
      }
      cluster_sync();  // the others may still be reading
    }
    if (!more) break;
  }
  cp_wait<0>();
}

// Rows of a CTA: 8, 16, 32, 64 (float32: blocks of 64), or, in bfloat16, blocks of 128.
int block_rows(int rows, int dtype) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || dtype == MUSE_F32 ? 64 : kTcRows;
}

template <typename T, int D, int Dv, int NB, int RT>
cudaError_t launch(AttendArgs a, const CacheView &v, int *status, cudaStream_t st) {
  using C = Shape<T, D, Dv, NB, RT>;
  const auto kernel = attend<T, D, Dv, NB, RT>;
  // CTAs that a device holds at once, looked up with the kernel's attribute once a device
  static std::atomic<int> resident[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int fit = resident[dev].load(std::memory_order_acquire);
  if (!fit) {
    int sms = 0, per_sm = 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * kWarps, C::kSmem);
    if (e != cudaSuccess) return e;
    fit = std::max(1, std::min(kMaxCtas, sms * per_sm));
    resident[dev].store(fit, std::memory_order_release);
  }
  const int rows = a.G * a.M;
  a.nrb = (rows + C::kRows - 1) / C::kRows;
  a.block_log2 = C::kRows == 8 ? 3 : C::kRows == 16 ? 4 : C::kRows == 32 ? 5 : 6;
  a.min_tiles = C::kSlices;
  a.tile_log2 = 5;
  a.item_tiles = kItemTiles;
  const int64_t items = (int64_t)a.B * v.Hkv * a.nrb;
  const int64_t cap = ((int64_t)v.max_pages << v.page_log2) / kTile;  // tiles a sequence can have
  if (C::kClusters && cap <= (items * kCluster <= fit ? kClusterTiles<T> : kClusterTilesTwice) * C::kSlices &&
      items * kCluster <= 2 * fit) {
    a.cluster = (int)std::max<int64_t>(1, std::min<int64_t>(kCluster, (cap + C::kSlices - 1) / C::kSlices));
    return launch_next(kernel, dim3((unsigned)(items * a.cluster)), 32 * kWarps, C::kSmem, st,
                       true, a.cluster, a, v, status);
  }
  // no more CTAs than the table could hold stretches for
  const int ctas = (int)std::min<int64_t>(fit, (items * cap + a.min_tiles - 1) / a.min_tiles);
  e = launch_next(kernel, dim3(ctas), 32 * kWarps, C::kSmem, st, false, 0, a, v, status);
  if (e != cudaSuccess) return e;
  return launch_next(attend_join<T, Dv, C::kRows>, dim3(rows, v.Hkv, a.B), 128, 0, st, true, 0, a, v,
                     status);
}

template <typename T, int D, int Dv>
cudaError_t by_rows(const AttendArgs &a, const CacheView &v, int *status, cudaStream_t st) {
  switch (block_rows(a.G * a.M, sizeof(T) == 4 ? MUSE_F32 : MUSE_BF16)) {
    case 8: return launch<T, D, Dv, 1, 1>(a, v, status, st);
    case 16: return launch<T, D, Dv, 2, 1>(a, v, status, st);
    case 32: return launch<T, D, Dv, 2, 2>(a, v, status, st);
    case 64: return launch<T, D, Dv, 2, 4>(a, v, status, st);
    default: return launch_attend_tc<D, Dv>(a, v, status, st);
  }
}

// Partial sums and references of two parts a CTA, and the ends of every item.
struct AttendWs {
  size_t part, part_ml, ends;
  AttendWs(int64_t B, int64_t H, int64_t M, int64_t Dv, int64_t Hkv, int dtype) {
    const int64_t all = H / Hkv * M, rows = block_rows((int)std::min<int64_t>(all, 1 << 20), dtype);
    const int64_t slots = 2 * (rows == kTcRows ? kTcMaxCtas : kMaxCtas);
    part = align_up((size_t)(slots * rows * Dv * 4));
    part_ml = align_up((size_t)(slots * rows * 8));
    ends = align_up((size_t)(B * Hkv * ((all + rows - 1) / rows) * 8));
  }
};

template <typename T>
cudaError_t by_width(const AttendArgs &a, const muse_dims &d, const CacheView &v, int *status,
                     cudaStream_t st) {
  if (d.D == 64)
    return d.Dv == 64 ? by_rows<T, 64, 64>(a, v, status, st) : by_rows<T, 64, 128>(a, v, status, st);
  return d.Dv == 64 ? by_rows<T, 128, 64>(a, v, status, st) : by_rows<T, 128, 128>(a, v, status, st);
}

}  // namespace

size_t cache_attend_ws(const muse_dims &d, int Hkv) {
  const AttendWs w(d.B, d.H, d.N, d.Dv, Hkv, d.dtype);
  return w.part + w.part_ml + w.ends;
}

cudaError_t run_cache_attend(const muse_rows &Q, const muse_dims &d, const muse_cache &c,
                             const int32_t *lens, const int32_t *counts, const muse_rows &O,
                             float *lse, void *ws, int *status, cudaStream_t st) {
  AttendArgs a;
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.lens = lens;
  a.counts = counts;
  a.B = d.B;
  a.H = d.H;
  a.M = d.N;
  a.G = d.H / c.Hkv;
  a.nrb = a.block_log2 = a.min_tiles = a.tile_log2 = a.item_tiles = a.cluster = 0;
  a.scale = d.scale;
  const AttendWs w(d.B, d.H, d.N, d.Dv, c.Hkv, d.dtype);
  char *p = static_cast<char *>(ws);
  a.part = reinterpret_cast<float *>(p);
  a.part_ml = reinterpret_cast<float *>(p + w.part);
  a.ends = reinterpret_cast<int2 *>(p + w.part + w.part_ml);
  const CacheView v = cache_view(c);
  return d.dtype == MUSE_F32 ? by_width<float>(a, d, v, status, st)
                             : by_width<__nv_bfloat16>(a, d, v, status, st);
}

}  // namespace muse
