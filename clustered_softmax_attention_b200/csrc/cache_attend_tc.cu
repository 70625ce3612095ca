// Causal attention over the 4-bit cache for many rows of a cache head (the chunk of a prompt, many
// drafted tokens): more than 64 bfloat16 rows, 128 at a time, on tcgen05.
//
// With that many rows the products bound it, not the cache's bytes, and a code is dequantised once
// for 128 rows into shared memory instead of into every warp's registers.  Per tile of 128 tokens:
//   producers (8 warps)  codes -> float16 K' and V' in 128-byte swizzled shared memory, two stages;
//   issuer               S = Q K'^T into TMEM (two buffers), O += P V' with P from TMEM;
//   softmax (4 warps)    a row a thread: S from TMEM, weights over it, O in TMEM moved only
//                        when the running reference moves.
// S of the next tile is issued before O += P V' of this one, so the softmax of one tile runs
// beside both products.
//   K' = code step 2^(12 - e), e the exponent of the largest step of sixteen tokens: exact for
//   steps down to 2^-26 of that; 2^(e - 12) multiplies their columns of S.  With a smaller step (zero
//   apart) the softmax warps form the sixteen tokens' logits in float32 from the codes.
//   V' = code step unit[group], a power of two that the group's first tile of the span that is not all
//   zeros sets by its usual largest step: exact for steps from 2^-17 to 2^9 of that.  Sixteen tokens with
//   a step outside of it (zero apart) have V' = 0, and the softmax warps add p v to O in float32 from
//   the codes.
// The order of channels inside K' and V' is the one in which a word's codes come out, two nibbles
// four apart a register; Q is laid out alike, and the output's columns are put back at the end.
//
// Two sequences, two cache heads of four query heads, 128 new rows (512 rows a cache head), 128 + 128
// channels: 64 to 68 us over 16384 tokens, of which about 25 are a call's beginning and end; from there
// 19 ns a tile of 128 x 128 (2.9 us an SM), 434 TFLOP/s of 1640: the three products (two of weights) are
// 1.1 of those 2.9 us, and the way of a tile through the three roles is the rest (ALU 25 %, tensor pipe
// 18 %, no unit is busy; stalls: loads, and instructions that are not there yet).
// The other form against this one, us behind a flushed L2, 64 rows a cache head and fewer, then more:
//   8 x 8 heads, 1024 tokens:    36 rows 44 and 56, 64 rows 48 and 58; 68 rows 67 and 58, 512 rows 185 and 128
//   2 x 2 heads, 16384 tokens:   36 rows 38 and 46, 64 rows 40 and 46; 68 rows 52 and 46, 512 rows 134 and 79
//   8 x 8 heads, 16384 tokens:   36 rows 243 and 204, 64 rows 247 and 206; 68 rows 463 and 208, 512 rows 1755 and 707
//   2 x 2 heads, 1024 tokens:    36 rows 21 and 30, 64 rows 21 and 30; 68 rows 22 and 30, 512 rows 32 and 40
#include <atomic>

#include "cache_attend.cuh"
#include "tc_ptx.cuh"

namespace muse {
namespace {

using namespace ptx;

constexpr int kTok = 128;               // tokens of a tile
constexpr int kSoftmaxWarps = 4, kProducers = 8, kIssuer = kSoftmaxWarps + kProducers;
constexpr int kThreads = 32 * (kIssuer + 1);
constexpr uint32_t kTmemCols = 512;
constexpr int kGone = 1;    // not in the cache
constexpr int kValues = 2;  // value steps that V' does not hold: it holds zeros
constexpr int kKeys = 4;    // key steps that K' does not hold
// TMEM columns: S (two of 128), O.  A weight takes the place of its S as two float16 pieces, 21 bits:
// sixteen tokens' columns hold eight of upper and eight of lower pieces.  In one piece (11 bits) results
// differed from float32 arithmetic's by 9e-4 in norm, in two by 1.6e-4.  One piece and two, 128 + 128
// channels: 2 x 2 heads of 16384 tokens, 512 rows a head, 55 and 64 us; 8 x 8 heads, 68 rows, 170 and 204
// (the second products take about 12 of the 34, the pieces and their stores the rest).
constexpr uint32_t kS = 0, kO = 256;

template <int D, int Dv>
struct __align__(1024) Smem {
  __half q[D / 64][kTcRows * 64];
  __half k[2][D / 64][kTok * 64];
  __half v[2][Dv / 64][kTok * 64];
  // a producer's sixteen tokens as they are held: key codes, value codes, key steps, value steps
  uint8_t raw[kProducers][2][9 * (D + Dv)];
  float scale[2][kProducers]; // what sixteen tokens' columns of S are multiplied by
  float unit[4][Dv / 32];     // by span
  alignas(4) uint16_t big[2][kProducers][Dv / 32];  // by exchange
  int exps[kTcRows];          // of the queries' powers of two
  float tokens[kSoftmaxWarps][16 * 16];  // sixteen tokens' keys or values, sixteen channels at a time
  alignas(8) uint8_t odd[2][kProducers];  // kGone, kValues, kKeys: what holds of sixteen tokens
  int64_t run[kThreads + kThreads / 32];
  uint64_t q_full, unit_full, kv_full[2], kv_empty[2], s_full[2], p_full[2], end;
  uint32_t tmem_base;
  int abort_flag;
};

// Instruction descriptor: float16 operands, float32 accumulators.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: 64 channels of a token a row, blocks of 64 channels 16 KB
// apart.
__device__ __forceinline__ uint64_t sdesc_mn(const void *p) {
  const uint32_t a = saddr(p);
  uint64_t d = 0;
  d |= (uint64_t)((a & 0x3FFFFu) >> 4);
  d |= (uint64_t)((16384u >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void async_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Waits for this thread's TMEM loads; x, the last of them, is not used before.
__device__ __forceinline__ void arrived(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]),
                 "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]),
                 "+r"(x[13]), "+r"(x[14]), "+r"(x[15])
               :
               : "memory");
}
__device__ __forceinline__ __half2 halves(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
// x and y as two float16 each, 21 bits: the upper pieces (cut to 11 bits) packed, the lower ones packed.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo) {
  const float a = __uint_as_float(__float_as_uint(x) & 0xffffe000u);
  const float b = __uint_as_float(__float_as_uint(y) & 0xffffe000u);
  hi = pack_f16(a, b);
  lo = pack_f16(x - a, y - b);
}
// The 16-byte chunk c of a 128-byte row.
__device__ __forceinline__ uint4 *chunk(__half *block, int row, int c) {
  return reinterpret_cast<uint4 *>(reinterpret_cast<char *>(block) + row * 128 + ((c ^ (row & 7)) << 4));
}
// Column of O (within 64) that holds channel c of 64.
__host__ __device__ constexpr int column_of(int c) {
  return 8 * (c % 8) + (c / 8 < 4 ? 2 * (c / 8) : 2 * (c / 8 - 4) + 1);
}

// The columns of S of sixteen tokens whose key steps K' does not hold, in float32 from the codes: a row a
// thread, `q` its block of queries.  `p`: their tile of 32 tokens, whose half `part` they are; `scale`: what
// the columns are multiplied by.  Small rather than fast (16 us), as exact_values.
template <int D>
__device__ __noinline__ void exact_logits(uint32_t columns, __half (*q)[kTcRows * 64], const uint8_t *p,
                                          const uint16_t *steps, int part, float scale, float *tokens) {
  const int lane = threadIdx.x & 31, t0 = 16 * part + (lane >> 1), e = -ilogbf(scale);
  const uint32_t *kw = reinterpret_cast<const uint32_t *>(p);
#pragma unroll 1
  for (int j = 0; j < D / 16; ++j) {
    // a lane a token and one of its words, the channels in the queries' order
    const uint32_t word = kw[key_word<D>(t0, 2 * (j & 1) + (lane & 1), j >> 1)];
    const float f = ldexpf(step_value(steps[t0 * (D / 32) + (j >> 1)]), e);
    float y[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) y[2 * (n & 3) + (n >> 2)] = code_value(word, n) * f;
    __syncwarp();  // the last channels have been read
    float4 *to = reinterpret_cast<float4 *>(tokens + (lane >> 1) * 16 + (lane & 1) * 8);
    to[0] = make_float4(y[0], y[1], y[2], y[3]);
    to[1] = make_float4(y[4], y[5], y[6], y[7]);
    __syncwarp();
    float x[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = *chunk(q[j >> 2], threadIdx.x, (2 * j + h) & 7);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 z = __half22float2(halves(w[k]));
        x[8 * h + 2 * k] = z.x;
        x[8 * h + 2 * k + 1] = z.y;
      }
    }
#pragma unroll 1
    for (int t = 0; t < 16; ++t) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(tokens + t * 16 + c);
        s = fmaf(x[c], k.x, fmaf(x[c + 1], k.y, fmaf(x[c + 2], k.z, fmaf(x[c + 3], k.w, s))));
      }
      if (j) s += tmem_ld1(columns + t);
      tmem_st1(columns + t, s);
    }
    tmem_st_wait();
  }
}

// O += p v of sixteen tokens whose value steps V' does not hold, in float32 from the codes: a row a
// thread.  `logits`: their columns of S; `left`: tokens of them that the row sees; `p`: their tile of 32
// tokens, whose half `part` they are; begin: O holds nothing yet.  Small rather than fast (7 us): a cold
// kernel waits for its instructions.
template <int D, int Dv>
__device__ __noinline__ void exact_values(uint32_t logits, float to2, float ref, int left, const uint8_t *p,
                                          int part, const float *unit, uint32_t o_at, float *tokens,
                                          bool begin) {
  using S = TileShape<D, Dv>;
  const int lane = threadIdx.x & 31, t0 = 16 * part + (lane >> 1);
  const uint32_t *vw = reinterpret_cast<const uint32_t *>(p + S::kV);
  const uint16_t *vs = reinterpret_cast<const uint16_t *>(p + S::kVStep) + t0 * (Dv / 32);
#pragma unroll 1
  for (int j = 0; j < Dv / 16; ++j) {
    // a lane a token and one of its words: channels g + 8 (0..7) of 64, in the order of the columns
    const uint32_t word = vw[value_word<Dv>(t0, 2 * (j & 3) + (lane & 1), j >> 2)];
    const int grp = 2 * (j >> 2);
    const float f[2] = {step_value(vs[grp]) * unit[grp], step_value(vs[grp + 1]) * unit[grp + 1]};
    float y[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) y[2 * (n & 3) + (n >> 2)] = code_value(word, n) * f[n >> 2];
    __syncwarp();  // the last columns' values have been read
    float4 *to = reinterpret_cast<float4 *>(tokens + (lane >> 1) * 16 + (lane & 1) * 8);
    to[0] = make_float4(y[0], y[1], y[2], y[3]);
    to[1] = make_float4(y[4], y[5], y[6], y[7]);
    __syncwarp();
    float o[16];
    tmem_ld16(o_at + j * 16, o);
    if (begin) {
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = 0.f;
    }
#pragma unroll 1
    for (int t = 0; t < 16; ++t) {
      const float w = ex2(__fmul_rn(tmem_ld1(logits + t), to2) - ref);
      if (t < left) {  // whatever others hold
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(tokens + t * 16 + e);
          o[e] = fmaf(w, x.x, o[e]);
          o[e + 1] = fmaf(w, x.y, o[e + 1]);
          o[e + 2] = fmaf(w, x.z, o[e + 2]);
          o[e + 3] = fmaf(w, x.w, o[e + 3]);
        }
      }
      __syncwarp();
    }
    uint32_t u[2][8];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e >> 3][e & 7] = __float_as_uint(o[e]);
    tmem_st8(o_at + j * 16, u[0]);
    tmem_st8(o_at + j * 16 + 8, u[1]);
  }
  tmem_st_wait();
}

template <int D, int Dv>
__global__ void __launch_bounds__(kThreads, 1)
attend_tc(const __grid_constant__ AttendArgs a, const __grid_constant__ CacheView v, int *status) {
  using S = TileShape<D, Dv>;
  constexpr int NGk = D / 32, NG = Dv / 32;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  Smem<D, Dv> &sm = *reinterpret_cast<Smem<D, Dv> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  volatile int *abort_flag = &sm.abort_flag;
  dependents_may_launch();
  wait_for_earlier();

  Walk walk;
  Span sp;
  int64_t per;
  if (!line_start<kThreads>(a, v, sm.run, walk, per)) return;
  if (!next_span(a, v, walk, sp, per)) return;

  if (tid == 0) {
    mbar_init(&sm.q_full, 128);
    mbar_init(&sm.unit_full, 32 * kProducers);
    mbar_init(&sm.end, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kv_full[i], 32 * kProducers);
      mbar_init(&sm.kv_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
    }
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    __syncwarp();  // lane 0 has set up the barriers
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  uint32_t it = 0;  // tiles so far, in every role alike
  // a wait that gives up ends the warp's role; the others end at their own next wait
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t phase) {
    ok = __all_sync(kAll, mbar_wait<true>(bar, phase & 1, abort_flag, status));
    return ok;
  };

  if (warp >= kSoftmaxWarps && warp < kIssuer) {
    // ------------------------------------------------------------ codes -> float16 operands
    const int pw = warp - kSoftmaxWarps;  // tokens 16 pw .. 16 pw + 15 of a tile
    constexpr int kRV = 8 * D, kRKS = 8 * (D + Dv), kRVS = kRKS + D;
    uint32_t shift[Dv / 64];
    uint32_t open = 0;       // groups that have no unit yet, in every producer alike
    uint32_t exchanges = 0;
    // (test hook: the first sixteen tokens of a tile are never handed on, so the waits for them run out)
    const bool withhold = pw == 0 && (test_hooks(status) & MUSE_TEST_WITHHOLD_CACHE);
    // the tile after the one at hand is under way: raw[it & 1] holds tile it
    bool next_here = false;
    auto fetch = [&](const Span &s, int t, uint32_t slot) {
      const int tile = 4 * t + (pw >> 1), part = pw & 1;
      const uint8_t *p = nullptr;
      if (tile * 32 + 16 * part < s.len) {
        p = cache_tile(v, s.b, s.hk, tile, S::kBytes);
        if (!p && lane == 0) report(status, MUSE_ERR_DEVICE);
      }
      if (p) {
        uint8_t *to = sm.raw[pw][slot & 1];
#pragma unroll
        for (int i = 0; i < D / 2; i += 32)
          cp_async16(to + (i + lane) * 16, p + S::kK + part * 8 * D + (i + lane) * 16, 16);
#pragma unroll
        for (int i = 0; i < Dv / 2; i += 32)
          cp_async16(to + kRV + (i + lane) * 16, p + S::kV + part * 8 * Dv + (i + lane) * 16, 16);
        if (lane < D / 16) cp_async16(to + kRKS + lane * 16, p + S::kKStep + part * D + lane * 16, 16);
        else if (lane >= 16 && lane < 16 + Dv / 16)
          cp_async16(to + kRVS + (lane - 16) * 16, p + S::kVStep + part * Dv + (lane - 16) * 16, 16);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      next_here = p != nullptr;
    };
    fetch(sp, sp.t0, 0);
    bool more = true;
    for (int span = 1; more && ok; ++span) {
      const Span cur = sp;
      more = next_span(a, v, walk, sp, per);
      for (int t = cur.t0; t < cur.t1 && ok; ++t, ++it) {
        const uint32_t st = it & 1;
        const int base = t * kTok + pw * 16;
        const bool here = next_here;
        if (t + 1 < cur.t1) fetch(cur, t + 1, it + 1);
        else if (more) fetch(sp, sp.t0, it + 1);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const uint8_t *raw = sm.raw[pw][st];
        const int n = here ? min(16, cur.len - base) : 0;  // its tokens
        if (t == cur.t0) {
          open = (1u << NG) - 1;
#pragma unroll
          for (int w = 0; w < Dv / 64; ++w) shift[w] = 0;
          if (pw == 0 && lane < NG) sm.unit[span & 3][lane] = 1.f;
        }
        if (open) {
          // The values' unit: in the group's first tile that has a step above zero, the largest of each
          // sixteen tokens, and of these the median, comes to [2^3, 2^4): neither a few large values nor
          // a few small ones put the others out of range.  Before that tile the group adds nothing to
          // O, and any unit is right.
#pragma unroll
          for (int w = 0; w < Dv / 64; ++w) {
            // a lane a token; NaN is negative here, and left out
            uint32_t top = lane < n ? __vmaxs2(0u, reinterpret_cast<const uint32_t *>(raw + kRVS)[lane * (Dv / 64) + w]) : 0u;
#pragma unroll
            for (int o = 8; o; o >>= 1) top = __vmaxs2(top, __shfl_xor_sync(kAll, top, o));
            if (lane == 0) reinterpret_cast<uint32_t *>(sm.big[exchanges & 1][pw])[w] = top;
          }
          mbar_arrive(&sm.unit_full);
          if (!wait(&sm.unit_full, exchanges)) break;
          // a lane a group and sixteen tokens: the place of its largest among those above zero
          const uint32_t mine = lane < NG * kProducers ? sm.big[exchanges & 1][lane / NG][lane % NG] : 0u;
          uint32_t many = 0, below = 0;
#pragma unroll 1
          for (int k = 0; k < kProducers; ++k) {
            const uint32_t x = __shfl_sync(kAll, mine, k * NG + lane % NG);
            many += x > 0;
            below += x > 0 && (x < mine || (x == mine && k < lane / NG));
          }
          uint32_t median = mine > 0 && below == (many - 1) / 2 ? mine : 0u;
#pragma unroll
          for (int o = NG; o < 32; o <<= 1) median = max(median, __shfl_xor_sync(kAll, median, o));
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
            const uint32_t step = __shfl_sync(kAll, median, grp);
            if (!step || !((open >> grp) & 1)) continue;
            open &= ~(1u << grp);
            const int ex = min(max((int)(step >> 7) - 127, -40), 60);
            // float16's exponent is 112 less than bfloat16's
            shift[grp >> 1] += (uint32_t)((3 - ex - 112) * 128) << (16 * (grp & 1));
            if (pw == 0 && lane == 0) sm.unit[span & 3][grp] = ldexpf(1.f, 3 - ex);
          }
          ++exchanges;
        }
        if (it >= 2 && !wait(&sm.kv_empty[st], (it - 2) >> 1)) break;
        // ---- steps as float16.  Keys: the sixteen tokens' largest (a NaN is left out: it makes its
        // token NaN) comes to exponent field 27; values: by the span's unit.
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < NGk / 2; ++w)
          if (lane < n) top = __vmaxs2(top, reinterpret_cast<const uint32_t *>(raw + kRKS)[lane * (NGk / 2) + w]);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
        const int e_top = (int)(__shfl_sync(kAll, top, 0) >> 7);
        if (lane == 0) sm.scale[st][pw] = ldexpf(1.f, e_top - 127 - 12);
        const uint32_t k_shift = (uint32_t)((27 - e_top) * 128) * 0x10001u;
        uint32_t ks[2][NGk / 2], vs[2][2][Dv / 64], off_range = 0;
        int odd = !here && base < cur.len ? kGone : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (D == 128) {
            const uint2 y = reinterpret_cast<const uint2 *>(raw + kRKS)[8 * i + g];
            ks[i][0] = y.x;
            ks[i][NGk / 2 - 1] = y.y;
          } else {
            ks[i][0] = reinterpret_cast<const uint32_t *>(raw + kRKS)[8 * i + g];
          }
          if (Dv == 128) {
            const uint4 y = reinterpret_cast<const uint4 *>(raw + kRVS)[4 * i + q];
            vs[i][0][0] = y.x;
            vs[i][0][Dv / 64 - 1] = y.y;
            vs[i][1][0] = y.z;
            vs[i][1][Dv / 64 - 1] = y.w;
          } else {
            const uint2 y = reinterpret_cast<const uint2 *>(raw + kRVS)[4 * i + q];
            vs[i][0][0] = y.x;
            vs[i][1][0] = y.y;
          }
          // fields 12..27 of keys, 8..23 of values (18: the first tile's usual largest).  Also the careful
          // way go n < 16, for the tokens that are not there, and keys so small (e_top < 16) that the shift
          // would bring steps without an exponent, or a NaN (0xffff), into range.
#pragma unroll
          for (int w = 0; w < NGk / 2; ++w) off_range |= ks[i][w] + k_shift - 0x06000600u;
#pragma unroll
          for (int w = 0; w < Dv / 64; ++w)
            off_range |= (vs[i][0][w] + shift[w] - 0x04000400u) | (vs[i][1][w] + shift[w] - 0x04000400u);
        }
        if (__builtin_expect(!__any_sync(kAll, (off_range & 0xf800f800u) != 0) && n >= 16 && e_top >= 16, 1)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int w = 0; w < NGk / 2; ++w) ks[i][w] = (ks[i][w] + k_shift) << 3;
#pragma unroll
            for (int w = 0; w < Dv / 64; ++w) {
              vs[i][0][w] = (vs[i][0][w] + shift[w]) << 3;
              vs[i][1][w] = (vs[i][1][w] + shift[w]) << 3;
            }
          }
        } else {
          // half by half: tokens that are not there and zero steps are zero, a key's NaN is NaN; with a value
          // step that float16 does not hold all values are zero here
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            auto careful = [&](uint32_t x, uint32_t by, bool live, bool value) {
              uint32_t d = 0;
              const int low = (short)(by & 0xffffu), high = (short)((by - (uint32_t)low) >> 16);
              for (int k = 0; k < 2; ++k) {
                const int s = (int)((x >> (16 * k)) & 0xffffu), f = s + (k ? high : low);
                if (!live || s == 0) continue;
                if (value && (s >= 0x7f80 || s < 128 || f < 128 || f >= 28 * 128)) odd |= kValues;
                else if (s >= 0x7f80) d |= 0x7e00u << (16 * k);
                else if (s < 128 || f < 128) odd |= kKeys;  // (of values: above)
                else d |= (uint32_t)(f << 3) << (16 * k);
              }
              return d;
            };
            for (int w = 0; w < NGk / 2; ++w) {
              const uint32_t d = careful(i ? ks[1][w] : ks[0][w], k_shift, 8 * i + g < n, false);
              (i ? ks[1][w] : ks[0][w]) = d;
            }
            for (int e = 0; e < 2; ++e)
              for (int w = 0; w < Dv / 64; ++w) {
                const uint32_t d = careful(i ? vs[1][e][w] : vs[0][e][w], shift[w], 8 * i + 2 * q + e < n, true);
                (i ? vs[1][e][w] : vs[0][e][w]) = d;
              }
          }
          odd = __reduce_or_sync(kAll, odd);
          if (odd & kValues) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int w = 0; w < Dv / 64; ++w) vs[i][0][w] = vs[i][1][w] = 0;
          }
        }
        if (lane == 0) sm.odd[st][pw] = (uint8_t)odd;
        // ---- codes: keys to row 8 i + g, chunk (w % 2) 4 + q; values to rows 8 i + 2 q + e, chunk g
        char *k_to = reinterpret_cast<char *>(sm.k[st][0]) + (pw * 16 + g) * 128;
        char *v_to = reinterpret_cast<char *>(sm.v[st][0]) + (pw * 16 + 2 * q) * 128;
        auto put = [&](char *to, uint32_t word, __half2 step) {
          uint32_t c[4];
          codes_f16(word, c);
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = bits(__hmul2(*reinterpret_cast<__half2 *>(&c[k]), step));
          *reinterpret_cast<uint4 *>(to) = make_uint4(c[0], c[1], c[2], c[3]);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t kw[NGk], vw[2][Dv / 64];
          if (D == 128) {
            const uint4 x = reinterpret_cast<const uint4 *>(raw)[i * 32 + lane];
            kw[0] = x.x;
            kw[1] = x.y;
            kw[NGk - 2] = x.z;
            kw[NGk - 1] = x.w;
          } else {
            const uint2 x = reinterpret_cast<const uint2 *>(raw)[lane * 2 + i];
            kw[0] = x.x;
            kw[1] = x.y;
          }
          if (Dv == 128) {
            const uint4 x = reinterpret_cast<const uint4 *>(raw + kRV)[i * 32 + lane];
            vw[0][0] = x.x;
            vw[0][Dv / 64 - 1] = x.y;
            vw[1][0] = x.z;
            vw[1][Dv / 64 - 1] = x.w;
          } else {
            const uint2 x = reinterpret_cast<const uint2 *>(raw + kRV)[lane * 2 + i];
            vw[0][0] = x.x;
            vw[1][0] = x.y;
          }
#pragma unroll
          for (int w = 0; w < NGk; ++w) {
            const __half2 two = *reinterpret_cast<__half2 *>(&ks[i][w >> 1]);
            put(k_to + (w >> 1) * (kTok * 128) + i * 1024 + ((((w & 1) * 4 + q) ^ g) << 4), kw[w],
                w & 1 ? __high2half2(two) : __low2half2(two));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < Dv / 64; ++w)  // a step for nibbles 0..3, one for 4..7
              put(v_to + w * (kTok * 128) + i * 1024 + e * 128 + ((g ^ (2 * q + e)) << 4), vw[e][w],
                  *reinterpret_cast<__half2 *>(&vs[i][e][w]));
        }
        async_fence();
        __syncwarp();  // all lanes have read raw[st]: the next fetch writes there
        if (!withhold) mbar_arrive(&sm.kv_full[st]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products
    bool more = true;
    for (int span = 1; more && ok; ++span) {
      const int n = sp.t1 - sp.t0;
      more = next_span(a, v, walk, sp, per);
      const uint32_t it0 = it;
      if (!wait(&sm.q_full, span - 1)) break;
      auto values = [&](uint32_t u) {  // O += P V' of tile u
        if (!wait(&sm.p_full[u & 1], u >> 1)) return;
        tc_fence_after();
        // O begins with the first tile's products, or with what the softmax warps have put there
        const uint2 odd = *reinterpret_cast<const uint2 *>(sm.odd[u & 1]);
        const bool begun = u > it0 || ((odd.x | odd.y) & (0x01010101u * kValues));
        if (lane == 0) {
          constexpr uint32_t id = idesc_f16(kTcRows, Dv) | (1u << 16);
          for (int kk = 0; kk < kTok / 16; ++kk) {
            const uint32_t p = tmem + kS + (u & 1) * 128 + kk * 16;
            const uint64_t rows = sdesc_mn(sm.v[u & 1][0] + kk * 16 * 64);
            tc_mma_ts(tmem + kO, p, rows, id, begun || kk > 0 ? 1u : 0u);
            tc_mma_ts(tmem + kO, p + 8, rows, id, 1u);
          }
          tc_commit(&sm.kv_empty[u & 1]);
        }
        __syncwarp();
      };
      for (int i = 0; i < n && ok; ++i, ++it) {
        if (!wait(&sm.kv_full[it & 1], it >> 1)) break;
        tc_fence_after();
        if (lane == 0) {
          constexpr uint32_t id = idesc_f16(kTcRows, kTok);
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma(tmem + kS + (it & 1) * 128, sdesc(sm.q[kk / 4] + (kk % 4) * 16),
                   sdesc(sm.k[it & 1][kk / 4] + (kk % 4) * 16), id, kk > 0 ? 1u : 0u);
          tc_commit(&sm.s_full[it & 1]);
        }
        __syncwarp();
        if (i) values(it - 1);
      }
      if (ok) values(it - 1);
    }
  } else {
    // ------------------------------------------------------------ softmax: row tid
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    bool more = true;
    for (int span = 1; more && ok; ++span) {
      const Span cur = sp;
      more = next_span(a, v, walk, sp, per);
      const int gr = cur.rb * kTcRows + tid;
      const int m = gr / a.G, h = cur.hk * a.G + (gr - m * a.G);
      const bool live = m < cur.rows;
      // a place without a row sees all, so that it masks nothing for its warp (it is not written)
      const int see = live ? min(max(cur.len - cur.rows + m + 1, 0), cur.len) : cur.len;
      int see_all = see;
#pragma unroll
      for (int x = 16; x; x >>= 1) see_all = min(see_all, __shfl_xor_sync(kAll, see_all, x));
      // ---- the queries as float16, a power of two a row: its largest in [2^14, 2^15).  A warp's 32
      // rows, eight channels a lane at a time.
      {
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int j = lane % kLanes;
        uint4 all[32 / kAtOnce];
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i) {
          const int gr2 = cur.rb * kTcRows + warp * 32 + i * kAtOnce + lane / kLanes;
          const int m2 = gr2 / a.G, h2 = cur.hk * a.G + (gr2 - m2 * a.G);
          all[i] = make_uint4(0, 0, 0, 0);
          if (m2 < cur.rows)
            all[i] = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.Q.p + cur.b * a.Q.sb +
                                                     h2 * a.Q.sh + m2 * a.Q.sn)[j];
        }
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i) {
          const int r = warp * 32 + i * kAtOnce + lane / kLanes;
          const uint4 x = all[i];
          uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                  __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          top = max(top << 16, top & 0xffff0000u);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
          const int e = min(max((int)(top >> 23) - 127 - 14, -114), 113);
          const float up = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, a normal number
          const float mul = top >= 0x7f800000u ? CUDART_NAN_F : a.scale < 0.f ? -up : up;
          if (j == 0) sm.exps[r] = e;
          // channels (0, 4), (1, 5), (2, 6), (3, 7) of eight
          *chunk(sm.q[j / 8], r, j % 8) =
              make_uint4(pack_f16(lo_f(x.x) * mul, lo_f(x.z) * mul), pack_f16(hi_f(x.x) * mul, hi_f(x.z) * mul),
                         pack_f16(lo_f(x.y) * mul, lo_f(x.w) * mul), pack_f16(hi_f(x.y) * mul, hi_f(x.w) * mul));
        }
        __syncwarp();
      }
      const float rf = ldexpf(fabsf(a.scale) * 1.44269504f, sm.exps[tid]);
      async_fence();
      mbar_arrive(&sm.q_full);

      float mx = -CUDART_INF_F, l = 0.f;
      bool far = false;  // of any row of the warp
      const uint32_t it0 = it;
      for (int t = cur.t0; t < cur.t1 && ok; ++t, ++it) {
        const uint32_t st = it & 1, col = tmem + lane_base + kS + st * 128;
        if (!wait(&sm.kv_full[st], it >> 1) || !wait(&sm.s_full[st], it >> 1)) break;
        tc_fence_after();
        const int left = see - t * kTok;
        const uint2 odd = *reinterpret_cast<const uint2 *>(sm.odd[st]);
        auto is = [&](int c, uint32_t what) { return ((c < 4 ? odd.x : odd.y) >> (8 * (c & 3))) & what; };
        const bool edge = see_all - t * kTok < kTok || ((odd.x | odd.y) & (0x01010101u * kGone));
        // to logits in units of log 2; above zero, so that what is hidden stays -infinity
        auto to2 = [&](int c) { return fmaxf(sm.scale[st][c] * rf, 1e-45f); };
        float sums[2] = {0.f, 0.f};
        // The reference moves: what was summed and weighed by it, the tile's first `done` chunks of
        // weights among them, is brought to the new one.
        auto move = [&](float top, int done) {
          const float now = fmaxf(mx, __fsub_ru(top, 9.f));
          const float fix = now == -CUDART_INF_F ? 1.f : ex2(mx - now);
          mx = now;
          far = __any_sync(kAll, fabsf(now) > kFar && now != -CUDART_INF_F);
          l *= fix;
          sums[0] *= fix;
          sums[1] *= fix;
          if (it > it0) {
            if (!wait(&sm.kv_empty[(it - 1) & 1], (it - 1) >> 1)) return;  // O holds all tiles so far
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < Dv / 16; ++c) {
              float o[16];
              uint32_t w[2][8];
              tmem_ld16(tmem + lane_base + kO + c * 16, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e >> 3][e & 7] = __float_as_uint(o[e] * fix);
              tmem_st8(tmem + lane_base + kO + c * 16, w[0]);
              tmem_st8(tmem + lane_base + kO + c * 16 + 8, w[1]);
            }
          }
          tmem_st_wait();
#pragma unroll 1
          for (int c = 0; c < done; ++c) {
            float o[16];
            uint32_t hi[8], lo[8];
            tmem_ld16(col + c * 16, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 u = __half22float2(halves(__float_as_uint(o[e])));
              const float2 v = __half22float2(halves(__float_as_uint(o[8 + e])));
              split_f16((u.x + v.x) * fix, (u.y + v.y) * fix, hi[e], lo[e]);
            }
            tmem_st8(col + c * 16, hi);
            tmem_st8(col + c * 16 + 8, lo);
          }
        };
        // The largest logit of two chunks of sixteen columns.  Weights are 2^9 at the reference, which
        // moves when one would pass 2^14 (in the first tile, a few more).
        auto top_of = [&](int c, const uint32_t (&x)[2][16]) {
          float top = -CUDART_INF_F;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              m[e] = fmaxf(fmaxf(__uint_as_float(x[k][e]), __uint_as_float(x[k][e + 4])),
                           fmaxf(__uint_as_float(x[k][e + 8]), __uint_as_float(x[k][e + 12])));
            top = fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * to2(c + k));
          }
          return top;
        };
        auto weigh = [&](int c, const uint32_t (&x)[2][16], bool scaled) {
          const float ref = mx == -CUDART_INF_F ? 0.f : mx;
          uint32_t w[32];  // the two chunks' upper and lower pieces
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float f = scaled ? 1.f : to2(c + k);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float p0 = ex2(fmaf(__uint_as_float(x[k][e]), f, -ref));
              const float p1 = ex2(fmaf(__uint_as_float(x[k][e + 1]), f, -ref));
              sums[(e >> 1) & 1] += p0 + p1;
              split_f16(p0, p1, w[16 * k + (e >> 1)], w[16 * k + 8 + (e >> 1)]);
            }
          }
          tmem_st32(col + c * 16, w);
        };
        if (__builtin_expect((odd.x | odd.y) & (0x01010101u * kKeys), 0)) {
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const uint8_t *p = is(k, kKeys) ? cache_tile(v, cur.b, cur.hk, 4 * t + (k >> 1), S::kBytes) : nullptr;
            if (p)
              exact_logits<D>(col + k * 16, sm.q, p, reinterpret_cast<const uint16_t *>(p + S::kKStep), k & 1,
                              sm.scale[st][k], sm.tokens[warp]);
          }
        }
        const bool values = (odd.x | odd.y) & (0x01010101u * kValues);
        // Most tiles: nothing hidden, nothing odd, and the reference stays.  Chunks from `begun` on are left
        // to the loop below, which does everything and is kept small.
        int begun = values ? -8 : 0;
        if (__builtin_expect(!(edge || values || far), 1)) {
          uint32_t x[2][2][16];
          tmem_ld16_async(col, x[0][0]);
          tmem_ld16_async(col + 16, x[0][1]);
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            const int k = (c >> 1) & 1;
            arrived(x[k][0]);
            arrived(x[k][1]);
            if (__any_sync(kAll, top_of(c, x[k]) - mx > 14.f)) break;
            if (c < 6) {
              tmem_ld16_async(col + (c + 2) * 16, x[k ^ 1][0]);
              tmem_ld16_async(col + (c + 3) * 16, x[k ^ 1][1]);
            }
            weigh(c, x[k], false);
            begun = c + 2;
          }
        }
        // where V' does not hold all values: the reference for the whole tile first (c below 0), and
        // these tokens' values by their logits
        float all = -CUDART_INF_F;
#pragma unroll 1
        for (int c = begun; c < 8; c += 2) {
          if (c == 0 && values) {
            if (__any_sync(kAll, all - mx > 14.f)) move(all, 0);
            if (it > it0 && ok) {
              wait(&sm.kv_empty[(it - 1) & 1], (it - 1) >> 1);
              tc_fence_after();
            }
            bool begin = it == it0;
#pragma unroll 1
            for (int k = 0; k < 8 && ok; ++k) {
              if (!is(k, kValues)) continue;
              const uint8_t *p = cache_tile(v, cur.b, cur.hk, 4 * t + (k >> 1), S::kBytes);
              if (!p) continue;
              exact_values<D, Dv>(col + k * 16, to2(k), mx == -CUDART_INF_F ? 0.f : mx, left - 16 * k, p,
                                  k & 1, sm.unit[span & 3], tmem + lane_base + kO, sm.tokens[warp], begin);
              begin = false;
            }
          }
          if (!ok) break;
          uint32_t x[2][16];
          tmem_ld16_async(col + (c & 7) * 16, x[0]);
          tmem_ld16_async(col + (c & 7) * 16 + 16, x[1]);
          arrived(x[0]);
          arrived(x[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = is((c & 7) + k, kGone) ? 0 : left - 16 * ((c & 7) + k);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e >= n) x[k][e] = 0xff800000u;  // -infinity
          }
          const float top = top_of(c & 7, x);
          all = fmaxf(all, top);
          if (c < 0) continue;
          if (__any_sync(kAll, top - mx > 14.f)) move(top, c);
          if (far) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                x[k][e] = __float_as_uint(__fmul_rn(__uint_as_float(x[k][e]), to2(c + k)));
          }
          weigh(c, x, far);
        }
        tmem_st_wait();
        if (!ok) break;
        l += sums[0] + sums[1];
        tc_fence_before();
        mbar_arrive(&sm.p_full[st]);
      }
      if (!ok) break;
      // ---- the span's sums
      if (!wait(&sm.kv_empty[(it - 1) & 1], (it - 1) >> 1)) break;
      tc_fence_after();
      const bool whole = cur.t0 == 0 && cur.t1 == cur.nt;
      const int slot = 2 * blockIdx.x + (span > 1 ? 1 : 0);
      if (cur.t0 == 0 && tid == 0)
        a.ends[((int64_t)cur.b * v.Hkv + cur.hk) * a.nrb + cur.rb] = make_int2(slot, blockIdx.x + cur.parts_in - 1);
#pragma unroll 1
      for (int c0 = 0; c0 < Dv; c0 += 64) {
        float y[64];
        __syncwarp();  // lanes without a row have not stored: the loads below take the whole warp
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float o[16];
          tmem_ld16(tmem + lane_base + kO + c0 + c * 16, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[c * 16 + e] = o[e];
        }
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float back = 1.f / sm.unit[span & 3][(c0 + c) / 32];
          float z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = y[column_of(c + e)] * back;
          if (whole) {
            finish_row<__nv_bfloat16>(a, cur.b, h, m, c0 + c, z, l, mx);
          } else {
            const int64_t at = (int64_t)slot * kTcRows + tid;
            *reinterpret_cast<float4 *>(a.part + at * Dv + c0 + c) = make_float4(z[0], z[1], z[2], z[3]);
            if (c0 + c == 0) *reinterpret_cast<float2 *>(a.part_ml + at * 2) = make_float2(mx, l);
          }
        }
      }
      tc_fence_before();
    }
  }
  // products still in flight land before shared memory and TMEM go: the last commit tracks them all
  __syncthreads();
  if (tid == kIssuer * 32) {
    tc_commit(&sm.end);
    mbar_drain(&sm.end, 0, status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace

template <int D, int Dv>
cudaError_t launch_attend_tc(AttendArgs a, const CacheView &v, int *status, cudaStream_t st) {
  const auto kernel = attend_tc<D, Dv>;
  const size_t smem = sizeof(Smem<D, Dv>) + 1024;
  // SMs of a device, looked up with the kernel's attribute once a device
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int sms = known[dev].load(std::memory_order_acquire);
  if (!sms) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known[dev].store(sms, std::memory_order_release);
  }
  const int rows = a.G * a.M;
  a.nrb = (rows + kTcRows - 1) / kTcRows;
  a.block_log2 = 7;
  a.min_tiles = 1;
  a.tile_log2 = 7;
  a.item_tiles = kTcItemTiles;
  const int64_t items = (int64_t)a.B * v.Hkv * a.nrb;
  const int64_t cap = (((int64_t)v.max_pages << v.page_log2) + kTok - 1) / kTok;
  const int ctas = (int)std::min<int64_t>(std::min(sms, kTcMaxCtas), items * (cap + a.item_tiles));
  e = launch_next(kernel, dim3(ctas), kThreads, smem, st, false, 0, a, v, status);
  if (e != cudaSuccess) return e;
  return launch_next(attend_join<__nv_bfloat16, Dv, kTcRows>, dim3(rows, v.Hkv, a.B), 128, 0, st, true,
                     0, a, v, status);
}

template cudaError_t launch_attend_tc<64, 64>(AttendArgs, const CacheView &, int *, cudaStream_t);
template cudaError_t launch_attend_tc<64, 128>(AttendArgs, const CacheView &, int *, cudaStream_t);
template cudaError_t launch_attend_tc<128, 64>(AttendArgs, const CacheView &, int *, cudaStream_t);
template cudaError_t launch_attend_tc<128, 128>(AttendArgs, const CacheView &, int *, cudaStream_t);

}  // namespace muse
