// Writing keys and values into the 4-bit cache and reading them back.
//
// A group of 32 neighbouring channels of one token has step = bf16(max|x| / 7) and codes
// round_half_even(x / step), the code of the exact quotient:
//   float32: t = x * (1 / step) rounded to a whole number (by adding 1.5 * 2^23) is within one
//   of it, r = x - t step is exact in float32 (t step has at most 12 bits, and r is a multiple of
//   the smaller of the two units and below x), and |r| against half a step, which is exact too,
//   says whether t has to move: when above, or when equal and t is odd;
//   bfloat16: x and step have 8 bits, so a quotient that is not half-way between two codes is at
//   least 2^-10 from there.  x * (1 / step), off by 2^-20 at most, is rounded to a multiple of
//   2^-14, which makes half-way quotients exact, and then to a whole number.
//
// Both directions read and write every byte once; a tile is put together, or taken apart, in
// shared memory, so that the cache and the rows are each moved 16 bytes a thread.  65536 tokens of
// 16 heads of 128 + 128 channels, bfloat16 (537 MB of rows, 151 MB of cache): written in 128 us
// (5.4 TB/s, 82 % of a copy's rate), read back in 114 us (6.0 TB/s, 92 %).  Writing is bound as much
// by its instructions (issue slots 71 % used: a code takes a fused multiplication, an
// addition and a shifted addition) as by its loads; reading by DRAM.  A token of 32 sequences: 9 us for both
// calls, two launches.
#include "cache.cuh"

namespace muse {
namespace {

struct CacheRows {
  muse_rows K, V;
  const int32_t *start, *counts;
  int N;
};

// 32 channels of one group as float32.
__device__ __forceinline__ void load_group(const float *p, float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = reinterpret_cast<const float4 *>(p)[i];
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}
// The step of a group whose largest magnitude has these bits; false when it holds an infinity or
// a NaN.
__device__ __forceinline__ bool group_step(uint32_t top, float &step, uint16_t &sb) {
  if (top >= 0x7f800000u) {
    sb = 0xffffu;
    return false;
  }
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.f));
  sb = __bfloat16_as_ushort(s);
  step = __bfloat162float(s);
  return true;
}
// Steps below 2^-100: 1 / step may overflow, and the step may be far from max|x| / 7.
__device__ __noinline__ uint32_t tiny_code(float x, float step) {
  const double t = step > 0.f ? rint((double)x / (double)step) : 0.0;
  return (uint32_t)(int)(fmin(fmax(t, -7.0), 7.0) + 8.0);
}

// Packs the codes + 8 of a group, u(i) of channel i, into words of eight: for keys the channels
// in order, for values channel 8 n + g as nibble n of half word g.
struct KeyOrder {
  static constexpr int kWords = 4, kNibbles = 8;
  static __device__ __forceinline__ int channel(int w, int n) { return 8 * w + n; }
};
struct ValueOrder {
  static constexpr int kWords = 8, kNibbles = 4;
  static __device__ __forceinline__ int channel(int w, int n) { return 8 * n + w; }
};

template <typename Order>
__device__ __forceinline__ uint16_t quantise(const float *p, uint32_t (&w)[Order::kWords]) {
  float x[32];
  load_group(p, x);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  float step = 0.f;
  uint16_t sb;
  const bool fine = group_step(top, step, sb);
  const bool tiny = !fine || step < 0x1p-100f;
  if (tiny) {
#pragma unroll
    for (int k = 0; k < Order::kWords; ++k) {
      w[k] = 0;
#pragma unroll
      for (int n = 0; n < Order::kNibbles; ++n)
        w[k] |= (fine ? tiny_code(x[Order::channel(k, n)], step) : 8u) << (4 * n);
    }
    return sb;
  }
  const float inv = __frcp_rn(step), half = 0.5f * step;
#pragma unroll
  for (int k = 0; k < Order::kWords; ++k) {
    uint32_t sum = 0, less = 0;
#pragma unroll
    for (int n = 0; n < Order::kNibbles; ++n) {
      const float y = x[Order::channel(k, n)];
      const float at = fmaf(y, inv, 12582912.f);  // its bits are 0x4B400000 + t
      const float r = fmaf(12582912.f - at, step, y);
      uint32_t t = __float_as_uint(at);
      // the float below half a step when t is odd: then |r| = half moves too
      if (fabsf(r) > __uint_as_float(__float_as_uint(half) - (t & 1u))) t += r > 0.f ? 1 : -1;
      sum += t << (4 * n);
      less += (0x4B400000u - 8u) << (4 * n);
    }
    w[k] = sum - less;
  }
  return sb;
}

template <typename Order>
__device__ __forceinline__ uint16_t quantise(const __nv_bfloat16 *p, uint32_t (&w)[Order::kWords]) {
  uint32_t x[16], top2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) top2 = __vmaxu2(top2, x[i] & 0x7fff7fffu);
  float step = 0.f;
  uint16_t sb;
  const bool fine = group_step(max(top2 << 16, top2 & 0xffff0000u), step, sb);
  if (fine && step >= 0x1p-100f) {
    const float inv = __frcp_rn(step);
#pragma unroll
    for (int k = 0; k < Order::kWords; ++k) {
      // a rounded number as bits is 0x4B400000 + 8 + code: the sum of them times 16^n, and what
      // the constants add up to, modulo 2^32
      uint32_t sum = 0, less = 0;
#pragma unroll
      for (int n = 0; n < Order::kNibbles; ++n) {
        const int c = Order::channel(k, n);
        const float y = __uint_as_float(c & 1 ? x[c >> 1] & 0xffff0000u : x[c >> 1] << 16);
        const float at = fmaf(y, inv, 768.f);               // multiples of 2^-14
        sum += __float_as_uint(at + 12582152.f) << (4 * n); // 2^23 + 2^22 + 8 - 768
        less += 0x4B400000u << (4 * n);
      }
      w[k] = sum - less;
    }
  } else {
#pragma unroll
    for (int k = 0; k < Order::kWords; ++k) {
      w[k] = 0;
#pragma unroll
      for (int n = 0; n < Order::kNibbles; ++n) {
        const int c = Order::channel(k, n);
        const float y = __uint_as_float(c & 1 ? x[c >> 1] & 0xffff0000u : x[c >> 1] << 16);
        w[k] |= (fine ? tiny_code(y, step) : 8u) << (4 * n);
      }
    }
  }
  return sb;
}

// One CTA per tile that the call touches: a thread quantises one group of one token into the
// tile's image in shared memory, and the words of the tokens that were written go out.
template <typename T, int D, int Dv>
__global__ void __launch_bounds__(D + Dv) cache_write(const CacheRows a, const CacheView v,
                                                     int *status) {
  using S = TileShape<D, Dv>;
  constexpr int kThreads = D + Dv;
  __shared__ __align__(16) uint32_t img[S::kBytes / 4];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  dependents_may_launch();
  wait_for_earlier();
  const int count = row_count(a.counts, b, a.N, status);
  const int start = a.start[b];
  // tiles are counted from the one that holds the first token (rounded down for start < 0)
  const int64_t tile = (int64_t)(start >> 5) + blockIdx.x;
  const int64_t n0 = tile * kTile - start;  // row of the tile's token 0
  const int lo = (int)max((int64_t)0, -n0), hi = (int)min((int64_t)kTile, count - n0);
  if (lo >= hi) return;
  uint8_t *dst = tile > 0x3ffffff ? nullptr : cache_tile(v, b, h, (int)tile, S::kBytes);
  if (!dst) {
    if (tid == 0) report(status, MUSE_ERR_DEVICE);
    return;
  }
  {
    const bool key = tid < D;  // D / 32 groups x 32 tokens
    const int id = key ? tid : tid - D, per = key ? D / 32 : Dv / 32;
    const int t = id / per, grp = id - t * per;
    if (t >= lo && t < hi) {
      const muse_rows &r = key ? a.K : a.V;
      const T *p = (const T *)r.p + b * r.sb + h * r.sh + (n0 + t) * r.sn + grp * 32;
      uint16_t *steps = reinterpret_cast<uint16_t *>(img) + (key ? S::kKStep : S::kVStep) / 2;
      if (key) {
        uint32_t w[4];
        steps[t * per + grp] = quantise<KeyOrder>(p, w);
#pragma unroll
        for (int q = 0; q < 4; ++q) img[key_word<D>(t, q, grp)] = w[q];
      } else {
        uint32_t w[8];
        steps[t * per + grp] = quantise<ValueOrder>(p, w);
        uint16_t *half = reinterpret_cast<uint16_t *>(img + S::kV / 4);
#pragma unroll
        for (int g = 0; g < 8; ++g)
          half[2 * value_word<Dv>(t, g, grp >> 1) + (grp & 1)] = (uint16_t)w[g];
      }
    }
  }
  __syncthreads();
  if (lo == 0 && hi == kTile) {
    for (int i = tid; i < S::kBytes / 16; i += kThreads)
      reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(img)[i];
    return;
  }
  uint32_t *out = reinterpret_cast<uint32_t *>(dst);
  for (int i = tid; i < S::kBytes / 4; i += kThreads) {
    int t;
    if (i < S::kV / 4) t = key_word_token<D>(i);
    else if (i < S::kKStep / 4) t = value_word_token<Dv>(i - S::kV / 4);
    else if (i < S::kVStep / 4) t = (i - S::kKStep / 4) / (D / 64);
    else t = (i - S::kVStep / 4) / (Dv / 64);
    if (t >= lo && t < hi) out[i] = img[i];
  }
}

// Eight channels of a token: codes times the step, rounded once.
__device__ __forceinline__ void store8(float *p, const float (&y)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
// (x & 0x000f000f) | 0x43004300 in one operation: two codes as bfloat16 128 + u; less 136 they are
// exact, and their product with the step is rounded once, as two values an operation.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t x, __nv_bfloat162 step) {
  uint32_t y;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(y) : "r"(x), "r"(0x43004300u));
  const __nv_bfloat162 less = __bfloat162bfloat162(__ushort_as_bfloat16(0xC308));  // -136
  const __nv_bfloat162 v = __hmul2(__hadd2(*reinterpret_cast<__nv_bfloat162 *>(&y), less), step);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void put_key(float *p, uint32_t w, uint16_t step) {
  const float s = step_value(step);
  float y[8];
#pragma unroll
  for (int n = 0; n < 8; ++n) y[n] = code_value(w, n) * s;
  store8(p, y);
}
__device__ __forceinline__ void put_key(__nv_bfloat16 *p, uint32_t w, uint16_t step) {
  const __nv_bfloat162 s = __bfloat162bfloat162(__ushort_as_bfloat16(step));
  uint32_t c[4];  // channels n and n + 4
#pragma unroll
  for (int n = 0; n < 4; ++n) c[n] = scaled_pair(w >> (4 * n), s);
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410),
                 __byte_perm(c[0], c[1], 0x7632), __byte_perm(c[2], c[3], 0x7632));
}
// w: the words of channel residues g = 0..7, of which nibble n is wanted.
__device__ __forceinline__ void put_value(float *p, const uint32_t (&w)[8], int n, uint16_t step) {
  const float s = step_value(step);
  float y[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) y[g] = code_value(w[g] >> (4 * n), 0) * s;
  store8(p, y);
}
__device__ __forceinline__ void put_value(__nv_bfloat16 *p, const uint32_t (&w)[8], int n,
                                          uint16_t step) {
  const __nv_bfloat162 s = __bfloat162bfloat162(__ushort_as_bfloat16(step));
  const uint32_t half = n & 4 ? 0x7632 : 0x5410;
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = scaled_pair(__byte_perm(w[2 * k], w[2 * k + 1], half) >> (4 * (n & 3)), s);
  *reinterpret_cast<uint4 *>(p) = make_uint4(c[0], c[1], c[2], c[3]);
}

// One CTA per tile: the tile to shared memory, then eight channels of a token a thread, so
// that neighbouring threads store neighbouring 16 (or 32) bytes.
template <typename T, int D, int Dv>
__global__ void __launch_bounds__(D + Dv) cache_read(const CacheRows a, const CacheView v,
                                                    int *status) {
  using S = TileShape<D, Dv>;
  constexpr int kThreads = D + Dv;
  __shared__ __align__(16) uint32_t img[S::kBytes / 4];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  dependents_may_launch();
  wait_for_earlier();
  const int count = row_count(a.counts, b, a.N, status);
  const int start = a.start[b];
  const int64_t tile = (int64_t)(start >> 5) + blockIdx.x;
  const int64_t n0 = tile * kTile - start;
  const int lo = (int)max((int64_t)0, -n0), hi = (int)min((int64_t)kTile, count - n0);
  if (lo >= hi) return;
  const uint8_t *src = tile > 0x3ffffff ? nullptr : cache_tile(v, b, h, (int)tile, S::kBytes);
  if (!src) {
    if (tid == 0) report(status, MUSE_ERR_DEVICE);
    return;
  }
  for (int i = tid; i < S::kBytes / 16; i += kThreads)
    reinterpret_cast<uint4 *>(img)[i] = reinterpret_cast<const uint4 *>(src)[i];
  __syncthreads();
  const uint16_t *ks = reinterpret_cast<const uint16_t *>(img) + S::kKStep / 2;
  const uint16_t *vs = reinterpret_cast<const uint16_t *>(img) + S::kVStep / 2;
  const uint32_t *vw = img + S::kV / 4;
  T *kp = (T *)a.K.p + b * a.K.sb + h * a.K.sh + n0 * a.K.sn;
  T *vp = (T *)a.V.p + b * a.V.sb + h * a.V.sh + n0 * a.V.sn;
#pragma unroll
  for (int i0 = 0; i0 < 32 * (D / 8); i0 += kThreads) {
    const int i = i0 + tid;
    if (32 * (D / 8) % kThreads && i >= 32 * (D / 8)) break;
    const int t = i / (D / 8), j = i % (D / 8);
    if (t >= lo && t < hi)
      put_key(kp + t * a.K.sn + 8 * j, img[key_word<D>(t, j & 3, j >> 2)], ks[t * (D / 32) + (j >> 2)]);
  }
  // a thread takes nibble n of all words of a token: Dv / 64 runs of eight channels
#pragma unroll
  for (int i0 = 0; i0 < 32 * 8; i0 += kThreads) {
    const int i = i0 + tid;
    if (32 * 8 % kThreads && i >= 32 * 8) break;
    const int t = i / 8, n = i % 8;
    if (t < lo || t >= hi) continue;
    uint32_t w[Dv / 64][8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const uint32_t *at = vw + value_word<Dv>(t, g, 0);
      if (Dv == 128) {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        w[0][g] = x.x;
        w[Dv / 64 - 1][g] = x.y;
      } else {
        w[0][g] = *at;
      }
    }
#pragma unroll
    for (int k = 0; k < Dv / 64; ++k)
      put_value(vp + t * a.V.sn + 64 * k + 8 * n, w[k], n, vs[t * (Dv / 32) + 2 * k + (n >> 2)]);
  }
}

template <typename T, int D, int Dv>
cudaError_t launch(bool write, const CacheRows &a, const CacheView &v, int B, int *status,
                   cudaStream_t st) {
  // N rows from any start touch at most (N + 30) / 32 + 1 tiles
  const dim3 grid((unsigned)((a.N + 30) / 32 + 1), (unsigned)v.Hkv, (unsigned)B);
  return launch_next(write ? cache_write<T, D, Dv> : cache_read<T, D, Dv>, grid, D + Dv, 0, st, true, 0, a,
                     v,
                     status);
}

template <typename T>
cudaError_t by_width(bool write, const CacheRows &a, const muse_dims &d, const muse_cache &c,
                     int *status, cudaStream_t st) {
  const CacheView v = cache_view(c);
  if (d.D == 64)
    return d.Dv == 64 ? launch<T, 64, 64>(write, a, v, d.B, status, st)
                      : launch<T, 64, 128>(write, a, v, d.B, status, st);
  return d.Dv == 64 ? launch<T, 128, 64>(write, a, v, d.B, status, st)
                    : launch<T, 128, 128>(write, a, v, d.B, status, st);
}

cudaError_t run(bool write, const muse_rows &K, const muse_rows &V, const muse_dims &d,
                const muse_cache &c, const int32_t *start, const int32_t *counts, int *status,
                cudaStream_t st) {
  const CacheRows a{K, V, start, counts, d.N};
  return d.dtype == MUSE_F32 ? by_width<float>(write, a, d, c, status, st)
                             : by_width<__nv_bfloat16>(write, a, d, c, status, st);
}

}  // namespace

cudaError_t run_cache_write(const muse_rows &K, const muse_rows &V, const muse_dims &d,
                            const muse_cache &c, const int32_t *start, const int32_t *counts,
                            int *status, cudaStream_t st) {
  return run(true, K, V, d, c, start, counts, status, st);
}
cudaError_t run_cache_read(const muse_dims &d, const muse_cache &c, const int32_t *start,
                           const int32_t *counts, const muse_rows &K, const muse_rows &V,
                           int *status, cudaStream_t st) {
  return run(false, K, V, d, c, start, counts, status, st);
}

}  // namespace muse
