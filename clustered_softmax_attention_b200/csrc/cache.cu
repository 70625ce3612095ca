// Writing keys and values into the 4-bit cache and reading them back.
//
// A group of 32 neighbouring channels of one token has step = bf16(max|x| / 7) and codes
// round_half_even(x / step), the code of the exact quotient:
//   float32: t = rint(x * (1 / step)) is within one of it, r = x - t step is exact in float32
//   (t step has at most 12 bits, and r is a multiple of the smaller of the two units and below
//   x), and r against half a step, which is exact too, says whether t has to move;
//   bfloat16: x and step have 8 bits, so a quotient that is not half-way between two codes is at
//   least 2^-10 from there.  x * (1 / step), off by 2^-20 at most, is rounded to a multiple of
//   2^-14, which makes half-way quotients exact, and then to a whole number.
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
  const float inv = tiny ? 0.f : __frcp_rn(step), half = 0.5f * step;
#pragma unroll
  for (int k = 0; k < Order::kWords; ++k) {
    w[k] = 0;
#pragma unroll
    for (int n = 0; n < Order::kNibbles; ++n) {
      const float y = x[Order::channel(k, n)];
      float t = rintf(y * inv);
      const float r = fmaf(-t, step, y);
      const bool odd = ((int)t & 1) != 0;
      if (r > half || (r == half && odd)) t += 1.f;
      else if (r < -half || (r == -half && odd)) t -= 1.f;
      const uint32_t u = !fine ? 8u : tiny ? tiny_code(y, step) : (uint32_t)((int)t + 8);
      w[k] |= u << (4 * n);
    }
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

__device__ __forceinline__ void store8(float *p, const float (&y)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&y)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
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
  for (int i = tid; i < 32 * (D / 8); i += kThreads) {
    const int t = i / (D / 8), j = i - t * (D / 8);
    if (t < lo || t >= hi) continue;
    const uint32_t w = img[key_word<D>(t, j & 3, j >> 2)];
    const float step = step_value(ks[t * (D / 32) + (j >> 2)]);
    float y[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) y[n] = code_value(w, n) * step;
    store8((T *)a.K.p + b * a.K.sb + h * a.K.sh + (n0 + t) * a.K.sn + 8 * j, y);
  }
  for (int i = tid; i < 32 * (Dv / 8); i += kThreads) {
    const int t = i / (Dv / 8), j = i - t * (Dv / 8);
    if (t < lo || t >= hi) continue;
    const float step = step_value(vs[t * (Dv / 32) + (j >> 2)]);
    float y[8];
#pragma unroll
    for (int g = 0; g < 8; ++g)
      y[g] = code_value(vw[value_word<Dv>(t, g, j >> 3)] >> (4 * (j & 7)), 0) * step;
    store8((T *)a.V.p + b * a.V.sb + h * a.V.sh + (n0 + t) * a.V.sn + 8 * j, y);
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
