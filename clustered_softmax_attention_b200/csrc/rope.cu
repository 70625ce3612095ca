// Rotary positions with several axes (muse_rope_axes).
//
// Pair i of a row turns by t = pos[axis(i)] * f_i.  Far positions lose their angle in
// float32 (pos * f has 24 bits, of which the turns take all but a few), so the angle is kept
// as a fraction of a turn in 64-bit integers: pos * turn[i] modulo 2^64 drops whole turns
// exactly, and its high 32 bits are half turns in [-1, 1).  Their float goes to sincospif, and what it
// rounded off (up to 2^-25 half turns, a thousandth of a sine next to zero) turns the result by that
// much more, so that an angle is off by 2^-31 half turns and the function's own error.
//
// Memory-bound: every element is read and written once.  The angles of a row are the same for
// every head, so a thread keeps its sines and cosines and walks the heads, four at a time, with
// the widest loads that both halves of its pairs are aligned for (16 bytes when P is a multiple
// of 8 in bfloat16, of 4 in float32, or for adjacent pairs; down to one element for odd P).
// Measured on a B200: 4 x 16384 tokens, 16 heads of 64 channels, bfloat16 (268 MB) in 46 us, 5.8 TB/s,
// 88 % of a copy's rate; float32, 2 x 5003 tokens, 32 heads of 128 (328 MB) in 61 us; one token of 16
// sequences 6.4 us, a launch's time.  It waits on its loads (4 heads are under way a thread, 38 % of
// the warps that fit).  With loads of two elements whatever P is, 16384 tokens of 32 heads of 128
// take 69 us instead of 54.
#include <algorithm>

#include "internal.h"

namespace muse {
namespace {

struct RopeArgs {
  muse_rows Q, K, Qo, Ko;
  const int32_t *pos;
  int64_t pos_sb;  // 0 when the batch shares its positions
  int B, H, Hk, N, heads_per_cta;
};

__device__ __forceinline__ void angle(const RopeTable &t, const int32_t *pos, int N, int i,
                                      float &s, float &c) {
  const int64_t p = pos[(int64_t)t.axis[i] * N];
  const uint64_t ph = (uint64_t)p * t.turn[i];
  const int32_t half_turns = (int32_t)(ph >> 32);
  const float x = __int2float_rn(half_turns);
  // 2^31 does not come back as an integer: it is off by one
  const float rest = (float)(half_turns - __float2int_rn(x)) * (3.14159265f * 0x1p-31f);
  float s0, c0;
  sincospif(x * 0x1p-31f, &s0, &c0);
  s = fmaf(c0, rest, s0);
  c = fmaf(-s0, rest, c0);
}

// VEC elements as one load; streamed, since nothing is read twice.
template <typename T, int VEC>
struct Vec {
  static constexpr int kBytes = VEC * sizeof(T);
  uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];
  __device__ __forceinline__ void load(const T *p) {
    if (kBytes == 16) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
      w[0] = v.x;
      w[kBytes / 4 > 1 ? 1 : 0] = v.y;
      w[kBytes / 4 > 2 ? 2 : 0] = v.z;
      w[kBytes / 4 > 3 ? 3 : 0] = v.w;
    } else if (kBytes == 8) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
      w[0] = v.x;
      w[kBytes / 4 > 1 ? 1 : 0] = v.y;
    } else if (kBytes == 4) {
      w[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint16_t *>(p));
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if (kBytes == 16)
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[kBytes / 4 > 1 ? 1 : 0],
                                                      w[kBytes / 4 > 2 ? 2 : 0], w[kBytes / 4 > 3 ? 3 : 0]));
    else if (kBytes == 8)
      __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[kBytes / 4 > 1 ? 1 : 0]));
    else if (kBytes == 4) __stcs(reinterpret_cast<uint32_t *>(p), w[0]);
    else __stcs(reinterpret_cast<uint16_t *>(p), (uint16_t)w[0]);
  }
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // elements i and i + 1 (i even), or the only one
  __device__ __forceinline__ void set(int i, float x, float y) {
    if (sizeof(T) == 4) {
      w[i] = __float_as_uint(x);
      if (VEC > 1) w[VEC > 1 ? i + 1 : i] = __float_as_uint(y);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      w[i >> 1] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
};

constexpr int kThreads = 128;
constexpr int kHeads = 4;  // heads whose loads are under way together

// A thread owns two vectors of a row: the two halves of VEC pairs, two vectors of adjacent
// pairs, or two vectors that are copied.
template <typename T, int D, int VEC, bool ADJ>
__global__ void __launch_bounds__(kThreads) rope(const RopeArgs a, const __grid_constant__ RopeTable t) {
  constexpr int kRow = D / (2 * VEC);  // threads of a row
  dependents_may_launch();
  wait_for_earlier();
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = id / kRow;
  const int u = (int)(id - row * kRow);
  if (row >= (int64_t)a.B * a.N) return;
  const int b = (int)(row / a.N), n = (int)(row - (int64_t)b * a.N);
  // channels of the two vectors, and the first pair of each (P or more: copied)
  int c0, c1;
  if (ADJ) {
    c0 = u * VEC;
    c1 = c0 + D / 2;
  } else {
    const int turned = t.P / VEC;
    c0 = u < turned ? u * VEC : 2 * t.P + (u - turned) * 2 * VEC;
    c1 = u < turned ? t.P + u * VEC : c0 + VEC;
  }
  float sn[VEC], cs[VEC];
  const int32_t *pos = a.pos + b * a.pos_sb + n;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int pair = ADJ ? (i < VEC / 2 ? c0 / 2 + i : c1 / 2 + i - VEC / 2) : u * VEC + i;
    sn[i] = 0.f;
    cs[i] = 1.f;
    if (pair < t.P) angle(t, pos, a.N, pair, sn[i], cs[i]);
  }
  const int h1 = min(a.H + a.Hk, (int)(blockIdx.y + 1) * a.heads_per_cta);
  for (int h0 = blockIdx.y * a.heads_per_cta; h0 < h1; h0 += kHeads) {
    Vec<T, VEC> x[kHeads], y[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k;
      if (h >= h1) break;
      const muse_rows &r = h < a.H ? a.Q : a.K;
      const T *p = (const T *)r.p + b * r.sb + (h < a.H ? h : h - a.H) * r.sh + n * r.sn;
      x[k].load(p + c0);
      y[k].load(p + c1);
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k;
      if (h >= h1) break;
      const muse_rows &r = h < a.H ? a.Qo : a.Ko;
      T *p = (T *)r.p + b * r.sb + (h < a.H ? h : h - a.H) * r.sh + n * r.sn;
      if (ADJ) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          Vec<T, VEC> &z = v ? y[k] : x[k];
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float s = sn[v * VEC / 2 + i], c = cs[v * VEC / 2 + i];
            const float e = z.get(2 * i), f = z.get(2 * i + 1);
            // a copied pair stays as it is, whatever it holds
            if ((v ? c1 : c0) / 2 + i < t.P) z.set(2 * i, e * c - f * s, e * s + f * c);
          }
        }
      } else if (u * VEC < t.P) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const int j = VEC > 1 ? i + 1 : i;
          const float e0 = x[k].get(i), f0 = y[k].get(i), e1 = x[k].get(j), f1 = y[k].get(j);
          x[k].set(i, e0 * cs[i] - f0 * sn[i], e1 * cs[j] - f1 * sn[j]);
          y[k].set(i, e0 * sn[i] + f0 * cs[i], e1 * sn[j] + f1 * cs[j]);
        }
      }
      x[k].store(p + c0);
      y[k].store(p + c1);
    }
  }
}

template <typename T, int D, int VEC, bool ADJ>
cudaError_t launch(RopeArgs a, const RopeTable &t, cudaStream_t st) {
  const int heads = a.H + a.Hk;
  const int64_t ctas = ((int64_t)a.B * a.N * (D / (2 * VEC)) + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  // Few rows: the heads are dealt out to more threads, each with its own angles; all heads to a
  // thread once that fills the card.  40 heads of 128 channels, split and not: 1 token 9 and 18 us,
  // 512 tokens 11 and 20, 2048 tokens 17 and 22.
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(heads, (148 * 8 + ctas - 1) / ctas));
  a.heads_per_cta = (int)((heads + split - 1) / split);
  const unsigned groups = (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta);
  return launch_next(rope<T, D, VEC, ADJ>, dim3((unsigned)ctas, groups), kThreads, 0, st, true, 0,
                     a, t);
}

template <typename T, int D>
cudaError_t by_width(const RopeArgs &a, const RopeTable &t, cudaStream_t st) {
  constexpr int kWide = 16 / sizeof(T);
  if (t.adjacent) return launch<T, D, kWide, true>(a, t, st);
  if (t.P % kWide == 0) return launch<T, D, kWide, false>(a, t, st);
  if (t.P % (kWide / 2) == 0) return launch<T, D, kWide / 2, false>(a, t, st);
  if (t.P % 2 == 0) return launch<T, D, 2, false>(a, t, st);
  return launch<T, D, 1, false>(a, t, st);
}

}  // namespace

cudaError_t run_rope(const muse_rows &Q, const muse_rows &K, int Hk, const muse_dims &d,
                     const int32_t *pos, int pos_batches, const RopeTable &t, const muse_rows &Qo,
                     const muse_rows &Ko, cudaStream_t st) {
  RopeArgs a;
  a.Q = Q;
  a.K = K;
  a.Qo = Qo;
  a.Ko = Ko;
  a.pos = pos;
  a.pos_sb = pos_batches == 1 ? 0 : (int64_t)t.axes * d.N;
  a.B = d.B;
  a.H = d.H;
  a.Hk = Hk;
  a.N = d.N;
  if (d.dtype == MUSE_F32)
    return d.D == 64 ? by_width<float, 64>(a, t, st) : by_width<float, 128>(a, t, st);
  return d.D == 64 ? by_width<__nv_bfloat16, 64>(a, t, st) : by_width<__nv_bfloat16, 128>(a, t, st);
}

}  // namespace muse
