// Rotary positions with several axes (muse_rope_axes).
//
// Pair i of a row turns by t = pos[axis(i)] * f_i.  Far positions lose their angle in
// float32 (pos * f has 24 bits, of which the turns take all but a few), so the angle is kept
// as a fraction of a turn in 64-bit integers: pos * turn[i] modulo 2^64 drops whole turns
// exactly, and its high 32 bits, as a float in [-1, 1) half turns, go to sincospif (error
// below 2^-24 half turns and the function's own).
//
// Memory-bound: every element is read and written once.  The angles of a row are the same for
// every head, so a thread keeps VEC sines and cosines and walks the heads with 16-byte loads.
#include "internal.h"

namespace muse {
namespace {

struct RopeArgs {
  muse_rows Q, K, Qo, Ko;
  const int32_t *pos;
  int64_t pos_sb;  // 0 when the batch shares its positions
  int B, H, Hk, N, heads_per_cta;
};

template <typename T>
__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
  const float u = x * c - y * s, v = x * s + y * c;
  x = u;
  y = v;
}

__device__ __forceinline__ void pair_angle(const RopeTable &t, const int32_t *pos, int N, int i,
                                           float &s, float &c) {
  const int64_t p = pos[(int64_t)t.axis[i] * N];
  const uint64_t ph = (uint64_t)p * t.turn[i];
  sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &s, &c);
}

// One thread per pair (or pair of copied channels) and row: any sections.
template <typename T, int D>
__global__ void __launch_bounds__(128) rope_pairs(const RopeArgs a,
                                                  const __grid_constant__ RopeTable t) {
  const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const int64_t row = id / (D / 2);
  const int i = (int)(id - row * (D / 2));
  if (row >= (int64_t)a.B * a.N) return;
  const int b = (int)(row / a.N), n = (int)(row - (int64_t)b * a.N);
  const bool turned = i < t.P;
  const int c0 = !turned || t.adjacent ? 2 * i : i;
  const int c1 = !turned || t.adjacent ? 2 * i + 1 : i + t.P;
  float s = 0.f, c = 1.f;
  if (turned) pair_angle(t, a.pos + b * a.pos_sb + n, a.N, i, s, c);
  const int h1 = min(a.H + a.Hk, (int)(blockIdx.y + 1) * a.heads_per_cta);
  for (int h = blockIdx.y * a.heads_per_cta; h < h1; ++h) {
    const bool q = h < a.H;
    const muse_rows &in = q ? a.Q : a.K, &out = q ? a.Qo : a.Ko;
    const int hh = q ? h : h - a.H;
    const T *x = (const T *)in.p + b * in.sb + hh * in.sh + n * in.sn;
    T *y = (T *)out.p + b * out.sb + hh * out.sh + n * out.sn;
    const T e0 = x[c0], e1 = x[c1];
    if (turned) {
      float u = ld_elem(&e0), v = ld_elem(&e1);
      turn<T>(u, v, c, s);
      st_elem(y + c0, u);
      st_elem(y + c1, v);
    } else {
      y[c0] = e0;
      y[c1] = e1;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const RopeArgs &a0, const RopeTable &t, cudaStream_t st) {
  RopeArgs a = a0;
  const int64_t work = (int64_t)a.B * a.N * (D / 2);
  const int64_t ctas = (work + 127) / 128;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  a.heads_per_cta = a.H + a.Hk;
  rope_pairs<T, D><<<dim3((unsigned)ctas, 1), 128, 0, st>>>(a, t);
  count_launches(1);
  return cudaGetLastError();
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
  if (d.dtype == MUSE_F32) return d.D == 64 ? launch<float, 64>(a, t, st) : launch<float, 128>(a, t, st);
  return d.D == 64 ? launch<__nv_bfloat16, 64>(a, t, st) : launch<__nv_bfloat16, 128>(a, t, st);
}

}  // namespace muse
