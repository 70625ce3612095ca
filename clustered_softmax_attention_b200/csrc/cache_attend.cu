// Causal attention of a sequence's newest rows over its 4-bit cache.
#include "cache.cuh"

namespace muse {
namespace {

struct AttendArgs {
  muse_rows Q, O;
  float *lse;
  const int32_t *lens, *counts;
  int B, H, M;
  float scale;
};

// One CTA per row (b, h, m); its four warps take tiles in turn, a lane a token for the logits
// and a channel of every group for the values.
template <typename T, int D, int Dv>
__global__ void __launch_bounds__(128) attend_rows(const AttendArgs a, const CacheView v,
                                                   int *status) {
  using S = TileShape<D, Dv>;
  constexpr int NGk = D / 32, NG = Dv / 32;
  __shared__ float q[D];
  __shared__ float sm[4], sl[4], so[4][Dv];
  const int m = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int count = row_count(a.counts, b, a.M, status);
  if (m >= count) return;
  int len = a.lens[b];
  const int64_t cap = (int64_t)v.max_pages << v.page_log2;
  if ((len < 0 || len > cap) && tid == 0) report(status, MUSE_ERR_DEVICE);
  len = (int)min((int64_t)max(len, 0), cap);
  const int see = max(0, len - count + m + 1);
  const int hk = h / (a.H / v.Hkv);
  if (tid < D)
    q[tid] = ld_elem((const T *)a.Q.p + b * a.Q.sb + h * a.Q.sh + m * a.Q.sn + tid) * a.scale;
  __syncthreads();
  float mx = -CUDART_INF_F, l = 0.f, o[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) o[g] = 0.f;
  for (int tile = warp; tile * 32 < see; tile += 4) {
    const uint8_t *p = cache_tile(v, b, hk, tile, S::kBytes);
    if (!p) {
      report(status, MUSE_ERR_DEVICE);
      continue;
    }
    const uint32_t *kw = (const uint32_t *)p, *vw = (const uint32_t *)(p + S::kV);
    const uint16_t *ks = (const uint16_t *)(p + S::kKStep), *vs = (const uint16_t *)(p + S::kVStep);
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < NGk; ++w) {
      float s = 0.f;
      for (int c = 0; c < 4; ++c) {
        const uint32_t u = kw[key_word<D>(lane, c, w)];
#pragma unroll
        for (int n = 0; n < 8; ++n) s = fmaf(code_value(u, n), q[32 * w + 8 * c + n], s);
      }
      x = fmaf(s, step_value(ks[lane * NGk + w]), x);
    }
    if (tile * 32 + lane >= see) x = -CUDART_INF_F;
    const float top = fmaxf(mx, warp_max(x));
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    const float fix = expf(mx - ref), e = expf(x - ref);
    mx = top;
    l = l * fix + warp_sum(e);
#pragma unroll
    for (int g = 0; g < NG; ++g) o[g] *= fix;
    const int live = min(32, see - tile * 32);
    for (int t = 0; t < live; ++t) {
      const float pt = __shfl_sync(0xffffffffu, e, t);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int c = 32 * g + lane;
        const uint32_t u = vw[value_word<Dv>(t, c & 7, c >> 6)] >> (4 * ((c & 63) >> 3));
        o[g] = fmaf(pt * step_value(vs[t * NG + g]), code_value(u, 0), o[g]);
      }
    }
  }
  if (lane == 0) {
    sm[warp] = mx;
    sl[warp] = l;
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) so[warp][32 * g + lane] = o[g];
  __syncthreads();
  float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  float z = 0.f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = expf(sm[w] - ref);
    z += f[w] * sl[w];
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  if (tid < Dv) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) y += f[w] * so[w][tid];
    st_elem((T *)a.O.p + b * a.O.sb + h * a.O.sh + m * a.O.sn + tid, y * inv);
  }
  if (tid == 0 && a.lse)
    a.lse[((int64_t)b * a.H + h) * a.M + m] = z == 0.f ? -CUDART_INF_F : ref + logf(z);
}

template <typename T, int D, int Dv>
cudaError_t launch(const AttendArgs &a, const CacheView &v, int *status, cudaStream_t st) {
  attend_rows<T, D, Dv><<<dim3(a.M, a.H, a.B), 128, 0, st>>>(a, v, status);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_width(const AttendArgs &a, const muse_dims &d, const CacheView &v, int *status,
                     cudaStream_t st) {
  if (d.D == 64)
    return d.Dv == 64 ? launch<T, 64, 64>(a, v, status, st) : launch<T, 64, 128>(a, v, status, st);
  return d.Dv == 64 ? launch<T, 128, 64>(a, v, status, st) : launch<T, 128, 128>(a, v, status, st);
}

}  // namespace

size_t cache_attend_ws(const muse_dims &d, int Hkv) { return 256; }

cudaError_t run_cache_attend(const muse_rows &Q, const muse_dims &d, const muse_cache &c,
                             const int32_t *lens, const int32_t *counts, const muse_rows &O,
                             float *lse, void *ws, int *status, cudaStream_t st) {
  const AttendArgs a{Q, O, lse, lens, counts, d.B, d.H, d.N, d.scale};
  const CacheView v = cache_view(c);
  return d.dtype == MUSE_F32 ? by_width<float>(a, d, v, status, st)
                             : by_width<__nv_bfloat16>(a, d, v, status, st);
}

}  // namespace muse
