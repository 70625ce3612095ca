// extern "C" entry points of the serving operators: argument validation and the launch of
// each.  Declarations and the meaning of every argument: include/muse.h.
#include <math.h>

#include "internal.h"

namespace muse {

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static muse_status check_shape(const muse_dims &d, bool need_dv) {
  if (d.dtype != MUSE_F32 && d.dtype != MUSE_BF16) return MUSE_ERR_DTYPE;
  if (d.B <= 0 || d.H <= 0 || d.N <= 0) return MUSE_ERR_SHAPE;
  if (d.D != 64 && d.D != 128) return MUSE_ERR_SHAPE;
  if (need_dv && d.Dv != 64 && d.Dv != 128) return MUSE_ERR_SHAPE;
  if ((int64_t)d.B * d.H > 65535) return MUSE_ERR_SHAPE;
  if ((int64_t)d.N * 128 > (int64_t)1 << 31) return MUSE_ERR_SHAPE;
  return MUSE_OK;
}

// A view of rows: 16-byte aligned, every stride a multiple of 16 bytes and not negative.
static bool valid_rows(const muse_rows &r, int dtype) {
  const int64_t unit = dtype == MUSE_F32 ? 4 : 8;
  if (!r.p || !aligned16(r.p)) return false;
  return r.sb >= 0 && r.sh >= 0 && r.sn >= 0 && r.sb % unit == 0 && r.sh % unit == 0 &&
         r.sn % unit == 0;
}

static muse_status check_cache(const muse_cache &c, const muse_dims &d) {
  if (!c.tiles || !aligned16(c.tiles) || !c.page_table) return MUSE_ERR_INVALID_ARG;
  if (c.pages <= 0 || c.Hkv <= 0 || c.max_pages <= 0) return MUSE_ERR_SHAPE;
  if (c.page < 32 || c.page > 1024 || (c.page & (c.page - 1))) return MUSE_ERR_SHAPE;
  const int64_t top = (int64_t)1 << 31;
  if ((int64_t)c.max_pages * c.page >= top || (int64_t)c.pages * c.Hkv >= top ||
      (int64_t)c.pages * c.Hkv * (c.page / 32) >= top)
    return MUSE_ERR_SHAPE;
  if ((int64_t)d.B * c.max_pages >= top) return MUSE_ERR_SHAPE;
  return MUSE_OK;
}

static muse_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MUSE_OK;
  const cudaError_t last = cudaGetLastError();
  return cuda_fail(last != cudaSuccess ? last : e);
}

// Frequencies of a muse_rope as 64-bit fractions of a turn; false when r is not valid for D.
static bool rope_table(const muse_rope &r, int D, RopeTable &t) {
  if (r.axes < 1 || r.axes > MUSE_ROPE_MAX_AXES) return false;
  if (r.flags & ~(MUSE_ROPE_INVERSE | MUSE_ROPE_ADJACENT | MUSE_ROPE_AXIS_LADDER)) return false;
  if (!(r.base >= 1.0) || !(r.base <= 1e12)) return false;
  int P = 0;
  for (int a = 0; a < r.axes; ++a) {
    if (r.sections[a] < 1 || r.sections[a] > D / 2) return false;
    P += r.sections[a];
  }
  if (P > D / 2) return false;
  t.P = P;
  t.axes = r.axes;
  t.adjacent = (r.flags & MUSE_ROPE_ADJACENT) != 0;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  for (int a = 0, i = 0; a < r.axes; ++a) {
    // base^-e down a ladder by its ratio: 64 products of 64 bits lose no more than 2^-58
    const bool own = (r.flags & MUSE_ROPE_AXIS_LADDER) != 0;
    const long double ratio = powl((long double)r.base, -1.0L / (own ? r.sections[a] : P));
    long double f = own ? 1.0L : powl(ratio, i);
    for (int j = 0; j < r.sections[a]; ++j, ++i, f *= ratio) {
      // below 1 / (2 pi) of a turn, so the fraction fits
      const uint64_t u = (uint64_t)(f / two_pi * 18446744073709551616.0L);
      t.turn[i] = (r.flags & MUSE_ROPE_INVERSE) ? 0 - u : u;
      t.axis[i] = (uint8_t)a;
    }
  }
  for (int i = P; i < 64; ++i) {
    t.turn[i] = 0;
    t.axis[i] = 0;
  }
  return true;
}

}  // namespace muse

using namespace muse;

extern "C" muse_status muse_rope_axes(muse_rows Q, muse_rows K, int Hk, muse_dims d,
                                      const int32_t *pos, int pos_batches, muse_rope r,
                                      muse_rows Qo, muse_rows Ko, muse_stream_t st) {
  const muse_status s = check_shape(d, false);
  if (s != MUSE_OK) return s;
  if (!valid_rows(Q, d.dtype) || !valid_rows(Qo, d.dtype) || !pos) return MUSE_ERR_INVALID_ARG;
  if (K.p) {
    if (!valid_rows(K, d.dtype) || !valid_rows(Ko, d.dtype)) return MUSE_ERR_INVALID_ARG;
    if (Hk <= 0 || (int64_t)d.B * Hk > 65535) return MUSE_ERR_SHAPE;
  } else {
    Hk = 0;
  }
  if (pos_batches != 1 && pos_batches != d.B) return MUSE_ERR_SHAPE;
  RopeTable t;
  if (!rope_table(r, d.D, t)) return MUSE_ERR_INVALID_ARG;
  return launched(run_rope(Q, K, Hk, d, pos, pos_batches, t, Qo, Ko, (cudaStream_t)st));
}

extern "C" size_t muse_cache_tile_bytes(int D, int Dv) {
  return (D == 64 || D == 128) && (Dv == 64 || Dv == 128) ? (size_t)18 * (D + Dv) : 0;
}

static muse_status check_cache_rows(const muse_rows &K, const muse_rows &V, const muse_dims &d,
                                    const muse_cache &c, const int32_t *start) {
  muse_status s = check_shape(d, true);
  if (s != MUSE_OK) return s;
  if (!valid_rows(K, d.dtype) || !valid_rows(V, d.dtype) || !start) return MUSE_ERR_INVALID_ARG;
  if (d.H != c.Hkv) return MUSE_ERR_SHAPE;
  return check_cache(c, d);
}

extern "C" muse_status muse_cache_write(muse_rows K, muse_rows V, muse_dims d, muse_cache c,
                                        const int32_t *start, const int32_t *counts,
                                        muse_stream_t st) {
  const muse_status s = check_cache_rows(K, V, d, c, start);
  if (s != MUSE_OK) return s;
  return launched(run_cache_write(K, V, d, c, start, counts, device_status_word(),
                                  (cudaStream_t)st));
}

extern "C" muse_status muse_cache_read(muse_dims d, muse_cache c, const int32_t *start,
                                       const int32_t *counts, muse_rows K, muse_rows V,
                                       muse_stream_t st) {
  const muse_status s = check_cache_rows(K, V, d, c, start);
  if (s != MUSE_OK) return s;
  return launched(run_cache_read(d, c, start, counts, K, V, device_status_word(),
                                 (cudaStream_t)st));
}

extern "C" muse_status muse_cache_attend(muse_rows Q, muse_dims d, muse_cache c,
                                         const int32_t *lens, const int32_t *counts, muse_rows O,
                                         float *lse, void *ws, size_t ws_bytes, muse_stream_t st) {
  muse_status s = check_shape(d, true);
  if (s != MUSE_OK) return s;
  if (!isfinite(d.scale)) return MUSE_ERR_INVALID_ARG;
  if (!valid_rows(Q, d.dtype) || !valid_rows(O, d.dtype) || !lens) return MUSE_ERR_INVALID_ARG;
  if (d.N > MUSE_CACHE_MAX_ROWS || c.Hkv <= 0 || d.H % c.Hkv) return MUSE_ERR_SHAPE;
  s = check_cache(c, d);
  if (s != MUSE_OK) return s;
  if (!ws || ws_bytes < cache_attend_ws(d, c.Hkv) || !aligned16(ws)) return MUSE_ERR_WORKSPACE;
  return launched(run_cache_attend(Q, d, c, lens, counts, O, lse, ws, device_status_word(),
                                   (cudaStream_t)st));
}
