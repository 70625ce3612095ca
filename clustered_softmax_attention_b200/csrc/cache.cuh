// The 4-bit cache as the kernels see it: where a tile lies and where a token's words are in it
// (layout: include/muse.h).
#pragma once

#include "internal.h"

namespace muse {

constexpr int kTile = 32;  // tokens of a tile

struct CacheView {
  uint8_t *tiles;
  const int32_t *table;
  int pages, Hkv, page_log2, max_pages;
};

inline CacheView cache_view(const muse_cache &c) {
  CacheView v;
  v.tiles = static_cast<uint8_t *>(c.tiles);
  v.table = c.page_table;
  v.pages = c.pages;
  v.Hkv = c.Hkv;
  v.page_log2 = 31 - __builtin_clz((unsigned)c.page);
  v.max_pages = c.max_pages;
  return v;
}

template <int D, int Dv>
struct TileShape {
  static constexpr int kK = 0;                    // byte offsets in a tile
  static constexpr int kV = 16 * D;
  static constexpr int kKStep = 16 * (D + Dv);
  static constexpr int kVStep = kKStep + 2 * D;
  static constexpr int kBytes = 18 * (D + Dv);
};

// Tile of tokens [32 T, 32 T + 32) of sequence b, head h; NULL when the table has no such
// place or names a page outside the cache.
__device__ __forceinline__ uint8_t *cache_tile(const CacheView &v, int b, int h, int T,
                                               int tile_bytes) {
  const int slot = (int)(((int64_t)T * kTile) >> v.page_log2);
  if (T < 0 || slot >= v.max_pages) return nullptr;
  const int pg = v.table[(int64_t)b * v.max_pages + slot];
  if ((unsigned)pg >= (unsigned)v.pages) return nullptr;
  const int per = 1 << (v.page_log2 - 5);
  const int64_t t = ((int64_t)pg * v.Hkv + h) * per + (T & (per - 1));
  return v.tiles + t * tile_bytes;
}

// Word of token t (0..31) that holds key channels 32 w + 8 q + (0..7).
template <int D>
__device__ __forceinline__ int key_word(int t, int q, int w) {
  return D == 128 ? t * 16 + q * 4 + w
                  : (t >> 4) * 128 + (t & 7) * 16 + q * 4 + ((t >> 3) & 1) * 2 + w;
}
// Word of token t that holds value channels 64 w + g + 8 (0..7) (w = 0 for Dv = 64).
template <int Dv>
__device__ __forceinline__ int value_word(int t, int g, int w) {
  return Dv == 128 ? (t >> 3) * 128 + g * 16 + ((t & 7) >> 1) * 4 + (t & 1) * 2 + w
                   : (t >> 4) * 128 + g * 16 + ((t & 7) >> 1) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
}
// The token that a word of the key codes, or of the value codes, belongs to.
template <int D>
__device__ __forceinline__ int key_word_token(int i) {
  return D == 128 ? i >> 4 : (i >> 7) * 16 + ((i >> 1) & 1) * 8 + ((i >> 4) & 7);
}
template <int Dv>
__device__ __forceinline__ int value_word_token(int i) {
  return Dv == 128 ? (i >> 7) * 8 + ((i >> 2) & 3) * 2 + ((i >> 1) & 1)
                   : (i >> 7) * 16 + ((i >> 1) & 1) * 8 + ((i >> 2) & 3) * 2 + (i & 1);
}

// Code n (0..7) of a word as a float: exact.
__device__ __forceinline__ float code_value(uint32_t w, int n) {
  return __uint_as_float(0x4B000000u | ((w >> (4 * n)) & 15u)) - 8388616.f;
}
__device__ __forceinline__ float step_value(uint16_t bits) {
  return __uint_as_float((uint32_t)bits << 16);
}

// Rows of one sequence that a write or a read takes: [0, count), token start + row.
__device__ __forceinline__ int row_count(const int32_t *counts, int b, int N, int *status) {
  if (!counts) return N;
  const int c = counts[b];
  if (c < 0 || c > N) report(status, MUSE_ERR_DEVICE);
  return min(max(c, 0), N);
}

}  // namespace muse
