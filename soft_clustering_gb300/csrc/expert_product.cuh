// expert_product.cuh - workspace and row tiles of the experts' products.
#pragma once

#include "expert_internal.cuh"

namespace gmm {

constexpr int kLeastTile = 64;  // fewest rows of a tile in any kernel's list

__host__ __device__ inline int64_t clamp_row(int64_t v, int64_t R) {
  return v < 0 ? 0 : v > R ? R : v;
}

// dW has a tile for every component and 128 x 256 of its matrix, each a sum
// over all the component's rows.  Where those are fewer than four a
// multiprocessor and the sums long, a component's rows are cut into stretches
// with a partial sum each, added in order afterwards: about this many
// stretches in all.  Cut and joined against whole: 522711 rows to 22
// components of 64 x 128 76 us (406), 200000 to 16 of 512 x 256 90 (189),
// 1000001 to 256 of 128 x 128 126 (128); but 16385 to 8 of 1024 x 1024 57
// (40): hence kDwLong rows a component.
constexpr int kDwTiles = 4 * 152, kDwLong = 4096;
inline int dw_stretches(int d_in, int d_out) {
  const int64_t tiles = (int64_t)((d_out + 127) / 128) * ((d_in + 255) / 256);
  return tiles > kDwTiles ? 0 : (int)(kDwTiles / tiles);
}
// Rows of a stretch; 0: components are not cut.
inline int64_t dw_stretch_rows(int64_t R, int d_in, int d_out, int K) {
  const int n = dw_stretches(d_in, d_out);
  if (n <= K || R < (int64_t)kDwLong * K) return 0;
  const int64_t each = (R + (n - K) - 1) / (n - K);
  const int64_t rows = each < 256 ? 256 : (each + 63) / 64 * 64;
  return rows < R ? rows : 0;
}

// What the tensor-core forms take, as far as types and widths say.
inline bool tc_widths_ok(int xdtype, int d_in, int d_out) {
  return xdtype != GMM_F32 && d_in % 8 == 0 && d_out % 8 == 0;
}

struct ProductLayout {
  size_t off_count, off_first, off_tiles, off_part, bytes;  // the DeviceStatus comes first
  // row tiles of K components and of the rows past them
  static int64_t most_tiles(int64_t R, int K, int T) { return R / T + K + 1; }
  static ProductLayout make(int64_t R, int d_in, int d_out, int K, int xdtype) {
    ProductLayout L;
    size_t o = align_up(sizeof(DeviceStatus));
    L.off_count = o; o = align_up(o + sizeof(int32_t));
    L.off_first = o; o = align_up(o + sizeof(uint32_t) * ((size_t)K + 2));
    L.off_tiles = o; o = align_up(o + sizeof(int4) * (size_t)most_tiles(R, K, kLeastTile));
    L.off_part = o;
    if (tc_widths_ok(xdtype, d_in, d_out) && dw_stretch_rows(R, d_in, d_out, K) > 0)
      o = align_up(o + sizeof(float) * (size_t)d_in * d_out * (dw_stretches(d_in, d_out) + 1));
    L.bytes = o;
    return L;
  }
};

// Fills the tile list {component or -1, first row, rows, 0}, its length and
// each component's first tile.
gmm_status list_tiles(const int64_t* offsets, int K, int64_t R, int T, void* ws,
                      const ProductLayout& L, cudaStream_t s);


// The tensor-core forms (expert_product_tc.cu) and what they take.
bool tc_product_ok(int xdtype, int64_t R, int d_in, int d_out, const void* a, const void* b, const void* c);
gmm_status tc_rows(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_from,
                   int d_to, int K, bool dx, const int64_t* offsets, void* ws, cudaStream_t s);
// ... and the one for few rows, 16-bit types as above.  Experts of 1024 x 2048
// in bf16, a call: 16 rows over 64 components 14.2 us, 32 rows 22.3 (the
// tensor-core form 19.0 and 25.4); 64 rows 35.1 (33.8); 32 rows over 8
// components, several to a component, 21.7 (15.8).  The rule sees the numbers
// and not the offsets: 32 rows of which all are one component's, of 64, take
// 29.7 us (33 rows on the tensor cores 13.6).  Its blocks count the offsets
// themselves, 256 at a time: worth it for a few thousand components.
inline bool few_rows(int64_t R, int K) { return R > 0 && R <= 32 && R <= 2 * (int64_t)K && K <= 4096; }
gmm_status few_rows_product(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_in,
                            int d_out, int K, const int64_t* offsets, cudaStream_t s);
gmm_status tc_weights(const void* dY, const void* A, int xdtype, int64_t R, int d_in, int d_out,
                      int K, const int64_t* offsets, void* dW, int wdtype, void* ws,
                      cudaStream_t s);

}  // namespace gmm
