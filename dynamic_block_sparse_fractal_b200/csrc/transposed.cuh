// The transposed block lists of the gradient kernels.
#pragma once
#include <cuda_runtime.h>

#include "layout.cuh"

namespace sa {

// One warp for unit = (bh, key tile): scan every q-block's keep bitmap for the
// tile's two k-blocks (the query-tile pairing applied to keys) and compact the
// q-blocks keeping either, ascending.
__device__ __forceinline__ void transposed_list(const uint32_t* __restrict__ bits,
                                                int32_t* __restrict__ kcnt,
                                                int32_t* __restrict__ kidx, const Geometry& g,
                                                long unit) {
  const int lane = threadIdx.x & 31;
  if (unit >= long(g.BH) * g.ntile) return;
  const int bh = int(unit / g.ntile), tile = int(unit - long(bh) * g.ntile);
  int ka, kb;
  tile_blocks(g, tile, ka, kb);
  const int words = bitmap_words(g);
  const uint32_t* rows = bits + size_t(bh) * g.nb * words;
  int32_t* out = kidx + size_t(unit) * g.nb;
  int n = 0;
  for (int i0 = 0; i0 < g.nb; i0 += 32) {
    const int i = i0 + lane;
    bool a = false, b = false;
    if (i < g.nb) {
      a = (rows[size_t(i) * words + (ka >> 5)] >> (ka & 31)) & 1u;
      if (kb >= 0) b = (rows[size_t(i) * words + (kb >> 5)] >> (kb & 31)) & 1u;
    }
    const unsigned m = __ballot_sync(0xFFFFFFFFu, a || b);
    if (a || b)
      out[n + __popc(m & ((1u << lane) - 1u))] =
          i | (a ? kEntryKeepA : 0) | (b ? kEntryKeepB : 0);
    n += __popc(m);
  }
  if (lane == 0) kcnt[unit] = n;
}

}  // namespace sa
