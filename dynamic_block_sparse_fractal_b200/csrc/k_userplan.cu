// A plan from the caller's own block mask: each q-block row of bytes becomes the
// keep bitmap, count and ascending list that the select and radius kernels
// write. Bound by the mask's bytes and the lists (nb^2 bytes read, up to 4 nb^2
// written per head); one warp per row, a word of the bitmap per ballot, four
// words' loads in flight.
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace sa {

__global__ void __launch_bounds__(256)
    mask_rows_kernel(const uint8_t* __restrict__ mask, size_t head_stride,
                     uint32_t* __restrict__ bits, int32_t* __restrict__ cnt,
                     int32_t* __restrict__ idx, Geometry g) {
  const int lane = threadIdx.x & 31;
  const long row = long(blockIdx.x) * 8 + (threadIdx.x >> 5);  // (bh, q-block)
  if (row >= long(g.BH) * g.nb) return;
  const int bh = int(row / g.nb), qb = int(row - long(bh) * g.nb);
  const uint8_t* src = mask + size_t(bh) * head_stride + size_t(qb) * g.nb;
  const int words = bitmap_words(g);
  uint32_t* b = bits + size_t(row) * words;
  int32_t* out = idx + size_t(row) * g.nb;
  int n = 0;
  for (int w0 = 0; w0 < words; w0 += 4) {
    uint8_t x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = 32 * (w0 + u) + lane;
      x[u] = j < g.nb ? __ldg(src + j) : uint8_t(0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (w0 + u >= words) break;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, x[u] != 0);
      if (x[u] != 0) out[n + __popc(m & ((1u << lane) - 1u))] = 32 * (w0 + u) + lane;
      if (lane == 0) b[w0 + u] = m;
      n += __popc(m);
    }
  }
  if (lane == 0) cnt[row] = n;
}

cudaError_t launch_mask_rows(const uint8_t* mask, size_t head_stride, uint32_t* bits, int32_t* cnt,
                             int32_t* idx, const Geometry& g, cudaStream_t stream) {
  const long rows = long(g.BH) * g.nb;
  mask_rows_kernel<<<unsigned((rows + 7) / 8), 256, 0, stream>>>(mask, head_stride, bits, cnt, idx,
                                                                 g);
  return cudaGetLastError();
}

}  // namespace sa
