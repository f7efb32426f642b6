// Learned relative position bias of a (query, key) pair as the attention
// kernels read it: bias = b_t[t_k - t_q] + b_h[h_k - h_q] + b_w[w_k - w_q], the
// three offset tables of the CTA's head expanded into shared memory in log2
// units. The coordinates are bit fields of a token's row in its block, so a
// block of 64 tokens with pw = 8 needs 8 values of b_t + b_h and 8 of b_w per
// thread, not 64.
#pragma once
#include <cuda_bf16.h>

#include "exp2_poly.cuh"
#include "kernels.cuh"
#include "sm100.cuh"

namespace sa {

// A table entry at or below this masks its offsets (the lowest finite value of
// the type, -inf): kept as -inf, so that no later rounding tells them apart.
constexpr float kRelBiasMasked = -1e30f;

__device__ __forceinline__ void relbias_load(float* dst, const BiasArgs& b, const Geometry& g,
                                             int bh, int tid, int threads, uint32_t* status) {
  const __nv_bfloat16* row = b.table + size_t(bh % b.H) * b.n_buckets;
  const int n = relbias_offsets(g);
  for (int i = tid; i < n; i += threads) {
    int k = __ldg(b.bucket + i);
    if (k < 0 || k >= b.n_buckets) {
      atomicOr(status, kDevErrBadIndex);
      k = 0;
    }
    const float v = __bfloat162float(row[k]);
    dst[i] = v <= kRelBiasMasked ? -INFINITY : v * 1.4426950408889634f;
  }
}

// One token's side of the offsets: indexes into the tables (or a histogram of
// the same layout) for a partner at coordinate 0. sign = +1: the thread's token
// is the query and the partners are keys; -1: the thread's token is the key.
struct RelBiasRow {
  int t, h, w;      // index of a partner at coordinate 0 along each axis
  uint32_t mf, mw;  // multipliers that divide a block id by nh * nw, and by nw
};

// n / d = umulhi(n, magic(d)) for n < 2^16, 1 < d < 2^16; 0 stands for d = 1.
__device__ __forceinline__ uint32_t div_magic(int d) {
  return d == 1 ? 0u : 0xFFFFFFFFu / uint32_t(d) + 1u;
}
__device__ __forceinline__ int div_by(int n, uint32_t m) {
  return m == 0u ? n : int(__umulhi(uint32_t(n), m));
}

__device__ __forceinline__ RelBiasRow relbias_row(const Geometry& g, int blk, int i, int sign) {
  RelBiasRow r;
  r.mf = div_magic(g.nh * g.nw);
  r.mw = div_magic(g.nw);
  int t, hp, wp;
  block_coords(g, blk < 0 ? 0 : blk, t, hp, wp);
  const int run = i >> g.lpw;
  r.t = g.T - 1 - sign * (t * g.pt + (run >> g.lph));
  r.h = 2 * g.T - 1 + g.Hh - 1 - sign * (hp * g.ph + (run & (g.ph - 1)));
  r.w = 2 * g.T - 1 + 2 * g.Hh - 1 + g.Ww - 1 - sign * (wp * g.pw + (i & (g.pw - 1)));
  return r;
}

// Indexes for partner 0 of block kb: the partner (dt, dh, dw) tokens further
// into the block is at t + sign dt, h + sign dh, w + sign dw.
__device__ __forceinline__ void relbias_block(const Geometry& g, const RelBiasRow& r, int kb,
                                              int sign, int& t, int& h, int& w) {
  kb = kb < g.nb ? kb : 0;  // as the loader reads, and reports, a list entry out of range
  const int tb = div_by(kb, r.mf);
  const int rest = kb - tb * (g.nh * g.nw);
  const int hb = div_by(rest, r.mw);
  t = r.t + sign * (tb * g.pt);
  h = r.h + sign * (hb * g.ph);
  w = r.w + sign * ((rest - hb * g.nw) * g.pw);
}

// The bias of 64 keys of block kb whose rows are 2^L tokens (pw == 2^L): f[a] of
// each row of the block, g of its columns in pairs.
template <int L>
struct BlockBias {
  static constexpr int kRows = 64 >> L, kPairs = (1 << L) / 2;
  float f[kRows];
  uint64_t g[kPairs];

  __device__ __forceinline__ void load(const float* bias, const RelBiasRow& r, const Geometry& geo,
                                       int kb) {
    int t, h, w;
    relbias_block(geo, r, kb, 1, t, h, w);
#pragma unroll
    for (int a = 0; a < kRows; ++a) f[a] = bias[t + (a >> geo.lph)] + bias[h + (a & (geo.ph - 1))];
#pragma unroll
    for (int c = 0; c < kPairs; ++c) g[c] = f2_pack(bias[w + 2 * c], bias[w + 2 * c + 1]);
  }

  // x[i] = x[i] * sl2 + g for those 64 keys (raw scores in, log2 units less f out);
  // returns the largest x + f.
  __device__ __forceinline__ float add_cols(float sl2, uint32_t* x) const {
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    float top = -INFINITY;
#pragma unroll
    for (int a = 0; a < kRows; ++a) {
      float m = -INFINITY;
#pragma unroll
      for (int c = 0; c < kPairs; ++c) {
        const int i = (a << L) + 2 * c;
        const uint64_t y =
            f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sl2x2, g[c]);
        float y0, y1;
        f2_unpack(y, y0, y1);
        x[i] = __float_as_uint(y0);
        x[i + 1] = __float_as_uint(y1);
        m = max3(m, y0, y1);
      }
      top = fmaxf(top, m + f[a]);
    }
    return top;
  }
};

// x[i] = x[i] * sl2 + bias for the 64 keys of block kb, any block shape.
__device__ __forceinline__ void relbias_add64(const float* bias, const RelBiasRow& r,
                                              const Geometry& g, int kb, float sl2, uint32_t* x) {
  int t, h, w;
  relbias_block(g, r, kb, 1, t, h, w);
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int run = i >> g.lpw;
    const float b = bias[t + (run >> g.lph)] + bias[h + (run & (g.ph - 1))] +
                    bias[w + (i & (g.pw - 1))];
    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), sl2, b));
  }
}

}  // namespace sa
