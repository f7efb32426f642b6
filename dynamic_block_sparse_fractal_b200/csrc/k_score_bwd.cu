// Gradients of the block-sparse attention with another score function: a
// learned relative position bias (one map) or differential attention (two maps
// that share the values, out = (P_1 - lambda P_2) V).
//
// With z the scores, P_m = 2^(z_m - lse_m) from the forward's row statistics,
// dP = dO V^T and D_m = rowsum(dO * P_m V):
//   dV = Pc^T dO            Pc = P (bias), P_1 - lambda P_2 (differential)
//   dS_1 = P_1 (dP - D_1),  dS_2 = -lambda P_2 (dP - D_2)
//   dQ_m = dS_m K_m * scale, dK_m = dS_m^T Q_m * scale
//   dtable[b] = sum of dS over the pairs in bucket b;  dlambda = -sum D_2
//
// Two tensor-core passes that each rebuild P and dP, instead of one pass that
// reduces dQ into memory: the query pass keeps a query tile and runs over its
// union list (dQ), the key pass keeps a key tile and runs over the q-blocks that
// keep it (dK, dV, dtable). Two products and the exponentials are done twice (8
// units of 2 N^2 d per kept pair instead of 5), but there are no atomics on dQ
// (the same bits at every run) and no fp32 accumulator to clear, reduce into and
// convert, and TMEM has room for two stages of scores, so that the products of
// one step run while the row warps work on the other.
//
// D. rowsum(dO * O) of a stored bf16 output carries its rounding, and the error
// of D is common to a whole row of dS. The query pass therefore starts from that
// value D~ (dS~ = P (dP - D~)) and sums D = rowsum(P * dP) in fp32 on the way; the
// key pass reads that D. For dQ one more product, P K, sets a row right: a row of
// dS sums to 0, so with R = the sum of the row's dS~ as rounded to bf16, dQ = dS~ K
// - R P K. That takes out D~'s error and the part of the roundings that lies along
// the row's mean key, which is the largest where keys share a component. (2-norm
// error of dQ against 64 bits, bf16 outputs: 4.5e-3 with D~ alone, 2.9e-3 with D,
// 2.2e-3 with R; the bf16 rounding of dQ itself is 1.7e-3. Gradients of the table
// and of lambda: up to 7e-3 with D~, 2e-3 with D.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "exp2_poly.cuh"
#include "relbias.cuh"
#include "transposed.cuh"
#include "sm100.cuh"

namespace sa {

namespace {

constexpr int kSbThreads = 640;   // warps 0, 2 TMA, 1, 3 MMA; 4-19 rows
constexpr int kSbRowWarps = 16;   // two groups of 8: the even and the odd steps; in a group two
                                  // warpgroups of 128 rows, half of a step's columns each
constexpr int kSbList = 2880;     // list entries staged in shared memory (the rest from L2)
constexpr int kSbSlots = 4;       // ring of streamed blocks (3 in the key pass with a table)
constexpr int kTile = 128 * 128;  // 128 rows x 128 B (64 bf16 channels)
constexpr int kBlk = 64 * 128;    // 64 rows x 128 B
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void fail_s(uint32_t* status, int* abort, uint32_t bit) {
  atomicOr(status, bit);
  *reinterpret_cast<volatile int*>(abort) = 1;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// One arrival for a warp whose lanes have all finished their TMEM accesses
// (tcgen05.wait before the call).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A and B both K-major, one accumulator of 128 x N: NK K steps of 16 channels
// from step k0 on; a_chunk / b_chunk bytes between 64-channel chunks.
template <int NK>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint64_t a, uint32_t a_chunk,
                                           uint64_t b, uint32_t b_chunk, uint32_t id, int k0) {
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) {
    const int ks = k0 + kk;
    const uint32_t in = uint32_t(ks & 3) * 32u;
    mma_ss(d_tmem, a + ((uint32_t(ks >> 2) * a_chunk + in) >> 4),
           b + ((uint32_t(ks >> 2) * b_chunk + in) >> 4), id, kk > 0);
  }
}

// A from TMEM, NK K steps 16 columns apart; B an MN-major block (16 rows a step).
template <int NK>
__device__ __forceinline__ void mma_from_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                              uint32_t id, uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < NK; ++kk)
    mma_ts(d_tmem, a_tmem + uint32_t(kk) * 16u, b + uint64_t(kk) * 128u, id, kk > 0 ? 1u : acc);
}

// mul * (32 accumulator columns of this lane's row, kFix: less fix * 32 columns at
// `sub`; zeros without a step) -> 32 elements of an output, bf16 or fp32.
template <bool kFix>
__device__ __forceinline__ void store_acc32(uint32_t col, uint32_t sub, bool any, float mul,
                                            float fix, void* out, size_t at, int fp32) {
  float x[32];
  if (any) {
    uint32_t o[32];
    tmem_ld32(col, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
    if constexpr (kFix) {
      tmem_ld32(sub, o);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = fmaf(-fix, __uint_as_float(o[i]), x[i]);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] *= mul;
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.f;
  }
  if (fp32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int v = 0; v < 8; ++v)
      dst[v] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      dst[v] = make_uint4(pack_bf16x2(x[8 * v], x[8 * v + 1]),
                          pack_bf16x2(x[8 * v + 2], x[8 * v + 3]),
                          pack_bf16x2(x[8 * v + 4], x[8 * v + 5]),
                          pack_bf16x2(x[8 * v + 6], x[8 * v + 7]));
  }
}

// TMEM column, relative to a [128 x d] accumulator, of output channel c (a
// multiple of 32): with two maps of 32 channels each map's product is taken over
// all 64 channels of the block, 64 columns apart, and half of it is used.
template <int D, bool kDiff>
__device__ __forceinline__ uint32_t acc_col(int c) {
  return uint32_t(kDiff && D == 64 && c >= 32 ? 64 + c : c);
}

// The bias of a row warp's 32 columns of a block, c = 32 wg + ..: with L =
// min(log2 pw, 5) it is f[c >> L] + g[c & (2^L - 1)], f from the time and row
// tables and g from the column table.
template <int L>
struct Cols {
  static constexpr int kG = 1 << L, kF = 32 >> L;
};

template <int L>
__device__ __forceinline__ int f_run(const Geometry& g, int wg, int x) {
  return (32 * wg + x * Cols<L>::kG) >> g.lpw;
}
template <int L>
__device__ __forceinline__ int g_col(const Geometry& g, int wg, int y) {
  return (32 * wg + y) & (g.pw - 1);
}

template <int L>
__device__ __forceinline__ void load_bias32(const float* bias, const Geometry& g, int t, int h,
                                            int w, int wg, int sign, float (&f)[Cols<L>::kF],
                                            float (&c)[Cols<L>::kG]) {
#pragma unroll
  for (int x = 0; x < Cols<L>::kF; ++x) {
    const int run = f_run<L>(g, wg, x);
    f[x] = bias[t + sign * (run >> g.lph)] + bias[h + sign * (run & (g.ph - 1))];
  }
#pragma unroll
  for (int y = 0; y < Cols<L>::kG; ++y) c[y] = bias[w + sign * g_col<L>(g, wg, y)];
}

// Sums N values of each lane over the lanes that differ in lane bits [LO, HI):
// while more than one value is left a bit halves them between the two lanes,
// after that it sums. Returns how many are left in v[0..); `first` is the index
// of v[0] among the N, and `writer` is false where another lane holds the same.
template <int N, int LO, int HI>
__device__ __forceinline__ int lane_sums(float (&v)[N], int lane, int& first, bool& writer) {
  int n = N;
  first = 0;
  writer = true;
#pragma unroll
  for (int bit = HI - 1; bit >= LO; --bit) {
    const bool up = (lane >> bit) & 1;
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        if (k < n) {
          const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
          v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 1 << bit);
        }
      }
      first += up ? n : 0;
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 1 << bit);
      writer = writer && !up;
    }
  }
  return n;
}

// dS of this thread's key against 32 query columns of a block, already summed
// over each run (f) and each column (c), added to the warp's own histogram over
// offsets (h, w: the block's indexes in it), for blocks of one frame with rows of
// 8 (the 8 x 8 patch); add_table_grad below is the same for the others. A warp holds
// 4 rows x 8 columns of keys against 4 rows x 8 columns of queries: 1 + 7 + 15
// offsets. The sums over one axis are brought together along their diagonals by
// shuffles, so that one addition to the histogram, each lane at an address of its
// own, ends the step. The frame offset's sum stays in a register (tsum, at index
// tcur) until another frame comes, which the ascending list makes rare.
__device__ __forceinline__ void add_table_grad_patch(float* hist, int h, int w, int wg, int lane,
                                                     const float (&f)[4], const float (&c)[8]) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  // rows: lane 8 a + 2 x holds the sum over the columns of key row a, query row x
  const bool u2 = lane & 4, u1 = lane & 2, u4 = lane & 16;
  const float a0 = (u2 ? f[2] : f[0]) + __shfl_xor_sync(kAll, u2 ? f[0] : f[2], 4);
  const float a1 = (u2 ? f[3] : f[1]) + __shfl_xor_sync(kAll, u2 ? f[1] : f[3], 4);
  float v = (u1 ? a1 : a0) + __shfl_xor_sync(kAll, u1 ? a0 : a1, 2);
  v += __shfl_xor_sync(kAll, v, 1);
  // columns: bit 4 halves the 8 sums (query columns 4 up ..), bit 3 is summed over;
  // then a half-warp's sums run along their diagonal, one lane on at each addition:
  // lane p of half up holds the offset p - 3 - 4 up
  float r = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x = (u4 ? c[k + 4] : c[k]) + __shfl_xor_sync(kAll, u4 ? c[k] : c[k + 4], 16);
    x += __shfl_xor_sync(kAll, x, 8);
    if (k > 0) {
      r = __shfl_up_sync(kAll, r, 1, 16);
      if ((lane & 15) == 0) r = 0.f;
    }
    if (!(lane & 8)) r += x;
  }
  // lane p < 7: row offset p - 3; lanes 8 .. 22: column offset lane - 15
  float s = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int a = lane - 3 + x;
    const float y = __shfl_sync(kAll, v, (8 * a + 2 * x) & 31);
    if (a >= 0 && a < 4) s += y;
  }
  const int o = lane - 8;
  const float lo = __shfl_sync(kAll, r, (o - 4) & 15), hi = __shfl_sync(kAll, r, 16 + (o & 15));
  if (lane >= 8) s = (o >= 4 ? lo : 0.f) + (o <= 10 ? hi : 0.f);
  // h, w: this lane's indexes for query row and column 0 (key row lane >> 3, column lane & 7)
  const int at = lane < 8 ? h - 4 * wg + lane - 3 : w - (lane & 7) + o - 7;
  if (lane != 7 && o <= 14) hist[at] += s;
  __syncwarp();
}

// The same for any block shape (t, h, w: the block's indexes in the histogram).
// Lanes of a warp are 32 tokens of one block: their low L bits are the column.
// Lanes that share an address sum first; then one group of lanes at a time adds
// one of its values, at addresses that all differ, so that no atomics are needed
// (histograms shared by the CTA's warps with atomic additions took 4,500 cycles a
// step, three times the step's products). A lane's next value meets its
// neighbour's last address: the warp synchronises between values. Blocks of
// several frames can still meet at an address and add atomically.
template <int L>
__device__ __forceinline__ void add_table_grad(float* hist, const Geometry& g, int t, int h, int w,
                                               int wg, int lane, float (&f)[Cols<L>::kF],
                                               float (&c)[Cols<L>::kG]) {
  constexpr int NG = Cols<L>::kG, NF = Cols<L>::kF;
  if (g.pt == 1) {  // one frame offset for the whole warp
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < NF; ++x) s += f[x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) hist[t] += s;
  }
  int first;
  bool writer;
  int n = lane_sums<NF, 0, L>(f, lane, first, writer);  // lanes of one row run
  if (g.pt == 1) {
    // lanes of equal column bits are different rows of the block
    constexpr int kStep = NF >= 1 << L ? 1 : (1 << L) / NF;  // (the others are no writers)
    for (int q = 0; q < 1 << L; q += kStep) {
      const bool mine = writer && (lane & ((1 << L) - 1)) == q;
#pragma unroll
      for (int k = 0; k < NF; ++k) {
        if (k >= n) break;
        if (mine) hist[h - (f_run<L>(g, wg, first + k) & (g.ph - 1))] += f[k];
        __syncwarp();
      }
    }
  } else if (writer) {
#pragma unroll
    for (int k = 0; k < NF; ++k) {
      if (k >= n) break;
      const int run = f_run<L>(g, wg, first + k);
      atomicAdd(hist + t - (run >> g.lph), f[k]);
      atomicAdd(hist + h - (run & (g.ph - 1)), f[k]);
    }
  }
  __syncwarp();
  n = lane_sums<NG, L, 5>(c, lane, first, writer);  // lanes of one column
#pragma unroll
  for (int q = 0; q < 32 >> L; ++q) {  // lanes of one row run: different columns
    const bool mine = writer && (lane >> L) == q;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      if (k >= n) break;
      if (mine) hist[w - g_col<L>(g, wg, first + k)] += c[k];
      __syncwarp();
    }
  }
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t f2_bf16(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint64_t f2_ex2(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return f2_pack(ex2_approx(lo), ex2_approx(hi));
}
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}

// What a CTA of either pass streams and waits on.
struct SbBars {
  uint64_t tile_full, full[kSbSlots], empty[kSbSlots];
  uint64_t s_full[2], out_full[2], x_done[2], y_done[2], acc_full, dsum_full, drain[2];
  uint32_t tmem_base;
  int abort;
};

template <int D, int kSlots>
struct __align__(1024) SbSmem {
  uint8_t ta[D / 64][kTile], tb[D / 64][kTile];               // the tile's K, V (or Q, dO)
  uint8_t sa[kSlots][D / 64][kBlk], sb[kSlots][D / 64][kBlk];  // streamed Q, dO (or K, V)
  float nlse[kSbSlots][2][64], ndsum[kSbSlots][2][64];        // of streamed query rows, per map
  float sums[2][2][4][128];  // query pass: four warps' parts of a row's D and R, per map
  int32_t list[kSbList];
  SbBars bar;
};
// Floats of one row warp's histogram: the offsets between a token of one block
// and any token, per axis.
SA_HD int hist_floats(const Geometry& g) {
  return (g.T + g.pt - 1) + (g.Hh + g.ph - 1) + (g.Ww + g.pw - 1);
}
// with the offset tables and the 16 histograms of the largest grid (pt + ph + pw
// <= 66), a CTA's 227 KB
static_assert(sizeof(SbSmem<128, 3>) + 1024 + sizeof(float) * (2 * kRelBiasMaxAxes - 3) +
                      16 * sizeof(float) * (kRelBiasMaxAxes + 63) <= kSmemLimit,
              "shared memory of the key pass");
static_assert(sizeof(SbSmem<128, 4>) + 1024 + sizeof(float) * (2 * kRelBiasMaxAxes - 3) <= kSmemLimit,
              "shared memory of the query pass");

}  // namespace

// -D_m and -lse_m * log2(e) of every row into fractal order (negated: both are
// addends; an empty row's lse = -inf stays -inf, so that 2^(z - lse) is 0). D/8 lanes per row, 32 rows
// per CTA, one head per CTA. The CTAs behind those make the transposed lists (see
// transposed_list), which need nothing from them: one launch less.
constexpr int kPrepRows = 32;

template <int D, bool kDiff>
__global__ void __launch_bounds__(256)
    score_prep_kernel(const void* __restrict__ o, const void* __restrict__ o2,
                      const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse,
                      const __nv_bfloat16* __restrict__ lam, int H, float* __restrict__ nlse,
                      float* __restrict__ ndsum, int fp32, int row_ctas,
                      const uint32_t* __restrict__ bits, int32_t* __restrict__ kcnt,
                      int32_t* __restrict__ kidx, Geometry g) {
  wait_for_stream();
  const int per_head = (g.S + kPrepRows - 1) / kPrepRows;
  if (int(blockIdx.x) >= row_ctas) {
    transposed_list(bits, kcnt, kidx, g, long(int(blockIdx.x) - row_ctas) * 8 + (threadIdx.x >> 5));
    return;
  }
  constexpr int kLanes = D / 8;
  const int sub = threadIdx.x % kLanes, bh = int(blockIdx.x) / per_head;
  const size_t all = size_t(g.BH) * g.S;
  const float lm = kDiff ? __bfloat162float(lam[bh % H]) : 0.f;
  for (int i = threadIdx.x / kLanes; i < kPrepRows; i += 256 / kLanes) {
    const int pos = (int(blockIdx.x) - bh * per_head) * kPrepRows + i;
    if (pos >= g.S) break;
    const size_t row = size_t(bh) * g.S + block_row_token(g, pos >> 6, pos & 63);
    const size_t at = row * D + 8 * sub;
    const uint4 dv = __ldg(reinterpret_cast<const uint4*>(dout + at));
    auto dot = [&](const void* p) {
      float acc = 0.f;
      const uint32_t* dw = &dv.x;
      if (fp32) {
        const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = __ldg(x), b = __ldg(x + 1);
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 d = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(dw + w));
          acc += d.x * y[2 * w] + d.y * y[2 * w + 1];
        }
      } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
        const uint32_t* xw = &x.x;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 d = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(dw + w));
          const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(xw + w));
          acc += d.x * y.x + d.y * y.y;
        }
      }
      return acc;
    };
    float d1 = dot(o), d2 = kDiff ? dot(o2) : 0.f;
    const unsigned mask = __activemask();  // whole groups of kLanes lanes
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) {
      d1 += __shfl_xor_sync(mask, d1, s);
      if (kDiff) d2 += __shfl_xor_sync(mask, d2, s);
    }
    if (sub == 0) {
      const size_t dst = size_t(bh) * g.S + pos;
#pragma unroll
      for (int m = 0; m < (kDiff ? 2 : 1); ++m) {
        const float l = lse[m * all + row];
        nlse[m * all + dst] = l == -INFINITY ? l : -l * kLog2e;
      }
      ndsum[dst] = kDiff ? -fmaf(lm, d2, d1) : -d1;  // out = O_1 - lambda O_2
      if (kDiff) ndsum[all + dst] = -d2;
    }
  }
}

// One pass over a tile of 128 rows (two blocks of one head): kQ = true, the
// query pass (rows are queries; Q and dO stay, K and V stream; -> dQ and D), or
// the key pass (rows are keys; K and V stay, Q, dO and their row statistics
// stream; -> dK, dV and the table's gradient). Rows are TMEM lanes in both:
//   S_m = A1_m B1_m^T, dP = A2 B2^T      (A1, A2 the tile's, B1, B2 a block's)
//   row warps: P_m and dS_m as bf16 over S and dP in TMEM
//   Y_m += dS_m B1_m                     (dQ or dK)
//   X  += Pc B2 (key pass: dV), X_m += P_m B1_m (query pass: P K)
// A step is W columns of a streamed block (64 with one map, 32 with two), in one
// of two TMEM stages; the row warps of group s work on stage s, so that one
// group's loads, stores and waits lie beside the other's exponentials.
// TMEM columns: X 0, Y 128, the stages at 256 and 384: S_1, (S_2,) dP, W each. A
// row thread owns 16-column chunks: P_m goes into the first 8 columns of its own
// chunk of S_m (key pass: Pc over S_1), dS_1 and dS_2 into the two halves of dP's,
// so nobody overwrites what another warp has still to read.
template <int D, AttnMode M, int L, bool kQ>
__global__ void __launch_bounds__(kSbThreads, 1)
    score_bwd_kernel(const __grid_constant__ ScoreBwdArgs a, const Geometry g) {
  constexpr bool kDiff = M == AttnMode::kDiff, kTable = !kDiff && !kQ;
  constexpr int NM = kDiff ? 2 : 1;
  constexpr int W = kDiff ? 32 : 64, kHalves = 64 / W;  // columns of a step, steps of a block
  constexpr int kSlots = kTable ? 3 : kSbSlots;
  using Smem = SbSmem<D, kSlots>;
  constexpr uint32_t kColX = 0, kColY = 128, kStage0 = 256, kStage = 128, kDP = W * NM;
  extern __shared__ uint8_t sb_raw[];
  // (an offset, not an address rounded up: the compiler then knows shared memory)
  Smem& sm = *reinterpret_cast<Smem*>(sb_raw + ((0u - smem_u32(sb_raw)) & 1023u));
  SbBars& br = sm.bar;
  float* bias = reinterpret_cast<float*>(&sm + 1);
  const int noff = relbias_offsets(g);
  float* hist = bias + noff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    br.abort = 0;
    mbar_init(&br.tile_full, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&br.full[s], 2);
      mbar_init(&br.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&br.s_full[s], 1);
      mbar_init(&br.out_full[s], kSbRowWarps / 2);
      mbar_init(&br.x_done[s], 1);
      mbar_init(&br.y_done[s], 1);
      mbar_init(&br.drain[s], 1);
    }
    mbar_init(&br.acc_full, 1);
    mbar_init(&br.dsum_full, kSbRowWarps);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&br.tmem_base, 512);
    tmem_relinquish();
  }
  wait_for_stream();

  // CTAs start heaviest tile first over a group of heads (see launch_pass)
  const int first_head = int(blockIdx.x) / (a.group * g.ntile) * a.group;
  const int heads = min(a.group, g.BH - first_head);
  const int in_group = int(blockIdx.x) - first_head * g.ntile;
  const int bh = first_head + in_group % heads;
  const int32_t* order = kQ ? a.order : a.korder;
  const int tile = order == nullptr ? in_group / heads
                                    : order[size_t(bh) * g.ntile + in_group / heads];
  int ba, bb;  // the tile's blocks (bb = -1: a lone block)
  tile_blocks(g, tile, ba, bb);
  const size_t unit = size_t(bh) * g.ntile + tile;
  const int nblk = kQ ? a.tcnt[unit] : a.kcnt[unit];
  const int n = nblk * kHalves;
  const int32_t* glist = (kQ ? a.tidx : a.kidx) + unit * g.nb;
  for (int i = threadIdx.x; i < nblk && i < kSbList; i += kSbThreads) sm.list[i] = glist[i];
  auto at = [&](int i) -> int { return i < kSbList ? sm.list[i] : __ldg(glist + i); };
  if constexpr (!kDiff) relbias_load(bias, a.bias, g, bh, threadIdx.x, kSbThreads, a.status);
  if constexpr (kTable)
    for (int i = threadIdx.x; i < kSbRowWarps * hist_floats(g); i += kSbThreads) hist[i] = 0.f;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, br.tmem_base, 0);
  volatile int* abort = &br.abort;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers
    // warp 0: the tile, then B1 (and the row statistics); warp 2: B2
    if (lane == 0 && nblk > 0) {
      const CUtensorMap* map =
          kQ ? (warp == 0 ? &a.map_k : &a.map_v) : (warp == 0 ? &a.map_q : &a.map_do);
      prefetch_tensormap(map);
      if (warp == 0) {
        mbar_arrive_expect_tx(&br.tile_full, 2u * 128u * D * 2u);
        for (int e = 0; e < 2; ++e) {
          const int blk = (e == 0 || bb < 0) ? ba : bb;  // a lone block: its copy fills the rest
          int t, hp, wp;
          block_coords(g, blk, t, hp, wp);
          for (int c = 0; c < D / 64; ++c) {
            tma_load_5d(&sm.ta[c][e * kBlk], kQ ? &a.map_q : &a.map_k, &br.tile_full, c * 64,
                        wp * g.pw, hp * g.ph, t * g.pt, bh);
            tma_load_5d(&sm.tb[c][e * kBlk], kQ ? &a.map_do : &a.map_v, &br.tile_full, c * 64,
                        wp * g.pw, hp * g.ph, t * g.pt, bh);
          }
        }
      }
      int last = -1;
      for (int j = 0; j < nblk; ++j) {
        const int s = j % kSlots;
        if (j >= kSlots && !mbar_wait(&br.empty[s], (j / kSlots - 1) & 1, abort)) {
          fail_s(a.status, &br.abort, kDevErrTimeoutLoad);
          break;
        }
        if (*abort) break;
        if (j == 0 && warp == 0 && (a.debug_flags & SA_DEBUG_STALL_LOADER)) continue;  // test hook
        int blk = at(j) & kEntryBlockMask;
        if (blk >= g.nb) {
          atomicOr(a.status, kDevErrBadIndex);
          blk = 0;
        }
        int t, hp, wp;
        block_coords(g, blk, t, hp, wp);
        mbar_arrive_expect_tx(&br.full[s],
                              64u * D * 2u + (!kQ && warp == 0 ? uint32_t(NM) * 512u : 0u));
        for (int c = 0; c < D / 64; ++c)
          tma_load_5d(warp == 0 ? &sm.sa[s][c][0] : &sm.sb[s][c][0], map, &br.full[s], c * 64,
                      wp * g.pw, hp * g.ph, t * g.pt, bh);
        if (!kQ && warp == 0) {
          for (int m = 0; m < NM; ++m) {
            const size_t off = (size_t(m) * g.BH + bh) * g.S + size_t(blk) * 64;
            bulk_load(&sm.nlse[s][m][0], a.nlse + off, 256u, &br.full[s]);
            bulk_load(&sm.ndsum[s][m][0], a.ndsum + off, 256u, &br.full[s]);
          }
        }
        last = j;
      }
      if (*abort) {
        // let the copies land before the CTA can exit (time-bounded, ignoring
        // the abort flag): at most the last use of each slot is open
        int never = 0;
        if (warp == 0) mbar_wait(&br.tile_full, 0, &never);
        for (int jj = last; jj >= 0 && jj > last - kSlots; --jj)
          mbar_wait(&br.full[jj % kSlots], (jj / kSlots) & 1, &never);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ MMA
    // Warp 3 issues a step's scores, warp 1 its products X and Y. The scores of step i
    // overwrite the P and dS that X and Y of step i - 2 read, in another MMA shape, and
    // only MMAs of one shape and accumulator are ordered by being issued one after the
    // other: S waits for X to have completed and dP for Y, while the products of step
    // i - 1 go out beside that wait. (One commit for X and Y together: 1,040 us where
    // this takes 980, differential, 12 x 8,192 tokens.) Each warp walks the steps as a
    // whole, so that the loop's values are uniform (the descriptors stay in uniform
    // registers); one elected lane issues.
    if (nblk > 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(128, W, 0, 0);
      constexpr uint32_t id_y = idesc_bf16_f32(128, kDiff ? 64 : D, 0, 1);
      constexpr uint32_t id_x = kQ ? id_y : idesc_bf16_f32(128, D, 0, 1);
      constexpr uint32_t kSlot = (D / 64) * kBlk / 16;   // a slot in descriptor units
      constexpr uint32_t kHalf = W * 128 / 16;           // W rows of a block
      constexpr uint32_t kMap = D == 128 ? kBlk / 16 : 0;  // a map's channels of a block
      const uint64_t b1 = sw128_desc(smem_u32(&sm.sa[0][0][0]), 16, 1024);
      const uint64_t b2 = sw128_desc(smem_u32(&sm.sb[0][0][0]), 16, 1024);
      auto where = [&](int i) -> uint64_t {
        return uint64_t((i / kHalves) % kSlots) * kSlot + uint64_t(i % kHalves) * kHalf;
      };
      auto block_here = [&](int i) {  // the streamed block of step i
        const int j = i / kHalves;
        return i % kHalves != 0 || mbar_wait(&br.full[j % kSlots], (j / kSlots) & 1, abort);
      };
      const bool one = elect_one();
      bool ok = true;
      if (warp == 3) {
        const uint64_t a1 = sw128_desc(smem_u32(&sm.ta[0][0]), 16, 1024);
        const uint64_t a2 = sw128_desc(smem_u32(&sm.tb[0][0]), 16, 1024);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&br.tile_full, 0, abort));
        for (int i = 0; ok && i < n; ++i) {  // S and dP of step i
          const uint32_t before = ((i >> 1) - 1) & 1;  // the stage's last step
          ok = block_here(i) && (i < 2 || mbar_wait(&br.x_done[i & 1], before, abort));
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t st = tmem + kStage0 + kStage * uint32_t(i & 1);
          if (one) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
              mma_scores<D / 16 / NM>(st + W * m, a1, kTile, b1 + where(i), kBlk, id_s,
                                      m * (D / 16 / NM));
          }
          __syncwarp();
          ok = __all_sync(0xFFFFFFFFu, i < 2 || mbar_wait(&br.y_done[i & 1], before, abort));
          if (!ok) break;
          tc_fence_after_sync();
          if (one) {
            mma_scores<D / 16>(st + kDP, a2, kTile, b2 + where(i), kBlk, id_s, 0);
            mma_commit(&br.s_full[i & 1]);
          }
          __syncwarp();
        }
      } else {
        const uint64_t b1_mn = sw128_desc(smem_u32(&sm.sa[0][0][0]), kBlk, 1024);
        const uint64_t b2_mn = sw128_desc(smem_u32(&sm.sb[0][0][0]), kBlk, 1024);
        for (int i = 0; ok && i < n; ++i) {  // X and Y of step i
          ok = block_here(i) && mbar_wait(&br.out_full[i & 1], (i >> 1) & 1, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after_sync();
          if (one) {
            const uint32_t st = tmem + kStage0 + kStage * uint32_t(i & 1);
            const uint32_t acc = i > 0 ? 1u : 0u;
#pragma unroll
            for (int m = 0; m < (kQ ? NM : 1); ++m) {
              if (kQ)
                mma_from_tmem<W / 16>(tmem + kColX + 64u * m, st + W * m,
                                      b1_mn + where(i) + m * kMap, id_x, acc);
              else
                mma_from_tmem<W / 16>(tmem + kColX, st, b2_mn + where(i), id_x, acc);
            }
            mma_commit(&br.x_done[i & 1]);
#pragma unroll
            for (int m = 0; m < NM; ++m)
              mma_from_tmem<W / 16>(tmem + kColY + 64u * m, st + kDP + 8u * m,
                                    b1_mn + where(i) + m * kMap, id_y, acc);
            mma_commit(&br.y_done[i & 1]);
            if ((i + 1) % kHalves == 0) mma_commit(&br.empty[(i / kHalves) % kSlots]);
          }
          __syncwarp();
        }
        if (ok && one) mma_commit(&br.acc_full);
      }
      if (!ok) {
        fail_s(a.status, &br.abort, kDevErrTimeoutMma);
        if (one) mma_commit(&br.drain[warp >> 1]);  // wait (bounded) for the MMAs issued before exit
        int never = 0;
        mbar_wait(&br.drain[warp >> 1], 0, &never);
      }
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------------- rows
    const int part = (warp - 4) >> 2;              // 0..3
    const int grp = part >> 1, wg = part & 1;      // steps of parity grp, half wg of the columns
    const int quad = warp & 3;
    const int r = quad * 32 + lane;                // TMEM lane: a row of the tile
    const uint32_t lane_base = tmem + (uint32_t(quad * 32) << 16);
    const bool valid = r < 64 || bb >= 0;          // uniform across the warp
    const int blk = r < 64 || bb < 0 ? ba : bb;
    const int my_keep = !valid ? 0 : r < 64 ? kEntryKeepA : kEntryKeepB;
    const uint64_t sl2x2 = f2_pack(a.scale_log2, a.scale_log2);
    const float lam = kDiff ? __bfloat162float(a.lam[bh % a.H]) : 0.f;
    const uint64_t nlam2 = f2_pack(-lam, -lam);
    const size_t my_pos = size_t(bh) * g.S + size_t(blk) * 64 + (r & 63);
    float nlse[NM], ndsum[NM];  // query pass: this row's
    uint64_t dfull2[NM], rsum2[NM];  // sums of P dP, and of dS as rounded
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      nlse[m] = kQ ? a.nlse[size_t(m) * g.BH * g.S + my_pos] : 0.f;
      ndsum[m] = kQ ? a.ndsum[size_t(m) * g.BH * g.S + my_pos] : 0.f;
      dfull2[m] = rsum2[m] = 0ull;
    }
    constexpr int kSign = kQ ? 1 : -1;
    constexpr int kG = Cols<L>::kG, kF = Cols<L>::kF;
    RelBiasRow rb;
    float* my_hist = hist + (warp - 4) * hist_floats(g);
    int to_h = 0, to_w = 0, to_t = 0;  // from an offset's index in the tables to the histogram's
    if constexpr (!kDiff) {
      rb = relbias_row(g, blk, r & 63, kSign);
      int t, hp, wp;
      block_coords(g, blk, t, hp, wp);
      to_t = t * g.pt;
      to_h = g.T - g.pt + hp * g.ph;
      to_w = (g.T - g.pt) + (g.Hh - g.ph) + wp * g.pw;
    }
    float tsum = 0.f;
    int tcur = to_t;
    auto flush_t = [&]() {
      float x = tsum;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      if (lane == 0) my_hist[tcur - to_t] += x;
      __syncwarp();
      tsum = 0.f;
    };
    const uint32_t st = lane_base + kStage0 + kStage * uint32_t(grp);
    bool ok = true;
    for (int i = grp; i < n; i += 2) {
      const int j = i / kHalves, s = j % kSlots;
      const int ent = at(j);
      const bool keep = (ent & my_keep) != 0;  // uniform across the warp
      // the bias of this thread's columns, while the scores are computed: f per
      // run, c per column in pairs (query pass: the row's -lse with it)
      float f[kF], c[kG];
      int it = 0, ih = 0, iw = 0;
      if constexpr (!kDiff) {
        if (keep) {
          relbias_block(g, rb, ent & kEntryBlockMask, kSign, it, ih, iw);
          load_bias32<L>(bias, g, it, ih, iw, wg, kSign, f, c);
          if (kQ) {
#pragma unroll
            for (int y = 0; y < kG; ++y) c[y] += nlse[0];
          }
        }
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&br.s_full[grp], (i >> 1) & 1, abort) &&
                                       (kQ || mbar_wait(&br.full[s], (j / kSlots) & 1, abort)));
      if (!ok) break;
      tc_fence_after_sync();
      uint64_t gf2[kF], gc2[(kG + 1) / 2];
      if constexpr (kTable) {
#pragma unroll
        for (int x = 0; x < kF; ++x) gf2[x] = 0ull;
#pragma unroll
        for (int y = 0; y < (kG + 1) / 2; ++y) gc2[y] = 0ull;
      }
#pragma unroll
      for (int ch = 0; ch < W / 32; ++ch) {
        const int col = (W / 2) * wg + 16 * ch;                   // in the stage
        const int qcol = (kDiff ? 32 * (i % kHalves) : 0) + col;  // in the streamed block
        uint32_t pk[NM][8], ds[NM][8];
        if (keep) {
          uint32_t x[NM][16], dp[16];
#pragma unroll
          for (int m = 0; m < NM; ++m) tmem_ld16(st + W * m + col, x[m]);
          tmem_ld16(st + kDP + col, dp);
          tmem_wait_ld();
#pragma unroll
          for (int k4 = 0; k4 < 16; k4 += 4) {
            uint64_t nls[NM][2], nds[NM][2];  // -lse and -D of four columns
            if (!kQ) {
#pragma unroll
              for (int m = 0; m < NM; ++m) {
                const float4 l = *reinterpret_cast<const float4*>(&sm.nlse[s][m][qcol + k4]);
                const float4 d = *reinterpret_cast<const float4*>(&sm.ndsum[s][m][qcol + k4]);
                nls[m][0] = f2_pack(l.x, l.y);
                nls[m][1] = f2_pack(l.z, l.w);
                nds[m][0] = f2_pack(d.x, d.y);
                nds[m][1] = f2_pack(d.z, d.w);
              }
            }
#pragma unroll
            for (int k = k4; k < k4 + 4; k += 2) {
              const uint64_t e2 = f2_pack(__uint_as_float(dp[k]), __uint_as_float(dp[k + 1]));
              uint64_t p2[NM];
#pragma unroll
              for (int m = 0; m < NM; ++m) {
                uint64_t nl2, nd2;
                if (kQ) {
                  nl2 = f2_pack(nlse[m], nlse[m]);
                  nd2 = f2_pack(ndsum[m], ndsum[m]);
                } else {
                  nl2 = nls[m][(k - k4) / 2];
                  nd2 = nds[m][(k - k4) / 2];
                }
                if constexpr (!kDiff) {
                  const int q = 16 * ch + k;
                  const uint64_t f2 = f2_pack(f[q / kG], f[(q + 1) / kG]);
                  const uint64_t c2 = f2_pack(c[q % kG], c[(q + 1) % kG]);
                  nl2 = kQ ? f2_add(f2, c2) : f2_add(f2_add(f2, c2), nl2);
                }
                p2[m] = f2_ex2(f2_fma(
                    f2_pack(__uint_as_float(x[m][k]), __uint_as_float(x[m][k + 1])), sl2x2, nl2));
                if (kQ) dfull2[m] = f2_fma(p2[m], e2, dfull2[m]);
                // (map 2: -lambda is applied to the finished dQ_2 and dK_2)
                const uint64_t d2 = f2_mul(p2[m], f2_add(e2, nd2));
                const uint32_t d16 = f2_bf16(d2);
                ds[m][k / 2] = d16;
                if (kQ)
                  rsum2[m] = f2_add(rsum2[m], f2_pack(__uint_as_float(d16 << 16),
                                                      __uint_as_float(d16 & 0xFFFF0000u)));
                if constexpr (kTable) {
                  const int q = 16 * ch + k;
                  gf2[kG > 1 ? q / kG : q / 2] = f2_add(gf2[kG > 1 ? q / kG : q / 2], d2);
                  gc2[(q % kG) / 2] = f2_add(gc2[(q % kG) / 2], d2);
                }
              }
              if constexpr (kDiff && !kQ) {
                pk[0][k / 2] = f2_bf16(f2_fma(nlam2, p2[NM - 1], p2[0]));
              } else {
#pragma unroll
                for (int m = 0; m < NM; ++m) pk[m][k / 2] = f2_bf16(p2[m]);
              }
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int m = 0; m < NM; ++m) pk[m][k] = ds[m][k] = 0u;
        }
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          if (kQ || m == 0) tmem_st8(st + W * m + col, pk[m]);
          tmem_st8(st + kDP + col + 8 * m, ds[m]);
        }
      }
      tmem_wait_st();
      warp_arrive(&br.out_full[grp], lane);
      if constexpr (kTable) {
        if (keep) {
#pragma unroll
          for (int x = 0; x < kF; ++x) {
            float lo, hi;
            f2_unpack(gf2[kG > 1 ? x : x / 2], lo, hi);
            f[x] = kG > 1 ? lo + hi : (x & 1 ? hi : lo);
          }
#pragma unroll
          for (int y = 0; y < kG; ++y) {
            float lo, hi;
            f2_unpack(gc2[y / 2], lo, hi);
            c[y] = kG == 1 ? lo + hi : (y & 1 ? hi : lo);
          }
          if constexpr (L == 3) {
            if (g.pt == 1) {
              if (it != tcur) {  // uniform across the warp
                flush_t();
                tcur = it;
              }
              tsum += (f[0] + f[1]) + (f[2] + f[3]);
              add_table_grad_patch(my_hist, ih - to_h, iw - to_w, wg, lane, f, c);
            } else {
              add_table_grad<L>(my_hist, g, it - to_t, ih - to_h, iw - to_w, wg, lane, f, c);
            }
          } else {
            add_table_grad<L>(my_hist, g, it - to_t, ih - to_h, iw - to_w, wg, lane, f, c);
          }
        }
      }
    }
    if constexpr (kTable && L == 3) flush_t();
    float dfull[NM], rsum[NM];
    if (kQ && ok) {
      // four warps' partial sums of every row, in a fixed order
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        sm.sums[0][m][part][r] = f2_sum(dfull2[m]);
        sm.sums[1][m][part][r] = f2_sum(rsum2[m]);
      }
      warp_arrive(&br.dsum_full, lane);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&br.dsum_full, 0, abort));
      if (ok) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          const auto& d = sm.sums[0][m];
          const auto& x = sm.sums[1][m];
          dfull[m] = (d[0][r] + d[1][r]) + (d[2][r] + d[3][r]);
          rsum[m] = (x[0][r] + x[1][r]) + (x[2][r] + x[3][r]);
        }
      }
    }
    if (!ok) {
      fail_s(a.status, &br.abort, kDevErrTimeoutSoftmax);
    } else if (valid) {  // uniform across the warp
      if (kQ && part == 0) {
#pragma unroll
        for (int m = 0; m < NM; ++m) a.ndsum[size_t(m) * g.BH * g.S + my_pos] = -dfull[m];
      }
      if (32 * part < D) {
        if (n > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&br.acc_full, 0, abort))) {
          fail_s(a.status, &br.abort, kDevErrTimeoutSoftmax);
        } else {
          if (n > 0) tc_fence_after_sync();
          const int c = 32 * part;
          const size_t dst = (size_t(bh) * g.S + block_row_token(g, blk, r & 63)) * D + c;
          const uint32_t y = lane_base + kColY + acc_col<D, kDiff>(c);
          const bool second = kDiff && c >= D / 2;
          const float mul = second ? -lam * a.scale : a.scale;  // dS_2 = -lambda P_2 (dP - D_2)
          if constexpr (kQ) {
            const float fix = second ? rsum[NM - 1] : rsum[0];
            store_acc32<true>(y, lane_base + kColX + acc_col<D, kDiff>(c), n > 0, mul, fix, a.dq, dst,
                        a.out_fp32);
          } else {
            store_acc32<false>(lane_base + kColX + c, 0u, n > 0, 1.f, 0.f, a.dv, dst, a.out_fp32);
            store_acc32<false>(y, 0u, n > 0, mul, 0.f, a.dk, dst, a.out_fp32);
          }
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if constexpr (kTable) {
    // the 16 warps' histograms (8 per block of the tile) joined in a fixed order
    float* dst = a.part + unit * noff;
    int o[2][3];  // table index - histogram index, per block and axis
    for (int e = 0; e < 2; ++e) {
      int t, hp, wp;
      block_coords(g, e == 0 || bb < 0 ? ba : bb, t, hp, wp);
      o[e][0] = t * g.pt;
      o[e][1] = g.T - g.pt + hp * g.ph;
      o[e][2] = (g.T - g.pt) + (g.Hh - g.ph) + wp * g.pw;
    }
    const int nt = g.T + g.pt - 1, nh = g.Hh + g.ph - 1, per = hist_floats(g);
    for (int i = threadIdx.x; i < noff; i += kSbThreads) {
      const int axis = i < 2 * g.T - 1 ? 0 : i < 2 * g.T - 1 + 2 * g.Hh - 1 ? 1 : 2;
      const int lo = axis == 0 ? 0 : axis == 1 ? nt : nt + nh;
      const int hi = axis == 0 ? nt : axis == 1 ? nt + nh : per;
      float sum = 0.f;
      for (int w = 0; w < kSbRowWarps; ++w) {
        const int k = i - o[(w & 3) >> 1][axis];  // quads 2 and 3 are the second block
        if (k >= lo && k < hi) sum += hist[w * per + k];
      }
      dst[i] = sum;
    }
  }
}

// dtable: per head, the tiles' partial sums over offsets (part [BH][ntile][noff])
// added over batch and tiles, a group of threads per share of the tiles, then over
// the offsets of each bucket, a warp per bucket; all in a fixed order. One CTA per
// head.
__global__ void __launch_bounds__(1024)
    dtable_kernel(const float* __restrict__ part, BiasArgs b, int B, void* __restrict__ dtable,
                  int fp32, Geometry g) {
  __shared__ float sums[2 * kRelBiasMaxAxes], red[1024];
  wait_for_stream();
  const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int noff = relbias_offsets(g);
  for (int o0 = 0; o0 < noff; o0 += 1024) {
    const int here = min(noff - o0, 1024), groups = 1024 / here;
    const int grp = threadIdx.x / here, o = threadIdx.x - grp * here;
    float s = 0.f;
    if (grp < groups) {
      for (int e = 0; e < B; ++e) {
        const float* src = part + (size_t(e) * b.H + h) * g.ntile * noff + o0 + o;
#pragma unroll 8
        for (int t = grp; t < g.ntile; t += groups) s += src[size_t(t) * noff];
      }
      red[threadIdx.x] = s;
    }
    __syncthreads();
    if (int(threadIdx.x) < here) {
      s = 0.f;
      for (int k = 0; k < groups; ++k) s += red[k * here + threadIdx.x];
      sums[o0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
  for (int k = warp; k < b.n_buckets; k += 32) {
    float s = 0.f;
    for (int i = lane; i < noff; i += 32) {
      int bk = __ldg(b.bucket + i);
      if (bk < 0 || bk >= b.n_buckets) bk = 0;  // as the kernels read it
      if (bk == k) s += sums[i];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    const size_t at = size_t(h) * b.n_buckets + k;
    if (lane == 0) {
      if (fp32) static_cast<float*>(dtable)[at] = s;
      else static_cast<__nv_bfloat16*>(dtable)[at] = __float2bfloat16_rn(s);
    }
  }
}

// dlambda[h] = sum of -D_2 (ndsum's second map, [BH][S]) over the batch and the
// rows, in a fixed order. One CTA per head.
__global__ void __launch_bounds__(1024)
    dlambda_kernel(const float* __restrict__ d2, int S, int B, int H, void* __restrict__ dlam,
                   int fp32) {
  __shared__ float red[32];
  wait_for_stream();
  const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float s = 0.f;
  for (int e = 0; e < B; ++e) {
    const float4* src = reinterpret_cast<const float4*>(d2 + (size_t(e) * H + h) * S);
#pragma unroll 4
    for (int i = threadIdx.x; i < S / 4; i += 1024) {
      const float4 x = __ldg(src + i);
      s += (x.x + x.y) + (x.z + x.w);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = red[lane];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    if (lane == 0) {
      if (fp32) static_cast<float*>(dlam)[h] = s;
      else static_cast<__nv_bfloat16*>(dlam)[h] = __float2bfloat16_rn(s);
    }
  }
}

// Heads whose tiles are dealt out together, heaviest first: as many as keep q, k,
// v and dO within 64 MB, half of L2. One head at a time leaves SMs idle behind
// the last head's heaviest tiles where heads are short (key pass, 12 heads of
// 8,192 tokens: 424 us in the tiles' own order); all heads at once would stream
// their blocks from HBM where they are long.
static int head_group(const Geometry& g) {
  const size_t head = size_t(4) * g.S * g.d * 2;
  const size_t n = (size_t(64) << 20) / head;
  return n < 1 ? 1 : n > size_t(g.BH) ? g.BH : int(n);
}

template <int D, AttnMode M, int L, bool kQ>
static cudaError_t launch_pass(const ScoreBwdArgs& a, const Geometry& g, cudaStream_t stream) {
  // the offset tables, and in the key pass the histogram behind them; at least
  // 120 KB, since each CTA allocates all 512 TMEM columns
  constexpr bool kTable = M != AttnMode::kDiff && !kQ;
  const size_t tables =
      M == AttnMode::kDiff
          ? 0
          : sizeof(float) * (relbias_offsets(g) + (kTable ? kSbRowWarps * hist_floats(g) : 0));
  const size_t need = sizeof(SbSmem<D, kTable ? 3 : kSbSlots>) + 1024 + tables;
  const int smem = int(need > 120 * 1024 ? need : 120 * 1024);
  // (the limit belongs to the process: the same for every grid, as in the forward)
  cudaError_t e = cudaFuncSetAttribute(score_bwd_kernel<D, M, L, kQ>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_early(score_bwd_kernel<D, M, L, kQ>, unsigned(g.ntile) * unsigned(g.BH),
                      kSbThreads, smem, stream, a, g);
}

template <int D, AttnMode M, int L>
static cudaError_t launch_passes(const ScoreBwdArgs& a, const Geometry& g, cudaStream_t stream) {
  const cudaError_t e = launch_pass<D, M, L, true>(a, g, stream);  // first: it corrects D
  return e != cudaSuccess ? e : launch_pass<D, M, L, false>(a, g, stream);
}

template <int D>
static cudaError_t launch_score_bwd_d(const ScoreBwdArgs& a, const Geometry& g,
                                      cudaStream_t stream) {
  if (a.lam != nullptr) return launch_passes<D, AttnMode::kDiff, 0>(a, g, stream);
  switch (g.lpw < 5 ? g.lpw : 5) {  // columns of a block that are one run of w
    case 0: return launch_passes<D, AttnMode::kBias, 0>(a, g, stream);
    case 1: return launch_passes<D, AttnMode::kBias, 1>(a, g, stream);
    case 2: return launch_passes<D, AttnMode::kBias, 2>(a, g, stream);
    case 3: return launch_passes<D, AttnMode::kBias, 3>(a, g, stream);
    case 4: return launch_passes<D, AttnMode::kBias, 4>(a, g, stream);
    default: return launch_passes<D, AttnMode::kBias, 5>(a, g, stream);
  }
}

cudaError_t launch_score_bwd(ScoreBwdArgs a, const Geometry& g, cudaStream_t stream) {
  a.group = head_group(g);
  const int row_ctas = (g.S + kPrepRows - 1) / kPrepRows * g.BH;
  const unsigned grid = unsigned(row_ctas) + unsigned((long(g.BH) * g.ntile + 7) / 8);
  const bool diff = a.lam != nullptr;
  cudaError_t e;
#define SA_PREP(D, DIFF)                                                                         \
  e = launch_early(score_prep_kernel<D, DIFF>, grid, 256, 0, stream, a.out, a.out2, a.dout, a.lse, \
                   a.lam, a.H, a.nlse, a.ndsum, a.out_fp32, row_ctas, a.bits, a.kcnt, a.kidx, g)
  if (g.d == 128) {
    if (diff) SA_PREP(128, true); else SA_PREP(128, false);
  } else {
    if (diff) SA_PREP(64, true); else SA_PREP(64, false);
  }
#undef SA_PREP
  // (no order where every key tile starts at once)
  if (long(g.ntile) * g.BH <= 148) a.korder = nullptr;
  else if (e == cudaSuccess) e = launch_tile_order(a.kcnt, a.korder, g, stream);
  if (e == cudaSuccess)
    e = g.d == 128 ? launch_score_bwd_d<128>(a, g, stream) : launch_score_bwd_d<64>(a, g, stream);
  if (e != cudaSuccess) return e;
  if (diff)
    return launch_early(dlambda_kernel, unsigned(a.H), 1024, 0, stream,
                        a.ndsum + size_t(g.BH) * g.S, g.S, g.BH / a.H, a.H, a.dparam, a.out_fp32);
  return launch_early(dtable_kernel, unsigned(a.H), 1024, 0, stream, a.part, a.bias, g.BH / a.H,
                      a.dparam, a.out_fp32, g);
}

}  // namespace sa
