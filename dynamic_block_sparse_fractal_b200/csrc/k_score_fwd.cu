// Block-sparse attention forward with another score function over the planned
// blocks: a learned relative position bias (O = softmax(z + b) V), or differential
// attention (O = (P_1 - lambda P_2) V, the maps of the two halves of the channels).
//
// A CTA runs two chains, A and B, of 128 query rows each: two query tiles (bias),
// the halves of one tile's list (bias, few tiles) or the two maps of one tile
// (differential). A step of a chain is one 64-key block:
//   S_X(j) = Q_X K^T   (M = 128, N = 64)      -> TMEM, two stages per chain
//   softmax warps of X: online softmax in fp32 (exp2 domain), P over S as bf16
//   O_X += P V         (K = 64)
// Two stages let the tensor core compute S_X(j + 1) while the softmax warps work
// on S_X(j): their chain load - maximum - exponentials - store is what bounds the
// kernel (the SFU's 16 exponentials per cycle and SM alone are 1,024 cycles for a
// step of both chains, the products 930 (differential) or 1,330 (bias); a step of
// a chain takes about 2,000). One stage of 128 keys per chain, as the plain kernel
// has it, took 2.10 ms where this takes 1.70 (differential, 4 heads of 61,440
// tokens) and 1.82 ms where this takes 1.44 to 1.55 (bias, 12 x 37,632).
//
//   warps 0, 2     TMA producers, one 16 KB ring slot per block of K or V, in the
//                  order the MMA warps consume them: a ring per chain (bias), or one
//                  that the maps share
//   warps 1, 3     one issues A's products and the other B's, a step at a time:
//                  PV_X(j), then S_X(j + 2) into the stage that it frees
//   warps 4-7, 8-11  softmax of chain A and B, one thread per query row
//
// S_X(j + 2) overwrites the P of step j. Only MMAs of one shape and accumulator are
// ordered by being issued one after the other, so it goes out after PV_X(j)'s commit
// has arrived; the other chain's products fill that wait, which is why the chains
// have a warp each (one warp for both, waiting: 250 and 350 us where two take 208
// and 290; bias and differential, 12 x 8,192 tokens). So S_X(j) complete means
// PV_X(j - 2) is; a rescale of O at step j waits for PV_X(j - 1). All waits are
// bounded; one that runs out records a status bit and raises the CTA's abort flag.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "exp2_poly.cuh"
#include "kernels.cuh"
#include "relbias.cuh"
#include "sm100.cuh"

namespace sa {

namespace {

constexpr int kFThreads = 384;
constexpr int kFSlots = 8;
constexpr int kFTile = 128 * 128;  // 128 rows x 128 B (64 bf16 channels)
constexpr int kFBlk = 64 * 128;    // 64 rows x 128 B
constexpr int kFList = 2880;       // union entries staged per chain (the rest from L2)
constexpr float kFRescale = 8.0f;  // log2 units

template <int D>
struct __align__(1024) ScoreFwdSmem {
  uint8_t q[2][D / 64][kFTile];
  uint8_t slot[kFSlots][D / 64][kFBlk];
  int32_t list[2][kFList];
  float m[2][128], l[2][128];  // row statistics of A and B where their outputs join
  uint64_t q_full[2], full[kFSlots], empty[kFSlots];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_final[2], join, drain[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(ScoreFwdSmem<128>) + 1024 + sizeof(float) * (2 * kRelBiasMaxAxes - 3) <=
                  kSmemLimit,
              "shared memory of the forward");

// Slot of ring position k: the differential chains share a ring of all slots, the
// others have half of them each.
template <bool kShared>
__device__ __forceinline__ int ring_slot(int x, int k) {
  return kShared ? k % kFSlots : x * (kFSlots / 2) + k % (kFSlots / 2);
}

template <int V>
struct Which {
  static constexpr int value = V;
};

struct Chain {
  int qa, qb;            // q-blocks (qb = -1: lone block)
  int n;                 // steps
  int first;             // list entry of step 0
  const int32_t* list;   // shared-memory copy of the first kFList entries
  const int32_t* glist;  // global memory
  __device__ __forceinline__ int at(int j) const {
    const int i = first + j;
    return i < kFList ? list[i] : __ldg(glist + i);
  }
};

__device__ __forceinline__ void fail_f(uint32_t* status, int* abort, uint32_t bit) {
  atomicOr(status, bit);
  *reinterpret_cast<volatile int*>(abort) = 1;
}

// 32 columns of O times `w`, or zeros when the chain ran no step.
__device__ __forceinline__ void load_o32(uint32_t col, int n, float w, float (&x)[32]) {
  if (n > 0) {
    uint32_t o[32];
    tmem_ld32(col, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]) * w;
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.f;
  }
}

// 32 values -> elements [at, at + 32) of an output, bf16 or fp32.
__device__ __forceinline__ void store_o32(void* out, size_t at, const float (&x)[32], int fp32) {
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

}  // namespace

// L: log2 of the tokens in a row of a block where the bias is taken row by row
// and column by column (24 values for the 64 keys at L = 3, held in registers);
// kAnyShape: three lookups per key (284 us against 122 for 12 x 5,760 tokens in
// blocks that both can take).
constexpr int kAnyShape = -1;

template <int D, AttnMode M, int L>
__global__ void __launch_bounds__(kFThreads, 1)
    score_fwd_kernel(const __grid_constant__ ScoreFwdArgs a, const Geometry g) {
  constexpr bool kDiff = M == AttnMode::kDiff, kRows = !kDiff && L != kAnyShape;
  const bool split = !kDiff && a.split;
  const bool one_tile = kDiff || split;
  constexpr int kRing = kDiff ? kFSlots : kFSlots / 2;
  extern __shared__ uint8_t sf_raw[];
  // (an offset, not an address rounded up: the compiler then knows shared memory)
  ScoreFwdSmem<D>& sm =
      *reinterpret_cast<ScoreFwdSmem<D>*>(sf_raw + ((0u - smem_u32(sf_raw)) & 1023u));
  float* bias = reinterpret_cast<float*>(&sm + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y;

  volatile int* abort = &sm.abort;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.q_full[x], 1);
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sm.s_full[x][s], 1);
        mbar_init(&sm.p_full[x][s], 4);  // one arrival per softmax warp
      }
      mbar_init(&sm.pv_done[x], 1);
      mbar_init(&sm.o_final[x], 1);
    }
    for (int s = 0; s < kFSlots; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kDiff ? 2 : 1);  // the maps share a slot
    }
    mbar_init(&sm.join, 256);
    for (int x = 0; x < 2; ++x) mbar_init(&sm.drain[x], 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  wait_for_stream();

  Chain chain[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int pos = one_tile ? int(blockIdx.x) : 2 * int(blockIdx.x) + x;  // in the tile order
    Chain& c = chain[x];
    c.qa = c.qb = -1;
    c.n = c.first = 0;
    c.list = sm.list[one_tile ? 0 : x];
    c.glist = nullptr;
    if (pos < g.ntile) {
      const int t = a.order[size_t(bh) * g.ntile + pos];
      tile_blocks(g, t, c.qa, c.qb);
      c.n = a.tcnt[size_t(bh) * g.ntile + t];
      c.glist = a.tidx + (size_t(bh) * g.ntile + t) * g.nb;
      if (!one_tile || x == 0)
        for (int i = threadIdx.x; i < c.n && i < kFList; i += kFThreads) sm.list[x][i] = c.glist[i];
    }
    if (split) {
      const int half = (c.n + 1) / 2;
      c.first = x == 0 ? 0 : half;
      c.n = x == 0 ? half : c.n - half;
    }
  }
  if constexpr (!kDiff) relbias_load(bias, a.bias, g, bh, threadIdx.x, kFThreads, a.status);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm.tmem_base, 0);
  auto col_s = [&](int x, int st) { return tmem + 128u * x + 64u * st; };
  auto col_o = [&](int x) { return tmem + 256u + 128u * x; };

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers
    // bias: warp 0 fills A's ring and warp 2 B's; the maps share one ring of all slots
    // and the warps take turns. A ring's order is K(0), K(1), then V(j), K(j + 2).
    const int prod = warp >> 1;
    if (lane == 0) {
      if (prod == 0) {
        prefetch_tensormap(&a.map_q);
        prefetch_tensormap(&a.map_k);
        prefetch_tensormap(&a.map_v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (chain[x].n == 0 || (one_tile && x == 1)) continue;
          mbar_arrive_expect_tx(&sm.q_full[x], 128u * D * 2u);
          for (int e = 0; e < 2; ++e) {
            const int blk = (e == 0 || chain[x].qb < 0) ? chain[x].qa : chain[x].qb;
            int t, hp, wp;
            block_coords(g, blk, t, hp, wp);
            for (int c = 0; c < D / 64; ++c)
              tma_load_5d(&sm.q[x][c][e * kFBlk], &a.map_q, &sm.q_full[x], c * 64, wp * g.pw,
                          hp * g.ph, t * g.pt, bh);
          }
        }
      }
      const Chain c = !kDiff && prod == 1 ? chain[1] : chain[0];
      int k = 0, last = -1;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int j) {  // the ring's next slot
        const int s = ring_slot<kDiff>(prod, k), use = k / kRing;
        if (kDiff && (k & 1) != prod) {
          ++k;
          return;
        }
        ++k;
        ok = ok && (use == 0 || mbar_wait(&sm.empty[s], (use - 1) & 1, abort)) && !*abort;
        if (!ok) return;
        if (k == 1 && (a.debug_flags & SA_DEBUG_STALL_LOADER)) return;  // test hook
        int kb = c.at(j) & kEntryBlockMask;
        if (kb >= g.nb) {
          atomicOr(a.status, kDevErrBadIndex);
          kb = 0;
        }
        int t, hp, wp;
        block_coords(g, kb, t, hp, wp);
        mbar_arrive_expect_tx(&sm.full[s], 64u * D * 2u);
        for (int ch = 0; ch < D / 64; ++ch)
          tma_load_5d(&sm.slot[s][ch][0], map, &sm.full[s], ch * 64, wp * g.pw, hp * g.ph,
                      t * g.pt, bh);
        last = k - 1;
      };
      for (int j = 0; j < 2 && j < c.n; ++j) load(&a.map_k, j);
      for (int j = 0; ok && j < c.n; ++j) {
        load(&a.map_v, j);
        if (j + 2 < c.n) load(&a.map_k, j + 2);
      }
      if (!ok) {
        fail_f(a.status, &sm.abort, kDevErrTimeoutLoad);
      }
      if (*abort && last >= 0) {
        // let this warp's own copies land before the CTA can exit (time-bounded,
        // ignoring the abort flag); at most one per slot is still in flight
        int never = 0;
        for (int kk = last; kk >= 0 && kk > last - kRing; kk -= kDiff ? 2 : 1)
          mbar_wait(&sm.full[ring_slot<kDiff>(prod, kk)], (kk / kRing) & 1, &never);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ MMA
    auto issue_chain = [&](auto which) {  // warp 1: chain 0 (A), warp 3: chain 1 (B)
      constexpr int x = decltype(which)::value;
      const int n = __shfl_sync(0xFFFFFFFFu, chain[x].n, 0);
      if (n == 0) return;
      constexpr uint32_t id_s = idesc_bf16_f32(128, 64, 0, 0);
      constexpr uint32_t id_pv = idesc_bf16_f32(128, D, 0, 1);
      constexpr uint32_t kSlotStep = (D / 64) * kFBlk / 16;
      const int qt = one_tile ? 0 : x;
      const uint64_t q = sw128_desc(smem_u32(&sm.q[qt][0][0]), 16, 1024);
      const uint64_t k0 = sw128_desc(smem_u32(&sm.slot[0][0][0]), 16, 1024);
      const uint64_t v0 = sw128_desc(smem_u32(&sm.slot[0][0][0]), kFBlk, 1024);
      const bool one = elect_one();
      auto mma_s = [&](int j, int s) {  // S_X(j), the K block in slot s
        const uint64_t k = k0 + uint64_t(s) * kSlotStep;
        constexpr int kSteps = kDiff ? D / 32 : D / 16;
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const int ks = kDiff ? x * kSteps + kk : kk;
          const uint32_t in = uint32_t(ks & 3) * 32u;
          mma_ss(col_s(x, j & 1), q + ((uint32_t(ks >> 2) * kFTile + in) >> 4),
                 k + ((uint32_t(ks >> 2) * kFBlk + in) >> 4), id_s, kk > 0);
        }
        mma_commit(&sm.s_full[x][j & 1]);
        mma_commit(&sm.empty[s]);
      };
      bool ok = mbar_wait(&sm.q_full[qt], 0, abort);
      int k = 0;  // ring position
      for (int j = 0; j < 2 && j < n; ++j, ++k) {
        const int sk = ring_slot<kDiff>(x, k);
        ok = ok && mbar_wait(&sm.full[sk], 0, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after_sync();
        if (ok && one) mma_s(j, sk);
        __syncwarp();
      }
      for (int j = 0; ok && j < n; ++j) {
        const bool has_s = j + 2 < n;
        const int sv = ring_slot<kDiff>(x, k), sk = ring_slot<kDiff>(x, k + 1);
        ok = mbar_wait(&sm.full[sv], (k / kRing) & 1, abort) &&
             mbar_wait(&sm.p_full[x][j & 1], (j >> 1) & 1, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (one) {
          mma_ts_k<4>(col_o(x), col_s(x, j & 1), v0 + uint64_t(sv) * kSlotStep, id_pv,
                      j > 0 ? 1u : 0u);
          mma_commit(j + 1 < n ? &sm.pv_done[x] : &sm.o_final[x]);
          mma_commit(&sm.empty[sv]);
        }
        __syncwarp();
        if (has_s) {  // PV_X(j) has to be done with the P that S_X(j + 2) overwrites
          ok = mbar_wait(&sm.full[sk], ((k + 1) / kRing) & 1, abort) &&
               mbar_wait(&sm.pv_done[x], j & 1, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after_sync();
          if (one) mma_s(j + 2, sk);
          __syncwarp();
        }
        k += has_s ? 2 : 1;
      }
      if (!ok) {
        fail_f(a.status, &sm.abort, kDevErrTimeoutMma);
        if (one) mma_commit(&sm.drain[x]);  // wait for the in-flight MMAs
        int never = 0;
        mbar_wait(&sm.drain[x], 0, &never);
      }
    };
    if (warp == 1) issue_chain(Which<0>{});
    else issue_chain(Which<1>{});
  } else {
    // -------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2;
    const Chain t = x ? chain[1] : chain[0];
    const int other = x ? chain[0].n : chain[1].n;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // tile row == TMEM lane
    const int half = r >> 6;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const int keep_bit = half ? (t.qb >= 0 ? kEntryKeepB : 0) : kEntryKeepA;
    const float sl2 = a.scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    RelBiasRow rb;
    if constexpr (!kDiff) rb = relbias_row(g, half && t.qb >= 0 ? t.qb : t.qa, r & 63, 1);
    for (int j = 0; j < t.n; ++j) {
      const int ent = t.at(j);
      const bool keep = (ent & keep_bit) != 0;  // uniform across the warp
      // the bias of the step's keys, while their scores are computed
      BlockBias<kRows ? L : 3> bb;
      if constexpr (kRows) {
        if (keep) bb.load(bias, rb, g, ent & kEntryBlockMask);
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.s_full[x][j & 1], (j >> 1) & 1, abort));
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t s_col = col_s(x, j & 1) + lanes;
      uint32_t sv[64];
      float mx = -INFINITY;
      if (keep) {
        tmem_ld32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_wait_ld();
        if constexpr (kRows) {
          mx = bb.add_cols(sl2, sv);  // log2 units, sv without the rows' f
        } else {
          if constexpr (!kDiff) relbias_add64(bias, rb, g, ent & kEntryBlockMask, sl2, sv);
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 2)
            mq[(i >> 1) & 3] =
                max3(mq[(i >> 1) & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
          mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
          if constexpr (kDiff) mx *= sl2;
        }
      }
      const bool need = mx > m + kFRescale;  // false while mx = -inf
      const float m_new = need ? mx : m;
      const float alpha = need ? ex2_approx(m - m_new) : 1.f;  // m = -inf -> 0
      if (__any_sync(0xFFFFFFFFu, need) && j > 0) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.pv_done[x], (j - 1) & 1, abort));
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(col_o(x) + lanes + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(col_o(x) + lanes + 32 * c, o);
        }
      }
      m = m_new;
      l *= alpha;
      uint32_t pk[32];
      if (keep) {
        // (a row whose offsets are all masked so far has m = -inf; p = 2^-inf = 0)
        const float negm = m == -INFINITY ? 0.f : -m;
        const uint64_t negm2 = f2_pack(negm, negm);
        uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint64_t s2 = f2_pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          uint64_t x2;
          if constexpr (kRows) {
            const float fm = bb.f[2 * i >> L] + negm;
            x2 = f2_add(s2, f2_pack(fm, fm));
          } else {
            x2 = kDiff ? f2_fma(s2, sl2x2, negm2) : f2_add(s2, negm2);
          }
          float x0, x1;
          f2_unpack(x2, x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          rs2[i & 3] = f2_add(rs2[i & 3], f2_pack(p0, p1));
          pk[i] = pack_bf16x2(p0, p1);
        }
        float lo, hi;
        f2_unpack(f2_add(f2_add(rs2[0], rs2[1]), f2_add(rs2[2], rs2[3])), lo, hi);
        l += lo + hi;
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = 0u;
      }
      tmem_st32(s_col, pk);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[x][j & 1]);
    }
    // ---- epilogue: O / l -> natural token position
    bool done = ok && (t.n == 0 ||
                       __all_sync(0xFFFFFFFFu, mbar_wait(&sm.o_final[x], 0, abort)));
    if (one_tile && done) {
      // the rows of A and B meet here: their statistics, then both O's in TMEM
      sm.m[x][r] = m;
      sm.l[x][r] = l;
      mbar_arrive(&sm.join);
      done = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.join, 0, abort)) &&
             (other == 0 || __all_sync(0xFFFFFFFFu, mbar_wait(&sm.o_final[x ^ 1], 0, abort)));
    }
    if (!done) {
      fail_f(a.status, &sm.abort, kDevErrTimeoutSoftmax);
    } else if (t.qa >= 0 && (half == 0 || t.qb >= 0)) {  // uniform across the warp
      tc_fence_after_sync();
      const size_t row = size_t(bh) * g.S + block_row_token(g, half ? t.qb : t.qa, r & 63);
      float w0 = l > 0.f ? 1.0f / l : 0.f, w1 = 0.f;  // what O_A and O_B count in the output
      if (one_tile) {
        const float m0 = sm.m[0][r], m1 = sm.m[1][r], l0 = sm.l[0][r], l1 = sm.l[1][r];
        if constexpr (kDiff) {
          w0 = l0 > 0.f ? 1.0f / l0 : 0.f;
          w1 = l1 > 0.f ? 1.0f / l1 : 0.f;
        } else {
          // one softmax over both halves of the list
          m = fmaxf(m0, m1);
          const float e0 = l0 > 0.f ? ex2_approx(m0 - m) : 0.f;
          const float e1 = l1 > 0.f ? ex2_approx(m1 - m) : 0.f;
          l = l0 * e0 + l1 * e1;
          w0 = l > 0.f ? e0 / l : 0.f;
          w1 = l > 0.f ? e1 / l : 0.f;
        }
      }
      // log-sum-exp of the row's kept scores (natural log): m is in log2 units and l
      // is the sum relative to 2^m
      if (a.lse != nullptr && !(split && x == 1))
        a.lse[row + (kDiff ? size_t(x) * g.BH * g.S : 0)] =
            l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
      if (one_tile) {
        // A's warps write the first half of the channels, B's the second
        const float lam = kDiff ? __bfloat162float(a.lam[bh % a.H]) : -1.f;
        const int na = chain[0].n, nb_ = chain[1].n;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int col = x * (D / 2) + 32 * c;
          float o1[32], o2[32];
          load_o32(col_o(0) + lanes + uint32_t(col), na, w0, o1);
          load_o32(col_o(1) + lanes + uint32_t(col), nb_, w1, o2);
#pragma unroll
          for (int i = 0; i < 32; ++i) o1[i] = fmaf(-lam, o2[i], o1[i]);
          store_o32(a.out, row * D + col, o1, a.out_fp32);
          if (kDiff && a.out2 != nullptr) store_o32(a.out2, row * D + col, o2, a.out_fp32);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          load_o32(col_o(x) + lanes + 32 * c, t.n, w0, o);
          store_o32(a.out, row * D + 32 * c, o, a.out_fp32);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Up to four query tiles per SM, A and B take the halves of one tile's list: twice
// the CTAs with half the steps each, where pairs of whole tiles leave SMs idle.
// Halves against whole tiles, d 128, lists of about 56 and 96 steps: 72.5 -> 40.6 and
// 129 -> 69 us (64 tiles), 81 -> 67 and 126 -> 114 (192), 137 -> 109 and 226 -> 175
// (384), 143 -> 140 and 228 -> 236 (512), 141 -> 155 and 242 -> 254 (576); beyond the
// bound the waves decide: 191 -> 180 and 349 -> 292 (640), 217 -> 213 and 376 -> 369
// (768), 294 -> 283 and 481 -> 461 (1,024), 425 -> 430 and 723 -> 710 (1,536), and with
// 12 % of 588 blocks kept 322 -> 338 (592), 508 -> 512 (888), 666 -> 688 (1,184).
constexpr long kSplitTiles = 4 * 148;

template <int D, AttnMode M, int L>
static cudaError_t launch_score_fwd_m(const ScoreFwdArgs& a, const Geometry& g,
                                      cudaStream_t stream) {
  // At least 120 KB: each CTA allocates all 512 TMEM columns.
  size_t need = sizeof(ScoreFwdSmem<D>) + 1024;
  if (M != AttnMode::kDiff) need += relbias_offsets(g) * sizeof(float);
  const int smem = int(need > 120 * 1024 ? need : 120 * 1024);
  // The limit belongs to the process, so it is the same for every grid: another
  // thread's call of a smaller one may stand between these two lines.
  cudaError_t e = cudaFuncSetAttribute(score_fwd_kernel<D, M, L>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  const bool one_tile = M == AttnMode::kDiff || a.split;
  const dim3 grid(unsigned(one_tile ? g.ntile : (g.ntile + 1) / 2), unsigned(g.BH));
  return launch_early(score_fwd_kernel<D, M, L>, grid, kFThreads, smem, stream, a, g);
}

template <int D>
static cudaError_t launch_score_fwd_d(const ScoreFwdArgs& a, const Geometry& g,
                                      cudaStream_t stream) {
  if (a.lam != nullptr) return launch_score_fwd_m<D, AttnMode::kDiff, kAnyShape>(a, g, stream);
  switch (g.lpw) {
    case 2: return launch_score_fwd_m<D, AttnMode::kBias, 2>(a, g, stream);
    case 3: return launch_score_fwd_m<D, AttnMode::kBias, 3>(a, g, stream);
    case 4: return launch_score_fwd_m<D, AttnMode::kBias, 4>(a, g, stream);
    default: return launch_score_fwd_m<D, AttnMode::kBias, kAnyShape>(a, g, stream);
  }
}

cudaError_t launch_score_fwd(ScoreFwdArgs a, const Geometry& g, cudaStream_t stream) {
  a.split = a.lam == nullptr && long(g.ntile) * g.BH <= kSplitTiles;
  return g.d == 128 ? launch_score_fwd_d<128>(a, g, stream) : launch_score_fwd_d<64>(a, g, stream);
}

}  // namespace sa
