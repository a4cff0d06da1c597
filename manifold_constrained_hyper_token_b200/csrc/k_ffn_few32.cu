// k_ffn_few32.cu -- the feed-forward products of up to 128 tokens, fp32.
//
// As in k_ffn_few.cu the weights are the tall operand and are read once, 128 rows
// per CTA, the k axis split over a cluster.  They arrive as they are, in fp32, by
// TMA; sixteen warps split each 128 x 32 tile into its three bf16 planes (split3x4)
// in shared memory, and the tensor cores take six of the nine products of planes with
// the tokens' planes (what is left out is 2^-24 of a product on average).  Splitting
// the weights beforehand, as the products of many tokens do, would move 16 bytes
// per weight instead of 4.
//
// X1 W1 has an accumulator of its own, the five smaller products share one.  (Three
// accumulators, one per order, and three MMAs over the stacked planes [X1 X2 X3],
// [X1 X2] and [X1] leave TMEM for fewer sets, and so force shorter parts: T = 64,
// C = 4096, F = 4736, 132 us against 104; T = 17, C = 7168, F = 14336, 441 against 409.)
//
// The tensor cores' adder cuts instead of rounding, so a long sum is spread over up
// to four sets of accumulators in turn and over the cluster, kGoodK per set where
// eight CTAs allow it; the rest of the sum is rounded fp32 addition in the epilogue.
//
// Warps: 0 weights' TMA, 1 the MMAs, 2 the tokens' TMA, 4-19 the split; then all of
// them the reduction over the cluster, as in k_ffn_few.cu.  Every warp takes part in
// every k block: a waiter that skipped phases of a barrier could take an earlier
// phase of the same parity for its own.
#include "ffn_few.h"

#include "ffn_common.cuh"
#include "tc_pair.cuh"

namespace mhc {

namespace {

namespace few32 {
constexpr int TM = 128, TK = 32;
constexpr int RAW = TM * TK * 4;      // a weight tile in fp32
constexpr int PLANE = TM * TK * 2;    // ... one of its planes
constexpr int NT = 640, NCONV = 16;   // threads; splitting warps
constexpr int MAXRAW = 12, MAXX = 6;  // ring stages, at most: weight tiles, k blocks of tokens
constexpr int ROOM = 222 * 1024, TAIL = 1024 + 512;
constexpr int BLOCK_NS = 450, FIXED_NS = 5000;  // a weight tile; a CTA's start and end
constexpr int kMaxK = 2048, kGoodK = 512;  // k per set of accumulators: at most; aimed at
static_assert(RAW / 2 == 32 * NCONV * 16, "a thread takes 16 bytes of each half of a tile");
}  // namespace few32

enum Epi32 { F32_STORE, F32_GATE, F32_DGATE };

struct Few32P {
  CUtensorMap w[2], x;
  int nseg, kblocks;
  int np, raws, xs;        // tokens rounded up to 16; weight tiles and token blocks on their way
  int sets;                // sets of two accumulators of a weight
  int64_t rows, t;
  void* o0;                // STORE: fp32 [t][rows]; else bf16 planes [3 or 6][t][rows]
  float *g, *u;            // GATE: kept unless null; DGATE: read
  int act;
  bool early;              // a later kernel of its call: the weights may be read at once
  bool beside;             // needs nothing from the kernel before it
  uint32_t tmem_cols;      // columns to allocate; an accumulator has np
  int* status;
  uint64_t wait_ns;
};

// Four consecutive values as three planes, `stride` elements apart.
__device__ __forceinline__ void store_planes(__nv_bfloat16* p, int64_t stride, const float (&v)[4]) {
  uint2 h, m, l;
  split3x4(make_float4(v[0], v[1], v[2], v[3]), h, m, l);
  *reinterpret_cast<uint2*>(p) = h;
  *reinterpret_cast<uint2*>(p + stride) = m;
  *reinterpret_cast<uint2*>(p + 2 * stride) = l;
}

template <Epi32 E, bool MN>
__global__ void __launch_bounds__(few32::NT, 1) k_ffn_few32(const __grid_constant__ Few32P P) {
  using namespace few32;
  constexpr int NW = E == F32_GATE ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  // a ring of weight tiles, two sets of [weight][plane] tiles, a ring of tokens' planes
  constexpr int SETB = NW * 3 * PLANE;
  const int xbytes = 3 * P.np * TK * 2;
  uint8_t* sets = smem + P.raws * RAW;
  uint8_t* xring = sets + 2 * SETB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(xring + P.xs * xbytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAXRAW + 2 * MAXX + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto raw_full = [&](int s) { return tc::smem_u32(bars + s); };
  auto raw_empty = [&](int s) { return tc::smem_u32(bars + MAXRAW + s); };
  auto set_full = [&](int s) { return tc::smem_u32(bars + 2 * MAXRAW + s); };
  auto set_empty = [&](int s) { return tc::smem_u32(bars + 2 * MAXRAW + 2 + s); };
  auto x_full = [&](int s) { return tc::smem_u32(bars + 2 * MAXRAW + 4 + s); };
  auto x_empty = [&](int s) { return tc::smem_u32(bars + 2 * MAXRAW + 4 + MAXX + s); };
  const uint32_t done_bar = tc::smem_u32(bars + 2 * MAXRAW + 4 + 2 * MAXX);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int parts = (int)csize, rank = (int)tc::cluster_rank();
  const int64_t row0 = (int64_t)(blockIdx.x / parts) * TM;
  const int nk = P.nseg * P.kblocks;
  // this CTA's k blocks: at least one, the launch has parts <= nk
  const int j0 = (int)((int64_t)nk * rank / parts), j1 = (int)((int64_t)nk * (rank + 1) / parts);
  const int blocks = j1 - j0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.raws; ++s) {
      tc::mbar_init(raw_full(s), 1);
      tc::mbar_init(raw_empty(s), NCONV);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(set_full(s), NCONV);
      tc::mbar_init(set_empty(s), 1);
    }
    for (int s = 0; s < P.xs; ++s) {
      tc::mbar_init(x_full(s), 1);
      tc::mbar_init(x_empty(s), 1);
    }
    tc::mbar_init(done_bar, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&P.w[0]);
    tc::tma_prefetch_desc(&P.x);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), P.tmem_cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_status(P.status, MHC_ERR_TIMEOUT);
  };

  // the first ring of weights needs nothing from the kernel before this one
  if (P.beside) {
    tc::grid_release();
  } else if (warp != 0 || !P.early) {
    tc::grid_wait();
    tc::grid_release();
  }

  if (warp == 0) {
    // ------------------------------------------------------- weights, as they are
    if (lane == 0) {
      const uint64_t stream = tc::policy_evict_first();
      int it = 0;  // tiles: a k block has NW
      for (; it < blocks * NW; ++it) {
        const int s = it % P.raws;
        // a tile is free once split, and the splitting warps wait for the kernel before
        // this one: its time is not this wait's
        if (P.early && it == P.raws) tc::grid_wait();
        if (it >= P.raws &&
            !tc::mbar_pipe_wait<false>(raw_empty(s), ((uint32_t)(it / P.raws) & 1u) ^ 1u,
                                       abort_flag, P.wait_ns)) {
          give_up();
          break;
        }
        const int j = j0 + it / NW, seg = j / P.kblocks, k0 = (j - seg * P.kblocks) * TK;
        tc::mbar_arrive_expect_tx(raw_full(s), RAW);
        const CUtensorMap* m = &P.w[NW == 2 ? it % NW : seg];
        const uint32_t dst = tc::smem_u32(smem + s * RAW);
        if (MN) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            tc::tma_load_2d(dst + b * (RAW / 4), m, raw_full(s), (int)row0 + 32 * b, k0, stream);
        } else {
          tc::tma_load_2d(dst, m, raw_full(s), k0, (int)row0, stream);
        }
      }
      for (int i = it > P.raws ? it - P.raws : 0; i < it; ++i)
        tc::mbar_wait(raw_full(i % P.raws), (uint32_t)(i / P.raws) & 1u, nullptr,
                      tc::kDrainWaitNs);
    }
    __syncwarp();
    if (P.early) tc::grid_wait();  // before the reduction reads g and u
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens' planes
    if (lane == 0) {
      const uint64_t keep = tc::policy_evict_last();
      int it = 0;
      for (; it < blocks; ++it) {
        const int s = it % P.xs;
        if (it >= P.xs && !tc::mbar_pipe_wait<false>(x_empty(s), ((uint32_t)(it / P.xs) & 1u) ^ 1u,
                                                     abort_flag, P.wait_ns)) {
          give_up();
          break;
        }
        const int j = j0 + it, seg = j / P.kblocks, k0 = (j - seg * P.kblocks) * TK;
        tc::mbar_arrive_expect_tx(x_full(s), xbytes);
        tc::tma_load_3d(tc::smem_u32(xring + s * xbytes), &P.x, x_full(s), k0, 0,
                        NW == 2 ? 0 : 3 * seg, keep);
      }
      for (int i = it > P.xs ? it - P.xs : 0; i < it; ++i)
        tc::mbar_wait(x_full(i % P.xs), (uint32_t)(i / P.xs) & 1u, nullptr, tc::kDrainWaitNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------------- MMA
    // A small MMA is over before its operands are made up.  So the descriptors are
    // prepared here (they count in 16 bytes), and the warp stays together and elects
    // the lane that issues, which makes them uniform (T = 17, C = 7168, F = 14336:
    // 633 us as a single lane's loop, 562 with the descriptors prepared, 441 so)
    const bool leader = tc::elect_one();
    const uint32_t np = (uint32_t)P.np, weight = (uint32_t)(2 * P.sets) * np;
    const uint32_t idesc = tc::idesc_bf16(TM, P.np, MN, false);
    const uint64_t adesc = MN ? tc::smem_desc(tc::smem_u32(sets), PLANE / 2, 1024, tc::SWZ_128B)
                              : tc::smem_desc(tc::smem_u32(sets), 16, 512, tc::SWZ_64B);
    const uint64_t bdesc = tc::smem_desc(tc::smem_u32(xring), 16, 512, tc::SWZ_64B);
    int xs = 0, set = 0;
    uint32_t xpar = 0, acc = tmem, add = 0;
    for (int it = 0; it < blocks; ++it) {
      const int s = it & 1;
      const bool ok =
          tc::mbar_pipe_wait<false>(x_full(xs), xpar, abort_flag, P.wait_ns) &&
          tc::mbar_pipe_wait<false>(set_full(s), (uint32_t)(it / 2) & 1u, abort_flag, P.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) give_up();
        break;
      }
      tc::tc_fence_after();
      const uint64_t a0 = adesc + (uint32_t)(s * (SETB / 16));
      const uint64_t b0 = bdesc + (uint32_t)(xs * (xbytes / 16));
#pragma unroll
      for (int k = 0; k < TK / 16; ++k) {
        if (leader) {
#pragma unroll
          for (int pw = 0; pw < 3; ++pw) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
              const uint64_t a = a0 + (uint32_t)((i * 3 + pw) * (PLANE / 16) + k * (MN ? 128 : 2));
              const uint64_t b = b0 + (uint32_t)(k * 2);
              const uint32_t d = acc + i * weight;
#pragma unroll
              for (int px = 0; px < 3 - pw; ++px)
                tc::mma_bf16(d + (pw + px > 0 ? np : 0), a, b + (uint32_t)px * np * 4, idesc,
                             pw > 0 || px > 1 ? 1u : add);
            }
          }
        }
        acc += 2 * np;
        if (++set == P.sets) {
          set = 0;
          acc = tmem;
          add = 1;
        }
      }
      if (leader) {
        tc::mma_commit(set_empty(s));
        tc::mma_commit(x_empty(xs));
      }
      if (++xs == P.xs) {
        xs = 0;
        xpar ^= 1u;
      }
    }
    // the sums are complete, and no MMA is under way when TMEM is freed
    if (leader) tc::mma_commit(done_bar);
    __syncwarp();
    tc::mbar_wait(done_bar, 0, nullptr, tc::kDrainWaitNs);
  } else if (warp >= 4) {
    // -------------------------------------------------------------------- split
    // this thread's 16 bytes of each half of a tile (row r of 128 bytes, piece p),
    // and where they go in a half of a plane
    const int c = threadIdx.x - 128, r = c >> 3, p = c & 7, k = r & 31;
    const int to0 = MN ? k * 128 + ((((r >> 5) * 4 + (p >> 1)) ^ (k & 7)) << 4) + (p & 1) * 8
                       : r * 64 + (((p >> 1) ^ ((r >> 1) & 3)) << 4) + (p & 1) * 8;
    for (int it = 0; it < blocks; ++it) {
      const int s = it & 1;
      bool ok = it < 2 || tc::mbar_pipe_wait<false>(set_empty(s), ((uint32_t)(it / 2) & 1u) ^ 1u,
                                                    abort_flag, P.wait_ns);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int n = it * NW + i, rs = n % P.raws;
        ok = ok && tc::mbar_pipe_wait<false>(raw_full(rs), (uint32_t)(n / P.raws) & 1u, abort_flag,
                                             P.wait_ns);
        if (!ok && !*abort_flag) give_up();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;  // a warp leaves as one
        const uint8_t* src = smem + rs * RAW;
        uint8_t* dst = sets + s * SETB + i * 3 * PLANE;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint2 h, m, l;
          split3x4(*reinterpret_cast<const float4*>(src + c * 16 + e * (RAW / 2)), h, m, l);
          // K-major: 64 rows further; MN: the tile is [32 rows of W at a time][k][32]
          // and the plane [64 rows at a time][k][64]
          const int to = to0 + e * (PLANE / 2);
          *reinterpret_cast<uint2*>(dst + to) = h;
          *reinterpret_cast<uint2*>(dst + PLANE + to) = m;
          *reinterpret_cast<uint2*>(dst + 2 * PLANE + to) = l;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(raw_empty(rs));
      }
      if (!ok) break;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(set_full(s));
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  // This CTA's part, [weight][token][row], over the stages, whose copies and MMAs
  // are done; then the ranks add up the tokens in turn, parts in rank order.
  float* part = reinterpret_cast<float*>(smem);
  if (warp < 4) {
    const int r = threadIdx.x;
    const uint32_t ta = tmem + ((uint32_t)(32 * warp) << 16);
    // the smaller products first, set by set
    const int steps = blocks * (TK / 16), used = steps < P.sets ? steps : P.sets;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      for (int c = 0; c < P.np; c += 16) {
        float v[16] = {}, m[16];
        for (int o = 1; o >= 0; --o)
          for (int q = 0; q < used; ++q) {
            tc::tmem_get16(ta + ((i * P.sets + q) * 2 + o) * P.np + c, m);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += m[e];
          }
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(i * P.np + c + e) * TM + r] = v[e];
      }
  }
  __syncwarp();
  if (parts > 1) tc::cluster_sync();
  else __syncthreads();
  const int64_t row = row0 + 4 * lane, plane = P.t * P.rows;
  if (row < P.rows) {
    for (int64_t c = rank + parts * warp; c < P.t; c += parts * (NT / 32)) {
      const int64_t o = c * P.rows + row;
      float4 gq, uq;
      if (E == F32_DGATE) {
        gq = *reinterpret_cast<const float4*>(P.g + o);
        uq = *reinterpret_cast<const float4*>(P.u + o);
      }
      float4 ld[NW][8];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint32_t at = tc::smem_u32(part + (i * P.np + c) * TM + 4 * lane);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          ld[i][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (q < parts) ld[i][q] = tc::ld_cluster_f32x4(tc::map_cta(at, q));
        }
      }
      float v[NW][4];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[i][0] += ld[i][q].x;
          v[i][1] += ld[i][q].y;
          v[i][2] += ld[i][q].z;
          v[i][3] += ld[i][q].w;
        }
      }
      if (E == F32_STORE) {
        *reinterpret_cast<float4*>((float*)P.o0 + o) = make_float4(v[0][0], v[0][1], v[0][2],
                                                                   v[0][3]);
      } else if (E == F32_GATE) {
        float a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = gate<false>(P.act, v[0][k]) * v[NW - 1][k];
        store_planes((__nv_bfloat16*)P.o0 + o, plane, a);
        if (P.g) {
          *reinterpret_cast<float4*>(P.g + o) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
          *reinterpret_cast<float4*>(P.u + o) =
              make_float4(v[NW - 1][0], v[NW - 1][1], v[NW - 1][2], v[NW - 1][3]);
        }
      } else {
        const float g[4] = {gq.x, gq.y, gq.z, gq.w}, u[4] = {uq.x, uq.y, uq.z, uq.w};
        float dg[4], du[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float h, dh;
          gate_both<false>(P.act, g[k], h, dh);
          dg[k] = v[0][k] * u[k] * dh;
          du[k] = v[0][k] * h;
        }
        store_planes((__nv_bfloat16*)P.o0 + o, plane, dg);
        store_planes((__nv_bfloat16*)P.o0 + 3 * plane + o, plane, du);
      }
    }
  }
  tc::tc_fence_before();
  __syncwarp();
  // nobody reads this CTA's part any more
  if (parts > 1) tc::cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, P.tmem_cols);
  }
  if (P.beside) tc::grid_wait();
}

#define TRY(call)                         \
  do {                                    \
    const cudaError_t e_ = (call);        \
    if (e_ != cudaSuccess) return e_;     \
  } while (0)

// An fp32 weight [rows][cols] as stored; mn: the products' rows run along cols.
cudaError_t weight_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, bool mn) {
  const uint64_t d[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t s[1] = {(uint64_t)cols * 4};
  const uint32_t b[2] = {32, mn ? (uint32_t)few32::TK : (uint32_t)few32::TM};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p, 2, d, s, b, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// The tokens' planes [planes][t][K], three at a time
cudaError_t token_map(CUtensorMap* m, const void* p, int64_t t, int64_t K, int planes, int np) {
  const uint64_t d[3] = {(uint64_t)K, (uint64_t)t, (uint64_t)planes};
  const uint64_t s[2] = {(uint64_t)K * 2, (uint64_t)K * t * 2};
  const uint32_t b[3] = {few32::TK, (uint32_t)np, 3};
  return make_tmap_bf16(m, p, 3, d, s, b, CU_TENSOR_MAP_SWIZZLE_64B);
}

int tokens16(int64_t t) { return (int)((t + 15) / 16 * 16); }

// Sets of two accumulators per weight, of a product with nw weights.
int sets_of(int64_t t, int nw) {
  const int n = 512 / (nw * 2 * tokens16(t));
  return n < 4 ? n : 4;
}

template <Epi32 E, bool MN>
cudaError_t launch(Few32P& P, const FewArgs& f, int64_t K, cudaStream_t s) {
  using namespace few32;
  constexpr int NW = E == F32_GATE ? 2 : 1;
  P.t = f.t;
  P.act = f.act;
  P.status = f.st;
  P.wait_ns = tc::wait_limit(f.wait_ns);
  P.kblocks = (int)((K + TK - 1) / TK);
  P.sets = sets_of(f.t, NW);
  P.tmem_cols = 32;
  while (P.tmem_cols < (uint32_t)(NW * P.sets * 2 * P.np)) P.tmem_cols *= 2;
  // What the planes leave is shared out between the weights' ring and the tokens':
  // a weight tile takes about 1.5 us from HBM and is free once split, a tokens' block
  // 1 us from the L2 and is free a block or two later, after its MMAs.
  const int sets = 2 * NW * 3 * PLANE, xbytes = 3 * P.np * TK * 2;
  int most = 0;
  for (int xs = 2; xs <= MAXX && ROOM - sets - xs * xbytes >= NW * RAW; ++xs) {
    const int fit = (ROOM - sets - xs * xbytes) / RAW, raws = fit < MAXRAW ? fit : MAXRAW;
    const int w = 2 * (2 * raws - NW), x = 3 * NW * (2 * xs - 3), score = w < x ? w : x;
    if (score > most) {
      most = score;
      P.xs = xs;
      P.raws = raws;
    }
  }
  // the parts take the stages' place: NW np 512 bytes, less than the rings and planes
  const int stage = P.raws * RAW + sets + P.xs * xbytes;
  const int64_t tiles = (P.rows + TM - 1) / TM;
  const int nk = P.nseg * P.kblocks, good = kGoodK / TK * P.sets;
  const int want = (nk + good - 1) / good, least = want < 8 ? want : 8;
  const int parts = split_sum(tiles, nk, 1, least, NW, BLOCK_NS * NW, FIXED_NS);
  auto kern = k_ffn_few32<E, MN>;
  TRY(allow_smem(kern, ROOM + TAIL));
  return launch_after(kern, (unsigned)(tiles * parts), NT, stage + TAIL, (unsigned)parts, s, P);
}

Few32P base(const FewArgs& f, int64_t rows, int nseg) {
  Few32P P{};
  P.rows = rows;
  P.nseg = nseg;
  P.np = tokens16(f.t);
  return P;
}

}  // namespace

bool few32_fits(int64_t t, int64_t C, int64_t F) {
  if (t > kFewTokens32) return false;
  const int64_t one = (int64_t)8 * few32::kMaxK;
  return C <= one * sets_of(t, 2) && 2 * F <= one * sets_of(t, 1);
}

cudaError_t few32_gate(const FewArgs& f, void* a, float* g, float* u, cudaStream_t s) {
  Few32P P = base(f, f.F, 1);
  TRY(weight_map(&P.w[0], f.wg, f.F, f.C, false));
  TRY(weight_map(&P.w[1], f.wu, f.F, f.C, false));
  TRY(token_map(&P.x, f.x, f.t, f.C, 3, P.np));
  P.o0 = a;
  P.g = g;
  P.u = u;
  return launch<F32_GATE, false>(P, f, f.C, s);
}

cudaError_t few32_down(const FewArgs& f, const void* a, float* y, cudaStream_t s) {
  Few32P P = base(f, f.C, 1);
  P.early = true;
  TRY(weight_map(&P.w[0], f.wd, f.C, f.F, false));
  TRY(token_map(&P.x, a, f.t, f.F, 3, P.np));
  P.o0 = y;
  return launch<F32_STORE, false>(P, f, f.F, s);
}

cudaError_t few32_dgate(const FewArgs& f, const float* g, const float* u, void* d, cudaStream_t s) {
  Few32P P = base(f, f.F, 1);
  P.beside = true;
  TRY(weight_map(&P.w[0], f.wd, f.C, f.F, true));
  TRY(token_map(&P.x, f.gy, f.t, f.C, 3, P.np));
  P.o0 = d;
  P.g = const_cast<float*>(g);
  P.u = const_cast<float*>(u);
  return launch<F32_DGATE, true>(P, f, f.C, s);
}

cudaError_t few32_grad_x(const FewArgs& f, const void* d, float* gx, cudaStream_t s) {
  Few32P P = base(f, f.C, 2);
  P.early = true;
  TRY(weight_map(&P.w[0], f.wg, f.F, f.C, true));
  TRY(weight_map(&P.w[1], f.wu, f.F, f.C, true));
  TRY(token_map(&P.x, d, f.t, f.F, 6, P.np));
  P.o0 = gx;
  return launch<F32_STORE, true>(P, f, f.F, s);
}

#undef TRY

}  // namespace mhc
