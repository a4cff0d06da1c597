// k_ffn_few.cu -- the feed-forward products of up to 256 tokens, bf16: decoding
// batches, short prompts, small gradient steps.
//
// These read every weight once and are bound by that, so the weights are the
// tall operand: D^T[w][t] = sum_k W(w, k) X(t, k), 128 weight rows per CTA (the
// MMA's M) by all the tokens at once (its N, rounded up to 16).  A CTA streams
// its rows in 64-wide k blocks through a TMA ring; one tcgen05 MMA per 16 k (two
// for the gated product, w_gate and w_up into two accumulators).  The k axis is
// split over the CTAs of a cluster so that the bytes in flight fill the machine:
// at C = 7168, F = 14336 there are only 56 or 112 row tiles for 148 SMs.  The
// parts meet in distributed shared memory and are added in rank order, so that
// results do not depend on timing; the activation, its derivative and the stores
// (consecutive rows of W are consecutive in memory) follow there.
//
// Weights stored along k (forward) or along their rows (the backward's da and
// gx) differ only in the TMA box and the MMA descriptor.  Waits are bounded as in
// the other tensor-core kernels; a CTA that gives up still takes part in its
// cluster's barriers.
#include "ffn_few.h"

#include "ffn_common.cuh"
#include "tc_pair.cuh"

namespace mhc {

namespace {

namespace few {
constexpr int TM = 128, TK = 64;
constexpr int WBYTES = TM * TK * 2;  // 16 KB of weights per k block
constexpr int NT = 128;
constexpr int MAXST = 12;            // stages of the ring, at most
constexpr int HALF_SMEM = 110 * 1024, FULL_SMEM = 222 * 1024;  // ring: two CTAs per SM, or one
constexpr int TAIL = 1024 + 256;     // alignment, barriers
constexpr int BLOCK_NS = 600, FIXED_NS = 4000;  // a k block; a CTA's start and end
}  // namespace few

enum FewEpi { FEW_STORE, FEW_GATE, FEW_DGATE };

struct FewP {
  CUtensorMap w[2], x;
  int nseg, kblocks;     // GATE: one segment, both maps; else segment s: w[s], plane s of x
  int np, stages, chunk; // tokens rounded up to 16; ring stages; tokens reduced at a time
  int64_t rows, t;       // weight rows; tokens
  __nv_bfloat16 *o0, *o1;
  float *g, *u;          // GATE: kept unless null; DGATE: read
  int act;
  bool early;            // a later kernel of its call: the weights may be read at once
  bool beside;           // needs nothing from the kernel before it
  uint32_t tmem_cols, acc1;  // columns to allocate; the second accumulator's column
  int* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

template <FewEpi E, bool MN>
__global__ void __launch_bounds__(few::NT) k_ffn_few(const __grid_constant__ FewP P) {
  using namespace few;
  constexpr int NW = E == FEW_GATE ? 2 : 1;  // weight tiles per stage, accumulators
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const int stage_bytes = NW * WBYTES + P.np * TK * 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P.stages * stage_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAXST + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full = [&](int s) { return tc::smem_u32(bars + s); };
  auto empty = [&](int s) { return tc::smem_u32(bars + MAXST + s); };
  const uint32_t done_bar = tc::smem_u32(bars + 2 * MAXST);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int parts = (int)csize, rank = (int)tc::cluster_rank();
  const int64_t row0 = (int64_t)(blockIdx.x / parts) * TM;
  const int nk = P.nseg * P.kblocks;
  // this CTA's k blocks: at least one, the launch has parts <= nk
  const int j0 = (int)((int64_t)nk * rank / parts), j1 = (int)((int64_t)nk * (rank + 1) / parts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      tc::mbar_init(full(s), 1);
      tc::mbar_init(empty(s), 1);
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

  const bool loader = warp == 0 && lane == 0;
  const uint64_t stream = tc::policy_evict_first(), keep = tc::policy_evict_last();
  auto load_weights = [&](int it) {
    const int s = it % P.stages, j = j0 + it, seg = j / P.kblocks;
    const int k0 = (j - seg * P.kblocks) * TK;
    const uint32_t base = tc::smem_u32(smem + s * stage_bytes);
    tc::mbar_arrive_expect_tx(full(s), stage_bytes);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const CUtensorMap* m = &P.w[NW == 2 ? i : seg];
      const uint32_t dst = base + i * WBYTES;
      if (MN) {
        tc::tma_load_2d(dst, m, full(s), (int)row0, k0, stream);
        tc::tma_load_2d(dst + WBYTES / 2, m, full(s), (int)row0 + 64, k0, stream);
      } else {
        tc::tma_load_2d(dst, m, full(s), k0, (int)row0, stream);
      }
    }
  };
  // a ring of weights is on its way while the kernel before this one ends
  const int blocks = j1 - j0;
  const int ahead = !P.early ? 0 : blocks < P.stages ? blocks : P.stages;
  if (loader)
    for (int it = 0; it < ahead; ++it) load_weights(it);
  if (!P.beside) tc::grid_wait();
  tc::grid_release();

  if (loader) {
    // ---------------------------------------------------------------- TMA
    int it = 0;
    for (; it < blocks; ++it) {
      const int s = it % P.stages;
      if (it >= P.stages &&
          !tc::mbar_pipe_wait<false>(empty(s), ((uint32_t)(it / P.stages) & 1u) ^ 1u, abort_flag,
                                     P.wait_ns)) {
        give_up();
        break;
      }
      if (it >= ahead) load_weights(it);
      const int j = j0 + it, seg = j / P.kblocks, k0 = (j - seg * P.kblocks) * TK;
      tc::tma_load_3d(tc::smem_u32(smem + s * stage_bytes) + NW * WBYTES, &P.x, full(s), k0, 0,
                      NW == 2 ? 0 : seg, keep);
    }
    // every copy issued here has landed before the CTA can exit
    for (int i = it > P.stages ? it - P.stages : 0; i < it; ++i)
      tc::mbar_wait(full(i % P.stages), (uint32_t)(i / P.stages) & 1u, nullptr, tc::kDrainWaitNs);
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc = tc::idesc_bf16(TM, P.np, MN, false);
    int it = 0;
    for (int j = j0; j < j1; ++j, ++it) {
      const int s = it % P.stages;
      if (!tc::mbar_pipe_wait<false>(full(s), (uint32_t)(it / P.stages) & 1u, abort_flag,
                                     P.wait_ns)) {
        give_up();
        break;
      }
      tc::tc_fence_after();
      const uint32_t base = tc::smem_u32(smem + s * stage_bytes);
#pragma unroll
      for (int k = 0; k < TK / 16; ++k) {
        const uint64_t b = tc::smem_desc(base + NW * WBYTES + k * 32, 16, 1024, tc::SWZ_128B);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const uint32_t wb = base + i * WBYTES;
          const uint64_t a = MN ? tc::smem_desc(wb + k * 2048, WBYTES / 2, 1024, tc::SWZ_128B)
                                : tc::smem_desc(wb + k * 32, 16, 1024, tc::SWZ_128B);
          tc::mma_bf16(tmem + i * P.acc1, a, b, idesc, it > 0 || k > 0 ? 1u : 0u);
        }
      }
      tc::mma_commit(empty(s));
    }
    // the sums are complete, and no MMA is under way when TMEM is freed
    tc::mma_commit(done_bar);
    tc::mbar_wait(done_bar, 0, nullptr, tc::kDrainWaitNs);
  }
  __syncthreads();
  tc::tc_fence_after();
  // This CTA's part: [accumulator][token][row] over the ring, whose copies and
  // MMAs are done; then rank r adds up tokens r, r + parts, ... of all parts.
  float* part = reinterpret_cast<float*>(smem);
  const int r = threadIdx.x;  // row of D^T: TMEM lane 32 warp + lane
  const uint32_t ta = tmem + ((uint32_t)(32 * warp) << 16);
  for (int c0 = 0; c0 < P.np; c0 += P.chunk) {
    const int cn = P.np - c0 < P.chunk ? P.np - c0 : P.chunk;
    for (int c = 0; c < cn; c += 16) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        float v[16];
        tc::tmem_get16(ta + i * P.acc1 + c0 + c, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(i * cn + c + e) * TM + r] = v[e];
      }
    }
    if (parts > 1) tc::cluster_sync();
    else __syncthreads();
    // a warp per token, four consecutive rows per lane (rows come in eights)
    const int64_t row = row0 + 4 * lane;
    if (row < P.rows) {
      for (int c = rank + parts * warp; c < cn && c0 + c < P.t; c += parts * 4) {
        const int64_t o = (c0 + c) * P.rows + row;
        // every load is under way before the first sum: one from another CTA takes
        // about a quarter of a microsecond
        float4 ld[NW][8];
        float4 gq, uq;
        if (E == FEW_DGATE) {
          gq = *reinterpret_cast<const float4*>(P.g + o);
          uq = *reinterpret_cast<const float4*>(P.u + o);
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const uint32_t at = tc::smem_u32(part + (i * cn + c) * TM + 4 * lane);
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
        if (E == FEW_STORE) {
          store4(P.o0 + o, v[0]);
        } else if (E == FEW_GATE) {
          float a[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) a[k] = gate<true>(P.act, v[0][k]) * v[NW - 1][k];
          store4(P.o0 + o, a);
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
            gate_both<true>(P.act, g[k], h, dh);
            dg[k] = v[0][k] * u[k] * dh;
            du[k] = v[0][k] * h;
          }
          store4(P.o0 + o, dg);
          store4(P.o1 + o, du);
        }
      }
    }
    __syncwarp();
    // nobody reads this part any more (before it is overwritten, or the CTA ends)
    if (parts > 1) tc::cluster_sync();
    else __syncthreads();
  }
  tc::tc_fence_before();
  __syncthreads();
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

// A weight [rows][cols] as stored; mn: the products' rows run along cols.
cudaError_t weight_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, bool mn) {
  const uint64_t d[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t s[1] = {(uint64_t)cols * 2};
  const uint32_t b[2] = {64, mn ? 64u : (uint32_t)few::TM};
  return make_tmap_bf16(m, p, 2, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Activations [planes][t][K]
cudaError_t token_map(CUtensorMap* m, const void* p, int64_t t, int64_t K, int planes, int np) {
  const uint64_t d[3] = {(uint64_t)K, (uint64_t)t, (uint64_t)planes};
  const uint64_t s[2] = {(uint64_t)K * 2, (uint64_t)K * t * 2};
  const uint32_t b[3] = {64, (uint32_t)np, 1};
  return make_tmap_bf16(m, p, 3, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <FewEpi E, bool MN> cudaError_t launch(FewP& P, const FewArgs& f, int64_t K, cudaStream_t s) {
  using namespace few;
  constexpr int NW = E == FEW_GATE ? 2 : 1;
  P.t = f.t;
  P.act = f.act;
  P.status = f.st;
  P.wait_ns = tc::wait_limit(f.wait_ns);
  P.kblocks = (int)((K + TK - 1) / TK);
  P.acc1 = (uint32_t)((P.np + 31) / 32 * 32);
  P.tmem_cols = 32;
  while (P.tmem_cols < NW * P.acc1) P.tmem_cols *= 2;
  const int per_sm = P.tmem_cols <= 256 ? 2 : 1;
  const int stage = NW * WBYTES + P.np * TK * 2;
  const int room = per_sm == 2 ? HALF_SMEM : FULL_SMEM;
  P.stages = room / stage < MAXST ? room / stage : MAXST;
  const int ring = P.stages * stage;
  P.chunk = ring / (NW * TM * 4) / 16 * 16;
  const int64_t tiles = (P.rows + TM - 1) / TM;
  // up to 8 kLongSum k come here
  const int64_t nk = (int64_t)P.nseg * P.kblocks;
  const int least = (int)((nk + kLongSum / TK - 1) / (kLongSum / TK));
  const int parts = split_sum(tiles, nk, per_sm, least, NW, BLOCK_NS, FIXED_NS);
  auto kern = k_ffn_few<E, MN>;
  TRY(allow_smem(kern, FULL_SMEM + TAIL));
  return launch_after(kern, (unsigned)(tiles * parts), NT, ring + TAIL, (unsigned)parts, s, P);
}

FewP base(const FewArgs& f, int64_t rows, int nseg) {
  FewP P{};
  P.rows = rows;
  P.nseg = nseg;
  P.np = (int)((f.t + 15) / 16 * 16);
  return P;
}

using bf16 = __nv_bfloat16;

}  // namespace

cudaError_t few_gate(const FewArgs& f, void* a, float* g, float* u, cudaStream_t s) {
  FewP P = base(f, f.F, 1);
  TRY(weight_map(&P.w[0], f.wg, f.F, f.C, false));
  TRY(weight_map(&P.w[1], f.wu, f.F, f.C, false));
  TRY(token_map(&P.x, f.x, f.t, f.C, 1, P.np));
  P.o0 = (bf16*)a;
  P.g = g;
  P.u = u;
  return launch<FEW_GATE, false>(P, f, f.C, s);
}

cudaError_t few_down(const FewArgs& f, const void* a, void* y, cudaStream_t s) {
  FewP P = base(f, f.C, 1);
  P.early = true;
  TRY(weight_map(&P.w[0], f.wd, f.C, f.F, false));
  TRY(token_map(&P.x, a, f.t, f.F, 1, P.np));
  P.o0 = (bf16*)y;
  return launch<FEW_STORE, false>(P, f, f.F, s);
}

cudaError_t few_dgate(const FewArgs& f, const float* g, const float* u, void* d, cudaStream_t s) {
  FewP P = base(f, f.F, 1);
  P.beside = true;
  TRY(weight_map(&P.w[0], f.wd, f.C, f.F, true));
  TRY(token_map(&P.x, f.gy, f.t, f.C, 1, P.np));
  P.o0 = (bf16*)d;
  P.o1 = (bf16*)d + f.t * f.F;
  P.g = const_cast<float*>(g);
  P.u = const_cast<float*>(u);
  return launch<FEW_DGATE, true>(P, f, f.C, s);
}

cudaError_t few_grad_x(const FewArgs& f, const void* d, void* gx, cudaStream_t s) {
  FewP P = base(f, f.C, 2);
  P.early = true;
  TRY(weight_map(&P.w[0], f.wg, f.F, f.C, true));
  TRY(weight_map(&P.w[1], f.wu, f.F, f.C, true));
  TRY(token_map(&P.x, d, f.t, f.F, 2, P.np));
  P.o0 = (bf16*)gx;
  return launch<FEW_STORE, true>(P, f, f.F, s);
}

#undef TRY

}  // namespace mhc
