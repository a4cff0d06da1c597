// k_ffn_tc.cu -- the matrix products of the gated feed-forward block on the
// 5th-generation tensor cores.
//
//   D[m][n] = sum_k A(m, k) B(n, k)
//
// with either operand stored along k or along its own rows, and four epilogues:
//   EPI_STORE  D itself
//   EPI_GATE   two products at once (A = x, B = w_gate and w_up): act(g) u
//   EPI_KEEP   the same, and g and u themselves (the backward's recompute)
//   EPI_DGATE  D = da: reads g and u, writes dg = da u act'(g), du = da act(g)
//
// Two CTAs (a cluster, one CTA per SM) make one 256 x 256 tile with paired
// MMAs (cta_group::2, 256 x 256 x 16): each brings 128 rows of A and 128 of B
// per 64-wide k block into a six-stage ring by TMA (32 KB a stage and CTA) and
// holds 128 rows of D in its TMEM, so an SM reads 64 bytes of operands from L2
// per 8192 multiply-adds where a single-CTA 128 x 256 tile would read 96.  Two
// accumulators (all 512 TMEM columns) let the epilogue of one tile run under the
// products of the next.  Tiles go over the pairs in bands of eight row tiles, so
// that the tiles in flight share operands in L2.
//
// fp32 operands come as three bf16 planes each (their exact split, split3);
// the six products of planes whose sum of orders is at most two are taken in one
// accumulator, the smallest first.  What is left out is below 2^-25 of a product.
//
// Warps of a CTA: 0 TMA; 1 the MMAs (first CTA only); 2 TMEM; 4-7 the epilogue.
// Both CTAs' copies complete on the first CTA's barriers.  (A thread of the
// second CTA that waited for its copies and then arrived there, an arrive with
// release at cluster scope, took about 0.9 us per stage: 600 TFLOP/s in all.)
// Every wait is bounded as in the other tensor-core kernels: on timeout the
// kernel records MHC_ERR_TIMEOUT, drains what it issued and returns.
#include "ffn_common.cuh"
#include "mhc_dispatch.h"
#include "tc_pair.cuh"

namespace mhc {

namespace ftc {
constexpr int TM = 256, TN = 256, TK = 64;  // the pair's tile, and the k block
constexpr int HALF = 128;                   // rows of A and of B that one CTA brings
constexpr int OPND = HALF * TK * 2;         // 16 KB
constexpr int STAGE = 2 * OPND;
constexpr int NS = 6;
constexpr int OUT = 32 * 128;               // one staged output box: 32 rows of 128 bytes
constexpr int NEPI = 4;                     // epilogue warps, two output boxes each
constexpr int OUT_OFF = NS * STAGE;
constexpr int BAR_OFF = OUT_OFF + NEPI * 2 * OUT;
constexpr int SMEM = BAR_OFF + 256 + 1024;
constexpr int NT = 256;
constexpr int BAND = 8;
static_assert(SMEM <= 232448, "shared memory");
}  // namespace ftc

namespace {

enum Epi { EPI_STORE, EPI_GATE, EPI_KEEP, EPI_DGATE };

constexpr int kMaxSegs = 12;

// One launch.  Segment s multiplies plane ap of A's map am by plane bp of B's
// map bm; all segments of a tile add into one accumulator.
struct GemmArgs {
  CUtensorMap a[2], b[2], d[3];
  uint8_t am[kMaxSegs], ap[kMaxSegs], bm[kMaxSegs], bp[kMaxSegs];
  int nseg, kblocks;
  int mt, nt, nz;         // tiles of a problem; problems (a plane of A and a map of D each)
  int zplanes;            // planes of A per problem
  int64_t M, N;           // rows and columns of D (columns of one product for GATE, KEEP)
  const void *g, *u;      // EPI_DGATE
  int act;
  int* status;
  uint64_t wait_ns;
};

// A tile's place: problem z, row tile, column tile; bands of BAND row tiles, row
// tiles fastest.
__device__ __forceinline__ void tile_at(const GemmArgs& P, int64_t id, int& z, int& mi, int& ni) {
  const int64_t per = (int64_t)P.mt * P.nt;
  z = (int)(id / per);
  id -= (int64_t)z * per;
  const int64_t band = id / ((int64_t)ftc::BAND * P.nt);
  const int m0 = (int)band * ftc::BAND;
  const int rows = P.mt - m0 < ftc::BAND ? P.mt - m0 : ftc::BAND;
  const int64_t in = id - band * ftc::BAND * P.nt;
  ni = (int)(in / rows);
  mi = m0 + (int)(in % rows);
}

// One operand half of a stage: 128 rows x 64 k.  Stored along k: one box.
// Stored along its rows (MN): two boxes of 64 rows.
template <bool MN>
__device__ __forceinline__ void load_half(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int row0, int k0, int plane, uint64_t pol) {
  if (MN) {
    tc::tma2_load_3d(dst, map, bar, row0, k0, plane, pol);
    tc::tma2_load_3d(dst + ftc::OPND / 2, map, bar, row0 + 64, k0, plane, pol);
  } else {
    tc::tma2_load_3d(dst, map, bar, k0, row0, plane, pol);
  }
}
// The descriptor of the k-th 16-wide slice of that half.
template <bool MN> __device__ __forceinline__ uint64_t half_desc(uint32_t base, int k) {
  return MN ? tc::smem_desc(base + k * 2048, ftc::OPND / 2, 1024, tc::SWZ_128B)
            : tc::smem_desc(base + k * 32, 16, 1024, tc::SWZ_128B);
}

// An epilogue warp's output boxes: 32 rows of 128 bytes each, two in turn.
struct Stager {
  uint8_t* buf;
  int n, lane;
  __device__ __forceinline__ uint8_t* next() {
    if (lane == 0) tc::bulk_wait_read<1>();
    __syncwarp();
    return buf + (n++ & 1) * ftc::OUT;
  }
  // piece p (16 bytes) of this lane's row
  __device__ __forceinline__ void put(uint8_t* b, int p, uint4 v) {
    *reinterpret_cast<uint4*>(b + lane * 128 + ((p ^ (lane & 7)) << 4)) = v;
  }
  __device__ __forceinline__ void send(uint8_t* b, const CUtensorMap* map, int64_t col,
                                       int64_t row, int plane, bool inside) {
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (inside) tc::tma_store_3d(map, tc::smem_u32(b), (int)col, (int)row, plane);
      tc::bulk_commit();
    }
  }
};

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 values of this lane's row to columns [32 half, 32 half + 32) of a bf16 box.
__device__ __forceinline__ void put_bf16(Stager& st, uint8_t* b, int half, const float (&v)[32]) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    st.put(b, 4 * half + p,
           make_uint4(bf2(v[8 * p], v[8 * p + 1]), bf2(v[8 * p + 2], v[8 * p + 3]),
                      bf2(v[8 * p + 4], v[8 * p + 5]), bf2(v[8 * p + 6], v[8 * p + 7])));
}
__device__ __forceinline__ void put_f32(Stager& st, uint8_t* b, const float (&v)[32]) {
#pragma unroll
  for (int p = 0; p < 8; ++p)
    st.put(b, p, make_uint4(__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]),
                            __float_as_uint(v[4 * p + 2]), __float_as_uint(v[4 * p + 3])));
}

// A 64-column chunk of this warp's 32 rows.  bf16: one box.  fp32: the three
// bf16 planes of the values (SPLIT; they are the next product's operand) or the
// values themselves as two boxes.
template <bool F32, bool SPLIT>
__device__ __forceinline__ void emit(Stager& st, const CUtensorMap* map, int64_t col, int64_t row,
                                     int plane, int64_t M, int64_t N, float (&v0)[32],
                                     float (&v1)[32]) {
  const bool in = row < M && col < N;
  if (!F32) {
    uint8_t* b = st.next();
    put_bf16(st, b, 0, v0);
    put_bf16(st, b, 1, v1);
    st.send(b, map, col, row, plane, in);
  } else if (SPLIT) {
#pragma unroll 1
    for (int pl = 0; pl < 3; ++pl) {
      uint8_t* b = st.next();
      float t0[32], t1[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float h, m, l;
        split3(v0[i], h, m, l);
        t0[i] = pl == 0 ? h : pl == 1 ? m : l;
        split3(v1[i], h, m, l);
        t1[i] = pl == 0 ? h : pl == 1 ? m : l;
      }
      put_bf16(st, b, 0, t0);
      put_bf16(st, b, 1, t1);
      st.send(b, map, col, row, 3 * plane + pl, in);
    }
  } else {
    uint8_t* b = st.next();
    put_f32(st, b, v0);
    st.send(b, map, col, row, plane, in);
    b = st.next();
    put_f32(st, b, v1);
    st.send(b, map, col + 32, row, plane, row < M && col + 32 < N);
  }
}

// 32 columns of this lane's row of g or u; columns past the end are not read.
template <bool F32>
__device__ __forceinline__ void row32(const void* base, int64_t row, int64_t col, int64_t M,
                                      int64_t N, float (&v)[32]) {
  constexpr int VN = F32 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < 32; i += VN) {
    if (row < M && col + i < N) {
      if (F32) {
        const float4 q = *reinterpret_cast<const float4*>((const float*)base + row * N + col + i);
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      } else {
        float t[8];
        Vec<__nv_bfloat16>::load((const __nv_bfloat16*)base + row * N + col + i, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i + e] = t[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < VN; ++e) v[i + e] = 0.0f;
    }
  }
}

template <Epi E, bool AMN, bool BMN, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(ftc::NT, 1)
    k_ffn_tc(const __grid_constant__ GemmArgs P) {
  using namespace ftc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  // full[NS] empty[NS] tfull[2] tempty[2] fin
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NS + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full = [&](int s) { return tc::smem_u32(bars + s); };
  auto empty = [&](int s) { return tc::smem_u32(bars + NS + s); };
  auto tfull = [&](int b) { return tc::smem_u32(bars + 2 * NS + b); };
  auto tempty = [&](int b) { return tc::smem_u32(bars + 2 * NS + 2 + b); };
  const uint32_t fin_bar = tc::smem_u32(bars + 2 * NS + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)tc::cluster_rank();
  const int64_t pair = blockIdx.x / 2, npairs = gridDim.x / 2;
  const int64_t tiles = (int64_t)P.mt * P.nt * P.nz;
  constexpr bool DUAL = E == EPI_GATE || E == EPI_KEEP;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(full(s), 1);  // the first CTA's: the bytes of both CTAs
      tc::mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tfull(b), 1);
      tc::mbar_init(tempty(b), 2 * NEPI);
    }
    tc::mbar_init(fin_bar, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch_desc(&P.a[0]);
    tc::tma_prefetch_desc(&P.b[0]);
    tc::tma_prefetch_desc(&P.d[0]);
  }
  if (warp == 2) {
    tc::tmem_alloc2(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish2();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // the partner's barriers exist
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto give_up = [&]() {
    *abort_flag = 1;
    flag_status(P.status, MHC_ERR_TIMEOUT);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      const uint64_t pol = tc::policy_evict_normal();
      int64_t it = 0;
      bool ok = true;
      for (int64_t id = pair; id < tiles && ok; id += npairs) {
        int z, mi, ni;
        tile_at(P, id, z, mi, ni);
        const int arow = mi * TM + rank * HALF;
        const int brow = DUAL ? ni * HALF : ni * TN + rank * HALF;
        for (int sg = 0; sg < P.nseg && ok; ++sg) {
          const CUtensorMap* am = &P.a[P.am[sg]];
          const CUtensorMap* bm = &P.b[DUAL ? rank : P.bm[sg]];
          const int ap = P.ap[sg] + z * P.zplanes, bp = P.bp[sg];
          for (int kb = 0; kb < P.kblocks; ++kb, ++it) {
            const int s = (int)(it % NS);
            if (it >= NS && !tc::mbar_pipe_wait<false>(empty(s), ((uint32_t)(it / NS) & 1u) ^ 1u,
                                                       abort_flag, P.wait_ns)) {
              give_up();
              ok = false;
              break;
            }
            const uint32_t base = tc::smem_u32(smem + s * STAGE);
            if (rank == 0) tc::mbar_arrive_expect_tx(full(s), 2 * STAGE);
            const uint32_t bar = tc::map_cta(full(s), 0);
            load_half<AMN>(base, am, bar, arow, kb * TK, ap, pol);
            load_half<BMN>(base + OPND, bm, bar, brow, kb * TK, bp, pol);
          }
        }
      }
      // Every copy has landed before the CTA can exit.  After an ordinary run the
      // MMAs have waited for all of them; after a give-up the first CTA waits for
      // the rounds that both CTAs issued, and the second, whose copies may be
      // ahead of the first CTA's count, for a millisecond.
      if (rank == 0) {
        for (int64_t i = it > NS ? it - NS : 0; i < it; ++i)
          if (!tc::mbar_wait(full((int)(i % NS)), (uint32_t)(i / NS) & 1u, nullptr,
                             tc::kDrainWaitNs))
            break;
      } else if (!ok) {
        const uint64_t t0 = tc::global_ns();
        while (tc::global_ns() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = tc::idesc_bf16(TM, TN, AMN, BMN);
      int64_t it = 0;
      int n = 0;
      bool ok = true, any = false;
      for (int64_t id = pair; id < tiles && ok; id += npairs, ++n) {
        const int buf = n & 1;
        if (n >= 2 && !tc::mbar_pipe_wait<true>(tempty(buf), ((uint32_t)(n / 2) & 1u) ^ 1u,
                                                abort_flag, P.wait_ns)) {
          give_up();
          break;
        }
        tc::tc_fence_after();
        for (int j = 0; j < P.nseg * P.kblocks; ++j, ++it) {
          const int s = (int)(it % NS);
          if (!tc::mbar_pipe_wait<false>(full(s), (uint32_t)(it / NS) & 1u, abort_flag,
                                         P.wait_ns)) {
            give_up();
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t base = tc::smem_u32(smem + s * STAGE);
#pragma unroll
          for (int k = 0; k < TK / 16; ++k)
            tc::mma2_bf16(tmem + buf * TN, half_desc<AMN>(base, k), half_desc<BMN>(base + OPND, k),
                          idesc, (j | k) != 0 ? 1u : 0u);
          any = true;
          tc::mma2_commit(empty(s));
        }
        if (ok) tc::mma2_commit(tfull(buf));
      }
      // every MMA issued here has finished before TMEM is freed
      if (any) {
        tc::mma2_commit(fin_bar);
        tc::mbar_wait(fin_bar, 0, nullptr, tc::kDrainWaitNs);
      }
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may read
    Stager st{smem + OUT_OFF + q * 2 * OUT, 0, lane};
    // a tile's products may rightly take longer than one wait: 4 us per k block more
    const uint64_t tile_ns = P.wait_ns + (uint64_t)P.nseg * P.kblocks * 4000;
    int n = 0;
    for (int64_t id = pair; id < tiles; id += npairs, ++n) {
      int z, mi, ni;
      tile_at(P, id, z, mi, ni);
      const int buf = n & 1;
      bool ok = tc::mbar_pipe_wait<false>(tfull(buf), (uint32_t)(n / 2) & 1u, abort_flag, tile_ns);
      if (!ok && !*abort_flag) give_up();
      ok = __all_sync(0xffffffffu, ok);  // the TMEM loads below are warp-collective
      if (!ok) break;
      tc::tc_fence_after();
      const int64_t row0 = (int64_t)mi * TM + rank * HALF + 32 * q, row = row0 + lane;
      const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16) + buf * TN;
      if (DUAL) {
#pragma unroll 1
        for (int c = 0; c < HALF; c += 64) {
          const int64_t col = (int64_t)ni * HALF + c;
          if (E == EPI_GATE) {
            float v[2][32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float u[32];
              tc::tmem_get32x2(ta + c + 32 * h, ta + HALF + c + 32 * h, v[h], u);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[h][i] = gate<!F32>(P.act, v[h][i]) * u[i];
            }
            emit<F32, true>(st, &P.d[0], col, row0, 0, P.M, P.N, v[0], v[1]);
          } else {
            float g[2][32], u[2][32];
            tc::tmem_get32x2(ta + c, ta + c + 32, g[0], g[1]);
            emit<F32, false>(st, &P.d[1], col, row0, 0, P.M, P.N, g[0], g[1]);
            tc::tmem_get32x2(ta + HALF + c, ta + HALF + c + 32, u[0], u[1]);
            emit<F32, false>(st, &P.d[2], col, row0, 0, P.M, P.N, u[0], u[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 32; ++i) g[h][i] = gate<!F32>(P.act, g[h][i]) * u[h][i];
            emit<F32, true>(st, &P.d[0], col, row0, 0, P.M, P.N, g[0], g[1]);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < TN; c += 64) {
          const int64_t col = (int64_t)ni * TN + c;
          if (E == EPI_STORE) {
            float v[2][32];
            tc::tmem_get32x2(ta + c, ta + c + 32, v[0], v[1]);
            emit<F32, false>(st, &P.d[z], col, row0, 0, P.M, P.N, v[0], v[1]);
          } else {
            float dg[2][32], du[2][32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float u[32], da[32];
              row32<F32>(P.g, row, col + 32 * h, P.M, P.N, dg[h]);
              row32<F32>(P.u, row, col + 32 * h, P.M, P.N, u);
              tc::tmem_get32(ta + c + 32 * h, da);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float a, da_dg;
                gate_both<!F32>(P.act, dg[h][i], a, da_dg);
                dg[h][i] = da[i] * u[i] * da_dg;
                du[h][i] = da[i] * a;
              }
            }
            emit<F32, true>(st, &P.d[0], col, row0, 0, P.M, P.N, dg[0], dg[1]);
            emit<F32, true>(st, &P.d[0], col, row0, 1, P.M, P.N, du[0], du[1]);
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::map_cta(tempty(buf), 0));
    }
    if (lane == 0) tc::bulk_wait<0>();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // no arrival or MMA of the partner is under way any more
  // the last commit of the first CTA has arrived here too
  if (rank == 1 && threadIdx.x == 0) tc::mbar_wait(fin_bar, 0, nullptr, tc::kDrainWaitNs);
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc2(tmem, 512);
  }
}

// [rows][cols] fp32 -> three bf16 planes of the same shape.
__global__ void __launch_bounds__(256) k_split3(int64_t n, const float* __restrict__ v,
                                                __nv_bfloat16* __restrict__ out) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n;
       i += (int64_t)gridDim.x * 256 * 8) {
    float p[3][8];
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      const float4 q = __ldcs(reinterpret_cast<const float4*>(v + i + h));
      const float w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) split3(w[e], p[0][h + e], p[1][h + e], p[2][h + e]);
    }
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
      *reinterpret_cast<uint4*>(out + pl * n + i) = Vec<__nv_bfloat16>::pack(p[pl]);
  }
}

cudaError_t split3_launch(int64_t n, const void* v, void* out, cudaStream_t s) {
  const int64_t blocks = (n / 8 + 255) / 256;
  k_split3<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(n, (const float*)v,
                                                                    (__nv_bfloat16*)out);
  return cudaGetLastError();
}

// A matrix in memory: [planes][rows][cols], bf16 (operands) or fp32 (results).
struct Mat {
  const void* p;
  int64_t rows, cols;
  int planes;
  bool f32;
};

// mn: the operand's own rows run along the stored columns.
cudaError_t operand_map(CUtensorMap* m, const Mat& x, bool mn) {
  const uint64_t d[3] = {(uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.planes};
  const uint64_t s[2] = {(uint64_t)x.cols * 2, (uint64_t)x.cols * x.rows * 2};
  const uint32_t b[3] = {64, mn ? 64u : (uint32_t)ftc::HALF, 1};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x.p, 3, d, s, b,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
cudaError_t result_map(CUtensorMap* m, const Mat& x) {
  const uint64_t e = x.f32 ? 4 : 2;
  const uint64_t d[3] = {(uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.planes};
  const uint64_t s[2] = {(uint64_t)x.cols * e, (uint64_t)x.cols * x.rows * e};
  const uint32_t b[3] = {(uint32_t)(128 / e), 32, 1};
  return make_tmap(m, x.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   x.p, 3, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// The segments of `pairs` products of operands with np planes each (1, or 3 with
// the smallest of the six products first); pair i takes planes [np i, np i + np)
// of A and map i of B.
void segments(GemmArgs& P, int pairs, int np) {
  P.nseg = 0;
  for (int order = np - 1; order >= 0; --order)
    for (int pr = 0; pr < pairs; ++pr)
      for (int i = 0; i <= order; ++i) {
        P.am[P.nseg] = 0;
        P.ap[P.nseg] = (uint8_t)(np * pr + i);
        P.bm[P.nseg] = (uint8_t)pr;
        P.bp[P.nseg] = (uint8_t)(order - i);
        ++P.nseg;
      }
}

template <Epi E, bool AMN, bool BMN, bool F32> cudaError_t launch(GemmArgs& P, cudaStream_t s) {
  auto kern = k_ffn_tc<E, AMN, BMN, F32>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ftc::SMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  const int64_t tiles = (int64_t)P.mt * P.nt * P.nz, pairs = sms / 2;
  kern<<<(unsigned)(2 * (tiles < pairs ? tiles : pairs)), ftc::NT, ftc::SMEM, s>>>(P);
  return cudaGetLastError();
}

int tiles_of(int64_t n, int t) { return (int)((n + t - 1) / t); }

// Operands as the products take them: the caller's bf16 arrays, or the split
// copies of its fp32 arrays.
struct Ffn {
  int64_t t, C, F;
  int act, np;  // planes per operand: 1 or 3
  const void *x, *wg, *wu, *wd, *gy;
  int* st;
  int64_t wait_ns;
};

GemmArgs base_args(const Ffn& f) {
  GemmArgs P{};
  P.nz = 1;
  P.act = f.act;
  P.status = f.st;
  P.wait_ns = tc::wait_limit(f.wait_ns);
  return P;
}

#define TRY(call)                         \
  do {                                    \
    const cudaError_t e_ = (call);        \
    if (e_ != cudaSuccess) return e_;     \
  } while (0)

// a = act(x wg^T) * (x wu^T) to a (and g, u where they are kept)
template <bool F32> cudaError_t gate_product(const Ffn& f, void* a, void* g, void* u,
                                             cudaStream_t s) {
  GemmArgs P = base_args(f);
  TRY(operand_map(&P.a[0], {f.x, f.t, f.C, f.np, false}, false));
  TRY(operand_map(&P.b[0], {f.wg, f.F, f.C, f.np, false}, false));
  TRY(operand_map(&P.b[1], {f.wu, f.F, f.C, f.np, false}, false));
  TRY(result_map(&P.d[0], {a, f.t, f.F, f.np, false}));
  segments(P, 1, f.np);
  P.kblocks = tiles_of(f.C, ftc::TK);
  P.mt = tiles_of(f.t, ftc::TM);
  P.nt = tiles_of(f.F, ftc::HALF);
  P.M = f.t;
  P.N = f.F;
  if (g == nullptr) return launch<EPI_GATE, false, false, F32>(P, s);
  TRY(result_map(&P.d[1], {g, f.t, f.F, 1, F32}));
  TRY(result_map(&P.d[2], {u, f.t, f.F, 1, F32}));
  return launch<EPI_KEEP, false, false, F32>(P, s);
}

// D (rows x cols) = A B^T over K; A, B given as stored
template <Epi E, bool AMN, bool BMN, bool F32>
cudaError_t product(GemmArgs& P, const Ffn& f, const Mat& A, const Mat& B, int64_t K, int64_t M,
                    int64_t N, cudaStream_t s) {
  TRY(operand_map(&P.a[0], A, AMN));
  TRY(operand_map(&P.b[0], B, BMN));
  P.kblocks = tiles_of(K, ftc::TK);
  P.mt = tiles_of(M, ftc::TM);
  P.nt = tiles_of(N, ftc::TN);
  P.M = M;
  P.N = N;
  return launch<E, AMN, BMN, F32>(P, s);
}

template <bool F32> cudaError_t fwd(const Ffn& f, void* y, void* a, cudaStream_t s) {
  TRY(gate_product<F32>(f, a, nullptr, nullptr, s));
  GemmArgs P = base_args(f);
  segments(P, 1, f.np);
  TRY(result_map(&P.d[0], {y, f.t, f.C, 1, F32}));
  return product<EPI_STORE, false, false, F32>(P, f, {a, f.t, f.F, f.np, false},
                                               {f.wd, f.C, f.F, f.np, false}, f.F, f.t, f.C, s);
}

// a [np][t][F], d [2 np][t][F] (dg, du), g and u [t][F] in the call's type.  For
// bf16 d may be the same memory as g and u: a tile reads its g and u before it
// writes dg and du there.
template <bool F32>
cudaError_t bwd(const Ffn& f, void* gx, void* gwg, void* gwu, void* gwd, void* a, void* d, void* g,
                void* u, cudaStream_t s) {
  const int np = f.np;
  TRY(gate_product<F32>(f, a, g, u, s));
  {
    GemmArgs P = base_args(f);
    segments(P, 1, np);
    TRY(result_map(&P.d[0], {d, f.t, f.F, 2 * np, false}));
    P.g = g;
    P.u = u;
    TRY((product<EPI_DGATE, false, true, F32>(P, f, {f.gy, f.t, f.C, np, false},
                                              {f.wd, f.C, f.F, np, false}, f.C, f.t, f.F, s)));
  }
  {
    GemmArgs P = base_args(f);
    segments(P, 1, np);
    TRY(result_map(&P.d[0], {gwd, f.C, f.F, 1, F32}));
    TRY((product<EPI_STORE, true, true, F32>(P, f, {f.gy, f.t, f.C, np, false},
                                             {a, f.t, f.F, np, false}, f.t, f.C, f.F, s)));
  }
  {
    GemmArgs P = base_args(f);
    segments(P, 1, np);
    P.nz = 2;
    P.zplanes = np;
    TRY(result_map(&P.d[0], {gwg, f.F, f.C, 1, F32}));
    TRY(result_map(&P.d[1], {gwu, f.F, f.C, 1, F32}));
    TRY((product<EPI_STORE, true, true, F32>(P, f, {d, f.t, f.F, 2 * np, false},
                                             {f.x, f.t, f.C, np, false}, f.t, f.F, f.C, s)));
  }
  GemmArgs P = base_args(f);
  segments(P, 2, np);
  TRY(result_map(&P.d[0], {gx, f.t, f.C, 1, F32}));
  TRY(operand_map(&P.b[1], {f.wu, f.F, f.C, np, false}, true));
  return product<EPI_STORE, false, true, F32>(P, f, {d, f.t, f.F, 2 * np, false},
                                              {f.wg, f.F, f.C, np, false}, f.F, f.t, f.C, s);
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Workspaces.  bf16: a; with the backward also dg and du (first g and u).
// fp32: the split copies of the inputs, the three planes of a (and of dg, du),
// and g, u as they are.
struct Layout {
  size_t a, d, g, u, x, wg, wu, wd, gy, total;
};
Layout layout(bool f32, bool backward, int64_t t, int64_t C, int64_t F) {
  Layout w{};
  size_t off = 0;
  const size_t np = f32 ? 3 : 1, hid = (size_t)t * F, io = (size_t)t * C, wt = (size_t)F * C;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = up(off + bytes);
    return o;
  };
  w.a = take(hid * 2 * np);
  if (backward) {
    w.d = take(hid * 2 * 2 * np);
    w.g = f32 ? take(hid * 4) : w.d;
    w.u = f32 ? take(hid * 4) : w.d + hid * 2;
  }
  if (f32) {
    w.x = take(io * 6);
    w.wg = take(wt * 6);
    w.wu = take(wt * 6);
    w.wd = take(wt * 6);
    if (backward) w.gy = take(io * 6);
  }
  w.total = off;
  return w;
}

// The inputs' split copies (fp32), or the inputs themselves.
cudaError_t operands(Ffn& f, bool f32, const Layout& w, char* ws, cudaStream_t s) {
  f.np = f32 ? 3 : 1;
  if (!f32) return cudaSuccess;
  const int64_t io = f.t * f.C, wt = f.F * f.C;
  TRY(split3_launch(io, f.x, ws + w.x, s));
  TRY(split3_launch(wt, f.wg, ws + w.wg, s));
  TRY(split3_launch(wt, f.wu, ws + w.wu, s));
  TRY(split3_launch(wt, f.wd, ws + w.wd, s));
  f.x = ws + w.x;
  f.wg = ws + w.wg;
  f.wu = ws + w.wu;
  f.wd = ws + w.wd;
  if (f.gy) {
    TRY(split3_launch(io, f.gy, ws + w.gy, s));
    f.gy = ws + w.gy;
  }
  return cudaSuccess;
}

}  // namespace

size_t ffn_fwd_workspace_bytes(int dtype, int64_t t, int64_t C, int64_t F) {
  return layout(dtype != MHC_DTYPE_BF16, false, t, C, F).total;
}

size_t ffn_bwd_workspace_bytes(int dtype, int64_t t, int64_t C, int64_t F) {
  return layout(dtype != MHC_DTYPE_BF16, true, t, C, F).total;
}

cudaError_t ffn_fwd_dispatch(int dtype, int act, int64_t t, int64_t C, int64_t F, const void* x,
                             const void* wg, const void* wu, const void* wd, void* y, void* ws,
                             int* st, int64_t wait_ns, cudaStream_t s) {
  const bool f32 = dtype != MHC_DTYPE_BF16;
  const Layout w = layout(f32, false, t, C, F);
  Ffn f{t, C, F, act, 1, x, wg, wu, wd, nullptr, st, wait_ns};
  TRY(operands(f, f32, w, (char*)ws, s));
  char* b = (char*)ws;
  return f32 ? fwd<true>(f, y, b + w.a, s) : fwd<false>(f, y, b + w.a, s);
}

cudaError_t ffn_bwd_dispatch(int dtype, int act, int64_t t, int64_t C, int64_t F, const void* x,
                             const void* wg, const void* wu, const void* wd, const void* gy,
                             void* gx, void* gwg, void* gwu, void* gwd, void* ws, int* st,
                             int64_t wait_ns, cudaStream_t s) {
  const bool f32 = dtype != MHC_DTYPE_BF16;
  const Layout w = layout(f32, true, t, C, F);
  Ffn f{t, C, F, act, 1, x, wg, wu, wd, gy, st, wait_ns};
  char* b = (char*)ws;
  TRY(operands(f, f32, w, b, s));
  return f32 ? bwd<true>(f, gx, gwg, gwu, gwd, b + w.a, b + w.d, b + w.g, b + w.u, s)
             : bwd<false>(f, gx, gwg, gwu, gwd, b + w.a, b + w.d, b + w.g, b + w.u, s);
}

#undef TRY

}  // namespace mhc
