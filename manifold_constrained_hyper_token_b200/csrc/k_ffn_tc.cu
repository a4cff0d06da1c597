// k_ffn_tc.cu -- the matrix products of the gated feed-forward block on the
// 5th-generation tensor cores.
//
//   D[m][n] = sum_k A(m, k) B(n, k)
//
// with either operand stored along k or along its own rows, and five epilogues:
//   EPI_STORE  D itself
//   EPI_PART   D's fp32 sums over a part of k (k_join adds the parts)
//   EPI_GATE   two products at once (A = x, B = w_gate and w_up): act(g) u
//   EPI_KEEP   the same, and g and u themselves (the backward's recompute)
//   EPI_DGATE  D = da: reads g and u, writes dg = da u act'(g), du = da act(g)
//
// Two CTAs (a cluster, one CTA per SM) make one 256 x TN tile with paired MMAs
// (cta_group::2, 256 x TN x 16): each brings 128 rows of A and TN / 2 of B per
// 64-wide k block into a six-stage ring by TMA and holds 128 rows of D in its
// TMEM.  With TN = 256 an SM reads 64 bytes of operands from L2 per 8192
// multiply-adds where a single-CTA 128 x 256 tile would read 96.  Two
// accumulators let the epilogue of one tile run under the products of the next.
// Tiles go over the pairs in bands of eight row tiles, so that the tiles in
// flight share operands in L2.
//
// fp32 operands come as three bf16 planes each (their exact split, split3x4).  A
// stage brings all planes of a 32-wide k block and six of the nine products of
// planes are taken, those whose orders add up to at most two; what is left out is
// 2^-24 of a product on average.  The tensor cores' adder cuts instead of rounding,
// about half a unit of the last place per 16-wide step, which adds up over a long
// sum (measured: 137 x 2^-24 at k = 5456).  So the first planes' products have
// accumulators of their own, which they leave every kChunk k blocks to be added
// up, rounded, in another TMEM region.  The other products are 2^-7 of them and
// less, five to each of theirs, and have one accumulator, which is emptied every
// kMinor such stays: what it loses by then is about 2^-20 of the sum of absolute
// products.  (Never emptied, it lost 2^-16.6 at k = 65536 and 2^-13.4 at 2^20.)
//
// bf16 sums stay in one accumulator for up to kLongSum k: plain products are split
// (plan), and the gate's and its derivative's over more channels (LONG) leave it as the
// first planes' sums do.
//
// The backward's g and u are kept in fp32: rounded to bf16 they would put as much
// error into dg and du as these take from their own rounding.
//
// Warps of a CTA: 0 TMA; 1 the MMAs (first CTA only); 2 TMEM; from 4 on the
// epilogue.
// Both CTAs' copies complete on the first CTA's barriers.  (A thread of the
// second CTA that waited for its copies and then arrived there, an arrive with
// release at cluster scope, took about 0.9 us per stage: 600 TFLOP/s in all.)
// Every wait is bounded as in the other tensor-core kernels: on timeout the
// kernel records MHC_ERR_TIMEOUT, drains what it issued and returns.
#include <algorithm>

#include "ffn_common.cuh"
#include "ffn_few.h"
#include "mhc_dispatch.h"
#include "tc_pair.cuh"

namespace mhc {

namespace ftc {
constexpr int TM = 256;           // the pair's rows
constexpr int HALF = 128;         // rows of A that one CTA brings
constexpr int BAND = 8;
constexpr int kChunk = 8;         // fp32: k blocks per stay of the first planes' products
constexpr int kMinor = 16;        // ... and such stays per stay of the others'
constexpr int BOX = 32 * 64;      // a staged box of results: 32 rows of 32 bf16 or 16 fp32

template <int TN, bool F32, bool MORE> struct Cfg {
  static constexpr int NEPI = MORE ? 8 : 4;             // epilogue warps
  static constexpr int NT = 128 + 32 * NEPI;
  static constexpr int TK = F32 ? 32 : 64;              // k block
  static constexpr int NP = F32 ? 3 : 1;                // planes of an operand
  static constexpr int NS = F32 ? 4 : 6;                // stages
  static constexpr int BROWS = TN / 2;                  // rows of B that one CTA brings
  static constexpr int APLANE = HALF * TK * 2, BPLANE = BROWS * TK * 2;
  static constexpr int ABYTES = NP * APLANE;
  static constexpr int STAGE = ABYTES + NP * BPLANE;
  static constexpr int OUT = (F32 ? 65536 : 32768) / NEPI;  // staged results per such warp
  static constexpr int OUT_OFF = NS * STAGE;
  static constexpr int BAR_OFF = OUT_OFF + NEPI * OUT;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  // TMEM columns: two accumulators; fp32: the lower planes' products, the sums
  static constexpr uint32_t MINOR = 2 * TN, SUMS = 3 * TN;
  static_assert(STAGE % 1024 == 0 && SMEM <= 232448, "shared memory");
  static_assert((F32 ? 4 : 2) * TN <= 512, "TMEM columns");
};
}  // namespace ftc

namespace {

enum Epi { EPI_STORE, EPI_GATE, EPI_KEEP, EPI_DGATE, EPI_PART };

// The epilogues with arithmetic take eight warps, two to a TMEM lane quarter: DGATE,
// T = 2368, C = 4096, F = 4736, 143 us with four warps, 116 with eight and g and u
// fetched ahead; T = 4096, C = F = 1024, forward pass (GATE) 47 -> 39 us, backward
// (KEEP) 134 -> 125.  Plain results gained nothing; fp32 stages more and has no room.
constexpr bool more_warps(Epi e, bool f32) {
  return !f32 && (e == EPI_GATE || e == EPI_KEEP || e == EPI_DGATE);
}

// One launch: the sum of nseg products into each tile, the s-th of A's planes
// from s NP on by B's map s.
struct GemmArgs {
  CUtensorMap a, b[2], d[3];
  int nseg, kblocks;
  int mt, nt, nz;         // tiles of a problem; problems (planes of A and a map of D each)
  int zplanes;            // planes of A per problem
  int split;              // PART: parts of k; part q of problem z goes to plane z split + q
  int64_t M, N;           // rows and columns of D (columns of one product for GATE, KEEP)
  const float *g, *u;     // EPI_DGATE
  int act;
  bool beside;            // needs nothing from the kernel before it
  int* status;
  uint64_t wait_ns;
};

// The stay in an accumulator that starts at k block j0 of a tile that ends at jb
// ends here.
template <bool F32, bool LONG> __device__ __forceinline__ int stay_end(int j0, int jb) {
  constexpr int chunk = F32 ? ftc::kChunk : (int)(kLongSum / 64);
  return !(F32 || LONG) || jb - j0 < chunk ? jb : j0 + chunk;
}

// ... and with it that of the lower planes' products.
__device__ __forceinline__ bool minor_end(int j1, int ja, int jb) {
  return j1 == jb || (j1 - ja) % (ftc::kChunk * ftc::kMinor) == 0;
}

// A tile's place: plane z of the results (problem z / split, part z % split), row
// tile, column tile, and its k blocks [ja, jb); bands of BAND row tiles, row tiles
// fastest.
__device__ __forceinline__ void tile_at(const GemmArgs& P, int64_t id, int& z, int& mi, int& ni,
                                        int& ja, int& jb) {
  const int64_t per = (int64_t)P.mt * P.nt, nk = (int64_t)P.nseg * P.kblocks;
  z = (int)(id / per);
  id -= (int64_t)z * per;
  const int q = z % P.split;
  ja = (int)(nk * q / P.split);
  jb = (int)(nk * (q + 1) / P.split);
  const int64_t band = id / ((int64_t)ftc::BAND * P.nt);
  const int m0 = (int)band * ftc::BAND;
  const int rows = P.mt - m0 < ftc::BAND ? P.mt - m0 : ftc::BAND;
  const int64_t in = id - band * ftc::BAND * P.nt;
  ni = (int)(in / rows);
  mi = m0 + (int)(in % rows);
}

// One operand of a stage, all its planes: ROWS rows x TK k.  Stored along k: one
// box [plane][row][k].  Stored along its rows (MN): boxes [plane][k][64 rows].
template <class G, int ROWS, bool MN>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int row0, int k0, int plane, uint64_t pol) {
  if (MN) {
#pragma unroll
    for (int r = 0; r < ROWS; r += 64)
      tc::tma2_load_3d(dst + (r / 64) * G::NP * G::TK * 128, map, bar, row0 + r, k0, plane, pol);
  } else {
    tc::tma2_load_3d(dst, map, bar, k0, row0, plane, pol);
  }
}
// The descriptor of the k-th 16-wide slice of a plane of that operand.
template <class G, int ROWS, bool MN>
__device__ __forceinline__ uint64_t rows_desc(uint32_t base, int plane, int k) {
  if (MN)
    return tc::smem_desc(base + plane * G::TK * 128 + k * 2048, G::NP * G::TK * 128, 1024,
                         tc::SWZ_128B);
  return tc::smem_desc(base + plane * ROWS * G::TK * 2 + k * 32, 16, G::TK * 16,
                       G::TK == 64 ? tc::SWZ_128B : tc::SWZ_64B);
}

// Row `lane` of a staged box (64-byte rows with the 64-byte swizzle): columns
// [16 g, 16 g + 16) of 32 bf16, or 16 fp32.
__device__ __forceinline__ uint4* box_piece(uint8_t* box, int lane, int p) {
  return reinterpret_cast<uint4*>(box + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4));
}
__device__ __forceinline__ void put_bf16(uint8_t* box, int lane, int g, const float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *box_piece(box, lane, 2 * g + p) =
        make_uint4(bf2(v[8 * p], v[8 * p + 1]), bf2(v[8 * p + 2], v[8 * p + 3]),
                   bf2(v[8 * p + 4], v[8 * p + 5]), bf2(v[8 * p + 6], v[8 * p + 7]));
}
__device__ __forceinline__ void put_f32(uint8_t* box, int lane, const float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *box_piece(box, lane, p) =
        make_uint4(__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]),
                   __float_as_uint(v[4 * p + 2]), __float_as_uint(v[4 * p + 3]));
}
// A value that the next product takes as an operand: itself in bf16, or its three
// planes in three boxes.
template <bool F32>
__device__ __forceinline__ void put_operand(uint8_t* box, int lane, int g, const float (&v)[16]) {
  if (!F32) {
    put_bf16(box, lane, g, v);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint2 h[2], m[2], l[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 8 * p + 4 * e;
        split3x4(make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]), h[e], m[e], l[e]);
      }
      *box_piece(box, lane, 2 * g + p) = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
      *box_piece(box + ftc::BOX, lane, 2 * g + p) = make_uint4(m[0].x, m[0].y, m[1].x, m[1].y);
      *box_piece(box + 2 * ftc::BOX, lane, 2 * g + p) = make_uint4(l[0].x, l[0].y, l[1].x, l[1].y);
    }
  }
}

// 16 columns of this lane's row of g or u, from column col on; what lies past the
// end is not read.
__device__ __forceinline__ void row16(const float* base, int64_t row, int64_t col, int64_t M,
                                      int64_t N, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < M && col + i < N)
      q = __ldcs(reinterpret_cast<const float4*>(base + row * N + col + i));
    v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
  }
}

template <Epi E, bool AMN, bool BMN, bool F32, int TN, bool LONG>
__global__ void __launch_bounds__(ftc::Cfg<TN, F32, more_warps(E, F32 || LONG)>::NT, 1)
    k_ffn_tc(const __grid_constant__ GemmArgs P) {
  using namespace ftc;
  using G = Cfg<TN, F32, more_warps(E, F32 || LONG)>;
  constexpr bool SUM = F32 || LONG;  // the results are sums of stays
  static_assert(!SUM || 4 * TN <= 512, "TMEM columns");
  constexpr int NEPI = G::NEPI;
  constexpr int STAGE = G::STAGE, NS = G::NS, TK = G::TK, HN = TN / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  // full[NS] empty[NS] tfull[2] tempty[2] mempty fin, the TMEM address and the abort
  // flag, the stages that this CTA's copies were issued for
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::BAR_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NS + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint64_t* issued = reinterpret_cast<volatile uint64_t*>(bars + 2 * NS + 7);
  auto full = [&](int s) { return tc::smem_u32(bars + s); };
  auto empty = [&](int s) { return tc::smem_u32(bars + NS + s); };
  auto tfull = [&](int b) { return tc::smem_u32(bars + 2 * NS + b); };
  auto tempty = [&](int b) { return tc::smem_u32(bars + 2 * NS + 2 + b); };
  const uint32_t mempty = tc::smem_u32(bars + 2 * NS + 4);  // fp32: the lower planes' sums
  const uint32_t fin_bar = tc::smem_u32(bars + 2 * NS + 5);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int rank = (int)tc::cluster_rank();
  const int64_t pair = blockIdx.x / 2, npairs = gridDim.x / 2;
  const int64_t tiles = (int64_t)P.mt * P.nt * P.nz * P.split;
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
    tc::mbar_init(mempty, 2 * NEPI);
    tc::mbar_init(fin_bar, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch_desc(&P.a);
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
  if (!P.beside) tc::grid_wait();
  tc::grid_release();
  const uint32_t tmem = *tmem_slot;

  auto give_up = [&]() {
    *abort_flag = 1;
    tc::st_cluster_u32(tc::map_cta(tc::smem_u32(tmem_slot + 1), (uint32_t)(rank ^ 1)), 1u);
    flag_status(P.status, MHC_ERR_TIMEOUT);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      const uint64_t pol = tc::policy_evict_normal();
      int64_t it = 0;
      bool ok = true;
      for (int64_t id = pair; id < tiles && ok; id += npairs) {
        int z, mi, ni, ja, jb;
        tile_at(P, id, z, mi, ni, ja, jb);
        const int arow = mi * TM + rank * HALF;
        const int brow = DUAL ? ni * HN : ni * TN + rank * HN;
        const int zplane = z / P.split * P.zplanes;
        int seg = ja / P.kblocks, kb = ja - seg * P.kblocks;
        for (int j = ja; j < jb; ++j, ++it) {
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
          load_rows<G, HALF, AMN>(base, &P.a, bar, arow, kb * TK, seg * G::NP + zplane, pol);
          load_rows<G, HN, BMN>(base + G::ABYTES, &P.b[DUAL ? rank : seg], bar, brow, kb * TK, 0,
                                pol);
          if (++kb == P.kblocks) {
            kb = 0;
            ++seg;
          }
        }
      }
      *issued = (uint64_t)it;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    // The warp waits together and elects the lane that issues, so that descriptors
    // stay uniform; made up for a single lane they took longer than an MMA of N = 128.
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_bf16(TM, TN, AMN, BMN);
      const bool leader = tc::elect_one();
      const uint32_t base0 = tc::smem_u32(smem);
      auto wait_all = [&](auto wait) {
        if (__all_sync(0xffffffffu, wait())) return true;
        if (lane == 0) give_up();
        return false;
      };
      int s = 0;
      uint32_t par = 0;
      int n = 0;  // accumulators filled so far
      bool ok = true;
      uint32_t minors = 0;  // stays of the lower planes' products begun so far
      for (int64_t id = pair; id < tiles && ok; id += npairs) {
        int z, mi, ni, ja, jb;
        tile_at(P, id, z, mi, ni, ja, jb);
        int jm = ja;  // where the current one began
        for (int j0 = ja, j1; j0 < jb && ok; j0 = j1, ++n) {
          j1 = stay_end<F32, LONG>(j0, jb);
          const int buf = n & 1;
          if (F32 && (j0 == ja || minor_end(j0, ja, jb))) {
            jm = j0;
            if (minors > 0 && !wait_all([&] {
                  return tc::mbar_pipe_wait<true>(mempty, (minors & 1u) ^ 1u, abort_flag,
                                                  P.wait_ns);
                })) {
              ok = false;
              break;
            }
            ++minors;
          }
          if (n >= 2 && !wait_all([&] {
                return tc::mbar_pipe_wait<true>(tempty(buf), ((uint32_t)(n / 2) & 1u) ^ 1u,
                                                abort_flag, P.wait_ns);
              })) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          for (int j = j0; j < j1; ++j) {
            if (!wait_all([&] {
                  return tc::mbar_pipe_wait<false>(full(s), par, abort_flag, P.wait_ns);
                })) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t base = base0 + s * STAGE;
            auto mma = [&](uint32_t col, int pa, int pb, int k, bool add) {
              tc::mma2_bf16(tmem + col, rows_desc<G, HALF, AMN>(base, pa, k),
                            rows_desc<G, HN, BMN>(base + G::ABYTES, pb, k), idesc, add ? 1u : 0u);
            };
            if (leader) {
#pragma unroll
              for (int k = 0; k < TK / 16; ++k) {
                if (F32) {
                  mma(G::MINOR, 2, 0, k, j > jm || k > 0);
                  mma(G::MINOR, 1, 1, k, true);
                  mma(G::MINOR, 0, 2, k, true);
                  mma(G::MINOR, 1, 0, k, true);
                  mma(G::MINOR, 0, 1, k, true);
                }
                mma(buf * TN, 0, 0, k, j > j0 || k > 0);
              }
              tc::mma2_commit(empty(s));
            }
            if (++s == NS) {
              s = 0;
              par ^= 1u;
            }
          }
          if (ok && leader) tc::mma2_commit(tfull(buf));
        }
      }
      // every MMA issued here has finished before TMEM is freed
      if (leader) tc::mma2_commit(fin_bar);
      __syncwarp();
      tc::mbar_wait(fin_bar, 0, nullptr, tc::kDrainWaitNs);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue
    // 32 or 64 columns at a time, staged as boxes of this warp's 32 rows and stored
    // by TMA; SETS of boxes in turn.  The loops stay rolled: in a small problem the
    // first pass over the code is a pass through instruction-cache misses.
    constexpr int NB = F32 ? 3 : 1;                // boxes of one operand
    constexpr bool WIDE = E == EPI_STORE && !F32;  // plain bf16: 64 columns at a time
    constexpr bool PLAIN = E == EPI_STORE || E == EPI_PART;
    constexpr int SET = PLAIN           ? 2 * BOX
                        : E == EPI_GATE ? NB * BOX
                        : E == EPI_KEEP ? (F32 ? 2 + NB : 2) * BOX
                                        : 2 * NB * BOX;
    constexpr int SETS = G::OUT / SET > 4 ? 4 : G::OUT / SET;
    static_assert(SETS >= 1, "staged results");
    // KEEP's a has boxes of its own in fp32, in bf16 it follows g and u through theirs
    constexpr int AOFF = E == EPI_KEEP && F32 ? 2 * BOX : 0;
    constexpr int COLS = DUAL ? HN : TN;  // columns of D's tile
    const int q = warp & 3;               // TMEM lane quarter this warp may read
    uint8_t* out = smem + G::OUT_OFF + (warp - 4) * G::OUT;
    // this warp's columns of the tile: all, or half
    constexpr int MINE = COLS * 4 / NEPI;
    const int first = (warp - 4) / 4 * MINE;
    const uint32_t sums = tmem + ((uint32_t)(32 * q) << 16) + G::SUMS;
    // a tile's products may rightly take longer than one wait: 4 us per k block more
    const uint64_t tile_ns = P.wait_ns + (uint64_t)P.nseg * P.kblocks * 4000;
    int n = 0, nset = 0;
    for (int64_t id = pair; id < tiles; id += npairs) {
      int z, mi, ni, ja, jb;
      tile_at(P, id, z, mi, ni, ja, jb);
      const int64_t row0 = (int64_t)mi * TM + rank * HALF + 32 * q, row = row0 + lane;
      bool ok = true;
      // DGATE: g and u are fetched 16 columns ahead, the first ones under the products
      // (without, their latency made the epilogue 43 us a tile, against 28 us of
      // products at k = 4096)
      float gnext[16], unext[16];
      if (E == EPI_DGATE) {
        row16(P.g, row, (int64_t)ni * COLS + first, P.M, P.N, gnext);
        row16(P.u, row, (int64_t)ni * COLS + first, P.M, P.N, unext);
      }
      for (int j0 = ja, j1; j0 < jb; j0 = j1, ++n) {
        j1 = stay_end<F32, LONG>(j0, jb);
        const int buf = n & 1;
        ok = tc::mbar_pipe_wait<false>(tfull(buf), (uint32_t)(n / 2) & 1u, abort_flag, tile_ns);
        if (!ok && !*abort_flag) give_up();
        ok = __all_sync(0xffffffffu, ok);  // the TMEM loads below are warp-collective
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16) + buf * TN;
        if (SUM) {
          // this stay's sums to those before it; at their end the lower planes' too
          const bool minor = F32 && minor_end(j1, ja, jb);
#pragma unroll 1
          for (int c = 0; c < TN; c += 16) {
            float v[16], m[16];
            if (j0 == ja) {
              tc::tmem_get16(ta + c, v);
            } else {
              tc::tmem_get16x2(ta + c, sums + c, v, m);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += m[i];
            }
            if (minor) {
              tc::tmem_get16(sums + c - G::SUMS + G::MINOR, m);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += m[i];
            }
            tc::tmem_put16(sums + c, v);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive_cluster(tc::map_cta(tempty(buf), 0));
            if (minor) tc::mbar_arrive_cluster(tc::map_cta(mempty, 0));
          }
        }
        if (j1 == jb) {
          const uint32_t at = SUM ? sums : ta;  // D's columns
#pragma unroll 1
          for (int c = first; c < first + MINE; c += WIDE ? 64 : 32) {
            const int64_t col = (int64_t)ni * COLS + c;
            const bool in = row0 < P.M && col < P.N;
            uint8_t* box = out + (nset++ % SETS) * SET;
            const uint32_t bu = tc::smem_u32(box);
            const int cc = (int)col, rr = (int)row0;
            float hold[16];
            if (lane == 0) tc::bulk_wait_read<SETS - 1>();
            __syncwarp();
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              const int cg = c + 16 * g;
              float v[16];
              if (WIDE) {
                float w[32];
                tc::tmem_get32(at + c + 32 * g, w);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                  *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * g + p) ^ (lane & 7)) << 4)) =
                      make_uint4(bf2(w[8 * p], w[8 * p + 1]), bf2(w[8 * p + 2], w[8 * p + 3]),
                                 bf2(w[8 * p + 4], w[8 * p + 5]), bf2(w[8 * p + 6], w[8 * p + 7]));
              } else if (PLAIN) {
                tc::tmem_get16(at + cg, v);
                put_f32(box + g * BOX, lane, v);
              } else if (DUAL) {
                float u[16];
                tc::tmem_get16x2(at + cg, at + HN + cg, v, u);
                if (E == EPI_KEEP) {
                  // g and u leave in boxes of 16 columns, a in one of 32
                  if (g == 1) {
                    if (lane == 0) tc::bulk_wait_read<0>();
                    __syncwarp();
                  }
                  put_f32(box, lane, v);
                  put_f32(box + BOX, lane, u);
                  tc::fence_proxy_async_smem();
                  __syncwarp();
                  if (lane == 0) {
                    if (in && col + 16 * g < P.N) {
                      tc::tma_store_3d(&P.d[1], bu, cc + 16 * g, rr, 0);
                      tc::tma_store_3d(&P.d[2], bu + BOX, cc + 16 * g, rr, 0);
                    }
                    tc::bulk_commit();
                  }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = gate<!F32>(P.act, v[i]) * u[i];
                if (E == EPI_GATE) {
                  put_operand<F32>(box, lane, g, v);
                } else if (g == 0) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) hold[i] = v[i];
                } else {
                  if (!F32) {
                    if (lane == 0) tc::bulk_wait_read<0>();
                    __syncwarp();
                  }
                  put_operand<F32>(box + AOFF, lane, 0, hold);
                  put_operand<F32>(box + AOFF, lane, 1, v);
                }
              } else {
                float u[16], gv[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  gv[i] = gnext[i];
                  u[i] = unext[i];
                }
                if (cg + 16 < first + MINE) {
                  row16(P.g, row, col + 16 * g + 16, P.M, P.N, gnext);
                  row16(P.u, row, col + 16 * g + 16, P.M, P.N, unext);
                }
                tc::tmem_get16(at + cg, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float h, dh;
                  gate_both<!F32>(P.act, gv[i], h, dh);
                  u[i] = v[i] * u[i] * dh;
                  v[i] *= h;
                }
                put_operand<F32>(box, lane, g, u);
                put_operand<F32>(box + NB * BOX, lane, g, v);
              }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (in) {
                if (WIDE) {
                  tc::tma_store_3d(&P.d[z], bu, cc, rr, 0);
                } else if (PLAIN) {
                  const CUtensorMap* d = &P.d[E == EPI_PART ? 0 : z];
                  const int plane = E == EPI_PART ? z : 0;
                  tc::tma_store_3d(d, bu, cc, rr, plane);
                  if (col + 16 < P.N) tc::tma_store_3d(d, bu + BOX, cc + 16, rr, plane);
                } else if (E == EPI_DGATE) {
                  for (int pl = 0; pl < 2 * NB; ++pl)
                    tc::tma_store_3d(&P.d[0], bu + pl * BOX, cc, rr, pl);
                } else {
                  for (int pl = 0; pl < NB; ++pl)
                    tc::tma_store_3d(&P.d[0], bu + AOFF + pl * BOX, cc, rr, pl);
                }
              }
              tc::bulk_commit();
            }
          }
        }
        if (!SUM) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(tc::map_cta(tempty(buf), 0));
        }
      }
      if (!ok) break;
    }
    if (lane == 0) tc::bulk_wait<0>();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // no arrival or MMA of the partner is under way any more
  // After an ordinary run the MMAs have waited for every copy.  When either CTA gave
  // up, copies may still be on their way, and the two need not have issued the same
  // ones.  A CTA is at most a ring ahead (a stage is refilled once the MMAs have read
  // both CTAs' copies in it), so each barrier has one open phase at most: the first
  // CTA settles what was never issued and waits for the rest.
  if (*abort_flag) {  // of both CTAs, or of neither
    if (rank == 0 && threadIdx.x == 0) {
      const uint64_t mine = *issued, other = tc::ld_cluster_u64(tc::map_cta(
                                         tc::smem_u32(bars + 2 * NS + 7), 1));
      const uint64_t most = mine > other ? mine : other;
      for (uint64_t i = most > NS ? most - NS : 0; i < most; ++i) {
        const uint32_t bar = full((int)(i % NS));
        if (i >= mine) tc::mbar_arrive_expect_tx(bar, STAGE);  // the partner's copies alone
        if (i >= other) tc::mbar_complete_tx(bar, STAGE);      // ... which do not come
        tc::mbar_wait(bar, (uint32_t)(i / NS) & 1u, nullptr, tc::kDrainWaitNs);
      }
    }
    __syncwarp();
    tc::cluster_sync();
  }
  // the last commit of the first CTA has arrived here too
  if (rank == 1 && threadIdx.x == 0) tc::mbar_wait(fin_bar, 0, nullptr, tc::kDrainWaitNs);
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc2(tmem, 512);
  }
  if (P.beside) tc::grid_wait();
}

// fp32 arrays of n[i] elements (multiples of 8) -> their three bf16 planes each.
struct SplitArgs {
  const float* src[5];
  __nv_bfloat16* dst[5];
  int64_t n[5];
  int count;
};
__global__ void __launch_bounds__(256) k_split3(const __grid_constant__ SplitArgs a) {
  tc::grid_wait();
  tc::grid_release();
  for (int q = 0; q < a.count; ++q) {
    const int64_t n = a.n[q];
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n;
         i += (int64_t)gridDim.x * 256 * 8) {
      uint2 p[3][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        split3x4(__ldcs(reinterpret_cast<const float4*>(a.src[q] + i + 4 * h)), p[0][h], p[1][h],
                 p[2][h]);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl)
        *reinterpret_cast<uint4*>(a.dst[q] + pl * n + i) =
            make_uint4(p[pl][0].x, p[pl][0].y, p[pl][1].x, p[pl][1].y);
    }
  }
}

// The parts of up to four results, added in order: n elements each, `split` planes
// of fp32 sums (split == 0: no such result).
struct JoinArgs {
  const float* part[4];
  void* out[4];
  int64_t n[4];
  int split[4];
};
template <bool F32>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ JoinArgs a) {
  tc::grid_wait();
  tc::grid_release();
  for (int q = 0; q < 4; ++q) {
    if (a.split[q] == 0) continue;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < a.n[q];
         i += (int64_t)gridDim.x * 256 * 4) {
      float4 v = __ldcs(reinterpret_cast<const float4*>(a.part[q] + i));
      for (int k = 1; k < a.split[q]; ++k) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(a.part[q] + k * a.n[q] + i));
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      if (F32)
        *reinterpret_cast<float4*>((float*)a.out[q] + i) = v;
      else
        *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out[q] + i) =
            make_uint2(bf2(v.x, v.y), bf2(v.z, v.w));
    }
  }
}

// A matrix in memory: [planes][rows][cols], bf16 (operands) or fp32 (results).
struct Mat {
  const void* p;
  int64_t rows, cols;
  int planes;
  bool f32;
};

// mn: the operand's own rows run along the stored columns; otherwise boxes of
// `rows` rows.  np planes at a time.
cudaError_t operand_map(CUtensorMap* m, const Mat& x, bool mn, int rows, int np) {
  const uint32_t tk = np == 3 ? 32 : 64;
  const uint64_t d[3] = {(uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.planes};
  const uint64_t s[2] = {(uint64_t)x.cols * 2, (uint64_t)x.cols * x.rows * 2};
  const uint32_t b[3] = {mn ? 64 : tk, mn ? tk : (uint32_t)rows, (uint32_t)np};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x.p, 3, d, s, b,
                   mn || tk == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// Boxes of 32 rows of 64 bytes, or of 64 bf16 for a plain bf16 result (`wide`).
cudaError_t result_map(CUtensorMap* m, const Mat& x, bool wide) {
  const uint64_t e = x.f32 ? 4 : 2;
  wide = wide && !x.f32;
  const uint64_t d[3] = {(uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.planes};
  const uint64_t s[2] = {(uint64_t)x.cols * e, (uint64_t)x.cols * x.rows * e};
  const uint32_t b[3] = {wide ? 64u : (uint32_t)(64 / e), 32, 1};
  return make_tmap(m, x.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   x.p, 3, d, s, b,
                   wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

int sm_pairs() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  return sms / 2;
}

int tiles_of(int64_t n, int t) { return (int)((n + t - 1) / t); }

#define TRY(call)                         \
  do {                                    \
    const cudaError_t e_ = (call);        \
    if (e_ != cudaSuccess) return e_;     \
  } while (0)

// The operands of a launch as stored, with the length of the sums.
struct Opnds {
  Mat a, b[2];
  int64_t K;
};

template <Epi E, bool AMN, bool BMN, bool F32, int TN, bool LONG = false>
cudaError_t launch_tn(GemmArgs& P, const Opnds& o, cudaStream_t s) {
  constexpr bool DUAL = E == EPI_GATE || E == EPI_KEEP;
  using G = ftc::Cfg<TN, F32, more_warps(E, F32 || LONG)>;
  TRY(operand_map(&P.a, o.a, AMN, ftc::HALF, G::NP));
  TRY(operand_map(&P.b[0], o.b[0], BMN, G::BROWS, G::NP));
  if (o.b[1].p) TRY(operand_map(&P.b[1], o.b[1], BMN, G::BROWS, G::NP));
  P.kblocks = tiles_of(o.K, G::TK);
  P.mt = tiles_of(P.M, ftc::TM);
  P.nt = tiles_of(P.N, DUAL ? TN / 2 : TN);
  auto kern = k_ffn_tc<E, AMN, BMN, F32, TN, LONG>;
  TRY(allow_smem(kern, G::SMEM));
  const int64_t tiles = (int64_t)P.mt * P.nt * P.nz * P.split, pairs = sm_pairs();
  return launch_after(kern, (unsigned)(2 * (tiles < pairs ? tiles : pairs)), G::NT, G::SMEM, 2, s,
                      P);
}

// How a product is cut.  fp32: 256 x 128 tiles (four TMEM regions).  bf16: 256 x
// 256, or 256 x 128 where its rounds over the pairs come to less: a narrow tile has
// half the work and takes 0.72 of the time (T = 8192, C = 7168, F = 14336: 5.41
// against 3.63 ms for the forward pass).  A plain result of few tiles and a long k
// is also split along k, into parts of eight k blocks at least, where that saves 24
// blocks of about a quarter of a microsecond: adding up the parts costs four.
// bf16 sums of any number of tiles are split where they are longer than kLongSum:
// they stay in one accumulator, whose adder cuts, and a sum of one sign is off by
// 2^-11.8 of itself at 65536 k, a sixth of its rounding to bf16 (2^-8.2 at 2^19; fp32
// sums leave the accumulator on their way).  The weight gradients' parts take 12 C bytes
// per hidden unit each, where g, u, dg, du and a take 14 T: a fifth at C = 7168.  T =
// 98304, C = F = 2048 backward: 5.64 ms, 5.56 without the split.
struct Plan {
  int tn, split;
};
Plan plan(bool f32, bool dual, bool plain, int64_t M, int64_t N, int nz, int64_t K, int nseg) {
  constexpr int64_t pairs = 74;  // of 148 SMs; the workspace's size follows from it
  const int64_t rows = (int64_t)tiles_of(M, ftc::TM) * nz;
  const int64_t wide = rows * tiles_of(N, dual ? 128 : 256);
  const int64_t half = rows * tiles_of(N, dual ? 64 : 128);
  Plan p{256, 1};
  if (f32 || 72 * ((half + pairs - 1) / pairs) < 100 * ((wide + pairs - 1) / pairs)) p.tn = 128;
  const int64_t tiles = p.tn == 128 ? half : wide, nk = (int64_t)nseg * tiles_of(K, f32 ? 32 : 64);
  if (plain && 2 * tiles <= pairs) {
    const int64_t s = std::min<int64_t>(std::min(pairs / tiles, nk / 8), 16);
    if (s > 1 && nk - nk / s >= 24) p.split = (int)s;
  }
  if (plain && !f32) p.split = (int)std::max<int64_t>(p.split, (nk * 64 + kLongSum - 1) / kLongSum);
  return p;
}
size_t part_bytes(const Plan& p, int64_t M, int64_t N, int nz) {
  return p.split > 1 ? (size_t)nz * p.split * M * N * 4 : 0;
}

template <Epi E, bool AMN, bool BMN, bool F32>
cudaError_t launch(GemmArgs& P, const Opnds& o, int tn, cudaStream_t s) {
  if constexpr (F32) {
    return launch_tn<E, AMN, BMN, true, 128>(P, o, s);
  } else {
    if constexpr (E == EPI_GATE || E == EPI_KEEP || E == EPI_DGATE) {
      if (o.K > kLongSum) return launch_tn<E, AMN, BMN, false, 128, true>(P, o, s);
    }
    return tn == 128 ? launch_tn<E, AMN, BMN, false, 128>(P, o, s)
                     : launch_tn<E, AMN, BMN, false, 256>(P, o, s);
  }
}

bool few_tokens(bool f32, int64_t t, int64_t C, int64_t F) {
  if (f32) return t <= kOneTokens || few32_fits(t, C, F);
  return t <= kFewTokens && std::max(C, 2 * F) <= 8 * kLongSum;  // a cluster's parts
}

// Operands as the products take them: the caller's bf16 arrays, or the split
// copies of its fp32 arrays.
struct Ffn {
  int64_t t, C, F;
  int act, np;  // planes per operand: 1 or 3
  const void *x, *wg, *wu, *wd, *gy;
  int* st;
  int64_t wait_ns;
  // fp32 inputs before their split (k_ffn_one32.cu reads them)
  const void *x32, *gy32;
  bool is_one() const { return np == 3 && t <= kOneTokens; }
  FewArgs one() const { return {t, C, F, act, x32, wg, wu, wd, gy32, st, wait_ns}; }
  bool is_few() const { return few_tokens(np == 3, t, C, F); }
  FewArgs few() const { return {t, C, F, act, x, wg, wu, wd, gy, st, wait_ns}; }
};

// A launch of `pairs` products into an M x N result.
GemmArgs base_args(const Ffn& f, int pairs, int64_t M, int64_t N) {
  GemmArgs P{};
  P.nz = 1;
  P.split = 1;
  P.M = M;
  P.N = N;
  P.act = f.act;
  P.status = f.st;
  P.wait_ns = tc::wait_limit(f.wait_ns);
  P.nseg = pairs;
  return P;
}

// a = act(x wg^T) * (x wu^T) to a (and g, u where they are kept)
template <bool F32> cudaError_t gate_product(const Ffn& f, void* a, float* g, float* u,
                                             cudaStream_t s) {
  GemmArgs P = base_args(f, 1, f.t, f.F);
  const Opnds o{{f.x, f.t, f.C, f.np, false},
                {{f.wg, f.F, f.C, f.np, false}, {f.wu, f.F, f.C, f.np, false}}, f.C};
  TRY(result_map(&P.d[0], {a, f.t, f.F, f.np, false}, false));
  const int tn = plan(F32, true, false, f.t, f.F, 1, f.C, 1).tn;
  if (g == nullptr) return launch<EPI_GATE, false, false, F32>(P, o, tn, s);
  TRY(result_map(&P.d[1], {g, f.t, f.F, 1, true}, false));
  TRY(result_map(&P.d[2], {u, f.t, f.F, 1, true}, false));
  return launch<EPI_KEEP, false, false, F32>(P, o, tn, s);
}

// The nz plain results of a product, into out[], at once or in parts that k_join
// adds up (J's next entries).
template <bool AMN, bool BMN, bool F32>
cudaError_t plain_product(GemmArgs& P, const Opnds& o, void* const* out, float* part, JoinArgs& J,
                          int& joins, cudaStream_t s) {
  const Plan p = plan(F32, false, true, P.M, P.N, P.nz, o.K, P.nseg);
  if (p.split == 1) {
    for (int z = 0; z < P.nz; ++z) TRY(result_map(&P.d[z], {out[z], P.M, P.N, 1, F32}, true));
    return launch<EPI_STORE, AMN, BMN, F32>(P, o, p.tn, s);
  }
  P.split = p.split;
  TRY(result_map(&P.d[0], {part, P.M, P.N, P.nz * p.split, true}, false));
  for (int z = 0; z < P.nz; ++z, ++joins) {
    J.part[joins] = part + (int64_t)z * p.split * P.M * P.N;
    J.out[joins] = out[z];
    J.n[joins] = P.M * P.N;
    J.split[joins] = p.split;
  }
  return launch<EPI_PART, AMN, BMN, F32>(P, o, p.tn, s);
}
template <bool F32> cudaError_t join(const JoinArgs& J, int joins, cudaStream_t s) {
  if (joins == 0) return cudaSuccess;
  int64_t most = 0;
  for (int q = 0; q < joins; ++q) most = std::max(most, J.n[q]);
  return launch_after(k_join<F32>, (unsigned)std::min<int64_t>((most / 4 + 255) / 256, 592), 256, 0,
                      1, s, J);
}

template <bool F32>
cudaError_t fwd(const Ffn& f, void* y, void* a, float* part, cudaStream_t s) {
  if (f.is_few()) {
    if constexpr (F32) {
      if (f.is_one()) {
        TRY(one32_gate(f.one(), (float*)a, nullptr, nullptr, nullptr, s));
        return one32_down(f.one(), (const float*)a, (float*)y, s);
      }
      TRY(few32_gate(f.few(), a, nullptr, nullptr, s));
      return few32_down(f.few(), a, (float*)y, s);
    } else {
      TRY(few_gate(f.few(), a, nullptr, nullptr, s));
      return few_down(f.few(), a, y, s);
    }
  }
  TRY(gate_product<F32>(f, a, nullptr, nullptr, s));
  GemmArgs P = base_args(f, 1, f.t, f.C);
  JoinArgs J{};
  int joins = 0;
  TRY((plain_product<false, false, F32>(
      P, {{a, f.t, f.F, f.np, false}, {{f.wd, f.C, f.F, f.np, false}}, f.F}, &y, part, J, joins,
      s)));
  return join<F32>(J, joins, s);
}

// Where the parts of the backward's plain products go (floats from the start).
struct Parts {
  size_t gx, gw, gwd, bytes;
};
Parts parts_of(bool f32, bool few, int64_t t, int64_t C, int64_t F) {
  Parts p{};
  auto take = [&](size_t bytes) {
    const size_t o = p.bytes / 4;
    p.bytes += (bytes + 255) / 256 * 256;
    return o;
  };
  p.gx = take(few ? 0 : part_bytes(plan(f32, false, true, t, C, 1, F, 2), t, C, 1));
  p.gw = take(part_bytes(plan(f32, false, true, F, C, 2, t, 1), F, C, 2));
  p.gwd = take(part_bytes(plan(f32, false, true, C, F, 1, t, 1), C, F, 1));
  return p;
}

// a [np][t][F], d [2 np][t][F] (dg, du), g and u [t][F].
template <bool F32>
cudaError_t bwd(const Ffn& f, void* gx, void* gwg, void* gwu, void* gwd, void* a, void* d,
                float* d32, float* g, float* u, float* part, cudaStream_t s) {
  const int np = f.np;
  const Mat X{f.x, f.t, f.C, np, false}, GY{f.gy, f.t, f.C, np, false};
  const Mat A{a, f.t, f.F, np, false}, D{d, f.t, f.F, 2 * np, false};
  const Mat WG{f.wg, f.F, f.C, np, false}, WU{f.wu, f.F, f.C, np, false};
  const Mat WD{f.wd, f.C, f.F, np, false};
  const bool few = f.is_few();
  const Parts parts = parts_of(F32, few, f.t, f.C, f.F);
  JoinArgs J{};
  int joins = 0;
  // Five products: g and u with a; gw_down, which needs a; dg and du, which need g
  // and u and run beside it; gx, which needs dg and du; gw_gate and gw_up beside it.
  // Those beside another fill the SMs that it leaves idle.
  if (f.is_one()) {
    TRY(one32_gate(f.one(), nullptr, a, g, u, s));
  } else if (few && F32) {
    TRY(few32_gate(f.few(), a, g, u, s));
  } else if (few) {
    TRY(few_gate(f.few(), a, g, u, s));
  } else {
    TRY(gate_product<F32>(f, a, g, u, s));
  }
  {
    GemmArgs P = base_args(f, 1, f.C, f.F);
    TRY((plain_product<true, true, F32>(P, {GY, {A}, f.t}, &gwd, part + parts.gwd, J, joins, s)));
  }
  if (f.is_one()) {
    TRY(one32_dgate(f.one(), g, u, d32, d, s));
  } else if (few && F32) {
    TRY(few32_dgate(f.few(), g, u, d, s));
  } else if (few) {
    TRY(few_dgate(f.few(), g, u, d, s));
  } else {
    GemmArgs P = base_args(f, 1, f.t, f.F);
    TRY(result_map(&P.d[0], D, false));
    P.g = g;
    P.u = u;
    P.beside = true;
    TRY((launch<EPI_DGATE, false, true, F32>(
        P, {GY, {WD}, f.C}, plan(F32, false, false, f.t, f.F, 1, f.C, 1).tn, s)));
  }
  if (f.is_one()) {
    TRY(one32_grad_x(f.one(), d32, (float*)gx, s));
  } else if (few && F32) {
    TRY(few32_grad_x(f.few(), d, (float*)gx, s));
  } else if (few) {
    TRY(few_grad_x(f.few(), d, gx, s));
  } else {
    GemmArgs P = base_args(f, 2, f.t, f.C);
    TRY((plain_product<false, true, F32>(P, {D, {WG, WU}, f.F}, &gx, part + parts.gx, J, joins,
                                         s)));
  }
  GemmArgs P = base_args(f, 1, f.F, f.C);
  P.nz = 2;
  P.zplanes = np;
  P.beside = true;
  void* const out[2] = {gwg, gwu};
  TRY((plain_product<true, true, F32>(P, {D, {X}, f.t}, out, part + parts.gw, J, joins, s)));
  return join<F32>(J, joins, s);
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Workspaces.  The planes of a (one in bf16, three in fp32); with the backward
// also of dg and du, and g and u in fp32.  fp32: the split copies of the inputs
// (with few tokens the weights are split on their way into the products).  The
// parts of products that are split along k.
struct Layout {
  size_t a, d, d32, g, u, x, wg, wu, wd, gy, part, total;
};
Layout layout(bool f32, bool backward, int64_t t, int64_t C, int64_t F) {
  Layout w{};
  size_t off = 0;
  const size_t np = f32 ? 3 : 1, hid = (size_t)t * F, io = (size_t)t * C, wt = (size_t)F * C;
  const bool few = few_tokens(f32, t, C, F);
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = up(off + bytes);
    return o;
  };
  w.a = take(hid * 2 * np);
  if (backward) {
    w.d = take(hid * 2 * 2 * np);
    w.g = take(hid * 4);
    w.u = take(hid * 4);
    if (f32 && t <= kOneTokens) w.d32 = take(hid * 8);
  }
  if (f32) {
    w.x = take(io * 6);
    if (backward) w.gy = take(io * 6);
    if (!few) {
      w.wg = take(wt * 6);
      w.wu = take(wt * 6);
      w.wd = take(wt * 6);
    }
  }
  w.part = take(backward ? parts_of(f32, few, t, C, F).bytes
                : few    ? 0
                         : part_bytes(plan(f32, false, true, t, C, 1, F, 1), t, C, 1));
  w.total = off;
  return w;
}

// The inputs' split copies (fp32), or the inputs themselves.
cudaError_t operands(Ffn& f, bool f32, const Layout& w, char* ws, cudaStream_t s) {
  f.np = f32 ? 3 : 1;
  if (!f32) return cudaSuccess;
  f.x32 = f.x;
  f.gy32 = f.gy;
  if (f.is_one() && !f.gy) return cudaSuccess;  // the forward takes them as they are
  const int64_t io = f.t * f.C, wt = f.F * f.C;
  SplitArgs a{};
  auto add = [&](const void*& p, size_t off, int64_t n) {
    a.src[a.count] = (const float*)p;
    a.dst[a.count] = (__nv_bfloat16*)(ws + off);
    a.n[a.count++] = n;
    p = ws + off;
  };
  add(f.x, w.x, io);
  if (f.gy) add(f.gy, w.gy, io);
  if (!f.is_few()) {
    add(f.wg, w.wg, wt);
    add(f.wu, w.wu, wt);
    add(f.wd, w.wd, wt);
  }
  const int64_t most = ((f.is_few() ? io : std::max(io, wt)) / 8 + 255) / 256;
  return launch_after(k_split3, (unsigned)std::min<int64_t>(most, 1184), 256, 0, 1, s, a);
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
  Ffn f{t, C, F, act, 1, x, wg, wu, wd, nullptr, st, wait_ns, nullptr, nullptr};
  TRY(operands(f, f32, w, (char*)ws, s));
  char* b = (char*)ws;
  float* part = (float*)(b + w.part);
  return f32 ? fwd<true>(f, y, b + w.a, part, s) : fwd<false>(f, y, b + w.a, part, s);
}

cudaError_t ffn_bwd_dispatch(int dtype, int act, int64_t t, int64_t C, int64_t F, const void* x,
                             const void* wg, const void* wu, const void* wd, const void* gy,
                             void* gx, void* gwg, void* gwu, void* gwd, void* ws, int* st,
                             int64_t wait_ns, cudaStream_t s) {
  const bool f32 = dtype != MHC_DTYPE_BF16;
  const Layout w = layout(f32, true, t, C, F);
  Ffn f{t, C, F, act, 1, x, wg, wu, wd, gy, st, wait_ns, nullptr, nullptr};
  char* b = (char*)ws;
  TRY(operands(f, f32, w, b, s));
  float *g = (float*)(b + w.g), *u = (float*)(b + w.u), *d32 = (float*)(b + w.d32);
  float* part = (float*)(b + w.part);
  return f32 ? bwd<true>(f, gx, gwg, gwu, gwd, b + w.a, b + w.d, d32, g, u, part, s)
             : bwd<false>(f, gx, gwg, gwu, gwd, b + w.a, b + w.d, nullptr, g, u, part, s);
}

#undef TRY

}  // namespace mhc
