// k_ffn_one32.cu -- the feed-forward products of up to 8 tokens, fp32, on the CUDA
// cores: plain fp32 multiply-adds, bound by reading the weights once.  Eight tokens
// take eight multiply-adds per weight, 16 weights a cycle and SM, against 5.8 that
// memory delivers (6.55 TB/s over 148 SMs).  Forward, C = 7168, F = 14336: 217 us
// with one token (5.7 TB/s), 241 with 4, 341 with 8; a variant for 16, whose sums
// leave one CTA per SM, took 809 us, the tensor cores (k_ffn_few32.cu) 407.
//
// k_rows: weights stored along k (forward).  A warp takes four rows, its lanes
// along k, and a row's tokens are reduced over the lanes at the end.
// k_cols: weights stored along their rows (the backward's da and gx).  Lanes run
// along the rows, four each, warps along k.
// Either way the tokens' chunk of k comes through shared memory, the k axis is split
// over the CTAs of a cluster where there are few row tiles, and the parts are added
// in a fixed order through distributed shared memory.
#include "ffn_few.h"

#include "ffn_common.cuh"
#include "tc_pair.cuh"

namespace mhc {

namespace {

constexpr int NTHR = 256, NWARP = 8;

enum OneEpi { ONE_STORE, ONE_GATE, ONE_DGATE };

struct OneP {
  const float *w[2], *x;       // weights; tokens [segments][t][K]
  int64_t K, rows, t;          // length of a product's sum; rows of D^T; tokens
  int nseg;                    // COLS: products added up (w[s] with plane s of x)
  int parts;
  float* o;                    // STORE: [t][rows]; GATE: a, null to leave out; DGATE: dg, du
  __nv_bfloat16* planes;       // GATE, DGATE: the planes of a, or of dg and du; may be null
  float *g, *u;                // GATE: kept unless null; DGATE: read
  int act;
  bool early;                  // a later kernel of its call: weights may be read at once
  bool beside;                 // COLS: needs nothing from the kernel before it
};

__device__ __forceinline__ float4 ld_once(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void put_planes(__nv_bfloat16* p, int64_t stride, float v) {
  uint2 h, m, l;
  split3x4(make_float4(v, 0.f, 0.f, 0.f), h, m, l);
  p[0] = __ushort_as_bfloat16((unsigned short)(h.x & 0xffffu));
  p[stride] = __ushort_as_bfloat16((unsigned short)(m.x & 0xffffu));
  p[2 * stride] = __ushort_as_bfloat16((unsigned short)(l.x & 0xffffu));
}

// One element of D^T, summed: v, and for GATE the other weight's sum.
template <OneEpi E>
__device__ __forceinline__ void finish(const OneP& P, int64_t tok, int64_t row, float v, float v2) {
  const int64_t o = tok * P.rows + row, plane = P.t * P.rows;
  if (E == ONE_STORE) {
    P.o[o] = v;
  } else if (E == ONE_GATE) {
    const float a = gate<false>(P.act, v) * v2;
    if (P.o) P.o[o] = a;
    if (P.planes) put_planes(P.planes + o, plane, a);
    if (P.g) {
      P.g[o] = v;
      P.u[o] = v2;
    }
  } else {
    float h, dh;
    gate_both<false>(P.act, P.g[o], h, dh);
    const float dg = v * P.u[o] * dh, du = v * h;
    P.o[o] = dg;
    P.o[plane + o] = du;
    put_planes(P.planes + o, plane, dg);
    put_planes(P.planes + 3 * plane + o, plane, du);
  }
}

__device__ __forceinline__ float ld_part(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];"
               : "=f"(v)
               : "r"(tc::map_cta(tc::smem_u32(p), rank))
               : "memory");
  return v;
}

// ------------------------------------------------------------ weights along k
constexpr int RPW = 4;             // rows per warp
constexpr int RCHUNK = 256;        // k per chunk: two float4 per lane

template <OneEpi E, int TT>
__global__ void __launch_bounds__(NTHR) k_rows(const __grid_constant__ OneP P) {
  constexpr int TILE = E == ONE_GATE ? NWARP * RPW / 2 : NWARP * RPW;  // rows of D^T per CTA
  __shared__ __align__(16) float xs[2][TT][RCHUNK];
  __shared__ float part[NWARP * RPW][TT];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)tc::cluster_rank();
  const int64_t row0 = (int64_t)(blockIdx.x / P.parts) * TILE;
  const int64_t chunks = (P.K + RCHUNK - 1) / RCHUNK;
  const int64_t c0 = chunks * rank / P.parts, c1 = chunks * (rank + 1) / P.parts;
  // this warp's rows; past the end the last one again (not stored)
  const float* wr[RPW];
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int64_t r = row0 + (E == ONE_GATE ? 2 * warp + i / 2 : RPW * warp + i);
    wr[i] = P.w[E == ONE_GATE ? i & 1 : 0] + (r < P.rows ? r : P.rows - 1) * P.K;
  }
  auto stage = [&](int64_t c, int b) {
    // tokens past the last, and k past the end, are zero
    for (int e = threadIdx.x; e < TT * RCHUNK / 4; e += NTHR) {
      const int tok = e / (RCHUNK / 4), q = e % (RCHUNK / 4);
      const int64_t k = c * RCHUNK + 4 * q;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tok < P.t && k < P.K)
        v = *reinterpret_cast<const float4*>(P.x + tok * P.K + k);
      *reinterpret_cast<float4*>(&xs[b][tok][4 * q]) = v;
    }
  };
  auto fetch = [&](int64_t c, float4 (&v)[2][RPW]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = c * RCHUNK + 128 * h + 4 * lane;
#pragma unroll
      for (int i = 0; i < RPW; ++i)
        v[h][i] = k < P.K ? ld_once(wr[i] + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  float acc[RPW][TT] = {};
  float4 next[2][RPW];
  if (P.early && c0 < c1) fetch(c0, next);
  tc::grid_wait();
  tc::grid_release();
  if (c0 < c1) {
    if (!P.early) fetch(c0, next);
    stage(c0, 0);
  }
  __syncthreads();
  for (int64_t c = c0; c < c1; ++c) {
    const int b = (int)(c - c0) & 1;
    float4 v[2][RPW];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RPW; ++i) v[h][i] = next[h][i];
    if (c + 1 < c1) {
      fetch(c + 1, next);
      stage(c + 1, b ^ 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int tok = 0; tok < TT; ++tok) {
        const float4 q = *reinterpret_cast<const float4*>(&xs[b][tok][128 * h + 4 * lane]);
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
          acc[i][tok] = fmaf(v[h][i].x, q.x, acc[i][tok]);
          acc[i][tok] = fmaf(v[h][i].y, q.y, acc[i][tok]);
          acc[i][tok] = fmaf(v[h][i].z, q.z, acc[i][tok]);
          acc[i][tok] = fmaf(v[h][i].w, q.w, acc[i][tok]);
        }
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < RPW; ++i)
#pragma unroll
    for (int tok = 0; tok < TT; ++tok) {
      float s = acc[i][tok];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) part[RPW * warp + i][tok] = s;
    }
  __syncwarp();
  if (P.parts > 1) tc::cluster_sync();
  else __syncthreads();
  for (int e = threadIdx.x; e < TILE * TT; e += NTHR) {
    const int tok = e / TILE, r = e % TILE;
    if (tok % P.parts != rank || tok >= P.t || row0 + r >= P.rows) continue;
    float v = 0.f, v2 = 0.f;
    for (int q = 0; q < P.parts; ++q) {
      if (E == ONE_GATE) {
        v += ld_part(&part[2 * r][tok], q);
        v2 += ld_part(&part[2 * r + 1][tok], q);
      } else {
        v += ld_part(&part[r][tok], q);
      }
    }
    finish<E>(P, tok, row0 + r, v, v2);
  }
  __syncwarp();
  // nobody reads this CTA's part any more
  if (P.parts > 1) tc::cluster_sync();
}

// ------------------------------------------------------- weights along their rows
constexpr int CTILE = 128;         // rows of D^T per CTA: four per lane
constexpr int CCHUNK = 64;         // k per chunk: eight per warp

template <OneEpi E, int TT>
__global__ void __launch_bounds__(NTHR) k_cols(const __grid_constant__ OneP P) {
  extern __shared__ float4 cols_smem[];
  float* xs = reinterpret_cast<float*>(cols_smem);                 // [2][CCHUNK][TT]
  float* wsum = xs + 2 * CCHUNK * TT;                              // [NWARP][TT][CTILE]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)tc::cluster_rank();
  const int64_t row0 = (int64_t)(blockIdx.x / P.parts) * CTILE, row = row0 + 4 * lane;
  const int64_t per = (P.K + CCHUNK - 1) / CCHUNK, chunks = per * P.nseg;
  const int64_t c0 = chunks * rank / P.parts, c1 = chunks * (rank + 1) / P.parts;
  auto stage = [&](int64_t c, int b) {
    const int64_t seg = c / per, kb = (c - seg * per) * CCHUNK;
    const float* x = P.x + seg * P.t * P.K;
    for (int e = threadIdx.x; e < TT * CCHUNK; e += NTHR) {
      const int tok = e / CCHUNK, k = e % CCHUNK;
      xs[(b * CCHUNK + k) * TT + tok] =
          tok < P.t && kb + k < P.K ? x[tok * P.K + kb + k] : 0.f;
    }
  };
  auto fetch = [&](int64_t c, float4 (&v)[8]) {
    const int64_t seg = c / per, kb = (c - seg * per) * CCHUNK;
    const float* w = P.w[seg];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t k = kb + 8 * warp + j;
      v[j] = k < P.K && row < P.rows ? ld_once(w + k * P.rows + row)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  float acc[TT][4] = {};
  float4 next[8];
  if (P.early && c0 < c1) fetch(c0, next);
  if (!P.beside) tc::grid_wait();
  tc::grid_release();
  if (c0 < c1) {
    if (!P.early) fetch(c0, next);
    stage(c0, 0);
  }
  __syncthreads();
  for (int64_t c = c0; c < c1; ++c) {
    const int b = (int)(c - c0) & 1;
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = next[j];
    if (c + 1 < c1) {
      fetch(c + 1, next);
      stage(c + 1, b ^ 1);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* q = xs + (b * CCHUNK + 8 * warp + j) * TT;
#pragma unroll
      for (int tok = 0; tok < TT; ++tok) {
        const float s = q[tok];
        acc[tok][0] = fmaf(v[j].x, s, acc[tok][0]);
        acc[tok][1] = fmaf(v[j].y, s, acc[tok][1]);
        acc[tok][2] = fmaf(v[j].z, s, acc[tok][2]);
        acc[tok][3] = fmaf(v[j].w, s, acc[tok][3]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int tok = 0; tok < TT; ++tok)
    *reinterpret_cast<float4*>(wsum + (warp * TT + tok) * CTILE + 4 * lane) =
        make_float4(acc[tok][0], acc[tok][1], acc[tok][2], acc[tok][3]);
  __syncthreads();
  // the warps' sums in warp order, into the first warp's place
  for (int e = threadIdx.x; e < TT * CTILE; e += NTHR) {
    float s = wsum[e];
#pragma unroll
    for (int q = 1; q < NWARP; ++q) s += wsum[q * TT * CTILE + e];
    wsum[e] = s;
  }
  __syncwarp();
  if (P.parts > 1) tc::cluster_sync();
  else __syncthreads();
  for (int e = threadIdx.x; e < TT * CTILE; e += NTHR) {
    const int tok = e / CTILE, r = e % CTILE;
    if (tok % P.parts != rank || tok >= P.t || row0 + r >= P.rows) continue;
    float v = 0.f;
    for (int q = 0; q < P.parts; ++q) v += ld_part(wsum + e, q);
    finish<E>(P, tok, row0 + r, v, 0.f);
  }
  __syncwarp();
  // nobody reads this CTA's part any more
  if (P.parts > 1) tc::cluster_sync();
  if (P.beside) tc::grid_wait();
}

// The split of k: a chunk of either kernel is 32 KB of weights.
int parts_of(int64_t tiles, int64_t chunks) { return split_sum(tiles, chunks, 2, 1, 2, 500, 3000); }

template <OneEpi E, int TT> cudaError_t rows_tt(OneP& P, cudaStream_t s) {
  const int64_t tile = E == ONE_GATE ? NWARP * RPW / 2 : NWARP * RPW;
  const int64_t tiles = (P.rows + tile - 1) / tile;
  P.parts = parts_of(tiles, (P.K + RCHUNK - 1) / RCHUNK);
  return launch_after(k_rows<E, TT>, (unsigned)(tiles * P.parts), NTHR, 0, (unsigned)P.parts, s, P);
}
template <OneEpi E, int TT> cudaError_t cols_tt(OneP& P, cudaStream_t s) {
  const int64_t tiles = (P.rows + CTILE - 1) / CTILE;
  P.parts = parts_of(tiles, (P.K + CCHUNK - 1) / CCHUNK * P.nseg);
  constexpr size_t sm = (size_t)(2 * CCHUNK * TT + NWARP * TT * CTILE) * 4;
  auto kern = k_cols<E, TT>;
  const cudaError_t e = allow_smem(kern, sm);
  if (e != cudaSuccess) return e;
  return launch_after(kern, (unsigned)(tiles * P.parts), NTHR, sm, (unsigned)P.parts, s, P);
}
template <OneEpi E> cudaError_t rows(OneP& P, cudaStream_t s) {
  return P.t <= 1   ? rows_tt<E, 1>(P, s)
         : P.t <= 4 ? rows_tt<E, 4>(P, s)
                    : rows_tt<E, 8>(P, s);
}
template <OneEpi E> cudaError_t cols(OneP& P, cudaStream_t s) {
  return P.t <= 1   ? cols_tt<E, 1>(P, s)
         : P.t <= 4 ? cols_tt<E, 4>(P, s)
                    : cols_tt<E, 8>(P, s);
}

}  // namespace

cudaError_t one32_gate(const FewArgs& f, float* a, void* planes, float* g, float* u,
                       cudaStream_t s) {
  OneP P{{(const float*)f.wg, (const float*)f.wu}, (const float*)f.x, f.C, f.F, f.t, 1, 1, a,
         (__nv_bfloat16*)planes, g, u, f.act, false, false};
  return rows<ONE_GATE>(P, s);
}

cudaError_t one32_down(const FewArgs& f, const float* a, float* y, cudaStream_t s) {
  OneP P{{(const float*)f.wd, nullptr}, a, f.F, f.C, f.t, 1, 1, y, nullptr, nullptr, nullptr, 0,
         true, false};
  return rows<ONE_STORE>(P, s);
}

cudaError_t one32_dgate(const FewArgs& f, const float* g, const float* u, float* d, void* planes,
                        cudaStream_t s) {
  OneP P{{(const float*)f.wd, nullptr}, (const float*)f.gy, f.C, f.F, f.t, 1, 1, d,
         (__nv_bfloat16*)planes, const_cast<float*>(g), const_cast<float*>(u), f.act,
         true, true};
  return cols<ONE_DGATE>(P, s);
}

cudaError_t one32_grad_x(const FewArgs& f, const float* d, float* gx, cudaStream_t s) {
  OneP P{{(const float*)f.wg, (const float*)f.wu}, d, f.F, f.C, f.t, 2, 1, gx, nullptr, nullptr,
         nullptr, 0, true, false};
  return cols<ONE_STORE>(P, s);
}

}  // namespace mhc
