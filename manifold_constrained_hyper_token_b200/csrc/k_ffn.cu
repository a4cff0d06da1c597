// k_ffn.cu -- the matrix products of the gated feed-forward block on the CUDA
// cores, with the activation and its derivative in their epilogues.
//
//   forward : a = act(x w_gate^T) * (x w_up^T);  y = a w_down^T
//   backward: g, u recomputed;  da = gy w_down, du = da act(g),
//             dg = da u act'(g);  gx = dg w_gate + du w_up;
//             gw_gate = dg^T x, gw_up = du^T x, gw_down = gy^T a
//
// One kernel: D[m][n] = sum_k A(m, k) B(n, k) with any strides, 64 x 64 tiles,
// 4 x 4 outputs per thread, fp32 sums in k order.
#include "mhc_common.cuh"
#include "mhc_dispatch.h"

namespace mhc {

namespace {

constexpr int TILE = 64, TK = 16;

enum Epi { E_STORE, E_GATE, E_GATE_KEEP, E_DGATE };

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// An operand: element (i, k) at p[i * si + k * sk].
template <typename T> struct Opnd {
  const T* p;
  int64_t si, sk;
};

__device__ __forceinline__ void act_both(int act, float g, float& h, float& dh) {
  if (act == MHC_ACT_SILU) {
    const float p = sigmoidf_(g);
    h = g * p;
    dh = p * (1.0f + g * (1.0f - p));
  } else {
    const float c = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
    h = g * c;
    dh = c + g * 0.39894228040143268f * expf(-0.5f * g * g);
  }
}

// E_STORE: D = A0 B0 (+ A1 B1 when pairs = 2) to o0.
// E_GATE / E_GATE_KEEP: g = A0 B0, u = A0 B1; act(g) u to o0 (and g, u to o1, o2).
// E_DGATE: da = A0 B0; reads g, u at o1, o2, writes act(g) u to o0 and dg, du
// over g and u.
template <typename T, Epi E>
__global__ void __launch_bounds__(256) k_ffn_simt(int64_t M, int64_t N, int64_t K, int pairs,
                                                  int act, Opnd<T> A0, Opnd<T> A1, Opnd<T> B0,
                                                  Opnd<T> B1, T* o0, T* o1, T* o2) {
  constexpr bool DUAL = E == E_GATE || E == E_GATE_KEEP;
  __shared__ float sa[TK][TILE + 1], sb[TK][TILE + 1], sc[DUAL ? TK : 1][TILE + 1];
  const int64_t m0 = (int64_t)blockIdx.y * TILE, n0 = (int64_t)blockIdx.x * TILE;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {}, acc2[4][4] = {};
  for (int pr = 0; pr < pairs; ++pr) {
    const Opnd<T> A = pr ? A1 : A0, B = pr ? B1 : B0;
    for (int64_t k0 = 0; k0 < K; k0 += TK) {
      for (int e = threadIdx.x; e < TILE * TK; e += 256) {
        // walk the operand's unit stride with neighbouring threads
        const int ka = A.sk == 1 ? e % TK : e / TILE, ia = A.sk == 1 ? e / TK : e % TILE;
        sa[ka][ia] = (m0 + ia < M && k0 + ka < K)
                         ? to_f32(A.p[(m0 + ia) * A.si + (k0 + ka) * A.sk]) : 0.f;
        const int kb = B.sk == 1 ? e % TK : e / TILE, ib = B.sk == 1 ? e / TK : e % TILE;
        const bool in = n0 + ib < N && k0 + kb < K;
        sb[kb][ib] = in ? to_f32(B.p[(n0 + ib) * B.si + (k0 + kb) * B.sk]) : 0.f;
        if (DUAL) sc[kb][ib] = in ? to_f32(B1.p[(n0 + ib) * B1.si + (k0 + kb) * B1.sk]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < TK; ++k) {
        float av[4], bv[4], cv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          av[i] = sa[k][ty + 16 * i];
          bv[i] = sb[k][tx + 16 * i];
          if (DUAL) cv[i] = sc[k][tx + 16 * i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            if (DUAL) acc2[i][j] = fmaf(av[i], cv[j], acc2[i][j]);
          }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= M || n >= N) continue;
      const int64_t o = m * N + n;
      float h, dh;
      if (E == E_STORE) {
        o0[o] = from_f32<T>(acc[i][j]);
      } else if (DUAL) {
        act_both(act, acc[i][j], h, dh);
        o0[o] = from_f32<T>(h * acc2[i][j]);
        if (E == E_GATE_KEEP) {
          o1[o] = from_f32<T>(acc[i][j]);
          o2[o] = from_f32<T>(acc2[i][j]);
        }
      } else {
        const float g = to_f32(o1[o]), u = to_f32(o2[o]), da = acc[i][j];
        act_both(act, g, h, dh);
        o1[o] = from_f32<T>(da * u * dh);
        o2[o] = from_f32<T>(da * h);
      }
    }
}

template <typename T, Epi E>
cudaError_t launch(int64_t M, int64_t N, int64_t K, int pairs, int act, Opnd<T> A0, Opnd<T> A1,
                   Opnd<T> B0, Opnd<T> B1, T* o0, T* o1, T* o2, cudaStream_t s) {
  // rows in slabs: gridDim.y is limited to 65535
  constexpr int64_t SLAB = (int64_t)65535 * TILE;
  for (int64_t m = 0; m < M; m += SLAB) {
    const int64_t mm = M - m < SLAB ? M - m : SLAB;
    const dim3 grid((unsigned)((N + TILE - 1) / TILE), (unsigned)((mm + TILE - 1) / TILE));
    Opnd<T> a0 = A0, a1 = A1;
    a0.p += m * A0.si;
    if (pairs == 2) a1.p += m * A1.si;
    k_ffn_simt<T, E><<<grid, 256, 0, s>>>(mm, N, K, pairs, act, a0, a1, B0, B1, o0 + m * N,
                                          o1 ? o1 + m * N : nullptr, o2 ? o2 + m * N : nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t fwd(int64_t t, int64_t C, int64_t F, int act, const T* x, const T* wg, const T* wu,
                const T* wd, T* y, T* a, cudaStream_t s) {
  const Opnd<T> X{x, C, 1}, G{wg, C, 1}, U{wu, C, 1}, A{a, F, 1}, D{wd, F, 1}, Z{nullptr, 0, 0};
  cudaError_t e = launch<T, E_GATE>(t, F, C, 1, act, X, Z, G, U, a, nullptr, nullptr, s);
  if (e != cudaSuccess) return e;
  return launch<T, E_STORE>(t, C, F, 1, act, A, Z, D, Z, y, nullptr, nullptr, s);
}

template <typename T>
cudaError_t bwd(int64_t t, int64_t C, int64_t F, int act, const T* x, const T* wg, const T* wu,
                const T* wd, const T* gy, T* gx, T* gwg, T* gwu, T* gwd, T* ws, cudaStream_t s) {
  T *a = ws, *dg = ws + t * F, *du = ws + 2 * t * F;
  const Opnd<T> Z{nullptr, 0, 0};
  const Opnd<T> X{x, C, 1}, G{wg, C, 1}, U{wu, C, 1}, GY{gy, C, 1}, DT{wd, 1, F};
  cudaError_t e = launch<T, E_GATE_KEEP>(t, F, C, 1, act, X, Z, G, U, a, dg, du, s);
  if (e == cudaSuccess) e = launch<T, E_DGATE>(t, F, C, 1, act, GY, Z, DT, Z, a, dg, du, s);
  const Opnd<T> XT{x, 1, C}, AT{a, 1, F}, DGT{dg, 1, F}, DUT{du, 1, F}, GYT{gy, 1, C};
  const Opnd<T> DG{dg, F, 1}, DU{du, F, 1}, GT{wg, 1, C}, UT{wu, 1, C};
  if (e == cudaSuccess) e = launch<T, E_STORE>(C, F, t, 1, act, GYT, Z, AT, Z, gwd, nullptr, nullptr, s);
  if (e == cudaSuccess) e = launch<T, E_STORE>(F, C, t, 1, act, DGT, Z, XT, Z, gwg, nullptr, nullptr, s);
  if (e == cudaSuccess) e = launch<T, E_STORE>(F, C, t, 1, act, DUT, Z, XT, Z, gwu, nullptr, nullptr, s);
  if (e == cudaSuccess) e = launch<T, E_STORE>(t, C, F, 2, act, DG, DU, GT, UT, gx, nullptr, nullptr, s);
  return e;
}

}  // namespace

size_t ffn_fwd_workspace_bytes(int dtype, int64_t t, int64_t C, int64_t F) {
  return (size_t)t * F * (dtype == MHC_DTYPE_BF16 ? 2 : 4);
}

size_t ffn_bwd_workspace_bytes(int dtype, int64_t t, int64_t C, int64_t F) {
  return (size_t)3 * t * F * (dtype == MHC_DTYPE_BF16 ? 2 : 4);
}

cudaError_t ffn_fwd_dispatch(int dtype, int act, int64_t t, int64_t C, int64_t F, const void* x,
                             const void* wg, const void* wu, const void* wd, void* y, void* ws,
                             int* st, int64_t wait_ns, cudaStream_t s) {
  (void)st;
  (void)wait_ns;
  using H = __nv_bfloat16;
  if (dtype == MHC_DTYPE_BF16)
    return fwd(t, C, F, act, (const H*)x, (const H*)wg, (const H*)wu, (const H*)wd, (H*)y, (H*)ws,
               s);
  return fwd(t, C, F, act, (const float*)x, (const float*)wg, (const float*)wu, (const float*)wd,
             (float*)y, (float*)ws, s);
}

cudaError_t ffn_bwd_dispatch(int dtype, int act, int64_t t, int64_t C, int64_t F, const void* x,
                             const void* wg, const void* wu, const void* wd, const void* gy,
                             void* gx, void* gwg, void* gwu, void* gwd, void* ws, int* st,
                             int64_t wait_ns, cudaStream_t s) {
  (void)st;
  (void)wait_ns;
  using H = __nv_bfloat16;
  if (dtype == MHC_DTYPE_BF16)
    return bwd(t, C, F, act, (const H*)x, (const H*)wg, (const H*)wu, (const H*)wd, (const H*)gy,
               (H*)gx, (H*)gwg, (H*)gwu, (H*)gwd, (H*)ws, s);
  return bwd(t, C, F, act, (const float*)x, (const float*)wg, (const float*)wu, (const float*)wd,
             (const float*)gy, (float*)gx, (float*)gwg, (float*)gwu, (float*)gwd, (float*)ws, s);
}

}  // namespace mhc
