// k_norm.cu -- layer norm over the channels of a token, forward and backward.
//
//   mean = 1/C sum x,  s = 1/sqrt(1/C sum (x - mean)^2 + eps),  xh = (x - mean) s
//   forward : y = xh w + b
//   backward: a = gy w,  gx = s (a - mean(a) - xh mean(a xh)),
//             gw = sum_t gy xh,  gb = sum_t gy
//
// HBM bound: one read of every input and one write of every output.  A token's
// row stays in registers between its statistics and its outputs.  Each warp
// takes its own share of a row in two passes (its sum, then the squares about
// its own mean), and the shares are joined as M2 = sum_w (M2_w + n_w (m_w -
// mean)^2): no difference of large sums, and one block barrier per row.
#include "mhc_common.cuh"
#include "mhc_dispatch.h"

namespace mhc {

namespace {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What one warp knows of its share of a row: how many channels, their mean, the
// squares about that mean and, in the backward, the sums of a and of a (x - m).
struct Share {
  float n, m, m2, a, ax;
};

// The row's statistics from its warps' shares (all lanes of all warps get them).
// Record w is read by lane w, so at most 32 warps.
template <bool BWD>
__device__ __forceinline__ Share join_shares(const Share& mine, Share* rec, int nwarps, int64_t C) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) rec[warp] = mine;
  __syncthreads();
  Share q = lane < nwarps ? rec[lane] : Share{0.f, 0.f, 0.f, 0.f, 0.f};
  Share r;
  r.n = (float)C;
  r.m = warp_sum(q.n * q.m) / (float)C;
  const float d = q.m - r.m;
  r.m2 = warp_sum(q.m2 + q.n * d * d);
  r.a = r.ax = 0.f;
  if (BWD) {
    r.a = warp_sum(q.a);
    r.ax = warp_sum(q.ax + d * q.a);
  }
  return r;
}

__device__ __forceinline__ void report(float mean, float s, int* status) {
  if (!isfinite(mean) || !isfinite(s)) flag_status(status, MHC_ERR_NONFINITE);
}

// ------------------------------------------------------------------ forward
// WARP: one row per warp (blockDim.x / 32 rows per CTA); otherwise one row per
// CTA.  A thread holds VPT 16-byte vectors of its row.
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(kMaxThreads) k_norm_fwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
                           const float* __restrict__ w, const float* __restrict__ b,
                           T* __restrict__ y, int* status) {
  constexpr int N = Vec<T>::N;
  __shared__ Share rec[32];
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32
                           : (int64_t)blockIdx.x;
  if (WARP && row >= rows) return;
  const int nvec = (int)(C / N);
  const T* xr = x + row * C;
  float v[VPT][N];
  float sum = 0.f;
  int cnt = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int k = t + i * tpr;
    if (k < nvec) {
      Vec<T>::load_stream(xr + (int64_t)k * N, v[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) sum += v[i][e];
      cnt += N;
    }
  }
  Share sh;
  sh.n = warp_sum((float)cnt);
  sh.m = sh.n > 0.f ? warp_sum(sum) / sh.n : 0.f;
  float m2 = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * tpr < nvec) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = v[i][e] - sh.m;
        m2 = fmaf(d, d, m2);
      }
    }
  sh.m2 = warp_sum(m2);
  if (!WARP) sh = join_shares<false>(sh, rec, blockDim.x / 32, C);
  const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
  if (t == 0) report(sh.m, s, status);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int k = t + i * tpr;
    if (k < nvec) {
      float o[N];
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 wv = __ldg(reinterpret_cast<const float4*>(w + (int64_t)k * N + e));
        const float4 bv = b ? __ldg(reinterpret_cast<const float4*>(b + (int64_t)k * N + e))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        o[e] = fmaf((v[i][e] - sh.m) * s, wv.x, bv.x);
        o[e + 1] = fmaf((v[i][e + 1] - sh.m) * s, wv.y, bv.y);
        o[e + 2] = fmaf((v[i][e + 2] - sh.m) * s, wv.z, bv.z);
        o[e + 3] = fmaf((v[i][e + 3] - sh.m) * s, wv.w, bv.w);
      }
      Vec<T>::store_stream(y + row * C + (int64_t)k * N, o);
    }
  }
}

// Rows too long for registers: one CTA per row, three walks over the row.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) k_norm_fwd_long(
    int64_t C, float eps, const T* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ b, T* __restrict__ y, int* status) {
  constexpr int N = Vec<T>::N;
  __shared__ Share rec[32];
  const int64_t row = blockIdx.x, nvec = C / N;
  const T* xr = x + row * C;
  float sum = 0.f, v[N];
  int64_t cnt = 0;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(xr + k * N, v);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) q += v[e];
    sum += q;
    cnt += N;
  }
  Share sh;
  sh.n = warp_sum((float)cnt);
  sh.m = sh.n > 0.f ? warp_sum(sum) / sh.n : 0.f;
  float m2 = 0.f;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(xr + k * N, v);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) q = fmaf(v[e] - sh.m, v[e] - sh.m, q);
    m2 += q;
  }
  sh.m2 = warp_sum(m2);
  sh = join_shares<false>(sh, rec, blockDim.x / 32, C);
  const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
  if (threadIdx.x == 0) report(sh.m, s, status);
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(xr + k * N, v);
    float o[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
      o[e] = fmaf((v[e] - sh.m) * s, __ldg(w + k * N + e), b ? __ldg(b + k * N + e) : 0.f);
    Vec<T>::store_stream(y + row * C + k * N, o);
  }
}

// ----------------------------------------------------------------- backward
// Persistent CTAs: each takes rows in a fixed stride and keeps its threads'
// channels of grad_weight and grad_bias in registers; one partial row pair
// [2][C] per CTA, summed in CTA order by k_norm_fin.  WARP: one row per warp at
// a time, the warps' sums joined in warp order through shared memory.
template <typename T, int VPT, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_bwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
                           const float* __restrict__ w, const T* __restrict__ gy,
                           T* __restrict__ gx, float* __restrict__ part, int* status) {
  constexpr int N = Vec<T>::N;
  __shared__ Share rec[2][32];
  extern __shared__ float wsum[];  // WARP: [2][C]
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int per = WARP ? blockDim.x / 32 : 1, g = WARP ? threadIdx.x / 32 : 0;
  const int nvec = (int)(C / N);
  float gw[VPT][N], gb[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) gw[i][e] = gb[i][e] = 0.f;
  int it = 0;
  for (int64_t row = (int64_t)blockIdx.x * per + g; row < rows;
       row += (int64_t)gridDim.x * per, ++it) {
    float xv[VPT][N], gv[VPT][N];
    float sum = 0.f, sa = 0.f;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        Vec<T>::load_stream(x + row * C + (int64_t)k * N, xv[i]);
        Vec<T>::load_stream(gy + row * C + (int64_t)k * N, gv[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) sum += xv[i][e];
        cnt += N;
      }
    }
    Share sh;
    sh.n = warp_sum((float)cnt);
    sh.m = sh.n > 0.f ? warp_sum(sum) / sh.n : 0.f;
    float m2 = 0.f, sax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d = xv[i][e] - sh.m, a = gv[i][e] * __ldg(w + (int64_t)k * N + e);
          m2 = fmaf(d, d, m2);
          sa += a;
          sax = fmaf(a, d, sax);
        }
      }
    }
    sh.m2 = warp_sum(m2);
    sh.a = warp_sum(sa);
    sh.ax = warp_sum(sax);
    if (!WARP) sh = join_shares<true>(sh, rec[it & 1], blockDim.x / 32, C);
    const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
    if (t == 0) report(sh.m, s, status);
    const float c1 = sh.a / (float)C, c2 = sh.ax * s / (float)C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float xh = (xv[i][e] - sh.m) * s, a = gv[i][e] * __ldg(w + (int64_t)k * N + e);
          o[e] = s * (a - c1 - xh * c2);
          gw[i][e] = fmaf(gv[i][e], xh, gw[i][e]);
          gb[i][e] += gv[i][e];
        }
        Vec<T>::store_stream(gx + row * C + (int64_t)k * N, o);
      }
    }
  }
  if (WARP) {
    for (int q = 0; q < per; ++q) {
      if (g == q) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int k = t + i * tpr;
          if (k < nvec) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              float* a = wsum + (int64_t)k * N + e;
              a[0] = (q ? a[0] : 0.f) + gw[i][e];
              a[C] = (q ? a[C] : 0.f) + gb[i][e];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * C; c += blockDim.x)
      part[(int64_t)blockIdx.x * 2 * C + c] = wsum[c];
  } else {
    float* p = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          *reinterpret_cast<float4*>(p + (int64_t)k * N + e) =
              make_float4(gw[i][e], gw[i][e + 1], gw[i][e + 2], gw[i][e + 3]);
          *reinterpret_cast<float4*>(p + C + (int64_t)k * N + e) =
              make_float4(gb[i][e], gb[i][e + 1], gb[i][e + 2], gb[i][e + 3]);
        }
      }
    }
  }
}

// Rows too long for registers: grad_x with one CTA per row, keeping (mean, s)
// per row in `stat`; then k_norm_bwd_cols sums the channels over slices of rows.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) k_norm_bwd_long(
    int64_t C, float eps, const T* __restrict__ x, const float* __restrict__ w,
    const T* __restrict__ gy, T* __restrict__ gx, float2* __restrict__ stat, int* status) {
  constexpr int N = Vec<T>::N;
  __shared__ Share rec[32];
  const int64_t row = blockIdx.x, nvec = C / N;
  float sum = 0.f, xv[N], gv[N];
  int64_t cnt = 0;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(x + row * C + k * N, xv);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) q += xv[e];
    sum += q;
    cnt += N;
  }
  Share sh;
  sh.n = warp_sum((float)cnt);
  sh.m = sh.n > 0.f ? warp_sum(sum) / sh.n : 0.f;
  float m2 = 0.f, sa = 0.f, sax = 0.f;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(x + row * C + k * N, xv);
    Vec<T>::load(gy + row * C + k * N, gv);
    float q2 = 0.f, qa = 0.f, qx = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = xv[e] - sh.m, a = gv[e] * __ldg(w + k * N + e);
      q2 = fmaf(d, d, q2);
      qa += a;
      qx = fmaf(a, d, qx);
    }
    m2 += q2;
    sa += qa;
    sax += qx;
  }
  sh.m2 = warp_sum(m2);
  sh.a = warp_sum(sa);
  sh.ax = warp_sum(sax);
  sh = join_shares<true>(sh, rec, blockDim.x / 32, C);
  const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
  const float c1 = sh.a / (float)C, c2 = sh.ax * s / (float)C;
  if (threadIdx.x == 0) {
    report(sh.m, s, status);
    stat[row] = make_float2(sh.m, s);
  }
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(x + row * C + k * N, xv);
    Vec<T>::load(gy + row * C + k * N, gv);
    float o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float xh = (xv[e] - sh.m) * s, a = gv[e] * __ldg(w + k * N + e);
      o[e] = s * (a - c1 - xh * c2);
    }
    Vec<T>::store_stream(gx + row * C + k * N, o);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_norm_bwd_cols(int64_t rows, int64_t C,
                                                       const T* __restrict__ x,
                                                       const T* __restrict__ gy,
                                                       const float2* __restrict__ stat,
                                                       float* __restrict__ part) {
  constexpr int N = Vec<T>::N;
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= C / N) return;
  float gw[N] = {}, gb[N] = {}, xv[N], gv[N];
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const float2 st = __ldg(stat + r);
    Vec<T>::load_stream(x + r * C + k * N, xv);
    Vec<T>::load_stream(gy + r * C + k * N, gv);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      gw[e] = fmaf(gv[e], (xv[e] - st.x) * st.y, gw[e]);
      gb[e] += gv[e];
    }
  }
  float* p = part + (int64_t)blockIdx.y * 2 * C + k * N;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    p[e] = gw[e];
    p[C + e] = gb[e];
  }
}

// grad_weight and grad_bias: column c of the nparts partial rows, added by
// kFinSlices threads in a fixed interleaving and then in slice order.
constexpr int kFinSlices = 8;
__global__ void __launch_bounds__(32 * kFinSlices) k_norm_fin(int64_t C, int nparts,
                                                              const float* __restrict__ part,
                                                              float* __restrict__ gw,
                                                              float* __restrict__ gb) {
  __shared__ float acc[kFinSlices][32];
  const int lane = threadIdx.x % 32, sl = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < 2 * C)
    for (int p = sl; p < nparts; p += kFinSlices) a += part[(int64_t)p * 2 * C + c];
  acc[sl][lane] = a;
  __syncthreads();
  if (sl == 0 && c < 2 * C) {
#pragma unroll
    for (int q = 1; q < kFinSlices; ++q) a += acc[q][lane];
    if (c < C)
      gw[c] = a;
    else if (gb)
      gb[c - C] = a;
  }
}

// ------------------------------------------------------------------- shapes
// How a row of nvec vectors is laid over threads.
struct Shape {
  bool warp, longrow;
  int vpt, threads;  // vectors per thread, threads per CTA
};

Shape fwd_shape(int64_t nvec) {
  Shape h{};
  if (nvec <= 128) {
    h.warp = true;
    h.vpt = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    h.threads = 256;
    return h;
  }
  h.vpt = nvec <= 512 ? 1 : nvec <= 2048 ? 2 : 4;
  h.longrow = nvec > 4 * kMaxThreads;
  h.threads = h.longrow ? kMaxThreads : (int)(((nvec + h.vpt - 1) / h.vpt + 31) / 32 * 32);
  return h;
}

// per16: vectors of 16 channels (2 for bf16, 4 for fp32)
Shape bwd_shape(int64_t nvec, int per16) {
  Shape h{};
  if (nvec <= 128) {
    h.warp = true;
    h.vpt = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    h.threads = 256;
    return h;
  }
  // 16 channels per thread: 512 threads (128 registers each) up to 8192
  // channels, 1024 (64 registers) up to 16384
  h.vpt = nvec <= 512 ? 1 : per16;
  h.longrow = nvec > (int64_t)per16 * kMaxThreads;
  h.threads = h.longrow ? kMaxThreads : (int)(((nvec + h.vpt - 1) / h.vpt + 31) / 32 * 32);
  return h;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

// Partial rows of grad_weight / grad_bias: the workspace is sized for this many.
constexpr int kMaxParts = 512;

template <typename T>
cudaError_t fwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const float* b,
                T* y, int* st, cudaStream_t s) {
  const Shape h = fwd_shape(C / Vec<T>::N);
  if (h.longrow) {
    k_norm_fwd_long<T><<<(unsigned)rows, h.threads, 0, s>>>(C, eps, x, w, b, y, st);
  } else if (h.warp) {
    const unsigned grid = (unsigned)((rows + h.threads / 32 - 1) / (h.threads / 32));
    if (h.vpt == 1) k_norm_fwd<T, 1, true><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
    else if (h.vpt == 2) k_norm_fwd<T, 2, true><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
    else k_norm_fwd<T, 4, true><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
  } else {
    const unsigned grid = (unsigned)rows;
    if (h.vpt == 1) k_norm_fwd<T, 1, false><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
    else if (h.vpt == 2) k_norm_fwd<T, 2, false><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
    else k_norm_fwd<T, 4, false><<<grid, h.threads, 0, s>>>(rows, C, eps, x, w, b, y, st);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const T* gy, T* gx,
                float* gw, float* gb, void* ws, int* st, cudaStream_t s) {
  const Shape h = bwd_shape(C / Vec<T>::N, 16 / Vec<T>::N);
  const int sms = sm_count();
  float* part = (float*)ws;
  int nparts;
  if (h.longrow) {
    float2* stat = (float2*)(part + (int64_t)kMaxParts * 2 * C);
    k_norm_bwd_long<T><<<(unsigned)rows, h.threads, 0, s>>>(C, eps, x, w, gy, gx, stat, st);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    nparts = (int)(rows < 64 ? rows : 64);
    const dim3 grid((unsigned)((C / Vec<T>::N + 255) / 256), (unsigned)nparts);
    k_norm_bwd_cols<T><<<grid, 256, 0, s>>>(rows, C, x, gy, stat, part);
  } else {
    const int per = h.warp ? h.threads / 32 : 1;
    const int64_t groups = (rows + per - 1) / per;
    const int resident = h.threads <= 512 ? 2 : 1;
    int64_t g = (int64_t)sms * resident;
    if (g > kMaxParts) g = kMaxParts;
    nparts = (int)(groups < g ? groups : g);
    const size_t sm = h.warp ? (size_t)2 * C * 4 : 0;
    if (h.warp) {
      if (h.vpt == 1) k_norm_bwd<T, 1, true, 256><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
      else if (h.vpt == 2) k_norm_bwd<T, 2, true, 256><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
      else k_norm_bwd<T, 4, true, 256><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
    } else {
      constexpr int V = 16 / Vec<T>::N;
      if (h.vpt == 1) k_norm_bwd<T, 1, false, 512><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
      else if (h.threads <= 512) k_norm_bwd<T, V, false, 512><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
      else k_norm_bwd<T, V, false, 1024><<<nparts, h.threads, sm, s>>>(rows, C, eps, x, w, gy, gx, part, st);
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_norm_fin<<<(unsigned)((2 * C + 31) / 32), 32 * kFinSlices, 0, s>>>(C, nparts, part, gw, gb);
  return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C, int dtype) {
  const int n = dtype == MHC_DTYPE_BF16 ? 8 : 4;
  const size_t part = (size_t)kMaxParts * 2 * C * 4;
  return part + (bwd_shape(C / n, 16 / n).longrow ? (size_t)rows * sizeof(float2) : 0);
}

cudaError_t norm_fwd_dispatch(int dtype, int64_t rows, int64_t C, float eps, const void* x,
                              const float* w, const float* b, void* y, int* st, cudaStream_t s) {
  if (dtype == MHC_DTYPE_BF16)
    return fwd(rows, C, eps, (const __nv_bfloat16*)x, w, b, (__nv_bfloat16*)y, st, s);
  return fwd(rows, C, eps, (const float*)x, w, b, (float*)y, st, s);
}

cudaError_t norm_bwd_dispatch(int dtype, int64_t rows, int64_t C, float eps, const void* x,
                              const float* w, const void* gy, void* gx, float* gw, float* gb,
                              void* ws, int* st, cudaStream_t s) {
  if (dtype == MHC_DTYPE_BF16)
    return bwd(rows, C, eps, (const __nv_bfloat16*)x, w, (const __nv_bfloat16*)gy,
               (__nv_bfloat16*)gx, gw, gb, ws, st, s);
  return bwd(rows, C, eps, (const float*)x, w, (const float*)gy, (float*)gx, gw, gb, ws, st, s);
}

}  // namespace mhc
