// k_norm.cu -- layer norm over the channels of a token, forward and backward.
//
//   mean = 1/C sum x,  s = 1/sqrt(1/C sum (x - mean)^2 + eps),  xh = (x - mean) s
//   forward : y = xh w + b
//   backward: a = gy w,  gx = s (a - mean(a) - xh mean(a xh)),
//             gw = sum_t gy xh,  gb = sum_t gy
//
// HBM bound: one read of every input and one write of every output.  A token's
// row stays on the chip between its statistics and its outputs.  Each warp takes
// its own share of a row in two passes (its sum, then the squares about its own
// mean), and the shares are joined as M2 = sum_w (M2_w + n_w (m_w - mean)^2): no
// difference of large sums, and one block barrier per row.
//
// What is left to care about is the number of instructions: with 16 channels per
// thread and scalar arithmetic the shuffles and joins of a row cost more than its
// elements (T = 16384, C = 7168 bf16: 187 us forward, 455 us backward).  So a
// thread takes up to 64 channels (forward) or 32 (backward) and works on pairs of
// floats (the paired fp32 instructions).
#include "mhc_common.cuh"
#include "mhc_dispatch.h"
#include "tc_pair.cuh"

namespace mhc {

namespace {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ uint64_t f2add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2dup(float v) { return f2pack(v, v); }
__device__ __forceinline__ float f2sum(uint64_t v) {
  return __uint_as_float((uint32_t)v) + __uint_as_float((uint32_t)(v >> 32));
}

// One 16-byte vector of the activations as P pairs of floats.
template <typename T> struct Pairs;
template <> struct Pairs<__nv_bfloat16> {
  static constexpr int P = 4;
  __device__ __forceinline__ static uint64_t get(const uint4& q, int i) {
    return bf2_to_f2(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w);
  }
  __device__ __forceinline__ static uint4 pack(const uint64_t (&v)[4]) {
    return make_uint4(f2_to_bf2(v[0]), f2_to_bf2(v[1]), f2_to_bf2(v[2]), f2_to_bf2(v[3]));
  }
};
template <> struct Pairs<float> {
  static constexpr int P = 2;
  __device__ __forceinline__ static uint64_t get(const uint4& q, int i) {
    return i == 0 ? (uint64_t)q.y << 32 | q.x : (uint64_t)q.w << 32 | q.z;
  }
  __device__ __forceinline__ static uint4 pack(const uint64_t (&v)[2]) {
    return make_uint4((uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1],
                      (uint32_t)(v[1] >> 32));
  }
};

// The fp32 parameters of a vector's channels, as pairs.
template <int P>
__device__ __forceinline__ void load_param(const float* p, uint64_t (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const ulonglong2 q = __ldg(reinterpret_cast<const ulonglong2*>(p + 2 * i));
    v[i] = q.x;
    v[i + 1] = q.y;
  }
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

// Channels of the vectors k = first + lane, first + lane + stride, ... below
// nvec that a warp's lanes hold, VPT per lane.
__device__ __forceinline__ int share_channels(int vpt, int n, int first, int stride, int nvec) {
  int c = 0;
  for (int i = 0; i < vpt; ++i) {
    const int left = nvec - first - i * stride;
    c += left <= 0 ? 0 : left < 32 ? left : 32;
  }
  return c * n;
}

// ------------------------------------------------------------------ forward
// WARP: one row per warp (blockDim.x / 32 rows per CTA); otherwise one row per
// CTA.  A thread holds VPT 16-byte vectors of its row.
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 512)
    k_norm_fwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
               const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
               int* status) {
  constexpr int N = Vec<T>::N, P = Pairs<T>::P;
  using PV = Pairs<T>;
  __shared__ Share rec[32];
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32
                           : (int64_t)blockIdx.x;
  tc::grid_wait();
  if (WARP && row >= rows) return;
  const int nvec = (int)(C / N);
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * C);
  uint4 v[VPT];
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int k = t + i * tpr;
    v[i] = k < nvec ? __ldcs(xr + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) sum = f2add(sum, PV::get(v[i], e));
  Share sh;
  sh.n = WARP ? (float)C : (float)share_channels(VPT, N, t & ~31, tpr, nvec);
  sh.m = sh.n > 0.f ? warp_sum(f2sum(sum)) / sh.n : 0.f;
  uint64_t m2 = 0, nm = f2dup(-sh.m);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * tpr < nvec) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const uint64_t d = f2add(PV::get(v[i], e), nm);
        m2 = f2fma(d, d, m2);
      }
    }
  sh.m2 = warp_sum(f2sum(m2));
  if (!WARP) sh = join_shares<false>(sh, rec, blockDim.x / 32, C);
  const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
  if (t == 0) report(sh.m, s, status);
  nm = f2dup(-sh.m);
  const uint64_t ss = f2dup(s);
  uint4* yr = reinterpret_cast<uint4*>(y + row * C);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int k = t + i * tpr;
    if (k < nvec) {
      uint64_t wv[P], bv[P] = {}, o[P];
      load_param<P>(w + (int64_t)k * N, wv);
      if (b) load_param<P>(b + (int64_t)k * N, bv);
#pragma unroll
      for (int e = 0; e < P; ++e)
        o[e] = f2fma(f2mul(f2add(PV::get(v[i], e), nm), ss), wv[e], bv[e]);
      __stcs(yr + k, PV::pack(o));
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
// [2][C] per CTA, summed in CTA order by k_norm_fin.  x and grad_y come through
// a ring of SLOTS rows in shared memory (cp.async: a thread copies what it later
// reads itself, so no barrier is needed), the next rows on their way while one is
// worked on.  WARP: one row per warp at a time, the warps' sums joined in warp
// order through the ring's memory.
__device__ __forceinline__ void cp16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src)
               : "memory");
}

template <typename T, int VPT, bool WARP, int SLOTS, int MAXT, int PERSM>
__global__ void __launch_bounds__(MAXT, PERSM)
    k_norm_bwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
               const float* __restrict__ w, const T* __restrict__ gy, T* __restrict__ gx,
               float* __restrict__ part, int* status) {
  constexpr int N = Vec<T>::N, P = Pairs<T>::P;
  using PV = Pairs<T>;
  __shared__ Share rec[2][32];
  extern __shared__ uint4 ring[];  // [group][SLOTS][x, gy][nvec]; WARP, at the end: [2][C] sums
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int per = WARP ? blockDim.x / 32 : 1, g = WARP ? threadIdx.x / 32 : 0;
  const int nvec = (int)(C / N);
  uint4* mine = ring + (int64_t)g * SLOTS * 2 * nvec;
  const int64_t row0 = (int64_t)blockIdx.x * per + g, step = (int64_t)gridDim.x * per;
  tc::grid_release();
  tc::grid_wait();
  auto fetch = [&](int64_t row, int slot) {
    if (row < rows) {
      uint4* d = mine + slot * 2 * nvec;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int k = t + i * tpr;
        if (k < nvec) {
          cp16(d + k, x + row * C + (int64_t)k * N);
          cp16(d + nvec + k, gy + row * C + (int64_t)k * N);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint64_t gw[VPT][P], gb[VPT][P];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) gw[i][e] = gb[i][e] = 0;
  const float share = WARP ? (float)C : (float)share_channels(VPT, N, t & ~31, tpr, nvec);
#pragma unroll
  for (int q = 0; q + 1 < SLOTS; ++q) fetch(row0 + q * step, q);
  int it = 0;
  for (int64_t row = row0; row < rows; row += step, ++it) {
    if (SLOTS == 1) fetch(row, 0);
    else fetch(row + (SLOTS - 1) * step, (it + SLOTS - 1) % SLOTS);
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    const uint4* xs = mine + (it % SLOTS) * 2 * nvec;
    const uint4* gs = xs + nvec;
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        const uint4 q = xs[k];
#pragma unroll
        for (int e = 0; e < P; ++e) sum = f2add(sum, PV::get(q, e));
      }
    }
    Share sh;
    sh.n = share;
    sh.m = share > 0.f ? warp_sum(f2sum(sum)) / share : 0.f;
    uint64_t m2 = 0, sa = 0, sax = 0, nm = f2dup(-sh.m);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        const uint4 q = xs[k], h = gs[k];
        uint64_t wv[P];
        load_param<P>(w + (int64_t)k * N, wv);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const uint64_t d = f2add(PV::get(q, e), nm), a = f2mul(PV::get(h, e), wv[e]);
          m2 = f2fma(d, d, m2);
          sa = f2add(sa, a);
          sax = f2fma(a, d, sax);
        }
      }
    }
    sh.m2 = warp_sum(f2sum(m2));
    sh.a = warp_sum(f2sum(sa));
    sh.ax = warp_sum(f2sum(sax));
    if (!WARP) sh = join_shares<true>(sh, rec[it & 1], blockDim.x / 32, C);
    const float s = 1.0f / sqrtf(sh.m2 / (float)C + eps);
    if (t == 0) report(sh.m, s, status);
    nm = f2dup(-sh.m);
    const uint64_t ss = f2dup(s), c1 = f2dup(-sh.a / (float)C),
                   c2 = f2dup(-(sh.ax * s / (float)C));
    uint4* gr = reinterpret_cast<uint4*>(gx + row * C);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        const uint4 q = xs[k], h = gs[k];
        uint64_t wv[P], o[P];
        load_param<P>(w + (int64_t)k * N, wv);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const uint64_t gv = PV::get(h, e), xh = f2mul(f2add(PV::get(q, e), nm), ss);
          o[e] = f2mul(f2fma(xh, c2, f2fma(gv, wv[e], c1)), ss);
          gw[i][e] = f2fma(gv, xh, gw[i][e]);
          gb[i][e] = f2add(gb[i][e], gv);
        }
        __stcs(gr + k, PV::pack(o));
      }
    }
  }
  float* sums = WARP ? reinterpret_cast<float*>(ring) : part + (int64_t)blockIdx.x * 2 * C;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (WARP) __syncthreads();
  for (int q = 0; q < per; ++q) {
    if (g == q) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int k = t + i * tpr;
        if (k < nvec) {
          ulonglong2* pw = reinterpret_cast<ulonglong2*>(sums + (int64_t)k * N);
          ulonglong2* pb = reinterpret_cast<ulonglong2*>(sums + C + (int64_t)k * N);
#pragma unroll
          for (int e = 0; e < P; e += 2) {
            ulonglong2 a = make_ulonglong2(gw[i][e], gw[i][e + 1]);
            ulonglong2 c = make_ulonglong2(gb[i][e], gb[i][e + 1]);
            if (q > 0) {
              const ulonglong2 a0 = pw[e / 2], c0 = pb[e / 2];
              a = make_ulonglong2(f2add(a0.x, a.x), f2add(a0.y, a.y));
              c = make_ulonglong2(f2add(c0.x, c.x), f2add(c0.y, c.y));
            }
            pw[e / 2] = a;
            pb[e / 2] = c;
          }
        }
      }
    }
    if (WARP) __syncthreads();
  }
  if (WARP)
    for (int c = threadIdx.x; c < C / 2; c += blockDim.x)
      reinterpret_cast<float4*>(part + (int64_t)blockIdx.x * 2 * C)[c] =
          reinterpret_cast<const float4*>(sums)[c];
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

// grad_weight and grad_bias: four columns per thread of the nparts partial rows,
// added by kFinSlices threads in a fixed interleaving and then in slice order.
constexpr int kFinSlices = 16, kFinCols = 16;
__global__ void __launch_bounds__(kFinCols * kFinSlices)
    k_norm_fin(int64_t C, int nparts, const float* __restrict__ part, float* __restrict__ gw,
               float* __restrict__ gb) {
  __shared__ float4 acc[kFinSlices][kFinCols];
  const int lane = threadIdx.x % kFinCols, sl = threadIdx.x / kFinCols;
  const int64_t c = ((int64_t)blockIdx.x * kFinCols + lane) * 4;
  tc::grid_wait();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& q) { a.x += q.x, a.y += q.y, a.z += q.z, a.w += q.w; };
  if (c < 2 * C) {
#pragma unroll 4
    for (int p = sl; p < nparts; p += kFinSlices)
      add(__ldcs(reinterpret_cast<const float4*>(part + (int64_t)p * 2 * C + c)));
  }
  acc[sl][lane] = a;
  __syncthreads();
  if (sl == 0 && c < 2 * C) {
#pragma unroll
    for (int q = 1; q < kFinSlices; ++q) add(acc[q][lane]);
    if (c < C) *reinterpret_cast<float4*>(gw + c) = a;
    else if (gb) *reinterpret_cast<float4*>(gb + c - C) = a;
  }
}

// ------------------------------------------------------------------- shapes
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

int round32(int64_t v) { return (int)((v + 31) / 32 * 32); }

// Partial rows of grad_weight / grad_bias: the workspace is sized for this many.
constexpr int kMaxParts = 320;
constexpr int64_t kBwdChannels = 16384;  // longer rows take the walks over memory

template <typename T>
cudaError_t fwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const float* b,
                T* y, int* st, cudaStream_t s) {
  const int64_t nvec = C / Vec<T>::N;
  if (nvec > 8 * 512) {
    k_norm_fwd_long<T><<<(unsigned)rows, kMaxThreads, 0, s>>>(C, eps, x, w, b, y, st);
    return cudaGetLastError();
  }
  if (nvec <= 8 * 32) {
    const unsigned grid = (unsigned)((rows + 3) / 4);
    auto kern = nvec <= 32   ? k_norm_fwd<T, 1, true>
                : nvec <= 64 ? k_norm_fwd<T, 2, true>
                : nvec <= 128 ? k_norm_fwd<T, 4, true>
                              : k_norm_fwd<T, 8, true>;
    return launch_after(kern, grid, 128, 0, 1, s, rows, C, eps, x, w, b, y, st);
  }
  return launch_after(k_norm_fwd<T, 8, false>, (unsigned)rows, round32((nvec + 7) / 8), 0, 1, s,
                      rows, C, eps, x, w, b, y, st);
}

template <typename T, int VPT, bool WARP, int SLOTS, int MAXT, int PERSM>
cudaError_t bwd_rows(int64_t rows, int64_t C, float eps, const T* x, const float* w, const T* gy,
                     T* gx, float* part, int threads, int* nparts, int* st, cudaStream_t s) {
  const int per = WARP ? threads / 32 : 1;
  const size_t slot = (size_t)2 * C * sizeof(T), sum = WARP ? (size_t)2 * C * 4 : 0;
  const size_t ring = per * SLOTS * slot, sm = ring > sum ? ring : sum;
  const int64_t groups = (rows + per - 1) / per;
  int64_t g = (int64_t)sm_count() * PERSM;
  if (g > kMaxParts) g = kMaxParts;
  *nparts = (int)(groups < g ? groups : g);
  auto kern = k_norm_bwd<T, VPT, WARP, SLOTS, MAXT, PERSM>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_after(kern, (unsigned)*nparts, (unsigned)threads, sm, 1, s, rows, C, eps, x, w, gy,
                      gx, part, st);
}

// 32 channels per thread: rows of up to 1024 channels on one warp, longer ones on
// a CTA of which two fit an SM (up to 8192 channels in bf16, 4778 in fp32) or
// one; three rows in the ring where they fit (an fp32 row pair of 16384 channels
// takes 128 KB: one).
template <typename T>
cudaError_t bwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const T* gy, T* gx,
                float* gw, float* gb, void* ws, int* st, cudaStream_t s) {
  constexpr int V = 32 / Vec<T>::N;  // vectors of a thread
  const int64_t nvec = C / Vec<T>::N;
  float* part = (float*)ws;
  int nparts = 0;
  cudaError_t e;
  const int threads = round32((nvec + V - 1) / V);
  if (C > kBwdChannels) {
    float2* stat = (float2*)(part + (int64_t)kMaxParts * 2 * C);
    k_norm_bwd_long<T><<<(unsigned)rows, kMaxThreads, 0, s>>>(C, eps, x, w, gy, gx, stat, st);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    nparts = (int)(rows < 64 ? rows : 64);
    const dim3 grid((unsigned)((nvec + 255) / 256), (unsigned)nparts);
    k_norm_bwd_cols<T><<<grid, 256, 0, s>>>(rows, C, x, gy, stat, part);
    e = cudaGetLastError();
  } else if (C <= 256) {
    e = bwd_rows<T, V / 4, true, 3, 256, 2>(rows, C, eps, x, w, gy, gx, part, 256, &nparts, st, s);
  } else if (C <= 512) {
    e = bwd_rows<T, V / 2, true, 3, 256, 2>(rows, C, eps, x, w, gy, gx, part, 256, &nparts, st, s);
  } else if (C <= 1024) {
    e = bwd_rows<T, V, true, 3, 128, 2>(rows, C, eps, x, w, gy, gx, part, 128, &nparts, st, s);
  } else if (threads <= 256 && 3 * 2 * C * sizeof(T) <= 112 * 1024) {
    e = bwd_rows<T, V, false, 3, 256, 2>(rows, C, eps, x, w, gy, gx, part, threads, &nparts, st, s);
  } else if (3 * 2 * C * sizeof(T) <= 224 * 1024) {
    e = bwd_rows<T, V, false, 3, 512, 1>(rows, C, eps, x, w, gy, gx, part, threads, &nparts, st, s);
  } else {
    e = bwd_rows<T, V, false, 1, 512, 1>(rows, C, eps, x, w, gy, gx, part, threads, &nparts, st, s);
  }
  if (e != cudaSuccess) return e;
  const int64_t cols = 2 * C / 4;
  return launch_after(k_norm_fin, (unsigned)((cols + kFinCols - 1) / kFinCols),
                      kFinCols * kFinSlices, 0, 1, s, C, nparts, (const float*)part, gw, gb);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C, int dtype) {
  (void)dtype;
  const size_t part = (size_t)kMaxParts * 2 * C * 4;
  return part + (C > kBwdChannels ? (size_t)rows * sizeof(float2) : 0);
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
