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
// mean m_w), and the shares are joined about the first warp's mean m_0:
//   mean = m_0 + 1/C sum_w (n_w (m_w - m_0) + r_w),  r_w = sum of x - m_w
//   M2   = sum_w (M2_w + d_w (2 r_w + n_w d_w)),     d_w = m_w - mean
// No difference of large sums, one block barrier per row, and a mean that is off by
// one rounding of itself where the row's values are close to one another: there s
// is as large as 1/sqrt(eps) and would make every further rounding of the mean (of
// a sum, a quotient, or of mean s in x s - mean s) part of the result.  r_w is what
// is left of the warp's own roundings; in bf16 the sums of such rows are exact and
// sum - n_w m_w gives it, in fp32 it is added up beside the squares.
//
// With 16 channels per thread and a row at a time the shuffles and joins of a row
// cost more than its elements (T = 16384, C = 7168 bf16: 187 us forward, 455 us
// backward).  So a thread takes 32 channels or 64 and, where there are many rows, two
// rows at a time, in paired fp32 instructions: 98 us (4.8 TB/s) and 173 us (4.1 TB/s;
// 2 and 6 us of them are the joined mean and x - mean).  What holds them back now is
// latency: less than half of the issue slots are taken, most often a warp waits for
// memory or for its own last result, and there are 14 warps to an SM.
// The backward's ring leaves an SM two CTAs of 7 warps at that width, and less L1 than
// the 28 KB of the weight, which is read twice for each pair of rows.
#include <algorithm>

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

// What one warp knows of its share of a row: the mean of its channels as rounded, the
// sum r and the squares of what is left about it and, in the backward, the sums of a
// and of a (x - m).
struct Share {
  float m, m2, a, ax, r;
};

// The squares about the mean of n values whose squares about m are m2 and whose sum
// about m is r, d = m - mean.  Roundings may leave it below zero.
__device__ __forceinline__ float about_mean(float m2, float r, float n, float d) {
  return fmaf(d, fmaf(n, d, 2.0f * r), m2);
}
// ... and 0 then; NaN stays.
__device__ __forceinline__ float not_below_0(float v) { return v < 0.f ? 0.f : v; }

// s is 0 only where the variance left fp32's range.
__device__ __forceinline__ void report(float mean, float s, int* status) {
  if (!isfinite(mean) || !isfinite(s) || s == 0.f) flag_status(status, MHC_ERR_NONFINITE);
}

// Channels that warp `warp` of a row of nvec vectors holds: vectors 32 warp + lane,
// and every `stride` vectors after that.
__device__ __forceinline__ float share_channels(int warp, int stride, int n, int nvec) {
  int c = 0;
  for (int k = 32 * warp; k < nvec; k += stride) c += nvec - k < 32 ? nvec - k : 32;
  return (float)(c * n);
}
__device__ __forceinline__ float inv_or_0(float n) { return n > 0.f ? 1.0f / n : 0.f; }

__device__ __forceinline__ void cp16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums over the warp of a (row 0) and b (row 1): lanes 0..15 get row 0's, lanes
// 16..31 row 1's.
__device__ __forceinline__ float pair_sum(float a, float b, int lane) {
  const bool hi = lane >= 16;
  float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// xh from d = x - m_w, the warp's own mean.  fp32: shift = m_w - mean, and d + shift is
// exact for values near one another, where m_w is a few roundings off.  bf16: their m_w
// is off by its own rounding only, and shift = (m_w - mean) s is no larger than the
// largest xh, so that its rounding is 2^-24 of that.
template <bool F32>
__device__ __forceinline__ uint64_t from_share(uint64_t d, uint64_t shift, uint64_t s) {
  return F32 ? f2mul(f2add(d, shift), s) : f2fma(d, s, shift);
}

// ------------------------------------------------------------------ forward
// WARP: one row per warp (blockDim.x / 32 rows per CTA); otherwise one row per
// CTA.  A thread holds VPT 16-byte vectors of its row.
template <typename T, int VPT, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_norm_fwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
               const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
               int* status) {
  constexpr int N = Vec<T>::N, P = Pairs<T>::P;
  constexpr bool F32 = sizeof(T) == 4;
  using PV = Pairs<T>;
  __shared__ float4 rec[16];
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32
                           : (int64_t)blockIdx.x;
  tc::grid_wait();
  if (WARP && row >= rows) return;
  const int nvec = (int)(C / N);
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * C);
  uint4 raw[VPT];
  uint64_t v[VPT][P], sum = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int k = t + i * tpr;
    raw[i] = k < nvec ? __ldcs(xr + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) {
      v[i][e] = PV::get(raw[i], e);
      sum = f2add(sum, v[i][e]);
    }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float n = WARP ? (float)C : share_channels(warp, tpr, N, nvec);
  const float all = warp_sum(f2sum(sum)), mw = all * inv_or_0(n);
  uint64_t m2 = 0, left = 0, nm = f2dup(-mw);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * tpr < nvec) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const uint64_t d = v[i][e] = f2add(v[i][e], nm);
        m2 = f2fma(d, d, m2);
        if (F32) left = f2add(left, d);
      }
    }
  float var = warp_sum(f2sum(m2)), m;
  const float r = F32 ? warp_sum(f2sum(left)) : fmaf(-n, mw, all);
  const float inv_c = 1.0f / (float)C;
  if (WARP) {
    m = fmaf(r, inv_c, mw);
    var = about_mean(var, r, n, mw - m);
  } else {
    if (lane == 0) rec[warp] = make_float4(n, mw, var, r);
    __syncthreads();
    const float4 q = lane < tpr / 32 ? rec[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    const float m0 = rec[0].y;
    m = fmaf(warp_sum(fmaf(q.x, q.y - m0, q.w)), inv_c, m0);
    var = warp_sum(about_mean(q.z, q.w, q.x, q.y - m));
  }
  const float s = rsqrtf(not_below_0(var) * inv_c + eps);
  if (t == 0) report(m, s, status);
  const uint64_t ss = f2dup(s), shift = f2dup(F32 ? mw - m : (mw - m) * s);
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
        o[e] = f2fma(from_share<F32>(v[i][e], shift, ss), wv[e], bv[e]);
      __stcs(yr + k, PV::pack(o));
    }
  }
}

// Many bf16 rows: persistent CTAs that take two rows at a time, as the backward does (see
// there), through a ring of two row pairs in shared memory.  Two rows share the
// loads of weight and bias and half the shuffles, and a CTA's fixed work is paid
// once: T = 16384, C = 7168 bf16 takes 98 us against 106 with a row per CTA.
template <int VPT, bool WARP, int MAXT, int PERSM>
__global__ void __launch_bounds__(MAXT, PERSM)
    k_norm_fwd_pairs(int64_t rows, int64_t C, float eps, const __nv_bfloat16* __restrict__ x,
                     const float* __restrict__ w, const float* __restrict__ b,
                     __nv_bfloat16* __restrict__ y, int* status) {
  using PV = Pairs<__nv_bfloat16>;
  constexpr int N = Vec<__nv_bfloat16>::N, P = PV::P;
  constexpr int W = WARP ? 1 : MAXT / 32;
  __shared__ float4 rec[WARP ? 1 : 2][2][W];
  extern __shared__ uint4 ring[];  // [group][2][row][nvec]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? lane : threadIdx.x;
  const int per = WARP ? blockDim.x / 32 : 1, g = WARP ? warp : 0;
  const int nvec = (int)(C / N);
  uint4* mine = ring + (int64_t)g * 4 * nvec;
  const int64_t row0 = 2 * ((int64_t)blockIdx.x * per + g), step = 2 * (int64_t)gridDim.x * per;
  const float inv_c = 1.0f / (float)C;
  const float n = WARP ? (float)C : share_channels(warp, tpr, N, nvec), inv_n = inv_or_0(n);
  const float nq =
      WARP || (lane & 15) >= tpr / 32 ? 0.f : share_channels(lane & 15, tpr, N, nvec);
  tc::grid_wait();
  auto fetch = [&](int64_t row, int slot) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (row + r < rows) {
        uint4* d = mine + (slot * 2 + r) * nvec;
        const uint4* xr = reinterpret_cast<const uint4*>(x + (row + r) * C);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int k = t + i * tpr;
          if (k < nvec) cp16(d + k, xr + k);
        }
      }
    }
    cp_commit();
  };
  fetch(row0, 0);
  int it = 0;
  for (int64_t row = row0; row < rows; row += step, ++it) {
    const int slot = it & 1;
    fetch(row + step, slot ^ 1);
    cp_wait<1>();
    const bool two = row + 1 < rows;
    const uint4* xs[2] = {mine + slot * 2 * nvec, mine + (slot * 2 + (two ? 1 : 0)) * nvec};
    uint64_t v[2][VPT][P], sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 q = k < nvec ? xs[r][k] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          v[r][i][e] = PV::get(q, e);
          sum[r] = f2add(sum[r], v[r][i][e]);
        }
      }
    }
    // from here to the join a lane's scalars are its half-warp's row's
    const float all = pair_sum(f2sum(sum[0]), f2sum(sum[1]), lane), mw = all * inv_n;
    const uint64_t nm[2] = {f2dup(-__shfl_sync(0xffffffffu, mw, 0)),
                            f2dup(-__shfl_sync(0xffffffffu, mw, 16))};
    uint64_t m2[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * tpr < nvec) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const uint64_t d = v[r][i][e] = f2add(v[r][i][e], nm[r]);
            m2[r] = f2fma(d, d, m2[r]);
          }
      }
    }
    float v2 = pair_sum(f2sum(m2[0]), f2sum(m2[1]), lane), m;
    const float rw = fmaf(-n, mw, all);
    if (WARP) {
      m = fmaf(rw, inv_c, mw);
      v2 = about_mean(v2, rw, n, mw - m);
    } else {
      if ((lane & 15) == 0) rec[it & 1][lane >> 4][warp] = make_float4(mw, v2, rw, 0.f);
      __syncthreads();
      const float4* recs = rec[it & 1][lane >> 4];
      const float4 q = nq > 0.f ? recs[lane & 15] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float m0 = recs[0].x;
      m = fmaf(half_sum(fmaf(nq, q.x - m0, q.z)), inv_c, m0);
      v2 = half_sum(about_mean(q.y, q.z, nq, q.x - m));
    }
    const float s = rsqrtf(not_below_0(v2) * inv_c + eps);
    if (t == 0 || (t == 16 && two)) report(m, s, status);
    const float off = (mw - m) * s;
    uint64_t ss[2], shift[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ss[r] = f2dup(__shfl_sync(0xffffffffu, s, 16 * r));
      shift[r] = f2dup(__shfl_sync(0xffffffffu, off, 16 * r));
    }
    uint4* yr = reinterpret_cast<uint4*>(y + row * C);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        uint64_t wv[P], bv[P] = {};
        load_param<P>(w + k * N, wv);
        if (b) load_param<P>(b + k * N, bv);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (r == 0 || two) {
            uint64_t o[P];
#pragma unroll
            for (int e = 0; e < P; ++e)
              o[e] = f2fma(from_share<false>(v[r][i][e], shift[r], ss[r]), wv[e], bv[e]);
            __stcs(yr + r * nvec + k, PV::pack(o));
          }
        }
      }
    }
  }
}

// A row's statistics from its warps' shares, for CTAs of kMaxThreads.
__device__ __forceinline__ Share join_shares(float n, const Share& mine, float4* rec, float2* cnt,
                                             int64_t C) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) {
    rec[warp] = make_float4(mine.m, mine.m2, mine.a, mine.ax);
    cnt[warp] = make_float2(n, mine.r);
  }
  __syncthreads();
  const float4 q = rec[lane];
  const float2 c = cnt[lane];
  const float m0 = rec[0].x;
  Share r;
  r.m = m0 + warp_sum(fmaf(c.x, q.x - m0, c.y)) / (float)C;
  const float d = q.x - r.m;
  r.m2 = not_below_0(warp_sum(about_mean(q.y, c.y, c.x, d)));
  r.a = warp_sum(q.z);
  r.ax = warp_sum(q.w + d * q.z);
  r.r = 0.f;
  return r;
}

// Rows too long for registers: one CTA per row, three walks over the row.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) k_norm_fwd_long(
    int64_t C, float eps, const T* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ b, T* __restrict__ y, int* status) {
  constexpr int N = Vec<T>::N;
  __shared__ float4 rec[32];
  __shared__ float2 num[32];
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
  Share sh = {};
  const float n = warp_sum((float)cnt);
  sh.m = warp_sum(sum) * inv_or_0(n);
  float m2 = 0.f, left = 0.f;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(xr + k * N, v);
    float q = 0.f, l = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = v[e] - sh.m;
      q = fmaf(d, d, q);
      l += d;
    }
    m2 += q;
    left += l;
  }
  sh.m2 = warp_sum(m2);
  sh.r = warp_sum(left);
  sh = join_shares(n, sh, rec, num, C);
  const float s = rsqrtf(sh.m2 / (float)C + eps);
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
// Persistent CTAs: each takes pairs of rows in a fixed stride and keeps its
// threads' channels of grad_weight and grad_bias in registers; one partial row
// pair [2][C] per CTA, summed in CTA order by k_norm_fin.  Two rows at a time
// share the loads of the weight and half the shuffles (one half-warp reduces
// each) and fill one row's waits with the other's work.  x and grad_y come
// through a ring of two row pairs in shared memory (cp.async: a thread copies
// what it later reads itself, so no barrier is needed).  WARP: a pair of rows per
// warp, the warps' sums joined in warp order through the ring's memory.

template <typename T, int VPT, bool WARP, int MAXT, int PERSM>
__global__ void __launch_bounds__(MAXT, PERSM)
    k_norm_bwd(int64_t rows, int64_t C, float eps, const T* __restrict__ x,
               const float* __restrict__ w, const T* __restrict__ gy, T* __restrict__ gx,
               float* __restrict__ part, int* status) {
  constexpr int N = Vec<T>::N, P = Pairs<T>::P;
  constexpr bool F32 = sizeof(T) == 4;
  using PV = Pairs<T>;
  constexpr int W = WARP ? 1 : MAXT / 32;
  __shared__ float4 rec[WARP ? 1 : 2][2][W];
  __shared__ float res[WARP ? 1 : 2][2][W];
  extern __shared__ uint4 ring[];  // [group][2][row][x, gy][nvec]; WARP, at the end: [2][C]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? lane : threadIdx.x;
  const int per = WARP ? blockDim.x / 32 : 1, g = WARP ? warp : 0;
  const int nvec = (int)(C / N);
  uint4* mine = ring + (int64_t)g * 8 * nvec;
  const int64_t row0 = 2 * ((int64_t)blockIdx.x * per + g), step = 2 * (int64_t)gridDim.x * per;
  const float inv_c = 1.0f / (float)C;
  // this warp's channels, and those of the warp whose record this lane joins
  const float n = WARP ? (float)C : share_channels(warp, tpr, N, nvec), inv_n = inv_or_0(n);
  const float nq =
      WARP || (lane & 15) >= tpr / 32 ? 0.f : share_channels(lane & 15, tpr, N, nvec);
  tc::grid_release();
  tc::grid_wait();
  auto fetch = [&](int64_t row, int slot) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (row + r < rows) {
        uint4* d = mine + (slot * 4 + 2 * r) * nvec;
        const uint4* xr = reinterpret_cast<const uint4*>(x + (row + r) * C);
        const uint4* gr = reinterpret_cast<const uint4*>(gy + (row + r) * C);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int k = t + i * tpr;
          if (k < nvec) {
            cp16(d + k, xr + k);
            cp16(d + nvec + k, gr + k);
          }
        }
      }
    }
    cp_commit();
  };
  uint64_t gw[VPT][P], gb[VPT][P];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) gw[i][e] = gb[i][e] = 0;
  fetch(row0, 0);
  int it = 0;
  for (int64_t row = row0; row < rows; row += step, ++it) {
    const int slot = it & 1;
    fetch(row + step, slot ^ 1);
    cp_wait<1>();
    const bool two = row + 1 < rows;
    // without a second row the first one is worked on twice, and counted once
    const uint4* xs[2] = {mine + slot * 4 * nvec, mine + (slot * 4 + (two ? 2 : 0)) * nvec};
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 q = xs[r][k];
#pragma unroll
          for (int e = 0; e < P; ++e) sum[r] = f2add(sum[r], PV::get(q, e));
        }
      }
    }
    // from here to the join a lane's scalars are its half-warp's row's
    const float all = pair_sum(f2sum(sum[0]), f2sum(sum[1]), lane), mw = all * inv_n;
    uint64_t nm[2] = {f2dup(-__shfl_sync(0xffffffffu, mw, 0)),
                      f2dup(-__shfl_sync(0xffffffffu, mw, 16))};
    uint64_t m2[2] = {0, 0}, sa[2] = {0, 0}, sax[2] = {0, 0}, left[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        uint64_t wv[P];
        load_param<P>(w + k * N, wv);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 q = xs[r][k], h = xs[r][nvec + k];
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const uint64_t d = f2add(PV::get(q, e), nm[r]), a = f2mul(PV::get(h, e), wv[e]);
            m2[r] = f2fma(d, d, m2[r]);
            sa[r] = f2add(sa[r], a);
            sax[r] = f2fma(a, d, sax[r]);
            if (F32) left[r] = f2add(left[r], d);
          }
        }
      }
    }
    float v2 = pair_sum(f2sum(m2[0]), f2sum(m2[1]), lane);
    float va = pair_sum(f2sum(sa[0]), f2sum(sa[1]), lane);
    float vx = pair_sum(f2sum(sax[0]), f2sum(sax[1]), lane), m;
    const float rw =
        F32 ? pair_sum(f2sum(left[0]), f2sum(left[1]), lane) : fmaf(-n, mw, all);
    if (WARP) {
      m = fmaf(rw, inv_c, mw);
      const float d = mw - m;
      v2 = about_mean(v2, rw, n, d);
      vx = fmaf(d, va, vx);
    } else {
      if ((lane & 15) == 0) {
        rec[it & 1][lane >> 4][warp] = make_float4(mw, v2, va, vx);
        res[it & 1][lane >> 4][warp] = rw;
      }
      __syncthreads();
      const float4* recs = rec[it & 1][lane >> 4];
      const float4 q = nq > 0.f ? recs[lane & 15] : make_float4(0, 0, 0, 0);
      const float qr = nq > 0.f ? res[it & 1][lane >> 4][lane & 15] : 0.f, m0 = recs[0].x;
      m = fmaf(half_sum(fmaf(nq, q.x - m0, qr)), inv_c, m0);
      const float d = q.x - m;
      v2 = half_sum(about_mean(q.y, qr, nq, d));
      va = half_sum(q.z);
      vx = half_sum(q.w + d * q.z);
    }
    const float s = rsqrtf(not_below_0(v2) * inv_c + eps);
    if (t == 0 || (t == 16 && two)) report(m, s, status);
    const float k1 = -va * inv_c, k2 = -vx * s * inv_c;
    uint64_t ss[2], c1[2], c2[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      nm[r] = f2dup(-__shfl_sync(0xffffffffu, m, 16 * r));
      ss[r] = f2dup(__shfl_sync(0xffffffffu, s, 16 * r));
      c1[r] = f2dup(__shfl_sync(0xffffffffu, k1, 16 * r));
      c2[r] = f2dup(__shfl_sync(0xffffffffu, k2, 16 * r));
    }
    uint4* gr = reinterpret_cast<uint4*>(gx + row * C);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = t + i * tpr;
      if (k < nvec) {
        uint64_t wv[P];
        load_param<P>(w + k * N, wv);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (r == 0 || two) {
            const uint4 q = xs[r][k], h = xs[r][nvec + k];
            uint64_t o[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const uint64_t gv = PV::get(h, e), xh = f2mul(f2add(PV::get(q, e), nm[r]), ss[r]);
              o[e] = f2mul(f2fma(xh, c2[r], f2fma(gv, wv[e], c1[r])), ss[r]);
              gw[i][e] = f2fma(gv, xh, gw[i][e]);
              gb[i][e] = f2add(gb[i][e], gv);
            }
            __stcs(gr + r * nvec + k, PV::pack(o));
          }
        }
      }
    }
  }
  float* sums = WARP ? reinterpret_cast<float*>(ring) : part + (int64_t)blockIdx.x * 2 * C;
  cp_wait<0>();
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
  __shared__ float4 rec[32];
  __shared__ float2 num[32];
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
  Share sh = {};
  const float n = warp_sum((float)cnt);
  sh.m = warp_sum(sum) * inv_or_0(n);
  float m2 = 0.f, sa = 0.f, sax = 0.f, left = 0.f;
  for (int64_t k = threadIdx.x; k < nvec; k += blockDim.x) {
    Vec<T>::load(x + row * C + k * N, xv);
    Vec<T>::load(gy + row * C + k * N, gv);
    float q2 = 0.f, qa = 0.f, qx = 0.f, l = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = xv[e] - sh.m, a = gv[e] * __ldg(w + k * N + e);
      q2 = fmaf(d, d, q2);
      qa += a;
      qx = fmaf(a, d, qx);
      l += d;
    }
    m2 += q2;
    sa += qa;
    sax += qx;
    left += l;
  }
  sh.m2 = warp_sum(m2);
  sh.r = warp_sum(left);
  sh.a = warp_sum(sa);
  sh.ax = warp_sum(sax);
  sh = join_shares(n, sh, rec, num, C);
  const float s = rsqrtf(sh.m2 / (float)C + eps);
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

// Partial rows of grad_weight and grad_bias: at most one per pair of rows and
// kMaxParts; kLongParts where a row's x and gy, more than kLongRow bytes, are walked
// in memory.
constexpr int64_t kMaxParts = 592, kLongParts = 64, kLongRow = 56 * 1024;
int64_t most_parts(int64_t rows, int64_t row_bytes) {
  return row_bytes > kLongRow ? std::min(rows, kLongParts) : std::min((rows + 1) / 2, kMaxParts);
}

// CTAs of `threads` threads and `smem` bytes that an SM holds, at 128 registers a
// thread (2 KB of shared memory beside: 1 KB for the records of 8 warps, 1 KB of the
// system's), and at most `most`.
int resident(int threads, size_t smem, int most) {
  const int by_regs = 512 / threads, by_smem = (int)(233472 / (smem + 2048));
  return std::max(1, std::min(most, std::min(by_regs, by_smem)));
}

template <int VPT, bool WARP, int MAXT, int PERSM>
cudaError_t fwd_pairs(int64_t rows, int64_t C, float eps, const __nv_bfloat16* x, const float* w,
                      const float* b, __nv_bfloat16* y, int threads, int* st, cudaStream_t s) {
  const int per = WARP ? threads / 32 : 1;
  const size_t sm = (size_t)per * 4 * C * 2;
  const int64_t groups = (rows + 2 * per - 1) / (2 * per);
  const int64_t g = (int64_t)sm_count() * resident(threads, sm, 8);
  auto kern = k_norm_fwd_pairs<VPT, WARP, MAXT, PERSM>;
  cudaError_t e = allow_smem(kern, 4 * MAXT * VPT * 16);
  if (e != cudaSuccess) return e;
  return launch_after(kern, (unsigned)(groups < g ? groups : g), (unsigned)threads, sm, 1, s, rows,
                      C, eps, x, w, b, y, st);
}

template <typename T>
cudaError_t fwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const float* b,
                T* y, int* st, cudaStream_t s) {
  const int64_t nvec = C / Vec<T>::N;
  // fp32 rows have half the arithmetic per byte and run faster one to a CTA (T =
  // 8192, C = 4096: 49 us against 61)
  if constexpr (sizeof(T) == 2) {
    if (rows >= 16 * sm_count()) {
      const int threads = round32((nvec + 3) / 4);  // four vectors, 32 channels, to a thread
      if (C > 512 && C <= 1024)
        return fwd_pairs<4, true, 128, 4>(rows, C, eps, x, w, b, y, 128, st, s);
      if (C > 1024 && C <= 8192)
        return fwd_pairs<4, false, 256, 2>(rows, C, eps, x, w, b, y, threads, st, s);
    }
  }
  if (nvec > 8 * 512) {
    k_norm_fwd_long<T><<<(unsigned)rows, kMaxThreads, 0, s>>>(C, eps, x, w, b, y, st);
    return cudaGetLastError();
  }
  if (nvec <= 8 * 32) {
    const unsigned grid = (unsigned)((rows + 3) / 4);
    auto kern = nvec <= 32    ? k_norm_fwd<T, 1, true, 128>
                : nvec <= 64  ? k_norm_fwd<T, 2, true, 128>
                : nvec <= 128 ? k_norm_fwd<T, 4, true, 128>
                              : k_norm_fwd<T, 8, true, 128>;
    return launch_after(kern, grid, 128, 0, 1, s, rows, C, eps, x, w, b, y, st);
  }
  auto kern = nvec <= 8 * 256 ? k_norm_fwd<T, 8, false, 256> : k_norm_fwd<T, 8, false, 512>;
  return launch_after(kern, (unsigned)rows, round32((nvec + 7) / 8), 0, 1, s, rows, C, eps, x, w, b,
                      y, st);
}

template <typename T, int VPT, bool WARP, int MAXT, int PERSM>
cudaError_t bwd_rows(int64_t rows, int64_t C, float eps, const T* x, const float* w, const T* gy,
                     T* gx, float* part, int threads, int* nparts, int* st, cudaStream_t s) {
  const int per = WARP ? threads / 32 : 1;
  const size_t ring = (size_t)per * 8 * C * sizeof(T);
  const size_t sum = WARP ? (size_t)2 * C * 4 : 0, sm = ring > sum ? ring : sum;
  const int64_t groups = (rows + 2 * per - 1) / (2 * per);
  const int64_t g = std::min<int64_t>(kMaxParts, (int64_t)sm_count() * resident(threads, sm, 4));
  *nparts = (int)(groups < g ? groups : g);  // at most most_parts()
  auto kern = k_norm_bwd<T, VPT, WARP, MAXT, PERSM>;
  cudaError_t e = allow_smem(kern, std::min<size_t>(8 * MAXT * VPT * 16, 4 * kLongRow));
  if (e != cudaSuccess) return e;
  return launch_after(kern, (unsigned)*nparts, (unsigned)threads, sm, 1, s, rows, C, eps, x, w, gy,
                      gx, part, st);
}

// Rows of up to 1024 channels on one warp; longer ones on a CTA, four vectors per
// thread (32 channels in bf16, 16 in fp32, whose rows leave shared memory for fewer
// CTAs), up to 14336 channels in bf16 and 7168 in fp32; what is longer does not fit
// the ring.
template <typename T>
cudaError_t bwd(int64_t rows, int64_t C, float eps, const T* x, const float* w, const T* gy, T* gx,
                float* gw, float* gb, void* ws, int* st, cudaStream_t s) {
  constexpr int V = 32 / Vec<T>::N;  // vectors of a lane at 1024 channels
  const int64_t nvec = C / Vec<T>::N, row = 2 * C * (int64_t)sizeof(T);  // x and gy
  float* part = (float*)ws;
  int nparts = 0;
  cudaError_t e;
  const int threads = round32((nvec + 3) / 4);
  if (row > kLongRow) {
    nparts = (int)most_parts(rows, row);
    float2* stat = (float2*)(part + (int64_t)nparts * 2 * C);
    k_norm_bwd_long<T><<<(unsigned)rows, kMaxThreads, 0, s>>>(C, eps, x, w, gy, gx, stat, st);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((nvec + 255) / 256), (unsigned)nparts);
    k_norm_bwd_cols<T><<<grid, 256, 0, s>>>(rows, C, x, gy, stat, part);
    e = cudaGetLastError();
  } else if (C <= 256) {
    e = bwd_rows<T, V / 4, true, 256, 2>(rows, C, eps, x, w, gy, gx, part, 256, &nparts, st, s);
  } else if (C <= 512) {
    e = bwd_rows<T, V / 2, true, 128, 3>(rows, C, eps, x, w, gy, gx, part, 128, &nparts, st, s);
  } else if (C <= 1024) {
    e = bwd_rows<T, V, true, 96, 2>(rows, C, eps, x, w, gy, gx, part, 96, &nparts, st, s);
  } else if (threads <= 256) {
    e = bwd_rows<T, 4, false, 256, 2>(rows, C, eps, x, w, gy, gx, part, threads, &nparts, st, s);
  } else {
    e = bwd_rows<T, 4, false, 512, 1>(rows, C, eps, x, w, gy, gx, part, threads, &nparts, st, s);
  }
  if (e != cudaSuccess) return e;
  const int64_t cols = 2 * C / 4;
  return launch_after(k_norm_fin, (unsigned)((cols + kFinCols - 1) / kFinCols),
                      kFinCols * kFinSlices, 0, 1, s, C, nparts, (const float*)part, gw, gb);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C, int dtype) {
  const int64_t row = 2 * C * (dtype == MHC_DTYPE_BF16 ? 2 : 4);
  return (size_t)most_parts(rows, row) * 2 * C * 4 +
         (row > kLongRow ? (size_t)rows * sizeof(float2) : 0);
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
