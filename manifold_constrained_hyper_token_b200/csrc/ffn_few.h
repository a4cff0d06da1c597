// ffn_few.h -- the feed-forward products of few tokens: bf16 in k_ffn_few.cu, fp32
// in k_ffn_one32.cu (up to 8) and k_ffn_few32.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mhc {

// Into how many parts (a cluster's CTAs) a sum of nk blocks of k is split, for `tiles`
// row tiles and per_sm CTAs per SM; at least `least` parts.  A wave of CTAs takes
// block_ns per block and what HBM needs to deliver one to each of them (2.5 ns per 16
// KB of weights), and fixed_ns for its start and end.  kClusters: clusters of 1 to 8
// CTAs that the machine holds at a time with one or two CTAs to an SM, a little below
// what an empty one does (a cluster stays in one group of SMs, so that clusters of 8
// leave 28 of 148 SMs idle, and a wave that filled the machine to the last place often
// took two: T = 130, C = 7168, F = 14336 bf16, 159 us against 136).
inline int split_sum(int64_t tiles, int64_t nk, int per_sm, int least, int tiles_16k,
                     int64_t block_ns, int64_t fixed_ns) {
  static constexpr int kClusters[2][8] = {{148, 74, 43, 32, 25, 21, 14, 14},
                                          {296, 148, 89, 68, 53, 43, 35, 32}};
  int parts = 0;
  int64_t best = 0;
  for (int p = least; p <= 8 && (p <= nk || p == least); ++p) {
    const int64_t cl = kClusters[per_sm - 1][p - 1], blocks = (nk + p - 1) / p;
    auto wave = [&](int64_t clusters) {
      const int64_t hbm = clusters * p * tiles_16k * 5 / 2;
      return clusters ? blocks * (block_ns + hbm) + fixed_ns : 0;
    };
    const int64_t cost = tiles / cl * wave(cl) + wave(tiles % cl);
    if (parts == 0 || cost < best) {
      best = cost;
      parts = p;
    }
  }
  return parts;
}

// bf16 sums longer than this do not stay in one accumulator (plan in k_ffn_tc.cu has the
// reason).
constexpr int64_t kLongSum = 65536;

// Up to this many tokens the weights are the tall operand of the products.
constexpr int64_t kFewTokens = 256;

struct FewArgs {
  int64_t t, C, F;
  int act;
  const void *x, *wg, *wu, *wd, *gy;
  int* st;
  int64_t wait_ns;
};

// a = act(x wg^T) * (x wu^T) [t][F], and g, u [t][F] unless g is null
cudaError_t few_gate(const FewArgs& f, void* a, float* g, float* u, cudaStream_t s);
// y = a wd^T [t][C]
cudaError_t few_down(const FewArgs& f, const void* a, void* y, cudaStream_t s);
// d = (dg, du) [2][t][F] from da = gy wd and g, u
cudaError_t few_dgate(const FewArgs& f, const float* g, const float* u, void* d, cudaStream_t s);
// gx = dg wg + du wu [t][C]
cudaError_t few_grad_x(const FewArgs& f, const void* d, void* gx, cudaStream_t s);

// k_ffn_few32.cu: the same in fp32, up to this many tokens.  x, gy, a and d are
// operands in three bf16 planes each ([3][t][..], d [6][t][F]); the weights are
// the caller's.
constexpr int64_t kFewTokens32 = 128;
bool few32_fits(int64_t t, int64_t C, int64_t F);
cudaError_t few32_gate(const FewArgs& f, void* a, float* g, float* u, cudaStream_t s);
cudaError_t few32_down(const FewArgs& f, const void* a, float* y, cudaStream_t s);
cudaError_t few32_dgate(const FewArgs& f, const float* g, const float* u, void* d, cudaStream_t s);
cudaError_t few32_grad_x(const FewArgs& f, const void* d, float* gx, cudaStream_t s);

// k_ffn_one32.cu: the same on the CUDA cores, up to this many tokens, from the
// caller's fp32 arrays; the planes of a and of dg, du are for the weight gradients
// (a or its planes may be null).
constexpr int64_t kOneTokens = 8;
cudaError_t one32_gate(const FewArgs& f, float* a, void* planes, float* g, float* u,
                       cudaStream_t s);
cudaError_t one32_down(const FewArgs& f, const float* a, float* y, cudaStream_t s);
cudaError_t one32_dgate(const FewArgs& f, const float* g, const float* u, float* d, void* planes,
                        cudaStream_t s);
cudaError_t one32_grad_x(const FewArgs& f, const float* d, float* gx, cudaStream_t s);

}  // namespace mhc
