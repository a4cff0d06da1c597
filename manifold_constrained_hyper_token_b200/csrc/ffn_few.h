// ffn_few.h -- the feed-forward products of few tokens: bf16 in k_ffn_few.cu, fp32
// in k_ffn_one32.cu (up to 8) and k_ffn_few32.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mhc {

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
