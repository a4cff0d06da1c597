// ffn_few.h -- the feed-forward products of few tokens (bf16), k_ffn_few.cu.
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

}  // namespace mhc
