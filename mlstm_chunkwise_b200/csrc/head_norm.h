// Layer norm of the cell output per (token, head), into token-major layout.
#pragma once

#include "common.cuh"

namespace mlstm {

struct HeadNormProblem {
  int B, NH, T, D;
  float eps;
  uint32_t* err;  // of the bounds-checked build (else nullptr)
};

constexpr int kHeadNormMaxD = 8192;

cudaError_t launch_head_norm_fw(const HeadNormProblem& p, mlstm_dtype dt, const void* X,
                                const float* weight, const float* bias, void* Y, float* mean,
                                float* rstd, cudaStream_t st);
size_t head_norm_bw_workspace(const HeadNormProblem& p, mlstm_dtype dt);
cudaError_t launch_head_norm_bw(const HeadNormProblem& p, mlstm_dtype dt, const void* X,
                                const void* dY, const float* weight, const float* mean,
                                const float* rstd, void* dX, float* dweight, float* dbias,
                                void* ws, cudaStream_t st);

}  // namespace mlstm
