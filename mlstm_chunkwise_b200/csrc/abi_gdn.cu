// C entry points of the gated delta rule and of the cell-output layer norm:
// argument checks and dispatch.  Every check happens before the first launch.
#include <math.h>

#include "abi.h"
#include "gdn.h"
#include "gdn_tc.h"
#include "head_norm.h"

namespace mlstm {
namespace {

bool valid_dtype(mlstm_dtype dt) { return dt == MLSTM_DT_F32 || dt == MLSTM_DT_BF16; }

mlstm_status gdn_problem(int B, int NHK, int NH, int T, int DK, int DV, float scale,
                         GdnProblem* out) {
  if (B < 1 || NHK < 1 || NH < 1 || T < 0 || DK < 1 || DV < 1) return MLSTM_ERR_INVALID_ARG;
  if (NH % NHK != 0 || !isfinite(scale)) return MLSTM_ERR_INVALID_ARG;
  if (DK > 1024 || DV > 1024 || T > (1 << 22) || (long long)B * NH > 65535)
    return MLSTM_ERR_UNSUPPORTED;
  GdnProblem p{};
  p.B = B;
  p.NHK = NHK;
  p.NH = NH;
  p.T = T;
  p.DK = DK;
  p.DV = DV;
  p.BH = B * NH;
  p.group = NH / NHK;
  p.scale = scale;
  p.max_polls = watchdog_polls();
  *out = p;
  return MLSTM_OK;
}

// Gradients of fewer head-tokens than this take the fp32 path: dg of a token is
// one sum over d_qk x d_v terms that may cancel to a hundredth of their size, and
// with a few tokens nothing averages that out (one token: 2.5e-5 of dg from the
// two-term operands, 4e-8 in fp32).  Costs 125 in place of 64 us at 4 tokens of 64
// x 64; from 64 head-tokens on the tensor cores' dg was within 7e-6.
constexpr long kFewHeadTokens = 64;

// Resolves AUTO and checks that the chosen algorithm takes the call.  The rule
// is one of type and sizes alone, so that the workspace size computed on the
// host always matches the algorithm a call picks.
mlstm_status gdn_algo(const GdnProblem& p, mlstm_dtype dt, mlstm_algo req, bool backward,
                      mlstm_algo* out) {
  if (!valid_dtype(dt)) return MLSTM_ERR_INVALID_ARG;
  const bool tc = dt == MLSTM_DT_BF16 && gdn_tc_supported(p);
  const bool few = backward && (long)p.BH * p.T < kFewHeadTokens;
  switch (req) {
    case MLSTM_ALGO_AUTO: *out = tc && !few ? MLSTM_ALGO_TC : MLSTM_ALGO_SIMT; return MLSTM_OK;
    case MLSTM_ALGO_SIMT: *out = req; return MLSTM_OK;
    case MLSTM_ALGO_TC: *out = req; return tc ? MLSTM_OK : MLSTM_ERR_UNSUPPORTED;
    case MLSTM_ALGO_TC_FUSED: return MLSTM_ERR_UNSUPPORTED;
  }
  return MLSTM_ERR_INVALID_ARG;
}

size_t gdn_workspace(const GdnProblem& p, mlstm_algo a, bool backward) {
  return a == MLSTM_ALGO_TC ? gdn_tc_workspace(p, backward) : gdn_simt_workspace(p, backward);
}

// Sizes of the training pair, where AUTO would take the tensor cores for the
// gradients.
mlstm_status gdn_train(const GdnProblem& p, mlstm_dtype dt, GdnTrainSizes* z) {
  mlstm_algo a;
  const mlstm_status s = gdn_algo(p, dt, MLSTM_ALGO_AUTO, true, &a);
  if (s != MLSTM_OK) return s;
  if (a != MLSTM_ALGO_TC) return MLSTM_ERR_UNSUPPORTED;
  *z = gdn_tc_train_sizes(p);
  return MLSTM_OK;
}

// dst = src, or zero without one.
mlstm_status copy_or_zero(float* dst, const float* src, size_t n, cudaStream_t st) {
  if (!dst || dst == src) return MLSTM_OK;
  const cudaError_t e =
      src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, st)
          : cudaMemsetAsync(dst, 0, n * sizeof(float), st);
  return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
}

mlstm_status norm_problem(int B, int NH, int T, int D, float eps, mlstm_dtype dt,
                          HeadNormProblem* out) {
  if (!valid_dtype(dt)) return MLSTM_ERR_INVALID_ARG;
  if (B < 1 || NH < 1 || T < 0 || D < 1 || !(eps >= 0.f) || !isfinite(eps))
    return MLSTM_ERR_INVALID_ARG;
  if (D > kHeadNormMaxD || T > (1 << 22) || (long long)B * NH > 65535)
    return MLSTM_ERR_UNSUPPORTED;
  *out = HeadNormProblem{B, NH, T, D, eps, nullptr};
#ifdef MLSTM_DEBUG_BOUNDS
  out->err = device_error_word();
#endif
  return MLSTM_OK;
}

template <size_t N>
bool all_aligned(unsigned n, const void* const (&ptrs)[N]) {
  for (const void* q : ptrs)
    if (!is_aligned(q, n)) return false;
  return true;
}

}  // namespace
}  // namespace mlstm

using namespace mlstm;

extern "C" {

mlstm_status mlstm_gated_delta_workspace_size(int B, int NHK, int NH, int T, int DK, int DV,
                                              mlstm_dtype dtype, mlstm_algo algo, int backward,
                                              size_t* bytes) {
  if (!bytes) return MLSTM_ERR_INVALID_ARG;
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, 1.f, &p);
  if (s != MLSTM_OK) return s;
  mlstm_algo a;
  s = gdn_algo(p, dtype, algo, backward != 0, &a);
  if (s != MLSTM_OK) return s;
  *bytes = gdn_workspace(p, a, backward != 0);
  return MLSTM_OK;
}

mlstm_status mlstm_gated_delta_fw(const void* Q, const void* K, const void* V, const float* g,
                                  const float* beta, const float* C0, void* H, float* C_T, int B,
                                  int NHK, int NH, int T, int DK, int DV, float scale,
                                  mlstm_dtype dtype, mlstm_algo algo, void* workspace,
                                  size_t workspace_bytes, mlstm_stream_t stream) {
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, scale, &p);
  if (s != MLSTM_OK) return s;
  mlstm_algo a;
  s = gdn_algo(p, dtype, algo, false, &a);
  if (s != MLSTM_OK) return s;
  if (T > 0 && (!Q || !K || !V || !g || !beta || !H)) return MLSTM_ERR_INVALID_ARG;
  if (!all_aligned(16, {Q, K, V, C0, H, C_T, workspace}) || !all_aligned(4, {g, beta}))
    return MLSTM_ERR_INVALID_ARG;
  const size_t need = gdn_workspace(p, a, false);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MLSTM_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return copy_or_zero(C_T, C0, (size_t)p.BH * DK * DV, st);
  p.err = device_error_word();
  if (!p.err) return MLSTM_ERR_CUDA;
  const GdnInputs x{Q, K, V, g, beta, C0};
  if (a == MLSTM_ALGO_TC)
    return run_family(MLSTM_KERNEL_GATED_DELTA_FW, gdn_tc_launches(p, false), st, [&] {
      return launch_gdn_tc_fw(p, x, H, C_T, workspace, st);
    });
  return run_family(MLSTM_KERNEL_GATED_DELTA_FW, gdn_simt_launches(p, false), st, [&] {
    return launch_gdn_simt_fw(p, dtype, x, H, C_T, workspace, st);
  });
}

mlstm_status mlstm_gated_delta_bw(const void* Q, const void* K, const void* V, const float* g,
                                  const float* beta, const float* C0, const void* dH,
                                  const float* dC_T, void* dQ, void* dK, void* dV, float* dg,
                                  float* dbeta, float* dC0, int B, int NHK, int NH, int T, int DK,
                                  int DV, float scale, mlstm_dtype dtype, mlstm_algo algo,
                                  void* workspace, size_t workspace_bytes, mlstm_stream_t stream) {
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, scale, &p);
  if (s != MLSTM_OK) return s;
  mlstm_algo a;
  s = gdn_algo(p, dtype, algo, true, &a);
  if (s != MLSTM_OK) return s;
  if (T > 0 && (!Q || !K || !V || !g || !beta || !dH || !dQ || !dK || !dV || !dg || !dbeta))
    return MLSTM_ERR_INVALID_ARG;
  if (!all_aligned(16, {Q, K, V, C0, dH, dC_T, dQ, dK, dV, dC0, workspace}) ||
      !all_aligned(4, {g, beta, dg, dbeta}))
    return MLSTM_ERR_INVALID_ARG;
  const size_t need = gdn_workspace(p, a, true);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MLSTM_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return copy_or_zero(dC0, dC_T, (size_t)p.BH * DK * DV, st);
  p.err = device_error_word();
  if (!p.err) return MLSTM_ERR_CUDA;
  const GdnInputs x{Q, K, V, g, beta, C0};
  const GdnGrads d{dH, dC_T, dQ, dK, dV, dg, dbeta, dC0};
  if (a == MLSTM_ALGO_TC)
    return run_family(MLSTM_KERNEL_GATED_DELTA_BW, gdn_tc_launches(p, true), st, [&] {
      return launch_gdn_tc_bw(p, x, d, workspace, st);
    });
  return run_family(MLSTM_KERNEL_GATED_DELTA_BW, gdn_simt_launches(p, true), st, [&] {
    return launch_gdn_simt_bw(p, dtype, x, d, workspace, st);
  });
}

mlstm_status mlstm_gated_delta_train_sizes(int B, int NHK, int NH, int T, int DK, int DV,
                                           mlstm_dtype dtype, size_t* saved_bytes,
                                           size_t* fw_workspace_bytes,
                                           size_t* bw_workspace_bytes) {
  if (!saved_bytes || !fw_workspace_bytes || !bw_workspace_bytes) return MLSTM_ERR_INVALID_ARG;
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, 1.f, &p);
  if (s != MLSTM_OK) return s;
  GdnTrainSizes z;
  s = gdn_train(p, dtype, &z);
  if (s != MLSTM_OK) return s;
  *saved_bytes = z.saved;
  *fw_workspace_bytes = z.fw;
  *bw_workspace_bytes = z.bw;
  return MLSTM_OK;
}

mlstm_status mlstm_gated_delta_fw_train(const void* Q, const void* K, const void* V,
                                        const float* g, const float* beta, const float* C0,
                                        void* H, float* C_T, void* saved, size_t saved_bytes,
                                        int B, int NHK, int NH, int T, int DK, int DV, float scale,
                                        mlstm_dtype dtype, void* workspace, size_t workspace_bytes,
                                        mlstm_stream_t stream) {
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, scale, &p);
  if (s != MLSTM_OK) return s;
  GdnTrainSizes z;
  s = gdn_train(p, dtype, &z);
  if (s != MLSTM_OK) return s;
  if (!Q || !K || !V || !g || !beta || !H || !saved || !workspace) return MLSTM_ERR_INVALID_ARG;
  if (!all_aligned(16, {Q, K, V, C0, H, C_T, saved, workspace}) || !all_aligned(4, {g, beta}))
    return MLSTM_ERR_INVALID_ARG;
  if (saved_bytes < z.saved || workspace_bytes < z.fw) return MLSTM_ERR_INVALID_ARG;
  p.err = device_error_word();
  if (!p.err) return MLSTM_ERR_CUDA;
  const GdnInputs x{Q, K, V, g, beta, C0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return run_family(MLSTM_KERNEL_GATED_DELTA_FW, gdn_tc_train_launches(p, false), st, [&] {
    return launch_gdn_tc_fw_train(p, x, H, C_T, saved, workspace, st);
  });
}

mlstm_status mlstm_gated_delta_bw_saved(const void* Q, const void* K, const void* V,
                                        const float* g, const float* beta, const void* saved,
                                        size_t saved_bytes, const void* dH, const float* dC_T,
                                        void* dQ, void* dK, void* dV, float* dg, float* dbeta,
                                        float* dC0, int B, int NHK, int NH, int T, int DK, int DV,
                                        float scale, mlstm_dtype dtype, void* workspace,
                                        size_t workspace_bytes, mlstm_stream_t stream) {
  GdnProblem p;
  mlstm_status s = gdn_problem(B, NHK, NH, T, DK, DV, scale, &p);
  if (s != MLSTM_OK) return s;
  GdnTrainSizes z;
  s = gdn_train(p, dtype, &z);
  if (s != MLSTM_OK) return s;
  if (!Q || !K || !V || !g || !beta || !saved || !dH || !dQ || !dK || !dV || !dg || !dbeta ||
      !workspace)
    return MLSTM_ERR_INVALID_ARG;
  if (!all_aligned(16, {Q, K, V, saved, dH, dC_T, dQ, dK, dV, dC0, workspace}) ||
      !all_aligned(4, {g, beta, dg, dbeta}))
    return MLSTM_ERR_INVALID_ARG;
  if (saved_bytes < z.saved || workspace_bytes < z.bw) return MLSTM_ERR_INVALID_ARG;
  p.err = device_error_word();
  if (!p.err) return MLSTM_ERR_CUDA;
  const GdnInputs x{Q, K, V, g, beta, nullptr};
  const GdnGrads d{dH, dC_T, dQ, dK, dV, dg, dbeta, dC0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return run_family(MLSTM_KERNEL_GATED_DELTA_BW, gdn_tc_train_launches(p, true), st, [&] {
    return launch_gdn_tc_bw_saved(p, x, d, saved, workspace, st);
  });
}

mlstm_status mlstm_gated_delta_step(const void* q, const void* k, const void* v, const float* g,
                                    const float* beta, float* C, void* h, int B, int NHK, int NH,
                                    int DK, int DV, float scale, mlstm_dtype dtype,
                                    mlstm_stream_t stream) {
  GdnProblem p;
  const mlstm_status s = gdn_problem(B, NHK, NH, 1, DK, DV, scale, &p);
  if (s != MLSTM_OK) return s;
  if (!valid_dtype(dtype) || !q || !k || !v || !g || !beta || !C || !h)
    return MLSTM_ERR_INVALID_ARG;
  // single elements are read, except of the state: one head's token of a longer
  // tensor need not start on a 16-byte boundary
  if (!all_aligned(dtype == MLSTM_DT_BF16 ? 2 : 4, {q, k, v, h}) || !all_aligned(4, {g, beta}) ||
      !all_aligned(16, {C}))
    return MLSTM_ERR_INVALID_ARG;
#ifdef MLSTM_DEBUG_BOUNDS
  p.err = device_error_word();
#endif
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return run_family(MLSTM_KERNEL_GATED_DELTA_STEP, 1, st, [&] {
    return launch_gdn_step(p, dtype, q, k, v, g, beta, C, h, st);
  });
}

mlstm_status mlstm_head_norm_fw(const void* X, const float* weight, const float* bias, void* Y,
                                float* mean, float* rstd, int B, int NH, int T, int D, float eps,
                                mlstm_dtype dtype, mlstm_stream_t stream) {
  HeadNormProblem p;
  const mlstm_status s = norm_problem(B, NH, T, D, eps, dtype, &p);
  if (s != MLSTM_OK) return s;
  if (!weight || (T > 0 && (!X || !Y)) || !all_aligned(16, {X, weight, bias, Y, mean, rstd}))
    return MLSTM_ERR_INVALID_ARG;
  if (T == 0) return MLSTM_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return run_family(MLSTM_KERNEL_HEAD_NORM_FW, 1, st, [&] {
    return launch_head_norm_fw(p, dtype, X, weight, bias, Y, mean, rstd, st);
  });
}

mlstm_status mlstm_head_norm_bw_workspace_size(int B, int NH, int T, int D, mlstm_dtype dtype,
                                               size_t* bytes) {
  HeadNormProblem p;
  const mlstm_status s = norm_problem(B, NH, T, D, 0.f, dtype, &p);
  if (s != MLSTM_OK || !bytes) return s != MLSTM_OK ? s : MLSTM_ERR_INVALID_ARG;
  *bytes = head_norm_bw_workspace(p, dtype);
  return MLSTM_OK;
}

mlstm_status mlstm_head_norm_bw(const void* X, const void* dY, const float* weight,
                                const float* mean, const float* rstd, void* dX, float* dweight,
                                float* dbias, int B, int NH, int T, int D, mlstm_dtype dtype,
                                void* workspace, size_t workspace_bytes, mlstm_stream_t stream) {
  HeadNormProblem p;
  const mlstm_status s = norm_problem(B, NH, T, D, 0.f, dtype, &p);
  if (s != MLSTM_OK) return s;
  if (!weight || !dweight || (T > 0 && (!X || !dY || !mean || !rstd || !dX)))
    return MLSTM_ERR_INVALID_ARG;
  if (!all_aligned(16, {X, dY, weight, mean, rstd, dX, dweight, dbias, workspace}))
    return MLSTM_ERR_INVALID_ARG;
  if (workspace_bytes < head_norm_bw_workspace(p, dtype) || !workspace)
    return MLSTM_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return run_family(MLSTM_KERNEL_HEAD_NORM_BW, 2, st, [&] {
    return launch_head_norm_bw(p, dtype, X, dY, weight, mean, rstd, dX, dweight, dbias, workspace,
                               st);
  });
}

}  // extern "C"
