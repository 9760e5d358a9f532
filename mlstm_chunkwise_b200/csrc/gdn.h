// Gated delta rule: problem description, workspace pieces and launchers.
//
// For every (batch b, value head h), with a_t = e^{g_t}:
//   y_t  = v_t - a_t C_{t-1}^T k_t
//   C_t  = a_t C_{t-1} + k_t (beta_t y_t)^T             C: [DK][DV]
//   h_t  = scale C_t^T q_t
// Chunkwise, for a chunk of L tokens entered with the state S (gc: inclusive
// sum of g inside the chunk, G its value at the chunk's end; Lam = e^{gc},
// D = e^{G - gc}, Gam_rs = e^{gc_r - gc_s}):
//   A_rs = Gam_rs beta_s k_r.k_s (s < r),   Tinv = (I + A)^{-1}
//   y    = Tinv (V - Lam K S)
//   H    = scale (Lam Q S + P y),            P_rs = Gam_rs beta_s q_r.k_s (s <= r)
//   S'   = e^G S + K^T (D beta y)
// and, given dH and the gradient dS' of the exit state,
//   dy~  = scale (Gam . QK^T)^T dH + D K dS'      (the gradient of beta y)
//   dz   = Tinv^T (beta dy~),                dV = dz
//   dS   = e^G dS' + Q^T (scale Lam dH) - K^T (Lam dz)
//   Rh   = scale (dH y^T) . Gam (s <= r),    Eh = -(dz y^T) . Gam (s < r)
//   dQ   = scale Lam (dH S^T) + (Rh beta) K
//   dK   = -Lam (dz S^T) + (Eh beta) K + beta (D (y dS'^T) + Rh^T Q + Eh^T K)
//   out_s = D_s k_s.(y dS'^T)_s,             Z = Rh . QK^T + Eh . KK^T
//   dbeta_s = out_s + sum_r Z_rs
//   dg_t = sum_{r >= t} [scale Lam_r dH_r.(S^T q_r) - Lam_r dz_r.(S^T k_r)]
//          + sum_{s < t} beta_s out_s + e^G <S, dS'> + sum_{r >= t > s} Z_rs beta_s
// The row and the column sums of the last term come from the same fp32 values
// of Z, so that what cancels between them cancels exactly: with strong decay
// dg is orders of magnitude smaller than the sums it is the difference of.
//
// (I + A)^{-1} is formed by forward substitution and by blocks
// (-T22 A21 T11), never as a power series: with alike keys the powers of A
// grow like binomials while the inverse stays of order one.
#pragma once

#include "common.cuh"

namespace mlstm {

struct GdnProblem {
  int B, NHK, NH, T, DK, DV;
  int BH;       // B * NH
  int group;    // NH / NHK
  float scale;
  uint32_t* err;
  unsigned long long max_polls;
};

// Head of Q and K (in [B * NHK]) that value head bh reads.
__host__ __device__ __forceinline__ int gdn_key_head(const GdnProblem& p, int bh) {
  return (bh / p.NH) * p.NHK + (bh % p.NH) / p.group;
}

// g below this decays any state to zero in fp32; clamping it (and -inf) keeps
// differences of sums finite.  A comparison, not fmaxf(), which drops a NaN: a
// diverged gate must not pass for a reset.
constexpr float kGdnMinLogDecay = -1000.f;
__device__ __forceinline__ float gdn_log_decay(float g) {
  return g < kGdnMinLogDecay ? kGdnMinLogDecay : g;
}

struct GdnInputs {
  const void *Q, *K, *V;
  const float *g, *beta, *C0;
};
struct GdnGrads {
  const void* dH;
  const float* dC_T;
  void *dQ, *dK, *dV;
  float *dg, *dbeta, *dC0;
};

// fp32 CUDA-core path (gdn_simt.cu): any sizes, chunks of 64.
size_t gdn_simt_workspace(const GdnProblem& p, bool backward);
int gdn_simt_launches(const GdnProblem& p, bool backward);
cudaError_t launch_gdn_simt_fw(const GdnProblem& p, mlstm_dtype dt, const GdnInputs& x, void* H,
                               float* C_T, void* ws, cudaStream_t st);
cudaError_t launch_gdn_simt_bw(const GdnProblem& p, mlstm_dtype dt, const GdnInputs& x,
                               const GdnGrads& d, void* ws, cudaStream_t st);

// Sums the per-value-head gradients of Q and K (fp32 [B * NH, T, DK]) over the
// value heads that share a key head.
cudaError_t launch_gdn_group_sum(const GdnProblem& p, mlstm_dtype dt, const float* dq,
                                 const float* dk, void* dQ, void* dK, cudaStream_t st);

// Single-token step (gdn_step.cu).
cudaError_t launch_gdn_step(const GdnProblem& p, mlstm_dtype dt, const void* q, const void* k,
                            const void* v, const float* g, const float* beta, float* C, void* h,
                            cudaStream_t st);

}  // namespace mlstm
