// Shared pieces of the gated delta rule's tensor-core kernels (bf16 inputs,
// d_qk up to 128, chunks of 128 tokens; formulas in gdn.h).
//
// Precision.  Q, K, V and dH are exact bf16 operands.  Every other operand of a
// product (state, inverse, z, y, the gated score matrices, and their
// gradients) is an fp32 value carried as two bf16 terms, hi = bf16(x) and
// lo = bf16(x - hi), off by at most 2^-16 of its value; the product of two such
// operands drops only lo.lo.  So fp32 outputs (state, gate gradients) keep
// about 17 bits at two or three tensor-core products in place of one.  A single
// bf16 rounding of the state or of the inverse would put 2e-3 of noise on
// every output, and dg, a difference of large sums, off by percents.
#pragma once

#include "gdn.h"
#include "tc_ptx.cuh"

namespace mlstm {

constexpr int kGdnL = 128;  // chunk length of the tensor-core path

inline int gdn_tc_chunks(const GdnProblem& p) { return (p.T + kGdnL - 1) / kGdnL; }

bool gdn_tc_supported(const GdnProblem& p);
size_t gdn_tc_workspace(const GdnProblem& p, bool backward);
int gdn_tc_launches(const GdnProblem& p, bool backward);
cudaError_t launch_gdn_tc_fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                             void* ws, cudaStream_t st);
cudaError_t launch_gdn_tc_bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
                             cudaStream_t st);

// Workspace pieces, per (bh, chunk):
//   gc    float2[128]      inclusive sums of g inside the chunk (hi, lo)
//   tinv  uint4[32][128]   Tinv by rows as bf16 terms: piece j < 16 holds columns
//                          8j .. 8j + 7 of hi, j >= 16 those of lo; row r at [j][r],
//                          so that a warp of row threads reads 512 contiguous bytes.
//                          Pieces right of the diagonal's 32 x 32 block are not
//                          written (they are zero).
//   tinvt uint4[32][128]   the same of Tinv^T (backward); pieces left of the
//                          diagonal's block are not written
//   y, dz [value tile][2 terms][16 KB]   operand images: 128 token rows of 128
//                          bytes (64 value columns), 128-byte swizzle
//   S, dS [value tile][2 terms][16 KB]   operand images of the state entering and
//                          of the state gradient leaving the chunk: 128 d_qk rows
//                          of 128 bytes
struct GdnTcWs {
  float2* gc;
  uint4 *tinv, *tinvt;
  uint8_t *y, *dz, *S, *dS;
  float *dq, *dk;  // fp32 [BH][T][DK], with shared key heads
  int NC, nvt;     // chunks, value tiles of 64 columns
  size_t bytes;
};

namespace tc {

// The two bf16 terms of eight fp32 values.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
    l[e] = pack_bf16x2(x[2 * e] - __uint_as_float(h[e] << 16),
                       x[2 * e + 1] - __uint_as_float(h[e] & 0xffff0000u));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

constexpr uint32_t kGdnImage = 16384;  // bytes of one term of an operand image

// Eight values as 16-byte chunk c of row r of an operand image (both terms).
__device__ __forceinline__ void put8(uint8_t* img, int r, int c, const float* x) {
  uint4 hi, lo;
  split8(x, hi, lo);
  *reinterpret_cast<uint4*>(img + sw128_offset(r, c)) = hi;
  *reinterpret_cast<uint4*>(img + kGdnImage + sw128_offset(r, c)) = lo;
}

constexpr float kLog2e = 1.4426950408889634f;
// e^{a - b} of two sums of g held as (hi, lo).
__device__ __forceinline__ float gdn_decay(float2 a, float2 b) {
  return ex2_approx(((a.x - b.x) + (a.y - b.y)) * kLog2e);
}

}  // namespace tc
}  // namespace mlstm
