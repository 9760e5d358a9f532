// Single-token step of the gated delta rule, in place on the fp32 state.
//
// With a = e^g and the old state C, both inner products of a column come out of
// one pass over it:
//   kc_j = sum_i k_i C_ij,  qc_j = sum_i q_i C_ij
//   vn_j = beta (v_j - a kc_j),  C'_ij = a C_ij + k_i vn_j
//   h_j  = scale (a qc_j + (q.k) vn_j)
// so the state is read once and written once: 8 d_qk d_v bytes per head against
// 6 d_qk d_v FLOPs, bound by HBM.  A CTA owns a (head, column tile): kTX lanes
// of four columns each side by side, kThreads / kTX row groups; a thread keeps
// its rows of the tile in registers between the reduction and the update (d_qk up
// to kRows row groups; larger states are read a second time).
//
// 1536 heads of 128 x 128 (201 MB moved): 40 us, 5.0 TB/s, 0.77 of the measured
// copy bandwidth.  Streaming loads and stores took it from 48 us, since a state
// read and written in place otherwise waits in L2 for its write-back.  Tiles of 32
// columns on 128 threads: 4.7 us for 16 heads against 6.2 with 64 columns on 256
// threads, the same for 1536; 512 threads a tile took twice as long (too few
// blocks to keep loads in flight while others reduce).
#include "gdn.h"

namespace mlstm {
namespace {

__device__ __forceinline__ float4 load_cols(const float* p, int left) {
  if (left >= 4) return __ldcs(reinterpret_cast<const float4*>(p));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (left > 0) v.x = p[0];
  if (left > 1) v.y = p[1];
  if (left > 2) v.z = p[2];
  return v;
}
__device__ __forceinline__ float4 load_unaligned(const float* p, int left) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (left > 0) v.x = p[0];
  if (left > 1) v.y = p[1];
  if (left > 2) v.z = p[2];
  if (left > 3) v.w = p[3];
  return v;
}
template <bool kVec>
__device__ __forceinline__ float4 load4(const float* p, int left) {
  return kVec ? load_cols(p, left) : load_unaligned(p, left);
}
template <bool kVec>
__device__ __forceinline__ void store4(float* p, int left, float4 v) {
  if (kVec) {
    if (left >= 4) __stcs(reinterpret_cast<float4*>(p), v);
  } else {
    if (left > 0) p[0] = v.x;
    if (left > 1) p[1] = v.y;
    if (left > 2) p[2] = v.z;
    if (left > 3) p[3] = v.w;
  }
}
__device__ __forceinline__ void fma4(float4& a, float s, float4 x) {
  a.x = fmaf(s, x.x, a.x);
  a.y = fmaf(s, x.y, a.y);
  a.z = fmaf(s, x.z, a.z);
  a.w = fmaf(s, x.w, a.w);
}

// kVec: DV is a multiple of 4 (every row starts on a 16-byte boundary and a
// lane's four columns are all inside or all outside).
template <typename T, int kThreads, int kTX, int kRows, bool kVec>
__global__ void __launch_bounds__(kThreads)
gdn_step_kernel(GdnProblem p, const T* __restrict__ q, const T* __restrict__ k,
                const T* __restrict__ v, const float* __restrict__ g,
                const float* __restrict__ beta, float* __restrict__ C, T* __restrict__ h) {
  constexpr int kTY = kThreads / kTX;
  extern __shared__ float sh[];
  float *sk = sh, *sq = sk + p.DK;
  float4* red = reinterpret_cast<float4*>(sq + p.DK + ((2 * p.DK) & 3 ? 4 - ((2 * p.DK) & 3) : 0));
  float* dots = reinterpret_cast<float*>(red + 2 * kTY * kTX);
  const int bh = blockIdx.y, tx = threadIdx.x % kTX, ty = threadIdx.x / kTX;
  const long kh = gdn_key_head(p, bh);
  const int col = (blockIdx.x * kTX + tx) * 4, left = p.DV - col;
  float* cp = C + (long)bh * p.DK * p.DV + col;

  float4 c[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = ty + i * kTY;
    c[i] = r < p.DK ? load4<kVec>(cp + (long)r * p.DV, left) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float a = expf(gdn_log_decay(g[bh])), b = beta[bh];
  float kq = 0.f;
  for (int i = threadIdx.x; i < p.DK; i += kThreads) {
    const float kk = to_float(k[kh * p.DK + i]), qq = to_float(q[kh * p.DK + i]);
    sk[i] = kk;
    sq[i] = qq;
    kq = fmaf(kk, qq, kq);
  }
  kq = warp_sum(kq);
  if ((threadIdx.x & 31) == 0) dots[threadIdx.x >> 5] = kq;
  __syncthreads();
  float4 kc = make_float4(0.f, 0.f, 0.f, 0.f), qc = kc;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = ty + i * kTY;
    if (r < p.DK) {
      fma4(kc, sk[r], c[i]);
      fma4(qc, sq[r], c[i]);
    }
  }
  for (int r = ty + kRows * kTY; r < p.DK; r += kTY) {
    const float4 x = load4<kVec>(cp + (long)r * p.DV, left);
    fma4(kc, sk[r], x);
    fma4(qc, sq[r], x);
  }
  red[ty * kTX + tx] = kc;
  red[(kTY + ty) * kTX + tx] = qc;
  __syncthreads();
  kc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kTY; ++i) fma4(kc, 1.f, red[i * kTX + tx]);
  // forgotten entirely, whatever it held: 0 times an infinity is a NaN
  const bool gone = a == 0.f;
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  if (gone) {
    kc = none;
#pragma unroll
    for (int i = 0; i < kRows; ++i) c[i] = none;
  }
  float4 vn;
  {
    const long vb = (long)bh * p.DV + col;
    vn.x = left > 0 ? b * (to_float(v[vb]) - a * kc.x) : 0.f;
    vn.y = left > 1 ? b * (to_float(v[vb + 1]) - a * kc.y) : 0.f;
    vn.z = left > 2 ? b * (to_float(v[vb + 2]) - a * kc.z) : 0.f;
    vn.w = left > 3 ? b * (to_float(v[vb + 3]) - a * kc.w) : 0.f;
  }
  auto put = [&](int r, float4 x) {
    float4 y = make_float4(a * x.x, a * x.y, a * x.z, a * x.w);
    fma4(y, sk[r], vn);
    if (MLSTM_IN_BOUNDS(p, bh < p.BH && r < p.DK && (!kVec || left <= 0 || left >= 4)))
      store4<kVec>(cp + (long)r * p.DV, left, y);
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (ty + i * kTY < p.DK) put(ty + i * kTY, c[i]);
  for (int r = ty + kRows * kTY; r < p.DK; r += kTY)
    put(r, gone ? none : load4<kVec>(cp + (long)r * p.DV, left));
  if (ty == 0) {
    qc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kTY; ++i) fma4(qc, 1.f, red[(kTY + i) * kTX + tx]);
    if (gone) qc = none;
    kq = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) kq += dots[i];
    T* hp = h + (long)bh * p.DV + col;
    if (left > 0) hp[0] = from_float<T>(p.scale * fmaf(a, qc.x, kq * vn.x));
    if (left > 1) hp[1] = from_float<T>(p.scale * fmaf(a, qc.y, kq * vn.y));
    if (left > 2) hp[2] = from_float<T>(p.scale * fmaf(a, qc.z, kq * vn.z));
    if (left > 3) hp[3] = from_float<T>(p.scale * fmaf(a, qc.w, kq * vn.w));
  }
}

template <typename T, int kThreads, int kTX, int kRows, bool kVec>
cudaError_t go(const GdnProblem& p, const void* q, const void* k, const void* v, const float* g,
               const float* beta, float* C, void* h, cudaStream_t st) {
  const size_t smem = ((size_t)(2 * p.DK + 3) / 4 * 4 + 8 * kThreads + kThreads / 32) * 4;
  gdn_step_kernel<T, kThreads, kTX, kRows, kVec>
      <<<dim3((p.DV + 4 * kTX - 1) / (4 * kTX), p.BH), kThreads, smem, st>>>(
          p, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), g, beta,
          C, static_cast<T*>(h));
  return cudaGetLastError();
}

template <typename T>
cudaError_t step(const GdnProblem& p, const void* q, const void* k, const void* v, const float* g,
                 const float* beta, float* C, void* h, cudaStream_t st) {
  if (p.DV % 4 != 0) return go<T, 128, 8, 8, false>(p, q, k, v, g, beta, C, h, st);
  return go<T, 128, 8, 8, true>(p, q, k, v, g, beta, C, h, st);
}

}  // namespace

cudaError_t launch_gdn_step(const GdnProblem& p, mlstm_dtype dt, const void* q, const void* k,
                            const void* v, const float* g, const float* beta, float* C, void* h,
                            cudaStream_t st) {
  return dt == MLSTM_DT_BF16 ? step<__nv_bfloat16>(p, q, k, v, g, beta, C, h, st)
                             : step<float>(p, q, k, v, g, beta, C, h, st);
}

}  // namespace mlstm
