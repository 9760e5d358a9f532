// Gated delta rule on the CUDA cores, fp32 throughout: the path for fp32
// inputs and for sizes that the tensor-core kernels do not take.  Formulas in
// gdn.h, in chunks of 64 tokens.  Every product is a block-level tiled matrix
// product whose operands are read through small functors (masks, decays and
// ragged ends are applied on the way in), so sizes need no padding in memory.
#include "gdn.h"

namespace mlstm {
namespace {

constexpr int kL = 64;        // chunk length
constexpr int kThreads = 256;
constexpr int kVT = 32;       // value columns per CTA of the sequential kernels
constexpr int kKB = 32;       // depth of one staged slab of a product

__host__ __device__ inline int chunks_of(int T) { return (T + kL - 1) / kL; }

// acc += A [64 x K] B [K x N], N = 16 * TN: thread (ty, tx) of 16 x 16 owns
// rows ty * 4 .. + 3 and columns tx * TN .. + TN - 1.  a(m, k), b(k, n) return
// the elements (zero outside).  AK / BK: consecutive threads read consecutive
// k (else consecutive m / n).
template <int TN, bool AK, bool BK, class FA, class FB>
__device__ __forceinline__ void block_mm(float (&acc)[4][TN], int K, FA a, FB b, float* sa,
                                         float* sb) {
  constexpr int N = 16 * TN, kA = 64 * kKB / kThreads, kB = N * kKB / kThreads;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  // a slab's elements are loaded together, while the slab before is worked on:
  // one by one, their latency made the recurrence four times slower
  float ra[kA], rb[kB];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int i = tid + u * kThreads, m = AK ? i / kKB : i % 64, k = AK ? i % kKB : i / 64;
      ra[u] = k0 + k < K ? a(m, k0 + k) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const int i = tid + u * kThreads, n = BK ? i / kKB : i % N, k = BK ? i % kKB : i / N;
      rb[u] = k0 + k < K ? b(k0 + k, n) : 0.f;
    }
  };
  __syncthreads();
  load(0);
  for (int k0 = 0; k0 < K; k0 += kKB) {
    if (k0) __syncthreads();
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int i = tid + u * kThreads, m = AK ? i / kKB : i % 64, k = AK ? i % kKB : i / 64;
      sa[k * 68 + m] = ra[u];
    }
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const int i = tid + u * kThreads, n = BK ? i / kKB : i % N, k = BK ? i % kKB : i / N;
      sb[k * (N + 4) + n] = rb[u];
    }
    __syncthreads();
    if (k0 + kKB < K) load(k0 + kKB);
#pragma unroll 8
    for (int k = 0; k < kKB; ++k) {
      const float4 av = *reinterpret_cast<const float4*>(sa + k * 68 + ty * 4);
      float bv[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) bv[j] = sb[k * (N + 4) + tx * TN + j];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        acc[0][j] = fmaf(av.x, bv[j], acc[0][j]);
        acc[1][j] = fmaf(av.y, bv[j], acc[1][j]);
        acc[2][j] = fmaf(av.z, bv[j], acc[2][j]);
        acc[3][j] = fmaf(av.w, bv[j], acc[3][j]);
      }
    }
  }
  __syncthreads();
}

template <int TN>
__device__ __forceinline__ void zero(float (&acc)[4][TN]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
}

constexpr int kSa = kKB * 68, kSb = kKB * 68;  // floats of the two staged slabs

// Workspace pieces (fp32): per (bh, chunk) Tinv and Gam . QK^T (without beta)
// [64][64], gc as (hi, lo) pairs per token; the backward adds y, dz
// [BH][NC * 64][DV], the states entering and the state gradients leaving every
// chunk [BH][NC][DK][DV], and with shared key heads dq, dk [BH][T][DK].
struct Ws {
  float *tinv, *p;
  float2* gc;
  float *y, *dz, *S, *dS, *dq, *dk;
  size_t bytes;
};
Ws layout(const GdnProblem& p, bool bw, char* base) {
  Ws w{};
  size_t at = 0;
  const size_t nc = (size_t)p.BH * chunks_of(p.T);
  auto take = [&](size_t floats) {
    float* r = base ? reinterpret_cast<float*>(base + at) : nullptr;
    at += (floats * 4 + 255) / 256 * 256;
    return r;
  };
  w.tinv = take(nc * kL * kL);
  w.p = take(nc * kL * kL);
  w.gc = reinterpret_cast<float2*>(take(nc * kL * 2));
  if (bw) {
    w.y = take(nc * kL * p.DV);
    w.dz = take(nc * kL * p.DV);
    w.S = take(nc * p.DK * p.DV);
    w.dS = take(nc * p.DK * p.DV);
    if (p.group > 1) {
      w.dq = take((size_t)p.BH * p.T * p.DK);
      w.dk = take((size_t)p.BH * p.T * p.DK);
    }
  }
  w.bytes = at;
  return w;
}

// Gam_rs for r >= s (callers mask the rest).
__device__ __forceinline__ float gam(float2 r, float2 s) {
  return expf((r.x - s.x) + (r.y - s.y));
}

// ---- per chunk: gc, Tinv, Gam . QK^T -----------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_simt_prep(GdnProblem p, const T* __restrict__ Q, const T* __restrict__ K,
              const float* __restrict__ g, const float* __restrict__ beta, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sA = sb + kSb;  // sA [64][65]
  float2* sgc = reinterpret_cast<float2*>(sA + 64 * 66);
  float* sbeta = reinterpret_cast<float*>(sgc + 64);
  const int c = blockIdx.x, bh = blockIdx.y, NC = gridDim.x;
  const int t0 = c * kL, n = min(kL, p.T - t0);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long kh = gdn_key_head(p, bh);
  const T* Kp = K + (kh * p.T + t0) * p.DK;
  const T* Qp = Q + (kh * p.T + t0) * p.DK;
  const long gt = (long)bh * p.T + t0;
  if (tid < 32) {  // inclusive sums in 64 bits, two tokens per lane
    double a = 2 * tid < n ? (double)fmaxf(g[gt + 2 * tid], kGdnMinLogDecay) : 0.;
    double b = 2 * tid + 1 < n ? (double)fmaxf(g[gt + 2 * tid + 1], kGdnMinLogDecay) : 0.;
    double s = a + b;
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(0xffffffffu, s, o);
      if (tid >= o) s += u;
    }
    const double x[2] = {s - b, s};
    for (int e = 0; e < 2; ++e) {
      const float hi = (float)x[e];
      sgc[2 * tid + e] = make_float2(hi, (float)(x[e] - hi));
    }
  }
  if (tid < kL) sbeta[tid] = tid < n ? beta[gt + tid] : 0.f;
  __syncthreads();
  const size_t cb = (size_t)bh * NC + c;
  if (tid < kL) w.gc[cb * kL + tid] = sgc[tid];
  auto row = [&](const T* P) {
    return [=](int m, int k) { return m < n ? to_float(P[(long)m * p.DK + k]) : 0.f; };
  };
  auto kcol = [&](int k, int m) { return m < n ? to_float(Kp[(long)m * p.DK + k]) : 0.f; };
  float acc[4][4];
  zero(acc);
  block_mm<4, true, true>(acc, p.DK, row(Qp), kcol, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = ty * 4 + i, s = tx * 4 + j;
      w.p[cb * kL * kL + r * kL + s] = s <= r ? gam(sgc[r], sgc[s]) * acc[i][j] : 0.f;
    }
  zero(acc);
  block_mm<4, true, true>(acc, p.DK, row(Kp), kcol, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = ty * 4 + i, s = tx * 4 + j;
      sA[r * 65 + s] = s < r ? gam(sgc[r], sgc[s]) * sbeta[s] * acc[i][j] : 0.f;
    }
  __syncthreads();
  // the inverse, sX[column][row]: the two 32 x 32 diagonal blocks by forward
  // substitution (a warp each, a lane per column: once x_s is known its multiples
  // leave all later rows, independent products), then -T22 A21 T11
  float* sX = sa;  // [64][65], over both slabs
  if (tid < kL) {
    const int b0 = tid & 32, c = tid & 31;
    float x[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = r == c ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < 31; ++k)
#pragma unroll
      for (int r = k + 1; r < 32; ++r) x[r] = fmaf(-sA[(b0 + r) * 65 + b0 + k], x[k], x[r]);
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      sX[tid * 65 + b0 + r] = x[r];
      if (b0) sX[tid * 65 + r] = 0.f;  // above the diagonal
    }
  }
  __syncthreads();
  {
    const int c = tid & 31, r0 = tid >> 5;
    float x[4] = {};
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = fmaf(sA[(32 + r0 + 8 * i) * 65 + k], sX[c * 65 + k], x[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sA[(32 + r0 + 8 * i) * 65 + c] = x[i];
      x[i] = 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = fmaf(-sX[(32 + k) * 65 + 32 + r0 + 8 * i], sA[(32 + k) * 65 + c], x[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sX[c * 65 + 32 + r0 + 8 * i] = x[i];
  }
  __syncthreads();
  for (int i = tid; i < kL * kL; i += kThreads)
    w.tinv[cb * kL * kL + i] = sX[(i % kL) * 65 + i / kL];
}

// ---- forward recurrence: one CTA per (bh, 32 value columns) ------------
// With kOut it also writes H; with w.S it keeps y and the entering states.
template <typename T, bool kOut>
__global__ void __launch_bounds__(kThreads)
gdn_simt_chain(GdnProblem p, const T* __restrict__ Q, const T* __restrict__ K,
               const T* __restrict__ V, const float* __restrict__ beta,
               const float* __restrict__ C0, T* __restrict__ H, float* __restrict__ C_T, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sz = sb + kSb;  // sz, sy [64][33]
  float *sy = sz + 64 * 33, *sS = sy + 64 * 33;    // sS [DK][33]
  float2* sgc = reinterpret_cast<float2*>(sS + p.DK * 33 + (p.DK & 1));
  float* sbeta = reinterpret_cast<float*>(sgc + 64);
  const int v0 = blockIdx.x * kVT, bh = blockIdx.y, NC = chunks_of(p.T);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long kh = gdn_key_head(p, bh);
  for (int i = tid; i < p.DK * kVT; i += kThreads) {
    const int d = i / kVT, v = i % kVT;
    sS[d * 33 + v] =
        C0 && v0 + v < p.DV ? C0[((long)bh * p.DK + d) * p.DV + v0 + v] : 0.f;
  }
  for (int c = 0; c < NC; ++c) {
    const int t0 = c * kL, n = min(kL, p.T - t0);
    const size_t cb = (size_t)bh * NC + c;
    const T* Kp = K + (kh * p.T + t0) * p.DK;
    const T* Qp = Q + (kh * p.T + t0) * p.DK;
    __syncthreads();
    if (tid < kL) {
      sgc[tid] = w.gc[cb * kL + tid];
      sbeta[tid] = tid < n ? beta[(long)bh * p.T + t0 + tid] : 0.f;
    }
    if (w.S)
      for (int i = tid; i < p.DK * kVT; i += kThreads) {
        const int d = i / kVT, v = i % kVT;
        if (v0 + v < p.DV) w.S[(cb * p.DK + d) * p.DV + v0 + v] = sS[d * 33 + v];
      }
    __syncthreads();
    auto krow = [&](int m, int k) { return m < n ? to_float(Kp[(long)m * p.DK + k]) : 0.f; };
    auto st = [&](int k, int v) { return sS[k * 33 + v]; };
    float acc[4][2], oacc[4][2];
    zero(acc);
    block_mm<2, true, false>(acc, p.DK, krow, st, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 2; ++j) {
        const int r = ty * 4 + i, v = tx * 2 + j;
        const float vv = r < n && v0 + v < p.DV
                             ? to_float(V[((long)bh * p.T + t0 + r) * p.DV + v0 + v])
                             : 0.f;
        sz[r * 33 + v] = vv - expf(sgc[r].x + sgc[r].y) * acc[i][j];
      }
    __syncthreads();
    zero(acc);
    block_mm<2, true, false>(
        acc, kL, [&](int m, int k) { return w.tinv[cb * kL * kL + m * kL + k]; },
        [&](int k, int v) { return sz[k * 33 + v]; }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 2; ++j) {
        const int r = ty * 4 + i, v = tx * 2 + j;
        sy[r * 33 + v] = sbeta[r] * acc[i][j];
        if (w.S && v0 + v < p.DV) w.y[(cb * kL + r) * p.DV + v0 + v] = acc[i][j];
      }
    __syncthreads();
    if (kOut) {
      zero(oacc);
      block_mm<2, true, false>(
          oacc, p.DK, [&](int m, int k) { return m < n ? to_float(Qp[(long)m * p.DK + k]) : 0.f; },
          st, sa, sb);
      for (int i = 0; i < 4; ++i) {
        const float2 gr = sgc[ty * 4 + i];
        for (int j = 0; j < 2; ++j) oacc[i][j] *= expf(gr.x + gr.y);
      }
      block_mm<2, true, false>(
          oacc, kL, [&](int m, int k) { return w.p[cb * kL * kL + m * kL + k]; },
          [&](int k, int v) { return sy[k * 33 + v]; }, sa, sb);
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 2; ++j) {
          const int r = ty * 4 + i, v = v0 + tx * 2 + j;
          if (r < n && v < p.DV)
            H[((long)bh * p.T + t0 + r) * p.DV + v] = from_float<T>(p.scale * oacc[i][j]);
        }
    }
    // S' = e^G S + K^T (D beta y), 64 state rows at a time (each product ends
    // with a barrier, and only this CTA's own rows are written)
    const float2 gl = sgc[kL - 1];
    const float eg = expf(gl.x + gl.y);
    for (int d0 = 0; d0 < p.DK; d0 += 64) {
      zero(acc);
      block_mm<2, false, false>(
          acc, kL,
          [&](int m, int k) {
            return k < n && d0 + m < p.DK ? to_float(Kp[(long)k * p.DK + d0 + m]) : 0.f;
          },
          [&](int k, int v) { return gam(gl, sgc[k]) * sy[k * 33 + v]; }, sa, sb);
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 2; ++j) {
          const int d = d0 + ty * 4 + i, v = tx * 2 + j;
          if (d < p.DK) sS[d * 33 + v] = fmaf(eg, sS[d * 33 + v], acc[i][j]);
        }
    }
  }
  __syncthreads();
  if (C_T)
    for (int i = tid; i < p.DK * kVT; i += kThreads) {
      const int d = i / kVT, v = i % kVT;
      if (v0 + v < p.DV) C_T[((long)bh * p.DK + d) * p.DV + v0 + v] = sS[d * 33 + v];
    }
}

// ---- reverse recurrence: dz (= dV) and the state gradients --------------
template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_simt_bchain(GdnProblem p, const T* __restrict__ Q, const T* __restrict__ K,
                const float* __restrict__ beta, const T* __restrict__ dH,
                const float* __restrict__ dC_T, T* __restrict__ dV, float* __restrict__ dC0, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sw = sb + kSb;  // sw, sd [64][33]
  float *sd = sw + 64 * 33, *sS = sd + 64 * 33;    // sS [DK][33]: the state gradient
  float2* sgc = reinterpret_cast<float2*>(sS + p.DK * 33 + (p.DK & 1));
  float* sbeta = reinterpret_cast<float*>(sgc + 64);
  const int v0 = blockIdx.x * kVT, bh = blockIdx.y, NC = chunks_of(p.T);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long kh = gdn_key_head(p, bh);
  for (int i = tid; i < p.DK * kVT; i += kThreads) {
    const int d = i / kVT, v = i % kVT;
    sS[d * 33 + v] =
        dC_T && v0 + v < p.DV ? dC_T[((long)bh * p.DK + d) * p.DV + v0 + v] : 0.f;
  }
  for (int c = NC - 1; c >= 0; --c) {
    const int t0 = c * kL, n = min(kL, p.T - t0);
    const size_t cb = (size_t)bh * NC + c;
    const T* Kp = K + (kh * p.T + t0) * p.DK;
    const T* Qp = Q + (kh * p.T + t0) * p.DK;
    __syncthreads();
    if (tid < kL) {
      sgc[tid] = w.gc[cb * kL + tid];
      sbeta[tid] = tid < n ? beta[(long)bh * p.T + t0 + tid] : 0.f;
    }
    for (int i = tid; i < p.DK * kVT; i += kThreads) {
      const int d = i / kVT, v = i % kVT;
      if (v0 + v < p.DV) w.dS[(cb * p.DK + d) * p.DV + v0 + v] = sS[d * 33 + v];
    }
    for (int i = tid; i < kL * kVT; i += kThreads) {
      const int r = i / kVT, v = i % kVT;
      sd[r * 33 + v] = r < n && v0 + v < p.DV
                           ? to_float(dH[((long)bh * p.T + t0 + r) * p.DV + v0 + v])
                           : 0.f;
    }
    __syncthreads();
    const float2 gl = sgc[kL - 1];
    float acc[4][2], acc2[4][2];
    zero(acc);
    zero(acc2);
    block_mm<2, false, false>(
        acc, kL, [&](int m, int k) { return w.p[cb * kL * kL + k * kL + m]; },
        [&](int k, int v) { return sd[k * 33 + v]; }, sa, sb);
    block_mm<2, true, false>(
        acc2, p.DK, [&](int m, int k) { return m < n ? to_float(Kp[(long)m * p.DK + k]) : 0.f; },
        [&](int k, int v) { return sS[k * 33 + v]; }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 2; ++j) {
        const int r = ty * 4 + i;
        sw[r * 33 + tx * 2 + j] =
            sbeta[r] * fmaf(p.scale, acc[i][j], gam(gl, sgc[r]) * acc2[i][j]);
      }
    __syncthreads();
    zero(acc);
    block_mm<2, false, false>(
        acc, kL, [&](int m, int k) { return w.tinv[cb * kL * kL + k * kL + m]; },
        [&](int k, int v) { return sw[k * 33 + v]; }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 2; ++j) {
        const int r = ty * 4 + i, v = tx * 2 + j;
        if (v0 + v < p.DV) {
          w.dz[(cb * kL + r) * p.DV + v0 + v] = acc[i][j];
          if (r < n) dV[((long)bh * p.T + t0 + r) * p.DV + v0 + v] = from_float<T>(acc[i][j]);
        }
        const float lam = expf(sgc[r].x + sgc[r].y);
        sw[r * 33 + v] = -lam * acc[i][j];
        sd[r * 33 + v] *= p.scale * lam;
      }
    __syncthreads();
    const float eg = expf(gl.x + gl.y);
    for (int d0 = 0; d0 < p.DK; d0 += 64) {
      auto col = [&](const T* P) {
        return [=](int m, int k) {
          return k < n && d0 + m < p.DK ? to_float(P[(long)k * p.DK + d0 + m]) : 0.f;
        };
      };
      zero(acc);
      block_mm<2, false, false>(acc, kL, col(Kp), [&](int k, int v) { return sw[k * 33 + v]; }, sa,
                                sb);
      block_mm<2, false, false>(acc, kL, col(Qp), [&](int k, int v) { return sd[k * 33 + v]; }, sa,
                                sb);
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 2; ++j) {
          const int d = d0 + ty * 4 + i, v = tx * 2 + j;
          if (d < p.DK) sS[d * 33 + v] = fmaf(eg, sS[d * 33 + v], acc[i][j]);
        }
    }
  }
  __syncthreads();
  if (dC0)
    for (int i = tid; i < p.DK * kVT; i += kThreads) {
      const int d = i / kVT, v = i % kVT;
      if (v0 + v < p.DV) dC0[((long)bh * p.DK + d) * p.DV + v0 + v] = sS[d * 33 + v];
    }
}

// ---- per chunk: dQ, dK, dg, dbeta ---------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_simt_grads(GdnProblem p, const T* __restrict__ Q, const T* __restrict__ K,
               const float* __restrict__ beta, const T* __restrict__ dH, T* __restrict__ dQ,
               T* __restrict__ dK, float* __restrict__ dg, float* __restrict__ dbeta, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sR = sb + kSb, *sE = sR + 64 * 65;  // Rh, Eh [64][65]
  float *srow = sE + 64 * 65;             // [64]: row sums of the strict part of Z beta
  float *scol = srow + 64, *sout = scol + 64, *sent = sout + 64, *sbeta = sent + 64;
  float* sred = sbeta + 64;               // [64][17]
  float2* sgc = reinterpret_cast<float2*>(sred + 64 * 17 + 64);
  const int c = blockIdx.x, bh = blockIdx.y, NC = gridDim.x;
  const int t0 = c * kL, n = min(kL, p.T - t0);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const size_t cb = (size_t)bh * NC + c;
  const long kh = gdn_key_head(p, bh);
  const T* Kp = K + (kh * p.T + t0) * p.DK;
  const T* Qp = Q + (kh * p.T + t0) * p.DK;
  const T* dHp = dH + ((long)bh * p.T + t0) * p.DV;
  const float* yp = w.y + cb * kL * p.DV;
  const float* zp = w.dz + cb * kL * p.DV;
  const float* Sp = w.S + cb * p.DK * p.DV;
  const float* dSp = w.dS + cb * p.DK * p.DV;
  if (tid < kL) {
    sgc[tid] = w.gc[cb * kL + tid];
    sbeta[tid] = tid < n ? beta[(long)bh * p.T + t0 + tid] : 0.f;
    srow[tid] = scol[tid] = sout[tid] = sent[tid] = 0.f;
  }
  __syncthreads();
  auto dhrow = [&](int m, int k) { return m < n ? to_float(dHp[(long)m * p.DV + k]) : 0.f; };
  auto zrow = [&](int m, int k) { return zp[(long)m * p.DV + k]; };
  auto yrow = [&](int m, int k) { return yp[(long)m * p.DV + k]; };
  auto ycol = [&](int k, int m) { return yp[(long)m * p.DV + k]; };
  auto qk = [&](const T* P) {
    return [=](int m, int k) { return m < n ? to_float(P[(long)m * p.DK + k]) : 0.f; };
  };
  auto kcol = [&](int k, int m) { return m < n ? to_float(Kp[(long)m * p.DK + k]) : 0.f; };
  // sums over the rows (columns) of the 64 x 64 tile that the threads hold
  auto row_sums = [&](const float (&part)[4], float* dst, float f) {
    for (int i = 0; i < 4; ++i) sred[(ty * 4 + i) * 17 + tx] = part[i];
    __syncthreads();
    if (tid < kL) {
      float s = 0.f;
      for (int j = 0; j < 16; ++j) s += sred[tid * 17 + j];
      dst[tid] += f * s;
    }
    __syncthreads();
  };
  float acc[4][4], zac[4][4], zsum[4][4];
  zero(zsum);
  for (int part = 0; part < 2; ++part) {  // Rh, then Eh, and their part of Z
    zero(acc);
    zero(zac);
    if (part == 0) {
      block_mm<4, true, true>(acc, p.DV, dhrow, ycol, sa, sb);
      block_mm<4, true, true>(zac, p.DK, qk(Qp), kcol, sa, sb);
    } else {
      block_mm<4, true, true>(acc, p.DV, zrow, ycol, sa, sb);
      block_mm<4, true, true>(zac, p.DK, qk(Kp), kcol, sa, sb);
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int r = ty * 4 + i, s = tx * 4 + j;
        const bool in = part == 0 ? s <= r : s < r;
        const float x = in ? (part == 0 ? p.scale : -1.f) * gam(sgc[r], sgc[s]) * acc[i][j] : 0.f;
        (part == 0 ? sR : sE)[r * 65 + s] = x;
        zsum[i][j] = fmaf(x, zac[i][j], zsum[i][j]);
      }
  }
  {
    float part[4];
    for (int i = 0; i < 4; ++i) {
      part[i] = 0.f;
      for (int j = 0; j < 4; ++j) {
        const int r = ty * 4 + i, s = tx * 4 + j;
        if (s < r) part[i] = fmaf(zsum[i][j], sbeta[s], part[i]);
      }
    }
    row_sums(part, srow, 1.f);
    // columns: [tx * 4 + j][ty]; the strict part (for dg) and the diagonal apart
    float pc[4];
    for (int j = 0; j < 4; ++j) {
      pc[j] = 0.f;
      for (int i = 0; i < 4; ++i)
        if (tx * 4 + j < ty * 4 + i) pc[j] += zsum[i][j];
    }
    for (int j = 0; j < 4; ++j) sred[(tx * 4 + j) * 17 + ty] = pc[j];
    __syncthreads();
    if (tid < kL) {
      float s = 0.f;
      for (int j = 0; j < 16; ++j) s += sred[tid * 17 + j];
      scol[tid] = s;
    }
    __syncthreads();
  }
  // diagonal of Z into dbeta: held by the threads with tx == ty
  float* sdiag = sred + 64 * 17;
  if (tx == ty)
    for (int i = 0; i < 4; ++i) sdiag[ty * 4 + i] = zsum[i][i];
  const float2 gl = sgc[kL - 1];
  for (int d0 = 0; d0 < p.DK; d0 += 64) {
    const int tn = tx * 4;
    auto srow_t = [&](const float* S) {
      return [=](int k, int d) { return d0 + d < p.DK ? S[(long)(d0 + d) * p.DV + k] : 0.f; };
    };
    auto kd = [&](const T* P) {
      return [=](int k, int d) {
        return k < n && d0 + d < p.DK ? to_float(P[(long)k * p.DK + d0 + d]) : 0.f;
      };
    };
    float part[4];
    auto el = [&](const T* P, int i, int j) {
      const int r = ty * 4 + i, d = d0 + tn + j;
      return r < n && d < p.DK ? to_float(P[(long)r * p.DK + d]) : 0.f;
    };
    // dQ
    zero(acc);
    block_mm<4, true, true>(acc, p.DV, dhrow, srow_t(Sp), sa, sb);
    for (int i = 0; i < 4; ++i) {
      const float f = p.scale * expf(sgc[ty * 4 + i].x + sgc[ty * 4 + i].y);
      part[i] = 0.f;
      for (int j = 0; j < 4; ++j) {
        acc[i][j] *= f;
        part[i] = fmaf(acc[i][j], el(Qp, i, j), part[i]);
      }
    }
    row_sums(part, sent, 1.f);
    block_mm<4, true, false>(acc, kL, [&](int m, int k) { return sR[m * 65 + k] * sbeta[k]; },
                             kd(Kp), sa, sb);
    auto put = [&](T* out, float* out32, float (&x)[4][4]) {
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
          const int r = ty * 4 + i, d = d0 + tn + j;
          if (r >= n || d >= p.DK) continue;
          const size_t at = ((size_t)(out32 ? (long)bh : kh) * p.T + t0 + r) * p.DK + d;
          if (out32)
            out32[at] = x[i][j];
          else
            out[at] = from_float<T>(x[i][j]);
        }
    };
    put(dQ, w.dq, acc);
    // dK: beta (D (y dS'^T) + Rh^T Q + Eh^T K) - Lam (dz S^T) + (Eh beta) K
    zero(acc);
    block_mm<4, true, true>(acc, p.DV, yrow, srow_t(dSp), sa, sb);
    for (int i = 0; i < 4; ++i) {
      const float f = gam(gl, sgc[ty * 4 + i]);
      part[i] = 0.f;
      for (int j = 0; j < 4; ++j) {
        acc[i][j] *= f;
        part[i] = fmaf(acc[i][j], el(Kp, i, j), part[i]);
      }
    }
    row_sums(part, sout, 1.f);
    block_mm<4, false, false>(acc, kL, [&](int m, int k) { return sR[k * 65 + m]; }, kd(Qp), sa,
                              sb);
    block_mm<4, false, false>(acc, kL, [&](int m, int k) { return sE[k * 65 + m]; }, kd(Kp), sa,
                              sb);
    zero(zac);
    block_mm<4, true, true>(zac, p.DV, zrow, srow_t(Sp), sa, sb);
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      const float lam = expf(sgc[r].x + sgc[r].y);
      part[i] = 0.f;
      for (int j = 0; j < 4; ++j) {
        zac[i][j] *= -lam;
        part[i] = fmaf(zac[i][j], el(Kp, i, j), part[i]);
        zac[i][j] = fmaf(sbeta[r], acc[i][j], zac[i][j]);
      }
    }
    row_sums(part, sent, 1.f);
    block_mm<4, true, false>(zac, kL, [&](int m, int k) { return sE[m * 65 + k] * sbeta[k]; },
                             kd(Kp), sa, sb);
    put(dK, w.dk, zac);
  }
  // <S, dS'>
  float ss = 0.f;
  for (long i = tid; i < (long)p.DK * p.DV; i += kThreads) ss = fmaf(Sp[i], dSp[i], ss);
  ss = warp_sum(ss);
  if ((tid & 31) == 0) sred[tid >> 5] = ss;
  __syncthreads();
  if (tid == 0) {
    float dG = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) dG += sred[i];
    dG *= expf(gl.x + gl.y);
    // dg_t: suffix sums of the entering terms and of Z's rows less its
    // columns, prefix sums of the leaving terms
    float suf = 0.f;
    for (int t = n - 1; t >= 0; --t) {
      suf += sent[t] + (srow[t] - sbeta[t] * scol[t]);
      sent[t] = suf;
    }
    float pre = 0.f;
    for (int t = 0; t < n; ++t) {
      sent[t] += pre + dG;
      pre = fmaf(sbeta[t], sout[t], pre);
    }
  }
  __syncthreads();
  if (tid < n) {
    dg[(long)bh * p.T + t0 + tid] = sent[tid];
    dbeta[(long)bh * p.T + t0 + tid] = sout[tid] + scol[tid] + sdiag[tid];
  }
}

template <typename T>
__global__ void gdn_group_sum(GdnProblem p, const float* __restrict__ dq,
                              const float* __restrict__ dk, T* __restrict__ dQ,
                              T* __restrict__ dK) {
  const size_t per = (size_t)p.T * p.DK, n = (size_t)p.B * p.NHK * per;
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x) {
    const size_t src = i / per * p.group * per + i % per;
    float a = 0.f, b = 0.f;
    for (int j = 0; j < p.group; ++j) {
      a += dq[src + j * per];
      b += dk[src + j * per];
    }
    dQ[i] = from_float<T>(a);
    dK[i] = from_float<T>(b);
  }
}

size_t chain_smem(const GdnProblem& p) {
  return (size_t)(kSa + kSb + 2 * 64 * 33 + p.DK * 33 + (p.DK & 1) + 64 * 3) * 4;
}
constexpr size_t kPrepSmem = (kSa + kSb + 64 * 66 + 64 * 3) * 4;
constexpr size_t kGradSmem = (kSa + kSb + 2 * 64 * 65 + 5 * 64 + 64 * 17 + 64 + 128) * 4;

template <class F>
cudaError_t allow(F* f, size_t smem) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <typename T>
cudaError_t prep(const GdnProblem& p, const GdnInputs& x, const Ws& w, cudaStream_t st) {
  cudaError_t e = allow(gdn_simt_prep<T>, kPrepSmem);
  if (e != cudaSuccess) return e;
  gdn_simt_prep<T><<<dim3(chunks_of(p.T), p.BH), kThreads, kPrepSmem, st>>>(
      p, (const T*)x.Q, (const T*)x.K, x.g, x.beta, w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T, void* ws,
               cudaStream_t st) {
  const Ws w = layout(p, false, static_cast<char*>(ws));
  if (p.T > 0) {
    const cudaError_t e = prep<T>(p, x, w, st);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = allow(gdn_simt_chain<T, true>, chain_smem(p));
  if (e != cudaSuccess) return e;
  gdn_simt_chain<T, true><<<dim3((p.DV + kVT - 1) / kVT, p.BH), kThreads, chain_smem(p), st>>>(
      p, (const T*)x.Q, (const T*)x.K, (const T*)x.V, x.beta, x.C0, (T*)H, C_T, w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
               cudaStream_t st) {
  const Ws w = layout(p, true, static_cast<char*>(ws));
  const dim3 cols((p.DV + kVT - 1) / kVT, p.BH), chunks(chunks_of(p.T), p.BH);
  cudaError_t e = prep<T>(p, x, w, st);
  if (e != cudaSuccess) return e;
  if ((e = allow(gdn_simt_chain<T, false>, chain_smem(p))) != cudaSuccess) return e;
  gdn_simt_chain<T, false><<<cols, kThreads, chain_smem(p), st>>>(
      p, (const T*)x.Q, (const T*)x.K, (const T*)x.V, x.beta, x.C0, nullptr, nullptr, w);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = allow(gdn_simt_bchain<T>, chain_smem(p))) != cudaSuccess) return e;
  gdn_simt_bchain<T><<<cols, kThreads, chain_smem(p), st>>>(
      p, (const T*)x.Q, (const T*)x.K, x.beta, (const T*)d.dH, d.dC_T, (T*)d.dV, d.dC0, w);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = allow(gdn_simt_grads<T>, kGradSmem)) != cudaSuccess) return e;
  gdn_simt_grads<T><<<chunks, kThreads, kGradSmem, st>>>(p, (const T*)x.Q, (const T*)x.K, x.beta,
                                                         (const T*)d.dH, (T*)d.dQ, (T*)d.dK, d.dg,
                                                         d.dbeta, w);
  if ((e = cudaGetLastError()) != cudaSuccess || p.group == 1) return e;
  return launch_gdn_group_sum(p, sizeof(T) == 2 ? MLSTM_DT_BF16 : MLSTM_DT_F32, w.dq, w.dk, d.dQ,
                              d.dK, st);
}

}  // namespace

size_t gdn_simt_workspace(const GdnProblem& p, bool backward) {
  return layout(p, backward, nullptr).bytes;
}
int gdn_simt_launches(const GdnProblem& p, bool backward) {
  return backward ? 4 + (p.group > 1) : 1 + (p.T > 0);
}
cudaError_t launch_gdn_simt_fw(const GdnProblem& p, mlstm_dtype dt, const GdnInputs& x, void* H,
                               float* C_T, void* ws, cudaStream_t st) {
  return dt == MLSTM_DT_BF16 ? fw<__nv_bfloat16>(p, x, H, C_T, ws, st)
                             : fw<float>(p, x, H, C_T, ws, st);
}
cudaError_t launch_gdn_simt_bw(const GdnProblem& p, mlstm_dtype dt, const GdnInputs& x,
                               const GdnGrads& d, void* ws, cudaStream_t st) {
  return dt == MLSTM_DT_BF16 ? bw<__nv_bfloat16>(p, x, d, ws, st) : bw<float>(p, x, d, ws, st);
}
cudaError_t launch_gdn_group_sum(const GdnProblem& p, mlstm_dtype dt, const float* dq,
                                 const float* dk, void* dQ, void* dK, cudaStream_t st) {
  const size_t n = (size_t)p.B * p.NHK * p.T * p.DK;
  const int grid = (int)((n + 255) / 256 < 148 * 16 ? (n + 255) / 256 : 148 * 16);
  if (dt == MLSTM_DT_BF16)
    gdn_group_sum<<<grid, 256, 0, st>>>(p, dq, dk, (__nv_bfloat16*)dQ, (__nv_bfloat16*)dK);
  else
    gdn_group_sum<<<grid, 256, 0, st>>>(p, dq, dk, (float*)dQ, (float*)dK);
  return cudaGetLastError();
}

}  // namespace mlstm
