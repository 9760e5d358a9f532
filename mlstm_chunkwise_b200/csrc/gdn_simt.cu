// Gated delta rule on the CUDA cores, fp32 throughout: the path for fp32
// inputs and for sizes that the tensor-core kernels do not take.  Formulas in
// gdn.h, in chunks of 64 tokens.  Every product is a block-level tiled matrix
// product whose operands are read through small functors (masks, decays and
// ragged ends are applied on the way in), so sizes need no padding in memory.
//
// What does not depend on the state (Tinv, W = Tinv Lam K, U = Tinv V and their
// counterparts of the gradients) is formed for all chunks in parallel, and so is
// what follows from the states; only y = U - W S and S' = e^G S + K^T (D beta y)
// run chunk after chunk.  1000 tokens x 4 heads of 64 x 96 in fp32: 117 us, 89 of
// them the recurrence (5.5 us a chunk of two dependent products, bound by their
// latency: an SM is 9% busy); with z, y and the output on the recurrence it was 206.
#include "device_address.h"
#include "gdn.h"

namespace mlstm {
namespace {

constexpr int kL = 64;        // chunk length
constexpr int kThreads = 256;
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

// Workspace pieces (fp32), per (bh, chunk): Tinv and Gam . QK^T (without beta)
// [64][64], gc as (hi, lo) pairs per token; W = Tinv Lam K [64][DK]; y [64][DV],
// in its place first U = Tinv V; S [DK][DV], the state entering.  The backward
// adds E = Tinv^T beta D K [64][DK]; dz [64][DV], first dz without its part from
// dS'; dS [DK][DV], the state gradient leaving, first Q^T (scale Lam dH); and with
// shared key heads dq, dk [BH][T][DK].
struct Ws {
  float *tinv, *p;
  float2* gc;
  float *W, *y, *S, *E, *dz, *dS, *dq, *dk;
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
  w.W = take(nc * kL * p.DK);
  w.y = take(nc * kL * p.DV);
  w.S = take(nc * p.DK * p.DV);
  if (bw) {
    w.E = take(nc * kL * p.DK);
    w.dz = take(nc * kL * p.DV);
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
__global__ void __launch_bounds__(kThreads, 2)
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
    double a = 2 * tid < n ? (double)gdn_log_decay(g[gt + 2 * tid]) : 0.;
    double b = 2 * tid + 1 < n ? (double)gdn_log_decay(g[gt + 2 * tid + 1]) : 0.;
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

// Gates of a chunk: gc, and per token Lam, D and beta.
struct Gates64 {
  float2 gc[kL];
  float lam[kL], d[kL], beta[kL];
};
__device__ __forceinline__ void load_gates(Gates64* g, const GdnProblem& p, const Ws& w, size_t cb,
                                           const float* beta, long at, int n) {
  const int t = threadIdx.x;
  if (t < kL) {
    const float2 x = w.gc[cb * kL + t];
    g->gc[t] = x;
    g->lam[t] = expf(x.x + x.y);
    g->d[t] = gam(w.gc[cb * kL + kL - 1], x);
    g->beta[t] = t < n ? beta[at + t] : 0.f;
  }
  __syncthreads();
}
// Rows of Q, K (or V, dH) of a chunk; zero outside.
template <typename T>
struct Rows {
  const T* p;
  int n, cols;
  __device__ float operator()(int r, int c) const {
    return r < n && c < cols ? to_float(p[(long)r * cols + c]) : 0.f;
  }
};

// ---- per chunk: W and U; for the backward E, dz0 and Q^T (scale Lam dH) ------
template <typename T, bool kBw>
__global__ void __launch_bounds__(kThreads, 2)
gdn_simt_chunk(GdnProblem p, const T* __restrict__ Q, const T* __restrict__ K,
               const T* __restrict__ V, const float* __restrict__ beta,
               const T* __restrict__ dH, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sw = sb + kSb;  // sw [64][65]
  Gates64* g = reinterpret_cast<Gates64*>(sw + 64 * 66);
  const int c = blockIdx.x, bh = blockIdx.y, NC = gridDim.x;
  const int t0 = c * kL, n = min(kL, p.T - t0);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const size_t cb = (size_t)bh * NC + c;
  const long kh = gdn_key_head(p, bh), at = (long)bh * p.T + t0;
  load_gates(g, p, w, cb, beta, at, n);
  const Rows<T> q{Q + (kh * p.T + t0) * p.DK, n, p.DK}, k{K + (kh * p.T + t0) * p.DK, n, p.DK};
  const float* tinv = w.tinv + cb * kL * kL;
  float acc[4][4];
  auto put = [&](float* dst, int rows, int cols, int r0, int c0) {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + ty * 4 + i, cc = c0 + tx * 4 + j;
        if (r < rows && cc < cols && MLSTM_IN_BOUNDS(p, cb < (size_t)p.BH * NC))
          dst[(long)r * cols + cc] = acc[i][j];
      }
  };
  for (int d0 = 0; d0 < p.DK; d0 += 64) {
    zero(acc);
    block_mm<4, true, false>(
        acc, kL, [&](int m, int s) { return tinv[m * kL + s] * g->lam[s]; },
        [&](int s, int d) { return k(s, d0 + d); }, sa, sb);
    put(w.W + cb * kL * p.DK, kL, p.DK, 0, d0);
    if (kBw) {
      zero(acc);
      block_mm<4, false, false>(
          acc, kL, [&](int m, int s) { return tinv[s * kL + m] * (g->beta[s] * g->d[s]); },
          [&](int s, int d) { return k(s, d0 + d); }, sa, sb);
      put(w.E + cb * kL * p.DK, kL, p.DK, 0, d0);
    }
  }
  const Rows<T> v{V + at * p.DV, n, p.DV};
  for (int v0 = 0; v0 < p.DV; v0 += 64) {
    zero(acc);
    block_mm<4, true, false>(
        acc, kL, [&](int m, int s) { return tinv[m * kL + s]; },
        [&](int s, int e) { return v(s, v0 + e); }, sa, sb);
    put(w.y + cb * kL * p.DV, kL, p.DV, 0, v0);
    if (!kBw) continue;
    const Rows<T> dh{dH + at * p.DV, n, p.DV};
    zero(acc);
    block_mm<4, false, false>(
        acc, kL, [&](int m, int s) { return w.p[cb * kL * kL + s * kL + m]; },
        [&](int s, int e) { return dh(s, v0 + e); }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j)
        sw[(ty * 4 + i) * 65 + tx * 4 + j] = p.scale * g->beta[ty * 4 + i] * acc[i][j];
    zero(acc);
    block_mm<4, false, false>(
        acc, kL, [&](int m, int s) { return tinv[s * kL + m]; },
        [&](int s, int e) { return sw[s * 65 + e]; }, sa, sb);
    put(w.dz + cb * kL * p.DV, kL, p.DV, 0, v0);
    for (int d0 = 0; d0 < p.DK; d0 += 64) {
      zero(acc);
      block_mm<4, false, false>(
          acc, kL, [&](int m, int s) { return q(s, d0 + m) * (p.scale * g->lam[s]); },
          [&](int s, int e) { return dh(s, v0 + e); }, sa, sb);
      put(w.dS + cb * p.DK * p.DV, p.DK, p.DV, d0, v0);
    }
  }
}

// ---- the recurrences: one CTA per (bh, 16 kTN value columns) ------------
// Forward: y = U - W S, S' = e^G S + K^T (D beta y).  Reverse: dz = dz0 + E dS',
// dS = e^G dS' + Q^T (scale Lam dH) - K^T (Lam dz).
template <typename T, bool kRev, int kTN>
__global__ void __launch_bounds__(kThreads)
gdn_simt_chain(GdnProblem p, const T* __restrict__ K, const float* __restrict__ beta,
               const float* __restrict__ init, float* __restrict__ fin, T* __restrict__ dV, Ws w) {
  constexpr int kVT = 16 * kTN;
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa, *sy = sb + kSb;  // sy [64][33]
  float* sS = sy + 64 * 33;                        // [DK][33]
  Gates64* g = reinterpret_cast<Gates64*>(sS + p.DK * 33 + (p.DK & 1));
  const int v0 = blockIdx.x * kVT, bh = blockIdx.y, NC = chunks_of(p.T);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long kh = gdn_key_head(p, bh);
  // a first token that forgets the state entirely: it may hold anything, and 0 times
  // an infinity is a NaN
  const float2 g0 = w.gc[(size_t)bh * NC * kL];
  const bool have = init && (kRev || expf(g0.x + g0.y) != 0.f);
  for (int i = tid; i < p.DK * kVT; i += kThreads) {
    const int d = i / kVT, v = i % kVT;
    sS[d * 33 + v] = have && v0 + v < p.DV ? init[((long)bh * p.DK + d) * p.DV + v0 + v] : 0.f;
  }
  const float* A = kRev ? w.E : w.W;
  float *Y = kRev ? w.dz : w.y, *St = kRev ? w.dS : w.S;
  for (int step = 0; step < NC; ++step) {
    const int c = kRev ? NC - 1 - step : step, t0 = c * kL, n = min(kL, p.T - t0);
    const size_t cb = (size_t)bh * NC + c;
    __syncthreads();
    load_gates(g, p, w, cb, beta, (long)bh * p.T + t0, n);
    const Rows<T> k{K + (kh * p.T + t0) * p.DK, n, p.DK};
    float acc[4][kTN], add[4][kTN];
    // what a product's result is added to is loaded ahead of the product
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < kTN; ++j) {
        const int r = ty * 4 + i, v = v0 + tx * kTN + j;
        add[i][j] = v < p.DV ? Y[(cb * kL + r) * p.DV + v] : 0.f;
      }
    zero(acc);
    block_mm<kTN, true, false>(
        acc, p.DK, [&](int m, int d) { return A[(cb * kL + m) * p.DK + d]; },
        [&](int d, int v) { return sS[d * 33 + v]; }, sa, sb);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < kTN; ++j) {
        const int r = ty * 4 + i, v = tx * kTN + j;
        const float y = kRev ? add[i][j] + acc[i][j] : add[i][j] - acc[i][j];
        if (v0 + v < p.DV && MLSTM_IN_BOUNDS(p, cb < (size_t)p.BH * NC && r < kL)) {
          Y[(cb * kL + r) * p.DV + v0 + v] = y;
          if (kRev && r < n) dV[((long)bh * p.T + t0 + r) * p.DV + v0 + v] = from_float<T>(y);
        }
        sy[r * 33 + v] = y * (kRev ? -g->lam[r] : g->d[r] * g->beta[r]);
      }
    __syncthreads();
    const float2 gl = g->gc[kL - 1];
    const float eg = expf(gl.x + gl.y);
    // 64 state rows at a time; a thread keeps the rows that it updates
    for (int d0 = 0; d0 < p.DK; d0 += 64) {
      if (kRev)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < kTN; ++j) {
            const int d = d0 + ty * 4 + i, v = v0 + tx * kTN + j;
            add[i][j] = d < p.DK && v < p.DV ? St[(cb * p.DK + d) * p.DV + v] : 0.f;
          }
      zero(acc);
      block_mm<kTN, false, false>(
          acc, kL, [&](int m, int s) { return k(s, d0 + m); },
          [&](int s, int v) { return sy[s * 33 + v]; }, sa, sb);
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < kTN; ++j) {
          const int d = d0 + ty * 4 + i, v = tx * kTN + j;
          if (d >= p.DK) continue;
          const float old = sS[d * 33 + v];
          if (v0 + v < p.DV && MLSTM_IN_BOUNDS(p, cb < (size_t)p.BH * NC))
            St[(cb * p.DK + d) * p.DV + v0 + v] = old;
          sS[d * 33 + v] = fmaf(eg, old, kRev ? acc[i][j] + add[i][j] : acc[i][j]);
        }
    }
  }
  __syncthreads();
  if (fin)
    for (int i = tid; i < p.DK * kVT; i += kThreads) {
      const int d = i / kVT, v = i % kVT;
      if (v0 + v < p.DV && MLSTM_IN_BOUNDS(p, bh < p.BH && d < p.DK))
        fin[((long)bh * p.DK + d) * p.DV + v0 + v] = sS[d * 33 + v];
    }
}

// ---- per chunk, 64 value columns: H = scale (Lam Q S + P beta y) --------
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
gdn_simt_out(GdnProblem p, const T* __restrict__ Q, const float* __restrict__ beta,
             T* __restrict__ H, Ws w) {
  extern __shared__ float sh[];
  float *sa = sh, *sb = sa + kSa;
  Gates64* g = reinterpret_cast<Gates64*>(sb + kSb);
  // chunks along x: there may be more than the 65535 blocks that y holds
  const int v0 = blockIdx.y * 64, c = blockIdx.x, bh = blockIdx.z, NC = gridDim.x;
  const int t0 = c * kL, n = min(kL, p.T - t0);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const size_t cb = (size_t)bh * NC + c;
  const long kh = gdn_key_head(p, bh), at = (long)bh * p.T + t0;
  load_gates(g, p, w, cb, beta, at, n);
  const Rows<T> q{Q + (kh * p.T + t0) * p.DK, n, p.DK};
  const Rows<float> s{w.S + cb * p.DK * p.DV, p.DK, p.DV}, y{w.y + cb * kL * p.DV, kL, p.DV};
  float acc[4][4];
  zero(acc);
  block_mm<4, true, false>(
      acc, p.DK, [&](int m, int d) { return q(m, d); },
      [&](int d, int v) { return s(d, v0 + v); }, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] *= g->lam[ty * 4 + i];
  block_mm<4, true, false>(
      acc, kL, [&](int m, int t) { return w.p[cb * kL * kL + m * kL + t]; },
      [&](int t, int v) { return g->beta[t] * y(t, v0 + v); }, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = ty * 4 + i, v = v0 + tx * 4 + j;
      if (r < n && v < p.DV && MLSTM_IN_BOUNDS(p, at + r < (long)p.BH * p.T))
        H[(at + r) * p.DV + v] = from_float<T>(p.scale * acc[i][j]);
    }
}

// ---- per chunk: dQ, dK, dg, dbeta ---------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
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
          if (r >= n || d >= p.DK || !MLSTM_IN_BOUNDS(p, t0 + r < p.T && bh < p.BH)) continue;
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
  if (tid < n && MLSTM_IN_BOUNDS(p, bh < p.BH && t0 + tid < p.T)) {
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

constexpr size_t chain_smem(int DK) {
  return (size_t)(kSa + kSb + 64 * 33 + DK * 33 + (DK & 1)) * 4 + sizeof(Gates64);
}
constexpr size_t kPrepSmem = (kSa + kSb + 64 * 66 + 64 * 3) * 4;
constexpr size_t kChunkSmem = (kSa + kSb + 64 * 66) * 4 + sizeof(Gates64);
constexpr size_t kOutSmem = (kSa + kSb) * 4 + sizeof(Gates64);
constexpr size_t kGradSmem = (kSa + kSb + 2 * 64 * 65 + 5 * 64 + 64 * 17 + 64 + 128) * 4;

template <typename T>
cudaError_t prep(const GdnProblem& p, const GdnInputs& x, const Ws& w, cudaStream_t st) {
  cudaError_t e = allow_smem(gdn_simt_prep<T>, kPrepSmem);
  if (e != cudaSuccess) return e;
  gdn_simt_prep<T><<<dim3(chunks_of(p.T), p.BH), kThreads, kPrepSmem, st>>>(
      p, (const T*)x.Q, (const T*)x.K, x.g, x.beta, w);
  return cudaGetLastError();
}

// A recurrence is bound by the latency of its products (10 us a chunk of 128 x 32
// state columns, an SM 9% busy), so that its columns are spread over twice the
// blocks, 16 each, while those still find free SMs.
template <typename T, bool kRev>
cudaError_t chain(const GdnProblem& p, const GdnInputs& x, const float* init, float* fin, T* dV,
                  const Ws& w, cudaStream_t st) {
  auto go = [&](auto* kern, int cols) {
    const cudaError_t e = allow_smem(kern, chain_smem(1024));  // the widest key's
    if (e != cudaSuccess) return e;
    kern<<<dim3((p.DV + cols - 1) / cols, p.BH), kThreads, chain_smem(p.DK), st>>>(
        p, (const T*)x.K, x.beta, init, fin, dV, w);
    return cudaGetLastError();
  };
  if ((long)p.BH * ((p.DV + 15) / 16) <= 148) return go(&gdn_simt_chain<T, kRev, 1>, 16);
  return go(&gdn_simt_chain<T, kRev, 2>, 32);
}

// prep and chunk quantities, then the forward recurrence
template <typename T, bool kBw>
cudaError_t states(const GdnProblem& p, const GdnInputs& x, const void* dH, float* C_T, const Ws& w,
                   cudaStream_t st) {
  cudaError_t e = prep<T>(p, x, w, st);
  if (e != cudaSuccess) return e;
  if ((e = allow_smem(gdn_simt_chunk<T, kBw>, kChunkSmem)) != cudaSuccess) return e;
  gdn_simt_chunk<T, kBw><<<dim3(chunks_of(p.T), p.BH), kThreads, kChunkSmem, st>>>(
      p, (const T*)x.Q, (const T*)x.K, (const T*)x.V, x.beta, (const T*)dH, w);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return chain<T, false>(p, x, x.C0, C_T, nullptr, w, st);
}

template <typename T>
cudaError_t fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T, void* ws,
               cudaStream_t st) {
  const Ws w = layout(p, false, static_cast<char*>(ws));
  cudaError_t e = states<T, false>(p, x, nullptr, C_T, w, st);
  if (e != cudaSuccess) return e;
  if ((e = allow_smem(gdn_simt_out<T>, kOutSmem)) != cudaSuccess) return e;
  gdn_simt_out<T><<<dim3(chunks_of(p.T), (p.DV + 63) / 64, p.BH), kThreads, kOutSmem, st>>>(
      p, (const T*)x.Q, x.beta, (T*)H, w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
               cudaStream_t st) {
  const Ws w = layout(p, true, static_cast<char*>(ws));
  const dim3 chunks(chunks_of(p.T), p.BH);
  cudaError_t e = states<T, true>(p, x, d.dH, nullptr, w, st);
  if (e != cudaSuccess) return e;
  if ((e = chain<T, true>(p, x, d.dC_T, d.dC0, (T*)d.dV, w, st)) != cudaSuccess) return e;
  if ((e = allow_smem(gdn_simt_grads<T>, kGradSmem)) != cudaSuccess) return e;
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
  return backward ? 5 + (p.group > 1) : 4;
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
