// Gated delta rule on the tensor cores: the per-chunk inverse, the forward
// recurrence fused with the output, and the path's host side.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

// ===========================================================================
// Per (bh, chunk): gc and Tinv = (I + A)^{-1}, A_rs = Gam_rs beta_s k_r.k_s.
//
// K K^T comes from tcgen05 (exact bf16 operands, fp32 sums); A^T goes to shared
// memory in fp32 and is inverted in place by blocks: the four 32 x 32 diagonal
// blocks by forward substitution (a warp per block, a lane per column), then
// T21 = -T22 A21 T11 for the two 64-blocks and for the whole.
// ===========================================================================
constexpr int kPrepThreads = 256;
constexpr int kLd = 132;  // floats per row of the transposed matrix
constexpr uint32_t kPrepMat = 128 * kLd * 4;
constexpr uint32_t kPrepOffGc = kPrepMat;                 // float2[128]
constexpr uint32_t kPrepOffBeta = kPrepOffGc + 1024;      // float[128]
constexpr uint32_t kPrepOffBar = kPrepOffBeta + 512;
constexpr uint32_t kPrepSmem = kPrepOffBar + 64 + 1024;

// m[k][r] holds element (row r, column k).  For the n x n blocks below the
// diagonal: [row0 + i][col0 + j] of the product X Y where X = block (row0,
// xcol0) and Y = block (yrow0, col0), sums over kdim.  Thread tile 4 x TN.
template <int TN>
__device__ __forceinline__ void tile_mm(const float* m, int r0, int xc0, int c0, int yr0, int k0,
                                        int k1, float (&acc)[4][TN]) {
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    const float4 a = *reinterpret_cast<const float4*>(m + (xc0 + k) * kLd + r0);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const float b = m[(c0 + j) * kLd + yr0 + k];
      acc[0][j] = fmaf(a.x, b, acc[0][j]);
      acc[1][j] = fmaf(a.y, b, acc[1][j]);
      acc[2][j] = fmaf(a.z, b, acc[2][j]);
      acc[3][j] = fmaf(a.w, b, acc[3][j]);
    }
  }
}

template <int TN>
__device__ __forceinline__ void tile_put(float* m, int r0, int c0, float sign,
                                         const float (&acc)[4][TN]) {
#pragma unroll
  for (int j = 0; j < TN; ++j)
    *reinterpret_cast<float4*>(m + (c0 + j) * kLd + r0) =
        make_float4(sign * acc[0][j], sign * acc[1][j], sign * acc[2][j], sign * acc[3][j]);
}

__global__ void __launch_bounds__(kPrepThreads, 3)
gdn_tc_prep_kernel(const __grid_constant__ CUtensorMap tm_k, GdnProblem p,
                   const float* __restrict__ g, const float* __restrict__ beta, GdnTcWs w,
                   int transposed) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* m = reinterpret_cast<float*>(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kPrepOffGc);
  float* sbeta = reinterpret_cast<float*>(smem + kPrepOffBeta);
  const uint32_t bar_k = sbase + kPrepOffBar, bar_mma = bar_k + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kPrepOffBar + 16);
  const int c = blockIdx.x, bh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0);
  const int slabs = (p.DK + 63) / 64;
  const size_t cb = (size_t)bh * w.NC + c;
  const Problem wait{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (tid == 0) {
    mbar_init(bar_k, 1);
    mbar_init(bar_mma, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_k, slabs * 16384);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(sbase + s * 16384, &tm_k, s * 64, t0, gdn_key_head(p, bh), bar_k);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 128);
    tmem_relinquish();
  }
  if (warp == 2) {  // inclusive sums of g in 64 bits, four tokens per lane
    double x[4], s = 0.;
    const float* gp = g + (long)bh * p.T + t0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * lane + e;
      s += t < n ? (double)fmaxf(gp[t], kGdnMinLogDecay) : 0.;
      x[e] = s;
    }
    double incl = s;
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double v = incl - s + x[e];
      const float hi = (float)v;
      const float2 pr = make_float2(hi, (float)(v - hi));
      gc[4 * lane + e] = pr;
      w.gc[cb * kGdnL + 4 * lane + e] = pr;
    }
  }
  if (warp >= 4) {
    const int t = tid - 128;
    sbeta[t] = t < n ? beta[(long)bh * p.T + t0 + t] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  bool ok = true;
  if (tid == 0) {
    ok = mbar_wait(bar_k, 0, wait, 0x41);
    tc_fence_after();
    constexpr uint32_t id = idesc_bf16(128, 128, 0, 0);
    if (ok)
      for (int s = 0; s < slabs; ++s)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = sdesc_sw128(sbase + s * 16384 + kk * 32, 16, 1024);
          mma_bf16_ss(tmem, d, d, id, (s | kk) != 0);
        }
    mma_commit(bar_mma);
  }
  ok = mbar_wait(bar_mma, 0, wait, 0x42) && ok;
  tc_fence_after();
  // A^T into shared memory (over K, which the product has read): thread (row r,
  // half h) takes 64 columns; blocks right of the diagonal are not needed.
  {
    const int q = warp & 3, r = q * 32 + lane, h = warp >> 2;
    const float2 gr = gc[r];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int s0 = h * 64 + b * 32;
      if (s0 > q * 32) continue;
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + s0, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int s = s0 + e;
        m[s * kLd + r] =
            s < r ? gdn_decay(gr, gc[s]) * sbeta[s] * __uint_as_float(v[e]) : 0.f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
  // diagonal 32 x 32 blocks: column `lane` of block `warp`.  Once x_s is known
  // its multiples leave all later rows (independent products).
  if (warp < 4) {
    float x[32];
    float* d = m + warp * 32 * kLd + warp * 32;
#pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = r == lane ? 1.f : 0.f;
#pragma unroll
    for (int s = 0; s < 31; ++s) {
      float a[32];
#pragma unroll
      for (int r4 = (s + 1) / 4; r4 < 8; ++r4) {
        const float4 v = *reinterpret_cast<const float4*>(d + s * kLd + r4 * 4);
        a[4 * r4] = v.x; a[4 * r4 + 1] = v.y; a[4 * r4 + 2] = v.z; a[4 * r4 + 3] = v.w;
      }
#pragma unroll
      for (int r = s + 1; r < 32; ++r) x[r] = fmaf(-a[r], x[s], x[r]);
    }
    __syncwarp();  // every lane has read the block
#pragma unroll
    for (int r4 = 0; r4 < 8; ++r4)
      *reinterpret_cast<float4*>(d + lane * kLd + r4 * 4) =
          make_float4(x[4 * r4], x[4 * r4 + 1], x[4 * r4 + 2], x[4 * r4 + 3]);
  }
  __syncthreads();
  // the two 64-blocks: 128 threads each, 32 x 32 outputs, tiles of 4 x 2
  {
    const int blk = tid >> 7, t = tid & 127, b0 = blk * 64;
    const int i0 = (t & 7) * 4, j0 = (t >> 3) * 2;
    float acc[4][2] = {};
    // A21 T11: T11 is lower triangular, columns j0.. start at row j0
    tile_mm<2>(m, b0 + 32 + i0, b0, b0 + j0, b0, j0, 32, acc);
    __syncthreads();
    tile_put<2>(m, b0 + 32 + i0, b0 + j0, 1.f, acc);
    __syncthreads();
    float out[4][2] = {};
    tile_mm<2>(m, b0 + 32 + i0, b0 + 32, b0 + j0, b0 + 32, 0, i0 + 4, out);
    __syncthreads();
    tile_put<2>(m, b0 + 32 + i0, b0 + j0, -1.f, out);
    __syncthreads();
  }
  {  // the whole: 64 x 64 outputs, tiles of 4 x 4
    const int i0 = (tid & 15) * 4, j0 = (tid >> 4) * 4;
    float acc[4][4] = {};
    tile_mm<4>(m, 64 + i0, 0, j0, 0, j0, 64, acc);
    __syncthreads();
    tile_put<4>(m, 64 + i0, j0, 1.f, acc);
    __syncthreads();
    float out[4][4] = {};
    tile_mm<4>(m, 64 + i0, 64, j0, 64, 0, i0 + 4, out);
    __syncthreads();
    tile_put<4>(m, 64 + i0, j0, -1.f, out);
    __syncthreads();
  }
  // rows (and, for the backward, columns) as bf16 terms
  {
    const int q = warp & 3, r = q * 32 + lane, h = warp >> 2;
    uint4* dst = w.tinv + cb * 32 * 128 + r;
    for (int j = h; j < 4 * (q + 1); j += 2) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 8 * j + e <= r ? m[(8 * j + e) * kLd + r] : 0.f;
      uint4 hi, lo;
      split8(x, hi, lo);
      dst[j * 128] = hi;
      dst[(16 + j) * 128] = lo;
    }
    if (transposed) {
      uint4* dt = w.tinvt + cb * 32 * 128 + r;
      for (int j = 4 * q + h; j < 16; j += 2) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(m + r * kLd + 8 * j + e);
          x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * j + e < r) x[e] = 0.f;
        uint4 hi, lo;
        split8(x, hi, lo);
        dt[j * 128] = hi;
        dt[(16 + j) * 128] = lo;
      }
    }
  }
}

// ===========================================================================
// Forward recurrence over the chunks of one (bh, 64 value columns), the state
// in TMEM.  Per chunk j:
//   X = K S                     S as a bf16 (hi, lo) operand image in smem
//   z = V - Lam X
//   Y = Tinv z                  Tinv rows in TMEM, three products
//   S = e^G S + K^T (D beta Y)
//   H = scale (Lam Q S + P Y)   P = Gam beta . Q K^T, in TMEM
// The chain X -> z -> Y -> S bounds the kernel (three dependent products with a
// pass through registers between them); the output's products fill its gaps.
// Warps (704 threads): 0 TMA producer; 1 MMA issuer; 2..9 the chain's row
// threads, two per row (state row or token), 32 columns each; 10..13 the
// output's row threads (P, H); 14..21 Tinv's terms from global memory (a chunk
// ahead, in registers) into TMEM.
// TMEM columns: S [0, 64), X and Y [64, 128), Q S [128, 192), P Y [192, 256),
// Q K^T then P [256, 384), Tinv [384, 512).
// kSave: keeps the images of S and of y for the backward (and writes no H).
// ===========================================================================
constexpr int kFwThreads = 704;
constexpr uint32_t kColS = 0, kColX = 64, kColQS = 128, kColPV = 192, kColP = 256, kColT = 384;

struct FwSmem {
  static constexpr uint32_t kK = 0;                   // 2 x 32 KB
  static constexpr uint32_t kQ = 65536;               // 32 KB
  static constexpr uint32_t kV = kQ + 32768;          // 16 KB
  static constexpr uint32_t kS = kV + 16384;          // state image, 2 x 16 KB
  static constexpr uint32_t kZ = kS + 32768;          // z, then y
  static constexpr uint32_t kU = kZ + 32768;          // D beta y
  static constexpr uint32_t kGc = kU + 32768;         // float2[2][128]
  static constexpr uint32_t kBeta = kGc + 2048;       // float[2][128]
  static constexpr uint32_t kBar = kBeta + 1024;
  static constexpr uint32_t kSlot = kBar + 256;
  static constexpr uint32_t kBytes = kSlot + 16 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
enum : uint32_t {  // barrier indexes
  kbQFull, kbQFree, kbKFull0, kbKFull1, kbKFree0, kbKFree1, kbVFull, kbVFree, kbQk, kbSop, kbX,
  kbORead, kbZ, kbT, kbY, kbYr, kbUpd, kbP, kbPv, kbIdle, kbCount
};

template <bool kSave>
__global__ void __launch_bounds__(kFwThreads, 1)
gdn_tc_fw_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, GdnProblem p,
                 const float* __restrict__ beta, const float* __restrict__ C0,
                 __nv_bfloat16* __restrict__ H, float* __restrict__ C_T, GdnTcWs w) {
  using F = FwSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](uint32_t i) { return sbase + F::kBar + 8 * i; };
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + F::kSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vt = blockIdx.x, bh = blockIdx.y, NC = w.NC;
  const int slabs = (p.DK + 63) / 64;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kbCount; ++i) {
      uint32_t n = 1;
      if (i == kbVFree || i == kbSop || i == kbZ || i == kbYr || i == kbT) n = 256;
      if (i == kbORead || i == kbP) n = 128;
      mbar_init(bar(i), n);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      const int kh = gdn_key_head(p, bh);
      for (int j = 0; j < NC && ok; ++j) {
        const int b = j & 1, t0 = j * kGdnL;
        if (j >= 2) ok = mbar_wait(bar(kbKFree0 + b), ((j >> 1) - 1) & 1, wt, 1);
        if (!ok) break;
        mbar_expect_tx(bar(kbKFull0 + b), slabs * 16384);
        for (int s = 0; s < slabs; ++s)
          tma_load_3d(sbase + F::kK + b * 32768 + s * 16384, &tm_k, s * 64, t0, kh,
                      bar(kbKFull0 + b));
        if (j >= 1) ok = mbar_wait(bar(kbVFree), (j - 1) & 1, wt, 2);
        if (!ok) break;
        mbar_expect_tx(bar(kbVFull), 16384);
        tma_load_3d(sbase + F::kV, &tm_v, vt * 64, t0, bh, bar(kbVFull));
        if (!kSave) {
          if (j >= 1) ok = mbar_wait(bar(kbQFree), (j - 1) & 1, wt, 3);
          if (!ok) break;
          mbar_expect_tx(bar(kbQFull), slabs * 16384);
          for (int s = 0; s < slabs; ++s)
            tma_load_3d(sbase + F::kQ + s * 16384, &tm_q, s * 64, t0, kh, bar(kbQFull));
        }
      }
      // the last loads of every buffer land before the CTA exits
      if (ok) {
        for (int j = NC > 2 ? NC - 2 : 0; j < NC; ++j)
          mbar_wait(bar(kbKFull0 + (j & 1)), (j >> 1) & 1, wt, 4);
        mbar_wait(bar(kbVFull), (NC - 1) & 1, wt, 4);
        if (!kSave) mbar_wait(bar(kbQFull), (NC - 1) & 1, wt, 4);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idQK = idesc_bf16(128, 128, 0, 0);  // K-major x K-major
      constexpr uint32_t idX = idesc_bf16(128, 64, 0, 1);    // K-major (or TMEM) x MN-major
      constexpr uint32_t idU = idesc_bf16(128, 64, 1, 1);    // MN-major x MN-major
      bool ok = true;
      const uint32_t qa = sbase + F::kQ, sa = sbase + F::kS, za = sbase + F::kZ, ua = sbase + F::kU;
      for (int j = 0; j < NC && ok; ++j) {
        const int b = j & 1, ph = j & 1;
        const uint32_t ka = sbase + F::kK + b * 32768;
        ok = ok && mbar_wait(bar(kbKFull0 + b), (j >> 1) & 1, wt, 5);
        if (!kSave) {
          ok = ok && mbar_wait(bar(kbQFull), ph, wt, 5);
          if (j >= 1) ok = ok && mbar_wait(bar(kbPv), (j - 1) & 1, wt, 6);  // P of j - 1 read
          tc_fence_after();
          if (!ok) break;
          for (int s = 0; s < slabs; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss(tmem + kColP, sdesc_sw128(qa + s * 16384 + kk * 32, 16, 1024),
                          sdesc_sw128(ka + s * 16384 + kk * 32, 16, 1024), idQK, (s | kk) != 0);
          mma_commit(bar(kbQk));
        }
        ok = ok && mbar_wait(bar(kbSop), ph, wt, 7);
        tc_fence_after();
        if (!ok) break;
        auto times_s = [&](uint32_t col, uint32_t a) {
          for (int term = 0; term < 2; ++term)
            for (int s = 0; s < slabs; ++s)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ss(tmem + col, sdesc_sw128(a + s * 16384 + kk * 32, 16, 1024),
                            sdesc_sw128(sa + term * kGdnImage + s * 8192 + kk * 2048, 8192, 1024),
                            idX, (term | s | kk) != 0);
        };
        times_s(kColX, ka);
        mma_commit(bar(kbX));
        if (!kSave) {
          if (j >= 1) ok = ok && mbar_wait(bar(kbORead), (j - 1) & 1, wt, 8);
          tc_fence_after();
          if (!ok) break;
          times_s(kColQS, qa);
          mma_commit(bar(kbQFree));
        }
        ok = ok && mbar_wait(bar(kbT), ph, wt, 9);
        ok = ok && mbar_wait(bar(kbZ), ph, wt, 9);
        tc_fence_after();
        if (!ok) break;
        // D = (hi + lo)(hi + lo) less lo.lo, A in TMEM (terms alo columns apart)
        auto three = [&](uint32_t col, uint32_t (*acol)(int, int), uint32_t bimg) {
#pragma unroll
          for (int t = 0; t < 3; ++t)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tmem + col, tmem + acol(t == 1, kk),
                          sdesc_sw128(bimg + (t == 2 ? kGdnImage : 0u) + kk * 2048, 8192, 1024),
                          idX, (t | kk) != 0);
        };
        three(kColX, [](int lo, int kk) -> uint32_t { return kColT + lo * 64 + kk * 8; }, za);
        mma_commit(bar(kbY));
        ok = ok && mbar_wait(bar(kbYr), ph, wt, 10);
        tc_fence_after();
        if (!ok) break;
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(tmem + kColS, sdesc_sw128(ka + kk * 2048, 16384, 1024),
                        sdesc_sw128(ua + term * kGdnImage + kk * 2048, 8192, 1024), idU, 1);
        mma_commit(bar(kbUpd));
        mma_commit(bar(kbKFree0 + b));
        if (!kSave) {
          ok = ok && mbar_wait(bar(kbP), ph, wt, 11);
          tc_fence_after();
          if (!ok) break;
          // P: the terms of keys 64 h .. 64 h + 63 in columns 64 h (hi), 64 h + 32 (lo)
          three(kColPV,
                [](int lo, int kk) -> uint32_t {
                  return kColP + (kk >> 2) * 64 + lo * 32 + (kk & 3) * 8;
                },
                za);
          mma_commit(bar(kbPv));
        }
      }
      mma_commit(bar(kbIdle));
      mbar_wait(bar(kbIdle), 0, wt, 12);
    }
  } else if (warp < 10) {
    // ------------------------------ the chain ------------------------------
    const int q = warp & 3, r = q * 32 + lane, h = (warp - 2) >> 2;
    const bool lead = threadIdx.x == 64;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + h * 32;
    const int v0 = vt * 64 + h * 32;  // first value column of this thread
    bool ok = true;
    auto load_gates = [&](int j, float2& gr, float2& gl, float& bt) {
      const float2* gp = w.gc + ((size_t)bh * NC + j) * kGdnL;
      gr = gp[r];
      gl = gp[kGdnL - 1];
      const int t = j * kGdnL + r;
      bt = t < p.T ? beta[(long)bh * p.T + t] : 0.f;
    };
    float2 gr, gl;
    float bt;
    load_gates(0, gr, gl, bt);
    for (int j = 0; j < NC && ok; ++j) {
      const int ph = j & 1;
      const size_t img = (((size_t)bh * NC + j) * w.nvt + vt) * 2 * kGdnImage;
      // the state entering the chunk: operand image, and the decayed master
      {
        uint32_t v[32];
        if (j == 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v[e] = __float_as_uint(C0 && r < p.DK && v0 + e < p.DV
                                       ? C0[((long)bh * p.DK + r) * p.DV + v0 + e]
                                       : 0.f);
        } else {
          ok = ok && mbar_wait(bar(kbUpd), (j - 1) & 1, wt, 13);
          tc_fence_after();
          tmem_ld32(trow + kColS, v);
          tmem_wait_ld();
          if (kSave) {  // the store of the last image has read it
            if (lead) tma_store_wait_read_all();
            named_bar_sync(1, 256);
          }
        }
#pragma unroll
        for (int cch = 0; cch < 4; ++cch)
          put8(smem + F::kS, r, h * 4 + cch, reinterpret_cast<const float*>(v) + 8 * cch);
        const float eg = expf(gl.x + gl.y);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(eg * __uint_as_float(v[e]));
        tmem_st32(trow + kColS, v);
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kbSop));
        if (kSave) {
          named_bar_sync(1, 256);
          if (lead) {
            bulk_store(w.S + img, sbase + F::kS, slabs * 8192);
            bulk_store(w.S + img + kGdnImage, sbase + F::kS + kGdnImage, slabs * 8192);
            tma_store_commit();
          }
        }
      }
      const float lam = expf(gr.x + gr.y), dec = bt * gdn_decay(gl, gr);
      float2 gr2 = gr, gl2 = gl;
      float bt2 = bt;
      if (j + 1 < NC) load_gates(j + 1, gr2, gl2, bt2);
      // z = V - Lam X
      {
        uint32_t v[32];
        ok = ok && mbar_wait(bar(kbVFull), ph, wt, 14);
        ok = ok && mbar_wait(bar(kbX), ph, wt, 15);
        if (!kSave && j >= 1) ok = ok && mbar_wait(bar(kbPv), (j - 1) & 1, wt, 16);  // y read
        tc_fence_after();
        tmem_ld32(trow + kColX, v);
        tmem_wait_ld();
#pragma unroll
        for (int cch = 0; cch < 4; ++cch) {
          const uint4 u = *reinterpret_cast<const uint4*>(smem + F::kV + sw128_offset(r, h * 4 + cch));
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] = fmaf(-lam, __uint_as_float(v[8 * cch + 2 * e]), __uint_as_float(uu[e] << 16));
            x[2 * e + 1] = fmaf(-lam, __uint_as_float(v[8 * cch + 2 * e + 1]),
                                __uint_as_float(uu[e] & 0xffff0000u));
          }
          put8(smem + F::kZ, r, h * 4 + cch, x);
        }
        mbar_arrive(bar(kbVFree));
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kbZ));
      }
      // y, and D beta y for the state
      {
        uint32_t v[32];
        ok = ok && mbar_wait(bar(kbY), ph, wt, 17);
        tc_fence_after();
        tmem_ld32(trow + kColX, v);
        tmem_wait_ld();
#pragma unroll
        for (int cch = 0; cch < 4; ++cch) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[8 * cch + e]);
          put8(smem + F::kZ, r, h * 4 + cch, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= dec;
          put8(smem + F::kU, r, h * 4 + cch, x);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kbYr));
        if (kSave) {
          named_bar_sync(1, 256);
          if (lead) {
            bulk_store(w.y + img, sbase + F::kZ, 2 * kGdnImage);
            tma_store_commit();
          }
        }
      }
      gr = gr2;
      gl = gl2;
      bt = bt2;
    }
    if (C_T) {
      ok = ok && mbar_wait(bar(kbUpd), (NC - 1) & 1, wt, 18);
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(trow + kColS, v);
      tmem_wait_ld();
      if (r < p.DK && ok)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (v0 + e < p.DV) C_T[((long)bh * p.DK + r) * p.DV + v0 + e] = __uint_as_float(v[e]);
    }
    if (kSave && lead) tma_store_wait_all();
  } else if (warp < 14) {
    // ------------------------------ the output ------------------------------
    if (!kSave) {
      const int q = warp & 3, r = q * 32 + lane, rt = threadIdx.x - 320;
      const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
      float2* sgc = reinterpret_cast<float2*>(smem + F::kGc);
      float* sbt = reinterpret_cast<float*>(smem + F::kBeta);
      bool ok = true;
      auto load_gates = [&](int j, float2& gv, float& bv) {
        gv = w.gc[((size_t)bh * NC + j) * kGdnL + rt];
        const int t = j * kGdnL + rt;
        bv = t < p.T ? beta[(long)bh * p.T + t] : 0.f;
      };
      float2 gn;
      float bn;
      load_gates(0, gn, bn);
      for (int j = 0; j < NC && ok; ++j) {
        const int ph = j & 1;
        float2* gcs = sgc + ph * 128;
        float* bts = sbt + ph * 128;
        gcs[rt] = gn;
        bts[rt] = bn;
        if (j + 1 < NC) load_gates(j + 1, gn, bn);
        named_bar_sync(2, 128);
        const float2 gr = gcs[r];
        ok = ok && mbar_wait(bar(kbQk), ph, wt, 19);
        tc_fence_after();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t keep[16];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int s0 = hh * 64 + b * 32;
            uint32_t hi[16], lo[16];
            if (s0 <= q * 32) {
              uint32_t v[32];
              tmem_ld32(trow + kColP + s0, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int s = s0 + e + i;
                  x[i] = s <= r ? gdn_decay(gr, gcs[s]) * bts[s] * __uint_as_float(v[e + i]) : 0.f;
                }
                uint4 a, c;
                split8(x, a, c);
                hi[e / 2] = a.x; hi[e / 2 + 1] = a.y; hi[e / 2 + 2] = a.z; hi[e / 2 + 3] = a.w;
                lo[e / 2] = c.x; lo[e / 2 + 1] = c.y; lo[e / 2 + 2] = c.z; lo[e / 2 + 3] = c.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
            }
            // 32 scores become 16 + 16 columns: the lo of the first batch waits
            // until the second's scores have been read
            tmem_st16(trow + kColP + hh * 64 + b * 16, hi);
            if (b == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) keep[e] = lo[e];
            } else {
              tmem_st16(trow + kColP + hh * 64 + 32, keep);
              tmem_st16(trow + kColP + hh * 64 + 48, lo);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kbP));
        const float lam = p.scale * expf(gr.x + gr.y);
        ok = ok && mbar_wait(bar(kbPv), ph, wt, 20);
        tc_fence_after();
        const int t = j * kGdnL + r;
        __nv_bfloat16* hp = H + ((long)bh * p.T + t) * p.DV + vt * 64;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t a[32], o[32];
          tmem_ld32(trow + kColQS + b * 32, a);
          tmem_ld32(trow + kColPV + b * 32, o);
          tmem_wait_ld();
          if (b == 1) {
            tc_fence_before();
            mbar_arrive(bar(kbORead));
          }
          if (t < p.T && ok)
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                u[i] = pack_bf16x2(fmaf(lam, __uint_as_float(a[e + 2 * i]),
                                        p.scale * __uint_as_float(o[e + 2 * i])),
                                   fmaf(lam, __uint_as_float(a[e + 2 * i + 1]),
                                        p.scale * __uint_as_float(o[e + 2 * i + 1])));
              if (vt * 64 + b * 32 + e < p.DV)
                *reinterpret_cast<uint4*>(hp + b * 32 + e) = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
      }
    }
  } else {
    // ----------------------------- Tinv loads ------------------------------
    const int q = warp & 3, r = q * 32 + lane, term = (warp - 14) >> 2;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + kColT + term * 64;
    uint4 t[16];
    auto load = [&](int j) {
      const uint4* src = w.tinv + (((size_t)bh * NC + j) * 32 + term * 16) * 128 + r;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < 4 * (q + 1)) t[i] = src[i * 128];
    };
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = make_uint4(0u, 0u, 0u, 0u);
    load(0);
    bool ok = true;
    for (int j = 0; j < NC && ok; ++j) {
      if (j >= 1) ok = mbar_wait(bar(kbY), (j - 1) & 1, wt, 21);  // Tinv of j - 1 read
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j == 0 || i <= q) {  // blocks right of the diagonal stay zero
          const uint32_t v[16] = {t[4 * i].x,     t[4 * i].y,     t[4 * i].z,     t[4 * i].w,
                                  t[4 * i + 1].x, t[4 * i + 1].y, t[4 * i + 1].z, t[4 * i + 1].w,
                                  t[4 * i + 2].x, t[4 * i + 2].y, t[4 * i + 2].z, t[4 * i + 2].w,
                                  t[4 * i + 3].x, t[4 * i + 3].y, t[4 * i + 3].z, t[4 * i + 3].w};
          tmem_st16(trow + i * 16, v);
        }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kbT));
      if (j + 1 < NC) load(j + 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr size_t round256(size_t x) { return (x + 255) / 256 * 256; }

GdnTcWs layout(const GdnProblem& p, bool bw, char* base) {
  GdnTcWs w{};
  w.NC = gdn_tc_chunks(p);
  w.nvt = (p.DV + 63) / 64;
  const size_t nc = (size_t)p.BH * w.NC;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + at : nullptr;
    at += round256(bytes);
    return r;
  };
  w.gc = reinterpret_cast<float2*>(take(nc * kGdnL * sizeof(float2)));
  w.tinv = reinterpret_cast<uint4*>(take(nc * 32 * 128 * sizeof(uint4)));
  w.bytes = at;
  return w;
}

cudaError_t launch_prep(const GdnProblem& p, const GdnInputs& x, const GdnTcWs& w, bool transposed,
                        cudaStream_t st) {
  CUtensorMap tk;
  if (!encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, (uint64_t)p.B * p.NHK, 64, kGdnL))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(gdn_tc_prep_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_prep_kernel<<<dim3(w.NC, p.BH), kPrepThreads, kPrepSmem, st>>>(tk, p, x.g, x.beta, w,
                                                                        transposed);
  return cudaGetLastError();
}

template <bool kSave>
cudaError_t launch_chain(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                         const GdnTcWs& w, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  const uint64_t kheads = (uint64_t)p.B * p.NHK;
  if (!encode_tmap_bf16_3d(&tq, x.Q, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tv, x.V, p.DV, p.T, p.BH, 64, kGdnL))
    return cudaErrorInvalidValue;
  auto kern = gdn_tc_fw_kernel<kSave>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FwSmem::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<dim3(w.nvt, p.BH), kFwThreads, FwSmem::kBytes, st>>>(
      tq, tk, tv, p, x.beta, x.C0, static_cast<__nv_bfloat16*>(H), C_T, w);
  return cudaGetLastError();
}

}  // namespace

bool gdn_tc_supported(const GdnProblem& p) {
  return p.DK <= 128 && p.DK % 8 == 0 && p.DV % 8 == 0;
}

size_t gdn_tc_workspace(const GdnProblem& p, bool backward) {
  return layout(p, backward, nullptr).bytes;
}

int gdn_tc_launches(const GdnProblem& p, bool backward) { return backward ? 4 + (p.group > 1) : 2; }

cudaError_t launch_gdn_tc_fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                             void* ws, cudaStream_t st) {
  const GdnTcWs w = layout(p, false, static_cast<char*>(ws));
  const cudaError_t e = launch_prep(p, x, w, false, st);
  if (e != cudaSuccess) return e;
  return launch_chain<false>(p, x, H, C_T, w, st);
}

}  // namespace mlstm
