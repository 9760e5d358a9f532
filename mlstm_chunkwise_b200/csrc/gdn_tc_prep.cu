// Gated delta rule, tensor cores: what a chunk contributes before the state that
// enters it is known.  Per (bh, chunk): the sums of g, Tinv = (I + A)^{-1} with
// A_rs = Gam_rs beta_s k_r.k_s (s < r), and M and N of the state recurrence.
//
// The inverse goes by blocks.  The four 32 x 32 diagonal blocks by forward
// substitution in fp32 (a warp per block, a lane per column); then
// T21 = -T22 A21 T11 for the two 64-blocks at once and for the whole, on the
// tensor cores with both operands as two bf16 terms (A21 and T22 in tensor
// memory, T11 and A21 T11 as images).  Every element of A is formed where it is
// used, from K K^T in tensor memory.
//
// About 11 products of 128^3 per chunk and a dozen dependent passes between
// tensor memory, registers and shared memory: bound by the latency of those
// passes, so two blocks share an SM (96 KB, 256 tensor-memory columns each).
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr uint32_t kOffK = 0;             // 2 blocks
constexpr uint32_t kOffR = 32768;         // 4 blocks: [term][block]
constexpr uint32_t kOffDiag = kOffR + kBlk;  // float[4][32][kLd], while inverting
constexpr uint32_t kOffGc = kOffR + 4 * kBlk;
constexpr uint32_t kOffBeta = kOffGc + 1024;
constexpr uint32_t kOffLam = kOffBeta + 512;
constexpr uint32_t kOffBar = kOffLam + 512;
constexpr uint32_t kSmem = kOffBar + 64 + 1024;
constexpr int kLd = 36;       // floats per row of a diagonal block
constexpr uint32_t kBi = 8192;  // lo term of the inversion's images (64 rows)

__global__ void __launch_bounds__(kThreads, 2)
gdn_tc_prep_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   GdnProblem p, const float* __restrict__ g, const float* __restrict__ beta,
                   GdnTcWs w, int transposed) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kOffGc);
  float* sbeta = reinterpret_cast<float*>(smem + kOffBeta);
  float* slam = reinterpret_cast<float*>(smem + kOffLam);
  uint8_t* img = smem + kOffR;
  const uint32_t ka = sbase + kOffK, ra = sbase + kOffR;
  const uint32_t bar_k = sbase + kOffBar, bar = bar_k + 8, bar_v = bar_k + 16;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 32);
  const int c = blockIdx.x, bh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0);
  const int slabs = (p.DK + 63) / 64;
  const size_t cb = (size_t)bh * w.NC + c;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (tid == 0) {
    mbar_init(bar_k, 1);
    mbar_init(bar, 1);
    mbar_init(bar_v, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_k, slabs * kBlk);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, gdn_key_head(p, bh), bar_k);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 256);
    tmem_relinquish();
  }
  if (warp == 2) gdn_chunk_sums(g + (long)bh * p.T + t0, n, lane, gc, w.gc + cb * kGdnL);
  if (warp >= 4) {
    const int t = tid - 128;
    sbeta[t] = t < n ? beta[(long)bh * p.T + t0 + t] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
  bool ok = true;
  uint32_t phase = 0;

  run_mma(bar, phase, ok, wt, 0x42, [&] {
    ok = mbar_wait(bar_k, 0, wt, 0x41);
    tc_fence_after();
    constexpr uint32_t id = idesc_bf16(128, 128, 0, 0);
    if (ok) mma_ss<false, false>(tmem, ka, ka, id, slabs, true);
  });
  const float2 gr = gc[r];
  const float dec = sbeta[r] * gdn_decay(gc[kGdnL - 1], gr);
  if (h == 0) slam[r] = gdn_exp(gr);
  // 32 elements of A's row r from column s0
  auto a_row = [&](int s0, float (&x)[32]) {
    uint32_t v[32];
    tmem_ld32(trow + s0, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int s = s0 + e;
      x[e] = s < r ? gdn_decay(gr, gc[s]) * sbeta[s] * __uint_as_float(v[e]) : 0.f;
    }
  };
  // A operand of the inversion: 64 inner columns, hi at 128, lo at 160
  auto put_a32 = [&](int col, const float (&x)[32]) {
    uint32_t hi[16], lo[16];
    split_pack<32>(x, hi, lo);
    tmem_st16(trow + 128 + col, hi);
    tmem_st16(trow + 160 + col, lo);
  };
  float* diag = reinterpret_cast<float*>(smem + kOffDiag);
  float* dq = diag + q * 32 * kLd;  // [s][r] of block q
  if (h == 0) {
    // the diagonal block: column s of A at [s], then the inverse's column at [s]
    {
      float x[32];
      a_row(q * 32, x);
#pragma unroll
      for (int e = 0; e < 32; ++e) dq[e * kLd + lane] = x[e];
    }
    __syncwarp();
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
    for (int s = 0; s < 31; ++s) {
      float a[32];
#pragma unroll
      for (int r4 = (s + 1) / 4; r4 < 8; ++r4) {
        const float4 v = *reinterpret_cast<const float4*>(dq + s * kLd + r4 * 4);
        a[4 * r4] = v.x; a[4 * r4 + 1] = v.y; a[4 * r4 + 2] = v.z; a[4 * r4 + 3] = v.w;
      }
#pragma unroll
      for (int i = s + 1; i < 32; ++i) x[i] = fmaf(-a[i], x[s], x[i]);
    }
    __syncwarp();  // every lane has read the block
#pragma unroll
    for (int r4 = 0; r4 < 8; ++r4)
      *reinterpret_cast<float4*>(dq + lane * kLd + r4 * 4) =
          make_float4(x[4 * r4], x[4 * r4 + 1], x[4 * r4 + 2], x[4 * r4 + 3]);
  } else if (q & 1) {
    // A21 of the 64-blocks: inner columns 0..31 the first block's, 32..63 the second's
    float x[32];
    a_row((q - 1) * 32, x);
    put_a32(q == 3 ? 16 : 0, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = 0.f;
    put_a32(q == 3 ? 0 : 16, x);
  }
  __syncthreads();
  // the image's rows: 0..31 and 32..63 are those of diagonal blocks 0 and 2
  {
    const int kr = tid & 63, cc = tid >> 6;
    const float* d = diag + (kr >> 5) * 2 * 32 * kLd;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = d[(8 * cc + e) * kLd + (kr & 31)];
    put8(img, kBi, kr, cc, x);
    put8(img, kBi, kr, cc + 4, x);  // columns 32..63 of the product are not used
  }
  auto inv_mma = [&] {
    constexpr uint32_t id = idesc_bf16(128, 64, 0, 1);
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ts(tmem + 192, tmem + 128 + (t == 1 ? 32 : 0) + kk * 8,
                    mnmaj(ra + (t == 2 ? kBi : 0u), kk), id, (t | kk) != 0);
  };
  run_mma(bar, phase, ok, wt, 0x43, inv_mma);
  if (q & 1) {
    uint32_t v[16];
    tmem_ld16(trow + 192 + h * 16, v);
    tmem_wait_ld();
    const int kr = (q >> 1) * 32 + lane;
    put8(img, kBi, kr, h * 2, reinterpret_cast<const float*>(v));
    put8(img, kBi, kr, h * 2 + 1, reinterpret_cast<const float*>(v) + 8);
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = dq[(h * 16 + e) * kLd + lane];
    uint32_t hi[8], lo[8];
    split_pack<16>(x, hi, lo);
    tmem_st8(trow + 128 + (q >> 1) * 16 + h * 8, hi);
    tmem_st8(trow + 160 + (q >> 1) * 16 + h * 8, lo);
  }
  run_mma(bar, phase, ok, wt, 0x44, inv_mma);
  // x: columns 32 h .. of this row inside its 64-block of the inverse
  float x[32], b[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = b[e] = 0.f;
  if (h == 0 && (q & 1)) {
    uint32_t v[32];
    tmem_ld32(trow + 192, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = -__uint_as_float(v[e]);
  } else if (h == (q & 1)) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = dq[e * kLd + lane];
  }
  if (q < 2) {
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) put8(img, kBi, r, h * 4 + cc, x + 8 * cc);
  } else {
    float a[32];
    a_row(h * 32, a);
    put_a32(h * 16, a);
  }
  run_mma(bar, phase, ok, wt, 0x45, inv_mma);
  if (q >= 2) {
    uint32_t v[32];
    tmem_ld32(trow + 192 + h * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int cc = 0; cc < 4; ++cc)
      put8(img, kBi, r - 64, h * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
    put_a32(h * 16, x);
  }
  run_mma(bar, phase, ok, wt, 0x46, inv_mma);
  if (q >= 2) {
    uint32_t v[32];
    tmem_ld32(trow + 192 + h * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) b[e] = -__uint_as_float(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      b[e] = x[e];
      x[e] = 0.f;
    }
  }
  // Now b: columns 32 h .. of row r of Tinv, x: columns 64 + 32 h ..
  {
    uint4* dst = w.tinv + cb * 32 * 128 + r;
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float y[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        y[e] = 2 * half + h == q && e == lane ? 0.f : (half ? x : b)[e];
      split_pack<32>(y, hi, lo);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = half * 8 + h * 4 + i;
        const uint4 uh = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        const uint4 ul = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        if (j < 4 * (q + 1)) {
          dst[j * 128] = uh;
          dst[(16 + j) * 128] = ul;
        }
        if (transposed) {
          *reinterpret_cast<uint4*>(img + half * kBlk + sw128_offset(r, h * 4 + i)) = uh;
          *reinterpret_cast<uint4*>(img + (2 + half) * kBlk + sw128_offset(r, h * 4 + i)) = ul;
        }
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = (half ? x : b)[e] * slam[half * 64 + h * 32 + e];
      split_pack<32>(y, hi, lo);
      tmem_st16(trow + half * 32 + h * 16, hi);
      tmem_st16(trow + 64 + half * 32 + h * 16, lo);
    }
  }
  // W = (Tinv Lam) K
  const uint32_t nk = idesc_bf16(128, slabs * 64, 0, 1), nkt = idesc_bf16(128, slabs * 64, 1, 1);
  run_mma(bar, phase, ok, wt, 0x47, [&] { mma_terms2(tmem + 128, tmem, ka, nk); });
  if (transposed) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(w.tinvt + cb * 32 * 128);
    for (int i = warp; i < 128; i += 8) {
      const int term = i >> 6, sb = (i >> 2) & 15, rg = i & 3;  // 8 columns s, 32 rows r
      if (rg < sb >> 2) continue;
      uint32_t v[4];
      ldmatrix4_trans(ra + (term * 2 + (sb >> 3)) * kBlk + sw128_offset(rg * 32 + lane, sb & 7), v);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        dst[((term * 16 + rg * 4 + m) * 128 + sb * 8 + (lane >> 2)) * 4 + (lane & 3)] = v[m];
    }
    __syncthreads();
  }
  // the image of D beta (columns in tensor memory), or its third term
  auto put_scaled = [&](int blocks, bool rest) {
    for (int s = 0; s < blocks; ++s) {
      uint32_t v[32];
      tmem_ld32(trow + 128 + s * 64 + h * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = dec * __uint_as_float(v[8 * cc + e]);
        if (!rest) {
          put8(img + s * kBlk, 2 * kBlk, r, h * 4 + cc, y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = third(y[e]);
          put8_one(img + s * kBlk, r, h * 4 + cc, y);
        }
      }
    }
  };
  auto kt_mma = [&](uint32_t d, uint32_t id) {
    mma_ss<true, true>(d, ka, ra, id, 2, true);
    mma_ss<true, true>(d, ka, ra + 2 * kBlk, id, 2, false);
  };
  put_scaled(slabs, false);
  run_mma(bar, phase, ok, wt, 0x48, [&] { kt_mma(tmem + 128, nkt); });
  for (int s = 0; s < slabs; ++s) {
    uint32_t v[32];
    tmem_ld32(trow + 128 + s * 64 + h * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int cc = 0; cc < 4; ++cc)
      put8(img + s * kBlk, 2 * kBlk, r, h * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    uint8_t* dst = w.M + cb * 4 * kBlk;
    for (int t = 0; t < 2; ++t)
      bulk_store(dst + t * 2 * kBlk, ra + t * 2 * kBlk, slabs * kBlk);
    tma_store_commit();
    tma_store_wait_read_all();
  }
  // two value tiles at a time
  for (int v0 = 0; v0 < w.nvt; v0 += 2) {
    const int tiles = min(2, w.nvt - v0);
    if (tid == 0) {  // the image has been read (above, or by the last products)
      mbar_expect_tx(bar_v, tiles * kBlk);
      for (int s = 0; s < tiles; ++s)
        tma_load_3d(ra + s * kBlk, &tm_v, (v0 + s) * 64, t0, bh, bar_v);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // Tinv, which N replaces
      uint32_t hi[16], lo[16];
      split_pack<32>(half ? x : b, hi, lo);
      tmem_st16(trow + half * 32 + h * 16, hi);
      tmem_st16(trow + 64 + half * 32 + h * 16, lo);
    }
    const uint32_t nv = idesc_bf16(128, tiles * 64, 0, 1), nvt = idesc_bf16(128, tiles * 64, 1, 1);
    run_mma(bar, phase, ok, wt, 0x49, [&] {
      ok = mbar_wait(bar_v, (v0 >> 1) & 1, wt, 0x4a);
      tc_fence_after();
      if (ok) mma_terms2(tmem + 128, tmem, ra, nv);
    });
    put_scaled(tiles, false);
    run_mma(bar, phase, ok, wt, 0x4b, [&] { kt_mma(tmem, nvt); });
    put_scaled(tiles, true);
    run_mma(bar, phase, ok, wt, 0x4c, [&] { mma_ss<true, true>(tmem, ka, ra, nvt, 2, false); });
    for (int s = 0; s < tiles; ++s) {
      uint32_t v[32];
      tmem_ld32(trow + s * 64 + h * 32, v);
      tmem_wait_ld();
      float4* dst = w.N + ((cb * w.nvt + v0 + s) * 16 + h * 8) * 128 + r;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e * 128] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                   __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  if (tid == 0) tma_store_wait_all();
}

}  // namespace

cudaError_t launch_gdn_tc_prep(const GdnProblem& p, const GdnInputs& x, const GdnTcWs& w,
                               bool transposed, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, (uint64_t)p.B * p.NHK, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tv, x.V, p.DV, p.T, p.BH, 64, kGdnL))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_tc_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_prep_kernel<<<dim3(w.NC, p.BH), kThreads, kSmem, st>>>(tk, tv, p, x.g, x.beta, w,
                                                                transposed);
  return cudaGetLastError();
}

}  // namespace mlstm
