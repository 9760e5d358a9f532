// Gated delta rule on the tensor cores: gradients (formulas in gdn.h).  Three
// kernels, each for all chunks in parallel, around the two recurrences:
//   dz0    Tinv^T (beta scale (Gam . QK^T)^T dH) and N' of the reverse recurrence
//   ydz    y, dz = dz0 + Tinv^T (beta D K dS') and dV, from both states
//   grads  dQ, dK, dg and dbeta
// The first two are chains of dependent products with a pass through registers
// after each, bound by latency: two blocks share an SM.  The third holds one
// chunk's operands (208 KB) and five 128 x 128 accumulators in turn in all of
// the tensor memory: about 90 products of 128 x 128 x 64 for 128 value columns.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

// ---------------------------------------------------------------- dz0, N'
constexpr int kThreads = 256;
constexpr uint32_t kOffGc = 6 * kBlk;
constexpr uint32_t kOffBeta = kOffGc + 1024;
constexpr uint32_t kOffBar = kOffBeta + 512;
constexpr uint32_t kSmem = kOffBar + 64 + 1024;

__device__ __forceinline__ void put_n(float4* dst, const uint32_t (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    dst[e * 128] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                               __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
}

__global__ void __launch_bounds__(kThreads, 2)
gdn_tc_dz0_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_dh, GdnProblem p,
                  const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kOffGc);
  uint8_t* img = smem + 4 * kBlk;  // dH, then the operands made of it (two terms)
  const uint32_t qa = sbase, ka = sbase + 2 * kBlk, ia = sbase + 4 * kBlk;
  const uint32_t bar_in = sbase + kOffBar, bar = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 32);
  const int vt = blockIdx.x, c = blockIdx.y, bh = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0);
  const int slabs = (p.DK + 63) / 64;
  const size_t cb = (size_t)bh * w.NC + c;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_in, (2 * slabs + 1) * kBlk);
    const int kh = gdn_key_head(p, bh);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, kh, bar_in);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, t0, kh, bar_in);
    }
    tma_load_3d(ia, &tm_dh, vt * 64, t0, bh, bar_in);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 256);
    tmem_relinquish();
  }
  if (h == 0) gc[r] = w.gc[cb * kGdnL + r];
  const float bt = r < n ? beta[(long)bh * p.T + t0 + r] : 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
  const float2 gr = gc[r];
  const float lam = gdn_exp(gr);
  bool ok = mbar_wait(bar_in, 0, wt, 0x70);
  uint32_t phase = 0;
  constexpr uint32_t id = idesc_bf16(128, 64, 0, 1), idt = idesc_bf16(128, 64, 1, 1);
  uint4 dh[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    dh[e] = *reinterpret_cast<const uint4*>(img + sw128_offset(r, h * 4 + e));

  run_mma(bar, phase, ok, wt, 0x71, [&] {
    mma_ss<false, false>(tmem, ka, qa, idesc_bf16(128, 128, 0, 0), slabs, true);
  });
  uint32_t v[32];
  // row s of (Gam . QK^T)^T: queries 64 h .. ; terms take the scores' columns
  if (h * 64 + 63 >= q * 32) {
    float x[64];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      tmem_ld32(trow + h * 64 + b * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int t = h * 64 + b * 32 + e;
        x[b * 32 + e] = t >= r ? gdn_decay(gc[t], gr) * __uint_as_float(v[e]) : 0.f;
      }
    }
    uint32_t hi[32], lo[32];
    split_pack<64>(x, hi, lo);
    tmem_st32(trow + h * 64, hi);
    tmem_st32(trow + h * 64 + 32, lo);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = 0u;
    tmem_st32(trow + h * 64, v);
    tmem_st32(trow + h * 64 + 32, v);
  }
  uint4 ti[16];
  load_tinv<true>(w.tinvt + cb * 32 * 128, r, h, 4 * q, 16, ti);
  run_mma(bar, phase, ok, wt, 0x72, [&] {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_bf16_ts(tmem + 128, tmem + (kk >> 2) * 64 + t * 32 + (kk & 3) * 8, mnmaj(ia, kk), id,
                    (t | kk) != 0);
  });
  put_tinv(trow, h, ti);
  const float wf = p.scale * bt;
  auto put = [&](float f) {  // f times the 32 columns in v
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = f * __uint_as_float(v[8 * cc + e]);
      put8(img, kBlk, r, h * 4 + cc, x);
    }
  };
  tmem_ld32(trow + 128 + h * 32, v);
  tmem_wait_ld();
  put(wf);
  run_mma(bar, phase, ok, wt, 0x73, [&] { mma_terms3(tmem + 128, tmem, ia, kBlk, id); });
  tmem_ld32(trow + 128 + h * 32, v);
  tmem_wait_ld();
  const size_t nb = ((cb * w.nvt + vt) * 16 + h * 8) * 128 + r;
  put_n(w.dz0 + nb, v);
  put(-lam);
  run_mma(bar, phase, ok, wt, 0x74, [&] {
    mma_ss<true, true>(tmem + 192, ka, ia, idt, 2, true);
    mma_ss<true, true>(tmem + 192, ka, ia + kBlk, idt, 2, false);
  });
  const float sl = p.scale * lam;
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    float x[8];
    unpack8(dh[cc], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= sl;
    put8(img, kBlk, r, h * 4 + cc, x);
  }
  run_mma(bar, phase, ok, wt, 0x75, [&] {
    mma_ss<true, true>(tmem + 192, qa, ia, idt, 2, false);
    mma_ss<true, true>(tmem + 192, qa, ia + kBlk, idt, 2, false);
  });
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    float x[8];
    unpack8(dh[cc], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = third(x[e] * sl);
    put8_one(img, r, h * 4 + cc, x);
  }
  run_mma(bar, phase, ok, wt, 0x6f,
          [&] { mma_ss<true, true>(tmem + 192, qa, ia, idt, 2, false); });
  tmem_ld32(trow + 192 + h * 32, v);
  tmem_wait_ld();
  put_n(w.N + nb, v);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- y, dz, dV
constexpr uint32_t kYBar = 7 * kBlk;
constexpr uint32_t kYSmem = kYBar + 64;

__global__ void __launch_bounds__(kThreads, 2)
gdn_tc_ydz_kernel(const __grid_constant__ CUtensorMap tm_k, GdnProblem p,
                  const float* __restrict__ beta, const __nv_bfloat16* __restrict__ V,
                  __nv_bfloat16* __restrict__ dV, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint8_t *img = smem + 2 * kBlk, *imgd = smem + 4 * kBlk;  // S, z, y; dS', its z, dz
  const uint32_t ka = sbase, ia = sbase + 2 * kBlk, da = sbase + 4 * kBlk;
  const uint32_t bar_in = sbase + kYBar, bar = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kYBar + 32);
  const int vt = blockIdx.x, c = blockIdx.y, bh = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0), v0 = vt * 64 + h * 32;
  const int slabs = (p.DK + 63) / 64;
  const size_t cb = (size_t)bh * w.NC + c, ct = cb * w.nvt + vt,
               tile = ct * 2 * kBlk;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_in, slabs * (kBlk + 5 * 8192));
    const int kh = gdn_key_head(p, bh);
    for (int s = 0; s < slabs; ++s) tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, kh, bar_in);
    for (int t = 0; t < 3; ++t) {
      if (t < 2) bulk_load(ia + t * kBlk, w.S + tile + t * kBlk, slabs * 8192, bar_in);
      bulk_load(da + t * kBlk, w.dS + (ct * 3 + t) * kBlk, slabs * 8192, bar_in);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 256);
    tmem_relinquish();
  }
  uint4 ti[16];
  load_tinv<false>(w.tinv + cb * 32 * 128, r, h, 0, 4 * (q + 1), ti);
  const size_t vb = ((size_t)bh * p.T + t0 + r) * p.DV + v0;
  uint4 vrow[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    vrow[e] = r < n && v0 + 8 * e < p.DV ? *reinterpret_cast<const uint4*>(V + vb + 8 * e)
                                         : make_uint4(0u, 0u, 0u, 0u);
  const float2 gr = w.gc[cb * kGdnL + r], gl = w.gc[cb * kGdnL + kGdnL - 1];
  const float bt = r < n ? beta[(long)bh * p.T + t0 + r] : 0.f;
  const float lam = gdn_exp(gr), dec = gdn_decay(gl, gr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
  bool ok = true;
  uint32_t phase = 0;
  constexpr uint32_t id = idesc_bf16(128, 64, 0, 1);
  put_tinv(trow, h, ti);
  run_mma(bar, phase, ok, wt, 0x76, [&] {
    ok = mbar_wait(bar_in, 0, wt, 0x79);
    tc_fence_after();
    if (!ok) return;
    for (int t = 0; t < 3; ++t) {
      if (t < 2) mma_ss<false, true>(tmem + 128, ka, ia + t * kBlk, id, slabs, t == 0);
      mma_ss<false, true>(tmem + 192, ka, da + t * kBlk, id, slabs, t == 0);
    }
  });
  uint32_t v[32];
  tmem_ld32(trow + 192 + h * 32, v);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = bt * dec * __uint_as_float(v[8 * cc + e]);
    put8(imgd, kBlk, r, h * 4 + cc, x);
  }
  float z[32];
  tmem_ld32(trow + 128 + h * 32, v);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    float x[8];
    unpack8(vrow[cc], x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      z[8 * cc + e] = fmaf(-lam, __uint_as_float(v[8 * cc + e]), x[e]);
    put8(img, kBlk, r, h * 4 + cc, z + 8 * cc);
  }
  load_tinv<true>(w.tinvt + cb * 32 * 128, r, h, 4 * q, 16, ti);
  run_mma(bar, phase, ok, wt, 0x77, [&] { mma_terms3(tmem + 128, tmem, ia, kBlk, id); });
  put_tinv(trow, h, ti);
  {
    uint32_t xd[32];
    tmem_ld32(trow + 128 + h * 32, v);
    tmem_ld32(trow + 192 + h * 32, xd);
    tmem_wait_ld();
    float o = 0.f;
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
#pragma unroll
      for (int e = 8 * cc; e < 8 * cc + 8; ++e) {
        z[e] += __uint_as_float(v[e]);
        o = fmaf(z[e], __uint_as_float(xd[e]), o);
      }
      put8(img, kBlk, r, h * 4 + cc, z + 8 * cc);
    }
    w.out[ct * 256 + h * 128 + r] = dec * o;
  }
  float4 z0[8];
  const float4* zp = w.dz0 + (ct * 16 + h * 8) * 128 + r;
#pragma unroll
  for (int e = 0; e < 8; ++e) z0[e] = zp[e * 128];
  run_mma(bar, phase, ok, wt, 0x78, [&] { mma_terms3(tmem + 192, tmem, da, kBlk, id); });
  if (tid == 0) {
    bulk_store(w.y + tile, ia, 2 * kBlk);
    tma_store_commit();
  }
  tmem_ld32(trow + 192 + h * 32, v);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    const float4 a = z0[2 * cc], b = z0[2 * cc + 1];
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += __uint_as_float(v[8 * cc + e]);
    put8(imgd, kBlk, r, h * 4 + cc, x);
    if (r < n && ok && v0 + 8 * cc < p.DV) *reinterpret_cast<uint4*>(dV + vb + 8 * cc) = pack8(x);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {  // every thread has read its part of dz0, which dz replaces
    bulk_store(w.dz + tile, da, 2 * kBlk);
    tma_store_commit();
    tma_store_wait_all();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- gradients
// 512 threads: thread (r, h) takes columns 32 h .. 32 h + 31 of row r of every
// 128 x 128 matrix.  Tensor memory:
//   [0, 128)    dH y^T over the value tiles, then QK^T
//   [128, 256)  dH S^T, scaled in place, then + (Rh beta) K: dQ
//   [256, 384)  dz S^T, combined in place with y dS'^T, then
//               + (Eh beta) K + (Rh beta)^T Q + (Eh beta)^T K: dK
//   [384, 512)  y dS'^T, then dz y^T, then KK^T
constexpr int kGThreads = 512;
constexpr uint32_t kGDh = 4 * kBlk, kGDz = 5 * kBlk, kGY = 7 * kBlk, kGS = 9 * kBlk,
                   kGDs = 11 * kBlk;
constexpr uint32_t kGR = 4 * kBlk, kGE = 8 * kBlk;  // images of Rh beta, Eh beta
constexpr uint32_t kGGc = 13 * kBlk;
constexpr uint32_t kGBeta = kGGc + 1024;
constexpr uint32_t kGRed = kGBeta + 512;          // float[3][4][128]: ent, rows, columns
constexpr uint32_t kGDiag = kGRed + 3 * 4 * 512;  // float[128]
constexpr uint32_t kGDot = kGDiag + 512;          // float[16]
constexpr uint32_t kGBar = kGDot + 64;
constexpr uint32_t kGSmem = kGBar + 64 + 1024;
static_assert(kGSmem <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(kGThreads, 1)
gdn_tc_grads_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_dh, GdnProblem p,
                    const float* __restrict__ beta, __nv_bfloat16* __restrict__ dQ,
                    __nv_bfloat16* __restrict__ dK, float* __restrict__ dg,
                    float* __restrict__ dbeta, GdnTcWs w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kGGc);
  float* sbeta = reinterpret_cast<float*>(smem + kGBeta);
  float* red = reinterpret_cast<float*>(smem + kGRed);
  float* sdiag = reinterpret_cast<float*>(smem + kGDiag);
  float* sdot = reinterpret_cast<float*>(smem + kGDot);
  const uint32_t qa = sbase, ka = sbase + 2 * kBlk;
  const uint32_t bar_in = sbase + kGBar, bar = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kGBar + 32);
  const int c = blockIdx.x, bh = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0);
  const int slabs = (p.DK + 63) / 64;
  const int kh = gdn_key_head(p, bh);
  const size_t cb = (size_t)bh * w.NC + c;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  // pieces of value tile vt: dH, y and both gradients' states; or y and dz alone
  auto load_tile = [&](int vt, bool states) {
    const size_t ct = cb * w.nvt + vt, tile = ct * 2 * kBlk;
    if (states) {
      tma_load_3d(sbase + kGDh, &tm_dh, vt * 64, t0, bh, bar_in);
      for (int t = 0; t < 2; ++t) {
        bulk_load(sbase + kGS + t * kBlk, w.S + tile + t * kBlk, slabs * 8192, bar_in);
        bulk_load(sbase + kGDs + t * kBlk, w.dS + (ct * 3 + t) * kBlk, slabs * 8192, bar_in);
      }
    }
    bulk_load(sbase + kGDz, w.dz + tile, 2 * kBlk, bar_in);
    bulk_load(sbase + kGY, w.y + tile, 2 * kBlk, bar_in);
  };
  const uint32_t all_bytes = 5 * kBlk + 4 * slabs * 8192;
  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_in, 2 * slabs * kBlk + all_bytes);
    load_tile(0, true);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, kh, bar_in);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, t0, kh, bar_in);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  if (tid < 128) {
    gc[tid] = w.gc[cb * kGdnL + tid];
    sbeta[tid] = tid < n ? beta[(long)bh * p.T + t0 + tid] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + h * 32;
  const float2 gr = gc[r], gl = gc[kGdnL - 1];
  const bool cols = h < 2 * slabs;  // this thread's columns exist in d_qk matrices
  bool ok = true;
  uint32_t phase = 0, in_phase = 0;
  constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);
  const uint32_t id_d = idesc_bf16(128, slabs * 64, 0, 0);

  // D (+)= A B^T over one block of 64 value columns, operands of two terms
  auto outer = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool a_terms, bool fresh) {
    mma_ss<false, false>(d, a, b, id, 1, fresh);
    mma_ss<false, false>(d, a, b + kBlk, id, 1, false);
    if (a_terms) mma_ss<false, false>(d, a + kBlk, b, id, 1, false);
  };
  float dot = 0.f;  // <S, dS'>
  for (int vt = 0; vt < w.nvt; ++vt) {
    if (ok) ok = mbar_wait(bar_in, in_phase, wt, 0x7b);
    in_phase ^= 1;
    run_mma(
        bar, phase, ok, wt, 0x7c,
        [&] {
          outer(tmem + 128, sbase + kGDh, sbase + kGS, id_d, false, vt == 0);
          outer(tmem + 256, sbase + kGDz, sbase + kGS, id_d, true, vt == 0);
          outer(tmem + 384, sbase + kGY, sbase + kGDs, id_d, true, vt == 0);
          outer(tmem, sbase + kGDh, sbase + kGY, id_s, false, vt == 0);
        },
        [&] {
          const int d = tid & 127;
          if (d < p.DK)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t at = sw128_offset(d, (tid >> 7) * 2 + e);
              float s[8], l[8], x[8], y[8];
              unpack8(*reinterpret_cast<const uint4*>(smem + kGS + at), s);
              unpack8(*reinterpret_cast<const uint4*>(smem + kGS + kBlk + at), l);
              unpack8(*reinterpret_cast<const uint4*>(smem + kGDs + at), x);
              unpack8(*reinterpret_cast<const uint4*>(smem + kGDs + kBlk + at), y);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot = fmaf(s[i] + l[i], x[i] + y[i], dot);
            }
        });
    if (w.nvt > 1) {
      fence_proxy_async_smem();
      __syncthreads();  // the tile has been read
      if (tid == 0) {
        const bool more = vt + 1 < w.nvt;
        mbar_expect_tx(bar_in, more ? all_bytes : 4 * kBlk);
        load_tile(more ? vt + 1 : 0, more);
      }
    }
  }
  dot = warp_sum(dot);
  if (lane == 0) sdot[warp] = dot;
  // rows of q and k against the products with the entering state; the scaled
  // products stay in place as the first terms of dQ and dK
  {
    float ent = 0.f;
    if (cols) {
      const float lam = gdn_exp(gr);
      const float fq = p.scale * lam, fo = sbeta[r] * gdn_decay(gl, gr);
      uint32_t a[32], b[32];
      auto piece = [&](uint32_t off, int cc, float* x) {
        unpack8(*reinterpret_cast<const uint4*>(smem + off + (h >> 1) * kBlk +
                                                sw128_offset(r, (h & 1) * 4 + cc)),
                x);
      };
      tmem_ld32(trow + 128, a);
      tmem_wait_ld();
      float s = 0.f;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float x[8];
        piece(0, cc, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = fq * __uint_as_float(a[8 * cc + e]);
          s = fmaf(x[e], y, s);
          a[8 * cc + e] = __float_as_uint(y);
        }
      }
      tmem_st32(trow + 128, a);
      tmem_ld32(trow + 256, a);
      tmem_ld32(trow + 384, b);
      tmem_wait_ld();
      float sz = 0.f;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float x[8];
        piece(2 * kBlk, cc, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = lam * __uint_as_float(a[8 * cc + e]), o = __uint_as_float(b[8 * cc + e]);
          sz = fmaf(x[e], y, sz);
          a[8 * cc + e] = __float_as_uint(fmaf(fo, o, -y));
        }
      }
      tmem_st32(trow + 256, a);
      ent = s - sz;
    }
    red[h * 128 + r] = ent;
  }
  // dz y^T
  for (int vt = 0; vt < w.nvt; ++vt) {
    if (w.nvt > 1) {
      if (ok) ok = mbar_wait(bar_in, in_phase, wt, 0x7d);
      in_phase ^= 1;
    }
    run_mma(bar, phase, ok, wt, 0x7e,
            [&] { outer(tmem + 384, sbase + kGDz, sbase + kGY, id_s, true, vt == 0); });
    if (vt + 1 < w.nvt && tid == 0) {
      mbar_expect_tx(bar_in, 4 * kBlk);
      load_tile(vt + 1, false);
    }
  }
  float rh[32], eh[32];
  const bool lower = h <= q;  // else all columns lie right of the diagonal
  if (lower) {
    uint32_t a[32], b[32];
    tmem_ld32(trow, a);
    tmem_ld32(trow + 384, b);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int s = h * 32 + e;
      const float f = s <= r ? gdn_decay(gr, gc[s]) : 0.f;
      rh[e] = s <= r ? p.scale * f * __uint_as_float(a[e]) : 0.f;
      eh[e] = s < r ? -f * __uint_as_float(b[e]) : 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) rh[e] = eh[e] = 0.f;
  }
  run_mma(
      bar, phase, ok, wt, 0x7f,
      [&] {
        mma_ss<false, false>(tmem, qa, ka, id_s, slabs, true);
        mma_ss<false, false>(tmem + 384, ka, ka, id_s, slabs, true);
      },
      [&] {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float x[8], y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float b = sbeta[h * 32 + 8 * cc + e];
            x[e] = rh[8 * cc + e] * b;
            y[e] = eh[8 * cc + e] * b;
          }
          put8(smem + kGR + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, x);
          put8(smem + kGE + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, y);
        }
      });
  // Z, its row sums (times beta) and column sums left of the diagonal
  {
    float row = 0.f, col = 0.f;
    if (lower) {
      uint32_t a[32], b[32];
      tmem_ld32(trow, a);
      tmem_ld32(trow + 384, b);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int s = h * 32 + e;
        float z = fmaf(rh[e], __uint_as_float(a[e]), eh[e] * __uint_as_float(b[e]));
        if (s == r) sdiag[r] = z;
        z = s < r ? z : 0.f;
        row = fmaf(z, sbeta[s], row);
        rh[e] = z;
      }
      // sums over the warp's rows: lane i ends with column i
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int e = 0; e < o; ++e) {
          const bool up = (lane & o) != 0;
          const float give = up ? rh[e] : rh[e + o], keep = up ? rh[e + o] : rh[e];
          rh[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      col = rh[0];
    }
    red[(4 + h) * 128 + r] = row;
    red[(8 + q) * 128 + h * 32 + lane] = col;
  }
  const uint32_t id_n = idesc_bf16(128, slabs * 64, 0, 1), id_t = idesc_bf16(128, slabs * 64, 1, 1);
  run_mma(
      bar, phase, ok, wt, 0x7a,
      [&] {
        const uint32_t ra = sbase + kGR, ea = sbase + kGE;
        for (int t = 0; t < 2; ++t) {
          mma_ss<false, true>(tmem + 128, ra + t * 2 * kBlk, ka, id_n, 2, false);
          mma_ss<false, true>(tmem + 256, ea + t * 2 * kBlk, ka, id_n, 2, false);
          mma_ss<true, true>(tmem + 256, ra + t * 2 * kBlk, qa, id_t, 2, false);
          mma_ss<true, true>(tmem + 256, ea + t * 2 * kBlk, ka, id_t, 2, false);
        }
      },
      [&] {
        if (warp != 0) return;
        // dg: suffix sums of what enters and of Z's rows less its columns, prefix
        // sums of what leaves; four tokens per lane
        float suf[4], pre[4], o[4], cs[4], ssuf = 0.f, spre = 0.f, dG = 0.f;
        for (int i = 0; i < kGThreads / 32; ++i) dG += sdot[i];
        dG *= gdn_exp(gl);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 4 * lane + e;
          float en = 0.f, rw = 0.f;
          o[e] = cs[e] = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            en += red[i * 128 + t];
            rw += red[(4 + i) * 128 + t];
            cs[e] += red[(8 + i) * 128 + t];
          }
          for (int i = 0; i < 2 * w.nvt; ++i) o[e] += w.out[(cb * w.nvt * 2 + i) * 128 + t];
          suf[e] = en + (rw - sbeta[t] * cs[e]);
          ssuf += suf[e];
          pre[e] = sbeta[t] * o[e];
          spre += pre[e];
        }
        float incl = ssuf, inclp = spre;  // over the lanes behind / before
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const float a = __shfl_down_sync(0xffffffffu, incl, i);
          const float b = __shfl_up_sync(0xffffffffu, inclp, i);
          if (lane + i < 32) incl += a;
          if (lane >= i) inclp += b;
        }
        float s = incl - ssuf, pr = inclp - spre, x[4];
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          s += suf[e];
          x[e] = s + dG;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 4 * lane + e;
          if (t < n) {
            dg[(long)bh * p.T + t0 + t] = x[e] + pr;
            dbeta[(long)bh * p.T + t0 + t] = o[e] + cs[e] + sdiag[t];
          }
          pr += pre[e];
        }
      });
  {
    const size_t at = ((size_t)(w.dq ? bh : kh) * p.T + t0 + r) * p.DK + h * 32;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (!cols) break;
      uint32_t a[32];
      tmem_ld32(trow + 128 + m * 128, a);
      tmem_wait_ld();
      if (r >= n || !ok) continue;
      if (w.dq) {
        float* dst = (m ? w.dk : w.dq) + at;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          if (h * 32 + e < p.DK)
            *reinterpret_cast<float4*>(dst + e) =
                make_float4(__uint_as_float(a[e]), __uint_as_float(a[e + 1]),
                            __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
      } else {
        __nv_bfloat16* dst = (m ? dK : dQ) + at;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          if (h * 32 + e < p.DK)
            *reinterpret_cast<uint4*>(dst + e) = pack8(reinterpret_cast<const float*>(a) + e);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_gdn_tc_dz0(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                              const GdnTcWs& w, cudaStream_t st) {
  CUtensorMap tq, tk, th;
  const uint64_t kheads = (uint64_t)p.B * p.NHK;
  if (!encode_tmap_bf16_3d(&tq, x.Q, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&th, d.dH, p.DV, p.T, p.BH, 64, kGdnL))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_tc_dz0_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_dz0_kernel<<<dim3(w.nvt, w.NC, p.BH), kThreads, kSmem, st>>>(tq, tk, th, p, x.beta, w);
  return cudaGetLastError();
}

cudaError_t launch_gdn_tc_ydz(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                              const GdnTcWs& w, cudaStream_t st) {
  CUtensorMap tk;
  if (!encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, (uint64_t)p.B * p.NHK, 64, kGdnL))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_tc_ydz_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kYSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_ydz_kernel<<<dim3(w.nvt, w.NC, p.BH), kThreads, kYSmem, st>>>(
      tk, p, x.beta, static_cast<const __nv_bfloat16*>(x.V), static_cast<__nv_bfloat16*>(d.dV), w);
  return cudaGetLastError();
}

cudaError_t launch_gdn_tc_grads(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                                const GdnTcWs& w, cudaStream_t st) {
  CUtensorMap tq, tk, th;
  const uint64_t kheads = (uint64_t)p.B * p.NHK;
  if (!encode_tmap_bf16_3d(&tq, x.Q, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&th, d.dH, p.DV, p.T, p.BH, 64, kGdnL))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(gdn_tc_grads_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_grads_kernel<<<dim3(w.NC, p.BH), kGThreads, kGSmem, st>>>(
      tq, tk, th, p, x.beta, static_cast<__nv_bfloat16*>(d.dQ), static_cast<__nv_bfloat16*>(d.dK),
      d.dg, d.dbeta, w);
  if ((e = cudaGetLastError()) != cudaSuccess || p.group == 1) return e;
  return launch_gdn_group_sum(p, MLSTM_DT_BF16, w.dq, w.dk, d.dQ, d.dK, st);
}

}  // namespace mlstm
