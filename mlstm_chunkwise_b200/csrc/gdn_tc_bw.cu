// Gated delta rule on the tensor cores: gradients (formulas in gdn.h).  Three
// kernels, each for all chunks in parallel, around the reverse recurrence:
//   dz0    Tinv^T (beta scale (Gam . QK^T)^T dH) and N' of the reverse recurrence
//   dz     dz = dz0 + Tinv^T (beta D K dS') and dV, from the gradient of the state
//   grads  dQ, dK, dg and dbeta
// The first two are persistent, one block of 512 threads per SM on up to 128
// value columns, thread (r, h) on columns 32 h .. of row r: rounds of products
// with a pass through registers after each.  The third holds one chunk's operands
// (208 KB) and five 128 x 128 accumulators in turn in all of the tensor memory:
// about 90 products of 128 x 128 x 64 for 128 value columns.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr long kSms = 148;

// (bh, chunk, pair of value tiles) of a persistent kernel's item.
struct Item {
  size_t cb;
  int bh, t0, n, vt, tiles;
  __device__ Item(long i, const GdnProblem& p, const GdnTcWs& w) {
    const int pairs = (w.nvt + 1) / 2;
    cb = (size_t)(i / pairs);
    vt = (int)(i % pairs) * 2;
    tiles = min(2, w.nvt - vt);
    bh = (int)(cb / w.NC);
    t0 = (int)(cb % w.NC) * kGdnL;
    n = min(kGdnL, p.T - t0);
  }
};
inline long items_of(const GdnProblem& p, const GdnTcWs& w) {
  return (long)p.BH * w.NC * ((w.nvt + 1) / 2);
}

// ---------------------------------------------------------------- dz0, N'
// Tensor memory: K Q^T then (Gam . QK^T)^T [0, 128), Tinv^T [128, 256), w0 then
// dz0 [256, 384), N' [384, 512).  The last operand of N', scale Lam dH, has three
// terms: two go under the first round, the third under the third.
constexpr uint32_t kZDh = 4 * kBlk, kZL = 6 * kBlk, kZW = 10 * kBlk;
constexpr uint32_t kZGc = 14 * kBlk;
constexpr uint32_t kZCol = kZGc + 1024;  // float[128]: the columns' factors
constexpr uint32_t kZBar = kZCol + 512;
constexpr uint32_t kZSmem = kZBar + 64;
static_assert(kZSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ void put_n(float4* dst, const uint32_t (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    dst[e * 128] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                               __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
}

__global__ void __launch_bounds__(kThreads, 1)
gdn_tc_dz0_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_dh, GdnProblem p,
                  const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kZGc);
  float* scol = reinterpret_cast<float*>(smem + kZCol);
  const uint32_t qa = sbase, ka = sbase + 2 * kBlk, ha = sbase + kZDh, la = sbase + kZL,
                 wa = sbase + kZW;
  const uint32_t bar_qk = sbase + kZBar, bar_h = bar_qk + 8, bar = bar_qk + 16;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kZBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};
  auto load_qk = [&](const Item& x) {
    mbar_expect_tx(bar_qk, 2 * slabs * kBlk);
    const int kh = gdn_key_head(p, x.bh);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, kh, bar_qk);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, x.t0, kh, bar_qk);
    }
  };
  auto load_dh = [&](const Item& x) {
    mbar_expect_tx(bar_h, x.tiles * kBlk);
    for (int v = 0; v < x.tiles; ++v)
      tma_load_3d(ha + v * kBlk, &tm_dh, (x.vt + v) * 64, x.t0, x.bh, bar_h);
  };
  uint4 ti[8];
  float2 ngc;
  float nbt;
  auto load_rows = [&](const Item& x) {
    load_tinv(w.tinvt + x.cb * 32 * 128, r, h, h >= q, ti);
    ngc = w.gc[x.cb * kGdnL + r];
    nbt = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  Item x(blockIdx.x, p, w);
  if (tid == 0) {
    mbar_init(bar_qk, 1);
    mbar_init(bar_h, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    load_qk(x);
    load_dh(x);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  load_rows(x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  const uint32_t at = (h >> 1) * kBlk;  // this thread's value tile in an image
  bool ok = true;
  uint32_t phase = 0, in_phase = 0;

  for (long i = blockIdx.x; i < items; i += gridDim.x, in_phase ^= 1) {
    const bool more = i + gridDim.x < items;
    const Item nx(more ? i + gridDim.x : i, p, w);
    const bool cols = h < 2 * x.tiles;
    const uint32_t id = idesc_bf16(128, x.tiles * 64, 0, 1), idt = idesc_bf16(128, x.tiles * 64, 1, 1);
    const float2 gr = ngc;
    const float bt = nbt, lam = gdn_exp(gr), sl = p.scale * lam;
    if (h == 0) {
      gc[r] = gr;
      scol[r] = gdn_col_factor(gr, 0);
    }
    add_identity(r, h, ti);
    put_tinv(tlane + 128, h, ti);
    if (more) load_rows(nx);
    uint4 dh[4];
    run_mma(
        bar, phase, ok, wt, 0x71,
        [&] {
          ok = mbar_wait(bar_qk, in_phase, wt, 0x70);
          tc_fence_after();
          if (ok) mma_ss<false, false>(tmem, ka, qa, idesc_bf16(128, 128, 0, 0), slabs, true);
        },
        [&] {
          if (ok) ok = mbar_wait(bar_h, in_phase, wt, 0x6e);
          if (!cols) return;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            dh[cc] = *reinterpret_cast<const uint4*>(smem + kZDh + at +
                                                     sw128_offset(r, (h & 1) * 4 + cc));
            float y[8];
            unpack8(dh[cc], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= sl;
            put8(smem + kZL + at, 2 * kBlk, r, (h & 1) * 4 + cc, y);
          }
        });
    uint32_t v[32];
    {  // row s of (Gam . QK^T)^T: 32 queries; terms take the scores' columns
      uint32_t hi[16], lo[16];
      if (h >= q) {
        tmem_ld32(trow, v);
        tmem_wait_ld();
        float g[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) g[e] = __uint_as_float(v[e]);
        if (h == q) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            g[e] = e >= lane ? gdn_decay(gc[h * 32 + e], gr) * g[e] : 0.f;
        } else {
          const float f = gdn_decay(gc[h * 32], gr);
#pragma unroll
          for (int e = 0; e < 32; ++e) g[e] *= f * scol[h * 32 + e];
        }
        split_pack<32>(g, hi, lo);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
      }
      tmem_st16(trow, hi);
      tmem_st16(trow + 16, lo);
    }
    run_mma(bar, phase, ok, wt, 0x72, [&] {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(tmem + 256, tmem + (kk >> 1) * 32 + t * 16 + (kk & 1) * 8, mnmaj(ha, kk), id,
                      (t | kk) != 0);
      for (int t = 0; t < 2; ++t)
        mma_ss<true, true>(tmem + 384, qa, la + 2 * t * kBlk, idt, 2, t == 0);
    });
    if (tid == 0 && more && ok) load_dh(nx);
    auto put = [&](float f) {  // f times the 32 columns in v
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = f * __uint_as_float(v[8 * cc + e]);
        put8(smem + kZW + at, 2 * kBlk, r, (h & 1) * 4 + cc, y);
      }
    };
    if (cols) {
      tmem_ld32(trow + 256, v);
      tmem_wait_ld();
      put(p.scale * bt);
    }
    run_mma(
        bar, phase, ok, wt, 0x73,
        [&] { mma_terms3(tmem + 256, tmem + 128, wa, 2 * kBlk, id); },
        [&] {
          if (!cols) return;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            float y[8];
            unpack8(dh[cc], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = third(y[e] * sl);
            put8_one(smem + kZL + at, r, (h & 1) * 4 + cc, y);
          }
        });
    const size_t nb = ((x.cb * w.nvt + x.vt + (h >> 1)) * 16 + (h & 1) * 8) * 128 + r;
    if (cols) {
      tmem_ld32(trow + 256, v);
      tmem_wait_ld();
      put_n(w.dz0 + nb, v);
      put(-lam);
    }
    run_mma(bar, phase, ok, wt, 0x74, [&] {
      for (int t = 0; t < 2; ++t) mma_ss<true, true>(tmem + 384, ka, wa + 2 * t * kBlk, idt, 2, false);
      mma_ss<true, true>(tmem + 384, qa, la, idt, 2, false);
    });
    if (tid == 0 && more && ok) load_qk(nx);
    if (cols) {
      tmem_ld32(trow + 384, v);
      tmem_wait_ld();
      put_n(w.N + nb, v);
    }
    x = nx;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dz, dV
// Tensor memory: Tinv^T [0, 128), K dS' [128, 256), dz [256, 384).
constexpr uint32_t kYDs = 2 * kBlk, kYW = 8 * kBlk, kYDv = 12 * kBlk, kYBar = 14 * kBlk;
constexpr uint32_t kYSmem = kYBar + 64;

__global__ void __launch_bounds__(kThreads, 1)
gdn_tc_dz_kernel(const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_dv, GdnProblem p,
                 const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ka = sbase, da = sbase + kYDs, wa = sbase + kYW;
  const uint32_t bar_in = sbase + kYBar, bar = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kYBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};
  auto load_tiles = [&](const Item& x) {
    mbar_expect_tx(bar_in, slabs * (kBlk + x.tiles * 3 * 8192));
    const int kh = gdn_key_head(p, x.bh);
    for (int s = 0; s < slabs; ++s) tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, kh, bar_in);
    for (int v = 0; v < x.tiles; ++v)
      for (int t = 0; t < 3; ++t)
        bulk_load(da + (2 * t + v) * kBlk, w.dS + ((x.cb * w.nvt + x.vt + v) * 3 + t) * kBlk,
                  slabs * 8192, bar_in);
  };
  uint4 ti[8];
  float2 ngc, ngl;
  float nbt;
  auto load_rows = [&](const Item& x) {
    load_tinv(w.tinvt + x.cb * 32 * 128, r, h, h >= q, ti);
    ngc = w.gc[x.cb * kGdnL + r];
    ngl = w.gc[x.cb * kGdnL + kGdnL - 1];
    nbt = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  Item x(blockIdx.x, p, w);
  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    load_tiles(x);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  load_rows(x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  uint8_t* img = smem + kYW + (h >> 1) * kBlk;
  bool ok = true;
  uint32_t phase = 0, in_phase = 0;

  for (long i = blockIdx.x; i < items; i += gridDim.x) {
    const bool more = i + gridDim.x < items;
    const Item nx(more ? i + gridDim.x : i, p, w);
    const bool cols = h < 2 * x.tiles;
    const uint32_t id = idesc_bf16(128, x.tiles * 64, 0, 1);
    const size_t ct = x.cb * w.nvt + x.vt + (h >> 1);
    const float dec = gdn_decay(ngl, ngc), bd = nbt * dec;
    add_identity(r, h, ti);
    put_tinv(tlane, h, ti);
    if (more) load_rows(nx);
    uint4 yh[4], yl[4];
    if (cols) {  // y of this thread's columns, both terms
      const uint8_t* src = w.y + ct * 2 * kBlk;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        const uint32_t off = sw128_offset(r, (h & 1) * 4 + cc);
        yh[cc] = *reinterpret_cast<const uint4*>(src + off);
        yl[cc] = *reinterpret_cast<const uint4*>(src + kBlk + off);
      }
    }
    if (tid == 0) tma_store_wait_read_all();  // dz of the item before has left
    run_mma(bar, phase, ok, wt, 0x76, [&] {
      ok = mbar_wait(bar_in, in_phase, wt, 0x79);
      tc_fence_after();
      if (!ok) return;
      for (int t = 0; t < 3; ++t)
        mma_ss<false, true>(tmem + 128, ka, da + 2 * t * kBlk, id, slabs, t == 0);
    });
    in_phase ^= 1;
    if (tid == 0 && more && ok) load_tiles(nx);
    uint32_t v[32];
    float4 z0[8];
    if (cols) {
      tmem_ld32(trow + 128, v);
      tmem_wait_ld();
      float o = 0.f;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float a[8], b[8];
        unpack8(yh[cc], a);
        unpack8(yl[cc], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xd = __uint_as_float(v[8 * cc + e]);
          o = fmaf(a[e] + b[e], xd, o);
          a[e] = bd * xd;
        }
        put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, a);
      }
      w.out[ct * 256 + (h & 1) * 128 + r] = dec * o;
      const float4* zp = w.dz0 + (ct * 16 + (h & 1) * 8) * 128 + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[e] = zp[e * 128];
    }
    run_mma(bar, phase, ok, wt, 0x78, [&] { mma_terms3(tmem + 256, tmem, wa, 2 * kBlk, id); });
    if (cols) {
      tmem_ld32(trow + 256, v);
      tmem_wait_ld();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        const float4 a = z0[2 * cc], b = z0[2 * cc + 1];
        float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += __uint_as_float(v[8 * cc + e]);
        put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, y);
        *reinterpret_cast<uint4*>(smem + kYDv + (h >> 1) * kBlk +
                                  sw128_offset(r, (h & 1) * 4 + cc)) = pack8(y);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {  // every thread has read its part of dz0, which dz replaces
      for (int t = 0; t < x.tiles; ++t)
        for (int term = 0; term < 2; ++term)
          bulk_store(w.dz + ((x.cb * w.nvt + x.vt + t) * 2 + term) * kBlk,
                     wa + (2 * term + t) * kBlk, kBlk);
      if (ok)  // rows past T and columns past d_v are clipped
        for (int t = 0; t < x.tiles; ++t)
          tma_store_3d(&tm_dv, sbase + kYDv + t * kBlk, (x.vt + t) * 64, x.t0, x.bh);
      tma_store_commit();
    }
    x = nx;
  }
  if (tid == 0) tma_store_wait_all();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
      gdn_tc_dz0_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kZSmem);
  if (e != cudaSuccess) return e;
  const long n = items_of(p, w);
  gdn_tc_dz0_kernel<<<(unsigned)(n < kSms ? n : kSms), kThreads, kZSmem, st>>>(tq, tk, th, p, x.beta,
                                                                              w);
  return cudaGetLastError();
}

cudaError_t launch_gdn_tc_dz(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                             const GdnTcWs& w, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, (uint64_t)p.B * p.NHK, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tv, d.dV, p.DV, p.T, p.BH, 64, kGdnL))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_tc_dz_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kYSmem);
  if (e != cudaSuccess) return e;
  const long n = items_of(p, w);
  gdn_tc_dz_kernel<<<(unsigned)(n < kSms ? n : kSms), kThreads, kYSmem, st>>>(
      tk, tv, p, x.beta, w);
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
