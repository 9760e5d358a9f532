// Gated delta rule on the tensor cores: gradients (formulas in gdn.h).  Three
// kernels, each for all chunks in parallel, around the reverse recurrence:
//   dz0    Tinv^T (beta scale (Gam . QK^T)^T dH) and N' of the reverse recurrence
//   dz     dz = dz0 + Tinv^T (beta D K dS') and dV, from the gradient of the state
//   grads  dQ, dK, dg and dbeta
// The first two are persistent, one block per SM on up to 128 value columns:
// rounds of products with a pass through registers after each.  The third works on
// one chunk's operands with six 128 x 128 accumulators in turn in all of the
// tensor memory: 184 products of 128 x 128 x 16 for 128 value columns.
//
// 1024 chunks of 128 x 128: dz0 94 us (88 products, four rounds: bound by the
// rounds' latency), dz 81 us (390 KB an item, HBM at 4.5 TB/s), grads 199 us (28 us
// an item: about 9 wait for the item's 224 KB of tiles, which fill the shared
// memory that a prefetch would need, and 7 are products).  Loading the 128 KB for
// <S, dS'> in larger batches slowed the tile loads (756 against 723 us for a whole
// training step); eight row warps in place of sixteen spilled as much (744).
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

// ---------------------------------------------------------------- dz0, N'
// Tensor memory: K Q^T then (Gam . QK^T)^T [0, 128), Tinv^T [128, 256), w0 then
// dz0 [256, 384), N' [384, 512).  The last operand of N', scale Lam dH, has three
// terms: two go under the first round, the third under the third.
constexpr uint32_t kZDh = 4 * kBlk, kZL = 6 * kBlk, kZW = 10 * kBlk;
constexpr uint32_t kZGc = 14 * kBlk;
constexpr uint32_t kZCol = kZGc + 1024;  // float[2][128]: the columns' factors
constexpr uint32_t kZBar = kZCol + 1024;
constexpr uint32_t kZSmem = kZBar + 64;
static_assert(kZSmem <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_dz0_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_dh, GdnProblem p,
                  const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kZGc);
  float* scol = reinterpret_cast<float*>(smem + kZCol);
  const uint32_t qa = sbase, ka = sbase + 2 * kBlk, ha = sbase + kZDh, la = sbase + kZL,
                 wa = sbase + kZW;
  const uint32_t bar_qk = sbase + kZBar, bar_h = bar_qk + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kZBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  GdnRounds rd{bar_qk + 16, 0u, true, Problem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls}};
  auto load_qk = [&](const GdnItem& x) {
    mbar_expect_tx(bar_qk, 2 * slabs * kBlk);
    const int kh = gdn_key_head(p, x.bh);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, kh, bar_qk);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, x.t0, kh, bar_qk);
    }
  };
  auto load_dh = [&](const GdnItem& x) {
    mbar_expect_tx(bar_h, x.tiles * kBlk);
    for (int v = 0; v < x.tiles; ++v)
      tma_load_3d(ha + v * kBlk, &tm_dh, (x.vt + v) * 64, x.t0, x.bh, bar_h);
  };
  uint4 ti[8];
  float2 ngc;
  float nbt;
  auto load_rows = [&](const GdnItem& x) {
    ngc = w.gc[x.cb * kGdnL + r];
    nbt = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  GdnItem x(blockIdx.x, p, w);
  gdn_next_stage();
  if (lead) {
    for (int i = 0; i < 3; ++i) mbar_init(bar_qk + 8 * i, 1);
    fence_barrier_init();
    load_qk(x);
    load_dh(x);
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  if (row) load_rows(x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  const uint32_t at = (h >> 1) * kBlk;  // this thread's value tile in an image
  uint32_t in_phase = 0;

  for (long i = blockIdx.x; i < items; i += gridDim.x, in_phase ^= 1) {
    const bool more = i + gridDim.x < items;
    const GdnItem nx(more ? i + gridDim.x : i, p, w);
    const bool cols = row && h < 2 * x.tiles;
    const uint32_t id = idesc_bf16(128, x.tiles * 64, 0, 1), idt = idesc_bf16(128, x.tiles * 64, 1, 1);
    float2 gr = make_float2(0.f, 0.f);
    float bt = 0.f;
    if (row) {
      gr = ngc;
      bt = nbt;
      if (h == 0) {
        gc[r] = gr;
        const float f = gdn_col_factor(gr, 0);
        scol[r] = f;
        scol[128 + r] = __fdividef(1.f, gdn_col_factor(gr, 31));
      }
      if (more) load_rows(nx);
    }
    const float lam = gdn_exp(gr), sl = p.scale * lam;
    gdn_round(
        rd, 0x71,
        [&] {
          rd.ok = mbar_wait(bar_qk, in_phase, rd.wt, 0x70);
          tc_fence_after();
          if (rd.ok) mma_ss<false, false>(tmem, ka, qa, idesc_bf16(128, 128, 0, 0), slabs, true);
        },
        [&] {
          if (rd.ok) rd.ok = mbar_wait(bar_h, in_phase, rd.wt, 0x6e);
          if (!cols) return;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            const uint32_t off = at + sw128_offset(r, (h & 1) * 4 + cc);
            float y[8];
            unpack8(*reinterpret_cast<const uint4*>(smem + kZDh + off), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= sl;
            put8(smem + kZL + at, 2 * kBlk, r, (h & 1) * 4 + cc, y);
          }
        },
        gdn_nothing, gdn_nothing);
    uint32_t v[32];
    if (row) {  // row s of (Gam . QK^T)^T: 32 queries; terms take the scores' columns
      uint32_t hi[16], lo[16];
      if (h >= q) {
        tmem_ld32(trow, v);
        tmem_wait_ld();
        float g[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) g[e] = __uint_as_float(v[e]);
        if (h == q && gc[h * 32].x - gc[h * 32 + 31].x > kGdnFlat) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            g[e] = e >= lane ? gdn_decay(gc[h * 32 + e], gr) * g[e] : 0.f;
        } else {
          const bool d = h == q;
          const float f = gdn_decay(gc[h * 32 + (d ? 31 : 0)], gr);
          const float* sc = scol + (d ? 128 : 0) + h * 32;
#pragma unroll
          for (int e = 0; e < 32; ++e) g[e] = d && e < lane ? 0.f : g[e] * (f * sc[e]);
        }
        split_pack<32>(g, hi, lo);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
      }
      tmem_st16(trow, hi);
      tmem_st16(trow + 16, lo);
      load_tinv(w.tinvt + x.cb * 32 * 128, r, h, h >= q, ti);  // for the third round
    }
    gdn_round(
        rd, 0x72,
        [&] {
          if (rd.ok) rd.ok = mbar_wait(bar_h, in_phase, rd.wt, 0x6d);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tmem + 256, tmem + (kk >> 1) * 32 + t * 16 + (kk & 1) * 8, mnmaj(ha, kk),
                          id, (t | kk) != 0);
          for (int t = 0; t < 2; ++t)
            mma_ss<true, true>(tmem + 384, qa, la + 2 * t * kBlk, idt, 2, t == 0);
        },
        [&] {
          add_identity(r, h, ti);
          put_tinv(tlane + 128, h, ti);
        },
        gdn_nothing, gdn_nothing);
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
    gdn_round(
        rd, 0x73, [&] { mma_terms3(tmem + 256, tmem + 128, wa, 2 * kBlk, id); },
        [&] {
          if (!cols) return;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            float y[8];
            unpack8(*reinterpret_cast<const uint4*>(smem + kZDh + at +
                                                    sw128_offset(r, (h & 1) * 4 + cc)),
                    y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= sl;
            put_terms<3, 2>(smem + kZL + at, 0, r, (h & 1) * 4 + cc, y);
          }
        },
        gdn_nothing, gdn_nothing);
    const size_t nb = ((x.cb * w.nvt + x.vt + (h >> 1)) * 16 + (h & 1) * 8) * 128 + r;
    if (cols) {
      tmem_ld32(trow + 256, v);
      tmem_wait_ld();
      gdn_put_n(p, w, w.dz0, nb, v);
      put(-lam);
    }
    gdn_round(
        rd, 0x74,
        [&] {
          for (int t = 0; t < 2; ++t)
            mma_ss<true, true>(tmem + 384, ka, wa + 2 * t * kBlk, idt, 2, false);
          mma_ss<true, true>(tmem + 384, qa, la, idt, 2, false);
        },
        gdn_nothing,
        [&] {
          if (more) load_dh(nx);
        },
        [&] {
          if (more) load_qk(nx);
        });
    if (cols) {
      tmem_ld32(trow + 384, v);
      tmem_wait_ld();
      gdn_put_n(p, w, w.N, nb, v);
    }
    x = nx;
  }
  tc_fence_before();
  __syncthreads();
  if (!row) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dz, dV
// Tensor memory: Tinv^T [0, 128), K dS' [128, 256), dz [256, 384).  The image
// holds y (for out), then beta D K dS', then dz.
constexpr uint32_t kYDs = 2 * kBlk, kYW = 8 * kBlk, kYDv = 12 * kBlk, kYBar = 14 * kBlk;
constexpr uint32_t kYSmem = kYBar + 64;

__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_dz_kernel(const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_dv, GdnProblem p,
                 const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ka = sbase, da = sbase + kYDs, wa = sbase + kYW;
  const uint32_t bar_in = sbase + kYBar, bar_y = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kYBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  GdnRounds rd{bar_in + 16, 0u, true, Problem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls}};
  auto load_tiles = [&](const GdnItem& x, bool wait) {
    mbar_expect_tx(bar_in, slabs * (kBlk + x.tiles * 3 * 8192));
    const int kh = gdn_key_head(p, x.bh);
    for (int s = 0; s < slabs; ++s) tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, kh, bar_in);
    if (wait) gdn_wait_stage();
    for (int v = 0; v < x.tiles; ++v)
      for (int t = 0; t < 3; ++t)
        gdn_load(p, w, da + (2 * t + v) * kBlk, w.dS, 3 * w.nvt,
                 (x.cb * w.nvt + x.vt + v) * 3 + t, slabs * 8192, bar_in);
  };
  auto load_y = [&](const GdnItem& x) {
    mbar_expect_tx(bar_y, x.tiles * 2 * kBlk);
    for (int v = 0; v < x.tiles; ++v)
      for (int t = 0; t < 2; ++t)
        gdn_load(p, w, wa + (2 * t + v) * kBlk, w.y, 2 * w.nvt,
                 (x.cb * w.nvt + x.vt + v) * 2 + t, kBlk, bar_y);
  };
  uint4 ti[8];
  float2 ngc, ngl;
  float nbt;
  auto load_rows = [&](const GdnItem& x) {
    ngc = w.gc[x.cb * kGdnL + r];
    ngl = w.gc[x.cb * kGdnL + kGdnL - 1];
    nbt = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  GdnItem x(blockIdx.x, p, w);
  gdn_next_stage();
  if (lead) {
    for (int i = 0; i < 3; ++i) mbar_init(bar_in + 8 * i, 1);
    fence_barrier_init();
    load_tiles(x, true);
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  if (row) load_rows(x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  uint8_t* img = smem + kYW + (h >> 1) * kBlk;
  uint32_t in_phase = 0;

  for (long i = blockIdx.x; i < items; i += gridDim.x, in_phase ^= 1) {
    const bool more = i + gridDim.x < items;
    const GdnItem nx(more ? i + gridDim.x : i, p, w);
    const bool cols = row && h < 2 * x.tiles;
    const uint32_t id = idesc_bf16(128, x.tiles * 64, 0, 1);
    const size_t ct = x.cb * w.nvt + x.vt + (h >> 1);
    float dec = 0.f, bd = 0.f;
    if (lead) {
      tma_store_wait_read_all();  // dz and dV of the item before have left
      load_y(x);
    }
    if (row) {
      dec = gdn_decay(ngl, ngc);
      bd = nbt * dec;
      load_tinv(w.tinvt + x.cb * 32 * 128, r, h, h >= q, ti);  // for the second round
      if (more) load_rows(nx);
    }
    float4 z0[8];
    gdn_round(
        rd, 0x76,
        [&] {
          rd.ok = mbar_wait(bar_in, in_phase, rd.wt, 0x79);
          tc_fence_after();
          if (!rd.ok) return;
          for (int t = 0; t < 3; ++t)
            mma_ss<false, true>(tmem + 128, ka, da + 2 * t * kBlk, id, slabs, t == 0);
        },
        [&] {
          add_identity(r, h, ti);
          put_tinv(tlane, h, ti);
          if (rd.ok) rd.ok = mbar_wait(bar_y, in_phase, rd.wt, 0x75);
        },
        gdn_nothing,
        [&] {
          if (more) load_tiles(nx, false);
        });
    uint32_t v[32];
    if (cols) {
      tmem_ld32(trow + 128, v);
      tmem_wait_ld();
      float o = 0.f;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        const uint32_t off = sw128_offset(r, (h & 1) * 4 + cc);
        float a[8], b[8];
        unpack8(*reinterpret_cast<const uint4*>(img + off), a);
        unpack8(*reinterpret_cast<const uint4*>(img + 2 * kBlk + off), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xd = __uint_as_float(v[8 * cc + e]);
          o = fmaf(a[e] + b[e], xd, o);
          a[e] = bd * xd;
        }
        put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, a);
      }
      if (MLSTM_IN_BOUNDS(p, ct < (size_t)p.BH * w.NC * w.nvt))
        w.out[ct * 256 + (h & 1) * 128 + r] = dec * o;
      const float4* zp = w.dz0 + (ct * 16 + (h & 1) * 8) * 128 + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[e] = zp[e * 128];
    }
    gdn_round(
        rd, 0x78, [&] { mma_terms3(tmem + 256, tmem, wa, 2 * kBlk, id); }, gdn_nothing,
        gdn_nothing, gdn_nothing);
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
    if (lead) {  // every thread has read its part of dz0, which dz replaces
      for (int t = 0; t < x.tiles; ++t)
        for (int term = 0; term < 2; ++term)
          gdn_store(p, w, w.dz, 2 * w.nvt, (x.cb * w.nvt + x.vt + t) * 2 + term,
                    wa + (2 * term + t) * kBlk, kBlk);
      if (rd.ok)  // rows past T and columns past d_v are clipped
        for (int t = 0; t < x.tiles; ++t)
          if (MLSTM_IN_BOUNDS(p, gdn_box_inside(p, (x.vt + t) * 64, p.DV, x.t0, x.bh, p.BH)))
            tma_store_3d(&tm_dv, sbase + kYDv + t * kBlk, (x.vt + t) * 64, x.t0, x.bh);
      tma_store_commit();
    }
    x = nx;
  }
  if (lead) tma_store_wait_all();
  __syncthreads();
  if (!row) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- gradients
// Persistent, one block per SM, per (bh, chunk) all value columns in pairs of
// tiles.  Rounds:
//   1  dH y^T, dz y^T, dH S^T, dz S^T               (80 products for 128 columns)
//   2  y dS'^T and Q K^T; meanwhile dH S^T and dz S^T are scaled in place: the
//      first terms of dQ and dK, and q, k against them (ent)
//   3  K K^T; meanwhile the images of Rh beta and Eh beta
//   4  dQ += (Rh beta) K, dK += (Eh beta) K + (Rh beta)^T Q + (Eh beta)^T K (64);
//      meanwhile dg and dbeta
// Tensor memory: dH y^T, y dS'^T, K K^T [0, 128); dz y^T, Q K^T [128, 256); dQ
// [256, 384); dK [384, 512).  Shared memory blocks: S, then K and Q 0..3; y, then
// Rh beta, then the results 4..7; dz, then dS', then Eh beta 8..11; dH, then the
// sums 12, 13.
constexpr uint32_t kGY = 4 * kBlk, kGZ = 8 * kBlk, kGH = 12 * kBlk;
constexpr uint32_t kGRed = 12 * kBlk;             // float[3][4][128]: ent, rows, columns
constexpr uint32_t kGOut = kGRed + 3 * 4 * 512;   // float[128]
constexpr uint32_t kGDiag = kGOut + 512;          // float[128]
constexpr uint32_t kGDot = kGDiag + 512;          // float[16]
constexpr uint32_t kGGc = 14 * kBlk;
constexpr uint32_t kGBeta = kGGc + 1024;
constexpr uint32_t kGCol = kGBeta + 512;
constexpr uint32_t kGBar = kGCol + 1024;
constexpr uint32_t kGSmem = kGBar + 64;
static_assert(kGSmem <= 227 * 1024, "shared memory");

// kShared: fp32 gradients per value head (key heads are shared).
template <bool kShared>
__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_grads_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_dh,
                    const __grid_constant__ CUtensorMap tm_dq,
                    const __grid_constant__ CUtensorMap tm_dk, GdnProblem p,
                    const float* __restrict__ beta, float* __restrict__ dg,
                    float* __restrict__ dbeta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kGGc);
  float* sbeta = reinterpret_cast<float*>(smem + kGBeta);
  float* scol = reinterpret_cast<float*>(smem + kGCol);
  float* red = reinterpret_cast<float*>(smem + kGRed);
  float* sout = reinterpret_cast<float*>(smem + kGOut);
  float* sdiag = reinterpret_cast<float*>(smem + kGDiag);
  float* sdot = reinterpret_cast<float*>(smem + kGDot);
  const uint32_t ka = sbase, qa = sbase + 2 * kBlk, sa = sbase, ya = sbase + kGY, za = sbase + kGZ,
                 ha = sbase + kGH;
  const uint32_t bar_a = sbase + kGBar, bar_q = bar_a + 8, bar_d = bar_a + 16;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kGBar + 40);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64, pairs = (w.nvt + 1) / 2;
  const int items = p.BH * w.NC;
  GdnRounds rd{bar_a + 24, 0u, true, Problem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls}};
  const uint32_t sbytes = slabs * 8192;

  auto tiles_of = [&](int pr) { return min(2, w.nvt - 2 * pr); };
  auto load_y = [&](size_t cb, int pr, uint32_t bar) {
    for (int v = 0; v < tiles_of(pr); ++v)
      for (int t = 0; t < 2; ++t)
        gdn_load(p, w, ya + (2 * t + v) * kBlk, w.y, 2 * w.nvt,
                 (cb * w.nvt + 2 * pr + v) * 2 + t, kBlk, bar);
  };
  // dH, S and dz of a pair; y apart (its place may still hold results)
  auto load_a = [&](int it, int pr) {
    const size_t cb = it;
    const int bh = it / w.NC, t0 = (it - bh * w.NC) * kGdnL, n = tiles_of(pr);
    mbar_expect_tx(bar_a, n * (5 * kBlk + 2 * sbytes));
    for (int v = 0; v < n; ++v) {
      const size_t ct = cb * w.nvt + 2 * pr + v;
      tma_load_3d(ha + v * kBlk, &tm_dh, (2 * pr + v) * 64, t0, bh, bar_a);
      for (int t = 0; t < 2; ++t) {
        gdn_load(p, w, sa + (2 * t + v) * kBlk, w.S, 2 * w.nvt, ct * 2 + t, sbytes, bar_a);
        gdn_load(p, w, za + (2 * t + v) * kBlk, w.dz, 2 * w.nvt, ct * 2 + t, kBlk, bar_a);
      }
    }
  };
  // the first two terms of dS' (and y again, where there are several pairs)
  auto load_d = [&](int it, int pr) {
    const int n = tiles_of(pr);
    mbar_expect_tx(bar_d, n * (2 * sbytes + (pairs > 1 ? 2 * kBlk : 0u)));
    for (int v = 0; v < n; ++v)
      for (int t = 0; t < 2; ++t)
        gdn_load(p, w, za + (2 * t + v) * kBlk, w.dS, 3 * w.nvt,
                 ((size_t)it * w.nvt + 2 * pr + v) * 3 + t, sbytes, bar_d);
    if (pairs > 1) load_y(it, pr, bar_d);
  };
  auto load_qk = [&](int it) {
    const int bh = it / w.NC, t0 = (it - bh * w.NC) * kGdnL;
    mbar_expect_tx(bar_q, 2 * slabs * kBlk);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, gdn_key_head(p, bh), bar_q);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, t0, gdn_key_head(p, bh), bar_q);
    }
  };
  float2 ngc, ngl;
  float nbt;
  auto load_rows = [&](int it) {
    const int bh = it / w.NC, t = (it - bh * w.NC) * kGdnL + r;
    ngc = w.gc[(size_t)it * kGdnL + r];
    ngl = w.gc[(size_t)it * kGdnL + kGdnL - 1];
    nbt = t < p.T ? beta[(long)bh * p.T + t] : 0.f;
  };

  if (lead) {
    for (int i = 0; i < 4; ++i) mbar_init(bar_a + 8 * i, 1);
    fence_barrier_init();
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  if (lead) {
    load_a(blockIdx.x, 0);
    load_y(blockIdx.x, 0, bar_a);
  }
  if (row) load_rows(blockIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + h * 32;
  const bool cols = row && h < 2 * slabs;  // this thread's columns exist in d_qk matrices
  const bool lower = row && h <= q;        // not all columns lie right of the diagonal
  constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);
  const uint32_t id_d = idesc_bf16(128, slabs * 64, 0, 0);
  uint32_t pa = 0, pq = 0, pd = 0;  // phases

  // D (+)= A B^T over a block of 64 value columns, operands of one or two terms
  auto outer = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool a_terms, bool fresh) {
    mma_ss<false, false>(d, a, b, id, 1, fresh);
    mma_ss<false, false>(d, a, b + 2 * kBlk, id, 1, false);
    if (a_terms) mma_ss<false, false>(d, a + 2 * kBlk, b, id, 1, false);
  };

  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int next = it + gridDim.x;
    const bool more = next < items;
    const int bh = it / w.NC, t0 = (it - bh * w.NC) * kGdnL, n = min(kGdnL, p.T - t0);
    float2 gr = make_float2(0.f, 0.f), gl = gr;
    if (row) {
      gr = ngc;
      gl = ngl;
      if (h == 0) {
        gc[r] = gr;
        sbeta[r] = nbt;
        scol[r] = gdn_col_factor(gr, 31);
        scol[128 + r] = __fdividef(1.f, gdn_col_factor(gr, 0));
      }
      if (more) load_rows(next);
    }
    float dot = 0.f;  // <S, dS'>
    for (int pr = 0; pr < pairs; ++pr) {
      const int nt = tiles_of(pr);
      gdn_round(
          rd, 0x7c,
          [&] {
            rd.ok = mbar_wait(bar_a, pa, rd.wt, 0x7b);
            tc_fence_after();
            if (!rd.ok) return;
            for (int v = 0; v < nt; ++v) {
              const uint32_t o = v * kBlk;
              const bool fresh = pr == 0 && v == 0;
              outer(tmem, ha + o, ya + o, id_s, false, fresh);
              outer(tmem + 128, za + o, ya + o, id_s, true, fresh);
              outer(tmem + 256, ha + o, sa + o, id_d, false, fresh);
              outer(tmem + 384, za + o, sa + o, id_d, true, fresh);
            }
          },
          [&] {
            // both states' images, in whatever order: 16-byte pieces of two terms
            for (int v = 0; v < nt; ++v) {
              const size_t ct = (size_t)it * w.nvt + 2 * pr + v;
              const uint4* s0 = reinterpret_cast<const uint4*>(w.S + ct * 2 * kBlk);
              const uint4* d0 = reinterpret_cast<const uint4*>(w.dS + ct * 3 * kBlk);
              for (int k = tid; k < (int)sbytes / 16; k += kGdnRows) {
                float a[8], b[8], c[8], d[8];
                unpack8(s0[k], a);
                unpack8(s0[k + kBlk / 16], b);
                unpack8(d0[k], c);
                unpack8(d0[k + kBlk / 16], d);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(a[e] + b[e], c[e] + d[e], dot);
              }
            }
          },
          gdn_nothing,
          [&] {
            if (pr + 1 < pairs) {
              load_a(it, pr + 1);
              load_y(it, pr + 1, bar_a);
            } else {
              load_qk(it);
              load_d(it, 0);
            }
          });
      pa ^= 1;
    }
    float rh[32], eh[32];
    if (lower) {
      uint32_t a[16];
      const bool d = h == q, steep = d && gc[h * 32].x - gc[h * 32 + 31].x > kGdnFlat;
      const float f = gdn_decay(gr, gc[h * 32 + (d ? 0 : 31)]);
      const float* sc = scol + (d ? 128 : 0) + h * 32;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float g[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = half * 16 + e;
          g[e] = d && k > lane ? 0.f : f * sc[k];
        }
        if (steep)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            g[e] = half * 16 + e <= lane ? gdn_decay(gr, gc[h * 32 + half * 16 + e]) : 0.f;
        tmem_ld16(trow + half * 16, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          rh[half * 16 + e] = p.scale * g[e] * __uint_as_float(a[e]);
        tmem_ld16(trow + 128 + half * 16, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          eh[half * 16 + e] =
              h == q && half * 16 + e == lane ? 0.f : -g[e] * __uint_as_float(a[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) rh[e] = eh[e] = 0.f;
    }
    const float lam = gdn_exp(gr);
    // four bf16 values of this thread's row of q or k
    auto piece = [&](uint32_t off, int cc, float* y) {
      unpack8(*reinterpret_cast<const uint4*>(smem + off + (h >> 1) * kBlk +
                                              sw128_offset(r, (h & 1) * 4 + cc)),
              y);
    };
    for (int pr = 0; pr < pairs; ++pr) {
      const int nt = tiles_of(pr);
      gdn_round(
          rd, 0x7d,
          [&] {
            rd.ok = mbar_wait(bar_d, pd, rd.wt, 0x7e);
            if (pr == 0) rd.ok = rd.ok && mbar_wait(bar_q, pq, rd.wt, 0x7f);
            tc_fence_after();
            if (!rd.ok) return;
            if (pr == 0) mma_ss<false, false>(tmem + 128, qa, ka, id_s, slabs, true);
            for (int v = 0; v < nt; ++v)
              outer(tmem, ya + v * kBlk, za + v * kBlk, id_d, true, pr == 0 && v == 0);
          },
          [&] {
            if (pr) return;
            if (rd.ok) rd.ok = mbar_wait(bar_q, pq, rd.wt, 0x7a);
            float ent = 0.f;
            if (cols)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t a[16];
                tmem_ld16(trow + 256 + half * 16, a);
                tmem_wait_ld();
                const float fq = p.scale * lam;
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2) {
                  float y[8];
                  piece(2 * kBlk, half * 2 + c2, y);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float u = fq * __uint_as_float(a[8 * c2 + e]);
                    ent = fmaf(y[e], u, ent);
                    a[8 * c2 + e] = __float_as_uint(u);
                  }
                }
                tmem_st16(trow + 256 + half * 16, a);
                tmem_ld16(trow + 384 + half * 16, a);
                tmem_wait_ld();
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2) {
                  float y[8];
                  piece(0, half * 2 + c2, y);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float u = -lam * __uint_as_float(a[8 * c2 + e]);
                    ent = fmaf(y[e], u, ent);
                    a[8 * c2 + e] = __float_as_uint(u);
                  }
                }
                tmem_st16(trow + 384 + half * 16, a);
              }
            red[h * 128 + r] = ent;
          },
          gdn_nothing,
          [&] {
            if (pr + 1 < pairs) load_d(it, pr + 1);
          });
      pd ^= 1;
    }
    pq ^= 1;
    // dK += beta D (y dS'^T); Z's first part
    float row_sum = 0.f;
    if (cols) {
      const float fo = sbeta[r] * gdn_decay(gl, gr);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t a[16], b[16];
        tmem_ld16(trow + half * 16, a);
        tmem_ld16(trow + 384 + half * 16, b);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          b[e] = __float_as_uint(fmaf(fo, __uint_as_float(a[e]), __uint_as_float(b[e])));
        tmem_st16(trow + 384 + half * 16, b);
      }
    }
    gdn_round(
        rd, 0x77, [&] { mma_ss<false, false>(tmem, ka, ka, id_s, slabs, true); },
        [&] {
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            float y[8], u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float b = sbeta[h * 32 + 8 * cc + e];
              y[e] = rh[8 * cc + e] * b;
              u[e] = eh[8 * cc + e] * b;
            }
            put8(smem + kGY + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, y);
            put8(smem + kGZ + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, u);
          }
          dot = warp_sum(dot);
          if (lane == 0) sdot[warp] = dot;
          if (h == 1) {
            float o = 0.f;
            for (int k = 0; k < 2 * w.nvt; ++k) o += w.out[((size_t)it * w.nvt * 2 + k) * 128 + r];
            sout[r] = o;
          }
        },
        gdn_nothing, gdn_nothing);
    // Z, its row sums (times beta) and column sums left of the diagonal
    if (row) {
      float col = 0.f;
      if (lower) {
        uint32_t a[16], b[16];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_ld16(trow + 128 + half * 16, a);
          tmem_ld16(trow + half * 16, b);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = half * 16 + e;
            float z = fmaf(rh[k], __uint_as_float(a[e]), eh[k] * __uint_as_float(b[e]));
            if (h == q) {
              if (k == lane) sdiag[r] = z;
              z = k < lane ? z : 0.f;
            }
            row_sum = fmaf(z, sbeta[h * 32 + k], row_sum);
            rh[k] = z;
          }
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
      red[(4 + h) * 128 + r] = row_sum;
      red[(8 + q) * 128 + h * 32 + lane] = col;
    }
    const uint32_t id_n = idesc_bf16(128, slabs * 64, 0, 1),
                   id_t = idesc_bf16(128, slabs * 64, 1, 1);
    gdn_round(
        rd, 0x78,
        [&] {
          for (int t = 0; t < 2; ++t) {
            mma_ss<false, true>(tmem + 256, ya + 2 * t * kBlk, ka, id_n, 2, false);
            mma_ss<false, true>(tmem + 384, za + 2 * t * kBlk, ka, id_n, 2, false);
            mma_ss<true, true>(tmem + 384, ya + 2 * t * kBlk, qa, id_t, 2, false);
            mma_ss<true, true>(tmem + 384, za + 2 * t * kBlk, ka, id_t, 2, false);
          }
        },
        [&] {
          if (warp != 0) return;
          // dg: suffix sums of what enters and of Z's rows less its columns, prefix
          // sums of what leaves; four tokens per lane
          float suf[4], pre[4], o[4], cs[4], ssuf = 0.f, spre = 0.f;
          float dG = warp_sum(lane < 16 ? sdot[lane] : 0.f) * gdn_exp(gl);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 4 * lane + e;
            float en = 0.f, rw = 0.f;
            o[e] = sout[t];
            cs[e] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              en += red[k * 128 + t];
              rw += red[(4 + k) * 128 + t];
              cs[e] += red[(8 + k) * 128 + t];
            }
            suf[e] = en + (rw - sbeta[t] * cs[e]);
            ssuf += suf[e];
            pre[e] = sbeta[t] * o[e];
            spre += pre[e];
          }
          float incl = ssuf, inclp = spre;  // over the lanes behind / before
#pragma unroll
          for (int k = 1; k < 32; k <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, incl, k);
            const float b = __shfl_up_sync(0xffffffffu, inclp, k);
            if (lane + k < 32) incl += a;
            if (lane >= k) inclp += b;
          }
          float s = incl - ssuf, before = inclp - spre, y[4];
#pragma unroll
          for (int e = 3; e >= 0; --e) {
            s += suf[e];
            y[e] = s + dG;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 4 * lane + e;
            if (t < n && MLSTM_IN_BOUNDS(p, bh < p.BH && t0 + t < p.T)) {
              dg[(long)bh * p.T + t0 + t] = y[e] + before;
              dbeta[(long)bh * p.T + t0 + t] = o[e] + cs[e] + sdiag[t];
            }
            before += pre[e];
          }
        },
        gdn_nothing, gdn_nothing);
    // results through shared memory (blocks 4 ..): bf16, two blocks each, or fp32,
    // four blocks of 32 columns each
    if (cols) {
      uint32_t a[16];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_ld16(trow + 256 + m * 128 + half * 16, a);
          tmem_wait_ld();
          const float* y = reinterpret_cast<const float*>(a);
          if (kShared) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(smem + kGY + (4 * m + h) * kBlk +
                                        sw128_offset(r, half * 4 + e)) =
                  make_uint4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(smem + kGY + (2 * m + (h >> 1)) * kBlk +
                                        sw128_offset(r, (h & 1) * 4 + half * 2 + e)) =
                  pack8(y + 8 * e);
          }
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (lead) {
      if (rd.ok) {  // rows past T and columns past d_qk are clipped
        const int hd = kShared ? bh : gdn_key_head(p, bh);
        constexpr int kW = kShared ? 32 : 64, kN = kShared ? 4 : 2;
        for (int m = 0; m < 2; ++m)
          for (int b = 0; b * kW < p.DK; ++b)
            if (MLSTM_IN_BOUNDS(p, gdn_box_inside(p, b * kW, p.DK, t0, hd,
                                                  kShared ? p.BH : p.B * p.NHK)))
              tma_store_3d(m ? &tm_dk : &tm_dq, ya + (kN * m + b) * kBlk, b * kW, t0, hd);
        tma_store_commit();
        if (more && !kShared) load_a(next, 0);
        tma_store_wait_read_all();
        if (more && kShared) load_a(next, 0);
        if (more) load_y(next, 0, bar_a);
      }
    }
  }
  if (lead) tma_store_wait_all();
  __syncthreads();
  if (!row) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_gdn_tc_dz0(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m, bool after,
                              const GdnTcWs& w, cudaStream_t st) {
  return gdn_launch(&gdn_tc_dz0_kernel, gdn_blocks(p, w), kGdnThreads, kZSmem, after, st, m.q, m.k,
                    m.dh, p, x.beta, w);
}

cudaError_t launch_gdn_tc_dz(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                             const GdnTcWs& w, cudaStream_t st) {
  return gdn_launch(&gdn_tc_dz_kernel, gdn_blocks(p, w), kGdnThreads, kYSmem, true, st, m.k, m.dv,
                    p, x.beta, w);
}

cudaError_t launch_gdn_tc_grads(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                                const GdnMaps& m, const GdnTcWs& w, cudaStream_t st) {
  const long n = (long)p.BH * w.NC;
  auto go = [&](auto* kern) {
    return gdn_launch(kern, (unsigned)(n < kGdnSms ? n : kGdnSms), kGdnThreads, kGSmem, true, st,
                      m.q, m.k, m.dh, m.dq, m.dk, p, x.beta, d.dg, d.dbeta, w);
  };
  if (!w.dq) return go(&gdn_tc_grads_kernel<false>);
  const cudaError_t e = go(&gdn_tc_grads_kernel<true>);
  return e == cudaSuccess ? launch_gdn_group_sum(p, MLSTM_DT_BF16, w.dq, w.dk, d.dQ, d.dK, st) : e;
}

}  // namespace mlstm
