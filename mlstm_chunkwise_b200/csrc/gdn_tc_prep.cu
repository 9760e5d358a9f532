// Gated delta rule, tensor cores: what a chunk contributes before the state that
// enters it is known: the sums of g and Tinv = (I + A)^{-1} with
// A_rs = Gam_rs beta_s k_r.k_s (s < r), then M and N of the state recurrence.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

// ------------------------------------------------------------------ inverse
// Persistent, blocks of 256 threads, thread (r, h) on one of two column halves of
// row r.  The inverse goes by blocks: the four 32 x 32 diagonal blocks by forward
// substitution in fp32 (a warp per block, a lane per column), while the other warps
// form the terms of A left of them; then T21 = -T22 A21 T11 for the two 64-blocks
// at once and for the whole, on the tensor cores with both operands as two bf16
// terms (A21 and T22 in tensor memory, T11 and A21 T11 as images).  Half a dozen
// dependent passes of little work each, bound by their latency: two blocks share
// an SM, and the next item's K, its K K^T and its sums are prepared meanwhile
// (8192 chunks 208 to 220 us, 512 chunks 21; a block per item 262 and 22).  What costs
// beyond that is instruction fetch, so loops whose copies would differ in little
// stay rolled, and anything in local memory, for which the shared memory leaves
// little L1 (a row's diagonal bit cleared by index, not by mask: 293 us).
// Tensor memory: operands [0, 64), products [64, 128), K K^T [128, 256), where the
// terms of A21 of the whole take the columns that they came from.
constexpr int kInvThreads = 256;
constexpr int kLd = 36;                     // floats per row of a diagonal block
constexpr uint32_t kBi = 8192;              // lo term of the products' images (64 rows)
// behind K twice (this item's, the next one's): float2[128] sums, beta, and
// float[2][128], beta times the column's factor
constexpr uint32_t kIGates = 2 * kBlk, kIGate = 1024 + 512 + 1024;
constexpr uint32_t kIBar = kIGates + 2 * kIGate;
constexpr uint32_t kIWork = kIGates + 6 * 1024;  // the products' image; with kT Tinv in the end
constexpr uint32_t kIDiag = kIWork + kBlk;       // float[4][32][kLd]
constexpr uint32_t inv_smem(bool kT) {
  return kT ? kIWork + 4 * kBlk : kIDiag + 4 * 32 * kLd * 4;
}
static_assert(2 * (inv_smem(true) + 1024) <= 228 * 1024, "two blocks per SM");

// kT: also Tinv^T.
template <bool kT>
__global__ void __launch_bounds__(kInvThreads, 2)
gdn_tc_inverse_kernel(const __grid_constant__ CUtensorMap tm_k, GdnProblem p,
                      const float* __restrict__ g, const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_k = sbase + kIBar, bar_kk = bar_k + 8, bar = bar_k + 16;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kIBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int slabs = (p.DK + 63) / 64;
  const int items = p.BH * w.NC;  // up to 65535 x 2^15: an int holds them and a grid more
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};
  // item i: chunk i % NC of head i / NC, so rows i * 128 of the workspace's arrays
  auto load_k = [&](int i) {
    const int bh = i / w.NC, t0 = (i - bh * w.NC) * kGdnL;
    mbar_expect_tx(bar_k, slabs * kBlk);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(sbase + s * kBlk, &tm_k, s * 64, t0, gdn_key_head(p, bh), bar_k);
  };
  auto put_gates = [&](int i, uint32_t buf) {  // by one warp
    const int bh = i / w.NC, t0 = (i - bh * w.NC) * kGdnL, n = min(kGdnL, p.T - t0);
    const long at = (long)bh * p.T + t0;
    float2* gc = reinterpret_cast<float2*>(smem + kIGates + buf * kIGate);
    float* sbeta = reinterpret_cast<float*>(gc + 128);
    float bt[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) bt[b] = b * 32 + lane < n ? beta[at + b * 32 + lane] : 0.f;
    gdn_chunk_sums(g + at, n, lane, gc, w.gc + (size_t)i * kGdnL);
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int t = b * 32 + lane;
      const float2 gt = gc[t];
      sbeta[t] = bt[b];
      sbeta[128 + t] = bt[b] * gdn_col_factor(gt, 31);
      sbeta[256 + t] = __fdividef(bt[b], gdn_col_factor(gt, 0));
    }
  };

  gdn_next_stage();
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(bar_k + 8 * i, 1);
    fence_barrier_init();
    load_k(blockIdx.x);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 256);
    tmem_relinquish();
  }
  if (warp == 4) put_gates(blockIdx.x, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
  bool ok = true;
  uint32_t phase = 0, ph = 0;
  auto k_product = [&](uint32_t k_phase) {  // by one lane
    if (ok) ok = mbar_wait(bar_k, k_phase, wt, 0x41);
    tc_fence_after();
    if (ok) mma_ss<false, false>(tmem + 128, sbase, sbase, idesc_bf16(128, 128, 0, 0), slabs, true);
    mma_commit(bar_kk);
  };
  if (warp == 0 && elect_one()) k_product(0);
  __syncwarp();

  float* diag = reinterpret_cast<float*>(smem + kIDiag);
  float* dq = diag + q * 32 * kLd;  // [s][r] of block q
  uint8_t* img = smem + kIWork;
  const uint32_t ia = sbase + kIWork;
  auto inv_mma = [&](uint32_t a) {
    constexpr uint32_t id = idesc_bf16(128, 64, 0, 1);
#pragma unroll 1
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ts(tmem + 64, a + (kk >> 1) * 32 + (t == 1 ? 16 : 0) + (kk & 1) * 8,
                    mnmaj(ia + (t == 2 ? kBi : 0u), kk), id, (t | kk) != 0);
  };

  for (int i = blockIdx.x; i < items; i += gridDim.x, ph ^= 1) {
    const bool more = i + gridDim.x < items;
    if (ok) ok = mbar_wait(bar_kk, ph, wt, 0x42);
    tc_fence_after();
    if (more && ok && tid == 128) load_k(i + gridDim.x);  // K has been read
    const float2* gc = reinterpret_cast<const float2*>(smem + kIGates + ph * kIGate);
    const float* sbeta = reinterpret_cast<const float*>(gc + 128);
    const float* scol = sbeta + 128;
    const float2 gr = gc[r];
    if (h == 0) {
      uint32_t v[32];
      tmem_ld32(trow + 128 + q * 32, v);
      tmem_wait_ld();
      if (gc[q * 32].x - gc[q * 32 + 31].x > kGdnFlat) {
#pragma unroll
        for (int e = 0; e < 32; ++e) dq[e * kLd + lane] = __uint_as_float(v[e]);
#pragma unroll 1
        for (int e = 0; e < 32; ++e) {
          const int s = q * 32 + e;
          float* x = dq + e * kLd + lane;
          *x = e < lane ? gdn_decay(gr, gc[s]) * sbeta[s] * *x : 0.f;
        }
      } else {
        const float f = gdn_decay(gr, gc[q * 32]);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          dq[e * kLd + lane] =
              e < lane ? f * scol[128 + q * 32 + e] * __uint_as_float(v[e]) : 0.f;
      }
      __syncwarp();
      // column `lane` of the block's inverse: once x_s is known its multiples leave
      // all later rows (independent products)
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = e == lane ? 1.f : 0.f;
#pragma unroll
      for (int s = 0; s < 31; ++s) {
#pragma unroll
        for (int r4 = (s + 1) / 4; r4 < 8; ++r4) {
          const float4 v = *reinterpret_cast<const float4*>(dq + s * kLd + r4 * 4);
          const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (4 * r4 + e > s) x[4 * r4 + e] = fmaf(-a[e], x[s], x[4 * r4 + e]);
        }
      }
      __syncwarp();  // every lane has read the block
#pragma unroll
      for (int r4 = 0; r4 < 8; ++r4)
        *reinterpret_cast<float4*>(dq + lane * kLd + r4 * 4) =
            make_float4(x[4 * r4], x[4 * r4 + 1], x[4 * r4 + 2], x[4 * r4 + 3]);
    } else if (q == 0) {
      if (more) put_gates(i + gridDim.x, ph ^ 1);
    } else {
      // Blocks of A's rows left of the diagonal's (columns 32 b ..), as terms: for
      // odd q that of A21 of the 64-blocks (inner columns 0..31 are the first one's,
      // 32..63 the second's), for q >= 2 the two of A21 of the whole, in place.
#pragma unroll 1
      for (int j = q & 1 ? 0 : 1; j < (q >= 2 ? 3 : 1); ++j) {
        const int b = j ? j - 1 : q - 1;
        uint32_t v[32], hi[16], lo[16];
        tmem_ld32(trow + 128 + b * 32, v);
        tmem_wait_ld();
        const float f = gdn_decay(gr, gc[b * 32 + 31]);
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = f * scol[b * 32 + e] * __uint_as_float(v[e]);
        split_pack<32>(x, hi, lo);
        const uint32_t to = trow + (j ? 128 + b * 32 : (q >> 1) * 32);
        tmem_st16(to, hi);
        tmem_st16(to + 16, lo);
        if (j == 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
          tmem_st32(trow + 32 - (q >> 1) * 32, v);
        }
      }
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
    run_mma(bar, phase, ok, wt, 0x43, [&] { inv_mma(tmem); });
    if (q & 1) {
      uint32_t v[16];
      tmem_ld16(trow + 64 + h * 16, v);
      tmem_wait_ld();
      const int kr = (q >> 1) * 32 + lane;
      put8(img, kBi, kr, h * 2, reinterpret_cast<const float*>(v));
      put8(img, kBi, kr, h * 2 + 1, reinterpret_cast<const float*>(v) + 8);
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = dq[(h * 16 + e) * kLd + lane];
      uint32_t hi[8], lo[8];
      split_pack<16>(x, hi, lo);
      tmem_st8(trow + (q >> 1) * 32 + h * 8, hi);
      tmem_st8(trow + (q >> 1) * 32 + 16 + h * 8, lo);
    }
    run_mma(bar, phase, ok, wt, 0x44, [&] { inv_mma(tmem); });
    // x: columns 32 h .. of this row inside its 64-block of the inverse
    float x[32];
    if (h == 0 && (q & 1)) {
      uint32_t v[32];
      tmem_ld32(trow + 64, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = -__uint_as_float(v[e]);
    } else if (h == (q & 1)) {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = dq[e * kLd + lane];
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = 0.f;
    }
    if (q < 2) {
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) put8(img, kBi, r, h * 4 + cc, x + 8 * cc);
    }
    run_mma(bar, phase, ok, wt, 0x45, [&] { inv_mma(tmem + 128); });
    uint32_t hi[16], lo[16];
    split_pack<32>(x, hi, lo);
    if (q >= 2) {
      uint32_t v[32];
      tmem_ld32(trow + 64 + h * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc)
        put8(img, kBi, r - 64, h * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
      tmem_st16(trow + h * 32, hi);
      tmem_st16(trow + h * 32 + 16, lo);
    }
    run_mma(bar, phase, ok, wt, 0x46, [&] { inv_mma(tmem); });
    if (more) {
      if (warp == 0 && elect_one()) k_product(ph ^ 1);
      __syncwarp();
    }
    // the row's terms, without the identity, by blocks (columns 32 b ..): that of
    // its 64-block of the inverse, and for q >= 2 that of T21 of the whole
    uint4* dst = w.tinv + (size_t)i * 32 * 128 + r;
#pragma unroll 1
    for (int j = 0; j < (q >= 2 ? 2 : 1); ++j) {
      const int b = j ? h : (q >> 1) * 2 + h;
      if (j) {
        uint32_t v[32];
        tmem_ld32(trow + 64 + h * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] ^= 0x80000000u;
        split_pack<32>(reinterpret_cast<const float*>(v), hi, lo);
      }
      if (b == q) {  // the diagonal's one sits in hi
#pragma unroll
        for (int e = 0; e < 16; ++e)
          hi[e] &= e != lane >> 1 ? 0xffffffffu : lane & 1 ? 0x0000ffffu : 0xffff0000u;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 uh = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
        const uint4 ul = make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
        if (b <= q && MLSTM_IN_BOUNDS(p, (size_t)i * 32 * 128 + r + (16 + b * 4 + k) * 128 <
                                             (size_t)p.BH * w.NC * 32 * 128)) {
          dst[(b * 4 + k) * 128] = uh;
          dst[(16 + b * 4 + k) * 128] = ul;
        }
        if (kT) {
          const uint32_t off = (b >> 1) * kBlk + sw128_offset(r, (b & 1) * 4 + k);
          *reinterpret_cast<uint4*>(img + off) = uh;
          *reinterpret_cast<uint4*>(img + 2 * kBlk + off) = ul;
        }
      }
    }
    if (kT) {  // 8 columns s by 32 rows r at a time; columns of rows above are zero
      __syncthreads();
      uint32_t* out = reinterpret_cast<uint32_t*>(w.tinvt + (size_t)i * 32 * 128);
      for (int j = warp; j < 128; j += 8) {
        const int term = j >> 6, sb = (j >> 2) & 15, rg = j & 3;
        if (rg < sb >> 2) continue;
        uint32_t v[4];
        ldmatrix4_trans(
            ia + (term * 2 + (sb >> 3)) * kBlk + sw128_offset(rg * 32 + lane, sb & 7), v);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (MLSTM_IN_BOUNDS(p, term * 16 + rg * 4 + m < 32 && sb * 8 + (lane >> 2) < 128))
            out[((term * 16 + rg * 4 + m) * 128 + sb * 8 + (lane >> 2)) * 4 + (lane & 3)] = v[m];
      }
      __syncthreads();  // the diagonal blocks' place is read
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------ M and N
// Per (bh, chunk, up to 128 value columns): two rounds,
//   {W = (Tinv Lam) K, U = Tinv V}, {M = K^T (D beta W), N = K^T (D beta U)}.
// 72 products of 128 x 128 x 16 (about 4900 cycles) and 230 KB of traffic per item.
// M only with the first pair of value tiles.  The next item's Tinv and Tinv Lam are
// put in place under the second round.  1024 items: 65 to 69 us, 9.8 us an item, of
// which 7.5 are products and passes; the rest waits for the next K and V.
// Tensor memory: Tinv [0, 128), W then M [128, 256), U then N
// [256, 384), Tinv Lam [384, 512).
constexpr uint32_t kMV = 2 * kBlk, kMW = 4 * kBlk, kMU = 8 * kBlk;
constexpr uint32_t kMLam = 14 * kBlk;
constexpr uint32_t kMBar = kMLam + 512;
constexpr uint32_t kMSmem = kMBar + 64;
static_assert(kMSmem <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_mn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 GdnProblem p, const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float* slam = reinterpret_cast<float*>(smem + kMLam);
  const uint32_t ka = sbase, va = sbase + kMV, wa = sbase + kMW, ua = sbase + kMU;
  // bar_f: M of the item before has left the image
  const uint32_t bar_k = sbase + kMBar, bar_v = bar_k + 8, bar_f = bar_k + 24;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kMBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  GdnRounds rd{bar_k + 16, 0u, true, Problem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls}};
  auto load_k = [&](const GdnItem& x) {
    mbar_expect_tx(bar_k, slabs * kBlk);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, gdn_key_head(p, x.bh), bar_k);
  };
  auto load_v = [&](const GdnItem& x) {
    mbar_expect_tx(bar_v, x.tiles * kBlk);
    for (int v = 0; v < x.tiles; ++v)
      tma_load_3d(va + v * kBlk, &tm_v, (x.vt + v) * 64, x.t0, x.bh, bar_v);
  };
  uint4 ti[8];
  float2 ngc, ngl;
  float nbt;
  auto load_rows = [&](const GdnItem& x) {
    load_tinv(w.tinv + x.cb * 32 * 128, r, h, h <= q, ti);
    ngc = w.gc[x.cb * kGdnL + r];
    ngl = w.gc[x.cb * kGdnL + kGdnL - 1];
    nbt = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  GdnItem x(blockIdx.x, p, w);
  gdn_next_stage();
  if (lead) {
    for (int i = 0; i < 4; ++i) mbar_init(bar_k + 8 * i, 1);
    fence_barrier_init();
    load_k(x);
    load_v(x);
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  if (row) {
    load_rows(x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  uint32_t in_phase = 0;
  // Tinv and Tinv Lam of the item that load_rows() fetched: under the second round
  // of the item before, which needs neither of its own
  auto put_operands = [&](bool with_lam) {
    if (h == 0) slam[r] = gdn_exp(ngc);
    add_identity(r, h, ti);
    put_tinv(tlane, h, ti);
    if (!with_lam) return;
    named_bar_sync(1, kGdnRows);
    uint32_t hi[16], lo[16];
    if (h <= q) {
      float y[32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a[8], b[8];
        unpack8(ti[k], a);
        unpack8(ti[4 + k], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[8 * k + e] = (a[e] + b[e]) * slam[h * 32 + 8 * k + e];
      }
      split_pack<32>(y, hi, lo);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
    }
    tmem_st16(tlane + 384 + h * 16, hi);
    tmem_st16(tlane + 448 + h * 16, lo);
  };
  if (row) put_operands(true);

  for (long i = blockIdx.x; i < items; i += gridDim.x, in_phase ^= 1) {
    const bool more = i + gridDim.x < items;
    const GdnItem nx(more ? i + gridDim.x : i, p, w);
    const bool first = x.vt == 0;
    const uint32_t nk = idesc_bf16(128, slabs * 64, 0, 1), nkt = idesc_bf16(128, slabs * 64, 1, 1);
    const uint32_t nv = idesc_bf16(128, x.tiles * 64, 0, 1),
                   nvt = idesc_bf16(128, x.tiles * 64, 1, 1);
    const float dec = row ? nbt * gdn_decay(ngl, ngc) : 0.f;
    gdn_round(
        rd, 0x47,
        [&] {
          rd.ok = mbar_wait(bar_k, in_phase, rd.wt, 0x48);
          rd.ok = rd.ok && mbar_wait(bar_v, in_phase, rd.wt, 0x49);
          tc_fence_after();
          if (!rd.ok) return;
          if (first) mma_terms2(tmem + 128, tmem + 384, ka, nk);
          mma_terms2(tmem + 256, tmem, va, nv);
        },
        [&] {
          if (more) load_rows(nx);
          if (rd.ok) rd.ok = mbar_wait(bar_f, in_phase, rd.wt, 0x4c);
        },
        [&] {
          tma_store_wait_read_all();
          mbar_arrive(bar_f);
        },
        [&] {
          if (more) load_v(nx);
        });
    uint32_t v[32];
    if (row) {
      if (first && h < 2 * slabs) {
        tmem_ld32(trow + 128, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = dec * __uint_as_float(v[8 * cc + e]);
          put8(smem + kMW + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, y);
        }
      }
      if (h < 2 * x.tiles) {
        tmem_ld32(trow + 256, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = dec * __uint_as_float(v[8 * cc + e]);
          put_terms<3>(smem + kMU + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc, y);
        }
      }
    }
    gdn_round(
        rd, 0x4a,
        [&] {
          if (first)
            for (int t = 0; t < 2; ++t)
              mma_ss<true, true>(tmem + 128, ka, wa + 2 * t * kBlk, nkt, 2, t == 0);
          for (int t = 0; t < 3; ++t)
            mma_ss<true, true>(tmem + 256, ka, ua + 2 * t * kBlk, nvt, 2, t == 0);
        },
        [&] {
          if (more) put_operands(nx.vt == 0);
        },
        gdn_nothing,
        [&] {
          if (more) load_k(nx);
        });
    if (row) {
      if (first && h < 2 * slabs) {
        tmem_ld32(trow + 128, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          put8(smem + kMW + (h >> 1) * kBlk, 2 * kBlk, r, (h & 1) * 4 + cc,
               reinterpret_cast<const float*>(v) + 8 * cc);
      }
      if (h < 2 * x.tiles) {
        tmem_ld32(trow + 256, v);
        tmem_wait_ld();
        gdn_put_n(p, w, w.N, ((x.cb * w.nvt + x.vt + (h >> 1)) * 16 + (h & 1) * 8) * 128 + r, v);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (lead && first) {
      for (int t = 0; t < 2; ++t)
        gdn_store(p, w, w.M, 4, x.cb * 4 + 2 * t, wa + 2 * t * kBlk, slabs * kBlk);
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

}  // namespace

cudaError_t launch_gdn_tc_inverse(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                                  const GdnTcWs& w, cudaStream_t st) {
  const long items = (long)p.BH * w.NC;
  const dim3 grid((unsigned)(items < 2 * kGdnSms ? items : 2 * kGdnSms));
  if (w.tinvt)
    return gdn_launch(&gdn_tc_inverse_kernel<true>, grid, kInvThreads, inv_smem(true), false, st,
                      m.k, p, x.g, x.beta, w);
  return gdn_launch(&gdn_tc_inverse_kernel<false>, grid, kInvThreads, inv_smem(false), false, st,
                    m.k, p, x.g, x.beta, w);
}

cudaError_t launch_gdn_tc_mn(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                             const GdnTcWs& w, cudaStream_t st) {
  return gdn_launch(&gdn_tc_mn_kernel, gdn_blocks(p, w), kGdnThreads, kMSmem, true, st, m.k, m.v, p,
                    x.beta, w);
}

}  // namespace mlstm
