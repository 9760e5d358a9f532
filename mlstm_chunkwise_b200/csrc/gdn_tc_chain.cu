// Gated delta rule, tensor cores: the recurrence over chunks, of the state
// (S' = e^G S + N - M S) or of its gradient (dS = e^G dS' + N' - M^T dS', from
// the last chunk to the first).  A CTA owns one (bh, 64 value columns); its
// 512 row threads keep the state in fp32 registers.  Per chunk: the state goes
// to shared memory as an operand image (two bf16 terms, which are also what
// the chunk's other kernels read), one product with M gives X, and the threads
// update.  M arrives two chunks ahead, N one chunk ahead in registers.
//
// The chain image -> product -> registers is what bounds it: 2250 cycles a chunk,
// 980 of them products, the rest the pass (300), the proxy fence (270) and the
// hand-overs to the issuing thread and back (430).  32 chunks of 16 heads: 47 us;
// with HBM mostly idle unless more than one wave of CTAs runs (256 heads: 256 us,
// 1.9 GB).
//
// Warps: 0 loads M, 1 issues the products and stores the images, 2..17 rows
// (four threads per row, 16 columns each).
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr int kRows = 512;  // row threads, four to a row
constexpr int kThreads = 64 + kRows;
constexpr uint32_t kOffM = 0;                // 2 x 64 KB
constexpr uint32_t kOffS = 8 * kBlk;         // 2 x 32 KB (reverse: three terms, 48 KB)
constexpr uint32_t kOffBar = 14 * kBlk;
constexpr uint32_t kSmem = kOffBar + 64 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
enum : uint32_t { kMFull0, kMFull1, kMFree0, kMFree1, kSop, kX, kBars };

template <bool kRev>
__global__ void __launch_bounds__(kThreads, 1)
gdn_tc_chain_kernel(GdnProblem p, const float* __restrict__ init, float* __restrict__ fin,
                    GdnTcWs w) {
  constexpr int kTerms = kRev ? 3 : 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](uint32_t i) { return sbase + kOffBar + 8 * i; };
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 56);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vt = blockIdx.x, bh = blockIdx.y, NC = w.NC;
  const int slabs = (p.DK + 63) / 64;
  // without a final state the last chunk only needs its image
  const int steps = fin ? NC : NC - 1;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};
  auto chunk = [&](int i) { return (size_t)bh * NC + (kRev ? NC - 1 - i : i); };

  gdn_next_stage();
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kBars; ++i) mbar_init(bar(i), i == kSop ? kRows / 32 : 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  gdn_wait_stage();

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < steps && ok; ++i) {
        const int b = i & 1;
        if (i >= 2) ok = mbar_wait(bar(kMFree0 + b), ((i >> 1) - 1) & 1, wt, 0x51);
        if (!ok) break;
        mbar_expect_tx(bar(kMFull0 + b), 2 * slabs * kBlk);
        for (int t = 0; t < 2; ++t)
          gdn_load(p, w, sbase + kOffM + (4 * b + 2 * t) * kBlk, w.M, 4, chunk(i) * 4 + 2 * t,
                   slabs * kBlk, bar(kMFull0 + b));
      }
      // every load has landed before the CTA exits
      for (int i = steps > 2 ? steps - 2 : 0; ok && i < steps; ++i)
        ok = mbar_wait(bar(kMFull0 + (i & 1)), (i >> 1) & 1, wt, 0x52);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // M's hi term against both terms of the state at once (128 columns), then its
      // lo term against hi: 16 issues of 16 inner indexes, 980 cycles, for 24 of
      // 64 columns, 1270
      constexpr uint32_t id2 = idesc_bf16(128, 128, kRev ? 1 : 0, 1);
      constexpr uint32_t id = idesc_bf16(128, 64, kRev ? 1 : 0, 1);
      bool ok = true;
      for (int i = 0; i < NC && ok; ++i) {
        const int b = i & 1;
        const uint32_t ma = sbase + kOffM + 4 * b * kBlk, sa = sbase + kOffS + kTerms * b * kBlk;
        if (i < steps) ok = mbar_wait(bar(kMFull0 + b), (i >> 1) & 1, wt, 0x53);
        ok = ok && mbar_wait(bar(kSop), i & 1, wt, 0x54);
        tc_fence_after();
        if (!ok) break;
        if (i < steps) {
          mma_ss<kRev, true>(tmem, ma, sa, id2, slabs, true);
          mma_ss<kRev, true>(tmem, ma + 2 * kBlk, sa, id, slabs, false);
          // the other image has left before X of this chunk lets the rows rewrite it
          tma_store_wait_read_all();
          mma_commit(bar(kX));
          mma_commit(bar(kMFree0 + b));
        }
        for (int t = 0; t < kTerms; ++t)
          gdn_store(p, w, kRev ? w.dS : w.S, kTerms * w.nvt, (chunk(i) * w.nvt + vt) * kTerms + t,
                    sa + t * kBlk, slabs * 8192);
        tma_store_commit();
      }
      tma_store_wait_all();
    }
  } else {
    const int q = warp & 3, r = q * 32 + lane, h = (warp - 2) >> 2;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + h * 16;
    const int v0 = vt * 64 + h * 16;  // first value column of this thread
    bool ok = true;
    float s[16];
    float4 n[4];
    float2 gl;
    auto load = [&](int i) {
      const float4* src = w.N + ((chunk(i) * w.nvt + vt) * 16 + h * 4) * 128 + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = src[e * 128];
      gl = w.gc[chunk(i) * kGdnL + kGdnL - 1];
    };
    if (steps > 0) load(0);
    const bool have = init && r < p.DK && (kRev || !gdn_starts_fresh(w.gc + chunk(0) * kGdnL));
#pragma unroll
    for (int e = 0; e < 16; ++e)
      s[e] = have && v0 + e < p.DV ? init[((long)bh * p.DK + r) * p.DV + v0 + e] : 0.f;
    for (int i = 0; i < NC; ++i) {
      uint8_t* img = smem + kOffS + (i & 1) * kTerms * kBlk;
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        put_terms<kTerms>(img, kBlk, r, h * 2 + cc, s + 8 * cc);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSop));
      if (i == steps) break;
      const float eg = gdn_exp(gl);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[4 * e] = fmaf(eg, s[4 * e], n[e].x);
        s[4 * e + 1] = fmaf(eg, s[4 * e + 1], n[e].y);
        s[4 * e + 2] = fmaf(eg, s[4 * e + 2], n[e].z);
        s[4 * e + 3] = fmaf(eg, s[4 * e + 3], n[e].w);
      }
      if (i + 1 < steps) load(i + 1);
      ok = ok && mbar_wait(bar(kX), i & 1, wt, 0x55);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[16], u[16];
      tmem_ld16(trow, v);
      tmem_ld16(trow + 64, u);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] -= __uint_as_float(v[e]) + __uint_as_float(u[e]);
    }
    if (fin && ok && r < p.DK)
#pragma unroll
      for (int e = 0; e < 16; e += 4)  // DV is a multiple of 8
        if (v0 + e < p.DV && MLSTM_IN_BOUNDS(p, bh < p.BH && v0 + e + 4 <= p.DV))
          *reinterpret_cast<float4*>(fin + ((long)bh * p.DK + r) * p.DV + v0 + e) =
              make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

}  // namespace

cudaError_t launch_gdn_tc_chain(const GdnProblem& p, bool reverse, const float* init, float* fin,
                                const GdnTcWs& w, cudaStream_t st) {
  const dim3 grid(w.nvt, p.BH);
  if (reverse)
    return gdn_launch(&gdn_tc_chain_kernel<true>, grid, kThreads, kSmem, true, st, p, init, fin, w);
  return gdn_launch(&gdn_tc_chain_kernel<false>, grid, kThreads, kSmem, true, st, p, init, fin, w);
}

}  // namespace mlstm
