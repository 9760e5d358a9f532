// Gated delta rule on the tensor cores: the output, and the path's host side.
//
// Per (bh, chunk, 64 value columns), from the state S entering the chunk:
//   X = K S,  z = V - Lam X,  y = Tinv z,  H = scale (Lam Q S + P y),
//   P_rs = Gam_rs beta_s q_r.k_s (s <= r)
// Four dependent products with a pass through registers after each, bound by
// their latency: two blocks share an SM (98 KB, 256 tensor-memory columns).
// Tinv, then Q K^T and P, take columns [0, 128); X, y and P y [128, 192); Q S
// [192, 256).  z and y replace the state's image in shared memory.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr uint32_t kOffQ = 0, kOffK = 2 * kBlk, kOffS = 4 * kBlk;
constexpr uint32_t kOffGc = 6 * kBlk;
constexpr uint32_t kOffBeta = kOffGc + 1024;
constexpr uint32_t kOffBar = kOffBeta + 512;
constexpr uint32_t kSmem = kOffBar + 64 + 1024;

__global__ void __launch_bounds__(kThreads, 2)
gdn_tc_out_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  GdnProblem p, const float* __restrict__ beta,
                  const __nv_bfloat16* __restrict__ V, __nv_bfloat16* __restrict__ H, GdnTcWs w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kOffGc);
  float* sbeta = reinterpret_cast<float*>(smem + kOffBeta);
  uint8_t* img = smem + kOffS;
  const uint32_t qa = sbase + kOffQ, ka = sbase + kOffK, sa = sbase + kOffS;
  const uint32_t bar_in = sbase + kOffBar, bar = bar_in + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 32);
  const int vt = blockIdx.x, c = blockIdx.y, bh = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const int t0 = c * kGdnL, n = min(kGdnL, p.T - t0), v0 = vt * 64 + h * 32;
  const int slabs = (p.DK + 63) / 64;
  const size_t cb = (size_t)bh * w.NC + c;
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};

  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar, 1);
    fence_barrier_init();
    mbar_expect_tx(bar_in, slabs * (2 * kBlk + 2 * 8192));
    const int kh = gdn_key_head(p, bh);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, t0, kh, bar_in);
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, t0, kh, bar_in);
    }
    const uint8_t* src = w.S + (cb * w.nvt + vt) * 2 * kBlk;
    for (int t = 0; t < 2; ++t) bulk_load(sa + t * kBlk, src + t * kBlk, slabs * 8192, bar_in);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)slot), 256);
    tmem_relinquish();
  }
  uint4 vrow[4];
  {
    const __nv_bfloat16* src = V + ((long)bh * p.T + t0 + r) * p.DV + v0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      vrow[e] = r < n && v0 + 8 * e < p.DV ? *reinterpret_cast<const uint4*>(src + 8 * e)
                                           : make_uint4(0u, 0u, 0u, 0u);
  }
  if (h == 0) {
    gc[r] = w.gc[cb * kGdnL + r];
  } else {
    sbeta[r] = r < n ? beta[(long)bh * p.T + t0 + r] : 0.f;
  }
  uint4 ti[16];
  load_tinv<true>(w.tinv + cb * 32 * 128, r, h, 0, 4 * (q + 1), ti);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
  const float2 gr = gc[r];
  const float lam = gdn_exp(gr);
  bool ok = true;
  uint32_t phase = 0;
  constexpr uint32_t id = idesc_bf16(128, 64, 0, 1);
  put_tinv(trow, h, ti);

  run_mma(bar, phase, ok, wt, 0x61, [&] {
    ok = mbar_wait(bar_in, 0, wt, 0x60);
    tc_fence_after();
    if (!ok) return;
    for (int t = 0; t < 2; ++t) {
      mma_ss<false, true>(tmem + 128, ka, sa + t * kBlk, id, slabs, t == 0);
      mma_ss<false, true>(tmem + 192, qa, sa + t * kBlk, id, slabs, t == 0);
    }
  });
  uint32_t v[32];
  tmem_ld32(trow + 128 + h * 32, v);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    float x[8];
    unpack8(vrow[cc], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(-lam, __uint_as_float(v[8 * cc + e]), x[e]);
    put8(img, kBlk, r, h * 4 + cc, x);
  }
  run_mma(bar, phase, ok, wt, 0x62, [&] { mma_terms3(tmem + 128, tmem, sa, kBlk, id); });
  tmem_ld32(trow + 128 + h * 32, v);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 4; ++cc)
    put8(img, kBlk, r, h * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
  run_mma(bar, phase, ok, wt, 0x63, [&] {
    mma_ss<false, false>(tmem, qa, ka, idesc_bf16(128, 128, 0, 0), slabs, true);
  });
  // P: keys 64 h .. of the row; its terms take the scores' columns, hi then lo
  if (h * 64 <= q * 32 + 31) {
    float x[64];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      tmem_ld32(trow + h * 64 + b * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int s = h * 64 + b * 32 + e;
        x[b * 32 + e] = s <= r ? gdn_decay(gr, gc[s]) * sbeta[s] * __uint_as_float(v[e]) : 0.f;
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
  run_mma(bar, phase, ok, wt, 0x64, [&] {
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_bf16_ts(tmem + 128, tmem + (kk >> 2) * 64 + (t == 1 ? 32 : 0) + (kk & 3) * 8,
                    mnmaj(sa + (t == 2 ? kBlk : 0u), kk), id, (t | kk) != 0);
  });
  {
    uint32_t o[32];
    tmem_ld32(trow + 128 + h * 32, o);
    tmem_ld32(trow + 192 + h * 32, v);
    tmem_wait_ld();
    __nv_bfloat16* hp = H + ((long)bh * p.T + t0 + r) * p.DV + v0;
    if (r < n && ok)
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = p.scale * fmaf(lam, __uint_as_float(v[8 * cc + e]), __uint_as_float(o[8 * cc + e]));
        if (v0 + 8 * cc < p.DV) *reinterpret_cast<uint4*>(hp + 8 * cc) = pack8(x);
      }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

constexpr size_t round256(size_t x) { return (x + 255) / 256 * 256; }

GdnTcWs layout(const GdnProblem& p, bool bw, char* base) {
  GdnTcWs w{};
  w.NC = gdn_tc_chunks(p);
  w.nvt = (p.DV + 63) / 64;
  const size_t nc = (size_t)p.BH * w.NC, tile = nc * w.nvt * 2 * tc::kBlk;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = base ? reinterpret_cast<uint8_t*>(base) + at : nullptr;
    at += round256(bytes);
    return r;
  };
  w.gc = reinterpret_cast<float2*>(take(nc * kGdnL * sizeof(float2)));
  w.tinv = reinterpret_cast<uint4*>(take(nc * 32 * 128 * sizeof(uint4)));
  w.M = take(nc * 4 * tc::kBlk);
  w.N = reinterpret_cast<float4*>(take(tile));
  w.S = take(tile);
  if (bw) {
    w.tinvt = reinterpret_cast<uint4*>(take(nc * 32 * 128 * sizeof(uint4)));
    w.dS = take(tile / 2 * 3);
    w.out = reinterpret_cast<float*>(take(nc * w.nvt * 256 * sizeof(float)));
    w.y = take(tile);
    w.dz = take(tile);
    w.dz0 = reinterpret_cast<float4*>(w.dz);
    if (p.group > 1) {
      w.dq = reinterpret_cast<float*>(take((size_t)p.BH * p.T * p.DK * sizeof(float)));
      w.dk = reinterpret_cast<float*>(take((size_t)p.BH * p.T * p.DK * sizeof(float)));
    }
  }
  w.bytes = at;
  return w;
}

}  // namespace

bool gdn_tc_supported(const GdnProblem& p) {
  return p.DK <= 128 && p.DK % 8 == 0 && p.DV % 8 == 0;
}

size_t gdn_tc_workspace(const GdnProblem& p, bool backward) {
  return p.T > 0 ? layout(p, backward, nullptr).bytes : 0;
}

int gdn_tc_launches(const GdnProblem& p, bool backward) { return backward ? 6 + (p.group > 1) : 3; }

cudaError_t launch_gdn_tc_out(const GdnProblem& p, const GdnInputs& x, void* H, const GdnTcWs& w,
                              cudaStream_t st) {
  CUtensorMap tq, tk;
  const uint64_t kheads = (uint64_t)p.B * p.NHK;
  if (!encode_tmap_bf16_3d(&tq, x.Q, p.DK, p.T, kheads, 64, kGdnL) ||
      !encode_tmap_bf16_3d(&tk, x.K, p.DK, p.T, kheads, 64, kGdnL))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_tc_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  gdn_tc_out_kernel<<<dim3(w.nvt, w.NC, p.BH), kThreads, kSmem, st>>>(
      tq, tk, p, x.beta, static_cast<const __nv_bfloat16*>(x.V), static_cast<__nv_bfloat16*>(H), w);
  return cudaGetLastError();
}

cudaError_t launch_gdn_tc_fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                             void* ws, cudaStream_t st) {
  const GdnTcWs w = layout(p, false, static_cast<char*>(ws));
  cudaError_t e = launch_gdn_tc_prep(p, x, w, false, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_gdn_tc_chain(p, false, x.C0, C_T, w, st)) != cudaSuccess) return e;
  return launch_gdn_tc_out(p, x, H, w, st);
}

cudaError_t launch_gdn_tc_bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
                             cudaStream_t st) {
  const GdnTcWs w = layout(p, true, static_cast<char*>(ws));
  cudaError_t e = launch_gdn_tc_prep(p, x, w, true, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_gdn_tc_chain(p, false, x.C0, nullptr, w, st)) != cudaSuccess) return e;
  if ((e = launch_gdn_tc_dz0(p, x, d, w, st)) != cudaSuccess) return e;
  if ((e = launch_gdn_tc_chain(p, true, d.dC_T, d.dC0, w, st)) != cudaSuccess) return e;
  if ((e = launch_gdn_tc_ydz(p, x, d, w, st)) != cudaSuccess) return e;
  return launch_gdn_tc_grads(p, x, d, w, st);
}

}  // namespace mlstm
