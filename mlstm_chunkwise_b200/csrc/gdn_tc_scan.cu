// Gated delta rule on the tensor cores: the forward of many heads, fused.
//
// A block walks the chunks of one (bh, up to 128 value columns) with the state in
// tensor memory, so that M, N and the chunks' states never reach memory: 210 KB
// of traffic per 128 tokens against 730 KB of the staged forward.  Per chunk:
//   X = K S               under H's pass of the chunk before
//   Q S                   under z's pass (z = V - Lam X)
//   y = Tinv z            meanwhile Q S is scaled in place
//                         the image of D beta y in three terms, the third in V's place
//   Q K^T, S = e^G S + K^T (D beta y)   meanwhile the image of y, then P
//   H = scale (Lam Q S + P y)           meanwhile the next state's image, e^G S
// 112 products of 128 x 128 x 16 (7900 cycles), behind each of which a barrier of its
// own lets the rows go on: 8.5 to 9 us a chunk (half a us of it the third term, without
// which the final state of one chunk was off by 3.4e-6 in place of 1.5e-6), against
// 10.5 when each of four rounds waited for all of its products.  Asking L2 for the
// next chunk's tiles ahead changed nothing.  Behind the staged forward where few
// heads with many chunks leave SMs idle, see gdn_tc_fw_fused().
// Tensor memory: S [0, 128), X and y [128, 256), Tinv then Q K^T and P [256, 384),
// Q S then H [384, 512).  Shared memory blocks: K 0, 1; Q 2, 3; V, then D beta y's third
// term 4, 5; z, y, H 6..9; D beta y, then the state's image 10..13.
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr uint32_t kOffQ = 2 * kBlk, kOffV = 4 * kBlk, kOffZ = 6 * kBlk, kOffU = 10 * kBlk;
constexpr uint32_t kOffGc = 14 * kBlk;            // float2[128]
constexpr uint32_t kOffBeta = kOffGc + 1024;      // float[128]
constexpr uint32_t kOffCol = kOffBeta + 512;      // float[2][128], as in gdn_tc.cu
constexpr uint32_t kOffBar = kOffCol + 1024;
constexpr uint32_t kSmem = kOffBar + 128;
static_assert(kSmem <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_scan_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_h, GdnProblem p,
                   const float* __restrict__ beta, const float* __restrict__ C0,
                   float* __restrict__ C_T, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kOffGc);
  float* sbeta = reinterpret_cast<float*>(smem + kOffBeta);
  float* scol = reinterpret_cast<float*>(smem + kOffCol);
  const uint32_t ka = sbase, qa = sbase + kOffQ, va = sbase + kOffV, za = sbase + kOffZ,
                 ua = sbase + kOffU;
  // loads of a chunk; its products; H has left the image
  const uint32_t bar_k = sbase + kOffBar, bar_q = bar_k + 8, bar_v = bar_k + 16,
                 bar_x = bar_k + 24, bar_qs = bar_k + 32, bar_y = bar_k + 40, bar_p = bar_k + 48,
                 bar_s = bar_k + 56, bar_hp = bar_k + 64, bar_h = bar_k + 72;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 96);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64;
  const int vt = blockIdx.x * 2, bh = blockIdx.y, NC = w.NC, tiles = min(2, w.nvt - vt);
  const bool cols = row && h < 2 * tiles;
  const int v0 = vt * 64 + h * 32;  // first value column of this thread
  const int kh = gdn_key_head(p, bh);
  const Problem wt{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls};
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t phase, uint32_t site) {
    if (ok) ok = mbar_wait(bar, phase, wt, site);
    tc_fence_after();
  };
  // everything written so far is visible to the products issued behind it
  auto sync = [&] {
    fence_proxy_async_smem();
    tmem_wait_st();
    tc_fence_before();
    named_bar_sync(1, kGdnThreads);
    tc_fence_after();
  };
  auto load_qk = [&](int c) {
    mbar_expect_tx(bar_k, slabs * kBlk);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, c * kGdnL, kh, bar_k);
    mbar_expect_tx(bar_q, slabs * kBlk);
    for (int s = 0; s < slabs; ++s)
      tma_load_3d(qa + s * kBlk, &tm_q, s * 64, c * kGdnL, kh, bar_q);
  };
  auto load_v = [&](int c) {
    mbar_expect_tx(bar_v, tiles * kBlk);
    for (int v = 0; v < tiles; ++v)
      tma_load_3d(va + v * kBlk, &tm_v, (vt + v) * 64, c * kGdnL, bh, bar_v);
  };
  uint4 ti[8];
  float2 ng, ngl;
  float nb;
  auto load_gates = [&](int c) {
    const size_t at = ((size_t)bh * NC + c) * kGdnL;
    ng = w.gc[at + r];
    ngl = w.gc[at + kGdnL - 1];
    nb = c * kGdnL + r < p.T ? beta[(long)bh * p.T + c * kGdnL + r] : 0.f;
  };

  if (lead) {
    for (int i = 0; i < 10; ++i) mbar_init(bar_k + 8 * i, 1);
    fence_barrier_init();
    load_qk(0);
    load_v(0);
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  uint8_t *img = smem + kOffZ + (h >> 1) * kBlk, *imgu = smem + kOffU + (h >> 1) * kBlk;
  const uint32_t id = idesc_bf16(128, tiles * 64, 0, 1), idt = idesc_bf16(128, tiles * 64, 1, 1);

  // the state's row r (of d_qk), columns 32 h ..: its image, and e^G times it
  auto split_state = [&](uint32_t (&v)[32], float eg) {
#pragma unroll
    for (int cc = 0; cc < 4; ++cc)
      put8(imgu, 2 * kBlk, r, (h & 1) * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(eg * __uint_as_float(v[e]));
    tmem_st32(trow, v);
  };
  if (row) load_gates(0);
  if (cols) {
    uint32_t v[32];
    const float* src = C0 + ((long)bh * p.DK + r) * p.DV + v0;
    const bool have = C0 && r < p.DK && !gdn_starts_fresh(w.gc + (size_t)bh * NC * kGdnL);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const bool in = have && v0 + e < p.DV;
      const float4 x = in ? *reinterpret_cast<const float4*>(src + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[e] = __float_as_uint(x.x);
      v[e + 1] = __float_as_uint(x.y);
      v[e + 2] = __float_as_uint(x.z);
      v[e + 3] = __float_as_uint(x.w);
    }
    split_state(v, gdn_exp(ngl));
  }

  sync();
  if (!row) {
    // X = K S of the chunk whose state's image stands
    auto issue_x = [&](uint32_t ph) {
      wait(bar_k, ph, 0x80);
      if (ok)
        for (int t = 0; t < 2; ++t)
          mma_ss<false, true>(tmem + 128, ka, ua + 2 * t * kBlk, id, slabs, t == 0);
      mma_commit(bar_x);
    };
    auto issue_qs = [&](uint32_t ph) {
      wait(bar_q, ph, 0x81);
      if (ok)
        for (int t = 0; t < 2; ++t)
          mma_ss<false, true>(tmem + 384, qa, ua + 2 * t * kBlk, id, slabs, t == 0);
      mma_commit(bar_qs);
    };
    if (elect_one()) {
      issue_x(0);
      issue_qs(0);
    }
    __syncwarp();
    for (int c = 0; c < NC; ++c) {
      const uint32_t ph = c & 1;
      const bool more = c + 1 < NC;
      sync();  // z, Tinv
      if (elect_one()) {
        if (ok) mma_terms3(tmem + 128, tmem + 256, za, 2 * kBlk, id);
        mma_commit(bar_y);
      }
      __syncwarp();
      sync();  // D beta y
      if (elect_one()) {
        if (ok)
          mma_ss<false, false>(tmem + 256, qa, ka, idesc_bf16(128, 128, 0, 0), slabs, true);
        mma_commit(bar_p);
        if (ok)
          for (int t = 0; t < 3; ++t)
            mma_ss<true, true>(tmem, ka, t < 2 ? ua + 2 * t * kBlk : va, idt, 2, false);
        mma_commit(bar_s);
      }
      __syncwarp();
      if (lead && more) {
        wait(bar_s, ph, 0x82);
        if (ok) {
          load_qk(c + 1);
          load_v(c + 1);
        }
      }
      __syncwarp();
      sync();  // P, y
      if (elect_one()) {
        if (ok)
#pragma unroll
          for (int t = 0; t < 3; ++t)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tmem + 384,
                          tmem + 256 + (kk >> 1) * 32 + (t == 1 ? 16 : 0) + (kk & 1) * 8,
                          mnmaj(za + (t == 2 ? 2 * kBlk : 0u), kk), id, 1);
        mma_commit(bar_hp);
      }
      __syncwarp();
      if (more) {
        sync();  // the next state
        if (elect_one()) issue_x(ph ^ 1);
        __syncwarp();
      }
      sync();  // H
      if (lead && ok) {  // rows past T and columns past d_v are clipped
        for (int t = 0; t < tiles; ++t)
          if (MLSTM_IN_BOUNDS(p, gdn_box_inside(p, (vt + t) * 64, p.DV, c * kGdnL, bh, p.BH)))
            tma_store_3d(&tm_h, za + t * kBlk, (vt + t) * 64, c * kGdnL, bh);
        tma_store_commit();
      }
      __syncwarp();
      if (!more) break;
      if (elect_one()) issue_qs(ph ^ 1);
      __syncwarp();
      if (lead) {
        tma_store_wait_read_all();
        mbar_arrive(bar_h);
      }
      __syncwarp();
    }
  } else {
    for (int c = 0; c < NC; ++c) {
      const uint32_t ph = c & 1;
      const bool more = c + 1 < NC;
      load_tinv(w.tinv + ((size_t)bh * NC + c) * 32 * 128, r, h, h <= q, ti);
      const float2 gr = ng;
      const float dec = nb * gdn_decay(ngl, gr), lam = gdn_exp(gr);
      if (h == 0) {
        gc[r] = gr;
        sbeta[r] = nb;
        scol[r] = nb * gdn_col_factor(gr, 31);
        scol[128 + r] = __fdividef(nb, gdn_col_factor(gr, 0));
      }
      uint32_t v[32];
      add_identity(r, h, ti);
      put_tinv(tlane + 256, h, ti);
      wait(bar_v, ph, 0x83);
      if (c > 0) wait(bar_h, ph ^ 1, 0x84);
      wait(bar_x, ph, 0x85);
      if (cols) {
        tmem_ld32(trow + 128, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float z[8];
          unpack8(*reinterpret_cast<const uint4*>(smem + kOffV + (h >> 1) * kBlk +
                                                  sw128_offset(r, (h & 1) * 4 + cc)),
                  z);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = fmaf(-lam, __uint_as_float(v[8 * cc + e]), z[e]);
          put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, z);
        }
      }
      sync();
      wait(bar_qs, ph, 0x86);
      if (cols) {
        const float f = p.scale * lam;
        tmem_ld32(trow + 384, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(f * __uint_as_float(v[e]));
        tmem_st32(trow + 384, v);
      }
      if (more) load_gates(c + 1);
      wait(bar_y, ph, 0x87);
      if (cols) {
        tmem_ld32(trow + 128, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = dec * __uint_as_float(v[8 * cc + e]);
          put_terms<3>(imgu, 2 * kBlk, r, (h & 1) * 4 + cc, y, (int)kOffV - (int)kOffU);
        }
      }
      sync();
      if (cols) {
        tmem_ld32(trow + 128, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
      }
      // P: 32 keys of the row; its terms take the scores' columns, hi then lo
      wait(bar_p, ph, 0x88);
      uint32_t hi[16], lo[16];
      if (h <= q) {
        tmem_ld32(trow + 256, v);
        tmem_wait_ld();
        float s[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = p.scale * __uint_as_float(v[e]);
        if (h == q && gc[h * 32].x - gc[h * 32 + 31].x > kGdnFlat) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int k = h * 32 + e;
            s[e] = e <= lane ? gdn_decay(gr, gc[k]) * sbeta[k] * s[e] : 0.f;
          }
        } else {
          const bool d = h == q;
          const float f = gdn_decay(gr, gc[h * 32 + (d ? 0 : 31)]);
          const float* sc = scol + (d ? 128 : 0) + h * 32;
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = d && e > lane ? 0.f : s[e] * (f * sc[e]);
        }
        split_pack<32>(s, hi, lo);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
      }
      tmem_st16(trow + 256, hi);
      tmem_st16(trow + 272, lo);
      sync();
      wait(bar_s, ph, 0x89);
      if (cols) {
        tmem_ld32(trow, v);
        tmem_wait_ld();
        if (more) {
          split_state(v, gdn_exp(ngl));
        } else if (C_T && r < p.DK && ok) {
          float* dst = C_T + ((long)bh * p.DK + r) * p.DV + v0;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            if (v0 + e < p.DV && MLSTM_IN_BOUNDS(p, bh < p.BH && v0 + e + 4 <= p.DV))
              *reinterpret_cast<float4*>(dst + e) =
                  make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                              __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        }
      }
      if (more) sync();
      wait(bar_hp, ph, 0x8a);
      if (cols) {
        tmem_ld32(trow + 384, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          *reinterpret_cast<uint4*>(img + sw128_offset(r, (h & 1) * 4 + cc)) =
              pack8(reinterpret_cast<const float*>(v) + 8 * cc);
      }
      sync();
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

// By what the two cost in us, measured: a chunk takes a fused block 9; the staged
// forward takes a wave of 148 (head, chunk, pair of value tiles) 21 (mn and out),
// its recurrence 1.45 a chunk, and two more launches 5.  So the fused one runs for
// one to three chunks, and from about a third of a wave of heads on.  (64 chunks,
// 128 x 128, us staged and fused: 32 heads 417, 585; 48 heads 574, 618; 56 heads 660,
// 635; 64 heads 740, 646.  32 chunks: 148 heads 890, 413; 256 heads 1480, 761.  16
// chunks: 16 heads 87, 153; 40 heads 157, 167; 48 heads 178, 171.  16 heads: 2 chunks
// 52, 42; 3 chunks 52, 50.)
bool gdn_tc_fw_fused(const GdnProblem& p) {
  const long nc = gdn_tc_chunks(p), heads = (long)p.BH * ((p.DV + 127) / 128);
  auto waves = [](long n) { return (n + kGdnSms - 1) / kGdnSms; };
  const long fused = 900 * nc * waves(heads);
  const long staged = 2100 * waves(heads * nc) +
                      145 * nc * waves((long)p.BH * ((p.DV + 63) / 64)) + 500;
  return fused <= staged;
}

cudaError_t launch_gdn_tc_scan(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m, float* C_T,
                               const GdnTcWs& w, cudaStream_t st) {
  return gdn_launch(&gdn_tc_scan_kernel, dim3((w.nvt + 1) / 2, p.BH), kGdnThreads, kSmem, true, st,
                    m.q, m.k, m.v, m.h, p, x.beta, x.C0, C_T, w);
}

}  // namespace mlstm
