// Gated delta rule on the tensor cores: the output, and the path's host side.
//
// Per (bh, chunk, up to 128 value columns), from the state S entering the chunk:
//   X = K S,  z = V - Lam X,  y = Tinv z,  H = scale (Lam Q S + P y),
//   P_rs = Gam_rs beta_s q_r.k_s (s <= r)
// Persistent, one block per SM.  Three rounds of products with a pass through
// registers after each: {K S, Q S, Q K^T}, under which Tinv goes to tensor memory;
// {Tinv z}, under which P is formed; {P y}.  The next item's tiles are copied in as
// soon as this one's have been read.  88 products of 128 x 128 x 16 (about 6000
// cycles) and 230 KB of traffic per item.  1024 items: 78 us (82 with y kept), 11 us
// an item, of which about 7 are products and passes; the rest waits for the next
// tiles, although HBM runs at 2.9 TB/s and nothing is saturated (tensor pipe 22%,
// issue slots 30%).  Two blocks per SM on 64 columns each with four rounds took
// 101 us (Tinv, Q, K and P twice, loads exposed).
// Tensor memory: Tinv [0, 128), Q K^T then P [128, 256), X, y, P y [256, 384),
// Q S [384, 512).
#include <cuda.h>

#include "gdn_tc.h"

namespace mlstm {
namespace {

using namespace tc;

constexpr uint32_t kOffQ = 0, kOffK = 2 * kBlk, kOffS = 4 * kBlk, kOffZ = 8 * kBlk;
constexpr uint32_t kOffV = 12 * kBlk;
constexpr uint32_t kOffGc = 14 * kBlk;            // float2[128]
constexpr uint32_t kOffBeta = kOffGc + 1024;      // float[128]
constexpr uint32_t kOffCol = kOffBeta + 512;      // float[2][128], beta times the column's factor
                                                  // (below the diagonal's block, in it)
constexpr uint32_t kOffBar = kOffCol + 1024;
constexpr uint32_t kSmem = kOffBar + 64;
static_assert(kSmem <= 227 * 1024, "shared memory");

// kH: writes H.  kY: keeps y for the backward.
template <bool kH, bool kY>
__global__ void __launch_bounds__(kGdnThreads, 1)
gdn_tc_out_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_h,
                  GdnProblem p, const float* __restrict__ beta, GdnTcWs w) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float2* gc = reinterpret_cast<float2*>(smem + kOffGc);
  float* sbeta = reinterpret_cast<float*>(smem + kOffBeta);
  float* scol = reinterpret_cast<float*>(smem + kOffCol);
  const uint32_t qa = sbase + kOffQ, ka = sbase + kOffK, sa = sbase + kOffS, za = sbase + kOffZ;
  // bar_f: what the image held (y or H of the item before) has left
  const uint32_t bar_in = sbase + kOffBar, bar_v = bar_in + 8, bar_f = bar_in + 24;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2, r = q * 32 + lane;
  const bool row = tid < kGdnRows, lead = tid == kGdnRows;
  const int slabs = (p.DK + 63) / 64;
  const long items = (long)p.BH * w.NC * ((w.nvt + 1) / 2);
  GdnRounds rd{bar_in + 16, 0u, true, Problem{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.f, 0, p.err, p.max_polls}};
  auto load_tiles = [&](const GdnItem& x, bool wait) {
    mbar_expect_tx(bar_in, slabs * ((kH ? 2 : 1) * kBlk + x.tiles * 2 * 8192));
    const int kh = gdn_key_head(p, x.bh);
    for (int s = 0; s < slabs; ++s) {
      tma_load_3d(ka + s * kBlk, &tm_k, s * 64, x.t0, kh, bar_in);
      if (kH) tma_load_3d(qa + s * kBlk, &tm_q, s * 64, x.t0, kh, bar_in);
    }
    if (wait) gdn_wait_stage();
    for (int v = 0; v < x.tiles; ++v)
      for (int t = 0; t < 2; ++t)
        gdn_load(p, w, sa + (2 * t + v) * kBlk, w.S, 2 * w.nvt,
                 (x.cb * w.nvt + x.vt + v) * 2 + t, slabs * 8192, bar_in);
  };
  auto load_v = [&](const GdnItem& x) {
    mbar_expect_tx(bar_v, x.tiles * kBlk);
    for (int v = 0; v < x.tiles; ++v)
      tma_load_3d(sbase + kOffV + v * kBlk, &tm_v, (x.vt + v) * 64, x.t0, x.bh, bar_v);
  };
  uint4 ti[8];
  float2 ng;
  float nb;
  auto load_gates = [&](const GdnItem& x) {
    ng = w.gc[x.cb * kGdnL + r];
    nb = r < x.n ? beta[(long)x.bh * p.T + x.t0 + r] : 0.f;
  };

  GdnItem x(blockIdx.x, p, w);
  gdn_next_stage();
  if (lead) {
    for (int i = 0; i < 4; ++i) mbar_init(bar_in + 8 * i, 1);
    fence_barrier_init();
    load_v(x);
    load_tiles(x, true);
  }
  if (!row) {
    __syncwarp();
    tmem_alloc(smem_u32((const void*)slot), 512);
    tmem_relinquish();
  }
  gdn_wait_stage();
  if (row) load_gates(x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16), trow = tlane + h * 32;
  uint8_t* img = smem + kOffZ + (h >> 1) * kBlk;
  uint32_t in_phase = 0;

  for (long i = blockIdx.x; i < items; i += gridDim.x, in_phase ^= 1) {
    const bool more = i + gridDim.x < items;
    const GdnItem nx(more ? i + gridDim.x : i, p, w);
    const bool cols = row && h < 2 * x.tiles;  // this thread's value columns exist
    const uint32_t id = idesc_bf16(128, x.tiles * 64, 0, 1);
    float2 gr = make_float2(0.f, 0.f);
    if (row) {
      gr = ng;
      if (kH && h == 0) {
        gc[r] = gr;
        sbeta[r] = nb;
        scol[r] = nb * gdn_col_factor(gr, 31);
        scol[128 + r] = __fdividef(nb, gdn_col_factor(gr, 0));
      }
      load_tinv(w.tinv + x.cb * 32 * 128, r, h, h <= q, ti);  // for the second round
    }
    gdn_round(
        rd, 0x61,
        [&] {
          rd.ok = mbar_wait(bar_in, in_phase, rd.wt, 0x60);
          tc_fence_after();
          if (!rd.ok) return;
          for (int t = 0; t < 2; ++t)
            mma_ss<false, true>(tmem + 256, ka, sa + 2 * t * kBlk, id, slabs, t == 0);
          if (kH) {
            mma_ss<false, false>(tmem + 128, qa, ka, idesc_bf16(128, 128, 0, 0), slabs, true);
            for (int t = 0; t < 2; ++t)
              mma_ss<false, true>(tmem + 384, qa, sa + 2 * t * kBlk, id, slabs, t == 0);
          }
        },
        [&] {
          add_identity(r, h, ti);
          put_tinv(tlane, h, ti);
          if (more) load_gates(nx);
          if (rd.ok) rd.ok = mbar_wait(bar_v, in_phase, rd.wt, 0x65);
          if (rd.ok) rd.ok = mbar_wait(bar_f, in_phase, rd.wt, 0x66);
        },
        [&] {
          tma_store_wait_read_all();
          mbar_arrive(bar_f);
        },
        [&] {
          if (more) load_tiles(nx, false);
        });
    const float lam = gdn_exp(gr);
    uint32_t v[32];
    if (cols) {
      tmem_ld32(trow + 256, v);
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
    gdn_round(
        rd, 0x62, [&] { mma_terms3(tmem + 256, tmem, za, 2 * kBlk, id); },
        [&] {
          if (!kH) return;
          // P: 32 keys of the row; its terms take the scores' columns, hi then lo
          uint32_t hi[16], lo[16];
          if (h <= q) {
            tmem_ld32(trow + 128, v);
            tmem_wait_ld();
            float s[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(v[e]);
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
          tmem_st16(trow + 128, hi);
          tmem_st16(trow + 144, lo);
        },
        [&] {
          if (more) load_v(nx);
        },
        gdn_nothing);
    if (cols) {
      tmem_ld32(trow + 256, v);
      tmem_wait_ld();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc)
        put8(img, 2 * kBlk, r, (h & 1) * 4 + cc, reinterpret_cast<const float*>(v) + 8 * cc);
    }
    auto keep_y = [&] {
      for (int t = 0; t < x.tiles; ++t)
        for (int term = 0; term < 2; ++term)
          gdn_store(p, w, w.y, 2 * w.nvt, (x.cb * w.nvt + x.vt + t) * 2 + term,
                    za + (2 * term + t) * kBlk, kBlk);
      tma_store_commit();
    };
    if (kH) {
      gdn_round(
          rd, 0x64,
          [&] {
#pragma unroll
            for (int t = 0; t < 3; ++t)
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ts(tmem + 256,
                            tmem + 128 + (kk >> 1) * 32 + (t == 1 ? 16 : 0) + (kk & 1) * 8,
                            mnmaj(za + (t == 2 ? 2 * kBlk : 0u), kk), id, (t | kk) != 0);
          },
          gdn_nothing,
          [&] {
            if (!kY) return;
            keep_y();
            tma_store_wait_read_all();
          },
          gdn_nothing);
      if (kY) __syncthreads();  // y has left: H takes its place
      if (cols) {
        uint32_t o[32];
        tmem_ld32(trow + 256, o);
        tmem_ld32(trow + 384, v);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = p.scale *
                   fmaf(lam, __uint_as_float(v[8 * cc + e]), __uint_as_float(o[8 * cc + e]));
          *reinterpret_cast<uint4*>(img + sw128_offset(r, (h & 1) * 4 + cc)) = pack8(y);
        }
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (lead && rd.ok) {
      if (kH) {  // rows past T and columns past d_v are clipped
        for (int t = 0; t < x.tiles; ++t)
          if (MLSTM_IN_BOUNDS(p, gdn_box_inside(p, (x.vt + t) * 64, p.DV, x.t0, x.bh, p.BH)))
            tma_store_3d(&tm_h, za + t * kBlk, (x.vt + t) * 64, x.t0, x.bh);
        tma_store_commit();
      } else {
        keep_y();
      }
    }
    x = nx;
  }
  if (lead) tma_store_wait_all();
  tc_fence_before();
  __syncthreads();
  if (!row) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Parts of the workspace.  kKeep: what outlives the forward of the training pair
// beside kState; kInverse and kN of the forward do not.
enum : int { kSums = 1, kState = 2, kKeep = 4, kInverse = 8, kN = 16, kGrad = 32 };

// Sets the pointers of `parts` in w from `base` on; returns their bytes.
size_t carve(const GdnProblem& p, int parts, const void* base, GdnTcWs* w) {
  w->NC = gdn_tc_chunks(p);
  w->nvt = (p.DV + 63) / 64;
  const size_t nc = (size_t)p.BH * w->NC, tile = nc * w->nvt * 2 * tc::kBlk;
  const size_t inverse = nc * 32 * 128 * sizeof(uint4);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = static_cast<uint8_t*>(const_cast<void*>(base));
    r = r ? r + at : nullptr;
    at += round256(bytes);
    return r;
  };
  if (parts & kSums) w->gc = reinterpret_cast<float2*>(take(nc * kGdnL * sizeof(float2)));
  if (parts & kState) {
    w->M = take(nc * 4 * tc::kBlk);
    w->S = take(tile);
  }
  if (parts & kKeep) {
    w->tinvt = reinterpret_cast<uint4*>(take(inverse));
    w->y = take(tile);
  }
  if (parts & kInverse) w->tinv = reinterpret_cast<uint4*>(take(inverse));
  if (parts & kN) w->N = reinterpret_cast<float4*>(take(tile));
  if (parts & kGrad) {
    w->dS = take(tile / 2 * 3);
    w->dz = take(tile);
    w->dz0 = reinterpret_cast<float4*>(w->dz);
    w->out = reinterpret_cast<float*>(take(nc * w->nvt * 256 * sizeof(float)));
    if (p.group > 1) {
      w->dq = reinterpret_cast<float*>(take((size_t)p.BH * p.T * p.DK * sizeof(float)));
      w->dk = reinterpret_cast<float*>(take((size_t)p.BH * p.T * p.DK * sizeof(float)));
    }
  }
  return at;
}
int fw_parts(const GdnProblem& p) {
  return kSums | kInverse | (gdn_tc_fw_fused(p) ? 0 : kState | kN);
}
constexpr int kBwParts = kSums | kState | kKeep | kInverse | kN | kGrad;
constexpr int kSaved = kSums | kState | kKeep;

bool map16(CUtensorMap* m, const void* base, int cols, int T, long heads) {
  return encode_tmap_bf16_3d(m, base, cols, T, heads, 64, kGdnL);
}

cudaError_t forward(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T, GdnMaps& m,
                    const GdnTcWs& w, cudaStream_t st) {
  const long kheads = (long)p.B * p.NHK;
  if (!map16(&m.k, x.K, p.DK, p.T, kheads) || !map16(&m.q, x.Q, p.DK, p.T, kheads) ||
      !map16(&m.v, x.V, p.DV, p.T, p.BH) || (H && !map16(&m.h, H, p.DV, p.T, p.BH)))
    return cudaErrorInvalidValue;
  if (!H) m.h = m.v;
  cudaError_t e = launch_gdn_tc_inverse(p, x, m, w, st);
  if (e != cudaSuccess) return e;
  if (!w.M) return launch_gdn_tc_scan(p, x, m, C_T, w, st);
  if ((e = launch_gdn_tc_mn(p, x, m, w, st)) != cudaSuccess) return e;
  if ((e = launch_gdn_tc_chain(p, false, x.C0, C_T, w, st)) != cudaSuccess) return e;
  return launch_gdn_tc_out(p, x, m, H != nullptr, w, st);
}
// behind: forward() ran before, with m's Q and K.
cudaError_t backward(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, bool behind,
                     GdnMaps& m, const GdnTcWs& w, cudaStream_t st) {
  const long kheads = (long)p.B * p.NHK;
  if (!behind && (!map16(&m.k, x.K, p.DK, p.T, kheads) || !map16(&m.q, x.Q, p.DK, p.T, kheads)))
    return cudaErrorInvalidValue;
  if (!map16(&m.dh, d.dH, p.DV, p.T, p.BH) || !map16(&m.dv, d.dV, p.DV, p.T, p.BH))
    return cudaErrorInvalidValue;
  if (w.dq ? !encode_tmap_3d(&m.dq, w.dq, 4, p.DK, p.T, p.BH, 32, kGdnL, 128) ||
                 !encode_tmap_3d(&m.dk, w.dk, 4, p.DK, p.T, p.BH, 32, kGdnL, 128)
           : !map16(&m.dq, d.dQ, p.DK, p.T, kheads) || !map16(&m.dk, d.dK, p.DK, p.T, kheads))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_gdn_tc_dz0(p, x, m, behind, w, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_gdn_tc_chain(p, true, d.dC_T, d.dC0, w, st)) != cudaSuccess) return e;
  if ((e = launch_gdn_tc_dz(p, x, m, w, st)) != cudaSuccess) return e;
  return launch_gdn_tc_grads(p, x, d, m, w, st);
}

}  // namespace

bool gdn_tc_supported(const GdnProblem& p) {
  return p.DK <= 128 && p.DK % 8 == 0 && p.DV % 8 == 0;
}

size_t gdn_tc_workspace(const GdnProblem& p, bool backward) {
  GdnTcWs w{};
  return p.T > 0 ? carve(p, backward ? kBwParts : fw_parts(p), nullptr, &w) : 0;
}
GdnTrainSizes gdn_tc_train_sizes(const GdnProblem& p) {
  GdnTcWs w{};
  return {carve(p, kSaved, nullptr, &w), carve(p, kInverse | kN, nullptr, &w),
          carve(p, kN | kGrad, nullptr, &w)};
}

int gdn_tc_train_launches(const GdnProblem& p, bool backward) {
  return backward ? 4 + (p.group > 1) : 4;
}
int gdn_tc_launches(const GdnProblem& p, bool backward) {
  return backward ? 4 + gdn_tc_train_launches(p, true) : gdn_tc_fw_fused(p) ? 2 : 4;
}

cudaError_t launch_gdn_tc_out(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                              bool with_h, const GdnTcWs& w, cudaStream_t st) {
  auto go = [&](auto* kern) {
    return gdn_launch(kern, gdn_blocks(p, w), kGdnThreads, kSmem, true, st, m.q, m.k, m.v, m.h, p,
                      x.beta, w);
  };
  if (!with_h) return go(&gdn_tc_out_kernel<false, true>);
  return w.y ? go(&gdn_tc_out_kernel<true, true>) : go(&gdn_tc_out_kernel<true, false>);
}

cudaError_t launch_gdn_tc_fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                             void* ws, cudaStream_t st) {
  GdnTcWs w{};
  carve(p, fw_parts(p), ws, &w);
  GdnMaps m;
  return forward(p, x, H, C_T, m, w, st);
}
cudaError_t launch_gdn_tc_bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
                             cudaStream_t st) {
  GdnTcWs w{};
  carve(p, kBwParts, ws, &w);
  GdnMaps m;
  const cudaError_t e = forward(p, x, nullptr, nullptr, m, w, st);
  return e == cudaSuccess ? backward(p, x, d, true, m, w, st) : e;
}
cudaError_t launch_gdn_tc_fw_train(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                                   void* saved, void* ws, cudaStream_t st) {
  GdnTcWs w{};
  carve(p, kSaved, saved, &w);
  carve(p, kInverse | kN, ws, &w);
  GdnMaps m;
  return forward(p, x, H, C_T, m, w, st);
}
cudaError_t launch_gdn_tc_bw_saved(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                                   const void* saved, void* ws, cudaStream_t st) {
  GdnTcWs w{};
  carve(p, kSaved, saved, &w);
  carve(p, kN | kGrad, ws, &w);
  GdnMaps m;
  return backward(p, x, d, false, m, w, st);
}

}  // namespace mlstm
