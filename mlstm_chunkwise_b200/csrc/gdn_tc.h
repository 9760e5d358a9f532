// Shared pieces of the gated delta rule's tensor-core kernels (bf16 inputs,
// d_qk up to 128, chunks of L = 128 tokens; formulas in gdn.h).
//
// The state entering a chunk obeys a recurrence with one product per chunk,
//   S' = e^G S + N - M S,   M = K^T (D beta W),  W = Tinv (Lam K),
//                           N = K^T (D beta U),  U = Tinv V,
// and the gradient of the state leaving it the transposed one,
//   dS = e^G dS' + N' - M^T dS',
//   N' = Q^T (scale Lam dH) - K^T (Lam Tinv^T (beta scale (Gam . QK^T)^T dH)).
// M, N and N' of all chunks are formed in parallel; only the recurrences run
// chunk after chunk (gdn_tc_chain.cu), and outputs and gradients are again
// formed for all chunks in parallel from the stored states.
//
// Precision.  Q, K, V and dH are exact bf16 operands.  Every other operand of a
// product (state, inverse, z, y, the gated score matrices, and their
// gradients) is an fp32 value carried as two bf16 terms, hi = bf16(x) and
// lo = bf16(x - hi), off by at most 2^-16 of its value; the product of two such
// operands drops only lo.lo.  So fp32 outputs (state, gate gradients) keep
// about 17 bits at two or three tensor-core products in place of one.  A single
// bf16 rounding of the state or of the inverse would put 2e-3 of noise on
// every output, and dg, a difference of large sums, off by percents.  Where one
// rounding alone would set the error of an fp32 output, the operand has a third
// term (24 bits) or the sum is taken in fp32: the last operands of N and N' and what
// the fused forward writes to the state (final state, dC0), the gradient of the state
// in K dS', and y against it (dbeta, dg).  In y dS'^T (a term of the bf16 dK) and in
// <S, dS'> (beside S, which has two) the gradient of the state enters with its first
// two terms.  Exponentials are ex2.approx (2^-22 of the value) with the exponent's
// rounding carried along, quotients of them __fdividef (2^-22): a quarter of 2^-20 at
// most, an order below two terms.
#pragma once

#include "device_address.h"
#include "gdn.h"
#include "tc_ptx.cuh"

namespace mlstm {

constexpr int kGdnL = 128;  // chunk length of the tensor-core path

inline int gdn_tc_chunks(const GdnProblem& p) { return (p.T + kGdnL - 1) / kGdnL; }

// Workspace pieces, per (bh, chunk).  Operand images hold rows of 128 bytes (64
// columns of one bf16 term, 128-byte swizzle), 128 rows to a block of 16 KB.
//   gc     float2[128]          inclusive sums of g inside the chunk (hi, lo)
//   tinv   uint4[32][128]       Tinv - I by rows as bf16 terms: piece j < 16 holds columns
//                               8j .. 8j + 7 of hi, j >= 16 those of lo; row r at [j][r],
//                               so that a warp of row threads reads 512 contiguous bytes.
//                               Pieces right of the diagonal's 32 x 32 block are not
//                               written (they are zero).
//   tinvt  uint4[32][128]       the same of Tinv^T (backward); pieces left of the
//                               diagonal's block are not written
//   M      [2 terms][2][16 KB]  image, rows i, columns j in two blocks of 64
//   N      [value tile] float4[16][128]: columns 4c .. 4c + 3 of row r at [c][r]; N', then
//                               dz without its part from dS', in the same form
//   S      [value tile][2 terms][16 KB]  state entering the chunk: rows d_qk, 64 value
//                               columns
//   dS     [value tile][3 terms][16 KB]  gradient of the state leaving the chunk
//   out    float[value tile][2][128]  D_s y_s.(dS'^T k_s) over 32 columns each
//   y, dz  [value tile][2 terms][16 KB]  rows are tokens
struct GdnTcWs {
  float2* gc;
  uint4 *tinv, *tinvt;
  uint8_t *M, *S, *dS, *y, *dz;
  float* out;
  float4 *N, *dz0;  // dz0 lies in dz: a tile's reader replaces it
  float *dq, *dk;   // fp32 [BH][T][DK], with shared key heads
  int NC, nvt;      // chunks, value tiles of 64 columns
  size_t bytes;
};

bool gdn_tc_supported(const GdnProblem& p);
size_t gdn_tc_workspace(const GdnProblem& p, bool backward);
int gdn_tc_launches(const GdnProblem& p, bool backward);
cudaError_t launch_gdn_tc_fw(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                             void* ws, cudaStream_t st);
cudaError_t launch_gdn_tc_bw(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d, void* ws,
                             cudaStream_t st);
// The pair that hands the chunks' sums, inverses, M, states and y on in `saved`.
struct GdnTrainSizes {
  size_t saved, fw, bw;
};
GdnTrainSizes gdn_tc_train_sizes(const GdnProblem& p);
int gdn_tc_train_launches(const GdnProblem& p, bool backward);
cudaError_t launch_gdn_tc_fw_train(const GdnProblem& p, const GdnInputs& x, void* H, float* C_T,
                                   void* saved, void* ws, cudaStream_t st);
cudaError_t launch_gdn_tc_bw_saved(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                                   const void* saved, void* ws, cudaStream_t st);

constexpr long kGdnSms = 148;
// Items of the persistent kernels, and their blocks.
inline long gdn_items(const GdnProblem& p, const GdnTcWs& w) {
  return (long)p.BH * w.NC * ((w.nvt + 1) / 2);
}
inline unsigned gdn_blocks(const GdnProblem& p, const GdnTcWs& w) {
  const long n = gdn_items(p, w);
  return (unsigned)(n < kGdnSms ? n : kGdnSms);
}

// Tensor maps of a call's arrays, encoded once for its launches: boxes of 64
// columns and 128 rows (dq32, dk32: of 32 fp32 columns).
struct GdnMaps {
  CUtensorMap q, k, v, h, dh, dv, dq, dk;
};

// Launches a stage.  `after`: it may start while the stage before it in the
// stream still runs (programmatic launch): its prologue and its loads of the
// caller's arrays then overlap that stage's end, and gdn_wait_stage() below
// orders the rest.  Saves 2 to 3 us between two short stages.
template <class K, class... A>
cudaError_t gdn_launch(K* kern, dim3 grid, int threads, size_t smem, bool after, cudaStream_t st,
                       const A&... args) {
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The stages, one launch each.
cudaError_t launch_gdn_tc_inverse(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                                  const GdnTcWs& w, cudaStream_t st);
cudaError_t launch_gdn_tc_mn(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                             const GdnTcWs& w, cudaStream_t st);
// reverse: the gradient's recurrence, from dC_T (init) to dC0 (fin).
cudaError_t launch_gdn_tc_chain(const GdnProblem& p, bool reverse, const float* init, float* fin,
                                const GdnTcWs& w, cudaStream_t st);
// with_h: H, else y alone.
cudaError_t launch_gdn_tc_out(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                              bool with_h, const GdnTcWs& w, cudaStream_t st);
// The forward fused, behind the inverse: instead of mn, chain and out.
bool gdn_tc_fw_fused(const GdnProblem& p);
cudaError_t launch_gdn_tc_scan(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m, float* C_T,
                               const GdnTcWs& w, cudaStream_t st);
// after: behind another stage (else first in its call).
cudaError_t launch_gdn_tc_dz0(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m, bool after,
                              const GdnTcWs& w, cudaStream_t st);
cudaError_t launch_gdn_tc_dz(const GdnProblem& p, const GdnInputs& x, const GdnMaps& m,
                             const GdnTcWs& w, cudaStream_t st);
// With shared key heads a second launch adds dQ and dK over the value heads.
cudaError_t launch_gdn_tc_grads(const GdnProblem& p, const GdnInputs& x, const GdnGrads& d,
                                const GdnMaps& m, const GdnTcWs& w, cudaStream_t st);

namespace tc {

constexpr uint32_t kBlk = 16384;  // bytes of a block: 128 rows x 64 columns of one term

// Lets the next stage start its prologue; waits for the stage before (a no-op
// without one).  What that stage wrote is read, and what it reads is written,
// only behind the wait.
__device__ __forceinline__ void gdn_next_stage() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void gdn_wait_stage() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Operand descriptors: step kk of 16 along the product's inner axis.
//   kmaj: rows are the outer axis, the inner axis runs along the columns
//   mnmaj: rows are the inner axis; outer columns past 64 in the next block
__device__ __forceinline__ uint64_t kmaj(uint32_t img, int kk) {
  return sdesc_sw128(img + (kk >> 2) * kBlk + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mnmaj(uint32_t img, int kk) {
  return sdesc_sw128(img + kk * 2048, kBlk, 1024);
}

// Bulk copies of blocks of a workspace array with `per` blocks a chunk; debug builds
// check them against its extent.
__device__ __forceinline__ bool gdn_blocks_inside(const GdnProblem& p, const GdnTcWs& w, int per,
                                                  size_t block, uint32_t bytes) {
  return block * kBlk + bytes <= (size_t)p.BH * w.NC * per * kBlk;
}
__device__ __forceinline__ void gdn_load(const GdnProblem& p, const GdnTcWs& w, uint32_t dst,
                                         const uint8_t* array, int per, size_t block,
                                         uint32_t bytes, uint32_t bar) {
  const bool in = MLSTM_IN_BOUNDS(p, gdn_blocks_inside(p, w, per, block, bytes));
  bulk_load(dst, array + (in ? block * kBlk : 0), bytes, bar);
}
__device__ __forceinline__ void gdn_store(const GdnProblem& p, const GdnTcWs& w, uint8_t* array,
                                          int per, size_t block, uint32_t src, uint32_t bytes) {
  if (MLSTM_IN_BOUNDS(p, gdn_blocks_inside(p, w, per, block, bytes)))
    bulk_store(array + block * kBlk, src, bytes);
}
// 32 columns of a row into an array of N's form.
__device__ __forceinline__ void gdn_put_n(const GdnProblem& p, const GdnTcWs& w, float4* array,
                                          size_t at, const uint32_t (&v)[32]) {
  if (!MLSTM_IN_BOUNDS(p, at + 7 * 128 < (size_t)p.BH * w.NC * w.nvt * 16 * 128)) return;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    array[at + e * 128] =
        make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                    __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
}
// Debug builds: token t0, column c of head bh (of `heads`) is where a tensor store of an
// array of `cols` columns may start.
__device__ __forceinline__ bool gdn_box_inside(const GdnProblem& p, int c, int cols, int t0, int bh,
                                               int heads) {
  return c >= 0 && c < cols && t0 >= 0 && t0 < p.T && bh >= 0 && bh < heads;
}

// Two values to a bf16 pair, and what the rounding left of them.  (Conversions
// of pairs: of single values they run at a quarter of the rate, which made a pass
// that forms three terms of 128 x 128 values take 2700 cycles in place of 1400.)
__device__ __forceinline__ uint32_t take_pair(float& a, float& b) {
  const uint32_t h = pack_bf16x2(a, b);
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
  return h;
}
// The terms of N values, packed in pairs.
template <int N>
__device__ __forceinline__ void split_pack(const float* x, uint32_t (&hi)[N / 2],
                                           uint32_t (&lo)[N / 2]) {
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    float a = x[2 * e], b = x[2 * e + 1];
    hi[e] = take_pair(a, b);
    lo[e] = pack_bf16x2(a, b);
  }
}
// Eight values as 16-byte piece c of row r of a block in kTerms terms, `term`
// bytes apart, but for the third where `third` says how far it lies from the first;
// kFrom: the first term that is written.
template <int kTerms, int kFrom = 0>
__device__ __forceinline__ void put_terms(uint8_t* img, uint32_t term, int r, int c,
                                          const float* x, int third = 0) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = x[e];
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = t + 1 < kTerms ? take_pair(y[2 * e], y[2 * e + 1])
                            : pack_bf16x2(y[2 * e], y[2 * e + 1]);
    if (t >= kFrom)
      *reinterpret_cast<uint4*>(img + (t == 2 && third ? third : (int)((t - kFrom) * term)) +
                                sw128_offset(r, c)) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}
__device__ __forceinline__ void put8(uint8_t* img, uint32_t term, int r, int c, const float* x) {
  put_terms<2>(img, term, r, c, x);
}
// Eight bf16 values of a row.
__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(v[e] << 16);
    x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = (float)(1.4426950408889634 - (double)kLog2e);
// e^{a - b} of two sums of g held as (hi, lo), off by no more than ex2.approx itself
// (2^-22 of the value): what the difference and the exponent lose in fp32, which
// grows with their size, is carried along and put right to first order.  Without
// that, factors e^{-x} and e^{x} whose product is of order one left 2.4e-6 of it
// at x = 15 and 8e-6 at 56.
__device__ __forceinline__ float gdn_decay(float2 a, float2 b) {
  const float d = a.x - b.x, v = d - a.x;
  const float dl = ((a.x - (d - v)) - (b.x + v)) + (a.y - b.y);
  const float t = d * kLog2e;
  const float tl = fmaf(d, kLog2e, -t) + fmaf(d, kLog2eLo, dl * kLog2e);
  const float e = ex2_approx(t);
  return fmaf(e, tl * 0.6931471805599453f, e);
}
__device__ __forceinline__ float gdn_exp(float2 a) { return expf(a.x + a.y); }

// Whether a head's first token forgets the initial state entirely (gc: the sums of its
// first chunk).  The state is then not read: it may hold anything, and 0 times an
// infinity is a NaN.
__device__ __forceinline__ bool gdn_starts_fresh(const float2* gc) { return gdn_exp(gc[0]) == 0.f; }

// True in one lane of a converged warp.  The compiler then knows that a single
// thread is active and keeps descriptors in uniform registers: a product with A
// in tensor memory and 64 columns issues in 25 cycles and takes 35, against 44
// and 50 from a thread picked by its index (measured, one block).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Gam of a 32-column block left of the diagonal's is a product of two factors
// below one, e^{gc_r - gc_m} e^{gc_m - gc_s} with m the block's last token (or,
// transposed, e^{gc_t - gc_m} e^{gc_m - gc_r} with m its first), so that one
// exponential per row and one per column replace one per element.
// In the diagonal's block the two are above and below one: as accurate there, as
// long as the block's whole decay stays within fp32 (kGdnFlat), else one by one.
constexpr float kGdnFlat = 60.f;
// Factor of column s, by the thread of token s (a warp holds a block).
__device__ __forceinline__ float gdn_col_factor(float2 g, int m) {
  const float2 gm = make_float2(__shfl_sync(0xffffffffu, g.x, m), __shfl_sync(0xffffffffu, g.y, m));
  return m ? gdn_decay(gm, g) : gdn_decay(g, gm);
}

// Persistent kernels of 16 row warps, thread (r, h) on columns 32 h .. of row r,
// and a control warp, which issues the products and moves the tiles: done by a
// row warp those cost its rows 1500 cycles a round.
constexpr int kGdnRows = 512;
constexpr int kGdnThreads = kGdnRows + 32;

struct GdnRounds {
  uint32_t bar, phase;
  bool ok;
  Problem wt;
};

// One round of the block: everything written so far (shared memory, tensor
// memory) is visible to the products that `issue` starts.  Meanwhile the row
// warps run `rows`, and lane 0 of the control warp `moves`; everyone waits for
// the products, then lane 0 runs `after` (loads into what they have read).
template <class F, class R, class M, class A>
__device__ __forceinline__ void gdn_round(GdnRounds& s, uint32_t site, F&& issue, R&& rows,
                                          M&& moves, A&& after) {
  fence_proxy_async_smem();
  tmem_wait_st();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x >= kGdnRows) {
    if (elect_one()) {
      tc_fence_after();
      if (s.ok) issue();
      mma_commit(s.bar);
    }
    __syncwarp();
    if (threadIdx.x == kGdnRows) {
      moves();
      if (s.ok) s.ok = mbar_wait(s.bar, s.phase, s.wt, site);
      if (s.ok) after();
    }
    __syncwarp();
  } else {
    rows();
    if (s.ok) s.ok = mbar_wait(s.bar, s.phase, s.wt, site);
    tc_fence_after();
  }
  s.phase ^= 1;
}
__device__ __forceinline__ void gdn_nothing() {}

// Item i of a persistent kernel: (bh, chunk, pair of value tiles).
struct GdnItem {
  size_t cb;
  int bh, t0, n, vt, tiles;
  __device__ GdnItem(long i, const GdnProblem& p, const GdnTcWs& w) {
    // an int holds the items: up to 65535 heads and 2^15 chunks do in any case, and
    // with pairs of value tiles each item has 136 KB of workspace or more
    const int pairs = (w.nvt + 1) / 2;
    const int k = (int)i, c = k / pairs;
    cb = (size_t)c;
    vt = (k - c * pairs) * 2;
    tiles = min(2, w.nvt - vt);
    bh = c / w.NC;
    t0 = (c - bh * w.NC) * kGdnL;
    n = min(kGdnL, p.T - t0);
  }
};

// The block as one, without a control warp: thread 0's warp issues.
template <class F>
__device__ __forceinline__ void run_mma(uint32_t bar, uint32_t& phase, bool& ok,
                                        const Problem& wt, uint32_t site, F&& issue) {
  fence_proxy_async_smem();
  tmem_wait_st();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32 && elect_one()) {
    tc_fence_after();
    if (ok) issue();
    mma_commit(bar);
  }
  __syncwarp();
  if (ok) ok = mbar_wait(bar, phase, wt, site);
  phase ^= 1;
  tc_fence_after();
}

// D (+)= A B over an inner axis of 64 * slabs, both operands in shared memory.
// AT / BT: the operand's rows are the inner axis.
template <bool AT, bool BT>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int slabs,
                                       bool fresh) {
  for (int s = 0; s < slabs; ++s) {
    const uint32_t as = a + s * (AT ? 8192 : kBlk), bs = b + s * (BT ? 8192 : kBlk);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      mma_bf16_ss(d, AT ? mnmaj(as, kk) : kmaj(as, kk), BT ? mnmaj(bs, kk) : kmaj(bs, kk), id,
                  !fresh || s > 0 || kk > 0);
  }
}

// Tinv (or Tinv^T) of row r into tensor memory as the A operand: hi in columns
// [0, 64), lo in [64, 128).  512 threads: thread h of the row takes both terms of
// columns 32 h ..: pieces 4 h .. 4 h + 3, t[0..3] hi and t[4..7] lo.  `have`: the
// row has them (else zero).  The identity is added on the way into tensor memory,
// not to the loads, which would wait for them.
__device__ __forceinline__ void load_tinv(const uint4* src, int r, int h, bool have,
                                          uint4 (&t)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    t[k] = have ? src[((k >> 2) * 16 + h * 4 + (k & 3)) * 128 + r] : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void add_identity(int r, int h, uint4 (&t)[8]) {
  const uint32_t one = 0x3f80u << (16 * (r & 1));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (h * 4 + k == r >> 3) {
      const int e = (r >> 1) & 3;
      t[k].x |= e == 0 ? one : 0u;
      t[k].y |= e == 1 ? one : 0u;
      t[k].z |= e == 2 ? one : 0u;
      t[k].w |= e == 3 ? one : 0u;
    }
}
// tlane: the thread's lane, first column of the operand.
__device__ __forceinline__ void put_tinv(uint32_t tlane, int h, const uint4 (&t)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v[16] = {t[4 * i].x,     t[4 * i].y,     t[4 * i].z,     t[4 * i].w,
                            t[4 * i + 1].x, t[4 * i + 1].y, t[4 * i + 1].z, t[4 * i + 1].w,
                            t[4 * i + 2].x, t[4 * i + 2].y, t[4 * i + 2].z, t[4 * i + 2].w,
                            t[4 * i + 3].x, t[4 * i + 3].y, t[4 * i + 3].z, t[4 * i + 3].w};
    tmem_st16(tlane + i * 64 + h * 16, v);
  }
}
// D = A B: A in tensor memory at `a` (hi, lo 64 columns behind), 128 inner
// indexes; B an image of two terms (`term` bytes apart) with inner rows.
__device__ __forceinline__ void mma_terms3(uint32_t d, uint32_t a, uint32_t b, uint32_t term,
                                           uint32_t id) {
#pragma unroll
  for (int t = 0; t < 3; ++t)
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16_ts(d, a + (t == 1 ? 64 : 0) + kk * 8, mnmaj(b + (t == 2 ? term : 0u), kk), id,
                  (t | kk) != 0);
}
__device__ __forceinline__ void mma_terms2(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16_ts(d, a + t * 64 + kk * 8, mnmaj(b, kk), id, (t | kk) != 0);
}

// 16 / 8 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// Four 8 x 8 blocks of 16-bit values, transposed: lane i supplies the address of
// row i % 8 of block i / 8 and gets, of each block, rows 2 (i % 4) and + 1 of
// column i / 4.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Sums of g inside the chunk by one warp, in 64 bits, four tokens per lane.
__device__ __forceinline__ void gdn_chunk_sums(const float* g, int n, int lane, float2* gc,
                                               float2* out) {
  double x[4], s = 0.;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = 4 * lane + e;
    s += t < n ? (double)gdn_log_decay(g[t]) : 0.;
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
    gc[4 * lane + e] = out[4 * lane + e] = make_float2(hi, (float)(v - hi));
  }
}

}  // namespace tc
}  // namespace mlstm
