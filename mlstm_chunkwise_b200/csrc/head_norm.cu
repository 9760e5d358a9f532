// Layer norm of the cell output: X [B, NH, T, D] is normalised over D for every
// (token, head), scaled and shifted per (head, column), and written token-major
// as Y [B, T, NH * D], the layout the block's output projection reads.
//   mean, var over D (var from the differences),  xh = (x - mean) rstd
//   y  = xh w + b
//   a  = dy w,  dx = rstd (a - mean(a) - xh mean(a xh))
//   dw = sum over (b, t) dy xh,  db = sum dy
//
// Bound by HBM: the forward moves x and y once, the backward x, dy and dx.  A
// row sits in registers between the statistics and the output (16-byte
// vectors where D allows): a warp per row up to 512 columns, else one block
// per row.  The backward's lanes own the same columns
// for every row they visit, so the weight gradient accumulates in registers
// over a block's rows of one head; blocks write partial sums and a second
// kernel adds them in a fixed order (no atomics: the result does not change
// from call to call).
#include <type_traits>

#include "device_address.h"
#include "head_norm.h"

namespace mlstm {
namespace {

template <typename T, int kVec>
struct Vec;
template <> struct Vec<float, 4> {
  __device__ static void load(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  __device__ static void store(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <> struct Vec<__nv_bfloat16, 8> {
  __device__ static void load(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(h[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};
template <typename T> struct Vec<T, 1> {
  __device__ static void load(const T* p, float (&x)[1]) { x[0] = to_float(*p); }
  __device__ static void store(T* p, const float (&x)[1]) { *p = from_float<T>(x[0]); }
};
template <int kVec>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[kVec]) {
  if constexpr (kVec >= 4) {
#pragma unroll
    for (int e = 0; e < kVec; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + e);
      x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
    }
  } else {
    x[0] = *p;
  }
}

// Sum over the threads of a row: a warp, or the whole block through `red`.
template <bool kBlockRow>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (kBlockRow) {
    const int warps = blockDim.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; ++i) v += red[i];
  }
  return v;
}

// Rows on their way: every thread copies its own vectors of the next kStages - 1
// rows into its own slots of shared memory (cp.async) and reads them back itself,
// so no barrier is needed and registers hold one row only.  Rows of single
// elements (D no whole number of 16-byte vectors) are loaded where they are used.
constexpr int kStages = 4;
template <int kNV>
constexpr int kBwStages = kNV < 4 ? 4 : 3;  // 512 threads of 128 bytes a stage must fit

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void copy_wait() {  // for the oldest of kN - 1 rows on their way
  asm volatile("cp.async.wait_group %0;" ::"n"(kN - 2) : "memory");
}

// A row of a head, (b, t), and the row `step` rows on, without a division per row
// (a 64-bit one costs as much as the row's arithmetic).
struct RowAt {
  int b, t;
  // no rows: past the last batch at once
  __device__ RowAt(long row, int T, int B)
      : b(T > 0 ? (int)(row / T) : B), t(T > 0 ? (int)(row % T) : 0) {}
  __device__ void advance(int step_b, int step_t, int T) {
    b += step_b;
    t += step_t;
    if (t >= T) {
      t -= T;
      ++b;
    }
  }
};

// Both kernels: grid (blocks, NH); block x handles rows x, x + gridDim.x, ...
// (warps interleaved) of head y's B * T rows, so that weight and bias stay in
// registers (loaded per row they were four times the row's own bytes, and the
// 7B-shaped forward took 244 us).
template <typename T, int kVec, int kNV, bool kBlockRow>
__global__ void __launch_bounds__(kBlockRow ? 512 : 256)
head_norm_fw_kernel(HeadNormProblem p, const T* __restrict__ X,
                    const float* __restrict__ weight,
                    const float* __restrict__ bias, T* __restrict__ Y,
                    float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[32];
  const int tpr = kBlockRow ? blockDim.x : 32;  // threads per row
  const int lane = threadIdx.x % tpr;
  const int h = blockIdx.y;
  const long per = kBlockRow ? 1 : blockDim.x / 32, step = gridDim.x * per;
  const float inv = 1.f / (float)p.D;
  const float *wp = weight + (long)h * p.D, *bp = bias + (long)h * p.D;
  float w[kNV][kVec], b[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * tpr + lane) * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) b[i][e] = 0.f;
    if (c < p.D) {
      load_f32<kVec>(wp + c, w[i]);
      if (bias) load_f32<kVec>(bp + c, b[i]);
    }
  }
  extern __shared__ uint4 ring[];  // [kStages][kNV][threads]
  const long row = blockIdx.x * per + threadIdx.x / tpr;
  const int step_b = (int)(step / max(p.T, 1)), step_t = (int)(step % max(p.T, 1));
  RowAt at(row, p.T, p.B), ahead = at;
  auto x_of = [&](const RowAt& a) { return ((long)a.b * p.NH + h) * p.T + a.t; };
  const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
  auto fetch = [&](int stage) {
    if (kVec > 1 && ahead.b < p.B) {
      const T* x = X + x_of(ahead) * p.D;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * tpr + lane) * kVec;
        if (c < p.D) copy16(slot + (stage * kNV + i) * blockDim.x * 16, x + c);
      }
    }
    copy_commit();
    ahead.advance(step_b, step_t, p.T);
  };
  for (int st = 0; st < kStages - 1; ++st) fetch(st);
  for (int st = 0; at.b < p.B; at.advance(step_b, step_t, p.T), st = (st + 1) % kStages) {
    float v[kNV][kVec];
    float s = 0.f;
    copy_wait<kStages>();
    const long xr = x_of(at);
    const T* x = X + xr * p.D;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        Vec<T, kVec>::load(kVec > 1 ? reinterpret_cast<const T*>(
                                          ring + (st * kNV + i) * blockDim.x + threadIdx.x)
                                    : x + c,
                           v[i]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s += v[i][e];
      }
    }
    fetch((st + kStages - 1) % kStages);
    const float mu = row_sum<kBlockRow>(s, red) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          v[i][e] -= mu;
          s = fmaf(v[i][e], v[i][e], s);
        }
      }
    }
    const float r = rsqrtf(row_sum<kBlockRow>(s, red) * inv + p.eps);
    T* y = Y + (((long)at.b * p.T + at.t) * p.NH + h) * p.D;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[i][e] = fmaf(v[i][e] * r, w[i][e], b[i][e]);
        if (MLSTM_IN_BOUNDS(p, at.b < p.B && at.t < p.T && c + kVec <= p.D))
          Vec<T, kVec>::store(y + c, v[i]);
      }
    }
    if (lane == 0 && MLSTM_IN_BOUNDS(p, xr < (long)p.B * p.NH * p.T)) {
      if (mean) mean[xr] = mu;
      if (rstd) rstd[xr] = r;
    }
  }
}

template <typename T, int kVec, int kNV, bool kBlockRow>
__global__ void __launch_bounds__(kBlockRow ? 512 : 256, kBlockRow ? 1 : 2)
head_norm_bw_kernel(HeadNormProblem p, const T* __restrict__ X,
                    const T* __restrict__ dY, const float* __restrict__ weight,
                    const float* __restrict__ mean,
                    const float* __restrict__ rstd, T* __restrict__ dX,
                    float* __restrict__ part, int has_db) {
  __shared__ float red[32];
  const int tpr = kBlockRow ? blockDim.x : 32;
  const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const int per = kBlockRow ? 1 : blockDim.x / 32;
  const int h = blockIdx.y;
  const long step = (long)gridDim.x * per;
  const float inv = 1.f / (float)p.D;
  const float* wp = weight + (long)h * p.D;
  float dw[kNV][kVec], db[kNV][kVec], w[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) dw[i][e] = db[i][e] = 0.f;
    const int c = (i * tpr + lane) * kVec;
    if (c < p.D) load_f32<kVec>(wp + c, w[i]);
  }
  // [kBwStages<kNV>][2 kNV][threads]
  extern __shared__ uint4 ring[];
  const long row = (long)blockIdx.x * per + sub;
  const int step_b = (int)(step / max(p.T, 1)), step_t = (int)(step % max(p.T, 1));
  RowAt at(row, p.T, p.B), ahead = at;
  auto x_of = [&](const RowAt& a) { return ((long)a.b * p.NH + h) * p.T + a.t; };
  auto y_of = [&](const RowAt& a) { return ((long)a.b * p.T + a.t) * p.NH + h; };
  const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
  auto fetch = [&](int stage) {
    if (kVec > 1 && ahead.b < p.B) {
      const long xr = x_of(ahead);
      const T *x = X + xr * p.D, *dy = dY + y_of(ahead) * p.D;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * tpr + lane) * kVec;
        if (c < p.D) {
          copy16(slot + (stage * 2 * kNV + 2 * i) * blockDim.x * 16, x + c);
          copy16(slot + (stage * 2 * kNV + 2 * i + 1) * blockDim.x * 16, dy + c);
        }
      }
    }
    copy_commit();
    ahead.advance(step_b, step_t, p.T);
  };
  for (int st = 0; st < kBwStages<kNV> - 1; ++st) fetch(st);
  float next_mu = 0.f, next_r = 0.f;
  auto load_stats = [&](const RowAt& a) {
    if (a.b >= p.B) return;
    next_mu = mean[x_of(a)];
    next_r = rstd[x_of(a)];
  };
  load_stats(at);
  for (int st = 0; at.b < p.B; at.advance(step_b, step_t, p.T), st = (st + 1) % kBwStages<kNV>) {
    copy_wait<kBwStages<kNV>>();
    const long xr = x_of(at);
    const float mu = next_mu, r = next_r;
    RowAt then = at;
    then.advance(step_b, step_t, p.T);
    load_stats(then);
    float xv[kNV][kVec], av[kNV][kVec];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        const uint4* in = ring + (st * 2 * kNV + 2 * i) * blockDim.x + threadIdx.x;
        Vec<T, kVec>::load(kVec > 1 ? reinterpret_cast<const T*>(in) : X + xr * p.D + c, xv[i]);
        Vec<T, kVec>::load(kVec > 1 ? reinterpret_cast<const T*>(in + blockDim.x)
                                    : dY + y_of(at) * p.D + c,
                           av[i]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float xh = (xv[i][e] - mu) * r, g = av[i][e];
          dw[i][e] = fmaf(g, xh, dw[i][e]);
          db[i][e] += g;
          xv[i][e] = xh;
          av[i][e] = g * w[i][e];
          s0 += av[i][e];
          s1 = fmaf(av[i][e], xh, s1);
        }
      }
    }
    fetch((st + kBwStages<kNV> - 1) % kBwStages<kNV>);
    if constexpr (kBlockRow) {
      s0 = row_sum<true>(s0, red) * inv;
      s1 = row_sum<true>(s1, red) * inv;
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      }
      s0 *= inv;
      s1 *= inv;
    }
    T* dx = dX + xr * p.D;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) av[i][e] = r * (av[i][e] - s0 - xv[i][e] * s1);
        if (MLSTM_IN_BOUNDS(p, xr < (long)p.B * p.NH * p.T && c + kVec <= p.D))
          Vec<T, kVec>::store(dx + c, av[i]);
      }
    }
  }
  // partial sums of this block: [block][2][NH][D]
  float* pw = part + ((size_t)blockIdx.x * 2 * p.NH + h) * p.D;
  float* pb = pw + (size_t)p.NH * p.D;
  if (kBlockRow) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          pw[c + e] = dw[i][e];
          if (has_db) pb[c + e] = db[i][e];
        }
      }
    }
    return;
  }
  __syncthreads();  // every row has left the ring
  float *sw = reinterpret_cast<float*>(ring), *sb = sw + p.D;
  for (int k = 0; k < per; ++k) {  // the warps in turn: a fixed order
    if (sub == k) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * 32 + lane) * kVec;
        if (c < p.D) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            sw[c + e] = k ? sw[c + e] + dw[i][e] : dw[i][e];
            sb[c + e] = k ? sb[c + e] + db[i][e] : db[i][e];
          }
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
    pw[c] = sw[c];
    if (has_db) pb[c] = sb[c];
  }
}

// Sum of the blocks' partial sums, 32 columns per block of 32 x 32 threads:
// thread row y adds every 32nd block, then the 32 in order (a fixed order).
__global__ void __launch_bounds__(1024)
head_norm_sum_kernel(const float* __restrict__ part, int blocks, size_t n, float* __restrict__ dw,
                     float* __restrict__ db) {
  __shared__ float s[32][33];
  const size_t c = (size_t)blockIdx.x * 32 + threadIdx.x;  // column over (NH, D)
  const int which = blockIdx.y;
  float a = 0.f;
  if (c < n)
    for (int b = threadIdx.y; b < blocks; b += 32) a += part[((size_t)b * 2 + which) * n + c];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += s[i][threadIdx.x];
    (which ? db : dw)[c] = a;
  }
}

struct Shape {
  bool block_row;
  int threads, nv, vec;
};
// Vectors of 16 bytes where a row is a whole number of them, else single
// elements; a warp per row while it holds at most 16 elements per lane (more
// and the backward's sums spill), else a block of 64 to 512 threads per row.
Shape shape_for(int D, int esz) {
  Shape s{};
  s.vec = D * esz % 16 == 0 ? 16 / esz : 1;
  const int most = 16 / s.vec;
  const int vecs = (D + s.vec - 1) / s.vec;
  s.block_row = vecs > 32 * most;
  s.threads = s.block_row ? 64 : 256;
  if (s.block_row)
    while (s.threads * most < vecs) s.threads *= 2;
  const int tpr = s.block_row ? s.threads : 32;
  const int need = (vecs + tpr - 1) / tpr;
  s.nv = 1;
  while (s.nv < need) s.nv *= 2;
  return s;
}

// Blocks per head: `per_sm` times 256 threads to an SM over all heads, each with
// at least `least` rows (or passes of one row per warp).
int blocks_per_head(const HeadNormProblem& p, const Shape& s, int per_sm, int least) {
  const long rows = (long)p.B * p.T, per = (s.block_row ? 1 : s.threads / 32) * least;
  const long n = 148l * per_sm * 256 / s.threads / p.NH, most = (rows + per - 1) / per;
  const long k = n < most ? n : most;
  return k > 1 ? (int)k : 1;
}
// Backward: 512 threads to an SM (their registers); every block leaves a row of
// partial sums, hence four rows each at least.
int bw_blocks(const HeadNormProblem& p, const Shape& s) { return blocks_per_head(p, s, 2, 4); }

// The largest ring of `slots` 16-byte vectors a thread, whatever this launch's is: 512
// threads where a block takes a row, 256 where a warp does.
template <class K>
cudaError_t allow_ring(K* kern, int slots, bool block_row) {
  const size_t most = (size_t)slots * 16 * (block_row ? 512 : 256);
  return most > 47 * 1024 ? allow_smem(kern, most) : cudaSuccess;  // 1 KB is static
}

template <typename T, int kVec, int kNV>
cudaError_t fw(const HeadNormProblem& p, const Shape& s, const void* X, const float* weight,
               const float* bias, void* Y, float* mean, float* rstd, cudaStream_t st) {
  const dim3 grid(blocks_per_head(p, s, 16, 1), p.NH);
  const size_t smem = kVec > 1 ? (size_t)kStages * kNV * 16 * s.threads : 0;
  auto kern = s.block_row ? head_norm_fw_kernel<T, kVec, kNV, true>
                          : head_norm_fw_kernel<T, kVec, kNV, false>;
  const cudaError_t e = allow_ring(kern, kVec > 1 ? kStages * kNV : 0, s.block_row);
  if (e != cudaSuccess) return e;
  kern<<<grid, s.threads, smem, st>>>(p, (const T*)X, weight, bias, (T*)Y, mean, rstd);
  return cudaGetLastError();
}

template <typename T, int kVec, int kNV>
cudaError_t bw(const HeadNormProblem& p, const Shape& s, const void* X, const void* dY,
               const float* weight, const float* mean, const float* rstd, void* dX,
               float* dweight, float* dbias, float* part, cudaStream_t st) {
  const int blocks = bw_blocks(p, s);
  const dim3 grid(blocks, p.NH);
  const size_t ring = kVec > 1 ? (size_t)kBwStages<kNV> * kNV * 32 * s.threads : 0;
  const size_t sums = s.block_row ? 0 : 8 * (size_t)p.D;  // reuses the ring
  const size_t smem = sums > ring ? sums : ring;
  auto kern = s.block_row ? head_norm_bw_kernel<T, kVec, kNV, true>
                          : head_norm_bw_kernel<T, kVec, kNV, false>;
  cudaError_t e = allow_ring(kern, kVec > 1 ? 2 * kBwStages<kNV> * kNV : 0, s.block_row);
  if (e != cudaSuccess) return e;
  kern<<<grid, s.threads, smem, st>>>(p, (const T*)X, (const T*)dY, weight, mean, rstd, (T*)dX,
                                      part, dbias != nullptr);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)p.NH * p.D;
  head_norm_sum_kernel<<<dim3((unsigned)((n + 31) / 32), dbias ? 2 : 1), dim3(32, 32), 0, st>>>(
      part, blocks, n, dweight, dbias);
  return cudaGetLastError();
}

// Calls f with the (T, vec, nv) of the shape as template arguments.
template <typename T, class F>
cudaError_t dispatch(const Shape& s, F&& f) {
  constexpr int kV = 16 / sizeof(T);
  if (s.vec > 1) {
    if (s.nv == 1) return f(std::integral_constant<int, kV>{}, std::integral_constant<int, 1>{});
    if (kV == 8 || s.nv == 2)
      return f(std::integral_constant<int, kV>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, kV>{}, std::integral_constant<int, kV == 8 ? 2 : 4>{});
  }
  if (s.nv <= 4) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
}

}  // namespace

cudaError_t launch_head_norm_fw(const HeadNormProblem& p, mlstm_dtype dt, const void* X,
                                const float* weight, const float* bias, void* Y, float* mean,
                                float* rstd, cudaStream_t st) {
  const Shape s = shape_for(p.D, dt == MLSTM_DT_BF16 ? 2 : 4);
  if (dt == MLSTM_DT_BF16)
    return dispatch<__nv_bfloat16>(s, [&](auto v, auto n) {
      return fw<__nv_bfloat16, v.value, n.value>(p, s, X, weight, bias, Y, mean, rstd, st);
    });
  return dispatch<float>(s, [&](auto v, auto n) {
    return fw<float, v.value, n.value>(p, s, X, weight, bias, Y, mean, rstd, st);
  });
}

size_t head_norm_bw_workspace(const HeadNormProblem& p, mlstm_dtype dt) {
  const Shape s = shape_for(p.D, dt == MLSTM_DT_BF16 ? 2 : 4);
  return (size_t)bw_blocks(p, s) * 2 * p.NH * p.D * sizeof(float);
}

cudaError_t launch_head_norm_bw(const HeadNormProblem& p, mlstm_dtype dt, const void* X,
                                const void* dY, const float* weight, const float* mean,
                                const float* rstd, void* dX, float* dweight, float* dbias,
                                void* ws, cudaStream_t st) {
  const Shape s = shape_for(p.D, dt == MLSTM_DT_BF16 ? 2 : 4);
  float* part = static_cast<float*>(ws);
  if (dt == MLSTM_DT_BF16)
    return dispatch<__nv_bfloat16>(s, [&](auto v, auto n) {
      return bw<__nv_bfloat16, v.value, n.value>(p, s, X, dY, weight, mean, rstd, dX, dweight,
                                                 dbias, part, st);
    });
  return dispatch<float>(s, [&](auto v, auto n) {
    return bw<float, v.value, n.value>(p, s, X, dY, weight, mean, rstd, dX, dweight, dbias, part,
                                       st);
  });
}

}  // namespace mlstm
