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
// vectors where D allows): a warp per row up to 1024 columns at 16 bits (512
// at 32), else one block per row.  The backward's lanes own the same columns
// for every row they visit, so the weight gradient accumulates in registers
// over a block's rows of one head; blocks write partial sums and a second
// kernel adds them in a fixed order (no atomics: the result does not change
// from call to call).
#include <type_traits>

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

// Row index (over B, NH, T) -> element offset of its Y row.
__device__ __forceinline__ size_t y_row(const HeadNormProblem& p, long bh, int t) {
  return (((size_t)(bh / p.NH) * p.T + t) * p.NH + bh % p.NH) * p.D;
}

template <typename T, int kVec, int kNV, bool kBlockRow>
__global__ void __launch_bounds__(kBlockRow ? 512 : 256)
head_norm_fw_kernel(HeadNormProblem p, const T* __restrict__ X,
                    const float* __restrict__ weight,
                    const float* __restrict__ bias, T* __restrict__ Y,
                    float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[32];
  const int tpr = kBlockRow ? blockDim.x : 32;  // threads per row
  const int lane = threadIdx.x % tpr;
  const long rows = (long)p.B * p.NH * p.T;
  const long per = kBlockRow ? 1 : blockDim.x / 32;
  const float inv = 1.f / (float)p.D;
  for (long row = blockIdx.x * per + threadIdx.x / tpr; row < rows; row += gridDim.x * per) {
    const T* x = X + row * p.D;
    float v[kNV][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        Vec<T, kVec>::load(x + c, v[i]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s += v[i][e];
      }
    }
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
    const long bh = row / p.T;
    const int h = (int)(bh % p.NH);
    T* y = Y + y_row(p, bh, (int)(row % p.T));
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        float w[kVec], b[kVec];
        load_f32<kVec>(weight + (long)h * p.D + c, w);
        if (bias) load_f32<kVec>(bias + (long)h * p.D + c, b);
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[i][e] = fmaf(v[i][e] * r, w[e], bias ? b[e] : 0.f);
        Vec<T, kVec>::store(y + c, v[i]);
      }
    }
    if (lane == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = r;
    }
  }
}

// Grid (blocks, NH): block x handles rows x, x + gridDim.x, ... (warps
// interleaved) of head y's B * T rows.
template <typename T, int kVec, int kNV, bool kBlockRow>
__global__ void __launch_bounds__(kBlockRow ? 512 : 256)
head_norm_bw_kernel(HeadNormProblem p, const T* __restrict__ X,
                    const T* __restrict__ dY, const float* __restrict__ weight,
                    const float* __restrict__ mean,
                    const float* __restrict__ rstd, T* __restrict__ dX,
                    float* __restrict__ part, int has_db) {
  extern __shared__ float sh[];  // red[32], then (warp rows) [2][D]
  float* red = sh;
  const int tpr = kBlockRow ? blockDim.x : 32;
  const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const int per = kBlockRow ? 1 : blockDim.x / 32;
  const int h = blockIdx.y;
  const long rows = (long)p.B * p.T;
  const float inv = 1.f / (float)p.D;
  float dw[kNV][kVec], db[kNV][kVec];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < kVec; ++e) dw[i][e] = db[i][e] = 0.f;
  for (long row = (long)blockIdx.x * per + sub; row < rows; row += (long)gridDim.x * per) {
    const long b = row / p.T, t = row % p.T;
    const size_t xr = ((size_t)(b * p.NH + h) * p.T + t);
    const T* x = X + xr * p.D;
    const T* dy = dY + y_row(p, b * p.NH + h, (int)t);
    const float mu = mean[xr], r = rstd[xr];
    float xv[kNV][kVec], av[kNV][kVec];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        Vec<T, kVec>::load(x + c, xv[i]);
        Vec<T, kVec>::load(dy + c, av[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
        float w[kVec];
        load_f32<kVec>(weight + (long)h * p.D + c, w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float xh = (xv[i][e] - mu) * r, g = av[i][e];
          dw[i][e] = fmaf(g, xh, dw[i][e]);
          db[i][e] += g;
          xv[i][e] = xh;
          av[i][e] = g * w[e];
          s0 += av[i][e];
          s1 = fmaf(av[i][e], xh, s1);
        }
      }
    }
    s0 = row_sum<kBlockRow>(s0, red) * inv;
    s1 = row_sum<kBlockRow>(s1, red) * inv;
    T* dx = dX + xr * p.D;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * tpr + lane) * kVec;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) av[i][e] = r * (av[i][e] - s0 - xv[i][e] * s1);
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
  float *sw = sh + 32, *sb = sw + p.D;
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

// Sum of the blocks' partial sums, 32 columns per block of 32 x 8 threads:
// thread row y adds every eighth block, then the eight in order.
__global__ void __launch_bounds__(256)
head_norm_sum_kernel(const float* __restrict__ part, int blocks, size_t n, float* __restrict__ dw,
                     float* __restrict__ db) {
  __shared__ float s[8][33];
  const size_t c = (size_t)blockIdx.x * 32 + threadIdx.x;  // column over (NH, D)
  const int which = blockIdx.y;
  float a = 0.f;
  if (c < n)
    for (int b = threadIdx.y; b < blocks; b += 8) a += part[((size_t)b * 2 + which) * n + c];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += s[i][threadIdx.x];
    (which ? db : dw)[c] = a;
  }
}

struct Shape {
  bool block_row;
  int threads, nv, vec;
};
// Vectors of 16 bytes where a row is a whole number of them, else single
// elements; a warp per row while it holds at most four vectors (sixteen
// elements) per lane, else a block of up to 512 threads per row.
Shape shape_for(int D, int esz) {
  Shape s{};
  s.vec = D * esz % 16 == 0 ? 16 / esz : 1;
  const int most = s.vec > 1 ? 4 : 16;
  const int vecs = (D + s.vec - 1) / s.vec;
  s.block_row = vecs > 32 * most;
  s.threads = 256;
  if (s.block_row)
    while (s.threads * most < vecs) s.threads *= 2;
  const int tpr = s.block_row ? s.threads : 32;
  const int need = (vecs + tpr - 1) / tpr;
  s.nv = 1;
  while (s.nv < need) s.nv *= 2;
  return s;
}

// Blocks per head of the backward: about two waves over all heads, fewer when
// there are few rows.
int bw_blocks(const HeadNormProblem& p, const Shape& s) {
  const long rows = (long)p.B * p.T, per = s.block_row ? 1 : s.threads / 32;
  long n = 148 * 4 / p.NH;
  if (n < 1) n = 1;
  const long most = (rows + per - 1) / per;
  return (int)(n < most ? n : (most > 0 ? most : 1));
}

template <typename T, int kVec, int kNV>
cudaError_t fw(const HeadNormProblem& p, const Shape& s, const void* X, const float* weight,
               const float* bias, void* Y, float* mean, float* rstd, cudaStream_t st) {
  const long rows = (long)p.B * p.NH * p.T, per = s.block_row ? 1 : s.threads / 32;
  const long need = (rows + per - 1) / per;
  const int grid = (int)(need < 148 * 32 ? need : 148 * 32);
  if (s.block_row)
    head_norm_fw_kernel<T, kVec, kNV, true><<<grid, s.threads, 0, st>>>(
        p, (const T*)X, weight, bias, (T*)Y, mean, rstd);
  else
    head_norm_fw_kernel<T, kVec, kNV, false><<<grid, s.threads, 0, st>>>(
        p, (const T*)X, weight, bias, (T*)Y, mean, rstd);
  return cudaGetLastError();
}

template <typename T, int kVec, int kNV>
cudaError_t bw(const HeadNormProblem& p, const Shape& s, const void* X, const void* dY,
               const float* weight, const float* mean, const float* rstd, void* dX,
               float* dweight, float* dbias, float* part, cudaStream_t st) {
  const int blocks = bw_blocks(p, s);
  const dim3 grid(blocks, p.NH);
  const size_t smem = (32 + (s.block_row ? 0 : 2 * (size_t)p.D)) * 4;
  if (s.block_row)
    head_norm_bw_kernel<T, kVec, kNV, true><<<grid, s.threads, smem, st>>>(
        p, (const T*)X, (const T*)dY, weight, mean, rstd, (T*)dX, part, dbias != nullptr);
  else
    head_norm_bw_kernel<T, kVec, kNV, false><<<grid, s.threads, smem, st>>>(
        p, (const T*)X, (const T*)dY, weight, mean, rstd, (T*)dX, part, dbias != nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)p.NH * p.D;
  head_norm_sum_kernel<<<dim3((unsigned)((n + 31) / 32), dbias ? 2 : 1), dim3(32, 8), 0, st>>>(
      part, blocks, n, dweight, dbias);
  return cudaGetLastError();
}

// Calls f with the (T, vec, nv) of the shape as template arguments.
template <typename T, class F>
cudaError_t dispatch(const Shape& s, F&& f) {
  constexpr int kV = 16 / sizeof(T);
  if (s.vec > 1) {
    if (s.nv == 1) return f(std::integral_constant<int, kV>{}, std::integral_constant<int, 1>{});
    if (s.nv == 2) return f(std::integral_constant<int, kV>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, kV>{}, std::integral_constant<int, 4>{});
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
