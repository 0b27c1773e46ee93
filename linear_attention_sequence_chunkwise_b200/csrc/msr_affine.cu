// msr_affine.cu -- the MSR epilogue ("阅读笔记：RetNet" §三.2) with a learnable affine, and its gradient:
//   x^ = (y - m) / sd over a (token, head) row,  n = w x^ + b,  out = swish(g) n,  swish(g) = g s(g);
//   db = sum_t swish(g) dout,  dw = sum_t swish(g) dout x^,  dg = dout n s(g) (1 + g (1 - s(g))),
//   with e = w swish(g) dout:  dy = (e - mean(e) - x^ mean(e x^)) / sd.
//
// Bound by HBM: y, g (and dout) are read once, out (dy, dg) written once.  A warp holds a row in
// registers, so the mean, the centred variance and the two means of the gradient are shuffles over
// registers; the statistics are recomputed by the gradient, which reads y anyway, instead of being
// kept.  dw and db are sums over all tokens of a head: a CTA stays on one head and strides over its
// tokens with the sums in registers, adds its warps' up in shared memory and writes one partial row;
// a second kernel adds the partial rows in order (no atomics: the same sums every time).
#include "launch.h"

namespace retnet {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

// Elements of a lane: 8 consecutive ones of each of MG groups (VEC), or every 32nd (odd widths and
// addresses).
template <bool VEC>
__device__ __forceinline__ int column(int lane, int m, int e) {
  return VEC ? (lane + 32 * m) * 8 + e : lane + 32 * (m * 8 + e);
}
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int lane, int m, int d_v, float (&x)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(lane, m, e);
      x[e] = c < d_v ? load_f(p, c) : 0.f;
    }
  } else {
    const int c = (lane + 32 * m) * 8;
    if (c >= d_v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p + c), b = *reinterpret_cast<const float4*>(p + c + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int lane, int m, int d_v, const float (&x)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(lane, m, e);
      if (c < d_v) store_f(p, c, x[e]);
    }
  } else {
    const int c = (lane + 32 * m) * 8;
    if (c >= d_v) return;
    if constexpr (sizeof(T) == 2) {
      uint4 u;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      *reinterpret_cast<uint4*>(p + c) = u;
    } else {
      *reinterpret_cast<float4*>(p + c) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(p + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// Mean and 1/sd of the row in x (elements past d_v are zero and stay out of the variance).
template <int MG, bool VEC>
__device__ __forceinline__ void row_stats(const float (&x)[MG][8], int lane, int d_v, float eps, float& mean, float& inv) {
  float s = 0.f;
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[m][e];
  mean = warp_sum(s) / static_cast<float>(d_v);
  float sq = 0.f;
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = column<VEC>(lane, m, e) < d_v ? x[m][e] - mean : 0.f;
      sq = fmaf(c, c, sq);
    }
  inv = rsqrtf(warp_sum(sq) / static_cast<float>(d_v) + eps);
}

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + expf(-g)); }

template <typename T, int MG, bool VEC>
__global__ void __launch_bounds__(kThreads) msr_affine_kernel(const T* y, const T* g,
                                                              const float* __restrict__ weight,
                                                              const float* __restrict__ bias, T* out,
                                                              int64_t tokens, int heads, int d_v, float eps) {
  const int lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= tokens * heads) return;
  const int h = static_cast<int>(row % heads);
  float x[MG][8], gv[MG][8];
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    load8<T, VEC>(y + row * d_v, lane, m, d_v, x[m]);
    load8<T, VEC>(g + row * d_v, lane, m, d_v, gv[m]);
  }
  float mean, inv;
  row_stats<MG, VEC>(x, lane, d_v, eps, mean, inv);
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    float w[8], b[8];
    if (weight) load8<float, VEC>(weight + static_cast<int64_t>(h) * d_v, lane, m, d_v, w);
    if (bias) load8<float, VEC>(bias + static_cast<int64_t>(h) * d_v, lane, m, d_v, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float n = (x[m][e] - mean) * inv;
      n = fmaf(n, weight ? w[e] : 1.f, bias ? b[e] : 0.f);
      x[m][e] = gv[m][e] * sigmoid(gv[m][e]) * n;
    }
    store8<T, VEC>(out + row * d_v, lane, m, d_v, x[m]);
  }
}

// grid (blocks, heads).  part: [blocks][2][heads][d_v], dw then db.
template <typename T, int MG, bool VEC>
__global__ void __launch_bounds__(kThreads) msr_backward_kernel(const T* __restrict__ y, const T* __restrict__ g,
                                                                const T* __restrict__ dout,
                                                                const float* __restrict__ weight,
                                                                const float* __restrict__ bias, T* __restrict__ dy,
                                                                T* __restrict__ dg, float* __restrict__ part,
                                                                int64_t tokens, int heads, int d_v, float eps) {
  extern __shared__ float red[];  // [kWarps][d_v]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, h = blockIdx.y;
  const float inv_n = 1.f / static_cast<float>(d_v);
  float w[MG][8], b[MG][8], dw[MG][8], db[MG][8];
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    if (weight) load8<float, VEC>(weight + static_cast<int64_t>(h) * d_v, lane, m, d_v, w[m]);
    if (bias) load8<float, VEC>(bias + static_cast<int64_t>(h) * d_v, lane, m, d_v, b[m]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!weight) w[m][e] = 1.f;
      if (!bias) b[m][e] = 0.f;
      dw[m][e] = db[m][e] = 0.f;
    }
  }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < tokens; t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t at = (t * heads + h) * d_v;
    float x[MG][8], gv[MG][8], d[MG][8];
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      load8<T, VEC>(y + at, lane, m, d_v, x[m]);
      load8<T, VEC>(g + at, lane, m, d_v, gv[m]);
      load8<T, VEC>(dout + at, lane, m, d_v, d[m]);
    }
    float mean, inv;
    row_stats<MG, VEC>(x, lane, d_v, eps, mean, inv);
    float se = 0.f, sx = 0.f;
#pragma unroll
    for (int m = 0; m < MG; ++m) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gg = gv[m][e], sg = sigmoid(gg);
        const bool in = VEC ? true : column<VEC>(lane, m, e) < d_v;
        const float xh = in ? (x[m][e] - mean) * inv : 0.f;
        const float n = fmaf(w[m][e], xh, b[m][e]);
        const float dn = d[m][e] * (gg * sg);
        gv[m][e] = d[m][e] * n * sg * fmaf(gg, 1.f - sg, 1.f);
        db[m][e] += dn;
        dw[m][e] = fmaf(dn, xh, dw[m][e]);
        const float ee = w[m][e] * dn;  // zero past d_v: dout is
        x[m][e] = xh;
        d[m][e] = ee;
        se += ee;
        sx = fmaf(ee, xh, sx);
      }
      store8<T, VEC>(dg + at, lane, m, d_v, gv[m]);
    }
    const float me = warp_sum(se) * inv_n, mx = warp_sum(sx) * inv_n;
#pragma unroll
    for (int m = 0; m < MG; ++m) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[m][e] = inv * (d[m][e] - me - x[m][e] * mx);
      store8<T, VEC>(dy + at, lane, m, d_v, d[m]);
    }
  }
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<VEC>(lane, m, e);
        if (c < d_v) red[warp * d_v + c] = which ? db[m][e] : dw[m][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < d_v; c += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += red[i * d_v + c];
      part[((static_cast<int64_t>(blockIdx.x) * 2 + which) * heads + h) * d_v + c] = s;
    }
  }
}

// Sum of the partial rows: one warp a column group, the rows split over the warp's CTA.
__global__ void __launch_bounds__(kThreads) msr_reduce_kernel(const float* __restrict__ part, int blocks, int64_t n,
                                                              float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float red[kWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // of 2 n columns: dw, then db
  float s = 0.f;
  if (c < 2 * n)
    for (int i = warp; i < blocks; i += kWarps) s += part[static_cast<int64_t>(i) * 2 * n + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * n) {
#pragma unroll
    for (int i = 1; i < kWarps; ++i) s += red[i][lane];
    float* to = c < n ? dweight : dbias;
    if (to) to[c < n ? c : c - n] = s;
  }
}

// CTAs of a head in the gradient: two an SM over all heads, no more than there are rows for.
int64_t backward_blocks(int64_t tokens, int64_t heads) {
  const int64_t want = (2 * 148 + heads - 1) / heads, most = (tokens + kWarps - 1) / kWarps;
  return want < most ? want : most;
}

bool vector_ok(const MsrAffineCall& c, const void* p0, const void* p1, const void* p2) {
  auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  return c.d_v % 8 == 0 && ok(c.y) && ok(c.g) && ok(c.weight) && ok(c.bias) && ok(p0) && ok(p1) && ok(p2);
}

template <typename T, int MG, bool VEC>
cudaError_t forward_launch(const MsrAffineCall& c, void* out, cudaStream_t s) {
  const int64_t blocks = (c.tokens * c.heads + kWarps - 1) / kWarps;
  msr_affine_kernel<T, MG, VEC><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      static_cast<const T*>(c.y), static_cast<const T*>(c.g), c.weight, c.bias, static_cast<T*>(out), c.tokens,
      static_cast<int>(c.heads), static_cast<int>(c.d_v), c.eps);
  return cudaGetLastError();
}
template <typename T, int MG, bool VEC>
cudaError_t backward_launch(const MsrAffineCall& c, const void* dout, void* dy, void* dg, float* part, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(backward_blocks(c.tokens, c.heads)), static_cast<unsigned>(c.heads));
  msr_backward_kernel<T, MG, VEC><<<grid, kThreads, sizeof(float) * kWarps * static_cast<size_t>(c.d_v), s>>>(
      static_cast<const T*>(c.y), static_cast<const T*>(c.g), static_cast<const T*>(dout), c.weight, c.bias,
      static_cast<T*>(dy), static_cast<T*>(dg), part, c.tokens, static_cast<int>(c.heads), static_cast<int>(c.d_v), c.eps);
  return cudaGetLastError();
}

// F: a functor template over (T, MG, VEC).
template <typename T, typename F>
cudaError_t by_width(int64_t d_v, bool vec, F f) {
  if (d_v <= 256) return vec ? f.template run<T, 1, true>() : f.template run<T, 1, false>();
  if (d_v <= 512) return vec ? f.template run<T, 2, true>() : f.template run<T, 2, false>();
  return vec ? f.template run<T, 4, true>() : f.template run<T, 4, false>();
}
struct Forward {
  const MsrAffineCall& c;
  void* out;
  cudaStream_t s;
  template <typename T, int MG, bool VEC>
  cudaError_t run() { return forward_launch<T, MG, VEC>(c, out, s); }
};
struct Backward {
  const MsrAffineCall& c;
  const void* dout;
  void* dy;
  void* dg;
  float* part;
  cudaStream_t s;
  template <typename T, int MG, bool VEC>
  cudaError_t run() { return backward_launch<T, MG, VEC>(c, dout, dy, dg, part, s); }
};

}  // namespace

cudaError_t launch_msr_affine(const MsrAffineCall& c, void* out, cudaStream_t s) {
  const bool vec = vector_ok(c, out, nullptr, nullptr);
  Forward f{c, out, s};
  return c.dtype == RETNET_F32 ? by_width<float>(c.d_v, vec, f) : by_width<__nv_bfloat16>(c.d_v, vec, f);
}

size_t msr_backward_workspace_bytes(int64_t tokens, int64_t heads, int64_t d_v) {
  return sizeof(float) * 2 * static_cast<size_t>(backward_blocks(tokens, heads)) * static_cast<size_t>(heads * d_v);
}

cudaError_t launch_msr_affine_backward(const MsrAffineCall& c, const void* dout, void* dy, void* dg, float* dweight,
                                       float* dbias, void* ws, cudaStream_t s) {
  const bool sums = dweight || dbias;
  const bool vec = vector_ok(c, dout, dy, dg);
  Backward f{c, dout, dy, dg, sums ? static_cast<float*>(ws) : nullptr, s};
  const cudaError_t e = c.dtype == RETNET_F32 ? by_width<float>(c.d_v, vec, f) : by_width<__nv_bfloat16>(c.d_v, vec, f);
  if (e != cudaSuccess || !sums) return e;
  const int64_t n = c.heads * c.d_v;
  msr_reduce_kernel<<<static_cast<unsigned>((2 * n + 31) / 32), kThreads, 0, s>>>(
      static_cast<const float*>(ws), static_cast<int>(backward_blocks(c.tokens, c.heads)), n, dweight, dbias);
  return cudaGetLastError();
}

}  // namespace retnet
