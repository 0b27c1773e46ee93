// msr_affine.cu -- the MSR epilogue ("阅读笔记：RetNet" §三.2) with a learnable affine, and its gradient:
//   x^ = (y - m) / sd over a (token, head) row,  n = w x^ + b,  out = swish(g) n,  swish(g) = g s(g);
//   db = sum_t swish(g) dout,  dw = sum_t swish(g) dout x^,  dg = dout n s(g) (1 + g (1 - s(g))),
//   with e = w swish(g) dout:  dy = (e - mean(e) - x^ mean(e x^)) / sd.
//
// Bound by HBM: y, g (and dout) are read once, out (dy, dg) written once.  LPR lanes (8, 16 or 32: the
// fewest that hold it at eight values a lane) keep a row in registers, so the mean, the centred
// variance and the two means of the gradient are shuffles over registers; the statistics are
// recomputed by the gradient, which reads y anyway, instead of being kept.  A CTA stays on one head
// and strides over its tokens: weight and bias stay in registers, the next row's loads are in flight
// while this one is worked on (without that, 24 KB a CTA pair in flight reached 43 % of the copy
// rate), and the gradient's dw and db, sums over all tokens, are kept in registers, added up over the
// CTA in shared memory and written as one partial row a CTA; a second kernel adds the partial rows in
// order (no atomics: the same sums every time).
#include "launch.h"
#include "pdl.cuh"

namespace retnet {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

// Eight values of a lane (group m of MG), W consecutive ones at a time: W = 8 (bf16 in 16 bytes), 4
// (fp32 in 16 bytes, bf16 in 8) or 1 (odd widths and addresses).
template <int W, int LPR>
__device__ __forceinline__ int column(int lane, int m, int e) {
  return (lane + LPR * (m * (8 / W) + e / W)) * W + e % W;
}
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float x[8];
};
template <>
struct Raw<__nv_bfloat16> {
  uint32_t x[4];
};
__device__ __forceinline__ float value(const Raw<float>& r, int e) { return r.x[e]; }
__device__ __forceinline__ float value(const Raw<__nv_bfloat16>& r, int e) {
  return __uint_as_float(e % 2 ? r.x[e / 2] & 0xffff0000u : r.x[e / 2] << 16);
}

template <int W, int LPR>
__device__ __forceinline__ void load(Raw<float>& r, const float* p, int lane, int m, int d_v) {
  if constexpr (W == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<1, LPR>(lane, m, e);
      r.x[e] = c < d_v ? p[c] : 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int c = column<W, LPR>(lane, m, e);
      const float4 v = c < d_v ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      r.x[e] = v.x; r.x[e + 1] = v.y; r.x[e + 2] = v.z; r.x[e + 3] = v.w;
    }
  }
}
template <int W, int LPR>
__device__ __forceinline__ void load(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p, int lane, int m, int d_v) {
  if constexpr (W == 8) {
    const int c = column<8, LPR>(lane, m, 0);
    const uint4 v = c < d_v ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
    r.x[0] = v.x; r.x[1] = v.y; r.x[2] = v.z; r.x[3] = v.w;
  } else if constexpr (W == 4) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int c = column<4, LPR>(lane, m, e);
      const uint2 v = c < d_v ? *reinterpret_cast<const uint2*>(p + c) : make_uint2(0, 0);
      r.x[e / 2] = v.x; r.x[e / 2 + 1] = v.y;
    }
  } else {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int c0 = column<1, LPR>(lane, m, e), c1 = column<1, LPR>(lane, m, e + 1);
      const uint32_t lo = c0 < d_v ? u[c0] : 0u, hi = c1 < d_v ? u[c1] : 0u;
      r.x[e / 2] = lo | (hi << 16);
    }
  }
}
template <int W, int LPR>
__device__ __forceinline__ void store(float* p, int lane, int m, int d_v, const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += W == 1 ? 1 : 4) {
    const int c = column<W, LPR>(lane, m, e);
    if (c >= d_v) continue;
    if constexpr (W == 1) p[c] = x[e];
    else *reinterpret_cast<float4*>(p + c) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int W, int LPR>
__device__ __forceinline__ void store(__nv_bfloat16* p, int lane, int m, int d_v, const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += W) {
    const int c = column<W, LPR>(lane, m, e);
    if (c >= d_v) continue;
    if constexpr (W == 8)
      *reinterpret_cast<uint4*>(p + c) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    else if constexpr (W == 4)
      *reinterpret_cast<uint2*>(p + c) = make_uint2(pack2(x[e], x[e + 1]), pack2(x[e + 2], x[e + 3]));
    else
      store_f(p, c, x[e]);
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// Mean and 1/sd of the row in x (values past d_v are zero and stay out of the variance).
template <int MG, int W, int LPR>
__device__ __forceinline__ void row_stats(const float (&x)[MG][8], int lane, int d_v, float eps, float& mean, float& inv) {
  float s = 0.f;
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[m][e];
  mean = row_sum<LPR>(s) / static_cast<float>(d_v);
  float sq = 0.f;
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = column<W, LPR>(lane, m, e) < d_v ? x[m][e] - mean : 0.f;
      sq = fmaf(c, c, sq);
    }
  inv = rsqrtf(row_sum<LPR>(sq) / static_cast<float>(d_v) + eps);
}

// (the approximate division is within 2 ulp, and 0 where exp passes 2^126, as the quotient nearly is)
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + expf(-g)); }

// Weight and bias of the CTA's head.
template <int MG, int W, int LPR>
__device__ __forceinline__ void load_affine(float (&w)[MG][8], float (&b)[MG][8], const float* weight, const float* bias,
                                            int h, int lane, int d_v) {
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    Raw<float> rw, rb;
    if (weight) load<W, LPR>(rw, weight + static_cast<int64_t>(h) * d_v, lane, m, d_v);
    if (bias) load<W, LPR>(rb, bias + static_cast<int64_t>(h) * d_v, lane, m, d_v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[m][e] = weight ? rw.x[e] : 1.f;
      b[m][e] = bias ? rb.x[e] : 0.f;
    }
  }
}

// grid (blocks, heads): the CTA's rows are tokens blockIdx.x * rows + i, + gridDim.x * rows, ...
template <typename T, int MG, int W, int LPR>
__global__ void __launch_bounds__(kThreads, MG == 1 ? 3 : 1)
    msr_affine_kernel(const T* y, const T* g, const float* __restrict__ weight, const float* __restrict__ bias, T* out,
                      int64_t tokens, int heads, int d_v, float eps) {
  constexpr int kRows = kThreads / LPR;
  const int lane = threadIdx.x % LPR, h = blockIdx.y;
  float w[MG][8], b[MG][8];
  load_affine<MG, W, LPR>(w, b, weight, bias, h, lane, d_v);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows, pitch = static_cast<int64_t>(heads) * d_v;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  int64_t t = first + threadIdx.x / LPR;
  Raw<T> ry[MG], rg[MG];
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      load<W, LPR>(ry[m], y + at * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v);
      load<W, LPR>(rg[m], g + at * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v);
    }
  };
  if (t < tokens) fetch(t);
  for (int64_t t0 = first; t0 < tokens; t0 += step, t += step) {  // all lanes of a warp alike: shuffles
    float x[MG][8], gv[MG][8];
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[m][e] = value(ry[m], e);
        gv[m][e] = value(rg[m], e);
      }
    if (t + step < tokens) fetch(t + step);
    float mean, inv;
    row_stats<MG, W, LPR>(x, lane, d_v, eps, mean, inv);
    if (t < tokens) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[m][e] = gv[m][e] * sigmoid(gv[m][e]) * fmaf((x[m][e] - mean) * inv, w[m][e], b[m][e]);
        store<W, LPR>(out + t * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v, x[m]);
      }
    }
  }
}

// grid (blocks, heads).  part: [blocks][2][heads][d_v], dw then db.
template <typename T, int MG, int W, int LPR>
__global__ void __launch_bounds__(kThreads, MG == 1 ? 2 : 1)
    msr_backward_kernel(const T* __restrict__ y, const T* __restrict__ g, const T* __restrict__ dout,
                        const float* __restrict__ weight, const float* __restrict__ bias, T* __restrict__ dy,
                        T* __restrict__ dg, float* __restrict__ part, int64_t tokens, int heads, int d_v, float eps) {
  extern __shared__ float red[];  // [rows][d_v]
  constexpr int kRows = kThreads / LPR;
  const int lane = threadIdx.x % LPR, row = threadIdx.x / LPR, h = blockIdx.y;
  const float inv_n = 1.f / static_cast<float>(d_v);
  float w[MG][8], b[MG][8], dw[MG][8], db[MG][8];
  load_affine<MG, W, LPR>(w, b, weight, bias, h, lane, d_v);
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[m][e] = db[m][e] = 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows, pitch = static_cast<int64_t>(heads) * d_v;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  int64_t t = first + row;
  Raw<T> ry[MG], rg[MG], rd[MG];
  auto fetch = [&](int64_t at) {
    at = at * pitch + static_cast<int64_t>(h) * d_v;
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      load<W, LPR>(ry[m], y + at, lane, m, d_v);
      load<W, LPR>(rg[m], g + at, lane, m, d_v);
      load<W, LPR>(rd[m], dout + at, lane, m, d_v);
    }
  };
  constexpr bool kAhead = MG < 4;  // at MG = 4 the registers are full without the next row
  if (kAhead && t < tokens) fetch(t);
  for (int64_t t0 = first; t0 < tokens; t0 += step, t += step) {
    float x[MG][8], gv[MG][8], d[MG][8];
    const bool live = t < tokens;
    if (!kAhead && live) fetch(t);
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[m][e] = value(ry[m], e);
        gv[m][e] = value(rg[m], e);
        d[m][e] = value(rd[m], e);
      }
    if (kAhead && t + step < tokens) fetch(t + step);
    float mean, inv;
    row_stats<MG, W, LPR>(x, lane, d_v, eps, mean, inv);
    const int64_t at = t * pitch + static_cast<int64_t>(h) * d_v;
    float se = 0.f, sx = 0.f;
    if (live) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gg = gv[m][e], sg = sigmoid(gg);
          const float xh = (x[m][e] - mean) * inv;
          const float n = fmaf(w[m][e], xh, b[m][e]);
          const float dn = d[m][e] * (gg * sg);
          gv[m][e] = d[m][e] * n * sg * fmaf(gg, 1.f - sg, 1.f);
          const float ee = w[m][e] * dn;  // past d_v dout is zero, and so are dn, ee and what they add to
          db[m][e] += dn;
          dw[m][e] = fmaf(dn, xh, dw[m][e]);
          x[m][e] = xh;
          d[m][e] = ee;
          se += ee;
          sx = fmaf(ee, xh, sx);
        }
        store<W, LPR>(dg + at, lane, m, d_v, gv[m]);
      }
    }
    const float me = row_sum<LPR>(se) * inv_n, mx = row_sum<LPR>(sx) * inv_n;
    if (live) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[m][e] = inv * (d[m][e] - me - x[m][e] * mx);
        store<W, LPR>(dy + at, lane, m, d_v, d[m]);
      }
    }
  }
  pdl_go();
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<W, LPR>(lane, m, e);
        if (c < d_v) red[row * d_v + c] = which ? db[m][e] : dw[m][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < d_v; c += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int i = 0; i < kRows; ++i) s += red[i * d_v + c];
      part[((static_cast<int64_t>(blockIdx.x) * 2 + which) * heads + h) * d_v + c] = s;
    }
  }
}

// Sum of the partial rows: one warp a column group, the rows split over the warp's CTA.
__global__ void __launch_bounds__(kThreads) msr_reduce_kernel(const float* part, int blocks, int64_t n,
                                                              float* dweight, float* dbias) {
  __shared__ float red[kWarps][32];
  pdl_wait();  // the partial rows are written
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

// CTAs of a head: `per_sm` an SM over all heads, no more than there are rows for.
int64_t blocks_of(int64_t tokens, int64_t heads, int rows, int per_sm) {
  const int64_t want = (per_sm * 148 + heads - 1) / heads, most = (tokens + rows - 1) / rows;
  return want < most ? want : most;
}
int lanes_per_row(int64_t d_v) { return d_v <= 64 ? 8 : d_v <= 128 ? 16 : 32; }
int64_t backward_blocks(int64_t tokens, int64_t heads, int64_t d_v) {
  return blocks_of(tokens, heads, kThreads / lanes_per_row(d_v), 2);
}

// The widest access that the width and every address allow.
template <typename T>
int vector_width(const MsrAffineCall& c, const void* p0, const void* p1, const void* p2) {
  auto ok = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!ok(c.weight, 16) || !ok(c.bias, 16)) return 1;
  auto data = [&](uintptr_t n) { return ok(c.y, n) && ok(c.g, n) && ok(p0, n) && ok(p1, n) && ok(p2, n); };
  if (sizeof(T) == 2 && c.d_v % 8 == 0 && data(16)) return 8;
  return c.d_v % 4 == 0 && data(4 * sizeof(T)) ? 4 : 1;
}

struct Forward {
  const MsrAffineCall& c;
  void* out;
  cudaStream_t s;
  template <typename T, int MG, int W, int LPR>
  cudaError_t run() {
    const dim3 grid(static_cast<unsigned>(blocks_of(c.tokens, c.heads, kThreads / LPR, 3)), static_cast<unsigned>(c.heads));
    msr_affine_kernel<T, MG, W, LPR><<<grid, kThreads, 0, s>>>(
        static_cast<const T*>(c.y), static_cast<const T*>(c.g), c.weight, c.bias, static_cast<T*>(out), c.tokens,
        static_cast<int>(c.heads), static_cast<int>(c.d_v), c.eps);
    return cudaGetLastError();
  }
};
struct Backward {
  const MsrAffineCall& c;
  const void* dout;
  void* dy;
  void* dg;
  float* part;
  cudaStream_t s;
  template <typename T, int MG, int W, int LPR>
  cudaError_t run() {
    const dim3 grid(static_cast<unsigned>(backward_blocks(c.tokens, c.heads, c.d_v)), static_cast<unsigned>(c.heads));
    // at most 32 KB: kThreads / LPR rows of at most 8 LPR (LPR < 32) or 1024 values
    const size_t smem = part ? sizeof(float) * (kThreads / LPR) * static_cast<size_t>(c.d_v) : 0;
    msr_backward_kernel<T, MG, W, LPR><<<grid, kThreads, smem, s>>>(
        static_cast<const T*>(c.y), static_cast<const T*>(c.g), static_cast<const T*>(dout), c.weight, c.bias,
        static_cast<T*>(dy), static_cast<T*>(dg), part, c.tokens, static_cast<int>(c.heads), static_cast<int>(c.d_v), c.eps);
    return cudaGetLastError();
  }
};
template <typename T, int W, typename F>
cudaError_t by_row(int64_t d_v, F& f) {
  if (d_v <= 64) return f.template run<T, 1, W, 8>();
  if (d_v <= 128) return f.template run<T, 1, W, 16>();
  if (d_v <= 256) return f.template run<T, 1, W, 32>();
  if (d_v <= 512) return f.template run<T, 2, W, 32>();
  return f.template run<T, 4, W, 32>();
}
template <typename F>
cudaError_t dispatch(const MsrAffineCall& c, F& f, const void* p0, const void* p1, const void* p2) {
  if (c.dtype == RETNET_F32)
    return vector_width<float>(c, p0, p1, p2) == 4 ? by_row<float, 4>(c.d_v, f) : by_row<float, 1>(c.d_v, f);
  const int w = vector_width<__nv_bfloat16>(c, p0, p1, p2);
  if (w == 8) return by_row<__nv_bfloat16, 8>(c.d_v, f);
  return w == 4 ? by_row<__nv_bfloat16, 4>(c.d_v, f) : by_row<__nv_bfloat16, 1>(c.d_v, f);
}

}  // namespace

cudaError_t launch_msr_affine(const MsrAffineCall& c, void* out, cudaStream_t s) {
  Forward f{c, out, s};
  return dispatch(c, f, out, nullptr, nullptr);
}

size_t msr_backward_workspace_bytes(int64_t tokens, int64_t heads, int64_t d_v) {
  return sizeof(float) * 2 * static_cast<size_t>(backward_blocks(tokens, heads, d_v)) * static_cast<size_t>(heads * d_v);
}

cudaError_t launch_msr_affine_backward(const MsrAffineCall& c, const void* dout, void* dy, void* dg, float* dweight,
                                       float* dbias, void* ws, cudaStream_t s) {
  const bool sums = dweight || dbias;
  Backward f{c, dout, dy, dg, sums ? static_cast<float*>(ws) : nullptr, s};
  const cudaError_t e = dispatch(c, f, dout, dy, dg);
  if (e != cudaSuccess || !sums) return e;
  const int64_t n = c.heads * c.d_v;
  return launch_dependent(msr_reduce_kernel, dim3(static_cast<unsigned>((2 * n + 31) / 32)), dim3(kThreads), 0, s,
                          static_cast<const float*>(ws), static_cast<int>(backward_blocks(c.tokens, c.heads, c.d_v)), n,
                          dweight, dbias);
}

}  // namespace retnet
