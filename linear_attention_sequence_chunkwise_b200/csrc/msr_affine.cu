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
// while this one is worked on (without that the gradient reached 43 % of the copy rate), and the
// gradient's dw and db, sums over all tokens, are kept in registers, added up over the
// CTA in shared memory and written as one partial row a CTA; a second kernel adds the partial rows in
// order (no atomics: the same sums every time).
//
// 16384 tokens, 8 heads of 256, bf16: forward 38 us, 5.3 TB/s (80 % of the copy rate); gradient 66 us, 5.1
// TB/s (77 %), where the warps issue in 60 % of the cycles and wait for loads, shuffles and the special
// functions in turn, and 3 us for the sums.  16 heads of 512: 133 us (92 %) and 261 us (78 %).  Beyond 512 a
// warp's row leaves one CTA an SM and no registers to fetch the next row ahead, and the two CTAs an SM that the
// gradient's grid has (four the forward's) run one after another: 8192 tokens, 8 heads of 1000, 91 us (66 %) and
// 208 us (48 %).
#include <algorithm>

#include "fp32x2.cuh"
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
// Values 2 i and 2 i + 1.
__device__ __forceinline__ Two value2(const Raw<float>& r, int i) { return two(r.x[2 * i], r.x[2 * i + 1]); }
__device__ __forceinline__ Two value2(const Raw<__nv_bfloat16>& r, int i) {
  return two(__uint_as_float(r.x[i] << 16), __uint_as_float(r.x[i] & 0xffff0000u));
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
__device__ __forceinline__ void spread(const Two (&v)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = parts(v[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}
template <int W, int LPR>
__device__ __forceinline__ void store(float* p, int lane, int m, int d_v, const Two (&v)[4]) {
  float x[8];
  spread(v, x);
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
__device__ __forceinline__ void store(__nv_bfloat16* p, int lane, int m, int d_v, const Two (&v)[4]) {
  float x[8];
  spread(v, x);
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

// x <- x - mean, and 1/sd (values past d_v, loaded as zeros, become zeros: out of the variance).  FULL:
// the lanes hold exactly d_v values.
template <int MG, int W, int LPR, bool FULL>
__device__ __forceinline__ float centre(Two (&x)[MG][4], int lane, int d_v, float inv_n, float eps) {
  Two s = two(0.f);
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) s = add2(s, x[m][i]);
  const Two less = two(-row_sum<LPR>(sum_of(s)) * inv_n);
  Two sq = two(0.f);
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[m][i] = add2(x[m][i], less);
      if (!FULL) {
        const float2 p = parts(x[m][i]);
        x[m][i] = two(column<W, LPR>(lane, m, 2 * i) < d_v ? p.x : 0.f, column<W, LPR>(lane, m, 2 * i + 1) < d_v ? p.y : 0.f);
      }
      sq = fma2(x[m][i], x[m][i], sq);
    }
  return rsqrtf(fmaf(row_sum<LPR>(sum_of(sq)), inv_n, eps));
}

// 1 / (1 + exp(-g)) of both lanes by the approximate exponential and division: a few 2^-23 of the value
// for |g| below ten, growing with |g| where 1 + exp(-g) is near 1 or the product with g is tiny.
__device__ __forceinline__ Two sigmoid2(Two g) {
  const float2 p = parts(g);
  return two(__fdividef(1.f, 1.f + __expf(-p.x)), __fdividef(1.f, 1.f + __expf(-p.y)));
}

// Weight and bias of the CTA's head.
template <int MG, int W, int LPR>
__device__ __forceinline__ void load_affine(Two (&w)[MG][4], Two (&b)[MG][4], const float* weight, const float* bias,
                                            int h, int lane, int d_v) {
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    Raw<float> rw, rb;
    if (weight) load<W, LPR>(rw, weight + static_cast<int64_t>(h) * d_v, lane, m, d_v);
    if (bias) load<W, LPR>(rb, bias + static_cast<int64_t>(h) * d_v, lane, m, d_v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[m][i] = weight ? value2(rw, i) : two(1.f);
      b[m][i] = bias ? value2(rb, i) : two(0.f);
    }
  }
}

// grid (blocks, heads): the CTA's rows are tokens blockIdx.x * rows + i, + gridDim.x * rows, ...
template <typename T, int MG, int W, int LPR, bool FULL>
__global__ void __launch_bounds__(kThreads, MG == 1 ? 4 : 1)
    msr_affine_kernel(const T* y, const T* g, const float* weight, const float* bias, T* out,
                      int64_t tokens, int heads, int d_v, float eps) {
  constexpr int kRows = kThreads / LPR;
  const int lane = threadIdx.x % LPR, h = blockIdx.y;
  const float inv_n = 1.f / static_cast<float>(d_v);
  Two w[MG][4], b[MG][4];
  pdl_wait();
  load_affine<MG, W, LPR>(w, b, weight, bias, h, lane, d_v);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows, pitch = static_cast<int64_t>(heads) * d_v;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  int64_t t = first + threadIdx.x / LPR;
  Raw<T> ry[MG], rg[MG];
  auto fetch = [&](int64_t at) {
    if (at >= tokens) return;
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      load<W, LPR>(ry[m], y + at * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v);
      load<W, LPR>(rg[m], g + at * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v);
    }
  };
  fetch(t);
  for (int64_t t0 = first; t0 < tokens; t0 += step, t += step) {  // all lanes of a warp alike: shuffles
    Two x[MG][4], gv[MG][4];
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[m][i] = value2(ry[m], i);
        gv[m][i] = value2(rg[m], i);
      }
    fetch(t + step);
    const Two inv = two(centre<MG, W, LPR, FULL>(x, lane, d_v, inv_n, eps));
    if (t < tokens) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[m][i] = mul2(mul2(gv[m][i], sigmoid2(gv[m][i])), fma2(mul2(x[m][i], inv), w[m][i], b[m][i]));
        store<W, LPR>(out + t * pitch + static_cast<int64_t>(h) * d_v, lane, m, d_v, x[m]);
      }
    }
  }
}

// grid (blocks, heads).  part: [blocks][2][heads][d_v], dw then db.
template <typename T, int MG, int W, int LPR, bool FULL>
__global__ void __launch_bounds__(kThreads, MG == 1 ? 2 : 1)
    msr_backward_kernel(const T* y, const T* g, const T* dout, const float* weight, const float* bias, T* dy, T* dg,
                        float* part, int64_t tokens, int heads, int d_v, float eps) {
  extern __shared__ float red[];  // [rows][d_v]
  constexpr int kRows = kThreads / LPR;
  const int lane = threadIdx.x % LPR, row = threadIdx.x / LPR, h = blockIdx.y;
  const float inv_n = 1.f / static_cast<float>(d_v);
  Two w[MG][4], b[MG][4], dw[MG][4], db[MG][4];
  pdl_wait();
  load_affine<MG, W, LPR>(w, b, weight, bias, h, lane, d_v);
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[m][i] = db[m][i] = two(0.f);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows, pitch = static_cast<int64_t>(heads) * d_v;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  int64_t t = first + row;
  constexpr bool kAhead = MG < 4;  // at MG = 4 the registers are full without the next row
  Raw<T> ry[MG], rg[MG], rd[MG];
  auto fetch = [&](int64_t at) {
    if (at >= tokens) return;
    at = at * pitch + static_cast<int64_t>(h) * d_v;
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      load<W, LPR>(ry[m], y + at, lane, m, d_v);
      load<W, LPR>(rg[m], g + at, lane, m, d_v);
      load<W, LPR>(rd[m], dout + at, lane, m, d_v);
    }
  };
  if (kAhead) fetch(t);
  for (int64_t t0 = first; t0 < tokens; t0 += step, t += step) {
    const bool live = t < tokens;
    if (!kAhead) fetch(t);
    Two x[MG][4], gv[MG][4], d[MG][4];
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[m][i] = value2(ry[m], i);
        gv[m][i] = value2(rg[m], i);
        d[m][i] = value2(rd[m], i);
      }
    if (kAhead) fetch(t + step);
    const float inv = centre<MG, W, LPR, FULL>(x, lane, d_v, inv_n, eps);
    const int64_t at = t * pitch + static_cast<int64_t>(h) * d_v;
    Two se = two(0.f), sx = two(0.f);
    if (live) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two gg = gv[m][i], sg = sigmoid2(gg);
          const Two xh = mul2(x[m][i], two(inv));
          const Two n = fma2(w[m][i], xh, b[m][i]);
          const Two ds = mul2(d[m][i], sg), dn = mul2(ds, gg);
          // swish'(g) = s (1 + g (1 - s)) = s + g s (1 - s)
          gv[m][i] = mul2(mul2(ds, n), fma2(gg, fma2(sg, two(-1.f), two(1.f)), two(1.f)));
          const Two ee = mul2(w[m][i], dn);  // past d_v dout is zero, and so are dn, ee and what they add to
          db[m][i] = add2(db[m][i], dn);
          dw[m][i] = fma2(dn, xh, dw[m][i]);
          x[m][i] = xh;
          d[m][i] = ee;
          se = add2(se, ee);
          sx = fma2(ee, xh, sx);
        }
        store<W, LPR>(dg + at, lane, m, d_v, gv[m]);
      }
    }
    const Two me = two(-row_sum<LPR>(sum_of(se)) * inv_n), mx = two(-row_sum<LPR>(sum_of(sx)) * inv_n);
    if (live) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[m][i] = mul2(two(inv), fma2(x[m][i], mx, add2(d[m][i], me)));
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
    for (int m = 0; m < MG; ++m) {
      float v[8];
      spread(which ? db[m] : dw[m], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<W, LPR>(lane, m, e);
        if (c < d_v) red[row * d_v + c] = v[e];
      }
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

// CTAs of a head: `per_sm` an SM over all heads, rounded down (four CTAs in a second wave took the
// forward from 42 to 60 us), no more than there are rows for.
int64_t blocks_of(int64_t tokens, int64_t heads, int rows, int per_sm) {
  const int64_t want = std::max<int64_t>(1, per_sm * 148 / heads);
  return std::min(want, (tokens + rows - 1) / rows);
}
// (with 32 lanes for all, forward and gradient of 16384 x 8 rows of 64 took 92 us instead of 30, of 128 94
// instead of 57)
int lanes_per_row(int64_t d_v) { return d_v <= 64 ? 8 : d_v <= 128 ? 16 : 32; }
int64_t backward_blocks(int64_t tokens, int64_t heads, int64_t d_v) {
  return blocks_of(tokens, heads, kThreads / lanes_per_row(d_v), 2);
}

// The widest access that the width and every address allow (8 values of bf16 against 4: 298 us against 340 at
// 8192 x 8 rows of 1000, no difference up to 512).
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
  template <typename T, int MG, int W, int LPR, bool FULL>
  cudaError_t run() {
    const dim3 grid(static_cast<unsigned>(blocks_of(c.tokens, c.heads, kThreads / LPR, 4)), static_cast<unsigned>(c.heads));
    return launch_dependent(msr_affine_kernel<T, MG, W, LPR, FULL>, grid, dim3(kThreads), 0, s, static_cast<const T*>(c.y),
                            static_cast<const T*>(c.g), c.weight, c.bias, static_cast<T*>(out), c.tokens,
                            static_cast<int>(c.heads), static_cast<int>(c.d_v), c.eps);
  }
};
struct Backward {
  const MsrAffineCall& c;
  const void* dout;
  void* dy;
  void* dg;
  float* part;
  cudaStream_t s;
  template <typename T, int MG, int W, int LPR, bool FULL>
  cudaError_t run() {
    const dim3 grid(static_cast<unsigned>(backward_blocks(c.tokens, c.heads, c.d_v)), static_cast<unsigned>(c.heads));
    // at most 32 KB: kThreads / LPR rows of at most 8 LPR (LPR < 32) or 1024 values
    const size_t smem = part ? sizeof(float) * (kThreads / LPR) * static_cast<size_t>(c.d_v) : 0;
    return launch_dependent(msr_backward_kernel<T, MG, W, LPR, FULL>, grid, dim3(kThreads), smem, s,
                            static_cast<const T*>(c.y), static_cast<const T*>(c.g), static_cast<const T*>(dout), c.weight,
                            c.bias, static_cast<T*>(dy), static_cast<T*>(dg), part, c.tokens, static_cast<int>(c.heads),
                            static_cast<int>(c.d_v), c.eps);
  }
};
// (forward and gradient of 16384 x 8 full rows of 256: 104.6 us, 106.5 without FULL)
template <typename T, int W, int MG, int LPR, typename F>
cudaError_t by_fullness(int64_t d_v, F& f) {
  return d_v == 8 * MG * LPR ? f.template run<T, MG, W, LPR, true>() : f.template run<T, MG, W, LPR, false>();
}
template <typename T, int W, typename F>
cudaError_t by_row(int64_t d_v, F& f) {
  if (d_v <= 64) return by_fullness<T, W, 1, 8>(d_v, f);
  if (d_v <= 128) return by_fullness<T, W, 1, 16>(d_v, f);
  if (d_v <= 256) return by_fullness<T, W, 1, 32>(d_v, f);
  if (d_v <= 512) return by_fullness<T, W, 2, 32>(d_v, f);
  return by_fullness<T, W, 4, 32>(d_v, f);
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
