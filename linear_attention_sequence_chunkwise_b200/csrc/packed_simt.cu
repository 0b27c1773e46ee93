// packed_simt.cu -- packed retention in fp32 on the CUDA cores: fp32 inputs (whose tolerance rules
// out 16-bit tensor-core operands) and every width, stride and decay that the tensor-core kernels do
// not take.  "阅读笔记：RetNet" §2.4 with the sequence cut into runs (packed.cuh):
//   rotate  q', k' in fp32, rows padded to four values, once a token (the angles in fp64);
//   state   W_u = sum_t gamma^(end-1-t) k'_t^T v_t of every run, all runs at once;
//   scan    a sequence's runs in order: R_u = the state before run u (written over W_u),
//           R <- gamma^len R + W; the last R goes to the pool;
//   output  o_n = f_n [ sum_{m in run, m<=n} gamma^(n-m) (q'_n . k'_m) v_m + gamma^(n-start+1) q'_n R_u ].
// Bound by the fp32 FMA rate and, with few tokens, by the latency of its five launches: tiles of 64 rows x
// 128 columns as packed pairs, operands in steps of 16 through shared memory with the next step's loads in
// flight.  Runs are 64 tokens (one tile: the least arithmetic) up to states of 128 x 256, 256 tokens beyond,
// where the states of shorter runs would be most of the workspace (2999 fp32 tokens, 8 heads, runs of 64
// against 256: 125 us against 185 at 128 x 128, 226 against 293 at 128 x 256, 452 against 480 at 256 x 256).
// 2999 tokens, 8 heads on 2, 80 x 120: 71 us, 39 of them the output kernel at about half the FMA rate.
#include "fp32x2.cuh"
#include "packed.cuh"
#include "pdl.cuh"

namespace retnet {
namespace {

constexpr int kTile = 64;     // tokens of a tile
constexpr int kWide = 128;    // columns of a tile
constexpr int kStep = 16;     // depth of one shared-memory step
constexpr int kThreads = 256;
constexpr int kPitch = kTile + 4, kWidePitch = kWide + 4;

int run_of(int64_t d_k, int64_t d_v) { return d_k * d_v <= 128 * 256 ? 64 : 256; }

template <typename T>
struct SimtPackedArgs {
  const T* q;
  const T* k;
  const T* v;
  T* o;
  float* pool;
  const RunDesc* desc;
  float* qf;      // [rows][heads][pitch] rotated
  float* kf;      // [rows][kv][pitch]
  float* factor;  // [rows][kv] row factors
  float* w;       // [units][kv][d_k][d_v]
  const int32_t* cu;
  int64_t units, stride_q, stride_k, stride_v, stride_o;
  int32_t run, heads, kv, group, d_k, d_v, pitch;
  uint32_t flags;
};

// grid (units, y): the CTA's share of the run's tokens, eight at a time: each one's rotations once, into
// shared memory, then all heads with 16-byte stores.
constexpr int kTokens = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_rotate_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  __shared__ __align__(16) float2 rot[kTokens][kMaxPairs];
  pdl_wait();
  pdl_go();
  const RunDesc d = a.desc[blockIdx.x];
  const bool xpos = (a.flags & RETNET_F_XPOS) != 0;
  const int pairs = a.pitch / 2, quads = a.pitch / 4, heads = a.heads + a.kv;
  for (int t0 = blockIdx.y * kTokens; t0 < d.tokens; t0 += gridDim.y * kTokens) {
    for (int e = threadIdx.x; e < kTokens * pairs; e += kThreads) {
      const int t = e / pairs, j = e % pairs;
      float s = 0.f, c = 1.f;
      if (xpos && 2 * j < a.d_k) position_sincos(d.pos + t0 + t, hp.theta[j], &s, &c);
      rot[t][j] = make_float2(c, s);
    }
    // the row factors, by the last threads: the first ones have most of the angles
    for (int e = kThreads - 1 - threadIdx.x; e < kTokens * a.kv; e += kThreads) {
      const int t = t0 + e / a.kv, h = e % a.kv;
      if (t < d.tokens) a.factor[static_cast<int64_t>(d.row + t) * a.kv + h] = row_factor(hp.gamma[h], a.d_k, d.pos + t, a.flags);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kTokens * heads * quads; e += kThreads) {
      const int i = e % quads * 4, h = e / quads % heads, t = e / quads / heads;
      if (t0 + t >= d.tokens) break;  // tokens are the slowest index
      const int64_t row = d.row + t0 + t;
      const T* from = h < a.heads ? a.q + row * a.stride_q + static_cast<int64_t>(h) * a.d_k
                                  : a.k + row * a.stride_k + static_cast<int64_t>(h - a.heads) * a.d_k;
      float* to = h < a.heads ? a.qf + (row * a.heads + h) * a.pitch : a.kf + (row * a.kv + h - a.heads) * a.pitch;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < a.d_k ? load_f(from, i + j) : 0.f;
      const float4 cs = *reinterpret_cast<const float4*>(&rot[t][i / 2]);
      *reinterpret_cast<float4*>(to + i) = make_float4(x[0] * cs.x - x[1] * cs.y, x[0] * cs.y + x[1] * cs.x,
                                                       x[2] * cs.z - x[3] * cs.w, x[2] * cs.w + x[3] * cs.z);
    }
    __syncthreads();
  }
}

// One step of a tile of 64 rows: a[r][i] (the first operand's 64 values), b[r][j].  A thread has R rows from
// R ty and 2 N columns: 4 tx .., 64 + 4 tx ...
template <int R, int N, int P>
__device__ __forceinline__ void fma_step(Two (&acc)[R][N], const float (*a)[kPitch], const float (*b)[P], int ty, int tx) {
#pragma unroll
  for (int r = 0; r < kStep; ++r) {
    Two xx[R];
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&a[r][ty * R + i]);
      xx[i] = two(x.x);
      xx[i + 1] = two(x.y);
      xx[i + 2] = two(x.z);
      xx[i + 3] = two(x.w);
    }
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&b[r][j * 32 + tx * 4]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        acc[i][j] = fma2(xx[i], y.x, acc[i][j]);
        acc[i][j + 1] = fma2(xx[i], y.y, acc[i][j + 1]);
      }
    }
  }
}

// grid (units, kv, tiles of d_k (64) x tiles of d_v (128))
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_state_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  __shared__ __align__(16) float ks[kStep][kPitch], vs[kStep][kWidePitch];
  pdl_wait();
  pdl_go();
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int h = blockIdx.y, tv = (a.d_v + kWide - 1) / kWide;
  const int i0 = (blockIdx.z / tv) * kTile, j0 = (blockIdx.z % tv) * kWide;
  const int tid = threadIdx.x, ty = tid / 64 * 4 + tid % 32 / 8, tx = tid / 32 % 2 * 8 + tid % 8;  // 4 x 8 lanes a warp
  const float lg = hp.log2g[h];
  Two acc[4][4] = {};
  float4 kr;
  float vr[8];
  const int kt = tid / 16, kc = tid % 16 * 4, vt = tid / 128, vc = tid % 128;
  auto fetch = [&](int t0) {
    const int t = t0 + kt;
    kr = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < d.tokens && i0 + kc < a.pitch)
      kr = *reinterpret_cast<const float4*>(a.kf + (static_cast<int64_t>(d.row + t) * a.kv + h) * a.pitch + i0 + kc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = t0 + vt + 2 * i;
      vr[i] = u < d.tokens && j0 + vc < a.d_v
                  ? load_f(a.v, static_cast<int64_t>(d.row + u) * a.stride_v + static_cast<int64_t>(h) * a.d_v + j0 + vc)
                  : 0.f;
    }
  };
  fetch(0);
  for (int t0 = 0; t0 < d.tokens; t0 += kStep) {
    const int t = t0 + kt;
    const float dec = t < d.tokens ? decay_pow(lg, d.tokens - 1 - t) : 0.f;
    *reinterpret_cast<float4*>(&ks[kt][kc]) = make_float4(kr.x * dec, kr.y * dec, kr.z * dec, kr.w * dec);
#pragma unroll
    for (int i = 0; i < 8; ++i) vs[vt + 2 * i][vc] = vr[i];
    __syncthreads();
    if (t0 + kStep < d.tokens) fetch(t0 + kStep);
    fma_step(acc, ks, vs, ty, tx);
    __syncthreads();
  }
  float* w = a.w + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * a.d_k * a.d_v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i0 + ty * 4 + i;
    if (r >= a.d_k) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = parts(acc[i][j]);
      const int c = j0 + (j / 2) * 64 + tx * 4 + (j % 2) * 2;
      if (c < a.d_v) w[static_cast<int64_t>(r) * a.d_v + c] = x.x;
      if (c + 1 < a.d_v) w[static_cast<int64_t>(r) * a.d_v + c + 1] = x.y;
    }
  }
}

// grid (blocks of d_k d_v, kv, seqs)
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_scan_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  pdl_wait();
  pdl_go();
  const int s = blockIdx.z, h = blockIdx.y;
  const int64_t n = static_cast<int64_t>(a.d_k) * a.d_v;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t u0 = a.cu[s] / a.run + s;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc first = a.desc[u0];
  if (first.tokens == 0 || first.seq != s || e >= n) return;
  float* slot = a.pool + (static_cast<int64_t>(first.slot) * a.kv + h) * n + e;
  float r = first.pos > 0 ? *slot : 0.f;
  const float lg = hp.log2g[h];
  const Decay full = decay_of(lg, a.run);
  const int64_t step = static_cast<int64_t>(a.kv) * n;
  float* w = a.w + (u0 * a.kv + h) * n + e;
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < first.runs; i0 += kAhead, w += kAhead * step) {
    float x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < first.runs) x[i] = w[i * step];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= first.runs) break;
      w[i * step] = r;
      const Decay d = i0 + i + 1 < first.runs ? full : decay_of(lg, a.desc[u0 + i0 + i].tokens);
      r = fmaf(d.by, r, (d.keep ? r : 0.f) + x[i]);
    }
  }
  *slot = r;
}

// grid (units x row tiles, heads, tiles of d_v).  128 threads of 8 x 8 values: with 256 of 4 x 8 the loads
// from shared memory, three for 16 packed FMAs instead of four for 32, held the warps up for most of the
// time.
constexpr int kOutThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kOutThreads, 3) simt_output_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  __shared__ __align__(16) float as[kStep][kPitch], bs[kStep][kWidePitch];
  __shared__ __align__(16) float ps[kTile][kPitch];  // [key][row]
  pdl_wait();
  const int tiles = a.run / kTile;
  const int64_t unit = blockIdx.x / tiles;
  const RunDesc d = a.desc[unit];
  const int r0 = blockIdx.x % tiles * kTile;
  if (r0 >= d.tokens) return;
  constexpr int R = 8;
  const int hq = blockIdx.y, h = hq / a.group, j0 = blockIdx.z * kWide;
  const int tid = threadIdx.x, ty = tid / 64 * 4 + tid % 32 / 8, tx = tid / 32 % 2 * 8 + tid % 8;  // 4 x 8 lanes a warp
  const float lg = hp.log2g[h];
  // values i0 + hc .. i0 + hc + 3 of tokens base + ht and base + ht + 32, to be transposed into a step
  const int ht = tid / 4, hc = tid % 4 * 4;
  struct Heads {
    float4 x[2];
  };
  auto head = [&](const float* p, int heads, int which, int base, int i0) {
    Heads y;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = base + ht + 32 * u;
      y.x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < d.tokens && i0 + hc < a.pitch)
        y.x[u] = *reinterpret_cast<const float4*>(p + (static_cast<int64_t>(d.row + t) * heads + which) * a.pitch + i0 + hc);
    }
    return y;
  };
  auto put = [&](float* to, int pitch, const Heads& y) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = ht + 32 * u;
      to[(hc + 0) * pitch + t] = y.x[u].x;
      to[(hc + 1) * pitch + t] = y.x[u].y;
      to[(hc + 2) * pitch + t] = y.x[u].z;
      to[(hc + 3) * pitch + t] = y.x[u].w;
    }
  };
  const bool in = j0 + tid < a.d_v;  // a thread's column of a wide step
  Two o[R][4] = {};
  if (!(d.index == 0 && d.pos == 0)) {  // the state before the run, decayed to each row
    const float* w = a.w + (unit * a.kv + h) * a.d_k * a.d_v + j0 + tid;
    Heads qr;
    float wr[kStep];
    auto fetch = [&](int i0) {
      qr = head(a.qf, a.heads, hq, r0, i0);
#pragma unroll
      for (int i = 0; i < kStep; ++i) wr[i] = i0 + i < a.d_k && in ? w[static_cast<int64_t>(i0 + i) * a.d_v] : 0.f;
    };
    fetch(0);
    for (int i0 = 0; i0 < a.d_k; i0 += kStep) {
      put(&as[0][0], kPitch, qr);
#pragma unroll
      for (int i = 0; i < kStep; ++i) bs[i][tid] = wr[i];
      __syncthreads();
      if (i0 + kStep < a.d_k) fetch(i0 + kStep);
      fma_step(o, as, bs, ty, tx);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Two xi = two(decay_pow(lg, r0 + ty * R + i + 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = mul2(o[i][j], xi);
    }
  }
  for (int k0 = 0; k0 <= r0; k0 += kTile) {
    Two sc[R][2] = {};
    Heads qr = head(a.qf, a.heads, hq, r0, 0), kr = head(a.kf, a.kv, h, k0, 0);
    for (int i0 = 0; i0 < a.d_k; i0 += kStep) {
      put(&as[0][0], kPitch, qr);
      put(&bs[0][0], kWidePitch, kr);
      __syncthreads();
      if (i0 + kStep < a.d_k) {
        qr = head(a.qf, a.heads, hq, r0, i0 + kStep);
        kr = head(a.kf, a.kv, h, k0, i0 + kStep);
      }
      fma_step(sc, as, bs, ty, tx);
      __syncthreads();
    }
    float vr[kStep];
    auto fetch = [&](int m0) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int t = k0 + m0 + i;
        vr[i] = t < d.tokens && in
                    ? load_f(a.v, static_cast<int64_t>(d.row + t) * a.stride_v + static_cast<int64_t>(h) * a.d_v + j0 + tid)
                    : 0.f;
      }
    };
    fetch(0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = parts(sc[i + e][j / 2]);
          const int gap = r0 + ty * R + i + e - k0 - tx * 4 - j;
          p[e] = gap >= 0 ? (j % 2 ? x.y : x.x) * decay_pow(lg, gap) : 0.f;
        }
        *reinterpret_cast<float4*>(&ps[tx * 4 + j][ty * R + i]) = make_float4(p[0], p[1], p[2], p[3]);
      }
    for (int m0 = 0; m0 < kTile; m0 += kStep) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) bs[i][tid] = vr[i];
      __syncthreads();
      if (m0 + kStep < kTile) fetch(m0 + kStep);
      fma_step(o, ps + m0, bs, ty, tx);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = r0 + ty * R + i;
    if (t >= d.tokens) continue;
    const float f = a.factor[static_cast<int64_t>(d.row + t) * a.kv + h];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = parts(o[i][j]);
      const int c = j0 + (j / 2) * 64 + tx * 4 + (j % 2) * 2;
      const int64_t at = static_cast<int64_t>(d.row + t) * a.stride_o + static_cast<int64_t>(hq) * a.d_v + c;
      if (c < a.d_v) store_f(a.o, at, x.x * f);
      if (c + 1 < a.d_v) store_f(a.o, at + 1, x.y * f);
    }
  }
}

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t pitch_of(int64_t d_k) { return (d_k + 3) / 4 * 4; }

template <typename T>
cudaError_t launch_typed(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  const int run = run_of(c.d_k, c.d_v);
  const int64_t units = packed_units(c.rows, c.seqs, run), pitch = pitch_of(c.d_k);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(c.ws) + 255) & ~static_cast<uintptr_t>(255));
  auto take = [&](size_t bytes) {
    char* p = ws;
    ws += a256(bytes);
    return p;
  };
  RunDesc* desc = reinterpret_cast<RunDesc*>(take(sizeof(RunDesc) * units));
  float* qf = reinterpret_cast<float*>(take(sizeof(float) * c.rows * c.heads * pitch));
  float* kf = reinterpret_cast<float*>(take(sizeof(float) * c.rows * c.heads_kv * pitch));
  float* factor = reinterpret_cast<float*>(take(sizeof(float) * c.rows * c.heads_kv));
  float* w = reinterpret_cast<float*>(take(sizeof(float) * units * c.heads_kv * c.d_k * c.d_v));
  const SimtPackedArgs<T> a{static_cast<const T*>(c.q), static_cast<const T*>(c.k), static_cast<const T*>(c.v),
                            static_cast<T*>(c.o), c.pool, desc, qf, kf, factor, w, c.cu, units, c.stride_q, c.stride_k,
                            c.stride_v, c.stride_o, run, static_cast<int32_t>(c.heads), static_cast<int32_t>(c.heads_kv),
                            static_cast<int32_t>(c.heads / c.heads_kv), static_cast<int32_t>(c.d_k),
                            static_cast<int32_t>(c.d_v), static_cast<int32_t>(pitch), c.flags};
  const PackedIndex ix{c.cu, c.slot, c.pos, c.rows, static_cast<int32_t>(c.seqs), static_cast<int32_t>(c.slots), run};
  cudaError_t e = launch_packed_plan(ix, desc, PackedRotation{nullptr, nullptr, 0, false}, hp, s);
  if (e != cudaSuccess) return e;
  const unsigned u = static_cast<unsigned>(units), kv = static_cast<unsigned>(c.heads_kv);
  const unsigned tk = static_cast<unsigned>((c.d_k + kTile - 1) / kTile), tv = static_cast<unsigned>((c.d_v + kWide - 1) / kWide);
  const unsigned nb = static_cast<unsigned>((c.d_k * c.d_v + kThreads - 1) / kThreads);
  const dim3 block(kThreads);
  e = launch_dependent(simt_rotate_kernel<T>, dim3(u, static_cast<unsigned>(run / kTokens)), block, 0, s, a, hp);
  if (e == cudaSuccess) e = launch_dependent(simt_state_kernel<T>, dim3(u, kv, tk * tv), block, 0, s, a, hp);
  if (e == cudaSuccess)
    e = launch_dependent(simt_scan_kernel<T>, dim3(nb, kv, static_cast<unsigned>(c.seqs)), block, 0, s, a, hp);
  if (e == cudaSuccess)
    e = launch_dependent(simt_output_kernel<T>, dim3(u * (run / kTile), static_cast<unsigned>(c.heads), tv),
                         dim3(kOutThreads), 0, s, a, hp);
  return e;
}

}  // namespace

size_t packed_simt_workspace_bytes(int64_t rows, int64_t seqs, int64_t heads, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  const size_t units = static_cast<size_t>(packed_units(rows, seqs, run_of(d_k, d_v))), r = static_cast<size_t>(rows);
  const size_t pitch = static_cast<size_t>(pitch_of(d_k)), hq = static_cast<size_t>(heads), hk = static_cast<size_t>(heads_kv);
  return 256 + a256(sizeof(RunDesc) * units) + a256(sizeof(float) * r * hq * pitch) + a256(sizeof(float) * r * hk * pitch) +
         a256(sizeof(float) * r * hk) + a256(sizeof(float) * units * hk * static_cast<size_t>(d_k * d_v));
}

cudaError_t launch_packed_simt(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  if (c.dtype == RETNET_F32) return launch_typed<float>(c, hp, s);
  return launch_typed<__nv_bfloat16>(c, hp, s);
}

}  // namespace retnet
