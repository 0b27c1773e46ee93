// packed_simt.cu -- packed retention in fp32 on the CUDA cores: fp32 inputs (whose tolerance rules
// out 16-bit tensor-core operands) and every width, stride and decay that the tensor-core kernels do
// not take.  "阅读笔记：RetNet" §2.4 with the sequence cut into runs (packed.cuh):
//   state   W_u = sum_t gamma^(end-1-t) k'_t^T v_t of every run, all runs at once;
//   scan    a sequence's runs in order: R_u = the state before run u (written over W_u),
//           R <- gamma^len R + W; the last R goes to the pool;
//   output  o_n = f_n [ sum_{m in run, m<=n} gamma^(n-m) (q'_n . k'_m) v_m + gamma^(n-start+1) q'_n R_u ].
// Bound by the fp32 FMA rate: 64 x 64 tiles, 4 x 4 values a thread, operands through shared memory.
// The rotations (fp64 angles) come from a table that a first kernel writes once a token, instead of
// once a token, tile and head.
#include "packed.cuh"

namespace retnet {
namespace {

constexpr int kRun = 256;     // tokens of a run: the state of a run (d_k d_v) against 256 (d_k + d_v) of its inputs
constexpr int kTile = 64;
constexpr int kStep = 16;     // depth of one shared-memory step
constexpr int kThreads = 256;
constexpr int kPitch = kTile + 4;

template <typename T>
struct SimtPackedArgs {
  const T* q;
  const T* k;
  const T* v;
  T* o;
  float* pool;
  const RunDesc* desc;
  const float2* rot;  // [rows][d_k / 2] (cos, sin) or nullptr
  float* w;           // [units][heads_kv][d_k][d_v]
  const int32_t* cu;
  int64_t stride_q, stride_k, stride_v, stride_o;
  int64_t units;
  int32_t kv, group, d_k, d_v;
  uint32_t flags;
};

__global__ void __launch_bounds__(kThreads) rotation_kernel(const RunDesc* __restrict__ desc, float2* __restrict__ rot,
                                                            int half, HeadParams hp) {
  const RunDesc d = desc[blockIdx.x];
  const int64_t n = static_cast<int64_t>(d.tokens) * half;
  for (int64_t e = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.y) * kThreads) {
    const int t = static_cast<int>(e / half), j = static_cast<int>(e % half);
    float s, c;
    position_sincos(d.pos + t, hp.theta[j], &s, &c);
    rot[static_cast<int64_t>(d.row + t) * half + j] = make_float2(c, s);
  }
}

// Element i of a head vector of token row (rotated where rot is given).
template <typename T>
__device__ __forceinline__ float rotated(const T* head, const float2* rot_row, int i, int d_k) {
  const float x = load_f(head, i);
  if (!rot_row || (i ^ 1) >= d_k) return x;
  const float y = load_f(head, i ^ 1);
  const float2 cs = rot_row[i / 2];
  return (i & 1) ? fmaf(y, cs.y, x * cs.x) : fmaf(-y, cs.y, x * cs.x);
}

// acc[i][j] += sum_r a[r][ty * 4 + i] * b[r][tx * 4 + j]
__device__ __forceinline__ void fma_step(float (&acc)[4][4], const float (*a)[kPitch], const float (*b)[kPitch], int ty,
                                         int tx) {
#pragma unroll
  for (int r = 0; r < kStep; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(&a[r][ty * 4]);
    const float4 y = *reinterpret_cast<const float4*>(&b[r][tx * 4]);
    const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xa[i], ya[j], acc[i][j]);
  }
}

// grid (units, heads_kv, tiles of d_k x tiles of d_v)
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_state_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  __shared__ __align__(16) float ks[kStep][kPitch], vs[kStep][kPitch];
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int h = blockIdx.y, tv = (a.d_v + kTile - 1) / kTile;
  const int i0 = (blockIdx.z / tv) * kTile, j0 = (blockIdx.z % tv) * kTile;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const float lg = hp.log2g[h];
  float acc[4][4] = {};
  for (int t0 = 0; t0 < d.tokens; t0 += kStep) {
    for (int e = tid; e < kStep * kTile; e += kThreads) {
      const int r = e / kTile, c = e % kTile, t = t0 + r;
      float x = 0.f, y = 0.f;
      if (t < d.tokens) {
        const int64_t row = d.row + t;
        if (i0 + c < a.d_k)
          x = rotated(a.k + row * a.stride_k + static_cast<int64_t>(h) * a.d_k,
                      a.rot ? a.rot + row * (a.d_k / 2) : nullptr, i0 + c, a.d_k) *
              decay_pow(lg, d.tokens - 1 - t);
        if (j0 + c < a.d_v) y = load_f(a.v, row * a.stride_v + static_cast<int64_t>(h) * a.d_v + j0 + c);
      }
      ks[r][c] = x;
      vs[r][c] = y;
    }
    __syncthreads();
    fma_step(acc, ks, vs, ty, tx);
    __syncthreads();
  }
  float* w = a.w + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * a.d_k * a.d_v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + ty * 4 + i < a.d_k && j0 + tx * 4 + j < a.d_v)
        w[static_cast<int64_t>(i0 + ty * 4 + i) * a.d_v + j0 + tx * 4 + j] = acc[i][j];
}

// grid (blocks of d_k d_v, heads_kv, seqs)
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_scan_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  const int s = blockIdx.z, h = blockIdx.y;
  const int64_t n = static_cast<int64_t>(a.d_k) * a.d_v;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t u0 = a.cu[s] / kRun + s;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc first = a.desc[u0];
  if (first.tokens == 0 || first.seq != s || e >= n) return;
  float* slot = a.pool + (static_cast<int64_t>(first.slot) * a.kv + h) * n + e;
  float r = first.pos > 0 ? *slot : 0.f;
  const float lg = hp.log2g[h], full = decay_pow(lg, kRun);
  for (int i = 0; i < first.runs; ++i) {
    float* w = a.w + ((u0 + i) * a.kv + h) * n + e;
    const float x = *w;
    *w = r;
    r = fmaf(i + 1 < first.runs ? full : decay_pow(lg, a.desc[u0 + i].tokens), r, x);
  }
  *slot = r;
}

// grid (units x row tiles, heads, tiles of d_v)
template <typename T>
__global__ void __launch_bounds__(kThreads) simt_output_kernel(SimtPackedArgs<T> a, HeadParams hp) {
  __shared__ __align__(16) float as[kStep][kPitch], bs[kStep][kPitch];
  __shared__ __align__(16) float ps[kTile][kPitch];  // [key][row]
  constexpr int kTiles = kRun / kTile;
  const RunDesc d = a.desc[blockIdx.x / kTiles];
  const int ti = blockIdx.x % kTiles, r0 = ti * kTile;
  if (r0 >= d.tokens) return;
  const int hq = blockIdx.y, h = hq / a.group, j0 = blockIdx.z * kTile;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const float lg = hp.log2g[h];
  const int half = a.d_k / 2;
  // as[r][c] <- element i0 + r of the q (k) vector of token base + c
  auto load_heads = [&](float (*to)[kPitch], const T* p, int64_t stride, int head, int base, int i0) {
    for (int e = tid; e < kStep * kTile; e += kThreads) {
      const int r = e % kStep, c = e / kStep, t = base + c, i = i0 + r;
      float x = 0.f;
      if (t < d.tokens && i < a.d_k) {
        const int64_t row = d.row + t;
        x = rotated(p + row * stride + static_cast<int64_t>(head) * a.d_k, a.rot ? a.rot + row * half : nullptr, i, a.d_k);
      }
      to[r][c] = x;
    }
  };
  float acc[4][4] = {};
  // the state before the run, decayed to each row
  const bool from_zero = d.index == 0 && d.pos == 0;
  if (!from_zero) {
    const float* w = a.w + (static_cast<int64_t>(blockIdx.x / kTiles) * a.kv + h) * a.d_k * a.d_v;
    for (int i0 = 0; i0 < a.d_k; i0 += kStep) {
      load_heads(as, a.q, a.stride_q, hq, r0, i0);
      for (int e = tid; e < kStep * kTile; e += kThreads) {
        const int r = e / kTile, c = e % kTile;
        bs[r][c] = i0 + r < a.d_k && j0 + c < a.d_v ? w[static_cast<int64_t>(i0 + r) * a.d_v + j0 + c] : 0.f;
      }
      __syncthreads();
      fma_step(acc, as, bs, ty, tx);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xi = decay_pow(lg, r0 + ty * 4 + i + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] *= xi;
    }
  }
  for (int k0 = 0; k0 <= r0; k0 += kTile) {
    float sc[4][4] = {};
    for (int i0 = 0; i0 < a.d_k; i0 += kStep) {
      load_heads(as, a.q, a.stride_q, hq, r0, i0);
      load_heads(bs, a.k, a.stride_k, h, k0, i0);
      __syncthreads();
      fma_step(sc, as, bs, ty, tx);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gap = r0 + ty * 4 + i - k0 - tx * 4 - j;
        ps[tx * 4 + j][ty * 4 + i] = gap >= 0 ? sc[i][j] * decay_pow(lg, gap) : 0.f;
      }
    __syncthreads();
    for (int m0 = 0; m0 < kTile; m0 += kStep) {
      for (int e = tid; e < kStep * kTile; e += kThreads) {
        const int r = e / kTile, c = e % kTile, t = k0 + m0 + r;
        bs[r][c] = t < d.tokens && j0 + c < a.d_v
                       ? load_f(a.v, (d.row + t) * a.stride_v + static_cast<int64_t>(h) * a.d_v + j0 + c)
                       : 0.f;
      }
      __syncthreads();
      fma_step(acc, ps + m0, bs, ty, tx);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = r0 + ty * 4 + i;
    if (t >= d.tokens) continue;
    const float f = row_factor(hp.gamma[h], a.d_k, d.pos + t, a.flags);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j0 + tx * 4 + j < a.d_v)
        store_f(a.o, (d.row + t) * a.stride_o + static_cast<int64_t>(hq) * a.d_v + j0 + tx * 4 + j, acc[i][j] * f);
  }
}

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename T>
cudaError_t launch_typed(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  const int64_t units = packed_units(c.rows, c.seqs, kRun);
  char* ws = static_cast<char*>(c.ws);
  RunDesc* desc = reinterpret_cast<RunDesc*>(ws);
  ws += a256(sizeof(RunDesc) * units);
  float2* rot = reinterpret_cast<float2*>(ws);
  ws += a256(sizeof(float2) * c.rows * (c.d_k / 2));
  const bool xpos = (c.flags & RETNET_F_XPOS) != 0;
  SimtPackedArgs<T> a{static_cast<const T*>(c.q), static_cast<const T*>(c.k), static_cast<const T*>(c.v),
                      static_cast<T*>(c.o), c.pool, desc, xpos ? rot : nullptr, reinterpret_cast<float*>(ws), c.cu,
                      c.stride_q, c.stride_k, c.stride_v, c.stride_o, units,
                      static_cast<int32_t>(c.heads_kv), static_cast<int32_t>(c.heads / c.heads_kv),
                      static_cast<int32_t>(c.d_k), static_cast<int32_t>(c.d_v), c.flags};
  const PackedIndex ix{c.cu, c.slot, c.pos, c.rows, static_cast<int32_t>(c.seqs), static_cast<int32_t>(c.slots), kRun};
  cudaError_t e = launch_packed_plan(ix, desc, PackedRotation{nullptr, nullptr, 0, false}, hp, s);
  if (e != cudaSuccess) return e;
  const unsigned u = static_cast<unsigned>(units), kv = static_cast<unsigned>(c.heads_kv);
  if (xpos) rotation_kernel<<<dim3(u, 8), kThreads, 0, s>>>(desc, rot, static_cast<int>(c.d_k / 2), hp);
  const unsigned tk = static_cast<unsigned>((c.d_k + kTile - 1) / kTile), tv = static_cast<unsigned>((c.d_v + kTile - 1) / kTile);
  simt_state_kernel<T><<<dim3(u, kv, tk * tv), kThreads, 0, s>>>(a, hp);
  const unsigned nb = static_cast<unsigned>((c.d_k * c.d_v + kThreads - 1) / kThreads);
  simt_scan_kernel<T><<<dim3(nb, kv, static_cast<unsigned>(c.seqs)), kThreads, 0, s>>>(a, hp);
  simt_output_kernel<T><<<dim3(u * (kRun / kTile), static_cast<unsigned>(c.heads), tv), kThreads, 0, s>>>(a, hp);
  return cudaGetLastError();
}

}  // namespace

size_t packed_simt_workspace_bytes(int64_t rows, int64_t seqs, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  const int64_t units = packed_units(rows, seqs, kRun);
  return a256(sizeof(RunDesc) * units) + a256(sizeof(float2) * rows * (d_k / 2)) +
         sizeof(float) * static_cast<size_t>(units * heads_kv * d_k * d_v);
}

cudaError_t launch_packed_simt(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  if (c.dtype == RETNET_F32) return launch_typed<float>(c, hp, s);
  return launch_typed<__nv_bfloat16>(c, hp, s);
}

}  // namespace retnet
