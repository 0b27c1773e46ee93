// step_slots.cu -- one recurrent token for each of many sequences whose states live in a pool:
//   S = pool[slot_r] (zeros at position 0),  S <- gamma S + k'^T v,  o_g = (q'_g S) f,
// k', q' rotated by the row's own position, g over the query heads that share the key/value head, f
// the row factor ("阅读笔记：RetNet" §2.2, §三.3).
//
// Bound by HBM: each named state is read once and written once, the rest is a few KB a row.  A CTA
// owns (row, key/value head, kCols columns of d_v): the lanes of a warp cover the columns with
// 16-byte accesses and the warps split the d_k rows, so a state is streamed in whole 128-byte (32
// columns) or 512-byte (128 columns) row segments.  The first kBatch state rows of every thread are
// loaded before the rotation is computed and the row's slot is checked against the others', so that
// latency is paid once.  62 rows of 16 states of 256 x 512 in 146 us: 5.9 TB/s, 90 % of the copy rate.
#include "launch.h"
#include "pdl.cuh"

namespace retnet {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;  // state rows of a thread in flight

__device__ unsigned int g_step_errors = 0;

template <typename T>
struct StepSlotsArgs {
  const T* q;
  const T* k;
  const T* v;
  T* o;
  float* pool;
  const int32_t* slots;
  const int64_t* pos;
  int64_t stride_q, stride_k, stride_v, stride_o;
  int32_t rows, n_slots, kv, group, d_k, d_v;
  int32_t width;  // columns of a CTA, at most VEC * LANES: d_v in equal parts
  uint32_t flags;
};

// VEC: columns of a lane (4, or 2 or 1 where d_v allows no wider access; 2 instead of 1 took 37 rows of
// 4 states of 100 x 130 from 10.3 to 8.2 us).  LANES: lanes that cover the
// CTA's columns.  G: query heads of one pass over the state (the group, rounded up; a
// larger group takes further passes that only read).
template <typename T, int VEC, int LANES, int G>
__global__ void __launch_bounds__(kThreads) step_slots_kernel(StepSlotsArgs<T> a, HeadParams hp) {
  constexpr int kCols = VEC * LANES;
  constexpr int kRowsPerPass = kThreads / LANES;  // state rows the CTA touches at once
  extern __shared__ float sm[];
  const int dk = a.d_k, dv = a.d_v, tid = threadIdx.x;
  float* ks = sm;                         // [dk] rotated k
  float* qs = ks + dk;                    // [G][dk] rotated q of this pass
  float* red = qs + G * dk;               // [warps][G][kCols] partial q S
  __shared__ float factor;
  const int row = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * a.width;
  const int c1 = c0 + a.width < dv ? c0 + a.width : dv;  // the CTA's columns end here
  pdl_wait();
  const int32_t slot = a.slots[row];
  const int64_t pos = a.pos ? a.pos[row] : 0;
  if (slot < 0) return;  // padding
  const bool bad_row = slot >= a.n_slots || pos < 0 || pos > RETNET_MAX_POSITION;
  const int lr = tid / LANES, col = c0 + (tid % LANES) * VEC;
  const bool live = col < c1;
  const bool fresh = pos == 0;
  float* S = a.pool + (static_cast<int64_t>(bad_row ? 0 : slot) * a.kv + h) * dk * dv + col;

  float st[kBatch][VEC];
  auto load_batch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kRowsPerPass;
#pragma unroll
      for (int c = 0; c < VEC; ++c) st[u][c] = 0.f;
      if (live && i < dk) {
        if constexpr (VEC == 4) {
          const float4 x = __ldcs(reinterpret_cast<const float4*>(S + static_cast<int64_t>(i) * dv));
          st[u][0] = x.x; st[u][1] = x.y; st[u][2] = x.z; st[u][3] = x.w;
        } else if constexpr (VEC == 2) {
          const float2 x = __ldcs(reinterpret_cast<const float2*>(S + static_cast<int64_t>(i) * dv));
          st[u][0] = x.x; st[u][1] = x.y;
        } else {
          st[u][0] = __ldcs(S + static_cast<int64_t>(i) * dv);
        }
      }
    }
  };
  if (!fresh && !bad_row) load_batch(lr);

  // A slot that an earlier row names is that row's.
  int dup = 0;
  for (int j = tid; j < row; j += kThreads) dup |= a.slots[j] == slot;
  const float gamma = hp.gamma[h];
  const bool xpos = (a.flags & RETNET_F_XPOS) != 0;
  const T* kp = a.k + row * a.stride_k + static_cast<int64_t>(h) * dk;
  const T* qp = a.q + row * a.stride_q + static_cast<int64_t>(h) * a.group * dk;
  auto rotate_into = [&](float* out, const T* in, int j, float s, float c) {
    const float x0 = load_f(in, 2 * j), x1 = load_f(in, 2 * j + 1);
    out[2 * j] = x0 * c - x1 * s;
    out[2 * j + 1] = x0 * s + x1 * c;
  };
  auto load_q = [&](int g0) {
    for (int j = tid; j < dk / 2; j += kThreads) {
      float s = 0.f, c = 1.f;
      if (xpos) position_sincos(pos, hp.theta[j], &s, &c);
      if (g0 == 0) rotate_into(ks, kp, j, s, c);
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (g0 + g < a.group) rotate_into(qs + g * dk, qp + static_cast<int64_t>(g0 + g) * dk, j, s, c);
    }
    if ((dk & 1) && tid == 0) {
      if (g0 == 0) ks[dk - 1] = load_f(kp, dk - 1);
      for (int g = 0; g < G && g0 + g < a.group; ++g) qs[g * dk + dk - 1] = load_f(qp, static_cast<int64_t>(g0 + g) * dk + dk - 1);
    }
  };
  load_q(0);
  if (tid / 32 == kThreads / 32 - 1) {  // fp64 work of one warp, beside the others' rotations
    const float f = row_factor(gamma, dk, bad_row ? 0 : pos, a.flags);
    if (tid % 32 == 0) factor = f;
  }
  float vv[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c)
    vv[c] = col + c < c1 ? load_f(a.v + row * a.stride_v + static_cast<int64_t>(h) * dv, col + c) : 0.f;
  if (__syncthreads_or(dup | static_cast<int>(bad_row))) {
    if (tid == 0 && h == 0 && blockIdx.z == 0) atomicAdd(&g_step_errors, 1u);
    return;
  }
  const float f = factor;

  for (int g0 = 0; g0 < a.group; g0 += G) {
    if (g0) {
      __syncthreads();
      load_q(g0);
      __syncthreads();
    }
    float acc[G][VEC];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int c = 0; c < VEC; ++c) acc[g][c] = 0.f;
    for (int i0 = lr; i0 < dk; i0 += kBatch * kRowsPerPass) {
      // the first batch is in registers already; a further pass reads what this thread wrote
      if (i0 != lr || g0) {
        if (!fresh || g0) load_batch(i0);
      }
      if (fresh && !g0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int c = 0; c < VEC; ++c) st[u][c] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kRowsPerPass;
        if (i >= dk) break;
        if (g0 == 0) {
          const float kr = ks[i];
#pragma unroll
          for (int c = 0; c < VEC; ++c) st[u][c] = fmaf(gamma, st[u][c], kr * vv[c]);
          if (live) {
            if constexpr (VEC == 4) {
              __stcs(reinterpret_cast<float4*>(S + static_cast<int64_t>(i) * dv),
                     make_float4(st[u][0], st[u][1], st[u][2], st[u][3]));
            } else if constexpr (VEC == 2) {
              __stcs(reinterpret_cast<float2*>(S + static_cast<int64_t>(i) * dv), make_float2(st[u][0], st[u][1]));
            } else {
              __stcs(S + static_cast<int64_t>(i) * dv, st[u][0]);
            }
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float qr = qs[g * dk + i];
#pragma unroll
          for (int c = 0; c < VEC; ++c) acc[g][c] = fmaf(qr, st[u][c], acc[g][c]);
        }
      }
    }
    // Partial sums of the CTA's row groups: lanes of a warp on the same columns first, then warps.
#pragma unroll
    for (int off = LANES; off < 32; off <<= 1)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[g][c] += __shfl_xor_sync(0xffffffffu, acc[g][c], off);
    const int warp = tid / 32, lane = tid % 32;
    if (lane < LANES) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < VEC; ++c) red[(warp * G + g) * kCols + lane * VEC + c] = acc[g][c];
    }
    __syncthreads();
    for (int e = tid; e < G * kCols; e += kThreads) {
      const int g = e / kCols, c = e % kCols;
      if (g0 + g < a.group && c0 + c < c1) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += red[(w * G + g) * kCols + c];
        store_f(a.o + row * a.stride_o, (static_cast<int64_t>(h) * a.group + g0 + g) * dv + c0 + c, s * f);
      }
    }
  }
}

template <typename T, int VEC, int LANES, int G>
cudaError_t launch_g(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  StepSlotsArgs<T> a{static_cast<const T*>(c.q), static_cast<const T*>(c.k), static_cast<const T*>(c.v),
                     static_cast<T*>(c.o), c.pool, c.slot, c.pos, c.stride_q, c.stride_k, c.stride_v, c.stride_o,
                     static_cast<int32_t>(c.rows), static_cast<int32_t>(c.slots), static_cast<int32_t>(c.heads_kv),
                     static_cast<int32_t>(c.heads / c.heads_kv), static_cast<int32_t>(c.d_k),
                     static_cast<int32_t>(c.d_v), 0, c.flags};
  constexpr int kCols = VEC * LANES;
  const int64_t parts = (c.d_v + kCols - 1) / kCols;
  a.width = static_cast<int32_t>(((c.d_v + parts - 1) / parts + VEC - 1) / VEC * VEC);
  // at most 4 * (9 * 512 + 8 * 8 * 128) = 51 KB
  const size_t smem = sizeof(float) * static_cast<size_t>((1 + G) * c.d_k + (kThreads / 32) * G * kCols);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(step_slots_kernel<T, VEC, LANES, G>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(c.rows), static_cast<unsigned>(c.heads_kv),
                  static_cast<unsigned>(parts));
  return launch_dependent(step_slots_kernel<T, VEC, LANES, G>, grid, dim3(kThreads), smem, s, a, hp);
}

template <typename T, int VEC, int LANES>
cudaError_t launch_lanes(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  const int64_t group = c.heads / c.heads_kv;
  if (group == 1) return launch_g<T, VEC, LANES, 1>(c, hp, s);
  if (group <= 2) return launch_g<T, VEC, LANES, 2>(c, hp, s);
  if (group <= 4) return launch_g<T, VEC, LANES, 4>(c, hp, s);
  return launch_g<T, VEC, LANES, 8>(c, hp, s);
}

template <typename T>
cudaError_t launch_typed(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  if (c.d_v % 2) return launch_lanes<T, 1, 32>(c, hp, s);
  if (c.d_v % 4) return launch_lanes<T, 2, 32>(c, hp, s);
  // 128-column CTAs read 512-byte segments; where they are fewer than 128, four times as many 32-column ones
  // (bf16, states of 128 x 128: 24 CTAs or 96 took 5.2 us against 4.0 from L2, 96 or 384 10.2 against 8.2
  // from HBM; 128 or 512 5.4 against 6.7 from L2, 512 or 2048 11.3 against 15.2)
  if (c.rows * c.heads_kv * ((c.d_v + 127) / 128) < 128) return launch_lanes<T, 4, 8>(c, hp, s);
  return launch_lanes<T, 4, 32>(c, hp, s);
}

}  // namespace

cudaError_t launch_step_slots(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  if (c.dtype == RETNET_F32) return launch_typed<float>(c, hp, s);
  return launch_typed<__nv_bfloat16>(c, hp, s);
}

cudaError_t step_index_errors(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_step_errors, sizeof(unsigned int));
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_step_errors, &zero, sizeof(zero));
  return e;
}

}  // namespace retnet
