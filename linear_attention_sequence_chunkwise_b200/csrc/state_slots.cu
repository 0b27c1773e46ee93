// state_slots.cu -- moving states between the slots of a pool: pool[dst_i] <- old pool[src_i], or
// zeros where src_i < 0, for all pairs at once ("old": every source is read as it was before the
// call, so a permutation, a beam's reorder in place, is one call).  Forking is one source with many
// destinations, compacting moves live slots into holes, freeing clears.
//
// Bound by HBM: each pair reads and writes one slot.  "All sources before any destination" needs no
// second copy of the pool when one CTA moves the SAME columns of every pair: a CTA owns a tile of
// `cols` floats of the slot, reads it for all pairs, then writes it for all pairs; tiles do not
// touch one another.  Only where some pair's source is another pair's destination does the read have
// to be complete before the first write (the tile is staged in shared memory, kStageBytes for all
// pairs); otherwise the tile streams through registers.
#include "launch.h"

namespace retnet {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = RETNET_MAX_SLOT_PAIRS;
constexpr int kStageBytes = 64 * 1024;  // three CTAs an SM
constexpr int kUnroll = 8;

__device__ unsigned int g_slot_errors = 0;

template <typename T>
__device__ __forceinline__ T zero_of();
template <>
__device__ __forceinline__ float zero_of<float>() { return 0.f; }
template <>
__device__ __forceinline__ float4 zero_of<float4>() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// T: float4, or float where a slot is no multiple of four floats.  n_cols, cols in units of T.
template <typename T>
__global__ void __launch_bounds__(kThreads) slots_copy_kernel(T* pool, int32_t n_slots, int64_t n_cols, int cols,
                                                              const int32_t* __restrict__ src,
                                                              const int32_t* __restrict__ dst, int n) {
  extern __shared__ __align__(16) unsigned char stage_raw[];
  T* stage = reinterpret_cast<T*>(stage_raw);
  __shared__ int32_t raw_dst[kMaxPairs], sp[kMaxPairs], dp[kMaxPairs];
  __shared__ int count;
  const int tid = threadIdx.x;
  if (tid == 0) count = 0;
  for (int i = tid; i < n; i += kThreads) raw_dst[i] = dst[i];
  __syncthreads();
  // The pairs to move, in any order (their destinations differ).  A pair with dst < 0 is padding;
  // one whose slots are out of range, or whose destination an earlier pair has, is refused.
  for (int i = tid; i < n; i += kThreads) {
    const int32_t d = raw_dst[i], s = src[i];
    if (d < 0) continue;
    bool bad = d >= n_slots || s >= n_slots;
    for (int j = 0; j < i; ++j) bad |= raw_dst[j] == d;
    if (bad) {
      if (blockIdx.x == 0) atomicAdd(&g_slot_errors, 1u);
      continue;
    }
    if (s == d) continue;
    const int at = atomicAdd(&count, 1);
    sp[at] = s;
    dp[at] = d;
  }
  __syncthreads();
  const int m = count;
  int mine = 0;
  for (int i = tid; i < m; i += kThreads) {
    const int32_t s = sp[i];
    if (s < 0) continue;
    for (int j = 0; j < m; ++j) mine |= dp[j] == s;
  }
  const bool hazard = __syncthreads_or(mine) != 0;

  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * cols; c0 < n_cols; c0 += static_cast<int64_t>(gridDim.x) * cols) {
    const int w = static_cast<int>(n_cols - c0 < cols ? n_cols - c0 : cols);
    const int total = m * w;
    for (int e0 = tid; e0 < total; e0 += kThreads * kUnroll) {
      T x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = e0 + u * kThreads;
        x[u] = zero_of<T>();
        if (e < total) {
          const int i = e / w;
          const int32_t s = sp[i];
          if (s >= 0) x[u] = pool[static_cast<int64_t>(s) * n_cols + c0 + (e - i * w)];
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = e0 + u * kThreads;
        if (e < total) {
          if (hazard) {
            stage[e] = x[u];
          } else {
            const int i = e / w;
            pool[static_cast<int64_t>(dp[i]) * n_cols + c0 + (e - i * w)] = x[u];
          }
        }
      }
    }
    if (hazard) {
      __syncthreads();
      for (int e = tid; e < total; e += kThreads) {
        const int i = e / w;
        pool[static_cast<int64_t>(dp[i]) * n_cols + c0 + (e - i * w)] = stage[e];
      }
      __syncthreads();
    }
  }
}

template <typename T>
cudaError_t launch_typed(float* pool, int64_t slots, int64_t slot_floats, const int32_t* src, const int32_t* dst,
                         int64_t n, cudaStream_t s) {
  const int64_t n_cols = slot_floats * static_cast<int64_t>(sizeof(float)) / static_cast<int64_t>(sizeof(T));
  int cols = kStageBytes / static_cast<int>(sizeof(T)) / static_cast<int>(n);
  if (cols >= 32) cols -= cols % 32;
  if (cols > n_cols) cols = static_cast<int>(n_cols);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(slots_copy_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (n_cols + cols - 1) / cols;
  const int64_t blocks = tiles < 2 * sms ? tiles : 2 * sms;
  slots_copy_kernel<T><<<static_cast<unsigned>(blocks), kThreads, static_cast<size_t>(cols) * n * sizeof(T), s>>>(
      reinterpret_cast<T*>(pool), static_cast<int32_t>(slots), n_cols, cols, src, dst, static_cast<int>(n));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_slots_copy(float* pool, int64_t slots, int64_t slot_floats, const int32_t* src, const int32_t* dst,
                              int64_t n, cudaStream_t s) {
  if (slot_floats % 4 == 0) return launch_typed<float4>(pool, slots, slot_floats, src, dst, n, s);
  return launch_typed<float>(pool, slots, slot_floats, src, dst, n, s);
}

cudaError_t slots_index_errors(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_slot_errors, sizeof(unsigned int));
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_slot_errors, &zero, sizeof(zero));
  return e;
}

}  // namespace retnet
