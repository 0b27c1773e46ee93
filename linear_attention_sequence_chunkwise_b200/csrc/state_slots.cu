// state_slots.cu -- moving states between the slots of a pool: pool[dst_i] <- old pool[src_i], or
// zeros where src_i < 0, for all pairs at once ("old": every source is read as it was before the
// call, so a permutation, a beam's reorder in place, is one call).  Forking is one source with many
// destinations, compacting moves live slots into holes, freeing clears.
//
// Bound by HBM: each pair reads and writes one slot.  "All sources before any destination" needs no
// second copy of the pool when one CTA moves the SAME columns of every pair: a CTA owns a tile of
// `cols` columns (16 bytes each) of the slot, reads it for all pairs, then writes it for all pairs;
// tiles do not touch one another.  The tile is staged in shared memory by asynchronous copies, 64 KB at
// once, two CTAs an SM, one storing while the other loads.  (Streaming through registers where no source
// is a destination was no faster: 30 slots of 8 MB in 97 us against 91.)  61 slots of 8 MB, sources
// shared, in 147 us: 7.0 TB/s of reads and writes, part of them from L2.
#include "launch.h"
#include "pdl.cuh"
#include "sm100_ptx.cuh"

namespace retnet {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = RETNET_MAX_SLOT_PAIRS;
constexpr int kStageBytes = 64 * 1024;

__device__ unsigned int g_slot_errors = 0;

template <typename T>
__device__ __forceinline__ T zero_of();
template <>
__device__ __forceinline__ float zero_of<float>() { return 0.f; }
template <>
__device__ __forceinline__ float4 zero_of<float4>() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// T: float4, or float where a slot is no multiple of four floats.  n_cols, cols in units of T; cols a
// power of two.
template <typename T>
__global__ void __launch_bounds__(kThreads) slots_copy_kernel(T* pool, int32_t n_slots, int64_t n_cols, int log_cols,
                                                              const int32_t* src, const int32_t* dst, int n) {
  extern __shared__ __align__(16) unsigned char stage_raw[];
  T* stage = reinterpret_cast<T*>(stage_raw);
  __shared__ int32_t raw_dst[kMaxPairs], sp[kMaxPairs], dp[kMaxPairs];
  __shared__ int count;
  const int tid = threadIdx.x;
  if (tid == 0) count = 0;
  pdl_wait();
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
  // element e of the tile: column e % cols of pair e / cols
  const int cols = 1 << log_cols, total = m << log_cols;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * cols; c0 < n_cols; c0 += static_cast<int64_t>(gridDim.x) * cols) {
    const int w = static_cast<int>(n_cols - c0 < cols ? n_cols - c0 : cols);
    T* at = pool + c0;
    for (int e = tid; e < total; e += kThreads) {
      const int c = e & (cols - 1);
      const int32_t s = sp[e >> log_cols];
      if (c >= w) continue;
      if (s < 0) {
        stage[e] = zero_of<T>();
      } else if constexpr (sizeof(T) == 16) {
        sm100::cp_async16(sm100::smem_addr(stage + e), at + static_cast<int64_t>(s) * n_cols + c, true);
      } else {
        stage[e] = at[static_cast<int64_t>(s) * n_cols + c];
      }
    }
    sm100::cp_async_wait_all();
    __syncthreads();
    for (int e = tid; e < total; e += kThreads) {
      const int c = e & (cols - 1);
      if (c < w) at[static_cast<int64_t>(dp[e >> log_cols]) * n_cols + c] = stage[e];
    }
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_typed(float* pool, int64_t slots, int64_t slot_floats, const int32_t* src, const int32_t* dst,
                         int64_t n, cudaStream_t s) {
  const int64_t n_cols = slot_floats * static_cast<int64_t>(sizeof(float)) / static_cast<int64_t>(sizeof(T));
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(slots_copy_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
  if (e != cudaSuccess) return e;
  // The widest power of two that the stage has room for (n <= 1024: at least 64 bytes), but no wider
  // than leaves two tiles an SM: four pairs of 512 KB slots took 8 us in 32 tiles.
  int log_cols = 0;
  while (static_cast<size_t>(2 << log_cols) * sizeof(T) * n <= kStageBytes && (n_cols >> (log_cols + 1)) >= 2 * sms) ++log_cols;
  const int64_t tiles = (n_cols + (1 << log_cols) - 1) >> log_cols;
  const int64_t blocks = tiles < 2 * sms ? tiles : 2 * sms;
  return launch_dependent(slots_copy_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                          (static_cast<size_t>(n) << log_cols) * sizeof(T), s, reinterpret_cast<T*>(pool),
                          static_cast<int32_t>(slots), n_cols, log_cols, src, dst, static_cast<int>(n));
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
