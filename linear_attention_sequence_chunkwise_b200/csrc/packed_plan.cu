// packed_plan.cu -- the parts of packed retention that both kernel families use: the run descriptors
// (packed.cuh), written on the device because the lengths live there, and the count of sequences
// that the device refused.
#include "packed.cuh"
#include "pdl.cuh"

namespace retnet {
namespace {

constexpr int kThreads = 512;

__device__ unsigned int g_packed_errors = 0;

// Rotation of pair j by position p, into its places: row[0] its cosine, row[4] its sine.
__device__ __forceinline__ void turn(float* row, const PackedRotation& rot, int64_t p, int j, const HeadParams& hp) {
  float s = 0.f, c = 1.f;
  if (rot.xpos) position_sincos(p, hp.theta[j], &s, &c);
  row[0] = c;
  row[4] = s;
}

// One CTA a unit.  The sequence of a unit is the last one whose first unit is not behind it.  A call
// whose cu_seqlens is out of order or leaves the rows has no runs; a sequence is refused (no run)
// when its slot is out of range or an earlier sequence with tokens has it, or its position is
// out of range; one with slot < 0 or no tokens has none either.  Bound by the latency of its few
// dependent steps: the arrays of up to kThreads sequences are fetched at once and the rest is done
// from shared memory.
__global__ void __launch_bounds__(kThreads) plan_kernel(PackedIndex ix, RunDesc* desc, PackedRotation rot,
                                                        HeadParams hp) {
  __shared__ int32_t cu[kThreads + 1], slots[kThreads];
  __shared__ int64_t poss[kThreads];
  __shared__ int total;
  const int tid = threadIdx.x;
  const int64_t u = blockIdx.x;
  pdl_wait();
  pdl_go();
  if (tid == 0) total = 0;
  int bad = 0, before = 0;
  for (int s0 = 0; s0 < ix.seqs; s0 += kThreads) {
    const int s = s0 + tid;
    if (s < ix.seqs) {
      const int64_t a = ix.cu[s], b = ix.cu[s + 1];
      if (s0 == 0) {
        cu[s] = static_cast<int32_t>(a);
        if (s + 1 == ix.seqs || tid + 1 == kThreads) cu[s + 1] = static_cast<int32_t>(b);
        slots[s] = ix.slots[s];
        poss[s] = ix.pos ? ix.pos[s] : 0;
      }
      bad |= a < 0 || b < a || b > ix.rows;
      before += a / ix.run + s <= u;
    }
  }
  __syncthreads();
  before = __reduce_add_sync(0xffffffffu, before);
  if (tid % 32 == 0 && before) atomicAdd(&total, before);
  bad = __syncthreads_or(bad);
  if (rot.offset)  // dealt out to the grid's threads
    for (int64_t e = u * kThreads + tid; e < 17 * rot.half; e += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int r = static_cast<int>(e / rot.half), j = static_cast<int>(e % rot.half);
      turn(rot.offset + r * 2 * rot.half + j / 4 * 8 + j % 4, rot, r, j, hp);
    }
  const int s = total - 1;  // -1: the first sequence starts behind this unit
  if (bad || s < 0) {
    if (tid == 0) {
      if (bad && u == 0) atomicAdd(&g_packed_errors, 1u);
      desc[u] = RunDesc{0, 0, 0, 0, 0, 0, 0};
    }
    return;
  }
  const bool cached = s < kThreads;
  const int64_t a = cached ? cu[s] : ix.cu[s], len = (cached ? cu[s + 1] : ix.cu[s + 1]) - a;
  const int32_t slot = cached ? slots[s] : ix.slots[s];
  const int64_t pos = cached ? poss[s] : ix.pos ? ix.pos[s] : 0;
  int dup = 0;
  for (int j = tid; j < s; j += kThreads)
    dup |= cached ? slots[j] == slot && cu[j + 1] > cu[j] : ix.slots[j] == slot && ix.cu[j + 1] > ix.cu[j];
  dup = __syncthreads_or(dup);
  const int64_t i = u - (a / ix.run + s), runs = (len + ix.run - 1) / ix.run, left = len - i * ix.run;
  const bool wanted = i < runs && slot >= 0, refused = dup || slot >= ix.n_slots || pos < 0 || pos > RETNET_MAX_POSITION;
  const bool live = wanted && !refused;
  if (tid == 0) {
    if (wanted && refused && i == 0) atomicAdd(&g_packed_errors, 1u);
    desc[u] = live ? RunDesc{s, static_cast<int32_t>(a + i * ix.run), static_cast<int32_t>(left < ix.run ? left : ix.run),
                             static_cast<int32_t>(i), static_cast<int32_t>(runs), slot, pos + i * ix.run}
                   : RunDesc{0, 0, 0, 0, 0, 0, 0};
  }
  if (!rot.base || !live) return;
  const int rows = ix.run / 16, width = 2 * rot.half < 128 ? 2 * rot.half : 128;
  for (int e = tid; e < rows * rot.half; e += kThreads) {
    const int r = e / rot.half, j = e % rot.half, col = j / 4 * 8 + j % 4;
    turn(rot.base + (u * rot.half * 2 + col / width * width) * rows + r * width + col % width, rot,
         pos + i * ix.run + 16 * r, j, hp);
  }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedIndex& ix, RunDesc* desc, const PackedRotation& rot, const HeadParams& hp,
                               cudaStream_t s) {
  return launch_dependent(plan_kernel, dim3(static_cast<unsigned>(packed_units(ix.rows, ix.seqs, ix.run))), dim3(kThreads), 0, s,
                          ix, desc, rot, hp);
}

cudaError_t packed_index_errors(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_packed_errors, sizeof(unsigned int));
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_packed_errors, &zero, sizeof(zero));
  return e;
}

}  // namespace retnet
