// packed_plan.cu -- the parts of packed retention that both kernel families use: the run descriptors
// (packed.cuh), written on the device because the lengths live there, and the count of sequences
// that the device refused.
#include "packed.cuh"

namespace retnet {
namespace {

constexpr int kThreads = 128;

__device__ unsigned int g_packed_errors = 0;

__device__ __forceinline__ float2 turn(const PackedRotation& rot, int64_t p, int j, const HeadParams& hp) {
  float s = 0.f, c = 1.f;
  if (rot.xpos) position_sincos(p, hp.theta[j], &s, &c);
  return make_float2(c, s);
}

// One CTA a unit.  The sequence of a unit is the last one whose first unit is not behind it.  A call
// whose cu_seqlens is out of order or leaves the rows has no runs; a sequence is refused (no run)
// when its slot is out of range or an earlier sequence with tokens has it, or its position is
// negative; one with slot < 0 or no tokens has none either.
__global__ void __launch_bounds__(kThreads) plan_kernel(PackedIndex ix, RunDesc* __restrict__ desc, PackedRotation rot,
                                                        HeadParams hp) {
  const int tid = threadIdx.x;
  const int64_t u = blockIdx.x;
  int bad = 0, before = 0;
  for (int s = tid; s < ix.seqs; s += kThreads) {
    const int64_t a = ix.cu[s], b = ix.cu[s + 1];
    bad |= a < 0 || b < a || b > ix.rows;
    before += a / ix.run + s <= u;
  }
  __shared__ int total;
  if (tid == 0) total = 0;
  bad = __syncthreads_or(bad);
  before = __reduce_add_sync(0xffffffffu, before);
  if (tid % 32 == 0) atomicAdd(&total, before);
  __syncthreads();
  RunDesc d{0, 0, 0, 0, 0, 0, 0};
  if (bad) {
    if (tid == 0) {
      if (u == 0) atomicAdd(&g_packed_errors, 1u);
      desc[u] = d;
    }
    return;
  }
  const int s = total - 1;  // -1: the first sequence starts behind this unit
  int dup = 0;
  if (s >= 0) {
    const int32_t slot = ix.slots[s];
    for (int j = tid; j < s; j += kThreads) dup |= ix.slots[j] == slot && ix.cu[j + 1] > ix.cu[j];
  }
  dup = __syncthreads_or(dup);
  __shared__ int64_t first;  // the run's position, -1 without a run
  if (tid == 0) first = -1;
  if (rot.offset && u == 0) {
    for (int e = tid; e < 16 * rot.half; e += kThreads) rot.offset[e] = turn(rot, e / rot.half, e % rot.half, hp);
  }
  if (tid == 0 && s >= 0) {
    const int64_t a = ix.cu[s], len = ix.cu[s + 1] - a, pos = ix.pos ? ix.pos[s] : 0;
    const int32_t slot = ix.slots[s];
    const int64_t i = u - (a / ix.run + s), runs = (len + ix.run - 1) / ix.run;
    if (i < runs && slot >= 0) {
      if (dup || slot >= ix.n_slots || pos < 0) {
        if (i == 0) atomicAdd(&g_packed_errors, 1u);
      } else {
        const int64_t left = len - i * ix.run;
        d.seq = s;
        d.row = static_cast<int32_t>(a + i * ix.run);
        d.tokens = static_cast<int32_t>(left < ix.run ? left : ix.run);
        d.index = static_cast<int32_t>(i);
        d.runs = static_cast<int32_t>(runs);
        d.slot = slot;
        d.pos = pos + i * ix.run;
        first = d.pos;
      }
    }
  }
  if (tid == 0) desc[u] = d;
  if (!rot.base) return;
  __syncthreads();
  if (first < 0) return;
  const int n = ix.run / 16 * rot.half;
  for (int e = tid; e < n; e += kThreads)
    rot.base[u * n + e] = turn(rot, first + 16 * (e / rot.half), e % rot.half, hp);
}

}  // namespace

cudaError_t launch_packed_plan(const PackedIndex& ix, RunDesc* desc, const PackedRotation& rot, const HeadParams& hp,
                               cudaStream_t s) {
  plan_kernel<<<static_cast<unsigned>(packed_units(ix.rows, ix.seqs, ix.run)), kThreads, 0, s>>>(ix, desc, rot, hp);
  return cudaGetLastError();
}

cudaError_t packed_index_errors(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_packed_errors, sizeof(unsigned int));
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_packed_errors, &zero, sizeof(zero));
  return e;
}

}  // namespace retnet
