// packed.cuh -- retention over sequences packed in one token axis: what its kernels share.
//
// A call's sequences are ragged and their lengths live on the device, so the host cannot plan the
// work.  It cuts every sequence into runs of `run` tokens and gives the grids room for the most
// runs there can be: sequence s owns the units from cu_seqlens[s] / run + s on.  Those first units
// grow by at least ceil(len / run) from one sequence to the next (floor(a + len) - floor(a) + 1 >=
// ceil(len) in units of run), so no two sequences share a unit, the last unit is below
// tokens / run + seqs, and a unit finds its sequence by counting, without a prefix sum over the
// lengths.  launch_packed_plan writes one descriptor a unit (tokens 0 where it has no work).
#pragma once

#include "launch.h"

namespace retnet {

struct RunDesc {
  int32_t seq;     // its sequence
  int32_t row;     // first row of the run in q, k, v, o
  int32_t tokens;  // rows of the run; 0: nothing to do
  int32_t index;   // the run's place in its sequence
  int32_t runs;    // runs of the sequence
  int32_t slot;    // the sequence's pool slot
  int64_t pos;     // absolute position of the run's first token
};
static_assert(sizeof(RunDesc) == 32, "two 16-byte words");

struct PackedIndex {
  const int32_t* cu;   // [seqs + 1]
  const int32_t* slots;  // [seqs]
  const int64_t* pos;  // [seqs] or nullptr (all 0)
  int64_t rows;        // rows of q, k, v, o
  int32_t seqs, n_slots, run;
};

inline int64_t packed_units(int64_t rows, int64_t seqs, int64_t run) { return rows / run + seqs; }

// The rotation of a token is base x offset (complex products): base[unit][i] turns the pairs by the
// angle of the run's token 16 i, offset[r] by that of r further tokens, so that a kernel needs no sine
// or cosine of its own.  base: [units][blocks of up to 128 columns][run / 16][columns] floats, offset:
// [17][2 half]; nullptr: not written.  A row holds, for every four pairs, their cosines and then their
// sines.
struct PackedRotation {
  float* base;
  float* offset;
  int half;
  bool xpos;
};
// Writes desc[0 .. packed_units) and the rotations.
cudaError_t launch_packed_plan(const PackedIndex& ix, RunDesc* desc, const PackedRotation& rot, const HeadParams& hp,
                               cudaStream_t s);

// A state S decayed by gamma^n and added to: by S + (keep ? S : 0) + what is added.  Above 1/2 by is
// gamma^n - 1 to full relative precision: the factor itself, near 1, would round the same way run after
// run.  Below, gamma^n: there the sum with S would leave a rounding as large as the old state's behind.
struct Decay {
  float by;
  bool keep;
};
__device__ __forceinline__ Decay decay_of(float log2g, int n) {
  const float f = decay_pow(log2g, n);
  if (f < 0.5f) return Decay{f, false};
  return Decay{expm1f(static_cast<float>(n) * log2g * 0.693147180559945309f), true};
}

}  // namespace retnet
