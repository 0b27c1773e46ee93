// packed_tc.cu -- packed retention on the tensor cores (bf16 inputs).  "阅读笔记：RetNet" §2.4 with
// chunks of 128 tokens, every chunk a run of its own (packed.cuh):
//   state   W_u = sum_t gamma^(127-t) k'_t^T v_t of every chunk        (tcgen05, d_k x d_v x 128)
//   scan    in order over a sequence's chunks: the state before each, rounded to fp16 once, for the
//           products; the fp32 state after the last, to the pool
//   output  O = (Q' K'^T (.) D) V + (Q' R) (.) xi                       (tcgen05, 128 rows a CTA)
// with the row factors in the output's epilogue.
//
// Numerics.  The state is an fp32 result that a sequence carries over thousands of tokens: k' in fp32
// (rotated, decayed) is cut into three bf16 numbers whose sum is k' (3 x 8 significant bits), v is
// bf16 already, so the products are those of fp32 arithmetic and no bf16 input leaves a range.  For
// the scores q' and k' are rounded to fp16 once (2^-11 of the value at most), decayed to the chunk's
// ends: (gamma^(r+1) q'_r) . (gamma^(127-c) k'_c) = gamma^128 gamma^(r-c) q'_r . k'_c, one constant
// factor instead of one a pair.  A warp's rows (8 or 16 of them) are first brought to fp16's upper end by
// a power of two, so that after a decay of up to gamma^128 >= 2^-12 an element 2^-16 of their largest is
// still normal; as they were, q and k of size 0.01 lost up to 1.6 % and of 1e-4 everything at gamma 0.94.
// The masked scores stay in tensor memory as two bf16 numbers (2^-17), so that v is read as it is.  Each
// rounding outside fp16's range is counted (retnet_fp16_range_errors): of states, and what is not finite.
#include <algorithm>

#include "fp32x2.cuh"
#include "packed.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"
#include "steps_done.h"
#include "tensor_map.h"

namespace retnet {
namespace {

using namespace sm100;

constexpr int kChunk = 128;
constexpr int kBlock = kChunk * 128;  // bytes of a 64-column 16-bit block of 128 rows

struct TcPackedArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  float* pool;
  const RunDesc* desc;
  const float* base;    // [units][d_k / M][8][M], M = min(d_k, 128): rotations (packed.cuh)
  const float* offset;  // [17][d_k]
  float* w;             // [units][heads_kv] states of chunks, in blocks of eight columns (below)
  __half* r16;          // [units][heads_kv] states before the chunks, the same
  const int32_t* cu;
  int64_t units, stride_q, stride_k, stride_v, stride_o;
  int32_t kv, group, d_k, d_v;
  uint32_t flags;
  bool o_wide;  // rows of o start on 32-byte boundaries
};

// States in the workspace are [d_k / M][d_v / 8][M][8], M = min(d_k, 128): a thread that holds a row of
// d_k writes eight columns at once beside its neighbours' (a row-major state cost 32 separate lines a
// store), and up to 128 columns of fp16 are the un-swizzled operand of the tensor cores as they lie.
__device__ __forceinline__ int64_t blocked(int row, int col, int m, int d_v) {
  return ((static_cast<int64_t>(row / m) * (d_v / 8) + col / 8) * m + row % m) * 8 + col % 8;
}

// Cosines and sines of four pairs, two and two.
struct Turn {
  Two c[2], s[2];
};
__device__ __forceinline__ Turn load_turn(const float* p) {
  const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(p), s = *reinterpret_cast<const ulonglong2*>(p + 4);
  return Turn{{c.x, c.y}, {s.x, s.y}};
}
// (past the L1 cache)
__device__ __forceinline__ Turn load_turn_l2(const float* p) {
  const ulonglong2 c = __ldcg(reinterpret_cast<const ulonglong2*>(p)), s = __ldcg(reinterpret_cast<const ulonglong2*>(p + 4));
  return Turn{{c.x, c.y}, {s.x, s.y}};
}
__device__ __forceinline__ RunDesc plan_entry(const RunDesc* p) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(p)), b = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  RunDesc d;
  d.seq = a.x; d.row = a.y; d.tokens = a.z; d.index = a.w; d.runs = b.x; d.slot = b.y;
  d.pos = static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(b.w)) << 32 | static_cast<uint32_t>(b.z));
  return d;
}
__device__ __forceinline__ Turn scaled(const Turn& t, float f) {
  const Two ff = two(f, f);
  return Turn{{mul2(t.c[0], ff), mul2(t.c[1], ff)}, {mul2(t.s[0], ff), mul2(t.s[1], ff)}};
}
__device__ __forceinline__ Turn product(const Turn& a, const Turn& b) {
  Turn r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.c[i] = fma2(neg2(a.s[i]), b.s[i], mul2(a.c[i], b.c[i]));
    r.s[i] = fma2(a.c[i], b.s[i], mul2(a.s[i], b.c[i]));
  }
  return r;
}
// Eight bf16 elements (four pairs) turned: first[i], second[i] are the first and second elements of
// pairs 2 i and 2 i + 1.
struct Eight {
  Two first[2], second[2];
};
__device__ __forceinline__ Eight turned(const uint4& raw, const Turn& t) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  Eight y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Two x0 = two(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
    const Two x1 = two(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
    y.first[i] = fma2(neg2(x1), t.s[i], mul2(x0, t.c[i]));
    y.second[i] = fma2(x0, t.s[i], mul2(x1, t.c[i]));
  }
  return y;
}

// The top 16 bits of a and b (bf16 by truncation) as one word.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// x less its truncation to bf16, both lanes (exact).
__device__ __forceinline__ Two rest2(Two x) { return fma2(x & 0xffff0000ffff0000ull, 0xbf800000bf800000ull, x); }
// The bf16 plane of y (truncated) to shared memory; y keeps what is left.
__device__ __forceinline__ void store_plane(unsigned char* to, Eight& y) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = parts(y.first[i]), b = parts(y.second[i]);
    w[2 * i] = top_halves(a.x, b.x);
    w[2 * i + 1] = top_halves(a.y, b.y);
    y.first[i] = rest2(y.first[i]);
    y.second[i] = rest2(y.second[i]);
  }
  *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Row factor s / c_p of §三.3 in fp32 (relative error of a few 2^-24; the output is bf16).
__device__ __forceinline__ float row_factor32(float gamma, int d_k, int64_t p, uint32_t flags) {
  float f = (flags & RETNET_F_SCALE_SQRT_D) ? rsqrtf(static_cast<float>(d_k)) : 1.f;
  if (flags & RETNET_F_NORM_D) {
    const float om = 1.f - gamma;
    f *= rsqrtf(-expm1f(static_cast<float>(p + 1) * log1pf(-om)) / om);
  }
  return f;
}

// Largest magnitude so far (NaN kept), for the fp16 range report.
__device__ __forceinline__ void track(float& mx, float a, float b) {
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(mx) : "f"(a), "f"(b));
}

// ---- states ----------------------------------------------------------------------------------
// One kernel, two walks.  A CTA holds up to 128 rows of d_k x NV columns of d_v and takes chunks in turn:
//   SEQ   the chunks of one (sequence, key/value head) in order: the fp32 state in registers (at most
//         64 values a thread); before each chunk its fp16 rounding goes to r16, after the last the
//         state goes to the pool.  No W, no scan.
//   else  every chunk of every head, dealt out to one CTA an SM: the products W of a chunk to memory.
// Chunks run in steps of 64 tokens through a ring of three: one warp fetches (TMA: k, v, and the step's
// rotations), the data warps rotate k and cut it into planes in place and, behind a chunk's last step,
// take the products of the chunk before out of one of two accumulators, one warp issues the products.
// A data warp that also issued them held the others up for as long as they ran, and one CTA a chunk
// spent a third of its 7 us on starting (32 us for 768 chunk-heads of 128 x 128, now 26).
// Bound by the data warps (converting a step, taking and rounding a state: 49 % of the issue cycles, the
// rest waits of warps that run in step) with the products close behind: a step of 64 tokens takes 4000 cycles
// at M 128, NV 256, its products 2100.  The walk of 10040 tokens, the longest of two documents, takes 336 to
// 341 us by itself; 297 with a third of the products, 315 without the small planes, 264 without both.  There
// 64 state values a thread stand beside the conversion and spill (480 bytes of stores, 316 of loads).
template <int M, int NV>
struct StateCfg {
  static constexpr int kData = 512, kThreads = kData + 128;  // a warpgroup for the copying and the issuing warp
  static constexpr int kHold = NV * 128 / kData;             // state values a thread
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2, kTurns = kStep / 16 * M * 4;
  static constexpr int kSmem = 3 * kPlane + 4 * kPlane + 3 * kVBytes + 3 * kTurns + 1024;
  static constexpr int kCols = 2 * NV;
  // 640 threads are launched with 96 registers each (61440); 512 x 112 + 128 x 32 are as many
};

template <int M, int NV, bool SEQ>
__global__ void __launch_bounds__(StateCfg<M, NV>::kThreads, 1)
    tc_state_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, TcPackedArgs a,
                    HeadParams hp) {
  using C = StateCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  // products of even / odd steps done; operands of even / odd steps ready; ring slots filled, free
  __shared__ uint64_t bars[10];
  __shared__ uint32_t tmem_at;
  const int slices = a.d_v / NV;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  unsigned char* smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  const uint32_t sm = smem_addr(smem), s2 = sm + 3 * C::kPlane, sv = s2 + 4 * C::kPlane, s_turns = sv + 3 * C::kVBytes;
  const uint32_t b_done = smem_addr(&bars[0]), b_ready = smem_addr(&bars[2]), b_full = smem_addr(&bars[4]),
                 b_free = smem_addr(&bars[7]);
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();  // or another CTA of the SM waits for this one's end
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_done + 8 * i, 1);
      mbar_init(b_ready + 8 * i, C::kData / 32);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_free + 8 * i, 1);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at;
  pdl_wait();
  pdl_go();  // not before: an output CTA that took this one's tensor memory would wait for it for ever
  // The CTA's chunks: units first .. first + count - 1 of head blockIdx.y, or the items blockIdx.x +
  // i gridDim.x of (head, unit).
  int64_t first = 0, count = 0;
  RunDesc d0{};
  if constexpr (SEQ) {
    first = a.cu[blockIdx.x] / kChunk + blockIdx.x;
    if (first >= 0 && first < a.units) d0 = a.desc[first];  // (cu_seqlens out of order: no run has tokens)
    if (d0.tokens == 0 || d0.seq != static_cast<int>(blockIdx.x)) {
      if (warp == 0) tmem_dealloc(tm, C::kCols);
      return;
    }
    count = d0.runs;
  } else {
    const int64_t items = a.units * a.kv;
    count = (items - blockIdx.x + gridDim.x - 1) / gridDim.x;
  }
  // Chunk i: its unit and head, and its tokens (0: none).
  struct Item {
    int64_t unit;
    int head, tokens, row;
  };
  auto item = [&](int64_t i) {
    Item it;
    if constexpr (SEQ) {
      it.unit = first + i;
      it.head = blockIdx.y;
      it.row = d0.row + static_cast<int>(i) * kChunk;
      it.tokens = i + 1 < count ? kChunk : a.desc[it.unit].tokens;
    } else {
      const int64_t n = blockIdx.x + i * gridDim.x;
      it.unit = n % a.units;
      it.head = static_cast<int>(n / a.units);
      const RunDesc d = a.desc[it.unit];
      it.tokens = d.tokens;
      it.row = d.row;
    }
    return it;
  };
  // n: steps of this CTA so far.  A wait that gives up ends its role: a data warp's lanes decide together (what
  // follows is a warp's), the data warps together before they exchange a state (its barriers are for all of
  // them), and the other two wait, with the full budget, for what they have issued.
  StepsDone steps;
  auto products_done = [&](int n) {
    if (!steps.must_wait(n)) return true;
    if (!__all_sync(0xffffffffu, mbar_wait(b_done + 8 * (n & 1), (n >> 1) & 1))) return false;
    steps.waited(n);
    return true;
  };
  auto filled = [&](int n) { return __all_sync(0xffffffffu, mbar_wait(b_full + 8 * (n % 3), (n / 3) & 1)); };

  if (tid >= C::kData) {
    registers_less<32>();
    if (warp == C::kData / 32) {  // ---- products
      if (lane == 0) {
        constexpr uint32_t ID = idesc_bf16_f32(M, NV, 1, 1);
        int n = 0, chunk = 0;
        bool alive = true;
        for (int64_t i = 0; alive && i < count; ++i) {
          const int tokens = item(i).tokens;
          for (int st = 0; st * C::kStep < tokens; ++st, ++n) {
            if (!(alive = mbar_wait(b_ready + 8 * (n & 1), (n >> 1) & 1))) break;
            tc_fence_after();
            const uint64_t dv = sdesc_sw128(sv + n % 3 * C::kVBytes, C::kStep * 128, 1024);
            const uint64_t dk0 = sdesc_sw128(sm + n % 3 * C::kPlane, C::kStep * 128, 1024);
            const uint64_t dk1 = sdesc_sw128(s2 + (n & 1) * 2 * C::kPlane, C::kStep * 128, 1024);
            const uint32_t tD = tm + (chunk & 1) * NV;
#pragma unroll
            for (int p = 2; p >= 0; --p) {  // the small planes first
              const uint64_t dk = p == 0 ? dk0 : dk1 + (((p - 1) * C::kPlane) >> 4);
#pragma unroll
              for (int ks = 0; ks < C::kStep / 16; ++ks)
                mma_f16_ss(tD, dk + ((ks * 2048) >> 4), dv + ((ks * 2048) >> 4), ID, st > 0 || p < 2 || ks > 0);
            }
            mma_commit(b_done + 8 * (n & 1));
            mma_commit(b_free + 8 * (n % 3));
          }
          chunk += tokens > 0;
        }
        for (int i = n > 3 ? n - 3 : 0; i < n; ++i) mbar_wait(b_free + 8 * (i % 3), (i / 3) & 1, kDrainBudget);
        for (int i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait(b_done + 8 * (i & 1), (i >> 1) & 1, kDrainBudget);
      }
    } else if (warp == C::kData / 32 + 1) {  // ---- copies
      if (lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        int n = 0;
        bool alive = true;
        for (int64_t i = 0; alive && i < count; ++i) {
          const Item it = item(i);
          for (int st = 0; st * C::kStep < it.tokens; ++st, ++n) {
            const int slot = n % 3;
            if (n >= 3 && !(alive = mbar_wait(b_free + 8 * slot, (n / 3 - 1) & 1))) break;
            const uint32_t bar = b_full + 8 * slot;
            mbar_arrive_expect_tx(bar, C::kPlane + C::kVBytes + C::kTurns);
            const int row = it.row + st * C::kStep;
            tma_load_3d(sm + slot * C::kPlane, &map_k, bar, 0, row, (it.head * a.d_k + k0) / 64);
            tma_load_3d(sv + slot * C::kVBytes, &map_v, bar, 0, row, (it.head * a.d_v + v0) / 64);
            bulk_load(s_turns + slot * C::kTurns, a.base + (it.unit * a.d_k + k0) * 8 + st * (C::kStep / 16) * M, C::kTurns, bar);
          }
        }
        // no copy in flight at the end
        for (int i = n > 3 ? n - 3 : 0; i < n; ++i) mbar_wait(b_full + 8 * (i % 3), (i / 3) & 1, kDrainBudget);
      }
    }
  } else {  // ---- data
    registers_more<112>();
    constexpr int kGroups = M / 8, kRows = C::kData / kGroups, kPer = C::kStep / kRows;
    static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
    const int g = tid % kGroups, tr = tid / kGroups;
    const uint32_t mine = (g / 8) * (C::kStep * 128) + sw128(tr, g % 8);  // kRows more rows: kRows * 128 bytes on
    const Turn off = load_turn(a.offset + (tr % 16) * a.d_k + k0 + g * 8);
    // this thread's piece of the state: row i of d_k in lane i (M = 128), or in lane 32 (i / 16) + i % 16
    // (M = 64); columns cols on
    const int quarter = warp % 4, cols = v0 + (warp / 4) * C::kHold;
    const bool holds = M == 128 || lane < 16;
    const int row = k0 + (M == 128 ? quarter * 32 + lane : quarter * 16 + lane % 16);
    const uint32_t t_mine = tm + (static_cast<uint32_t>(quarter * 32) << 16) + (warp / 4) * C::kHold;
    const int64_t head_size = static_cast<int64_t>(a.d_k) * a.d_v, state_size = a.kv * head_size;
    const int64_t at = blocked(row, cols, M, a.d_v);
    float mx = 0.f;
    Two S[SEQ ? C::kHold / 2 : 1];
    float lg = 0.f;
    Decay full{0.f, true};
    __half* r16 = nullptr;
    auto emit = [&](int64_t chunk) {  // the state before chunk `chunk`, rounded
      if (holds) {  // (what is in the other lanes of tensor memory is no state: not to be reported)
        __half* to = r16 + chunk * state_size;
#pragma unroll
        for (int e = 0; e < C::kHold; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = parts(S[e / 2 + j]);
            track(mx, x.x, x.y);
            w[j] = pack_f16x2(x.x, x.y);
          }
          *reinterpret_cast<uint4*>(to + e * M) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (M != 128) __syncwarp();
    };
    // S <- decay S + up D, D the products of the CTA's chunk-th chunk; or D to W of (unit, head)
    auto take = [&](int chunk, Decay decay, float up, int64_t unit, int head) {
      tc_fence_after();
      const Two kept = decay.keep ? ~0ull : 0ull;
      float* w = nullptr;
      if constexpr (!SEQ) w = a.w + (unit * a.kv + head) * head_size + at;
#pragma unroll
      for (int e = 0; e < C::kHold; e += 16) {
        uint32_t r[1][16];
        tmem_ld_wait(t_mine + (chunk & 1) * NV + e, r);
        if constexpr (SEQ) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            Two& x = S[e / 2 + j];
            x = fma2(two(decay.by), x, fma2(two(up), two(__uint_as_float(r[0][2 * j]), __uint_as_float(r[0][2 * j + 1])), x & kept));
          }
        } else if (holds) {
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint32_t x[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) x[m] = r[0][j + m];
            st_global_v8(w + (e + j) * M, x);
          }
        }
      }
      tc_fence_before();
    };
    float decays[2 * kPer];  // gamma^(127-t) of this thread's rows
    auto set_head = [&](int head) {
      lg = hp.log2g[head];
#pragma unroll
      for (int r = 0; r < 2 * kPer; ++r) decays[r] = decay_pow(lg, 127 - tr - r * kRows);
    };
    // S from the pool, or to it, 128 columns at a time through shared memory (the small planes' place, free
    // before the first step and behind the last), so that the pool is read and written in whole rows: a
    // thread's own row, 16 bytes an access, took 4000 cycles each way.
    auto exchange_pool = [&](bool out) {
      constexpr int kPart = NV < 128 ? NV : 128, kChunks = kPart / 4;
      unsigned char* tile = smem + (s2 - sm);
      float* rows = a.pool + d0.slot * state_size + blockIdx.y * head_size + static_cast<int64_t>(k0) * a.d_v + v0;
      const int my = row - k0, my_col = (warp / 4) * C::kHold;
#pragma unroll
      for (int p = 0; p < NV; p += kPart) {
        const bool here = holds && my_col / kPart * kPart == p;
        if (out && here) {
#pragma unroll
          for (int e = 0; e < C::kHold; e += 4) {
            const float2 x = parts(S[SEQ ? e / 2 : 0]), y = parts(S[SEQ ? e / 2 + 1 : 0]);
            const int c = (my_col - p + e) / 4;
            *reinterpret_cast<float4*>(tile + (my * kChunks + (c ^ (my & 7))) * 16) = make_float4(x.x, x.y, y.x, y.y);
          }
        }
        if (out) named_bar_sync(1, C::kData);
#pragma unroll 8
        for (int e = tid; e < M * kChunks; e += C::kData) {
          const int r = e / kChunks, c = e % kChunks;
          float4* at_pool = reinterpret_cast<float4*>(rows + static_cast<int64_t>(r) * a.d_v + p) + c;
          float4* at_tile = reinterpret_cast<float4*>(tile + (r * kChunks + (c ^ (r & 7))) * 16);
          if (out) *at_pool = *at_tile;
          else *at_tile = *at_pool;
        }
        named_bar_sync(1, C::kData);
        if (!out && here) {
#pragma unroll
          for (int e = 0; e < C::kHold; e += 4) {
            const int c = (my_col - p + e) / 4;
            const float4 x = *reinterpret_cast<const float4*>(tile + (my * kChunks + (c ^ (my & 7))) * 16);
            S[SEQ ? e / 2 : 0] = two(x.x, x.y);
            S[SEQ ? e / 2 + 1 : 0] = two(x.z, x.w);
          }
        }
        if (!out) named_bar_sync(1, C::kData);
      }
    };
    if constexpr (SEQ) {
      set_head(blockIdx.y);
      full = decay_of(lg, kChunk);
      r16 = a.r16 + first * state_size + blockIdx.y * head_size + at;
#pragma unroll
      for (int e = 0; e < C::kHold / 2; ++e) S[e] = two(0.f);
      if (d0.pos > 0) exchange_pool(false);
      if (d0.pos > 0) emit(0);
    }
    int n = 0, chunk = 0, last_step = -1;  // steps, chunks so far; the last step of the chunk before
    int64_t last_unit = 0;
    int last_head = 0, last_tokens = 0;
    bool alive = true;
    for (int64_t i = 0; alive && i < count; ++i) {
      const Item it = item(i);
      if (it.tokens == 0) continue;
      if constexpr (!SEQ) set_head(it.head);
      for (int st = 0; st * C::kStep < it.tokens; ++st, ++n) {
        // the step's copies have landed; the small planes of two steps ago have been read
        if (!(alive = (n < 2 || products_done(n - 2)) && filled(n))) break;
        const int slot = n % 3, left = it.tokens - st * C::kStep;
        unsigned char* hi = smem + slot * C::kPlane + mine;
        unsigned char* low = smem + (3 + (n & 1) * 2) * C::kPlane + mine;
        const unsigned char* turns = smem + 7 * C::kPlane + 3 * C::kVBytes + slot * C::kTurns + g * 32;
        uint4 raw[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          raw[r] = *reinterpret_cast<const uint4*>(hi + r * kRows * 128);
        }
        if (left < C::kStep) {  // rows behind the sequence
#pragma unroll
          for (int r = 0; r < kPer; ++r)
            if (tr + r * kRows >= left) raw[r] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const int t = tr + r * kRows, o = r * kRows * 128;
          const Turn base = load_turn(reinterpret_cast<const float*>(turns + t / 16 * (M * 4)));
          Eight y = turned(raw[r], product(scaled(base, st ? decays[kPer + r] : decays[r]), off));
          store_plane(hi + o, y);
          store_plane(low + o, y);
          store_plane(low + C::kPlane + o, y);
        }
        if (left < C::kStep) {  // 0 x v of another sequence may not be 0
          for (int e = tid; e < (C::kStep - left) * (NV / 8); e += C::kData)
            st_shared_v4(sv + slot * C::kVBytes + (e % (NV / 8) / 8) * (C::kStep * 128) + (left + e / (NV / 8)) * 128 + e % 8 * 16,
                         0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ready + 8 * (n & 1));
      }
      if (!alive) break;
      if (chunk > 0) {  // its products ran beside this chunk's first steps
        if (!(alive = products_done(last_step))) break;
        take(chunk - 1, full, 1.f, last_unit, last_head);
        if constexpr (SEQ) emit(i);
      }
      ++chunk;
      last_step = n - 1;
      last_unit = it.unit;
      last_head = it.head;
      last_tokens = it.tokens;
    }
    alive = alive && chunk > 0 && products_done(last_step);
    if constexpr (SEQ) alive = named_bar_all(1, C::kData, alive);
    if (alive) {
      take(chunk - 1, SEQ ? decay_of(lg, last_tokens) : full,
           SEQ ? exp2f(static_cast<float>(last_tokens - kChunk) * lg) : 1.f, last_unit, last_head);
      if constexpr (SEQ) exchange_pool(true);
    }
    if constexpr (SEQ) report_fp16_range(mx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tm, C::kCols);
  }
}

// ---- scan ------------------------------------------------------------------------------------
// Thread = four columns of one (sequence, head) state, in the order of the blocked states.  The decay after a chunk is gamma^128 except
// the last's; a short last chunk's W is relative to token 127, so it is scaled back by
// gamma^(len-128) <= 2^12.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) tc_scan_kernel(TcPackedArgs a, HeadParams hp) {
  pdl_wait();
  pdl_go();
  const int s = blockIdx.z, h = blockIdx.y;
  const int64_t n4 = static_cast<int64_t>(a.d_k) * a.d_v / 4;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
  const int64_t u0 = a.cu[s] / kChunk + s;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc first = a.desc[u0];
  if (first.tokens == 0 || first.seq != s || e >= n4) return;
  const int m = a.d_k < 128 ? a.d_k : 128, block = static_cast<int>(e / (2 * m)), in = static_cast<int>(e % (2 * m));
  const int row = block / (a.d_v / 8) * m + in / 2, col = block % (a.d_v / 8) * 8 + in % 2 * 4;
  float4* slot = reinterpret_cast<float4*>(a.pool + (static_cast<int64_t>(first.slot) * a.kv + h) * 4 * n4 +
                                           static_cast<int64_t>(row) * a.d_v + col);
  float4 r = first.pos > 0 ? *slot : make_float4(0.f, 0.f, 0.f, 0.f);
  const float lg = hp.log2g[h];
  const Decay full = decay_of(lg, kChunk);
  const int64_t step = static_cast<int64_t>(a.kv) * n4;
  const float4* w = reinterpret_cast<const float4*>(a.w) + (u0 * a.kv + h) * n4 + e;
  uint2* r16 = reinterpret_cast<uint2*>(a.r16) + (u0 * a.kv + h) * n4 + e;
  float mx = 0.f;
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < first.runs; i0 += kAhead) {
    float4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < first.runs) x[i] = __ldcs(w + (i0 + i) * step);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = i0 + i;
      if (u >= first.runs) break;
      if (u > 0 || first.pos > 0) {
        track(mx, r.x, r.y);
        track(mx, r.z, r.w);
        r16[u * step] = make_uint2(pack_f16x2(r.x, r.y), pack_f16x2(r.z, r.w));
      }
      Decay by = full;
      float up = 1.f;
      if (u + 1 == first.runs) {
        const int len = a.desc[u0 + u].tokens;
        by = decay_of(lg, len);
        up = exp2f(static_cast<float>(len - kChunk) * lg);
      }
      r.x = fmaf(by.by, r.x, fmaf(up, x[i].x, by.keep ? r.x : 0.f));
      r.y = fmaf(by.by, r.y, fmaf(up, x[i].y, by.keep ? r.y : 0.f));
      r.z = fmaf(by.by, r.z, fmaf(up, x[i].z, by.keep ? r.z : 0.f));
      r.w = fmaf(by.by, r.w, fmaf(up, x[i].w, by.keep ? r.w : 0.f));
    }
  }
  *slot = r;
  report_fp16_range(mx);
}

// The largest magnitude (15 bits) of each half of N 16-byte pieces of bf16; with FINITE of those that are finite.
template <bool FINITE, int N>
__device__ __forceinline__ uint32_t largest(const uint4 (&raw)[N]) {
  auto size = [](uint32_t w) {
    w &= 0x7fff7fffu;
    return FINITE ? w & __vcmpltu2(w, 0x7f807f80u) : w;
  };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(size(raw[i].x), size(raw[i].y)), __vmaxu2(size(raw[i].z), size(raw[i].w))));
  return top;
}
// The exponent of the power of two that brings magnitudes up to `top` (a finite bf16's 15 bits) below 2^15 and
// the largest to 2^14 at least: turned by a rotation, sqrt(2) larger at most, they are below fp16's 65504.  At
// most 126, so that neither power leaves fp32: magnitudes below 2^-112 reach less than 2^14.
__device__ __forceinline__ int fit_exponent(uint32_t top) { return min(14 + 127 - static_cast<int>(top >> 7), 126); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// ---- output ----------------------------------------------------------------------------------
// CTA = (chunk, query head).  The data warps fetch q and k by asynchronous copies, rotate and round
// them in place, turn the scores into bf16 pairs in tensor memory, and store the outputs: a slice of up
// to 128 columns of d_v is the work of eight of them, the other eight's slice (d_k 256) runs beside it.
// One warp issues all products (P V + Q R of a slice into the accumulator of its warps), one fetches V
// and R in pieces of 32 KB through a ring whose last buffers lie over k, free after the scores.  V comes
// by TMA, or in a sequence's last, shorter chunk by plain copies that leave zeros behind it; R by bulk
// copies: the workspace holds it as the tensor cores take it.
//   When the data warps did all of this in turn, a 64-column slice cost 4800 cycles at d_k 256; with the
// issuing and copying warps 2300, bound by shared memory: a product of 64 columns reads as much of q as
// one of 128, which is what the slices are now.  Bound by HBM at d_k 256, d_v 512: q, k, v, the states and
// o of 16381 tokens and 16 heads are 1.34 GB, in 281 us 4.8 TB/s (73 % of the copy rate).
template <int DK>
struct OutCfg {
  static constexpr int kData = DK == 256 ? 512 : 256;
  static constexpr int kThreads = kData + 64;
  static constexpr int NV = 128, kTeams = kData / 256;            // teams of eight warps, an accumulator each
  static constexpr int M = DK < 128 ? DK : 128;                   // rows of a piece of R
  static constexpr int kQ = kChunk * DK * 2, kPiece = kChunk * NV * 2, kR = M * NV * 2;
  static constexpr int kOwn = DK == 256 ? 3 : DK == 128 ? 1 : 2;  // buffers besides those in k's area
  static constexpr int kRing = kOwn + kQ / kPiece;
  static constexpr int kSmem = 2 * kQ + kOwn * kPiece + 1024;
  static constexpr int kCtas = kSmem <= 110 * 1024 ? 2 : 1;
  static constexpr int kCols = 128 + kTeams * NV <= 256 ? 256 : 512;  // S / P: 0..127, then the accumulators
};

template <int DK>
__global__ void __launch_bounds__(OutCfg<DK>::kThreads, OutCfg<DK>::kCtas)
    tc_output_kernel(const __grid_constant__ CUtensorMap map_v, TcPackedArgs a, HeadParams hp) {
  using C = OutCfg<DK>;
  constexpr int NV = C::NV;
  extern __shared__ unsigned char raw_smem[];
  // q and k ready; scores done; P ready; per buffer: filled, free; per team: products done, read
  __shared__ uint64_t bars[3 + 2 * C::kRing + 2 * C::kTeams];
  __shared__ uint32_t tmem_at;
  __shared__ float factor[kChunk];                       // of the rows of o
  __shared__ float undo_q[kChunk];                       // 1 / the power of two in q's row
  __shared__ __align__(16) float undo_k[kChunk];         // gamma^-128 / the power of two in k's row
  // This grid starts when every CTA of the kernel before it has passed its own wait, so the plan, and all that
  // came before this call, is complete; the plan is read past the L1 cache, q, k and v are read and o, which
  // the state kernel does not touch, is written at any time.  The states are not complete: the copying warp
  // waits before it fetches R (and before the CTA ends, so that no later kernel runs beside the state kernel), and
  // so do the others before they wait for what depends on R: the state kernel may run for longer than their budget.
  const RunDesc d = plan_entry(a.desc + blockIdx.x);
  if (d.tokens == 0) {
    pdl_wait();
    return;
  }
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int hq = blockIdx.y, h = hq / a.group, slices = (a.d_v + NV - 1) / NV;
  unsigned char* smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  const uint32_t sq = smem_addr(smem), sk = sq + C::kQ, own = sk + C::kQ;
  const uint32_t b_qk = smem_addr(bars), b_s = b_qk + 8, b_p = b_qk + 16, b_full = b_qk + 24, b_free = b_full + 8 * C::kRing,
                 b_done = b_free + 8 * C::kRing, b_read = b_done + 8 * C::kTeams;
  const bool has_r = !(d.index == 0 && d.pos == 0);
  const int pieces = 1 + (has_r ? DK / C::M : 0);  // of a slice: V, then R by rows of M
  auto buffer = [&](int n) -> uint32_t {  // of the n-th piece
    const int i = n % C::kRing;
    return i < C::kOwn ? own + i * C::kPiece : sk + (i - C::kOwn) * C::kPiece;
  };
  auto columns = [&](int s) { return a.d_v - s * NV < NV ? a.d_v - s * NV : NV; };  // 64 or 128
  // A wait that gives up ends its role: a warp's lanes decide together (what follows is a warp's), and who has
  // issued products or copies waits, with the full budget, for those.
  auto wait = [](uint32_t bar, int phase) { return mbar_wait(bar, phase & 1); };
  auto wait_all = [](uint32_t bar, int phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1)); };
  auto drain = [](uint32_t bar, int phase) { mbar_wait(bar, phase & 1, kDrainBudget); };
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();
  }
  if (tid == C::kData) {
    mbar_init(b_qk, C::kData / 32);
    mbar_init(b_s, 1);
    mbar_init(b_p, C::kData / 32);
    for (int i = 0; i < 2 * C::kRing; ++i) mbar_init(b_full + 8 * i, 1);
    for (int i = 0; i < C::kTeams; ++i) {
      mbar_init(b_done + 8 * i, 1);
      mbar_init(b_read + 8 * i, 8);
    }
    fence_mbar_init();
  }

  constexpr int kGroups = DK / 8, kRows = C::kData / kGroups, kPer = kChunk / kRows;
  static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
  const int g = tid % kGroups, tr = tid / kGroups;
  const uint32_t mine = (g / 8) * kBlock + sw128(tr, g % 8);  // kRows more rows: kRows * 128 bytes on
  if (tid < C::kData) {
    auto fetch_rows = [&](uint32_t to, const __nv_bfloat16* p, int64_t stride) {
      const __nv_bfloat16* q = p + static_cast<int64_t>(tr) * stride;
#pragma unroll
      for (int i = 0; i < kPer; ++i, q += kRows * stride) {
        const bool in = tr + i * kRows < d.tokens;
        cp_async16(to + mine + i * kRows * 128, in ? q : p, in);
      }
      cp_async_commit();
    };
    fetch_rows(sq, a.q + static_cast<int64_t>(d.row) * a.stride_q + static_cast<int64_t>(hq) * DK + g * 8, a.stride_q);
    fetch_rows(sk, a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * DK + g * 8, a.stride_k);
  } else {
    for (int i = tid - C::kData; i < kChunk; i += 64) factor[i] = row_factor32(hp.gamma[h], DK, d.pos + i, a.flags);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at, tS = tm;

  if (warp == C::kData / 32) {  // ---- products
    if (lane == 0) {
      // descriptors once, then constants added
      const uint64_t dq = sdesc_sw128(sq, 16, 1024), dk = sdesc_sw128(sk, 16, 1024);
      auto kstep = [](int ks) -> uint64_t { return static_cast<uint64_t>(((ks / 4) * kBlock + (ks % 4) * 32) >> 4); };
      bool ok = wait(b_qk, 0);
      const bool scores = ok;
      if (scores) {
        tc_fence_after();
        constexpr uint32_t ID = idesc_f16_f32(kChunk, kChunk, 0, 0);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) mma_f16_ss(tS, dq + kstep(ks), dk + kstep(ks), ID, ks > 0);
        mma_commit(b_s);
        ok = wait(b_p, 0);
      }
      int s = 0, n = 0;
      for (; ok && s < slices; ++s) {
        const int team = s % C::kTeams;
        const uint32_t tO = tm + 128 + team * NV;
        const bool wide = columns(s) == NV;
        if (!(ok = s < C::kTeams || wait(b_read + 8 * team, s / C::kTeams - 1))) break;
        for (int p = 0; p < pieces; ++p, ++n) {
          if (n == 1 && p == 1) pdl_wait();
          if (!(ok = wait(b_full + 8 * (n % C::kRing), n / C::kRing))) break;
          tc_fence_after();
          const uint32_t at = buffer(n);
          if (p == 0) {
            const uint32_t ID = wide ? idesc_bf16_f32(kChunk, NV, 0, 1) : idesc_bf16_f32(kChunk, 64, 0, 1);
            const uint64_t dv = sdesc_sw128(at, kBlock, 1024);
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int ks = 0; ks < kChunk / 16; ++ks)
                mma_f16_ts(tO, tS + (ks / 2) * 32 + part * 16 + (ks % 2) * 8, dv + ((ks * 2048) >> 4), ID, part == 0 || ks > 0);
          } else {
            const uint32_t ID = wide ? idesc_f16_f32(kChunk, NV, 0, 1) : idesc_f16_f32(kChunk, 64, 0, 1);
            const uint64_t dr = sdesc_cores(at, C::M * 16, 128), da = dq + kstep((p - 1) * (C::M / 16));
#pragma unroll
            for (int ks = 0; ks < C::M / 16; ++ks) mma_f16_ss(tO, da + kstep(ks), dr + ((ks * 256) >> 4), ID, 1);
          }
          mma_commit(b_free + 8 * (n % C::kRing));
        }
        if (!ok) break;
        mma_commit(b_done + 8 * team);
      }
      // nothing in flight when the tensor memory is freed
      if (scores) drain(b_s, 0);
      for (int i = n > C::kRing ? n - C::kRing : 0; i < n; ++i) drain(b_free + 8 * (i % C::kRing), i / C::kRing);
      if (s > 0) drain(b_done + 8 * ((s - 1) % C::kTeams), (s - 1) / C::kTeams);
    }
  } else if (warp == C::kData / 32 + 1) {  // ---- V and R
    const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v;
    const __half* rp = a.r16 + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * DK * a.d_v;
    bool ok = true, waited = false;
    int n = 0;
    for (int s = 0; ok && s < slices; ++s) {
      for (int p = 0; p < pieces; ++p, ++n) {
        const int i = n % C::kRing;
        const uint32_t to = buffer(n), bar = b_full + 8 * i;
        ok = n >= C::kRing ? wait_all(b_free + 8 * i, n / C::kRing - 1) : i < C::kOwn || wait_all(b_s, 0);
        if (!ok) break;
        if (p > 0) {
          if (!waited) pdl_wait();
          waited = true;
          if (lane == 0) {
            const uint32_t bytes = C::M * columns(s) * 2;
            mbar_arrive_expect_tx(bar, bytes);
            bulk_load(to, rp + (static_cast<int64_t>(p - 1) * a.d_v + s * NV) * C::M, bytes, bar);
          }
        } else if (d.tokens == kChunk) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::kPiece);
            tma_load_3d(to, &map_v, bar, 0, d.row, (h * a.d_v + s * NV) / 64);
          }
        } else {  // rows behind the sequence are zeros: 0 x v of another sequence may not be 0
          const int chunks = columns(s) / 8;
          for (int e = lane; e < kChunk * chunks; e += 32) {
            const int r = e / chunks, c = e % chunks;
            const bool in = r < d.tokens;
            cp_async16(to + (c / 8) * kBlock + sw128(r, c % 8), vp + static_cast<int64_t>(in ? r : 0) * a.stride_v + s * NV + c * 8, in);
          }
          cp_async_wait_all();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        }
      }
    }
    if (!waited) pdl_wait();
    for (int i = n > C::kRing ? n - C::kRing : 0; i < n; ++i) drain(b_full + 8 * (i % C::kRing), i / C::kRing);
  } else {  // ---- data
    const float lg = hp.log2g[h];
    constexpr int kBase = DK < 128 ? DK : 128;  // columns of a block of the rotations
    // rows t = tr + kRows i: each one's rotation is the last one's times a constant step
    const Turn first = product(load_turn_l2(a.base + (static_cast<int64_t>(blockIdx.x) * DK + g * 8 / kBase * kBase) * 8 +
                                            tr / 16 * kBase + g * 8 % kBase),
                               load_turn_l2(a.offset + (tr % 16) * DK + g * 8));
    Turn step = load_turn_l2(a.offset + 16 * DK + g * 8);
    if (kRows == 32) step = product(step, step);
    float mx = 0.f;
    // q by gamma^(t+1), k by gamma^(127-t), and the warp's rows by the power of two that fits them; undo: what
    // takes that off, times `by`, by row (read behind the scores, which wait for all of this)
    auto convert = [&](unsigned char* area, float scale, float grow, float* undo, float by) {
      uint4 raw[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) raw[i] = *reinterpret_cast<const uint4*>(area + mine + i * kRows * 128);
      auto of_warp = [](uint32_t top) { return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)); };
      uint32_t top = of_warp(largest<false>(raw));
      if (top >= 0x7f80u) top = of_warp(largest<true>(raw));  // (what is not finite stays so at any scale)
      const int fit = fit_exponent(top);
      const float off = by * power_of_two(-fit);
      Turn t = scaled(first, scale * power_of_two(fit));
      const Turn next = scaled(step, grow);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const Eight y = turned(raw[i], t);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 u = parts(y.first[e]), v = parts(y.second[e]);
          track(mx, u.x, u.y);
          track(mx, v.x, v.y);
          w[2 * e] = pack_f16x2(u.x, v.x);
          w[2 * e + 1] = pack_f16x2(u.y, v.y);
        }
        *reinterpret_cast<uint4*>(area + mine + i * kRows * 128) = make_uint4(w[0], w[1], w[2], w[3]);
        if (g == 0) undo[tr + i * kRows] = off;
        if (i + 1 < kPer) t = product(t, next);
      }
    };
    cp_async_wait<1>();
    convert(smem, decay_pow(lg, tr + 1), decay_pow(lg, kRows), undo_q, 1.f);
    cp_async_wait<0>();
    convert(smem + C::kQ, decay_pow(lg, kChunk - 1 - tr), exp2f(-static_cast<float>(kRows) * lg), undo_k,
            exp2f(-static_cast<float>(kChunk) * lg));
    report_fp16_range(mx);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b_qk);
    const int quarter = warp % 4, row = quarter * 32 + lane, team = warp / 8;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    if (wait_all(b_s, 0)) {
      tc_fence_after();
#pragma unroll
      for (int c = (warp / 4) * 32; c < kChunk; c += C::kData / 4) {
        uint32_t r[2][16], p[2][16];
        tmem_ld_wait(tS + lanes + c, r);
        const int keep = c < quarter * 32 ? 31 : c > quarter * 32 ? -1 : lane;  // the row's last column here
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 back = *reinterpret_cast<const float2*>(&undo_k[c + 2 * e]);
          const float x0 = 2 * e <= keep ? __uint_as_float(r[e / 8][2 * e % 16]) * back.x : 0.f;
          const float x1 = 2 * e + 1 <= keep ? __uint_as_float(r[e / 8][2 * e % 16 + 1]) * back.y : 0.f;
          p[0][e] = top_halves(x0, x1);
          const __nv_bfloat162 low = __floats2bfloat162_rn(rest(x0), rest(x1));
          p[1][e] = *reinterpret_cast<const uint32_t*>(&low);
        }
        tmem_st_wait(tS + lanes + c, p);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_p);
      if (has_r) pdl_wait();
      const float f = factor[row] * undo_q[row];
      const int c0 = (warp / 4) % 2 * 64;  // this warp's columns of a slice
      __nv_bfloat16* op = a.o + (static_cast<int64_t>(d.row) + row) * a.stride_o + static_cast<int64_t>(hq) * a.d_v + c0;
      const bool in = row < d.tokens, wide = a.o_wide;
      for (int s = team; s < slices; s += C::kTeams) {
        if (!wait_all(b_done + 8 * team, s / C::kTeams)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t r[2][16];
          tmem_ld_wait(tm + 128 + team * NV + lanes + c0 + c, r);
          if (c == 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_read + 8 * team);
          }
          if (!in || c0 >= columns(s)) continue;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 x =
                  __floats2bfloat162_rn(__uint_as_float(r[e][2 * j]) * f, __uint_as_float(r[e][2 * j + 1]) * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&x);
            }
            __nv_bfloat16* to = op + s * NV + c + e * 16;
            if (wide) {
              st_global_v8(to, w);
            } else {
              reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tm, C::kCols);
  }
}

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename K>
cudaError_t prepare(K kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int M, int NV, bool SEQ>
cudaError_t launch_states(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  using C = StateCfg<M, NV>;
  cudaError_t e = prepare(tc_state_kernel<M, NV, SEQ>, C::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!encode_token_rows(&mk, c.k, c.rows, c.heads_kv * c.d_k, c.stride_k, C::kStep, M / 64) ||
      !encode_token_rows(&mv, c.v, c.rows, c.heads_kv * c.d_v, c.stride_v, C::kStep, NV / 64))
    return cudaErrorUnknown;
  const unsigned kv = static_cast<unsigned>(a.kv), z = static_cast<unsigned>((a.d_k / M) * (a.d_v / NV));
  const dim3 block(C::kThreads);
  if (SEQ)
    return launch_dependent(tc_state_kernel<M, NV, SEQ>, dim3(static_cast<unsigned>(c.seqs), kv, z), block, C::kSmem, s, mk,
                            mv, a, hp);
  const int64_t items = a.units * a.kv, most = std::max<int64_t>(1, 148 / z);
  e = launch_dependent(tc_state_kernel<M, NV, SEQ>, dim3(static_cast<unsigned>(std::min(items, most)), 1, z), block, C::kSmem, s,
                       mk, mv, a, hp);
  if (e != cudaSuccess) return e;
  const unsigned nb = static_cast<unsigned>((static_cast<int64_t>(a.d_k) * a.d_v / 4 + kScanThreads - 1) / kScanThreads);
  return launch_dependent(tc_scan_kernel, dim3(nb, kv, static_cast<unsigned>(c.seqs)), dim3(kScanThreads), 0, s, a, hp);
}

// Whether the states are walked sequence by sequence.  Chunk by chunk takes one more launch and one
// more pass over every chunk's fp32 state, written and read (at d_k 256, d_v 512 more bytes than q, k,
// v and o together); a sequence's walk takes the time of its longest one, so it needs enough CTAs to
// fill the GPU, or sequences short enough (two chunks on average) that there is nothing to spread.
// A call by sequence against one by chunk (bursts of 30 calls; sustained, the first takes 674 us): 16381
// tokens in 2 (the longer 10040), 16 heads of 256 x 512 (128 CTAs) 588 us against 904; 12800 in 64 alike, 8
// heads of 128 x 128 (512) 105 against 139; 157 in 6 (48, short) 16.5 against 26; 12289 in 9 (72), the longest up to
// 4.5 times the shortest, 93 against 84; 16000 in 4 alike, 16 heads of 128 x 256 (64) 260 against 281.
// The host knows how many sequences there are, not how long each is (and counts empty and padding ones), so
// one long among many short ones is walked by few CTAs: 12000 tokens and 63 sequences of 1 to 8, 8 heads of
// 128 x 128, 317 us against 134 by chunk; 12000 and 63 empty ones 282 against 104.
// Slices of 256 columns read k from memory and rotate it for twice as many columns as 128 do: 588 us
// against 695 for the documents.  (Where only 128 columns make 96 CTAs they would be the better choice: the
// 16000 tokens in 4 take 209 us with them, by sequence.)
int state_columns(int64_t d_v) { return d_v % 256 == 0 ? 256 : d_v % 128 == 0 ? 128 : 64; }
bool by_sequence(int64_t rows, int64_t seqs, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  return rows <= 2 * kChunk * seqs ||
         seqs * heads_kv * (d_k > 128 ? d_k / 128 : 1) * (d_v / state_columns(d_v)) >= 96;
}

template <int DK>
cudaError_t launch_shape(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  constexpr int M = DK < 128 ? DK : 128;
  using O = OutCfg<DK>;
  cudaError_t e = prepare(tc_output_kernel<DK>, O::kSmem);
  if (e != cudaSuccess) return e;
  const int nv = state_columns(c.d_v);
  if (by_sequence(c.rows, c.seqs, c.heads_kv, c.d_k, c.d_v)) {
    e = nv == 256 ? launch_states<M, 256, true>(c, a, hp, s)
                  : nv == 128 ? launch_states<M, 128, true>(c, a, hp, s) : launch_states<M, 64, true>(c, a, hp, s);
  } else {
    e = nv == 256 ? launch_states<M, 256, false>(c, a, hp, s)
                  : nv == 128 ? launch_states<M, 128, false>(c, a, hp, s) : launch_states<M, 64, false>(c, a, hp, s);
  }
  if (e != cudaSuccess) return e;
  CUtensorMap mv;
  if (!encode_token_rows(&mv, c.v, c.rows, c.heads_kv * c.d_v, c.stride_v, kChunk, 2)) return cudaErrorUnknown;
  return launch_dependent(tc_output_kernel<DK>, dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(c.heads)),
                          dim3(O::kThreads), O::kSmem, s, mv, a, hp);
}

}  // namespace

bool packed_tc_shape(int64_t d_k, int64_t d_v) { return (d_k == 64 || d_k == 128 || d_k == 256) && d_v % 64 == 0; }

bool packed_tc_supported(const PackedCall& c, const HeadParams& hp) {
  if (c.dtype != RETNET_BF16 || (c.flags & RETNET_F_PRECISE)) return false;
  if (!packed_tc_shape(c.d_k, c.d_v)) return false;
  if ((c.stride_q | c.stride_k | c.stride_v | c.stride_o) % 8) return false;
  auto ok = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!ok(c.q) || !ok(c.k) || !ok(c.v) || !ok(c.o)) return false;
  for (int64_t h = 0; h < c.heads_kv; ++h)
    if (hp.log2g[h] * kChunk < -12.f) return false;
  return true;
}

size_t packed_tc_workspace_bytes(int64_t rows, int64_t seqs, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  const size_t units = static_cast<size_t>(packed_units(rows, seqs, kChunk));
  const size_t states = units * static_cast<size_t>(heads_kv * d_k * d_v);
  const bool chunks = !by_sequence(rows, seqs, heads_kv, d_k, d_v);
  return 256 + a256(sizeof(RunDesc) * units) + a256(sizeof(float) * units * 8 * static_cast<size_t>(d_k)) +
         a256(sizeof(float) * 17 * static_cast<size_t>(d_k)) + (chunks ? a256(sizeof(float) * states) : 0) + sizeof(__half) * states;
}

cudaError_t launch_packed_tc(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  const int64_t units = packed_units(c.rows, c.seqs, kChunk);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(c.ws) + 255) & ~static_cast<uintptr_t>(255));
  auto take = [&](size_t bytes) {
    char* p = ws;
    ws += a256(bytes);
    return p;
  };
  RunDesc* desc = reinterpret_cast<RunDesc*>(take(sizeof(RunDesc) * units));
  float* base = reinterpret_cast<float*>(take(sizeof(float) * units * 8 * c.d_k));
  float* offset = reinterpret_cast<float*>(take(sizeof(float) * 17 * c.d_k));
  const size_t states = static_cast<size_t>(units * c.heads_kv * c.d_k * c.d_v);
  float* w = by_sequence(c.rows, c.seqs, c.heads_kv, c.d_k, c.d_v) ? nullptr : reinterpret_cast<float*>(take(sizeof(float) * states));
  __half* r16 = reinterpret_cast<__half*>(take(sizeof(__half) * states));
  const TcPackedArgs a{static_cast<const __nv_bfloat16*>(c.q), static_cast<const __nv_bfloat16*>(c.k),
                       static_cast<const __nv_bfloat16*>(c.v), static_cast<__nv_bfloat16*>(c.o), c.pool, desc, base,
                       offset, w, r16, c.cu, units, c.stride_q, c.stride_k, c.stride_v, c.stride_o,
                       static_cast<int32_t>(c.heads_kv), static_cast<int32_t>(c.heads / c.heads_kv),
                       static_cast<int32_t>(c.d_k), static_cast<int32_t>(c.d_v), c.flags,
                       c.stride_o % 16 == 0 && (reinterpret_cast<uintptr_t>(c.o) & 31u) == 0};
  const PackedIndex ix{c.cu, c.slot, c.pos, c.rows, static_cast<int32_t>(c.seqs), static_cast<int32_t>(c.slots), kChunk};
  const cudaError_t e = launch_packed_plan(
      ix, desc, PackedRotation{base, offset, static_cast<int>(c.d_k / 2), (c.flags & RETNET_F_XPOS) != 0}, hp, s);
  if (e != cudaSuccess) return e;
  if (c.d_k == 64) return launch_shape<64>(c, a, hp, s);
  if (c.d_k == 128) return launch_shape<128>(c, a, hp, s);
  return launch_shape<256>(c, a, hp, s);
}

cudaError_t packed_set_wait_budget(long long cycles) {
  const long long v = cycles > 0 ? cycles : kDrainBudget;
  return cudaMemcpyToSymbol(g_wait_budget, &v, sizeof(long long));
}

cudaError_t packed_wait_timeouts(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
  if (e != cudaSuccess || !clear || *count == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
}

cudaError_t packed_fp16_overflows(unsigned int* count, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_fp16_overflows, sizeof(unsigned int));
  if (e != cudaSuccess || !clear || *count == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_fp16_overflows, &zero, sizeof(unsigned int));
}

}  // namespace retnet
