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
// factor instead of one a pair; gamma^128 >= 2^-12 keeps both in fp16's normal range.  The masked
// scores stay in tensor memory as two bf16 numbers (2^-17), so that v is read as it is.  Each
// rounding outside fp16's range is counted (retnet_fp16_range_errors).
#include "fp32x2.cuh"
#include "packed.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"
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
  const float* base;    // [units][8][d_k], rotations (packed.cuh)
  const float* offset;  // [17][d_k]
  float* w;             // [units][heads_kv] states of chunks, in blocks of eight columns (below)
  __half* r16;          // [units][heads_kv] states before the chunks, the same
  const int32_t* cu;
  int64_t units, stride_q, stride_k, stride_v, stride_o;
  int32_t kv, group, d_k, d_v;
  uint32_t flags;
  bool o_wide;  // rows of o start on 32-byte boundaries
};

// States in the workspace are [d_v / 8][d_k][8]: a thread that holds a row of d_k writes eight columns
// at once beside its neighbours' (a row-major state cost 32 separate lines a store), and 64 columns of
// fp16 are the un-swizzled operand of the tensor cores as they lie.
__device__ __forceinline__ int64_t blocked(int row, int col, int d_k) {
  return (static_cast<int64_t>(col / 8) * d_k + row) * 8 + col % 8;
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
__device__ __forceinline__ void store_plane(uint32_t to, Eight& y) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = parts(y.first[i]), b = parts(y.second[i]);
    w[2 * i] = top_halves(a.x, b.x);
    w[2 * i + 1] = top_halves(a.y, b.y);
    y.first[i] = rest2(y.first[i]);
    y.second[i] = rest2(y.second[i]);
  }
  st_shared_v4(to, w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t at) {
  uint4 x;
  ld_shared_v4(at, x.x, x.y, x.z, x.w);
  return x;
}
// gamma^n - 1 to full relative precision: a state decayed by fma(that, S, S) keeps the factor's
// accuracy where the factor itself, near 1, would round the same way chunk after chunk.
__device__ __forceinline__ float decay_less_one(float log2g, int n) {
  return expm1f(static_cast<float>(n) * log2g * 0.693147180559945309f);
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

// fp16 range check of packed pairs: the largest magnitude so far, NaN kept.
__device__ __forceinline__ void track(__half2& mx, uint32_t w) {
  mx = __hmax2_nan(mx, __habs2(*reinterpret_cast<const __half2*>(&w)));
}
__device__ __forceinline__ void report(const __half2& mx) {
  const float2 f = __half22float2(mx);
  report_fp16_range(fmaxf(f.x, f.y) + (f.x - f.x) + (f.y - f.y));
}

// ---- state: W of one chunk -------------------------------------------------------------------
// CTA = (chunk, key/value head, up to 128 rows of d_k x NV columns of d_v).  All of the chunk's k and v
// is fetched at once by asynchronous copies; k is rotated and cut in two steps of 64 tokens, its first
// plane written over the raw rows.  The first planes' products and the other two's go to
// accumulators of their own: a tensor-core sum drops what lies below its running value's last bit, so
// it is kept to the 8 steps that one plane takes.  Two CTAs an SM cover one another's waits.
template <int M, int NV>
struct StateCfg {
  static constexpr int kThreads = M == 128 ? 512 : 256;
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2;
  static constexpr int kSmem = 4 * kPlane + 2 * kVBytes + 1024;  // raw / first planes x 2, second, third, v x 2
  static constexpr int kCols = NV;
};

template <int M, int NV>
__global__ void __launch_bounds__(StateCfg<M, NV>::kThreads, 2) tc_state_kernel(TcPackedArgs a, HeadParams hp) {
  using C = StateCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_at;
  pdl_wait();
  pdl_go();
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.y, slices = a.d_v / NV;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  const uint32_t sm = (smem_addr(raw_smem) + 1023u) & ~1023u, s2 = sm + 2 * C::kPlane, sv = sm + 4 * C::kPlane,
                 b = smem_addr(&bar);
  constexpr int kGroups = M / 8, kRows = C::kThreads / kGroups, kPer = C::kStep / kRows;  // rows at once, rows a thread
  const int g = tid % kGroups, tr = tid / kGroups;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * a.d_k + k0 + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v + v0;
  const int steps = d.tokens > C::kStep ? 2 : 1;
  const uint32_t mine = (g / 8) * (C::kStep * 128) + sw128(tr, g % 8);  // kRows more rows: kRows * 128 bytes on
  constexpr int kVPer = C::kStep * (NV / 8) / C::kThreads, kVRows = C::kThreads / (NV / 8);
  static_assert(kVRows % 8 == 0 && kRows % 16 == 0, "rows kVRows apart are swizzled alike; a thread's rows share t % 16");
  const int vr = tid / (NV / 8), vc = tid % (NV / 8);
  const uint32_t v_mine = (vc / 8) * (C::kStep * 128) + sw128(vr, vc % 8);
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    if (st < steps) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = st * C::kStep + tr + i * kRows;
        const bool in = t < d.tokens;
        cp_async16(sm + st * C::kPlane + mine + i * kRows * 128, kp + static_cast<int64_t>(in ? t : 0) * a.stride_k, in);
      }
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int t = st * C::kStep + vr + i * kVRows;
        const bool in = t < d.tokens;
        cp_async16(sv + st * C::kVBytes + v_mine + i * kVRows * 128, vp + static_cast<int64_t>(in ? t : 0) * a.stride_v + vc * 8, in);
      }
    }
    cp_async_commit();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();  // or the SM's next CTA waits for this one's end
  }
  if (tid == 0) {
    mbar_init(b, 1);
    fence_mbar_init();
  }
  const float lg = hp.log2g[h];
  // the decay to the chunk's end, gamma^(127-t) = gamma^(112-16i) gamma^(15-r), t = 16 i + r
  const Turn off = scaled(load_turn(a.offset + (tr % 16) * a.d_k + k0 + g * 8), decay_pow(lg, 15 - tr % 16));
  const float* base = a.base + static_cast<int64_t>(blockIdx.x) * 8 * a.d_k + k0 + g * 8;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at;
  constexpr uint32_t ID = idesc_bf16_f32(M, NV, 1, 1);
  bool dead = false;
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    if (st >= steps) break;
    if (st == 0) cp_async_wait<1>();
    else cp_async_wait<0>();
    Eight y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = tr + i * kRows, at = (st * C::kStep + r) / 16;
      const uint32_t to = sm + st * C::kPlane + mine + i * kRows * 128;
      y[i] = turned(ld_shared_u4(to), product(scaled(load_turn(base + at * a.d_k), decay_pow(lg, 112 - 16 * at)), off));
      store_plane(to, y[i]);
    }
    if (st == 1) dead = !mbar_wait(b, 0, kDrainBudget);  // the first step's products have read planes 2 and 3
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t to = s2 + mine + i * kRows * 128;
      store_plane(to, y[i]);
      store_plane(to + C::kPlane, y[i]);
    }
    fence_proxy_async_smem();
    if (__syncthreads_or(dead)) {
      dead = true;
      break;
    }
    if (tid == 0) {
      const uint64_t dv = sdesc_sw128(sv + st * C::kVBytes, C::kStep * 128, 1024);
#pragma unroll
      for (int p = 2; p >= 0; --p) {
        const uint64_t dk = sdesc_sw128(p == 0 ? sm + st * C::kPlane : s2 + (p - 1) * C::kPlane, C::kStep * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < C::kStep / 16; ++ks)
          mma_f16_ss(tm, dk + ((ks * 2048) >> 4), dv + ((ks * 2048) >> 4), ID, st > 0 || p < 2 || ks > 0);
      }
      mma_commit(b);
    }
  }
  if (!dead) dead = !mbar_wait(b, (steps - 1) & 1, kDrainBudget);
  dead = __syncthreads_or(dead);
  tc_fence_after();
  if (!dead) {
    // row i of d_k in lane i (M = 128), or in lane 32 (i / 16) + i % 16 (M = 64)
    const int quarter = warp % 4;
    const int row = k0 + (M == 128 ? quarter * 32 + lane : quarter * 16 + lane);
    const uint32_t lanes = tm + (static_cast<uint32_t>(quarter * 32) << 16);
    float* w = a.w + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * a.d_k * a.d_v;
#pragma unroll
    for (int c = (warp / 4) * 32; c < NV; c += C::kThreads / 4) {
      uint32_t r[2][16];
      tmem_ld_wait(lanes + c, r);
      if (M == 128 || lane < 16) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = r[e / 16][e % 16 + j];
          st_global_v8(w + blocked(row, v0 + c + e, a.d_k), x);
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

// ---- state of whole sequences ----------------------------------------------------------------
// CTA = (sequence, key/value head, up to 128 rows of d_k x NV columns of d_v): the chunks in order, the
// fp32 state in registers (at most 64 values a thread); before each chunk its fp16 rounding goes to
// r16, after the last the state goes to the pool.  No W, no scan.  Steps of 64 tokens run through a
// ring of three: one warp fetches (TMA: k, v, and the step's rotations), the data warps rotate k and cut
// it in place and, every second step, add and round the chunk before while the products run, one warp
// issues the products.  A data warp that also issued them held the others up for as long as they ran.
template <int M, int NV>
struct SeqCfg {
  static constexpr int kData = NV == 256 ? 512 : 256;
  static constexpr int kThreads = kData + 128;    // a warpgroup for the copying and the issuing warp
  static constexpr int kHold = NV * 128 / kData;  // state values a thread
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2, kTurns = kStep / 16 * M * 4;
  static constexpr int kSmem = 3 * kPlane + 4 * kPlane + 3 * kVBytes + 3 * kTurns + 1024;
  static constexpr int kCols = 2 * NV;
  // 640 threads are launched with 96 registers each (61440); 512 x 112 + 128 x 24 = 60416 of them
  static constexpr bool kMoveRegisters = kData == 512;
};

template <int M, int NV>
__global__ void __launch_bounds__(SeqCfg<M, NV>::kThreads, 1)
    tc_sequence_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, TcPackedArgs a,
                       HeadParams hp) {
  using C = SeqCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  // products of even / odd steps done; operands of even / odd steps ready; ring slots filled, free
  __shared__ uint64_t bars[10];
  __shared__ uint32_t tmem_at;
  pdl_wait();
  pdl_go();
  const int seq = blockIdx.x, h = blockIdx.y, slices = a.d_v / NV;
  const int64_t u0 = a.cu[seq] / kChunk + seq;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc d = a.desc[u0];
  if (d.tokens == 0 || d.seq != seq) return;
  const int len = (d.runs - 1) * kChunk + a.desc[u0 + d.runs - 1].tokens, steps = (len + C::kStep - 1) / C::kStep;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  const uint32_t sm = (smem_addr(raw_smem) + 1023u) & ~1023u, s2 = sm + 3 * C::kPlane, sv = s2 + 4 * C::kPlane,
                 st_turns = sv + 3 * C::kVBytes;
  const uint32_t b_done = smem_addr(&bars[0]), b_ready = smem_addr(&bars[2]), b_full = smem_addr(&bars[4]),
                 b_free = smem_addr(&bars[7]);
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();
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
  auto slot_of = [](int st) { return st % 3; };
  auto products_done = [&](int st) { return mbar_wait(b_done + 8 * (st & 1), (st >> 1) & 1, kDrainBudget); };
  auto filled = [&](int st) { return mbar_wait(b_full + 8 * slot_of(st), (st / 3) & 1, kDrainBudget); };

  if (tid >= C::kData) {
    if constexpr (C::kMoveRegisters) registers_less<24>();
    if (warp == C::kData / 32) {  // ---- products
      if (lane == 0) {
        constexpr uint32_t ID = idesc_bf16_f32(M, NV, 1, 1);
        int st = 0;
        for (; st < steps; ++st) {
          if (!mbar_wait(b_ready + 8 * (st & 1), (st >> 1) & 1, kDrainBudget)) break;
          tc_fence_after();
          const uint64_t dv = sdesc_sw128(sv + slot_of(st) * C::kVBytes, C::kStep * 128, 1024);
          const uint64_t d0 = sdesc_sw128(sm + slot_of(st) * C::kPlane, C::kStep * 128, 1024);
          const uint64_t d1 = sdesc_sw128(s2 + (st & 1) * 2 * C::kPlane, C::kStep * 128, 1024);
          const uint32_t tD = tm + ((st >> 1) & 1) * NV;
#pragma unroll
          for (int p = 2; p >= 0; --p) {  // the small planes first
            const uint64_t dk = p == 0 ? d0 : d1 + (((p - 1) * C::kPlane) >> 4);
#pragma unroll
            for (int ks = 0; ks < C::kStep / 16; ++ks)
              mma_f16_ss(tD, dk + ((ks * 2048) >> 4), dv + ((ks * 2048) >> 4), ID, st % 2 || p < 2 || ks > 0);
          }
          mma_commit(b_done + 8 * (st & 1));
          mma_commit(b_free + 8 * slot_of(st));
        }
        for (int i = st > 3 ? st - 3 : 0; i < st; ++i) mbar_wait(b_free + 8 * slot_of(i), (i / 3) & 1, kDrainBudget);
      }
    } else if (warp == C::kData / 32 + 1) {  // ---- copies
      if (lane == 0) {
        int st = 0;
        for (; st < steps; ++st) {
          const int slot = slot_of(st);
          if (st >= 3 && !mbar_wait(b_free + 8 * slot, (st / 3 - 1) & 1, kDrainBudget)) break;
          const uint32_t bar = b_full + 8 * slot;
          mbar_arrive_expect_tx(bar, C::kPlane + C::kVBytes + C::kTurns);
          const int row = d.row + st * C::kStep;
#pragma unroll
          for (int c = 0; c < M; c += 64)
            tma_load_2d(sm + slot * C::kPlane + c * (C::kStep * 2), &map_k, bar, h * a.d_k + k0 + c, row);
#pragma unroll
          for (int c = 0; c < NV; c += 64)
            tma_load_2d(sv + slot * C::kVBytes + c * (C::kStep * 2), &map_v, bar, h * a.d_v + v0 + c, row);
#pragma unroll
          for (int i = 0; i < C::kStep / 16; ++i)
            bulk_load(st_turns + slot * C::kTurns + i * M * 4,
                      a.base + (u0 * 8 + st * (C::kStep / 16) + i) * static_cast<int64_t>(a.d_k) + k0, M * 4, bar);
        }
        for (int i = st > 3 ? st - 3 : 0; i < st; ++i) filled(i);  // no copy in flight at the end
      }
    }
  } else {  // ---- data
    if constexpr (C::kMoveRegisters) registers_more<112>();
    constexpr int kGroups = M / 8, kRows = C::kData / kGroups, kPer = C::kStep / kRows;
    static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
    const int g = tid % kGroups, tr = tid / kGroups;
    const uint32_t mine = (g / 8) * (C::kStep * 128) + sw128(tr, g % 8);  // kRows more rows: kRows * 128 bytes on
    const float lg = hp.log2g[h];
    const Turn off = scaled(load_turn(a.offset + (tr % 16) * a.d_k + k0 + g * 8), decay_pow(lg, 15 - tr % 16));
    // this thread's piece of the state: row (k0 + row), columns v0 + cols on
    const int quarter = warp % 4, cols = v0 + (warp / 4) * C::kHold;
    const bool holds = M == 128 || lane < 16;
    const int row = k0 + (M == 128 ? quarter * 32 + lane : quarter * 16 + lane % 16);
    const int64_t state_size = static_cast<int64_t>(a.kv) * a.d_k * a.d_v, at_head = static_cast<int64_t>(h) * a.d_k * a.d_v;
    float* pool = a.pool + d.slot * state_size + at_head + static_cast<int64_t>(row) * a.d_v + cols;
    __half* r16 = a.r16 + u0 * state_size + at_head + blocked(row, cols, a.d_k);
    float S[C::kHold];
#pragma unroll
    for (int e = 0; e < C::kHold; e += 4) {
      const float4 x = d.pos > 0 && holds ? *reinterpret_cast<const float4*>(pool + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
    }
    __half2 mx = __float2half2_rn(0.f);
    auto emit = [&](int chunk) {
      __half* to = r16 + chunk * state_size;
#pragma unroll
      for (int e = 0; e < C::kHold; e += 8) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = pack_f16x2(S[e + 2 * j], S[e + 2 * j + 1]);
          track(mx, w[j]);
        }
        if (holds) *reinterpret_cast<uint4*>(to + static_cast<int64_t>(e) * a.d_k) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    if (d.pos > 0) emit(0);
    // S <- S + less S + up D, D the products of a chunk
    auto add_chunk = [&](int chunk, float less, float up) {
      tc_fence_after();
#pragma unroll
      for (int e = 0; e < C::kHold; e += 16) {
        uint32_t r[1][16];
        tmem_ld_wait(tm + (static_cast<uint32_t>(quarter * 32) << 16) + (chunk & 1) * NV + (warp / 4) * C::kHold + e, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) S[e + j] = fmaf(less, S[e + j], fmaf(up, __uint_as_float(r[0][j]), S[e + j]));
      }
      tc_fence_before();
    };
    const float full_less = decay_less_one(lg, kChunk);
    bool alive = true;
    for (int st = 0; st < steps; ++st) {
      // the step's copies have landed; the small planes of two steps ago have been read
      if (!(alive = (st < 2 || products_done(st - 2)) && filled(st))) break;
      const int slot = slot_of(st), left = len - st * C::kStep;
      const uint32_t hi = sm + slot * C::kPlane + mine, low = s2 + (st & 1) * 2 * C::kPlane + mine;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = tr + i * kRows;
        const uint32_t o = i * kRows * 128;
        const uint32_t at = st_turns + slot * C::kTurns + (t / 16) * (M * 4) + g * 32;
        const uint4 c = ld_shared_u4(at), s = ld_shared_u4(at + 16);
        const Turn base{{static_cast<Two>(c.y) << 32 | c.x, static_cast<Two>(c.w) << 32 | c.z},
                        {static_cast<Two>(s.y) << 32 | s.x, static_cast<Two>(s.w) << 32 | s.z}};
        uint4 raw = ld_shared_u4(hi + o);
        if (t >= left) raw = make_uint4(0, 0, 0, 0);  // rows behind the sequence
        Eight y = turned(raw, product(scaled(base, decay_pow(lg, 112 - 64 * (st & 1) - t / 16 * 16)), off));
        store_plane(hi + o, y);
        store_plane(low + o, y);
        store_plane(low + C::kPlane + o, y);
      }
      if (left < C::kStep) {  // 0 x v of another sequence may not be 0
        for (int e = tid; e < (C::kStep - left) * (NV / 8); e += C::kData)
          st_shared_v4(sv + slot * C::kVBytes + (e % (NV / 8) / 8) * (C::kStep * 128) + (left + e / (NV / 8)) * 128 + e % 8 * 16, 0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_ready + 8 * (st & 1));
      if (st >= 3 && st % 2) {  // (awaited above) the products of chunk st / 2 - 1
        add_chunk(st / 2 - 1, full_less, 1.f);
        emit(st / 2);
      }
    }
    if (alive && steps % 2 && steps > 1 && (alive = products_done(steps - 2))) {
      add_chunk(d.runs - 2, full_less, 1.f);
      emit(d.runs - 1);
    }
    if (alive && products_done(steps - 1)) {
      const int last = len - (d.runs - 1) * kChunk;
      add_chunk(d.runs - 1, decay_less_one(lg, last), exp2f(static_cast<float>(last - kChunk) * lg));
      if (holds) {
#pragma unroll
        for (int e = 0; e < C::kHold; e += 4)
          *reinterpret_cast<float4*>(pool + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
      }
    }
    report(mx);
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
  const int block = static_cast<int>(e / (2 * a.d_k)), in = static_cast<int>(e % (2 * a.d_k));  // (column block, half row)
  float4* slot = reinterpret_cast<float4*>(a.pool + (static_cast<int64_t>(first.slot) * a.kv + h) * 4 * n4 +
                                           static_cast<int64_t>(in / 2) * a.d_v + block * 8 + in % 2 * 4);
  float4 r = first.pos > 0 ? *slot : make_float4(0.f, 0.f, 0.f, 0.f);
  const float lg = hp.log2g[h], full_less = decay_less_one(lg, kChunk);
  const int64_t step = static_cast<int64_t>(a.kv) * n4;
  const float4* w = reinterpret_cast<const float4*>(a.w) + (u0 * a.kv + h) * n4 + e;
  uint2* r16 = reinterpret_cast<uint2*>(a.r16) + (u0 * a.kv + h) * n4 + e;
  __half2 mx = __float2half2_rn(0.f);
  constexpr int kAhead = 4;
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
        const uint32_t lo = pack_f16x2(r.x, r.y), hi = pack_f16x2(r.z, r.w);
        track(mx, lo);
        track(mx, hi);
        r16[u * step] = make_uint2(lo, hi);
      }
      float less = full_less, up = 1.f;
      if (u + 1 == first.runs) {
        const int len = a.desc[u0 + u].tokens;
        less = decay_less_one(lg, len);
        up = exp2f(static_cast<float>(len - kChunk) * lg);
      }
      r.x = fmaf(less, r.x, fmaf(up, x[i].x, r.x));
      r.y = fmaf(less, r.y, fmaf(up, x[i].y, r.y));
      r.z = fmaf(less, r.z, fmaf(up, x[i].z, r.z));
      r.w = fmaf(less, r.w, fmaf(up, x[i].w, r.w));
    }
  }
  *slot = r;
  report(mx);
}

// ---- output ----------------------------------------------------------------------------------
// CTA = (chunk, query head).  The data warps fetch q and k by asynchronous copies, rotate and round
// them in place, turn the scores into bf16 pairs in tensor memory, and store the outputs: slice s
// (64 columns of d_v) is the work of four of them, the others' slices run beside it.  One warp issues
// all products (Q R + P V of a slice into the accumulator of its four warps), one fetches R (a bulk
// copy: the workspace holds it as the tensor cores take it) and V through a ring whose last stage lies
// over k, free after the scores.  When the data warps did all of this in turn, a slice cost 4800 cycles
// (products 1800, copies 570, stores 1100, the rest barriers) at d_k 256.
template <int DK>
struct OutCfg {
  static constexpr int kData = DK == 256 ? 512 : 256;
  static constexpr int kThreads = kData + 64;
  static constexpr int NV = 64, kTeams = kData / 128;
  static constexpr int kQ = kChunk * DK * 2;
  static constexpr int kR = DK * NV * 2, kV = kChunk * NV * 2, kStage = kR + kV;
  static constexpr int kOwn = DK == 128 ? 1 : 2;                 // ring stages besides k's area
  static constexpr int kRing = kOwn + (kQ >= kStage ? 1 : 0);
  static constexpr int kSmem = 2 * kQ + kOwn * kStage + 1024;
  static constexpr int kCtas = kSmem <= 110 * 1024 ? 2 : 1;
  static constexpr int kCols = 128 + kTeams * NV <= 256 ? 256 : 512;  // S / P: 0..127, then the accumulators
  // A slice is fetched again only when the one kRing before it is done, and its accumulator's next
  // products wait for that fetch: no barrier runs two phases ahead of one who waits.
  static_assert(kRing <= kTeams, "phases");
};

template <int DK>
__global__ void __launch_bounds__(OutCfg<DK>::kThreads, OutCfg<DK>::kCtas) tc_output_kernel(TcPackedArgs a, HeadParams hp) {
  using C = OutCfg<DK>;
  constexpr int NV = C::NV;
  extern __shared__ unsigned char raw_smem[];
  // q and k ready; scores done; P ready; per ring stage: filled; per team: products done, read
  __shared__ uint64_t bars[3 + C::kRing + 2 * C::kTeams];
  __shared__ uint32_t tmem_at;
  __shared__ float factor[kChunk];
  // This grid starts when the state kernel before it has passed its own wait, so the plan is complete;
  // it is read past the L1 cache.  The states are not: the copying warp waits before it fetches R (and
  // before the CTA ends, so that no later kernel runs beside the state kernel).
  const RunDesc d = plan_entry(a.desc + blockIdx.x);
  if (d.tokens == 0) {
    pdl_wait();
    return;
  }
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int hq = blockIdx.y, h = hq / a.group, slices = a.d_v / NV;
  const uint32_t sq = (smem_addr(raw_smem) + 1023u) & ~1023u, sk = sq + C::kQ, own = sk + C::kQ;
  const uint32_t b_qk = smem_addr(bars), b_s = b_qk + 8, b_p = b_qk + 16, b_full = b_qk + 24, b_done = b_full + 8 * C::kRing,
                 b_read = b_done + 8 * C::kTeams;
  const bool has_r = !(d.index == 0 && d.pos == 0);
  auto stage = [&](int s) -> uint32_t {
    const int i = s % C::kRing;
    return i < C::kOwn ? own + i * C::kStage : sk;
  };
  auto wait = [](uint32_t bar, int phase) { return mbar_wait(bar, phase & 1, kDrainBudget); };
  auto done = [&](int s) { return wait(b_done + 8 * (s % C::kTeams), s / C::kTeams); };
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();
  }
  if (tid == C::kData) {
    mbar_init(b_qk, C::kData / 32);
    mbar_init(b_s, 1);
    mbar_init(b_p, C::kData / 32);
    for (int i = 0; i < C::kRing; ++i) mbar_init(b_full + 8 * i, 2);
    for (int i = 0; i < C::kTeams; ++i) {
      mbar_init(b_done + 8 * i, 1);
      mbar_init(b_read + 8 * i, 4);
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
      if (ok) {
        tc_fence_after();
        constexpr uint32_t ID = idesc_f16_f32(kChunk, kChunk, 0, 0);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) mma_f16_ss(tS, dq + kstep(ks), dk + kstep(ks), ID, ks > 0);
        mma_commit(b_s);
        ok = wait(b_p, 0);
      }
      int s = 0;
      for (; ok && s < slices; ++s) {
        const int team = s % C::kTeams;
        ok = wait(b_full + 8 * (s % C::kRing), s / C::kRing) && (s < C::kTeams || wait(b_read + 8 * team, s / C::kTeams - 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t tO = tm + 128 + team * NV, at = stage(s);
        const uint64_t dr = sdesc_cores(at, DK * 16, 128), dv = sdesc_sw128(at + C::kR, kBlock, 1024);
        if (has_r) {
          constexpr uint32_t ID = idesc_f16_f32(kChunk, NV, 0, 1);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks) mma_f16_ss(tO, dq + kstep(ks), dr + ((ks * 256) >> 4), ID, ks > 0);
        }
        constexpr uint32_t ID = idesc_bf16_f32(kChunk, NV, 0, 1);
#pragma unroll
        for (int part = 1; part >= 0; --part)
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            mma_f16_ts(tO, tS + (ks / 2) * 32 + part * 16 + (ks % 2) * 8, dv + ((ks * 2048) >> 4), ID,
                       has_r || part == 0 || ks > 0);
        mma_commit(b_done + 8 * team);
      }
      wait(b_s, 0);
      if (s > 0) done(s - 1);  // nothing in flight when the tensor memory is freed
    }
  } else if (warp == C::kData / 32 + 1) {  // ---- R and V
    const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v +
                              static_cast<int64_t>(lane / 8) * a.stride_v + lane % 8 * 8;
    const __half* rp = a.r16 + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * DK * a.d_v;
    auto filled = [&](int s) {  // this warp's copies of slice s have landed
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_full + 8 * (s % C::kRing));
    };
    pdl_wait();
    bool ok = true;
    int s = 0;
    for (; s < slices; ++s) {
      if (s >= C::kRing) ok = done(s - C::kRing);
      else if (s >= C::kOwn) ok = wait(b_s, 0);
      if (!ok) break;
      const uint32_t to = stage(s), bar = b_full + 8 * (s % C::kRing);
      if (lane == 0) {
        if (has_r) {
          mbar_arrive_expect_tx(bar, C::kR);
          bulk_load(to, rp + static_cast<int64_t>(s) * NV * DK, C::kR, bar);
        } else {
          mbar_arrive(bar);
        }
      }
      const __nv_bfloat16* p = vp + s * NV;
#pragma unroll
      for (int i = 0; i < kChunk / 4; ++i) {
        const int r = lane / 8 + 4 * i;
        const bool in = r < d.tokens;
        cp_async16(to + C::kR + sw128(r, lane % 8), p + static_cast<int64_t>(in ? 4 * i : 0) * a.stride_v - (in ? 0 : lane / 8 * a.stride_v), in);
      }
      cp_async_commit();
      if (s > 0) {
        cp_async_wait<1>();
        filled(s - 1);
      }
    }
    cp_async_wait<0>();
    if (s > 0) filled(s - 1);
    for (int i = s > C::kRing ? s - C::kRing : 0; i < s; ++i) wait(b_full + 8 * (i % C::kRing), i / C::kRing);
  } else {  // ---- data
    const float lg = hp.log2g[h];
    // rows t = tr + kRows i: each one's rotation is the last one's times a constant step
    const Turn first = product(load_turn_l2(a.base + (static_cast<int64_t>(blockIdx.x) * 8 + tr / 16) * DK + g * 8),
                               load_turn_l2(a.offset + (tr % 16) * DK + g * 8));
    Turn step = load_turn_l2(a.offset + 16 * DK + g * 8);
    if (kRows == 32) step = product(step, step);
    __half2 mx = __float2half2_rn(0.f);
    // q by gamma^(t+1), k by gamma^(127-t)
    auto convert = [&](uint32_t area, float scale, float grow) {
      Turn t = scaled(first, scale);
      const Turn by = scaled(step, grow);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t to = area + mine + i * kRows * 128;
        const Eight y = turned(ld_shared_u4(to), t);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 u = parts(y.first[e]), v = parts(y.second[e]);
          w[2 * e] = pack_f16x2(u.x, v.x);
          w[2 * e + 1] = pack_f16x2(u.y, v.y);
          track(mx, w[2 * e]);
          track(mx, w[2 * e + 1]);
        }
        st_shared_v4(to, w[0], w[1], w[2], w[3]);
        if (i + 1 < kPer) t = product(t, by);
      }
    };
    cp_async_wait<1>();
    convert(sq, decay_pow(lg, tr + 1), decay_pow(lg, kRows));
    cp_async_wait<0>();
    convert(sk, decay_pow(lg, kChunk - 1 - tr), exp2f(-static_cast<float>(kRows) * lg));
    report(mx);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b_qk);
    const int quarter = warp % 4, row = quarter * 32 + lane, team = warp / 4;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float back = exp2f(-static_cast<float>(kChunk) * lg);
    if (wait(b_s, 0)) {
      tc_fence_after();
#pragma unroll
      for (int c = team * 32; c < kChunk; c += C::kTeams * 32) {
        uint32_t r[2][16], p[2][16];
        tmem_ld_wait(tS + lanes + c, r);
        const int keep = c < quarter * 32 ? 31 : c > quarter * 32 ? -1 : lane;  // the row's last column here
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x0 = 2 * e <= keep ? __uint_as_float(r[e / 8][2 * e % 16]) * back : 0.f;
          const float x1 = 2 * e + 1 <= keep ? __uint_as_float(r[e / 8][2 * e % 16 + 1]) * back : 0.f;
          p[0][e] = top_halves(x0, x1);
          const __nv_bfloat162 low = __floats2bfloat162_rn(rest(x0), rest(x1));
          p[1][e] = *reinterpret_cast<const uint32_t*>(&low);
        }
        tmem_st_wait(tS + lanes + c, p);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_p);
      const float f = factor[row];
      __nv_bfloat16* op = a.o + (static_cast<int64_t>(d.row) + row) * a.stride_o + static_cast<int64_t>(hq) * a.d_v;
      const bool in = row < d.tokens, wide = a.o_wide;
      for (int s = team; s < slices; s += C::kTeams) {
        if (!done(s)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NV; c += 32) {
          uint32_t r[2][16];
          tmem_ld_wait(tm + 128 + team * NV + lanes + c, r);
          if (c + 32 == NV) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_read + 8 * team);
          }
          if (!in) continue;
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

template <int M, int NV>
cudaError_t launch_sequences(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  using C = SeqCfg<M, NV>;
  const cudaError_t e = prepare(tc_sequence_kernel<M, NV>, C::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!encode_token_rows(&mk, c.k, c.rows, c.heads_kv * c.d_k, c.stride_k, C::kStep) ||
      !encode_token_rows(&mv, c.v, c.rows, c.heads_kv * c.d_v, c.stride_v, C::kStep))
    return cudaErrorUnknown;
  return launch_dependent(tc_sequence_kernel<M, NV>,
                          dim3(static_cast<unsigned>(c.seqs), static_cast<unsigned>(a.kv),
                               static_cast<unsigned>((a.d_k / M) * (a.d_v / NV))),
                          dim3(C::kThreads), C::kSmem, s, mk, mv, a, hp);
}
template <int M, int NV>
cudaError_t launch_chunks(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  using C = StateCfg<M, NV>;
  cudaError_t e = prepare(tc_state_kernel<M, NV>, C::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned kv = static_cast<unsigned>(a.kv);
  e = launch_dependent(tc_state_kernel<M, NV>,
                       dim3(static_cast<unsigned>(a.units), kv, static_cast<unsigned>((a.d_k / M) * (a.d_v / NV))),
                       dim3(C::kThreads), C::kSmem, s, a, hp);
  if (e != cudaSuccess) return e;
  const unsigned nb = static_cast<unsigned>((static_cast<int64_t>(a.d_k) * a.d_v / 4 + kScanThreads - 1) / kScanThreads);
  return launch_dependent(tc_scan_kernel, dim3(nb, kv, static_cast<unsigned>(c.seqs)), dim3(kScanThreads), 0, s, a, hp);
}

// Whether the states are walked sequence by sequence.  Chunk by chunk takes one more launch and one
// more pass over every chunk's fp32 state, written and read (at d_k 256, d_v 512 more bytes than q, k,
// v and o together); a sequence's walk takes the time of its longest one, so it needs enough CTAs to
// fill the GPU, or sequences short enough (two chunks on average) that there is nothing to spread.
int sequence_columns(int64_t d_v) { return d_v % 256 == 0 ? 256 : d_v % 128 == 0 ? 128 : 64; }
bool by_sequence(int64_t rows, int64_t seqs, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  return rows <= 2 * kChunk * seqs ||
         seqs * heads_kv * (d_k > 128 ? d_k / 128 : 1) * (d_v / sequence_columns(d_v)) >= 96;
}

template <int DK>
cudaError_t launch_shape(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  constexpr int M = DK < 128 ? DK : 128;
  using O = OutCfg<DK>;
  cudaError_t e = prepare(tc_output_kernel<DK>, O::kSmem);
  if (e != cudaSuccess) return e;
  if (by_sequence(c.rows, c.seqs, c.heads_kv, c.d_k, c.d_v)) {
    const int nv = sequence_columns(c.d_v);
    e = nv == 256 ? launch_sequences<M, 256>(c, a, hp, s)
                  : nv == 128 ? launch_sequences<M, 128>(c, a, hp, s) : launch_sequences<M, 64>(c, a, hp, s);
  } else {
    e = c.d_v % 128 == 0 ? launch_chunks<M, 128>(c, a, hp, s) : launch_chunks<M, 64>(c, a, hp, s);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(tc_output_kernel<DK>, dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(c.heads)),
                          dim3(O::kThreads), O::kSmem, s, a, hp);
}

}  // namespace

bool packed_tc_supported(const PackedCall& c, const HeadParams& hp) {
  if (c.dtype != RETNET_BF16 || (c.flags & RETNET_F_PRECISE)) return false;
  if ((c.d_k != 64 && c.d_k != 128 && c.d_k != 256) || c.d_v % 64) return false;
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
  const bool chunks = d_v < 64 || !by_sequence(rows, seqs, heads_kv, d_k, d_v);
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
