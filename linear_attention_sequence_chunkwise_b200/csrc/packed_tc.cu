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
#include "packed.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"

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
  float* w;              // [units][heads_kv][d_k][d_v]
  __half* r16;           // [units][heads_kv][d_k][d_v]
  const int32_t* cu;
  int64_t units, stride_q, stride_k, stride_v, stride_o;
  int32_t kv, group, d_k, d_v;
  uint32_t flags;
};

// Pairs of floats for the packed fp32 instructions (two lanes an instruction).
using Two = uint64_t;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 parts(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two neg2(Two a) { return a ^ 0x8000000080000000ull; }

// Cosines and sines of four pairs, two and two.
struct Turn {
  Two c[2], s[2];
};
__device__ __forceinline__ Turn load_turn(const float* p) {
  const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(p), s = *reinterpret_cast<const ulonglong2*>(p + 4);
  return Turn{{c.x, c.y}, {s.x, s.y}};
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
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2;
  static constexpr int kSmem = 4 * kPlane + 2 * kVBytes + 1024;  // raw / first planes x 2, second, third, v x 2
  static constexpr int kCols = NV;
  static_assert(M * NV * 4 <= 4 * kPlane + 2 * kVBytes, "the result is staged over the operands");
};

template <int M, int NV>
__global__ void __launch_bounds__(256, 2) tc_state_kernel(TcPackedArgs a, HeadParams hp) {
  using C = StateCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_at;
  pdl_go();
  pdl_wait();
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.y, slices = a.d_v / NV;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  const uint32_t sm = (smem_addr(raw_smem) + 1023u) & ~1023u, s2 = sm + 2 * C::kPlane, sv = sm + 4 * C::kPlane,
                 b = smem_addr(&bar);
  constexpr int kGroups = M / 8, kRows = 256 / kGroups, kPer = C::kStep / kRows;  // rows at once, rows a thread
  const int g = tid % kGroups, tr = tid / kGroups;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * a.d_k + k0 + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v + v0;
  const int steps = d.tokens > C::kStep ? 2 : 1;
  const uint32_t mine = (g / 8) * (C::kStep * 128);  // this thread's column block
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    if (st < steps) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = tr + i * kRows, t = st * C::kStep + r;
        const bool in = t < d.tokens;
        cp_async16(sm + st * C::kPlane + mine + sw128(r, g % 8), kp + static_cast<int64_t>(in ? t : 0) * a.stride_k, in);
      }
#pragma unroll
      for (int e = tid; e < C::kStep * (NV / 8); e += 256) {
        const int r = e / (NV / 8), c = e % (NV / 8), t = st * C::kStep + r;
        const bool in = t < d.tokens;
        cp_async16(sv + st * C::kVBytes + (c / 8) * (C::kStep * 128) + sw128(r, c % 8),
                   vp + static_cast<int64_t>(in ? t : 0) * a.stride_v + c * 8, in);
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
      const uint32_t to = sm + st * C::kPlane + mine + sw128(r, g % 8);
      y[i] = turned(ld_shared_u4(to), product(scaled(load_turn(base + at * a.d_k), decay_pow(lg, 112 - 16 * at)), off));
      store_plane(to, y[i]);
    }
    if (st == 1) dead = !mbar_wait(b, 0, kDrainBudget);  // the first step's products have read planes 2 and 3
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t to = s2 + mine + sw128(tr + i * kRows, g % 8);
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
    // Row i of d_k in lane i (M = 128), or in lane 32 (i / 16) + i % 16 (M = 64).  Staged in shared
    // memory, 16-byte pieces swizzled by the row, so that global rows are written whole.
    const int quarter = warp % 4;
    const int row = M == 128 ? quarter * 32 + lane : quarter * 16 + lane;
    const uint32_t lanes = tm + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
    for (int c = (warp / 4) * 32; c < NV; c += 64) {
      uint32_t r[2][16];
      tmem_ld_wait(lanes + c, r);
      if (M == 128 || lane < 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          st_shared_v4(sm + row * (NV * 4) + (((c / 4 + e) ^ (row & 7)) << 4), r[e / 4][(e % 4) * 4], r[e / 4][(e % 4) * 4 + 1],
                       r[e / 4][(e % 4) * 4 + 2], r[e / 4][(e % 4) * 4 + 3]);
      }
    }
    __syncthreads();
    float* w = a.w + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * a.d_k * a.d_v + v0;
    for (int e = tid; e < M * NV / 4; e += 256) {
      const int i = e / (NV / 4), c = e % (NV / 4);
      *reinterpret_cast<uint4*>(w + static_cast<int64_t>(k0 + i) * a.d_v + c * 4) =
          ld_shared_u4(sm + i * (NV * 4) + ((c ^ (i & 7)) << 4));
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
// fp32 state in registers (at most 64 values a thread); before each chunk its fp16 rounding goes to r16, after
// the last the state goes to the pool.  No W, no scan.  Steps of 64 tokens run through a ring: copies
// two steps ahead, k of the next step is cut while the products of this one run.
template <int M, int NV>
struct SeqCfg {
  static constexpr int kThreads = NV == 256 ? 512 : 256;
  static constexpr int kHold = NV * 128 / kThreads;  // state values a thread
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2;
  static constexpr int kSmem = 3 * kPlane + 4 * kPlane + 3 * kVBytes + 1024;
  static constexpr int kCols = 2 * NV;
};

template <int M, int NV>
__global__ void __launch_bounds__(SeqCfg<M, NV>::kThreads, 1) tc_sequence_kernel(TcPackedArgs a, HeadParams hp) {
  using C = SeqCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bars[2];
  __shared__ uint32_t tmem_at;
  pdl_go();
  pdl_wait();
  const int seq = blockIdx.x, h = blockIdx.y, slices = a.d_v / NV;
  const int64_t u0 = a.cu[seq] / kChunk + seq;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc d = a.desc[u0];
  if (d.tokens == 0 || d.seq != seq) return;
  const int len = (d.runs - 1) * kChunk + a.desc[u0 + d.runs - 1].tokens, steps = (len + C::kStep - 1) / C::kStep;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  const uint32_t sm = (smem_addr(raw_smem) + 1023u) & ~1023u, s2 = sm + 3 * C::kPlane, sv = s2 + 4 * C::kPlane;
  const uint32_t b0 = smem_addr(&bars[0]), b1 = smem_addr(&bars[1]);
  constexpr int kGroups = M / 8, kRows = C::kThreads / kGroups, kPer = C::kStep / kRows;
  static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
  const int g = tid % kGroups, tr = tid / kGroups;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * a.d_k + k0 + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v + v0;
  const uint32_t mine = (g / 8) * (C::kStep * 128);
  auto fetch = [&](int st) {
    if (st < steps) {
      const int slot = st % 3;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = tr + i * kRows, t = st * C::kStep + r;
        const bool in = t < len;
        cp_async16(sm + slot * C::kPlane + mine + sw128(r, g % 8), kp + static_cast<int64_t>(in ? t : 0) * a.stride_k, in);
      }
#pragma unroll
      for (int i = 0; i < C::kStep * (NV / 8) / C::kThreads; ++i) {
        const int e = tid + i * C::kThreads, r = e / (NV / 8), c = e % (NV / 8), t = st * C::kStep + r;
        const bool in = t < len;
        cp_async16(sv + slot * C::kVBytes + (c / 8) * (C::kStep * 128) + sw128(r, c % 8),
                   vp + static_cast<int64_t>(in ? t : 0) * a.stride_v + c * 8, in);
      }
    }
    cp_async_commit();
  };
  fetch(0);
  fetch(1);
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(b0, 1);
    mbar_init(b1, 1);
    fence_mbar_init();
  }
  const float lg = hp.log2g[h];
  const Turn off = scaled(load_turn(a.offset + (tr % 16) * a.d_k + k0 + g * 8), decay_pow(lg, 15 - tr % 16));
  const float* base = a.base + u0 * 8 * a.d_k + k0 + g * 8;
  // this thread's piece of the state: row (k0 + row), columns v0 + cols on
  const int quarter = warp % 4, cols = (warp / 4) * C::kHold;
  const bool holds = M == 128 || lane < 16;
  const int row = k0 + (M == 128 ? quarter * 32 + lane : quarter * 16 + lane % 16);
  const int64_t at_state = static_cast<int64_t>(h) * a.d_k * a.d_v + static_cast<int64_t>(row) * a.d_v + v0 + cols;
  const int64_t state_size = static_cast<int64_t>(a.kv) * a.d_k * a.d_v;
  float* pool = a.pool + d.slot * state_size + at_state;
  __half* r16 = a.r16 + u0 * state_size + at_state;
  float S[C::kHold];
#pragma unroll
  for (int e = 0; e < C::kHold; e += 4) {
    const float4 x = d.pos > 0 && holds ? *reinterpret_cast<const float4*>(pool + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
  }
  __half2 mx = __float2half2_rn(0.f);
  auto emit = [&](int chunk) {
#pragma unroll
    for (int e = 0; e < C::kHold; e += 16) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = pack_f16x2(S[e + 2 * j], S[e + 2 * j + 1]);
        track(mx, w[j]);
      }
      if (holds) st_global_v8(r16 + chunk * state_size + e, w);
    }
  };
  if (d.pos > 0) emit(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at;
  // S <- S + less S + up D, D the products of a chunk
  auto add_chunk = [&](int chunk, float less, float up) {
#pragma unroll
    for (int e = 0; e < C::kHold; e += 32) {
      uint32_t r[2][16];
      tmem_ld_wait(tm + (static_cast<uint32_t>(quarter * 32) << 16) + (chunk & 1) * NV + cols + e, r);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        S[e + j] = fmaf(less, S[e + j], fmaf(up, __uint_as_float(r[j / 16][j % 16]), S[e + j]));
    }
    tc_fence_before();
  };
  constexpr uint32_t ID = idesc_bf16_f32(M, NV, 1, 1);
  const float full_less = decay_less_one(lg, kChunk);
  bool dead = false;
  auto wait_step = [&](int st) { dead |= !mbar_wait(st & 1 ? b1 : b0, (st >> 1) & 1, kDrainBudget); };
  for (int st = 0; st < steps; ++st) {
    cp_async_wait<1>();
    const uint32_t hi = sm + (st % 3) * C::kPlane, low = s2 + (st & 1) * 2 * C::kPlane;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = tr + i * kRows, at = st * (C::kStep / 16) + r / 16;  // base rows of a chunk are 8, in order
      const uint32_t to = mine + sw128(r, g % 8);
      Eight y = turned(ld_shared_u4(hi + to), product(scaled(load_turn(base + static_cast<int64_t>(at) * a.d_k),
                                                             decay_pow(lg, 112 - 16 * (at % 8))), off));
      store_plane(hi + to, y);
      store_plane(low + to, y);
      store_plane(low + C::kPlane + to, y);
    }
    fence_proxy_async_smem();
    if (__syncthreads_or(dead)) {
      dead = true;
      break;
    }
    tc_fence_after();
    if (tid == 0) {
      const uint64_t dv = sdesc_sw128(sv + (st % 3) * C::kVBytes, C::kStep * 128, 1024);
      const uint32_t tD = tm + ((st >> 1) & 1) * NV;
#pragma unroll
      for (int p = 2; p >= 0; --p) {
        const uint64_t dk = sdesc_sw128(p == 0 ? hi : low + (p - 1) * C::kPlane, C::kStep * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < C::kStep / 16; ++ks)
          mma_f16_ss(tD, dk + ((ks * 2048) >> 4), dv + ((ks * 2048) >> 4), ID, st % 2 || p < 2 || ks > 0);
      }
      mma_commit(st & 1 ? b1 : b0);
    }
    if (st > 0) wait_step(st - 1);  // its ring slot is free
    fetch(st + 2);
    if (st > 0 && st % 2 == 0) {  // the chunk before this step is complete; the next one's products run
      tc_fence_after();
      add_chunk(st / 2 - 1, full_less, 1.f);
      emit(st / 2);
    }
  }
  if (!dead) wait_step(steps - 1);
  dead = __syncthreads_or(dead);
  if (!dead) {
    tc_fence_after();
    const int last = len - (d.runs - 1) * kChunk;
    add_chunk(d.runs - 1, decay_less_one(lg, last), exp2f(static_cast<float>(last - kChunk) * lg));
    if (holds) {
#pragma unroll
      for (int e = 0; e < C::kHold; e += 4)
        *reinterpret_cast<float4*>(pool + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }
  report(mx);
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tm, C::kCols);
  }
}

// ---- scan ------------------------------------------------------------------------------------
// Thread = four columns of one (sequence, head) state.  The decay after a chunk is gamma^128 except
// the last's; a short last chunk's W is relative to token 127, so it is scaled back by
// gamma^(len-128) <= 2^12.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) tc_scan_kernel(TcPackedArgs a, HeadParams hp) {
  pdl_go();
  pdl_wait();
  const int s = blockIdx.z, h = blockIdx.y;
  const int64_t n4 = static_cast<int64_t>(a.d_k) * a.d_v / 4;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
  const int64_t u0 = a.cu[s] / kChunk + s;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc first = a.desc[u0];
  if (first.tokens == 0 || first.seq != s || e >= n4) return;
  float4* slot = reinterpret_cast<float4*>(a.pool) + (static_cast<int64_t>(first.slot) * a.kv + h) * n4 + e;
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
// CTA = (chunk, query head).  q and k arrive by asynchronous copies and are rotated and rounded in
// place; the scores are computed once and kept in tensor memory as bf16 pairs.  Then, for every 64
// columns of d_v, Q R + P V into one of two accumulators: R and V come through a ring whose last
// stage lies over k (free after the scores), and a slice's epilogue (row factors, store) runs under
// the next one's products.
template <int DK>
struct OutCfg {
  static constexpr int kThreads = DK == 256 ? 512 : 256;
  static constexpr int NV = 64;
  static constexpr int kQ = kChunk * DK * 2;
  static constexpr int kR = DK * NV * 2, kV = kChunk * NV * 2, kStage = kR + kV;
  static constexpr int kOwn = DK == 128 ? 1 : 2;                 // ring stages besides k's area
  static constexpr int kRing = kOwn + (kQ >= kStage ? 1 : 0);
  static constexpr int kSmem = 2 * kQ + kOwn * kStage + 1024;
  static constexpr int kCtas = kSmem <= 110 * 1024 ? 2 : 1;
  static constexpr int kCols = 256;  // S / P: 0..127, O: 128.. and 192..
};

template <int DK>
__global__ void __launch_bounds__(OutCfg<DK>::kThreads, OutCfg<DK>::kCtas) tc_output_kernel(TcPackedArgs a, HeadParams hp) {
  using C = OutCfg<DK>;
  constexpr int NV = C::NV;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bars[3];
  __shared__ uint32_t tmem_at;
  __shared__ float factor[kChunk];
  pdl_wait();
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int hq = blockIdx.y, h = hq / a.group, slices = a.d_v / NV;
  const uint32_t sq = (smem_addr(raw_smem) + 1023u) & ~1023u, sk = sq + C::kQ, own = sk + C::kQ;
  const uint32_t bs = smem_addr(&bars[0]), bo[2] = {smem_addr(&bars[1]), smem_addr(&bars[2])};
  constexpr int kGroups = DK / 8, kRows = C::kThreads / kGroups, kPer = kChunk / kRows;
  static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
  const int g = tid % kGroups, tr = tid / kGroups;
  const float lg = hp.log2g[h];
  const __nv_bfloat16* qp = a.q + static_cast<int64_t>(d.row) * a.stride_q + static_cast<int64_t>(hq) * DK + g * 8;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * DK + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v;
  const __half* rp = a.r16 + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * DK * a.d_v;
  const bool has_r = !(d.index == 0 && d.pos == 0);
  const uint32_t mine = (g / 8) * kBlock;
  auto fetch_rows = [&](uint32_t to, const __nv_bfloat16* p, int64_t stride) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tr + i * kRows;
      const bool in = t < d.tokens;
      cp_async16(to + mine + sw128(t, g % 8), p + static_cast<int64_t>(in ? t : 0) * stride, in);
    }
    cp_async_commit();
  };
  auto stage = [&](int s) -> uint32_t {
    const int i = s % C::kRing;
    return i < C::kOwn ? own + i * C::kStage : sk;
  };
  auto fetch_slice = [&](int s) {
    if (s < slices) {
      const uint32_t to = stage(s), tv = to + C::kR;
      const int v0 = s * NV;
      if (has_r) {
#pragma unroll
        for (int i = 0; i < DK * (NV / 8) / C::kThreads; ++i) {
          const int e = tid + i * C::kThreads, r = e / (NV / 8), c = e % (NV / 8);
          cp_async16(to + sw128(r, c), rp + static_cast<int64_t>(r) * a.d_v + v0 + c * 8, true);
        }
      }
#pragma unroll
      for (int i = 0; i < kChunk * (NV / 8) / C::kThreads; ++i) {
        const int e = tid + i * C::kThreads, r = e / (NV / 8), c = e % (NV / 8);
        const bool in = r < d.tokens;
        cp_async16(tv + sw128(r, c), vp + static_cast<int64_t>(in ? r : 0) * a.stride_v + v0 + c * 8, in);
      }
    }
    cp_async_commit();
  };
  fetch_rows(sq, qp, a.stride_q);
  fetch_rows(sk, kp, a.stride_k);
#pragma unroll
  for (int s = 0; s < C::kOwn; ++s) fetch_slice(s);
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_at), C::kCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bs, 1);
    mbar_init(bo[0], 1);
    mbar_init(bo[1], 1);
    fence_mbar_init();
  }
  // rows t = tr + kRows i: each one's rotation is the last one's times a constant step
  const Turn first = product(load_turn(a.base + (static_cast<int64_t>(blockIdx.x) * 8 + tr / 16) * DK + g * 8),
                             load_turn(a.offset + (tr % 16) * DK + g * 8));
  Turn step = load_turn(a.offset + 16 * DK + g * 8);
  if (kRows == 32) step = product(step, step);
  for (int i = tid; i < kChunk; i += C::kThreads) factor[i] = row_factor32(hp.gamma[h], DK, d.pos + i, a.flags);
  __half2 mx = __float2half2_rn(0.f);
  // q by gamma^(t+1), k by gamma^(127-t)
  auto convert = [&](uint32_t area, float scale, float grow) {
    Turn t = scaled(first, scale);
    const Turn s = scaled(step, grow);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t to = area + mine + sw128(tr + i * kRows, g % 8);
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
      if (i + 1 < kPer) t = product(t, s);
    }
  };
  cp_async_wait<C::kOwn + 1>();
  convert(sq, decay_pow(lg, tr + 1), decay_pow(lg, kRows));
  cp_async_wait<C::kOwn>();
  convert(sk, decay_pow(lg, kChunk - 1 - tr), exp2f(-static_cast<float>(kRows) * lg));
  report(mx);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at, tS = tm;
  // descriptors once, then constants added: built anew for every product they were most of a slice's time
  const uint64_t dq = sdesc_sw128(sq, 16, 1024);
  auto kstep = [](int ks) -> uint64_t { return static_cast<uint64_t>(((ks / 4) * kBlock + (ks % 4) * 32) >> 4); };
  if (tid == 0) {
    constexpr uint32_t ID = idesc_f16_f32(kChunk, kChunk, 0, 0);
    const uint64_t dk = sdesc_sw128(sk, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) mma_f16_ss(tS, dq + kstep(ks), dk + kstep(ks), ID, ks > 0);
    mma_commit(bs);
  }
  bool dead = !mbar_wait(bs, 0, kDrainBudget);
  if (!__syncthreads_or(dead)) {
    tc_fence_after();
    if (C::kRing > C::kOwn) fetch_slice(C::kOwn);
    const int quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    {
      const float back = exp2f(-static_cast<float>(kChunk) * lg);
#pragma unroll
      for (int c = (warp / 4) * 32; c < kChunk; c += (C::kThreads / 128) * 32) {
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
    }
    const float f = factor[row];
    __nv_bfloat16* op = a.o + (static_cast<int64_t>(d.row) + row) * a.stride_o + static_cast<int64_t>(hq) * a.d_v;
    // Slice s out of its accumulator: 16 columns a thread and turn.
    auto epilogue = [&](int s) {
      const uint32_t tO = tm + 128 + (s & 1) * NV;
#pragma unroll
      for (int c = (warp / 4) * 16; c < NV; c += (C::kThreads / 128) * 16) {
        uint32_t r[1][16];
        tmem_ld_wait(tO + lanes + c, r);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 x =
              __floats2bfloat162_rn(__uint_as_float(r[0][2 * j]) * f, __uint_as_float(r[0][2 * j + 1]) * f);
          w[j] = *reinterpret_cast<const uint32_t*>(&x);
        }
        if (row < d.tokens) {
          uint4* to = reinterpret_cast<uint4*>(op + s * NV + c);
          to[0] = make_uint4(w[0], w[1], w[2], w[3]);
          to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      tc_fence_before();
    };
    for (int s = 0; s <= slices; ++s) {
      if (s < slices) {
        if (s == 0) cp_async_wait<C::kRing - 1>();
        else cp_async_wait<C::kRing - 2>();
        fence_proxy_async_smem();
        __syncthreads();
        tc_fence_after();
        if (tid == 0) {
          const uint32_t tO = tm + 128 + (s & 1) * NV;
          const uint64_t dr = sdesc_sw128(stage(s), DK * 128, 1024), dv = sdesc_sw128(stage(s) + C::kR, kBlock, 1024);
          if (has_r) {
            constexpr uint32_t ID = idesc_f16_f32(kChunk, NV, 0, 1);
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) mma_f16_ss(tO, dq + kstep(ks), dr + ((ks * 2048) >> 4), ID, ks > 0);
          }
          constexpr uint32_t ID = idesc_bf16_f32(kChunk, NV, 0, 1);
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int ks = 0; ks < kChunk / 16; ++ks)
              mma_f16_ts(tO, tS + (ks / 2) * 32 + part * 16 + (ks % 2) * 8, dv + ((ks * 2048) >> 4), ID,
                         has_r || part == 0 || ks > 0);
          mma_commit(bo[s & 1]);
        }
      }
      if (s > 0) {
        dead = !mbar_wait(bo[(s - 1) & 1], ((s - 1) >> 1) & 1, kDrainBudget);
        if (__syncthreads_or(dead)) break;
        tc_fence_after();
        fetch_slice(s - 1 + C::kRing);
        epilogue(s - 1);
      }
    }
  }
  cp_async_wait_all();
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
  return launch_dependent(tc_sequence_kernel<M, NV>,
                          dim3(static_cast<unsigned>(c.seqs), static_cast<unsigned>(a.kv),
                               static_cast<unsigned>((a.d_k / M) * (a.d_v / NV))),
                          dim3(C::kThreads), C::kSmem, s, a, hp);
}
template <int M, int NV>
cudaError_t launch_chunks(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  using C = StateCfg<M, NV>;
  cudaError_t e = prepare(tc_state_kernel<M, NV>, C::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned kv = static_cast<unsigned>(a.kv);
  e = launch_dependent(tc_state_kernel<M, NV>,
                       dim3(static_cast<unsigned>(a.units), kv, static_cast<unsigned>((a.d_k / M) * (a.d_v / NV))), dim3(256),
                       C::kSmem, s, a, hp);
  if (e != cudaSuccess) return e;
  const unsigned nb = static_cast<unsigned>((static_cast<int64_t>(a.d_k) * a.d_v / 4 + kScanThreads - 1) / kScanThreads);
  return launch_dependent(tc_scan_kernel, dim3(nb, kv, static_cast<unsigned>(c.seqs)), dim3(kScanThreads), 0, s, a, hp);
}

// Whether the states are walked sequence by sequence.  Chunk by chunk takes one more pass over every
// chunk's fp32 state, written and read (at d_k 256, d_v 512 more bytes than q, k, v and o together);
// a sequence's walk takes the time of its longest one, so it needs enough CTAs to fill the GPU.
int sequence_columns(int64_t d_v) { return d_v % 256 == 0 ? 256 : d_v % 128 == 0 ? 128 : 64; }
bool by_sequence(int64_t seqs, int64_t heads_kv, int64_t d_k, int64_t d_v) {
  return seqs * heads_kv * (d_k > 128 ? d_k / 128 : 1) * (d_v / sequence_columns(d_v)) >= 96;
}

template <int DK>
cudaError_t launch_shape(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  constexpr int M = DK < 128 ? DK : 128;
  using O = OutCfg<DK>;
  cudaError_t e = prepare(tc_output_kernel<DK>, O::kSmem);
  if (e != cudaSuccess) return e;
  if (by_sequence(c.seqs, c.heads_kv, c.d_k, c.d_v)) {
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
  const bool chunks = d_v < 64 || !by_sequence(seqs, heads_kv, d_k, d_v);
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
  float* w = by_sequence(c.seqs, c.heads_kv, c.d_k, c.d_v) ? nullptr : reinterpret_cast<float*>(take(sizeof(float) * states));
  __half* r16 = reinterpret_cast<__half*>(take(sizeof(__half) * states));
  const TcPackedArgs a{static_cast<const __nv_bfloat16*>(c.q), static_cast<const __nv_bfloat16*>(c.k),
                       static_cast<const __nv_bfloat16*>(c.v), static_cast<__nv_bfloat16*>(c.o), c.pool, desc, base,
                       offset, w, r16, c.cu, units, c.stride_q, c.stride_k, c.stride_v, c.stride_o,
                       static_cast<int32_t>(c.heads_kv), static_cast<int32_t>(c.heads / c.heads_kv),
                       static_cast<int32_t>(c.d_k), static_cast<int32_t>(c.d_v), c.flags};
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
