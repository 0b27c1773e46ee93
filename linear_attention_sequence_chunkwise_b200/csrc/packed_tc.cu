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
  const float2* base;    // [units][8][d_k / 2]
  const float2* offset;  // [16][d_k / 2]
  float* w;              // [units][heads_kv][d_k][d_v]
  __half* r16;           // [units][heads_kv][d_k][d_v]
  const int32_t* cu;
  int64_t units, stride_q, stride_k, stride_v, stride_o;
  int32_t kv, group, d_k, d_v;
  uint32_t flags;
};

// Eight elements (four pairs) of a rotated head vector: x turned by base x off, times scale.
__device__ __forceinline__ void rotate8(const uint4& raw, const float2* base, const float2 (&off)[4], float scale,
                                        float (&y)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const float4 b01 = *reinterpret_cast<const float4*>(base), b23 = *reinterpret_cast<const float4*>(base + 2);
  const float2 b[4] = {{b01.x, b01.y}, {b01.z, b01.w}, {b23.x, b23.y}, {b23.z, b23.w}};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float bc = b[i].x * scale, bs = b[i].y * scale;
    const float c = bc * off[i].x - bs * off[i].y, s = bc * off[i].y + bs * off[i].x;
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xffff0000u);
    y[2 * i] = x0 * c - x1 * s;
    y[2 * i + 1] = x0 * s + x1 * c;
  }
}

// The top 16 bits of a and b (bf16 by truncation) as one word.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// fp16 range check of packed pairs: the largest magnitude so far, NaN kept.
__device__ __forceinline__ void track(__half2& mx, uint32_t w) {
  mx = __hmax2_nan(mx, __habs2(*reinterpret_cast<const __half2*>(&w)));
}
__device__ __forceinline__ void report(const __half2& mx) {
  const float2 f = __half22float2(mx);
  report_fp16_range(fmaxf(f.x, f.y) + (f.x - f.x) + (f.y - f.y));
}

// ---- state: W of one chunk -------------------------------------------------------------------
// CTA = (chunk, key/value head, up to 128 rows of d_k x NV columns of d_v).  Steps of 64 tokens: the
// three planes of k' (each [64][M], M contiguous) and v ([64][NV]) fill 128-byte-swizzled blocks, one
// thread issues 4 x 3 MMAs, the next step's k is in registers meanwhile.  Two CTAs an SM cover one
// another's conversion and products.
template <int M, int NV>
struct StateCfg {
  static constexpr int kThreads = 256;
  static constexpr int kStep = 64;
  static constexpr int kPlane = kStep * M * 2, kVBytes = kStep * NV * 2;
  static constexpr int kStage = 3 * kPlane + kVBytes;
  static constexpr int kOut = M * NV * 4;  // the result, staged for whole-row stores
  static constexpr int kSmem = (kStage > kOut ? kStage : kOut) + 1024;
};

template <int M, int NV>
__global__ void __launch_bounds__(256, 2) tc_state_kernel(TcPackedArgs a, HeadParams hp) {
  using C = StateCfg<M, NV>;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_at;
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.y, slices = a.d_v / NV;
  const int k0 = (blockIdx.z / slices) * M, v0 = (blockIdx.z % slices) * NV;
  const uint32_t sm = (smem_addr(raw_smem) + 1023u) & ~1023u, sv = sm + 3 * C::kPlane, b = smem_addr(&bar);
  if (warp == 0) tmem_alloc(smem_addr(&tmem_at), NV);
  if (tid == 0) {
    mbar_init(b, 1);
    fence_mbar_init();
  }
  constexpr int kGroups = M / 8, kRows = 256 / kGroups, kPer = C::kStep / kRows;  // rows at once, rows a thread
  const int g = tid % kGroups, tr = tid / kGroups;
  const float lg = hp.log2g[h];
  float2 off[4];
  {
    // the decay to the chunk's end, gamma^(127-t) = gamma^(112-16i) gamma^(15-r), t = 16 i + r
    const float dec = decay_pow(lg, 15 - tr % 16);
    const float2* o = a.offset + (tr % 16) * (a.d_k / 2) + k0 / 2 + g * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = make_float2(o[i].x * dec, o[i].y * dec);
  }
  const float2* base = a.base + static_cast<int64_t>(blockIdx.x) * 8 * (a.d_k / 2) + k0 / 2 + g * 4;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * a.d_k + k0 + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v + v0;
  uint4 kr[kPer];
  auto load_k = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + tr + i * kRows;
      kr[i] = t < d.tokens ? *reinterpret_cast<const uint4*>(kp + static_cast<int64_t>(t) * a.stride_k) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](int t0) {
    constexpr int kVG = NV / 8;
#pragma unroll
    for (int e = tid; e < C::kStep * kVG; e += 256) {
      const int r = e / kVG, c = e % kVG, t = t0 + r;
      const bool in = t < d.tokens;
      cp_async16(sv + (c / 8) * (C::kStep * 128) + sw128(r, c % 8), vp + static_cast<int64_t>(in ? t : 0) * a.stride_v + c * 8, in);
    }
  };
  load_k(0);
  load_v(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at;
  constexpr uint32_t ID = idesc_bf16_f32(M, NV, 1, 1);
  bool dead = false;
#pragma unroll
  for (int st = 0; st < kChunk / C::kStep; ++st) {
    if (st * C::kStep >= d.tokens) break;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tr + i * kRows, at = (st * C::kStep + t) / 16;
      float y[8];
      rotate8(kr[i], base + at * (a.d_k / 2), off, decay_pow(lg, 112 - 16 * at), y);
      const uint32_t to = sm + (g / 8) * (C::kStep * 128) + sw128(t, g % 8);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        st_shared_v4(to + p * C::kPlane, top_halves(y[0], y[1]), top_halves(y[2], y[3]), top_halves(y[4], y[5]),
                     top_halves(y[6], y[7]));
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = rest(y[e]);
      }
    }
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int p = 2; p >= 0; --p) {  // the small planes first
        const uint64_t da = sdesc_sw128(sm + p * C::kPlane, C::kStep * 128, 1024), db = sdesc_sw128(sv, C::kStep * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < C::kStep / 16; ++ks)
          mma_f16_ss(tm, da + ((ks * 2048) >> 4), db + ((ks * 2048) >> 4), ID, st > 0 || p < 2 || ks > 0);
      }
      mma_commit(b);
    }
    const bool more = (st + 1) * C::kStep < d.tokens && st + 1 < kChunk / C::kStep;
    if (more) load_k((st + 1) * C::kStep);
    dead = !mbar_wait(b, st & 1, kDrainBudget);
    if (__syncthreads_or(dead)) {
      dead = true;
      break;
    }
    if (more) load_v((st + 1) * C::kStep);
  }
  tc_fence_after();
  if (!dead) {
    // D: row i of d_k in lane i (M = 128), or in lane 32 (i / 16) + i % 16 (M = 64).  Staged in
    // shared memory, 16-byte pieces swizzled by the row, so that global rows are written whole.
    const int quarter = warp % 4;
    const int row = M == 128 ? quarter * 32 + lane : quarter * 16 + lane;
#pragma unroll
    for (int c = (warp / 4) * 32; c < NV; c += 64) {
      uint32_t r[2][16];
      tmem_ld_wait(tm + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
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
      uint32_t x[4];
      ld_shared_v4(sm + i * (NV * 4) + ((c ^ (i & 7)) << 4), x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(w + static_cast<int64_t>(k0 + i) * a.d_v + c * 4) = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tm, NV);
  }
}

// ---- scan ------------------------------------------------------------------------------------
// Thread = four columns of one (sequence, head) state.  The decay after a chunk is gamma^128 except
// the last's; a short last chunk's W is relative to token 127, so it is scaled back by
// gamma^(len-128) <= 2^12.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) tc_scan_kernel(TcPackedArgs a, HeadParams hp) {
  const int s = blockIdx.z, h = blockIdx.y;
  const int64_t n4 = static_cast<int64_t>(a.d_k) * a.d_v / 4;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
  const int64_t u0 = a.cu[s] / kChunk + s;
  if (u0 < 0 || u0 >= a.units) return;  // cu_seqlens out of order: no run has tokens
  const RunDesc first = a.desc[u0];
  if (first.tokens == 0 || first.seq != s || e >= n4) return;
  float4* slot = reinterpret_cast<float4*>(a.pool) + (static_cast<int64_t>(first.slot) * a.kv + h) * n4 + e;
  float4 r = first.pos > 0 ? *slot : make_float4(0.f, 0.f, 0.f, 0.f);
  const float lg = hp.log2g[h], full = decay_pow(lg, kChunk);
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
      float dec = full, up = 1.f;
      if (u + 1 == first.runs) {
        const int len = a.desc[u0 + u].tokens;
        dec = decay_pow(lg, len);
        up = exp2f(static_cast<float>(len - kChunk) * lg);
      }
      r.x = fmaf(dec, r.x, up * x[i].x);
      r.y = fmaf(dec, r.y, up * x[i].y);
      r.z = fmaf(dec, r.z, up * x[i].z);
      r.w = fmaf(dec, r.w, up * x[i].w);
    }
  }
  *slot = r;
  report(mx);
}

// ---- output ----------------------------------------------------------------------------------
// CTA = (chunk, query head).  Scores once, kept in tensor memory as bf16 pairs; then for every NV
// columns of d_v: R and V into shared memory (the next columns' copies run under this one's epilogue),
// Q R + P V into one accumulator, row factors, store.
template <int DK, int NV>
struct OutCfg {
  static constexpr int kThreads = DK == 256 ? 512 : 256;
  static constexpr int kQ = kChunk * DK * 2;
  static constexpr int kB = DK * (NV > kChunk ? NV : kChunk) * 2;  // k', then R
  static constexpr int kV = kChunk * NV * 2;
  static constexpr int kSmem = kQ + kB + kV + 1024;
  static constexpr int kCtas = kSmem <= 110 * 1024 ? 2 : 1;
  static constexpr int kCols = 256;  // S / P: 0..127, O: 128..128+NV-1
};

template <int DK, int NV>
__global__ void __launch_bounds__(OutCfg<DK, NV>::kThreads, OutCfg<DK, NV>::kCtas)
    tc_output_kernel(TcPackedArgs a, HeadParams hp) {
  using C = OutCfg<DK, NV>;
  extern __shared__ unsigned char raw_smem[];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_at;
  __shared__ float factor[kChunk];
  const RunDesc d = a.desc[blockIdx.x];
  if (d.tokens == 0) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int hq = blockIdx.y, h = hq / a.group;
  const uint32_t sq = (smem_addr(raw_smem) + 1023u) & ~1023u, sb = sq + C::kQ, sv = sb + C::kB, b = smem_addr(&bar);
  if (warp == 0) tmem_alloc(smem_addr(&tmem_at), C::kCols);
  if (tid == 0) {
    mbar_init(b, 1);
    fence_mbar_init();
  }
  constexpr int kGroups = DK / 8, kRows = C::kThreads / kGroups, kPer = kChunk / kRows;
  static_assert(kRows % 16 == 0, "a thread's rows share their place in a group of 16 tokens");
  const int g = tid % kGroups, tr = tid / kGroups;
  const float lg = hp.log2g[h];
  const __nv_bfloat16* qp = a.q + static_cast<int64_t>(d.row) * a.stride_q + static_cast<int64_t>(hq) * DK + g * 8;
  const __nv_bfloat16* kp = a.k + static_cast<int64_t>(d.row) * a.stride_k + static_cast<int64_t>(h) * DK + g * 8;
  const __nv_bfloat16* vp = a.v + static_cast<int64_t>(d.row) * a.stride_v + static_cast<int64_t>(h) * a.d_v;
  const __half* rp = a.r16 + (static_cast<int64_t>(blockIdx.x) * a.kv + h) * DK * a.d_v;
  const bool has_r = !(d.index == 0 && d.pos == 0);
  uint4 raw[kPer];
  auto load_rows = [&](const __nv_bfloat16* p, int64_t stride) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tr + i * kRows;
      raw[i] = t < d.tokens ? *reinterpret_cast<const uint4*>(p + static_cast<int64_t>(t) * stride) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](int v0) {
#pragma unroll
    for (int e = tid; e < kChunk * (NV / 8); e += C::kThreads) {
      const int r = e / (NV / 8), c = e % (NV / 8);
      const bool in = r < d.tokens;
      cp_async16(sv + (c / 8) * kBlock + sw128(r, c % 8), vp + static_cast<int64_t>(in ? r : 0) * a.stride_v + v0 + c * 8, in);
    }
  };
  auto load_r = [&](int v0) {
    if (!has_r) return;
#pragma unroll
    for (int e = tid; e < DK * (NV / 8); e += C::kThreads) {
      const int r = e / (NV / 8), c = e % (NV / 8);
      cp_async16(sb + (c / 8) * (DK * 128) + sw128(r, c % 8), rp + static_cast<int64_t>(r) * a.d_v + v0 + c * 8, true);
    }
  };
  load_rows(qp, a.stride_q);
  load_v(0);
  const float2* base = a.base + static_cast<int64_t>(blockIdx.x) * 8 * (DK / 2) + g * 4;
  float2 off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) off[i] = a.offset[(tr % 16) * (DK / 2) + g * 4 + i];
  for (int i = tid; i < kChunk; i += C::kThreads) factor[i] = row_factor(hp.gamma[h], DK, d.pos + i, a.flags);
  __half2 mx = __float2half2_rn(0.f);
  // q by gamma^(t+1), k by gamma^(127-t); t = 16 at + tr % 16
  auto convert = [&](uint32_t to, bool is_q) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tr + i * kRows, at = t / 16;
      float y[8];
      rotate8(raw[i], base + at * (DK / 2), off, decay_pow(lg, is_q ? t + 1 : kChunk - 1 - t), y);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = pack_f16x2(y[2 * e], y[2 * e + 1]);
        track(mx, w[e]);
      }
      st_shared_v4(to + (g / 8) * kBlock + sw128(t, g % 8), w[0], w[1], w[2], w[3]);
    }
  };
  convert(sq, true);
  load_rows(kp, a.stride_k);
  convert(sb, false);
  report(mx);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_at, tS = tm, tO = tm + 128;
  if (tid == 0) {
    constexpr uint32_t ID = idesc_f16_f32(kChunk, kChunk, 0, 0);
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      const uint32_t at = (ks / 4) * kBlock + (ks % 4) * 32;
      mma_f16_ss(tS, sdesc_sw128(sq + at, 16, 1024), sdesc_sw128(sb + at, 16, 1024), ID, ks > 0);
    }
    mma_commit(b);
  }
  uint32_t phase = 0;
  bool dead = !mbar_wait(b, phase, kDrainBudget);
  phase ^= 1;
  if (!__syncthreads_or(dead)) {
    tc_fence_after();
    load_r(0);
    const int quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    {
      const float back = exp2f(-static_cast<float>(kChunk) * lg);
#pragma unroll
      for (int c = (warp / 4) * 32; c < kChunk; c += (C::kThreads / 128) * 32) {
        uint32_t r[2][16], p[2][16];
        tmem_ld_wait(tS + lanes + c, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = 2 * e + j;
            x[j] = c + col <= row ? __uint_as_float(r[col / 16][col % 16]) * back : 0.f;
          }
          p[0][e] = top_halves(x[0], x[1]);
          const __nv_bfloat162 low = __floats2bfloat162_rn(rest(x[0]), rest(x[1]));
          p[1][e] = *reinterpret_cast<const uint32_t*>(&low);
        }
        tmem_st_wait(tS + lanes + c, p);
      }
      tc_fence_before();
    }
    for (int v0 = 0; v0 < a.d_v; v0 += NV) {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncthreads();
      tc_fence_after();
      if (tid == 0) {
        if (has_r) {
          constexpr uint32_t ID = idesc_f16_f32(kChunk, NV, 0, 1);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_f16_ss(tO, sdesc_sw128(sq + (ks / 4) * kBlock + (ks % 4) * 32, 16, 1024),
                       sdesc_sw128(sb + ks * 2048, DK * 128, 1024), ID, ks > 0);
        }
        constexpr uint32_t ID = idesc_bf16_f32(kChunk, NV, 0, 1);
#pragma unroll
        for (int part = 1; part >= 0; --part)
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            mma_f16_ts(tO, tS + (ks / 2) * 32 + part * 16 + (ks % 2) * 8, sdesc_sw128(sv + ks * 2048, kBlock, 1024), ID,
                       has_r || part == 0 || ks > 0);
        mma_commit(b);
      }
      dead = !mbar_wait(b, phase, kDrainBudget);
      phase ^= 1;
      if (__syncthreads_or(dead)) break;
      tc_fence_after();
      if (v0 + NV < a.d_v) {
        load_r(v0 + NV);
        load_v(v0 + NV);
      }
      const float f = factor[row];
      __nv_bfloat16* op = a.o + (static_cast<int64_t>(d.row) + row) * a.stride_o + static_cast<int64_t>(hq) * a.d_v + v0;
#pragma unroll
      for (int c = (warp / 4) * 32; c < NV; c += (C::kThreads / 128) * 32) {
        uint32_t r[2][16];
        tmem_ld_wait(tO + lanes + c, r);
        if (row < d.tokens) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int col = e * 8 + j * 2;
              const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(r[col / 16][col % 16]) * f,
                                                             __uint_as_float(r[col / 16][col % 16 + 1]) * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(op + c + e * 8) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
    }
  }
  cp_async_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tm, C::kCols);
  }
}

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename K>
cudaError_t prepare(K kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int DK, int NV>
cudaError_t launch_shape(const PackedCall& c, const TcPackedArgs& a, const HeadParams& hp, cudaStream_t s) {
  constexpr int M = DK < 128 ? DK : 128;
  using S = StateCfg<M, NV>;
  using O = OutCfg<DK, NV>;
  cudaError_t e = prepare(tc_state_kernel<M, NV>, S::kSmem);
  if (e == cudaSuccess) e = prepare(tc_output_kernel<DK, NV>, O::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned u = static_cast<unsigned>(a.units), kv = static_cast<unsigned>(a.kv);
  tc_state_kernel<M, NV><<<dim3(u, kv, static_cast<unsigned>((DK / M) * (a.d_v / NV))), S::kThreads, S::kSmem, s>>>(a, hp);
  const unsigned nb = static_cast<unsigned>((static_cast<int64_t>(DK) * a.d_v / 4 + kScanThreads - 1) / kScanThreads);
  tc_scan_kernel<<<dim3(nb, kv, static_cast<unsigned>(c.seqs)), kScanThreads, 0, s>>>(a, hp);
  tc_output_kernel<DK, NV><<<dim3(u, static_cast<unsigned>(c.heads)), O::kThreads, O::kSmem, s>>>(a, hp);
  return cudaGetLastError();
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
  const size_t units = static_cast<size_t>(packed_units(rows, seqs, kChunk)), half = static_cast<size_t>(d_k / 2);
  const size_t states = units * static_cast<size_t>(heads_kv * d_k * d_v);
  return a256(sizeof(RunDesc) * units) + a256(sizeof(float2) * units * 8 * half) + a256(sizeof(float2) * 16 * half) +
         a256(sizeof(float) * states) + sizeof(__half) * states;
}

cudaError_t launch_packed_tc(const PackedCall& c, const HeadParams& hp, cudaStream_t s) {
  const int64_t units = packed_units(c.rows, c.seqs, kChunk), half = c.d_k / 2;
  char* ws = static_cast<char*>(c.ws);
  auto take = [&](size_t bytes) {
    char* p = ws;
    ws += a256(bytes);
    return p;
  };
  RunDesc* desc = reinterpret_cast<RunDesc*>(take(sizeof(RunDesc) * units));
  float2* base = reinterpret_cast<float2*>(take(sizeof(float2) * units * 8 * half));
  float2* offset = reinterpret_cast<float2*>(take(sizeof(float2) * 16 * half));
  const size_t states = static_cast<size_t>(units * c.heads_kv * c.d_k * c.d_v);
  float* w = reinterpret_cast<float*>(take(sizeof(float) * states));
  __half* r16 = reinterpret_cast<__half*>(take(sizeof(__half) * states));
  const TcPackedArgs a{static_cast<const __nv_bfloat16*>(c.q), static_cast<const __nv_bfloat16*>(c.k),
                       static_cast<const __nv_bfloat16*>(c.v), static_cast<__nv_bfloat16*>(c.o), c.pool, desc, base,
                       offset, w, r16, c.cu, units, c.stride_q, c.stride_k, c.stride_v, c.stride_o,
                       static_cast<int32_t>(c.heads_kv), static_cast<int32_t>(c.heads / c.heads_kv),
                       static_cast<int32_t>(c.d_k), static_cast<int32_t>(c.d_v), c.flags};
  const PackedIndex ix{c.cu, c.slot, c.pos, c.rows, static_cast<int32_t>(c.seqs), static_cast<int32_t>(c.slots), kChunk};
  const cudaError_t e = launch_packed_plan(
      ix, desc, PackedRotation{base, offset, static_cast<int>(half), (c.flags & RETNET_F_XPOS) != 0}, hp, s);
  if (e != cudaSuccess) return e;
  const bool wide = c.d_v % 128 == 0;
  if (c.d_k == 64) return wide ? launch_shape<64, 128>(c, a, hp, s) : launch_shape<64, 64>(c, a, hp, s);
  if (c.d_k == 128) return wide ? launch_shape<128, 128>(c, a, hp, s) : launch_shape<128, 64>(c, a, hp, s);
  return wide ? launch_shape<256, 128>(c, a, hp, s) : launch_shape<256, 64>(c, a, hp, s);
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
