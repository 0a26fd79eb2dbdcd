// Orthogonalised updates of stacked matrices (the Muon optimiser's step for the weight
// gradients that the backward writes).  Host side in muon_api.cuh.  For each matrix
// G [rows, cols] of a stack:
//
//   m' = beta m + G,   u = G + beta m' (Nesterov) | m' | G (no momentum),
//   X_0 = u / (|u|_F + eps),
//   X_{k+1} = a X_k + (b A + c A^2) X_k,   A = X_k X_k^T      (rows <= cols),
//   X_{k+1} = a X_k + X_k (b A + c A^2),   A = X_k^T X_k      (rows > cols),
//   w' = keep * w - step * X.
//
// Numbers: the products run on tcgen05 (kind::f16, fp16 operands, fp32 accumulation); X is
// held as hi + lo, two fp16 (22 bits), and the linear term a X is formed from both, apart
// from the products.  With bf16 operands the result is 1e-2 (full-rank u) to 1.6e-1
// (rank-deficient u) off the exact one, with fp16 operands and aI folded into the polynomial
// 1.2e-3 to 2e-2: a rounding of X has parts along directions that u does not have, and those
// grow by a^5 = 485.  With the linear term apart only b A X and c A^2 X see rounded operands,
// and those products have no part along such directions.  What the roundings of A and
// B = b A + c A^2 do is mostly their diagonals' doing (A is near I at the end): the diagonals'
// remainders are kept in fp32 and put back by the epilogues.  Together 3e-4 to 1.2e-3 on
// every spectrum tried, below the output's own bf16 rounding (1.7e-3).
// Matrices with at most 128 rows or columns have few roundings to average over (one, for a
// single row); their products take hi lo and lo hi as well (SPLIT), which costs nothing there.
// Powers of two keep every operand in fp16's range, from the largest value (bounded by the
// spectral norm) to 1e-9 of it: X 2^15, A 2^14, B 2^13.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "wgrad.cuh"

namespace moe {

constexpr float kNsSx = 32768.f, kNsSa = 16384.f, kNsSb = 8192.f;

// ---------------------------------------------------------------------------
// Momentum, norm and X_0.
// ---------------------------------------------------------------------------
struct MuonInArgs {
  const void* grad;         // [groups, rows, cols] fp32 or bf16
  const float* mom_in;      // or null: no momentum
  float* mom_out;           // the same shape; may be mom_in
  double* part;             // [groups, chunks]: sums of u^2
  __half* hi; __half* lo;   // X_0: [groups, rows, ld]
  int64_t n;                // rows * cols
  int cols, ld, chunk, chunks, nesterov;
  float beta, eps;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Momentum and each chunk's sum of u^2, in 64 bits (the squares of 1e-30 or 1e30 stay in
// range), added in an order fixed by the shape.  VEC: four elements an access.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) muon_norm_kernel(const __grid_constant__ MuonInArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double red[8];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * a.n;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t i1 = min(i0 + a.chunk, a.n);
  const T* g = static_cast<const T*>(a.grad) + base;
  double s = 0.0;
  auto one = [&](float gv, float mv, float& mo) -> float {
    if (!a.mom_in) return gv;
    mo = fmaf(a.beta, mv, gv);
    return a.nesterov ? fmaf(a.beta, mo, gv) : mo;
  };
  if constexpr (VEC) {
    for (int64_t i = i0 + threadIdx.x * 4; i < i1; i += 1024) {
      const float4 gv = load4<T>(g + i);
      float4 mv = make_float4(0, 0, 0, 0), mo = mv, u;
      if (a.mom_in) mv = *reinterpret_cast<const float4*>(a.mom_in + base + i);
      u.x = one(gv.x, mv.x, mo.x);
      u.y = one(gv.y, mv.y, mo.y);
      u.z = one(gv.z, mv.z, mo.z);
      u.w = one(gv.w, mv.w, mo.w);
      if (a.mom_in) *reinterpret_cast<float4*>(a.mom_out + base + i) = mo;
      s += static_cast<double>(u.x) * u.x + static_cast<double>(u.y) * u.y +
           static_cast<double>(u.z) * u.z + static_cast<double>(u.w) * u.w;
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
      float mo = 0.f;
      const float u = one(load1(g + i), a.mom_in ? a.mom_in[base + i] : 0.f, mo);
      if (a.mom_in) a.mom_out[base + i] = mo;
      s += static_cast<double>(u) * u;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane_id() == 0) red[warp_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 8; ++i) s += red[i];
    a.part[static_cast<int64_t>(blockIdx.y) * a.chunks + blockIdx.x] = s;
  }
}

// x = hi + lo in fp16, each rounded to nearest (lo is subnormal below 2^-29 of 1: 2^-40 off).
__device__ __forceinline__ void split_half(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(x - __half2float(hi));
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) muon_scale_kernel(const __grid_constant__ MuonInArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double red[8];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * a.n;
  double s = 0.0;
  for (int i = threadIdx.x; i < a.chunks; i += 256)
    s += a.part[static_cast<int64_t>(blockIdx.y) * a.chunks + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane_id() == 0) red[warp_id()] = s;
  __syncthreads();
  s = 0.0;
  for (int i = 0; i < 8; ++i) s += red[i];
  const float scale = static_cast<float>(static_cast<double>(kNsSx) / (sqrt(s) + a.eps));
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t i1 = min(i0 + a.chunk, a.n);
  const T* g = static_cast<const T*>(a.grad) + base;
  const float* m = a.mom_in ? a.mom_out + base : nullptr;
  const int rows = static_cast<int>(a.n / a.cols);
  const int64_t xb = static_cast<int64_t>(blockIdx.y) * rows * a.ld;
  auto one = [&](float gv, float mo) -> float {
    return scale * (!m ? gv : (a.nesterov ? fmaf(a.beta, mo, gv) : mo));
  };
  if constexpr (VEC) {
    for (int64_t i = i0 + threadIdx.x * 4; i < i1; i += 1024) {
      float4 gv = make_float4(0, 0, 0, 0), mo = gv;
      if (!m || a.nesterov) gv = load4<T>(g + i);
      if (m) mo = *reinterpret_cast<const float4*>(m + i);
      __align__(8) __half h[4], l[4];
      split_half(one(gv.x, mo.x), h[0], l[0]);
      split_half(one(gv.y, mo.y), h[1], l[1]);
      split_half(one(gv.z, mo.z), h[2], l[2]);
      split_half(one(gv.w, mo.w), h[3], l[3]);
      const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.cols);
      const int64_t o = xb + static_cast<int64_t>(r) * a.ld + (i - static_cast<int64_t>(r) * a.cols);
      *reinterpret_cast<uint2*>(a.hi + o) = *reinterpret_cast<const uint2*>(h);
      *reinterpret_cast<uint2*>(a.lo + o) = *reinterpret_cast<const uint2*>(l);
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
      __half h, l;
      split_half(one(!m || a.nesterov ? load1(g + i) : 0.f, m ? m[i] : 0.f), h, l);
      const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.cols);
      const int64_t o = xb + static_cast<int64_t>(r) * a.ld + (i - static_cast<int64_t>(r) * a.cols);
      a.hi[o] = h;
      a.lo[o] = l;
    }
  }
}

// ---------------------------------------------------------------------------
// The three products of a step, one matrix of the stack after another.
// ---------------------------------------------------------------------------
enum { kNsGram = 0, kNsPoly = 1, kNsApply = 2 };

constexpr int kNsBK = 64;
constexpr int kNsOpBytes = 128 * kNsBK * 2;  // 16 KB an operand, stage and CTA
constexpr int kNsStages = 6;
constexpr int kNsEpiWarps = 8;
constexpr int kNsThreads = 32 * (2 + kNsEpiWarps);
constexpr int kNsSmemBytes = kNsStages * 2 * kNsOpBytes + 256 + 1024;

struct NsParams {
  // [groups, rows, K] K-major (box 64 x 128) or [groups, K, cols] (box 64 x 64)
  CUtensorMap a, b;        // hi parts
  CUtensorMap a_lo, b_lo;  // SPLIT: lo parts
  int32_t M, N, ksteps;    // output extents; 64-wide steps of the contraction
  int32_t n_tiles, per_group, total;  // tiles
  const __half* in_hi;     // poly: A; apply: X
  const __half* in_lo;     // apply; SPLIT poly
  __half* out_hi;          // gram, poly: the symmetric result; apply: X'
  __half* out_lo;          // apply; SPLIT gram and poly
  const float* in_diag;    // not SPLIT: [groups, r] remainders of A's (poly) or B's (apply) diagonal
  float* out_diag;         // not SPLIT gram and poly
  int64_t ld, stride;      // of in_* and out_* (elements)
  __nv_bfloat16* out;      // last apply: [groups, M, N]
  const __nv_bfloat16* w;  // last apply: weights to update, or null (out = X)
  float alpha, beta;       // result = alpha * product + beta * in
  float diag_scale;        // apply: in_diag times this is added to beta
  float keep, step;        // weights: keep * w - step * X
  int32_t tall;            // apply: B stands on the right, its diagonal goes with the columns
  int32_t* status;
};

struct NsTile {
  int g, m0, n0;
};

// Symmetric results: only tiles on and above the diagonal are computed, and written twice.
template <int MODE, int TILE>
__device__ __forceinline__ NsTile ns_decode(const NsParams& p, int u) {
  NsTile t;
  t.g = u / p.per_group;
  int v = u - t.g * p.per_group;
  if (MODE == kNsApply) {
    t.m0 = v / p.n_tiles;
    t.n0 = (v - t.m0 * p.n_tiles) * TILE;
    t.m0 *= TILE;
  } else {
    int i = 0;
    while (v >= p.n_tiles - i) {
      v -= p.n_tiles - i;
      ++i;
    }
    t.m0 = i * TILE;
    t.n0 = (i + v) * TILE;
  }
  return t;
}

// kind::f16 instruction descriptor with fp16 operands.
template <bool A_MN, bool B_MN>
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// PAIR: clusters of two CTAs on 256 x 256 tiles (each CTA holds 128 rows of A and of B),
// otherwise one CTA on 128 x 128 tiles, with the SPLIT products.  Persistent; two accumulators in TMEM, so that
// one tile's epilogue overlaps the next one's products.
template <int MODE, bool A_MN, bool B_MN, bool PAIR, bool LAST>
__global__ void __launch_bounds__(kNsThreads, 1) ns_gemm_kernel(const __grid_constant__ NsParams p) {
  constexpr int TILE = PAIR ? 256 : 128;
  constexpr bool SPLIT = !PAIR;
  const int steps = (SPLIT ? 3 : 1) * p.ksteps;  // hi hi, then hi lo and lo hi
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kNsStages * 2 * kNsOpBytes);
  uint64_t* empty = full + kNsStages;
  uint64_t* acc_full = empty + kNsStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = PAIR ? blockIdx.x / 2 : blockIdx.x;
  const int step = PAIR ? gridDim.x / 2 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], PAIR ? 2 * kNsEpiWarps : kNsEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.a);
    tma_prefetch_desc(&p.b);
    if (SPLIT) {
      tma_prefetch_desc(&p.a_lo);
      tma_prefetch_desc(&p.b_lo);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * TILE);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * TILE);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t last[kNsStages];
#pragma unroll
      for (int s = 0; s < kNsStages; ++s) last[s] = 2;  // 2: nothing issued
      bool ok = true;
      for (int u = first; u < p.total && ok; u += step) {
        const NsTile t = ns_decode<MODE, TILE>(p, u);
        const int am = t.m0 + rank * 128, bn = t.n0 + rank * 128;
        for (int kk = 0; kk < steps; ++kk) {
          const int pass = SPLIT ? kk / p.ksteps : 0, k = kk - pass * p.ksteps;
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) { ok = false; break; }
          uint8_t* sa = ring + stage * 2 * kNsOpBytes;
          uint8_t* sb = sa + kNsOpBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], (PAIR ? 4 : 2) * kNsOpBytes);
          auto load = [&](uint8_t* dst, const CUtensorMap* map, bool mn, int row) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!mn && j) break;
              const int c0 = mn ? row + 64 * j : k * kNsBK, c1 = mn ? k * kNsBK : row;
              if constexpr (PAIR)
                tma_load_3d_pair(dst + 8192 * j, map, cluster_addr(&full[stage], 0), c0, c1, t.g, pol);
              else
                tma_load_3d(dst + 8192 * j, map, &full[stage], c0, c1, t.g, pol);
            }
          };
          load(sa, pass == 2 ? &p.a_lo : &p.a, A_MN, am);
          load(sb, pass == 1 ? &p.b_lo : &p.b, B_MN, bn);
#pragma unroll
          for (int s = 0; s < kNsStages; ++s)
            if (s == stage) last[s] = phase;
          if (++stage == kNsStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!PAIR) {
        // every load issued lands before the CTA may leave (bounded: 20 ms); pairs: the
        // issuer waits for every stage of either CTA, and the closing barrier for it
        const uint64_t t0 = global_timer_ns();
#pragma unroll
        for (int s = 0; s < kNsStages; ++s) {
          if (last[s] > 1) continue;
          while (!mbar_try_wait(&full[s], last[s]) && global_timer_ns() - t0 < 20000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (pairs: rank 0) ----------------
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_f16<A_MN, B_MN>(TILE, TILE);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = first; u < p.total && ok; u += step) {
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * TILE;
        for (int k = 0; k < steps; ++k) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + stage * 2 * kNsOpBytes);
          const uint32_t sb = sa + kNsOpBytes;
#pragma unroll
          for (int kk = 0; kk < kNsBK / 16; ++kk) {
            const uint64_t da = A_MN ? sdesc_mnmajor_sw128(sa + kk * 2048, 8192)
                                     : sdesc_kmajor_sw128(sa) + 2 * kk;
            const uint64_t db = B_MN ? sdesc_mnmajor_sw128(sb + kk * 2048, 8192)
                                     : sdesc_kmajor_sw128(sb) + 2 * kk;
            if constexpr (PAIR) mma_bf16_pair(d, da, db, idesc, (k | kk) != 0 ? 1u : 0u);
            else mma_bf16(d, da, db, idesc, (k | kk) != 0 ? 1u : 0u);
          }
          if constexpr (PAIR) {
            mma_commit_pair(cluster_addr(&empty[stage], 0));
            mma_commit_pair(cluster_addr(&empty[stage], 1));
          } else {
            mma_commit(&empty[stage]);
          }
          if (++stage == kNsStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if constexpr (PAIR) {
          mma_commit_pair(cluster_addr(&acc_full[acc], 0));
          mma_commit_pair(cluster_addr(&acc_full[acc], 1));
        } else {
          mma_commit(&acc_full[acc]);
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if constexpr (PAIR) mma_commit_pair(cluster_addr(drain, 0)); else mma_commit(drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < 20000000ull) {
      }
    }
  } else {
    // ---------------- epilogue ----------------
    const int quarter = warp & 3;      // TMEM lanes 32 * quarter ..
    const int half = (warp - 2) >> 2;  // column half of the tile
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < p.total; u += step) {
      const NsTile t = ns_decode<MODE, TILE>(p, u);
      const int m = t.m0 + rank * 128 + quarter * 32 + lane;
      const int64_t row = t.g * p.stride + static_cast<int64_t>(m) * p.ld;
      if (!mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * TILE + half * (TILE / 2);
#pragma unroll 1
      for (int c = 0; c < TILE / 2; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + c, r);
        tmem_ld_wait();
        const int n = t.n0 + half * (TILE / 2) + c;
        if (n >= p.N) continue;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = p.alpha * __uint_as_float(r[j]);
        if (MODE != kNsGram && m < p.M) {
          // rows of in_* are padded to whole 16-byte vectors
          const float* cd = p.in_diag + static_cast<int64_t>(t.g) * (MODE == kNsPoly || p.tall ? p.N : p.M);
          const float dm = SPLIT || (MODE == kNsApply && p.tall) ? 0.f : cd[m];
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (n + j >= p.N) break;
            const uint4 h4 = *reinterpret_cast<const uint4*>(p.in_hi + row + n + j);
            const __half2* h2 = reinterpret_cast<const __half2*>(&h4);
            uint4 l4 = make_uint4(0, 0, 0, 0);
            if (MODE == kNsApply || SPLIT) l4 = *reinterpret_cast<const uint4*>(p.in_lo + row + n + j);
            const __half2* l2 = reinterpret_cast<const __half2*>(&l4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x2 = __half22float2(h2[i / 2]), y2 = __half22float2(l2[i / 2]);
              float x = i & 1 ? x2.y : x2.x;
              if (MODE == kNsApply || SPLIT) x += i & 1 ? y2.y : y2.x;
              float f = p.beta;
              if (!SPLIT) {
                const float dn = (MODE == kNsPoly || p.tall) && n + j + i < p.N ? cd[n + j + i] : 0.f;
                if (MODE == kNsApply) {
                  f = fmaf(p.diag_scale, dm + dn, f);
                } else {  // (A + D)^2 = A^2 + D A + A D, and b D on the diagonal
                  f = fmaf(p.alpha, dm + dn, f);
                  if (n + j + i == m) v[j + i] = fmaf(p.beta, dm, v[j + i]);
                }
              }
              v[j + i] = fmaf(f, x, v[j + i]);
            }
          }
        }
        if constexpr (LAST) {
          if (m < p.M) {
            const int64_t o = (static_cast<int64_t>(t.g) * p.M + m) * p.N + n;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (n + j >= p.N) break;
              float x = v[j] * (1.f / kNsSx);
              if (p.w) x = fmaf(p.keep, __bfloat162float(p.w[o + j]), -p.step * x);
              p.out[o + j] = __float2bfloat16_rn(x);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (n + j >= p.N || m >= p.M) break;
            __align__(16) __half h[8], l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              split_half(v[j + i], h[i], l[i]);
              if (!SPLIT && MODE != kNsApply && n + j + i == m)
                p.out_diag[static_cast<int64_t>(t.g) * p.M + m] = v[j + i] - __half2float(h[i]);
            }
            *reinterpret_cast<uint4*>(p.out_hi + row + n + j) = *reinterpret_cast<const uint4*>(h);
            if (MODE == kNsApply || SPLIT)
              *reinterpret_cast<uint4*>(p.out_lo + row + n + j) = *reinterpret_cast<const uint4*>(l);
          }
          if (MODE != kNsApply && t.m0 != t.n0) {
            // the mirrored tile: 32 lanes write 64 consecutive bytes
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (n + j < p.N && m < p.M) {
                __half h, l;
                split_half(v[j], h, l);
                const int64_t o = t.g * p.stride + static_cast<int64_t>(n + j) * p.ld + m;
                p.out_hi[o] = h;
                if (SPLIT) p.out_lo[o] = l;
              }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(cluster_addr(&acc_empty[acc], 0));
        else mbar_arrive(&acc_empty[acc]);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  }

  tc_fence_before();
  if (PAIR) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 2 * TILE);
    else tmem_dealloc(tmem_base, 2 * TILE);
  }
}

}  // namespace moe
