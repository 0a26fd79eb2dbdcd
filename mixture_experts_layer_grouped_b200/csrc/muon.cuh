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
#include "grouped_gemm.cuh"  // packed f32x2 arithmetic
#include "wgrad.cuh"         // MN-major descriptors

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
constexpr int kNsEpiWarps = 8;
constexpr int kNsThreads = 32 * (2 + kNsEpiWarps);
constexpr int kNsBlkBytes = 32 * 32 * 2;     // an epilogue warp's block: 32 rows x 32 columns

// What a form of the kernel stages and how: its values are hi + lo (LO), it adds to the
// product what a block brings (IN); the blocks an epilogue warp keeps in flight, and the
// load stages in what they leave of shared memory.
template <int MODE, bool PAIR, bool LAST>
struct NsCfg {
  static constexpr int TILE = PAIR ? 256 : 128;
  static constexpr bool SPLIT = !PAIR;
  static constexpr bool LO = MODE == kNsApply || SPLIT;
  static constexpr bool IN = MODE != kNsGram;
  static constexpr int ARR = (LO ? 2 : 1) + (LAST ? 1 : 0);  // arrays of a block
  static constexpr int SETS = LAST ? 2 : (LO ? 3 : 4);
  static constexpr int STAGES = LO ? 4 : 5;
  static constexpr int STG = kNsEpiWarps * SETS * ARR * kNsBlkBytes;
  static constexpr int SMEM_BYTES = STAGES * 2 * kNsOpBytes + STG + kNsEpiWarps * 32 * 4 + 512 + 1024;
};

struct NsParams {
  // [groups, rows, K] K-major (box 64 x 128) or [groups, K, cols] (box 64 x 64)
  CUtensorMap a, b;        // hi parts
  CUtensorMap a_lo, b_lo;  // SPLIT: lo parts
  CUtensorMap sym;         // not SPLIT poly and apply: the symmetric operand with box 64 x 64
  // blocks of the epilogue (box 32 x 32, 64-byte swizzle)
  CUtensorMap in_hi;       // poly: A; apply: X
  CUtensorMap in_lo;       // apply; SPLIT poly
  CUtensorMap out_hi;      // gram, poly: the symmetric result; apply: X'; last apply: out, if tma_out
  CUtensorMap out_lo;      // apply; SPLIT gram and poly
  CUtensorMap w_in;        // last apply: w, if tma_out
  int32_t M, N, ksteps;    // output extents; 64-wide steps of the contraction
  int32_t n_tiles, per_group, total;  // tiles
  const float* in_diag;    // not SPLIT: [groups, r] remainders of A's (poly) or B's (apply) diagonal
  float* out_diag;         // not SPLIT gram and poly
  __nv_bfloat16* out;      // last apply: [groups, M, N]
  const __nv_bfloat16* w;  // last apply: weights to update, or null (out = X)
  int32_t tma_out;         // last apply: out and w have rows of whole 16-byte vectors
  float alpha, beta;       // result = alpha * product + beta * in
  float diag_scale;        // apply: in_diag times this is added to beta
  float keep, step;        // weights: keep * w - step * X
  int32_t* status;
};

struct NsTile {
  int g, m0, n0;
};

// Symmetric results: only tiles on and above the diagonal are computed and stored.
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

// TMA store of a staged block; committed groups are waited for until their shared memory
// is read (the buffer may be written again) or until their writes are done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t c0,
                                             int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>  // all but the N latest groups
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Orders this thread's accesses to shared memory before later TMA (async proxy) ones.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// kind::f16 instruction descriptor with fp16 operands, K-major or MN-major each.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// One of a step's products.  PAIR: clusters of two CTAs on 256 x 256 tiles (each CTA holds
// 128 rows of A and of B), otherwise one CTA on 128 x 128 tiles, with the SPLIT products.
// Persistent; two accumulators in TMEM, so that one tile's epilogue overlaps the next one's
// products.  TALL: X stands on the left (rows > cols).
//
// A symmetric operand (A, B of the formulas) has only its tiles on and above the diagonal in
// memory.  A k-step that needs rows of a tile below it loads the mirrored tile's rows and
// hands them to the tensor cores MN-major: nothing is ever transposed in software.
//
// Epilogue: blocks of 32 x 32.  A TMA load brings what a block adds to the product two blocks
// ahead, each lane works on one row of it in place, and a TMA store takes the result away
// while the next blocks are worked on; loads and stores clip at the matrix's edges.  (Plain
// loads and stores, one row a lane: 18 us a 256 x 256 tile, of which the products need 4.3.)
template <int MODE, bool TALL, bool PAIR, bool LAST>
__global__ void __launch_bounds__(kNsThreads, 1) ns_gemm_kernel(const __grid_constant__ NsParams p) {
  using C = NsCfg<MODE, PAIR, LAST>;
  constexpr int TILE = C::TILE;
  constexpr bool SPLIT = C::SPLIT, LO = C::LO, IN = C::IN;
  constexpr bool A_MN = MODE == kNsGram && TALL;
  constexpr bool B_MN = (MODE == kNsGram && TALL) || (MODE == kNsApply && !TALL);
  constexpr bool A_SYM = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && !TALL));
  constexpr bool B_SYM = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && TALL));
  constexpr bool COL_DIAG = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && TALL));
  constexpr bool ROW_DIAG = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && !TALL));
  const int steps = (SPLIT ? 3 : 1) * p.ksteps;  // hi hi, then hi lo and lo hi
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stg = ring + C::STAGES * 2 * kNsOpBytes;
  float* dcols = reinterpret_cast<float*>(stg + C::STG);  // [kNsEpiWarps][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(dcols + kNsEpiWarps * 32);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint64_t* in_full = drain + 1;           // [kNsEpiWarps][SETS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + kNsEpiWarps * C::SETS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = PAIR ? blockIdx.x / 2 : blockIdx.x;
  const int step = PAIR ? gridDim.x / 2 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], PAIR ? 2 * kNsEpiWarps : kNsEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kNsEpiWarps * C::SETS; ++i) mbar_init(&in_full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.a);
    tma_prefetch_desc(&p.b);
    tma_prefetch_desc(&p.out_hi);
    if (IN) tma_prefetch_desc(&p.in_hi);
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
      uint32_t last[C::STAGES];
#pragma unroll
      for (int s = 0; s < C::STAGES; ++s) last[s] = 2;  // 2: nothing issued
      bool ok = true;
      for (int u = first; u < p.total && ok; u += step) {
        const NsTile t = ns_decode<MODE, TILE>(p, u);
        const int am = t.m0 + rank * 128, bn = t.n0 + rank * 128;
        for (int kk = 0; kk < steps; ++kk) {
          const int pass = SPLIT ? kk / p.ksteps : 0, k = (kk - pass * p.ksteps) * kNsBK;
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) { ok = false; break; }
          uint8_t* sa = ring + stage * 2 * kNsOpBytes;
          uint8_t* sb = sa + kNsOpBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], (PAIR ? 4 : 2) * kNsOpBytes);
          auto load = [&](uint8_t* dst, const CUtensorMap* map, bool mn, int row) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!mn && j) break;
              const int c0 = mn ? row + 64 * j : k, c1 = mn ? k : row;
              if constexpr (PAIR)
                tma_load_3d_pair(dst + 8192 * j, map, cluster_addr(&full[stage], 0), c0, c1, t.g, pol);
              else
                tma_load_3d(dst + 8192 * j, map, &full[stage], c0, c1, t.g, pol);
            }
          };
          if (A_SYM && k < t.m0) load(sa, &p.sym, true, am);
          else load(sa, pass == 2 ? &p.a_lo : &p.a, A_MN, am);
          if (B_SYM && k < t.n0) load(sb, &p.sym, true, bn);
          else load(sb, pass == 1 ? &p.b_lo : &p.b, B_MN, bn);
#pragma unroll
          for (int s = 0; s < C::STAGES; ++s)
            if (s == stage) last[s] = phase;
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (!PAIR) {
        // every load issued lands before the CTA may leave (bounded: 20 ms); pairs: the
        // issuer waits for every stage of either CTA, and the closing barrier for it
        const uint64_t t0 = global_timer_ns();
#pragma unroll
        for (int s = 0; s < C::STAGES; ++s) {
          if (last[s] > 1) continue;
          while (!mbar_try_wait(&full[s], last[s]) && global_timer_ns() - t0 < 20000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (pairs: rank 0) ----------------
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = first; u < p.total && ok; u += step) {
        const NsTile t = ns_decode<MODE, TILE>(p, u);
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * TILE;
        for (int k = 0; k < steps; ++k) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + stage * 2 * kNsOpBytes);
          const uint32_t sb = sa + kNsOpBytes;
          const bool a_mn = A_MN || (A_SYM && k * kNsBK < t.m0);
          const bool b_mn = B_MN || (B_SYM && k * kNsBK < t.n0);
          const uint32_t idesc = idesc_f16(TILE, TILE, a_mn, b_mn);
          // 16 of K on: 32 bytes inside the swizzle atom, or two groups of eight 128-byte rows
          const uint64_t da = a_mn ? sdesc_mnmajor_sw128(sa, 8192) : sdesc_kmajor_sw128(sa);
          const uint64_t db = b_mn ? sdesc_mnmajor_sw128(sb, 8192) : sdesc_kmajor_sw128(sb);
          const uint32_t ka = a_mn ? 2048 >> 4 : 2, kb = b_mn ? 2048 >> 4 : 2;
#pragma unroll
          for (int kk = 0; kk < kNsBK / 16; ++kk) {
            const uint32_t accum = (k | kk) != 0 ? 1u : 0u;
            if constexpr (PAIR) mma_bf16_pair(d, da + kk * ka, db + kk * kb, idesc, accum);
            else mma_bf16(d, da + kk * ka, db + kk * kb, idesc, accum);
          }
          if constexpr (PAIR) {
            mma_commit_pair(cluster_addr(&empty[stage], 0));
            mma_commit_pair(cluster_addr(&empty[stage], 1));
          } else {
            mma_commit(&empty[stage]);
          }
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
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
    constexpr int BLKS = TILE / 64;    // blocks a warp has of a tile
    constexpr int AHEAD = C::SETS - 1;
    const int quarter = warp & 3;      // TMEM lanes 32 * quarter ..
    const int half = (warp - 2) >> 2;  // column half of the tile
    uint8_t* buf0 = stg + (warp - 2) * C::SETS * C::ARR * kNsBlkBytes;
    float* dcol = dcols + (warp - 2) * 32;
    uint64_t* my_full = in_full + (warp - 2) * C::SETS;
    const bool weights = LAST && p.w != nullptr;
    const uint64_t pol = l2_policy_evict_last();
    // 16-byte vector v of this lane's row of array b of a set (64-byte swizzle)
    auto vec = [&](uint8_t* set, int b, int v) -> uint4* {
      return reinterpret_cast<uint4*>(set + b * kNsBlkBytes + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4));
    };
    // the blocks asked for: a cursor AHEAD blocks in front (lane 0's loads, every lane's count)
    int lu = first, lc = 0, lset = 0, asked = 0, taken = 0;
    auto load_next = [&]() {
      if (lu >= p.total) return;
      if (lane == 0) {
        const NsTile t = ns_decode<MODE, TILE>(p, lu);
        const int m = t.m0 + rank * 128 + quarter * 32, n = t.n0 + half * (TILE / 2) + lc * 32;
        const bool w_too = weights && p.tma_out;
        uint8_t* set = buf0 + lset * C::ARR * kNsBlkBytes;
        uint64_t* bar = my_full + lset;
        mbar_arrive_expect_tx(bar, (1 + (LO ? 1 : 0) + (w_too ? 1 : 0)) * kNsBlkBytes);
        tma_load_3d(set, &p.in_hi, bar, n, m, t.g, pol);
        if (LO) tma_load_3d(set + kNsBlkBytes, &p.in_lo, bar, n, m, t.g, pol);
        if (w_too) tma_load_3d(set + 2 * kNsBlkBytes, &p.w_in, bar, n, m, t.g, pol);
      }
      ++asked;
      if (++lset == C::SETS) lset = 0;
      if (++lc == BLKS) { lc = 0; lu += step; }
    };
    if (IN)
      for (int i = 0; i < AHEAD; ++i) load_next();
    int acc = 0, set_i = 0;
    uint32_t acc_phase = 0, in_phase = 0;
    bool ok = true;
    const uint64_t alpha2 = f32x2_pack(p.alpha, p.alpha);
    for (int u = first; u < p.total && ok; u += step) {
      const NsTile t = ns_decode<MODE, TILE>(p, u);
      const int mw = t.m0 + rank * 128 + quarter * 32, m = mw + lane;
      const float* cd = p.in_diag + static_cast<int64_t>(t.g) * (COL_DIAG ? p.N : p.M);
      const float dm = ROW_DIAG && m < p.M ? __ldg(cd + m) : 0.f;
      const float f_row = fmaf(p.diag_scale, dm, p.beta);
      // (a lane that gave up takes its warp along)
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.status))) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BLKS; ++c) {
        const int n = t.n0 + half * (TILE / 2) + c * 32;
        uint8_t* set = buf0 + set_i * C::ARR * kNsBlkBytes;
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * TILE +
                               half * (TILE / 2) + c * 32, r);
        if (COL_DIAG) dcol[lane] = n + lane < p.N ? __ldg(cd + n + lane) : 0.f;
        if (IN) {
          ok = __all_sync(0xffffffffu, mbar_wait(my_full + set_i, in_phase, abort_flag, p.status));
          if (ok) ++taken;
        }
        tmem_ld_wait();
        if (!ok) break;
        if (c == BLKS - 1) {  // the accumulator is in registers: hand it back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR) mbar_arrive_cluster(cluster_addr(&acc_empty[acc], 0));
            else mbar_arrive(&acc_empty[acc]);
          }
        } else if (COL_DIAG) {
          __syncwarp();
        }
        const bool some = mw < p.M && n < p.N;
        const bool on_diag = MODE != kNsApply && mw == n;
        if (some) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // eight columns
            uint64_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = f32x2_mul(alpha2, f32x2_pack(__uint_as_float(r[8 * q + 2 * i]),
                                                  __uint_as_float(r[8 * q + 2 * i + 1])));
            if (IN) {
              const uint4 h4 = *vec(set, 0, q);
              uint4 l4 = make_uint4(0, 0, 0, 0);
              if (LO) l4 = *vec(set, 1, q);
              const __half2* h2 = reinterpret_cast<const __half2*>(&h4);
              const __half2* l2 = reinterpret_cast<const __half2*>(&l4);
              float d[8];
              if (COL_DIAG) {
                *reinterpret_cast<float4*>(d) = *reinterpret_cast<const float4*>(dcol + 8 * q);
                *reinterpret_cast<float4*>(d + 4) = *reinterpret_cast<const float4*>(dcol + 8 * q + 4);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 hf = __half22float2(h2[i]);
                uint64_t x = f32x2_pack(hf.x, hf.y);
                if (LO) {
                  const float2 lf = __half22float2(l2[i]);
                  x = f32x2_add(x, f32x2_pack(lf.x, lf.y));
                }
                // the remainders of the diagonals: X's rows or columns times theirs, or in
                // (A + D)^2 = A^2 + D A + A D
                uint64_t f = f32x2_pack(f_row, f_row);
                if (COL_DIAG)
                  f = f32x2_fma(f32x2_pack(p.diag_scale, p.diag_scale), f32x2_pack(d[2 * i], d[2 * i + 1]), f);
                v[i] = f32x2_fma(f, x, v[i]);
              }
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f32x2_unpack(v[i], y[2 * i], y[2 * i + 1]);
            if (MODE == kNsPoly && !SPLIT && on_diag && (lane >> 3) == q) {  // b D
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if ((lane & 7) == i) y[i] = fmaf(p.beta, dm, y[i]);
            }
            if constexpr (LAST) {
              if (weights && p.tma_out) {
                const uint4 w4 = *vec(set, 2, q);
                const __nv_bfloat162* w2 = reinterpret_cast<const __nv_bfloat162*>(&w4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 wf = __bfloat1622float2(w2[i]);
                  y[2 * i] = fmaf(p.keep, wf.x, -p.step * y[2 * i]);
                  y[2 * i + 1] = fmaf(p.keep, wf.y, -p.step * y[2 * i + 1]);
                }
              }
              if (p.tma_out) {
                *vec(set, 0, q) = make_uint4(bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]),
                                             bf16x2_bits(y[4], y[5]), bf16x2_bits(y[6], y[7]));
              } else {  // fp32 over the lane's own hi and lo vectors, written out below
                *reinterpret_cast<float4*>(vec(set, 0, q)) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(vec(set, 1, q)) = make_float4(y[4], y[5], y[6], y[7]);
              }
            } else {
              uint4 h4, l4;
              __half2* h2 = reinterpret_cast<__half2*>(&h4);
              __half2* l2 = reinterpret_cast<__half2*>(&l4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                h2[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
                if (LO) {
                  const float2 f = __half22float2(h2[i]);
                  l2[i] = __floats2half2_rn(y[2 * i] - f.x, y[2 * i + 1] - f.y);
                }
              }
              *vec(set, 0, q) = h4;
              if (LO) *vec(set, 1, q) = l4;
              if (MODE != kNsApply && !SPLIT && on_diag && (lane >> 3) == q && m < p.M) {
                const __half* hh = reinterpret_cast<const __half*>(&h4);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if ((lane & 7) == i)
                    p.out_diag[static_cast<int64_t>(t.g) * p.M + m] = y[i] - __half2float(hh[i]);
              }
            }
          }
        }
        if (LAST && !p.tma_out && some) {
          // rows of any alignment: one column a lane, one row after another
          __syncwarp();
          if (n + lane < p.N) {
            const int b = (lane >> 2) & 1, v8 = lane >> 3;
            for (int i = 0; i < 32 && mw + i < p.M; ++i) {
              const int64_t o = (static_cast<int64_t>(t.g) * p.M + mw + i) * p.N + n + lane;
              float x = *reinterpret_cast<const float*>(set + b * kNsBlkBytes + i * 64 +
                                                        ((v8 ^ ((i >> 1) & 3)) << 4) + (lane & 3) * 4);
              if (weights) x = fmaf(p.keep, __bfloat162float(p.w[o]), -p.step * x);
              p.out[o] = __float2bfloat16_rn(x);
            }
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (some && !(LAST && !p.tma_out)) {
            tma_store_3d(&p.out_hi, set, n, mw, t.g);
            if (LO && !LAST) tma_store_3d(&p.out_lo, set + kNsBlkBytes, n, mw, t.g);
          }
          bulk_commit();
          // the set that the next load (IN) or the next block uses: its store is done reading
          bulk_wait_read<IN ? 1 : C::SETS - 1>();
        }
        if (IN) load_next();
        __syncwarp();
        if (++set_i == C::SETS) { set_i = 0; in_phase ^= 1; }
      }
      if (!ok) break;
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (IN && lane == 0 && taken < asked) {
      // gave up: the blocks asked for land before the CTA may leave (20 ms at most)
      const uint64_t t0 = global_timer_ns();
      for (; taken < asked; ++taken)
        while (!mbar_try_wait(my_full + taken % C::SETS, (taken / C::SETS) & 1) &&
               global_timer_ns() - t0 < 20000000ull) {
        }
    }
    if (lane == 0) bulk_wait_all();
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
