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

#include <type_traits>

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
  int32_t* counters;        // zeroed here, for the products that follow
  int n_counters;
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
// range), added in an order fixed by the shape.  Four accesses in flight (mom_out may be
// mom_in, so the compiler may not move loads over stores itself), VEC: of four elements.
// HBM-bound: 2.7 GB in 0.45 ms (32 x [2048, 4096], bf16 gradients: 5.9 TB/s).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) muon_norm_kernel(const __grid_constant__ MuonInArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double red[8];
  const int mat = blockIdx.y;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * gridDim.y * 256;
  for (int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
       i < a.n_counters; i += threads)
    a.counters[i] = 0;
  const int64_t base = static_cast<int64_t>(mat) * a.n;
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
    for (int64_t j = i0 + threadIdx.x * 4; j < i1; j += 4096) {
      float4 gv[4], mv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 1024;
        gv[k] = mv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < i1) gv[k] = load4<T>(g + i);
        if (i < i1 && a.mom_in) mv[k] = __ldcs(reinterpret_cast<const float4*>(a.mom_in + base + i));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 1024;
        float4 mo, u;
        u.x = one(gv[k].x, mv[k].x, mo.x);
        u.y = one(gv[k].y, mv[k].y, mo.y);
        u.z = one(gv[k].z, mv[k].z, mo.z);
        u.w = one(gv[k].w, mv[k].w, mo.w);
        if (a.mom_in && i < i1) *reinterpret_cast<float4*>(a.mom_out + base + i) = mo;
        s += static_cast<double>(u.x) * u.x + static_cast<double>(u.y) * u.y +
             static_cast<double>(u.z) * u.z + static_cast<double>(u.w) * u.w;
      }
    }
  } else {
    for (int64_t j = i0 + threadIdx.x; j < i1; j += 1024) {
      float gv[4], mv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 256;
        gv[k] = i < i1 ? load1(g + i) : 0.f;
        mv[k] = i < i1 && a.mom_in ? a.mom_in[base + i] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 256;
        float mo = 0.f;
        const float u = one(gv[k], mv[k], mo);
        if (a.mom_in && i < i1) a.mom_out[base + i] = mo;
        s += static_cast<double>(u) * u;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane_id() == 0) red[warp_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 8; ++i) s += red[i];
    a.part[static_cast<int64_t>(mat) * a.chunks + blockIdx.x] = s;
  }
}

// x = hi + lo in fp16, each rounded to nearest (lo is subnormal below 2^-29 of 1: 2^-40 off).
__device__ __forceinline__ void split_half(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(x - __half2float(hi));
}

// u again, over its norm, as hi and lo parts; HBM-bound (2.7 GB in 0.47 ms at the same sizes:
// 5.7 TB/s).  Both passes a few matrices at a time, so that this one reads L2: no faster (the
// whole step of 64 x [2048, 1024] 3.88 ms against 3.91).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) muon_scale_kernel(const __grid_constant__ MuonInArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double red[8];
  const int mat = blockIdx.y;
  const int64_t base = static_cast<int64_t>(mat) * a.n;
  double s = 0.0;
  for (int i = threadIdx.x; i < a.chunks; i += 256)
    s += a.part[static_cast<int64_t>(mat) * a.chunks + i];
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
  const int64_t xb = static_cast<int64_t>(mat) * rows * a.ld;
  auto one = [&](float gv, float mo) -> float {
    return scale * (!m ? gv : (a.nesterov ? fmaf(a.beta, mo, gv) : mo));
  };
  if constexpr (VEC) {
    for (int64_t j = i0 + threadIdx.x * 4; j < i1; j += 4096) {
      float4 gv[4], mo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 1024;
        gv[k] = mo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < i1 && (!m || a.nesterov)) gv[k] = load4<T>(g + i);
        if (i < i1 && m) mo[k] = *reinterpret_cast<const float4*>(m + i);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 1024;
        __align__(8) __half h[4], l[4];
        split_half(one(gv[k].x, mo[k].x), h[0], l[0]);
        split_half(one(gv[k].y, mo[k].y), h[1], l[1]);
        split_half(one(gv[k].z, mo[k].z), h[2], l[2]);
        split_half(one(gv[k].w, mo[k].w), h[3], l[3]);
        if (i >= i1) continue;
        const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.cols);
        const int64_t o = xb + static_cast<int64_t>(r) * a.ld + (i - static_cast<int64_t>(r) * a.cols);
        __stcs(reinterpret_cast<uint2*>(a.hi + o), *reinterpret_cast<const uint2*>(h));
        __stcs(reinterpret_cast<uint2*>(a.lo + o), *reinterpret_cast<const uint2*>(l));
      }
    }
  } else {
    for (int64_t j = i0 + threadIdx.x; j < i1; j += 1024) {
      float gv[4], mo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 256;
        gv[k] = i < i1 && (!m || a.nesterov) ? load1(g + i) : 0.f;
        mo[k] = i < i1 && m ? m[i] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = j + k * 256;
        if (i >= i1) continue;
        __half h, l;
        split_half(one(gv[k], mo[k]), h, l);
        const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.cols);
        const int64_t o = xb + static_cast<int64_t>(r) * a.ld + (i - static_cast<int64_t>(r) * a.cols);
        a.hi[o] = h;
        a.lo[o] = l;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The products of all steps, in one persistent kernel.
// ---------------------------------------------------------------------------
enum { kNsGram = 0, kNsPoly = 1, kNsApply = 2, kNsSum = 3 };

constexpr int kNsBK = 64;
constexpr int kNsOpBytes = 128 * kNsBK * 2;  // 16 KB an operand, stage and CTA
constexpr int kNsStages = 4;
constexpr int kNsEpiWarps = 8;
constexpr int kNsThreads = 32 * (2 + kNsEpiWarps);
constexpr int kNsBlkBytes = 32 * 32 * 2;     // an epilogue warp's block: 32 rows x 32 columns
constexpr int kNsWarpBytes = 6 * kNsBlkBytes;  // the blocks it has in flight
constexpr int kNsSets = 4;                   // at most, of one to three arrays each
constexpr int kNsMaxSplits = 8;
constexpr int kNsSmemBytes = kNsStages * 2 * kNsOpBytes + kNsEpiWarps * (kNsWarpBytes + 32 * 4) + 768 + 1024;

// Work units in order: for each step, the Gram tiles of all matrices (`splits` units each, and
// with more than one `sums` units that add them up), the polynomial's tiles, the application's
// tiles.  Symmetric results: only tiles on and above the diagonal.  CTAs (or pairs) claim units
// in this order, so what a claimed unit waits for was claimed before by a running CTA, and
// every wait ends.
struct NsParams {
  // [groups, rows, K] K-major (box 64 x 128) or [groups, K, cols] (box 64 x 64); [buffer][hi, lo]
  CUtensorMap x_gram[2][2], x_apply[2][2];
  CUtensorMap ab_op[2][2];   // A and B [hi, lo]; lo only with SPLIT
  CUtensorMap ab_mir[2];     // A and B with box 64 x 64, for the tiles below the diagonal
  // blocks of the epilogue (box 32 x 32, 64-byte swizzle)
  CUtensorMap x_blk[2][2], ab_blk[2][2];
  CUtensorMap out_map, w_map;  // last application, if tma_out
  int32_t groups, rows, cols, r, steps;
  int32_t sym_tiles, sym_n, app_tiles, app_n;  // tiles a matrix (n: tiles along a side, along columns)
  int32_t k_gram, k_r;                         // 64-wide steps of the contractions
  int32_t splits, sums;                        // sums: 0 with one split
  int32_t total;
  int32_t* unit_counter;       // [1]: claims
  int32_t* done;               // [groups][3 * steps]: epilogue warps that finished a unit
  int32_t* split_done;         // [groups][sym_tiles]: epilogue warps that left a partial tile
  float4* partial;             // [groups][sym_tiles][splits][tile]
  float* diag[2];              // [groups, r]: remainders of A's and B's diagonals (not SPLIT)
  __nv_bfloat16* out;          // [groups, rows, cols]
  const __nv_bfloat16* w;      // weights to update, or null (out = X)
  int32_t tma_out;             // out and w have rows of whole 16-byte vectors
  float a, b, c;
  float keep, step;            // weights: keep * w - step * X
  int32_t* status;
};

struct NsUnit {
  int k, mode, g, tile, split, m0, n0;
};

template <int TILE>
__device__ __forceinline__ NsUnit ns_decode(const NsParams& p, int u) {
  NsUnit t;
  const int per = p.sym_tiles * (p.splits + p.sums + 1) + p.app_tiles;  // units a matrix and step
  const int n = p.groups;
  t.k = u / (n * per);
  int v = u - t.k * n * per;
  t.split = 0;
  if (v < n * p.sym_tiles * p.splits) {
    t.mode = kNsGram;
    t.g = v / (p.sym_tiles * p.splits);
    v -= t.g * p.sym_tiles * p.splits;
    t.tile = v / p.splits;
    t.split = v - t.tile * p.splits;
  } else if ((v -= n * p.sym_tiles * p.splits) < n * p.sym_tiles * p.sums) {
    t.mode = kNsSum;  // split: the block column of the tile that it adds up
    t.g = v / (p.sym_tiles * p.sums);
    v -= t.g * p.sym_tiles * p.sums;
    t.tile = v / p.sums;
    t.split = v - t.tile * p.sums;
  } else if ((v -= n * p.sym_tiles * p.sums) < n * p.sym_tiles) {
    t.mode = kNsPoly;
    t.g = v / p.sym_tiles;
    t.tile = v - t.g * p.sym_tiles;
  } else {
    v -= n * p.sym_tiles;
    t.mode = kNsApply;
    t.g = v / p.app_tiles;
    t.tile = v - t.g * p.app_tiles;
  }
  if (t.mode == kNsApply) {
    t.m0 = t.tile / p.app_n;
    t.n0 = (t.tile - t.m0 * p.app_n) * TILE;
    t.m0 *= TILE;
  } else {
    int i = 0, w = t.tile;
    while (w >= p.sym_n - i) {
      w -= p.sym_n - i;
      ++i;
    }
    t.m0 = i * TILE;
    t.n0 = (i + w) * TILE;
  }
  return t;
}

// 64-wide steps [k0, k1) of the contraction of a unit (of one pass).
__device__ __forceinline__ void ns_ksteps(const NsParams& p, const NsUnit& t, int& k0, int& k1) {
  k0 = 0;
  k1 = p.k_r;
  if (t.mode == kNsGram) {
    k0 = p.k_gram * t.split / p.splits;
    k1 = p.k_gram * (t.split + 1) / p.splits;
  }
}

// counter_wait with short sleeps: a wait here is on the way of everything that follows.
__device__ __forceinline__ bool ns_wait(const int32_t* p, int32_t target, volatile int* abort,
                                        int32_t* status) {
  uint64_t t0 = 0;
  for (int i = 0;; ++i) {
    int32_t v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= target) return true;
    if (*abort) return false;
    if (i == 0) {
      t0 = global_timer_ns();
    } else if (global_timer_ns() - t0 > 2000000000ull) {
      *abort = 1;
      set_status(status, MOE_ERR_TIMEOUT);
      return false;
    }
    __nanosleep(20);
  }
}

// What a unit reads is written: the product before it, of the same matrix, is complete.
// (The applications before that one, too: each product waits for the one before.)
template <int WARPS>
__device__ __forceinline__ bool ns_ready(const NsParams& p, const NsUnit& t, volatile int* abort) {
  if (t.mode == kNsSum)
    return ns_wait(p.split_done + static_cast<int64_t>(t.g) * p.sym_tiles + t.tile,
                        (t.k + 1) * p.splits * WARPS, abort, p.status);
  const int phase = 3 * t.k + t.mode;
  if (phase == 0) return true;
  const int units = t.mode == kNsGram ? p.app_tiles
                                      : p.sym_tiles * (t.mode == kNsPoly && p.sums > 0 ? p.sums : 1);
  const bool ok = ns_wait(p.done + static_cast<int64_t>(t.g) * 3 * p.steps + phase - 1, units * WARPS,
                               abort, p.status);
  fence_proxy_async_global();
  return ok;
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

// Adds one to a counter, after this thread's earlier writes (and those it knows of).
__device__ __forceinline__ void counter_add(int32_t* p) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}

// PAIR: clusters of two CTAs on 256 x 256 tiles (each CTA holds 128 rows of A and of B),
// otherwise one CTA on 128 x 128 tiles.  SPLIT: products of hi and lo parts (see the top).
// Two accumulators in TMEM, so that one unit's epilogue overlaps the next one's products.
// TALL: X stands on the left.
//
// One kernel for all steps: a launch each took 12 us at 5 x [333, 215] (set-up, cold
// instructions, drain) for 2 us of products; and a matrix goes on as soon as its own tiles
// are done, not when the slowest of the stack are.
//
// A symmetric operand (A, B of the formulas) has only its tiles on and above the diagonal in
// memory.  A k-step that needs rows of a tile below it loads the mirrored tile's rows and
// hands them to the tensor cores MN-major: nothing is ever transposed in software.
//
// Few tiles and a long contraction (one wide matrix): a Gram tile is `splits` units that leave
// their fp32 sums in memory, and a unit for each block column adds them in order.
//
// Epilogue: blocks of 32 x 32.  A TMA load brings what a block adds to the product, ahead of
// it, each lane works on one row of it in place, and a TMA store takes the result away: with
// the others where the warp's blocks of a tile fit its buffers, otherwise while the next
// blocks are worked on.  Loads and stores clip at the matrix's edges.  (Plain
// loads and stores, one row a lane: 18 us a 256 x 256 tile, of which the products need 4.3.)
//
// Bound: 64 x [2048, 1024] 2.9 ms (0.82 PFLOP/s of the formulas' products), 32 x [2048, 4096] 9.0 ms
// (1.07 PFLOP/s): a k-step of a pair takes 670-780 clocks for its 64 KB from L2, 512 of the tensor
// pipe, at the clock that the power cap leaves.  One small stack or matrix: 15 dependent products
// of 7 to 14 us, most of it a unit's way in and out.
template <bool TALL, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kNsThreads, 1) ns_steps_kernel(const __grid_constant__ NsParams p) {
  constexpr int TILE = PAIR ? 256 : 128;
  constexpr int WARPS = PAIR ? 2 * kNsEpiWarps : kNsEpiWarps;  // epilogue warps of a unit
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stg = ring + kNsStages * 2 * kNsOpBytes;
  float* dcols = reinterpret_cast<float*>(stg + kNsEpiWarps * kNsWarpBytes);  // [kNsEpiWarps][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(dcols + kNsEpiWarps * 32);
  uint64_t* empty = full + kNsStages;
  uint64_t* acc_full = empty + kNsStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_empty + 2;
  uint64_t* in_full = drain + 1;           // [kNsEpiWarps][kNsSets]
  uint64_t* sched_full = in_full + kNsEpiWarps * kNsSets;  // [kSched]
  uint64_t* sched_empty = sched_full + kSched;             // [kSched]
  int* sched_u = reinterpret_cast<int*>(sched_empty + kSched);  // [kSched]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sched_u + kSched);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], WARPS);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kNsEpiWarps * kNsSets; ++i) mbar_init(&in_full[i], 1);
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&sched_full[i], 1);
      mbar_init(&sched_empty[i], PAIR ? 2 * (1 + kNsEpiWarps) : 1 + kNsEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
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
  TileQueue tq{sched_full, sched_empty, sched_u, 0, 0u, 0, 0, true};
  // (A or B) is a symmetric operand of a mode
  auto a_sym = [](int mode) { return !SPLIT && (mode == kNsPoly || (mode == kNsApply && !TALL)); };
  auto b_sym = [](int mode) { return !SPLIT && (mode == kNsPoly || (mode == kNsApply && TALL)); };
  auto a_is_mn = [](int mode) { return mode == kNsGram && TALL; };
  auto b_is_mn = [](int mode) { return (mode == kNsGram && TALL) || (mode == kNsApply && !TALL); };

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
      while (ok) {
        const int u = rank == 0 ? claim_tile<PAIR>(tq, p, p.total, abort_flag, ok)
                                : next_tile<PAIR>(tq, p, p.total, rank, false, abort_flag);
        if (u >= p.total) break;
        const NsUnit t = ns_decode<TILE>(p, u);
        if (t.mode == kNsSum) continue;
        if (!ns_ready<WARPS>(p, t, abort_flag)) break;
        const int am = t.m0 + rank * 128, bn = t.n0 + rank * 128, in = t.k & 1;
        // operands [hi, lo]
        const CUtensorMap* ma[2] = {&p.x_gram[in][0], &p.x_gram[in][1]};
        const CUtensorMap* mb[2] = {ma[0], ma[1]};
        const CUtensorMap* sym = &p.ab_mir[0];
        if (t.mode != kNsGram) {
          const int m = t.mode == kNsPoly ? 0 : 1;  // A, or B
          sym = &p.ab_mir[m];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            ma[j] = mb[j] = &p.ab_op[m][j];
            if (t.mode == kNsApply) (TALL ? ma : mb)[j] = &p.x_apply[in][j];
          }
        }
        const bool amn = a_is_mn(t.mode), bmn = b_is_mn(t.mode), as = a_sym(t.mode), bs = b_sym(t.mode);
        int k0, k1;
        ns_ksteps(p, t, k0, k1);
        for (int pass = 0; pass < (SPLIT ? 3 : 1) && ok; ++pass) {  // hi hi, then hi lo and lo hi
          for (int kk = k0; kk < k1; ++kk) {
            const int k = kk * kNsBK;
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
            const bool at = as && k < t.m0, bt = bs && k < t.n0;  // below the diagonal
            load(sa, at ? sym : ma[pass == 2], amn || at, am);
            load(sb, bt ? sym : mb[pass == 1], bmn || bt, bn);
#pragma unroll
            for (int s = 0; s < kNsStages; ++s)
              if (s == stage) last[s] = phase;
            if (++stage == kNsStages) { stage = 0; phase ^= 1; }
          }
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
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok) {
        const int u = next_tile<PAIR>(tq, p, p.total, 0, false, abort_flag);
        if (u >= p.total) break;
        const NsUnit t = ns_decode<TILE>(p, u);
        if (t.mode == kNsSum) continue;
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * TILE;
        const bool amn = a_is_mn(t.mode), bmn = b_is_mn(t.mode), as = a_sym(t.mode), bs = b_sym(t.mode);
        int k0, k1;
        ns_ksteps(p, t, k0, k1);
        uint32_t accum = 0u;
        for (int pass = 0; pass < (SPLIT ? 3 : 1) && ok; ++pass) {
          for (int k = k0; k < k1; ++k) {
            if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(ring + stage * 2 * kNsOpBytes);
            const uint32_t sb = sa + kNsOpBytes;
            const bool a_mn = amn || (as && k * kNsBK < t.m0);
            const bool b_mn = bmn || (bs && k * kNsBK < t.n0);
            const uint32_t idesc = idesc_f16(TILE, TILE, a_mn, b_mn);
            // 16 of K on: 32 bytes inside the swizzle atom, or two groups of eight 128-byte rows
            const uint64_t da = a_mn ? sdesc_mnmajor_sw128(sa, 8192) : sdesc_kmajor_sw128(sa);
            const uint64_t db = b_mn ? sdesc_mnmajor_sw128(sb, 8192) : sdesc_kmajor_sw128(sb);
            const uint32_t ka = a_mn ? 2048 >> 4 : 2, kb = b_mn ? 2048 >> 4 : 2;
#pragma unroll
            for (int kk = 0; kk < kNsBK / 16; ++kk) {
              if constexpr (PAIR) mma_bf16_pair(d, da + kk * ka, db + kk * kb, idesc, accum);
              else mma_bf16(d, da + kk * ka, db + kk * kb, idesc, accum);
              accum = 1u;
            }
            if constexpr (PAIR) {
              mma_commit_pair(cluster_addr(&empty[stage], 0));
              mma_commit_pair(cluster_addr(&empty[stage], 1));
            } else {
              mma_commit(&empty[stage]);
            }
            if (++stage == kNsStages) { stage = 0; phase ^= 1; }
          }
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
    const int quarter = warp & 3;      // TMEM lanes 32 * quarter ..
    const int half = (warp - 2) >> 2;  // column half of the tile
    uint8_t* buf0 = stg + (warp - 2) * kNsWarpBytes;
    float* dcol = dcols + (warp - 2) * 32;
    uint64_t* my_full = in_full + (warp - 2) * kNsSets;
    const uint64_t pol = l2_policy_evict_last();
    uint32_t in_phase = 0;             // a bit for each set
    int acc = 0;
    uint32_t acc_phase = 0;
    // 16-byte vector v of this lane's row of array b of a set (64-byte swizzle)
    auto vec = [&](uint8_t* set, int b, int v) -> uint4* {
      return reinterpret_cast<uint4*>(set + b * kNsBlkBytes + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4));
    };

    // A unit's blocks; false: gave up.  MODE kNsSum is the Gram tile's epilogue on sums of parts.
    auto work = [&](const NsUnit& t, auto mode_c, auto last_c) -> bool {
      constexpr int MODE = decltype(mode_c)::value;
      constexpr bool LAST = decltype(last_c)::value;
      constexpr bool GRAM = MODE == kNsGram || MODE == kNsSum;
      constexpr bool LO = MODE == kNsApply || SPLIT;  // values are hi + lo
      constexpr bool IN = !GRAM;
      constexpr int ARR = (LO ? 2 : 1) + (LAST ? 1 : 0);
      constexpr int SETS = BLKS < 6 / ARR ? BLKS : 6 / ARR;
      constexpr bool ALL = SETS == BLKS;              // every block has its own buffers
      constexpr int AHEAD = ALL ? SETS : SETS - 1;
      constexpr bool COL_DIAG = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && TALL));
      constexpr bool ROW_DIAG = !SPLIT && (MODE == kNsPoly || (MODE == kNsApply && !TALL));
      static_assert(SETS <= kNsSets, "blocks of a warp");
      const int M = MODE == kNsApply ? p.rows : p.r, N = MODE == kNsApply ? p.cols : p.r;
      const int in = t.k & 1;
      const CUtensorMap *in_hi = nullptr, *in_lo = nullptr, *out_hi, *out_lo;
      float alpha, beta = 0.f, diag_scale = 0.f;
      if (GRAM) {
        out_hi = &p.ab_blk[0][0];
        out_lo = &p.ab_blk[0][1];
        alpha = kNsSa / (kNsSx * kNsSx);
      } else if (MODE == kNsPoly) {
        in_hi = &p.ab_blk[0][0];
        in_lo = &p.ab_blk[0][1];
        out_hi = &p.ab_blk[1][0];
        out_lo = &p.ab_blk[1][1];
        alpha = p.c * (kNsSb / (kNsSa * kNsSa));
        beta = p.b * (kNsSb / kNsSa);
        diag_scale = alpha;
      } else {
        constexpr float f = LAST ? 1.f / kNsSx : 1.f;  // the last one is X itself
        in_hi = &p.x_blk[in][0];
        in_lo = &p.x_blk[in][1];
        out_hi = LAST ? &p.out_map : &p.x_blk[in ^ 1][0];
        out_lo = &p.x_blk[in ^ 1][1];
        alpha = f / kNsSb;
        beta = p.a * f;
        diag_scale = alpha;
      }
      const bool weights = LAST && p.w != nullptr, tma_out = !LAST || p.tma_out;
      const int mw = t.m0 + rank * 128 + quarter * 32, m = mw + lane;
      const int nw = t.n0 + half * (TILE / 2);
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * TILE +
                             half * (TILE / 2);
      int asked = 0, taken = 0;
      auto load_next = [&]() {  // lane 0
        const int c = asked++, set_i = c % SETS;
        uint8_t* set = buf0 + set_i * ARR * kNsBlkBytes;
        uint64_t* bar = my_full + set_i;
        mbar_arrive_expect_tx(bar, ((LO ? 2 : 1) + (weights && tma_out ? 1 : 0)) * kNsBlkBytes);
        tma_load_3d(set, in_hi, bar, nw + 32 * c, mw, t.g, pol);
        if (LO) tma_load_3d(set + kNsBlkBytes, in_lo, bar, nw + 32 * c, mw, t.g, pol);
        if (weights && tma_out) tma_load_3d(set + 2 * kNsBlkBytes, &p.w_map, bar, nw + 32 * c, mw, t.g, pol);
      };
      auto store = [&](int c) {  // lane 0
        uint8_t* set = buf0 + (c % SETS) * ARR * kNsBlkBytes;
        if (mw < M && nw + 32 * c < N && tma_out) {
          tma_store_3d(out_hi, set, nw + 32 * c, mw, t.g);
          if (LO && !LAST) tma_store_3d(out_lo, set + kNsBlkBytes, nw + 32 * c, mw, t.g);
        }
      };
      bool ok = true;
      if (IN || MODE == kNsSum) {
        if (lane == 0) ok = ns_ready<WARPS>(p, t, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        __syncwarp();  // what lane 0 has seen, the warp has
        if (IN && ok && lane == 0)
          for (int i = 0; i < AHEAD; ++i) load_next();
      }
      // A's or B's diagonal remainders (rewritten every step: no ldg)
      const float* cd = p.diag[MODE == kNsPoly ? 0 : 1] + static_cast<int64_t>(t.g) * p.r;
      const float dm = ROW_DIAG && ok && m < M ? __ldcg(cd + m) : 0.f;
      float dn[BLKS];
#pragma unroll
      for (int c = 0; c < BLKS; ++c)
        dn[c] = COL_DIAG && ok && nw + 32 * c + lane < N ? __ldcg(cd + nw + 32 * c + lane) : 0.f;
      const float f_row = fmaf(diag_scale, dm, beta);
      // (a lane that gave up takes its warp along)
      if (MODE != kNsSum) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.status));
        tc_fence_after();
      }
      const uint64_t alpha2 = f32x2_pack(alpha, alpha);
      const int c_first = MODE == kNsSum ? t.split : 0, c_end = MODE == kNsSum ? t.split + 1 : BLKS;
#pragma unroll 1
      for (int c = c_first; c < c_end && ok; ++c) {
        const int n = nw + c * 32, set_i = c % SETS;
        uint8_t* set = buf0 + set_i * ARR * kNsBlkBytes;
        const bool some = mw < M && n < N;
        uint32_t wv[LAST ? 16 : 1];  // weights of any alignment: one column a lane, two rows a word
        if (LAST && weights && !tma_out && some && n + lane < N) {
          const int64_t o = (static_cast<int64_t>(t.g) * M + mw) * N + n + lane;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint32_t w0 = mw + i < M ? __bfloat16_as_ushort(p.w[o + static_cast<int64_t>(i) * N]) : 0u;
            const uint32_t w1 = mw + i + 1 < M ? __bfloat16_as_ushort(p.w[o + static_cast<int64_t>(i + 1) * N]) : 0u;
            wv[LAST ? i / 2 : 0] = w0 | (w1 << 16);
          }
        }
        if (COL_DIAG) {
          float d = dn[0];
#pragma unroll
          for (int i = 1; i < BLKS; ++i)
            if (c == i) d = dn[i];
          dcol[lane] = d;
        }
        if (IN) {
          ok = __all_sync(0xffffffffu, mbar_wait(my_full + set_i, (in_phase >> set_i) & 1, abort_flag, p.status));
          if (!ok) break;
          in_phase ^= 1u << set_i;
          ++taken;
        }
        __syncwarp();
        const bool on_diag = MODE != kNsApply && mw == n;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 16 columns
          uint32_t r[16];
          if constexpr (MODE == kNsSum) {
            // parts as the other CTAs' same warps and lanes left them: [split][block][h][4][lane]
            const float4* part = p.partial +
                (static_cast<int64_t>(t.g) * p.sym_tiles + t.tile) * p.splits * (TILE * TILE / 4) +
                (rank * kNsEpiWarps + warp - 2) * (BLKS * 256) + (2 * c + h) * 128 + lane;
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 x = __ldcg(part + static_cast<int64_t>(s) * (TILE * TILE / 4) + 32 * i);
                v[i].x += x.x;
                v[i].y += x.y;
                v[i].z += x.z;
                v[i].w += x.w;
              }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[4 * i] = __float_as_uint(v[i].x);
              r[4 * i + 1] = __float_as_uint(v[i].y);
              r[4 * i + 2] = __float_as_uint(v[i].z);
              r[4 * i + 3] = __float_as_uint(v[i].w);
            }
          } else {
            tmem_ld_32x32b_x16(taddr + 32 * c + 16 * h, r);
            tmem_ld_wait();
          }
          if (!some) continue;
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {  // eight columns
            const int q = 2 * h + qq;
            uint64_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = f32x2_mul(alpha2, f32x2_pack(__uint_as_float(r[8 * qq + 2 * i]),
                                                  __uint_as_float(r[8 * qq + 2 * i + 1])));
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
                  f = f32x2_fma(f32x2_pack(diag_scale, diag_scale), f32x2_pack(d[2 * i], d[2 * i + 1]), f);
                v[i] = f32x2_fma(f, x, v[i]);
              }
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f32x2_unpack(v[i], y[2 * i], y[2 * i + 1]);
            if (MODE == kNsPoly && !SPLIT && on_diag && (lane >> 3) == q) {  // b D
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if ((lane & 7) == i) y[i] = fmaf(beta, dm, y[i]);
            }
            if constexpr (LAST) {
              if (weights && tma_out) {
                const uint4 w4 = *vec(set, 2, q);
                const __nv_bfloat162* w2 = reinterpret_cast<const __nv_bfloat162*>(&w4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 wf = __bfloat1622float2(w2[i]);
                  y[2 * i] = fmaf(p.keep, wf.x, -p.step * y[2 * i]);
                  y[2 * i + 1] = fmaf(p.keep, wf.y, -p.step * y[2 * i + 1]);
                }
              }
              if (tma_out) {
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
              if (MODE != kNsApply && !SPLIT && on_diag && (lane >> 3) == q && m < M) {
                const __half* hh = reinterpret_cast<const __half*>(&h4);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if ((lane & 7) == i)
                    p.diag[MODE == kNsPoly ? 1 : 0][static_cast<int64_t>(t.g) * p.r + m] =
                        y[i] - __half2float(hh[i]);
              }
            }
          }
        }
        if (MODE != kNsSum && c == BLKS - 1) {  // the accumulator is read: hand it back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR) mbar_arrive_cluster(cluster_addr(&acc_empty[acc], 0));
            else mbar_arrive(&acc_empty[acc]);
          }
        }
        if (LAST && !tma_out && some) {
          __syncwarp();
          if (n + lane < N) {
            const int b = (lane >> 2) & 1, v8 = lane >> 3;
            const int64_t o = (static_cast<int64_t>(t.g) * M + mw) * N + n + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x = *reinterpret_cast<const float*>(set + b * kNsBlkBytes + i * 64 +
                                                        ((v8 ^ ((i >> 1) & 3)) << 4) + (lane & 3) * 4);
              if (weights)
                x = fmaf(p.keep, __uint_as_float(i & 1 ? wv[LAST ? i / 2 : 0] & 0xFFFF0000u : wv[LAST ? i / 2 : 0] << 16),
                         -p.step * x);
              if (mw + i < M) p.out[o + static_cast<int64_t>(i) * N] = __float2bfloat16_rn(x);
            }
          }
        }
        if (!ALL) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            store(c);
            bulk_commit();
            bulk_wait_read<1>();  // the store before: the set that the next load uses
            if (asked < BLKS) load_next();
          }
        }
        __syncwarp();
      }
      if (ALL && ok) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          for (int c = c_first; c < c_end; ++c) store(c);
          bulk_commit();
        }
      }
      if (IN && !ok && lane == 0) {
        // gave up: the blocks asked for land before the CTA may leave (20 ms at most)
        const uint64_t t0 = global_timer_ns();
        for (; taken < asked; ++taken) {
          const int set_i = taken % SETS;
          while (!mbar_try_wait(my_full + set_i, (in_phase >> set_i) & 1) &&
                 global_timer_ns() - t0 < 20000000ull) {
          }
          in_phase ^= 1u << set_i;
        }
      }
      return ok;
    };

    // A part of a Gram tile: the accumulator as it is, [block][h][4][lane] of float4 a warp.
    auto leave_part = [&](const NsUnit& t) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.status))) return false;
      tc_fence_after();
      float4* part = p.partial +
          ((static_cast<int64_t>(t.g) * p.sym_tiles + t.tile) * p.splits + t.split) * (TILE * TILE / 4) +
          (rank * kNsEpiWarps + warp - 2) * (BLKS * 256) + lane;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * TILE +
                             half * (TILE / 2);
#pragma unroll 1
      for (int c = 0; c < 2 * BLKS; ++c) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(taddr + 16 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          part[c * 128 + 32 * i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                               __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(cluster_addr(&acc_empty[acc], 0));
        else mbar_arrive(&acc_empty[acc]);
        counter_add(p.split_done + static_cast<int64_t>(t.g) * p.sym_tiles + t.tile);
      }
      return true;
    };

    while (true) {
      const int u = next_tile<PAIR>(tq, p, p.total, rank, true, abort_flag);
      if (u >= p.total) break;
      const NsUnit t = ns_decode<TILE>(p, u);
      using std::integral_constant;
      using No = integral_constant<bool, false>;
      bool ok;
      if (t.mode == kNsGram && p.sums > 0) {
        ok = leave_part(t);
      } else {
        if (t.mode == kNsSum) ok = work(t, integral_constant<int, kNsSum>(), No());
        else if (t.mode == kNsGram) ok = work(t, integral_constant<int, kNsGram>(), No());
        else if (t.mode == kNsPoly) ok = work(t, integral_constant<int, kNsPoly>(), No());
        else if (t.k + 1 < p.steps) ok = work(t, integral_constant<int, kNsApply>(), No());
        else ok = work(t, integral_constant<int, kNsApply>(), integral_constant<bool, true>());
        if (ok && lane == 0) {
          // the stores are done, and seen before the count is (also by other CTAs' TMA loads)
          bulk_wait_all();
          fence_proxy_async_global();
          counter_add(p.done + static_cast<int64_t>(t.g) * 3 * p.steps + 3 * t.k +
                      (t.mode == kNsSum ? static_cast<int>(kNsGram) : t.mode));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (t.mode != kNsSum && ++acc == 2) { acc = 0; acc_phase ^= 1; }
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
