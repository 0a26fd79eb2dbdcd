// Orthogonalised updates of matrices with at most 128 rows or 128 columns (r of them; n is
// the other extent), in three kernels.  X_5 = Q X_0 where Q is a polynomial of S = X_0 X_0^T,
// and with S_k = X_k X_k^T the steps never touch X:
//
//   P = a I + b S + c S^2,   Q <- P Q,   S <- P S P       (all r x r, all commuting),
//
//   muon_gram_kernel    momentum; partial sums of u u^T over 128-wide pieces of n;
//   muon_chain_kernel   one CTA a matrix: S = sum / (|u|_F + eps)^2 (the trace is |u|_F^2),
//                       then every step in shared memory and TMEM;
//   muon_apply_kernel   X = Q u / (|u|_F + eps) and the weights, 128-wide pieces of n.
//
// So u is read twice whatever the number of steps, and nothing of it is stored between.
// Every product takes fp16 hi and lo parts (hi hi + hi lo + lo hi, 22 bits): the square roots
// of S's roundings are what small singular values see, and with 11 bits those would be gone.
// Measured against 64 bits: 1e-6 (full rank) to 1e-3 (rank 1), far below the bf16 result.
// Measured: 16 x [128, 256] fp32 58 us (the chain takes most of it);
// 64 x [100, 7000] with momentum and weights 0.40 ms (1.1 GB: 2.7 TB/s).
// The pieces are scaled by a power of two from their largest value; partial sums carry the
// exponent, so the range of fp32 gradients is covered.
#pragma once

#include "muon.cuh"
#include "route_scored.cuh"  // warp_sum

namespace moe {

constexpr int kMsThreads = 512;
constexpr int kMsWarps = kMsThreads / 32;
constexpr int kMsSlots = 128 / kMsWarps;     // rows of a piece that a warp loads
constexpr int kMsBlock = 128 * 128;          // bytes of 128 rows x 64 fp16
constexpr int kMsImage = 2 * kMsBlock;       // 128 x 128 fp16: two such blocks
constexpr int kMsMaxParts = 16;              // CTAs that share a matrix's sum
constexpr float kMsSs = 16384.f, kMsSp = 4096.f, kMsSt = 8192.f;  // scales of S, P, P S

struct MuonSmallArgs {
  const void* grad;         // [groups, rows, cols] fp32 or bf16
  const float* mom_in;      // or null: no momentum
  float* mom_out;
  const __nv_bfloat16* w;   // or null: out = X
  __nv_bfloat16* out;
  float4* part;             // [slots, 8, 512]: a CTA's sums of a matrix, 32 a thread
  int32_t* part_exp;        // [slots]: the sums are u u^T 2^(2 exp)
  uint8_t* q;               // [groups, 2, kMsImage]: Q's shared-memory images, hi and lo
  double* inv_norm;         // [groups]: 1 / (|u|_F + eps), over Q's scale
  int rows, cols, r, r16, pieces, steps;  // r16: r rounded up to 16
  int64_t units;            // groups * pieces, dealt to the CTAs in equal runs
  int gram_ctas;            // CTAs of the gram kernel
  int tall, nesterov;
  float beta, a, b, c, eps, keep, step, sq;      // sq: scale of Q
  int32_t* status;
};

// Byte offset of element (row, col) in an image: blocks of 64 columns, 128-byte swizzle.
__device__ __forceinline__ int ms_at(int row, int col) {
  return (col >> 6) * kMsBlock + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}

__device__ __forceinline__ float pow2f(int e) {  // 2^e, e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Eight neighbouring fp32 values as hi and lo parts of an image pair.
__device__ __forceinline__ void ms_store8(uint8_t* hi, uint8_t* lo, int row, int col, const float (&v)[8]) {
  uint4 h4, l4;
  __half2* h = reinterpret_cast<__half2*>(&h4);
  __half2* l = reinterpret_cast<__half2*>(&l4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    const float2 f = __half22float2(h[i]);
    l[i] = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
  }
  const int at = ms_at(row, col);
  *reinterpret_cast<uint4*>(hi + at) = h4;
  *reinterpret_cast<uint4*>(lo + at) = l4;
}
// Four of them.
__device__ __forceinline__ void ms_store4(uint8_t* hi, uint8_t* lo, int row, int col, float4 v) {
  const __half2 h0 = __floats2half2_rn(v.x, v.y), h1 = __floats2half2_rn(v.z, v.w);
  const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
  const __half2 l0 = __floats2half2_rn(v.x - f0.x, v.y - f0.y), l1 = __floats2half2_rn(v.z - f1.x, v.w - f1.y);
  const int at = ms_at(row, col);
  *reinterpret_cast<uint2*>(hi + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&h0),
                                                  *reinterpret_cast<const uint32_t*>(&h1));
  *reinterpret_cast<uint2*>(lo + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&l0),
                                                  *reinterpret_cast<const uint32_t*>(&l1));
}

// D (+)= A B^T over K of two image pairs, hi hi + hi lo + lo hi (one thread issues).
template <bool A_MN, bool B_MN>
__device__ __forceinline__ void ms_mma(uint32_t d, uint32_t a_hi, uint32_t a_lo, uint32_t b_hi,
                                       uint32_t b_lo, int N, int K) {
  const uint32_t idesc = idesc_f16(128, N, A_MN, B_MN);
  uint32_t accum = 0u;
  for (int pass = 0; pass < 3; ++pass) {
    const uint32_t a = pass == 2 ? a_lo : a_hi, b = pass == 1 ? b_lo : b_hi;
    for (int k = 0; k < K; k += 16) {
      // K-major: 16 of K inside a block, 64 to the next block; MN-major: rows of 128 bytes
      const uint64_t da = A_MN ? sdesc_mnmajor_sw128(a + k * 128, kMsBlock)
                               : sdesc_kmajor_sw128(a + (k >> 6) * kMsBlock) + ((k & 63) >> 3);
      const uint64_t db = B_MN ? sdesc_mnmajor_sw128(b + k * 128, kMsBlock)
                               : sdesc_kmajor_sw128(b + (k >> 6) * kMsBlock) + ((k & 63) >> 3);
      mma_bf16(d, da, db, idesc, accum);
      accum = 1u;
    }
  }
}

// What u of a 128 x 128 piece is made of, eight rows a warp and four columns a lane: asked for
// here, used by ms_form, so that a piece's loads run beside the one before it.  FIRST: the
// momentum is formed and written, otherwise it is read back.
struct MsRaw {
  float4 g[kMsSlots], m[kMsSlots];
};

template <typename T, bool VEC, bool FIRST>
__device__ __forceinline__ void ms_load(const MuonSmallArgs& a, int g, int piece, MsRaw& u) {
  const int warp = warp_id(), lane = lane_id();
  const int r0 = a.tall ? piece * 128 : 0, c0 = a.tall ? 0 : piece * 128;
  const int64_t base = static_cast<int64_t>(g) * a.rows * a.cols;
  const T* grad = static_cast<const T*>(a.grad) + base;
  const float* mom = (FIRST ? a.mom_in : a.mom_out);
  const bool need_g = FIRST || !mom || a.nesterov;
  const int col = c0 + 4 * lane;
  const int r_end = min(a.rows, r0 + 128);
#pragma unroll
  for (int i = 0; i < kMsSlots; ++i) {
    const int row = r0 + warp + kMsWarps * i;
    u.g[i] = u.m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row >= r_end || col >= a.cols) continue;
    const int64_t at = static_cast<int64_t>(row) * a.cols + col;
    if constexpr (VEC) {
      if (need_g) u.g[i] = load4<T>(grad + at);
      if (mom) u.m[i] = *reinterpret_cast<const float4*>(mom + base + at);
    } else {
      float* up = &u.g[i].x;
      float* mp = &u.m[i].x;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < a.cols) {
          if (need_g) up[j] = load1(grad + at + j);
          if (mom) mp[j] = mom[base + at + j];
        }
    }
  }
}

// u in place of the gradient; FIRST: the new momentum goes out.
template <bool VEC, bool FIRST>
__device__ __forceinline__ void ms_form(const MuonSmallArgs& a, int g, int piece, MsRaw& u) {
  if (!a.mom_in) return;
  const int warp = warp_id(), lane = lane_id();
  const int r0 = a.tall ? piece * 128 : 0, c0 = a.tall ? 0 : piece * 128;
  const int64_t base = static_cast<int64_t>(g) * a.rows * a.cols;
  const int col = c0 + 4 * lane;
  const int r_end = min(a.rows, r0 + 128);
#pragma unroll
  for (int i = 0; i < kMsSlots; ++i) {
    const int row = r0 + warp + kMsWarps * i;
    float* up = &u.g[i].x;
    float* mp = &u.m[i].x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (FIRST) mp[j] = fmaf(a.beta, mp[j], up[j]);
      up[j] = a.nesterov ? fmaf(a.beta, mp[j], up[j]) : mp[j];
    }
    if (FIRST && row < r_end && col < a.cols) {
      const int64_t at = base + static_cast<int64_t>(row) * a.cols + col;
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(a.mom_out + at) = u.m[i];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < a.cols) a.mom_out[at + j] = mp[j];
      }
    }
  }
}

// The piece's image pair, scaled so that its largest value is in [2^13, 2^14); returns the
// exponent of the scale.  Rows past what the products read are left out.
__device__ __forceinline__ int ms_image(const MuonSmallArgs& a, const float4 (&u)[kMsSlots], uint8_t* hi, uint8_t* lo,
                                        float* red) {
  const int warp = warp_id(), lane = lane_id();
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kMsSlots; ++i)
    m = fmaxf(fmaxf(fmaxf(m, fabsf(u[i].x)), fmaxf(fabsf(u[i].y), fabsf(u[i].z))), fabsf(u[i].w));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < kMsWarps; ++i) m = fmaxf(m, red[i]);
  // exponent of the largest value (an infinity or zero: no scale; far below fp32: clamped)
  const int em = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  const int e = (m == 0.f || em == 128) ? 0 : min(13 - em, 126);
  const float s = pow2f(max(e, -126));
  const int rows = a.tall ? 128 : a.r16;
#pragma unroll
  for (int i = 0; i < kMsSlots; ++i) {
    const int row = warp + kMsWarps * i;
    if (row >= rows) break;
    ms_store4(hi, lo, row, 4 * lane, make_float4(u[i].x * s, u[i].y * s, u[i].z * s, u[i].w * s));
  }
  return max(e, -126);
}

// Shared parts of the three kernels: TMEM, one mbarrier for the products, flags.
struct MsCtl {
  uint64_t bar;
  uint32_t tmem;
  int abort;
  float red[kMsWarps];
};

__device__ __forceinline__ uint32_t ms_begin(MsCtl* ctl, uint32_t cols) {
  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp_id() == 0) {
    tmem_alloc(&ctl->tmem, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return ctl->tmem;
}
__device__ __forceinline__ void ms_end(uint32_t tmem, uint32_t cols) {
  tc_fence_before();
  __syncthreads();
  if (warp_id() == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}
// The products issued since the last call are done, for the whole block (false: gave up).
__device__ __forceinline__ bool ms_wait(MsCtl* ctl, uint32_t& phase, int32_t* status) {
  const bool ok = mbar_wait(&ctl->bar, phase, &ctl->abort, status);
  phase ^= 1;
  const bool all = __syncthreads_and(ok);
  tc_fence_after();
  return all;
}
// Shared memory written by the block is what the tensor cores read next.
__device__ __forceinline__ void ms_publish() {
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

constexpr int kMsCtlBytes = 256;
constexpr int kMsGramSmem = 1024 + 2 * kMsImage + kMsCtlBytes;
constexpr int kMsChainSmem = 1024 + 6 * kMsImage + kMsCtlBytes;
constexpr int kMsApplySmem = 1024 + 4 * kMsImage + kMsCtlBytes;

__device__ __forceinline__ uint8_t* ms_smem(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// The units (matrix, piece) of CTA b of n: equal runs.
__device__ __forceinline__ int64_t ms_first(const MuonSmallArgs& a, int b, int n) {
  return a.units * b / n;
}

// A CTA takes a run of units; for each matrix that it meets it leaves its sums in slot
// (CTA + matrix), which no other pair has.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMsThreads, 1) muon_gram_kernel(const __grid_constant__ MuonSmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* hi = ms_smem(smem_raw);
  uint8_t* lo = hi + kMsImage;
  MsCtl* ctl = reinterpret_cast<MsCtl*>(lo + kMsImage);
  const uint32_t tmem = ms_begin(ctl, 128);
  pdl_wait();
  pdl_trigger();
  const int warp = warp_id(), lane = lane_id();
  const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
  const int64_t u0 = ms_first(a, blockIdx.x, a.gram_ctas), u1 = ms_first(a, blockIdx.x + 1, a.gram_ctas);
  float acc[32];
  int exp = 0;
  uint32_t phase = 0;
  MsRaw u;
  int g = static_cast<int>(u0 / a.pieces), piece = static_cast<int>(u0 - static_cast<int64_t>(g) * a.pieces);
  bool first = true;
  if (u0 < u1) ms_load<T, VEC, true>(a, g, piece, u);
  for (int64_t v = u0; v < u1; ++v) {
    ms_form<VEC, true>(a, g, piece, u);
    const int e = ms_image(a, u.g, hi, lo, ctl->red);
    const int g_next = piece + 1 == a.pieces ? g + 1 : g, p_next = piece + 1 == a.pieces ? 0 : piece + 1;
    if (v + 1 < u1) ms_load<T, VEC, true>(a, g_next, p_next, u);
    ms_publish();
    if (threadIdx.x == 0) {
      const uint32_t h = smem_u32(hi), l = smem_u32(lo);
      if (a.tall) ms_mma<true, true>(tmem, h, l, h, l, a.r16, 128);
      else ms_mma<false, false>(tmem, h, l, h, l, a.r16, 128);
      mma_commit(&ctl->bar);
    }
    if (!ms_wait(ctl, phase, a.status)) break;
    // the sums keep the smaller exponent: what has the larger one is scaled down
    float f_acc = 1.f, f_new = 1.f;
    if (first) {
      exp = e;
    } else if (e < exp) {
      f_acc = 2 * (e - exp) < -126 ? 0.f : pow2f(2 * (e - exp));
      exp = e;
    } else {
      f_new = 2 * (exp - e) < -126 ? 0.f : pow2f(2 * (exp - e));
    }
    uint32_t d[32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, d);
    tmem_ld_wait();
    if (first) {
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = __uint_as_float(d[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(d[j]), f_new, acc[j] * f_acc);
    }
    first = false;
    if (g_next != g || v + 1 == u1) {
      const int64_t slot = static_cast<int64_t>(blockIdx.x) + g;
      float4* dst = a.part + slot * (8 * kMsThreads) + threadIdx.x;
      if (row < a.r16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + 4 * i < a.r16)
            dst[i * kMsThreads] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      }
      if (threadIdx.x == 0) a.part_exp[slot] = exp;
      first = true;
    }
    g = g_next;
    piece = p_next;
    tc_fence_before();
    __syncthreads();  // images and TMEM may be written again
    tc_fence_after();
  }
  ms_end(tmem, 128);
}

// One CTA a matrix.  A thread holds a quarter of a row of S in fp32; P, Q and S (or P S) live
// in shared memory as image pairs.  Three dependent products a step: at r = 128 each reads
// 192 KB of shared memory (1536 clk of its bandwidth) and 256 KB of new images are written.
// Latency: 48 us for the 14 of five steps, however few the matrices.  (r <= 32 in fp32 on the
// ordinary cores: 16 rows 29 -> 24 us a call, but 64 x [32, 2000] 74 -> 81.)
__global__ void __launch_bounds__(kMsThreads, 1) muon_chain_kernel(const __grid_constant__ MuonSmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = ms_smem(smem_raw);
  uint8_t *s_hi = base, *s_lo = base + kMsImage, *p_hi = base + 2 * kMsImage, *p_lo = base + 3 * kMsImage,
          *q_hi = base + 4 * kMsImage, *q_lo = base + 5 * kMsImage;
  MsCtl* ctl = reinterpret_cast<MsCtl*>(base + 6 * kMsImage);
  const uint32_t tmem = ms_begin(ctl, 256);
  pdl_wait();
  pdl_trigger();
  const int warp = warp_id(), lane = lane_id(), g = blockIdx.x;
  const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
  const bool mine = row < a.r16 && c0 < a.r16;
  const bool warp_mine = (warp & 3) * 32 < a.r16 && c0 < a.r16;  // (TMEM loads are whole warps')
  const int vecs = mine ? min(4, (a.r16 - c0) / 8) : 0;  // of eight columns
  // S: the CTAs' sums under one exponent.  CTA b met this matrix if its run does.
  const int64_t v0 = static_cast<int64_t>(g) * a.pieces, v1 = v0 + a.pieces;
  int b0 = static_cast<int>(v0 * a.gram_ctas / a.units), b1 = static_cast<int>(v1 * a.gram_ctas / a.units);
  while (b0 > 0 && ms_first(a, b0, a.gram_ctas) > v0) --b0;
  while (ms_first(a, b0 + 1, a.gram_ctas) <= v0) ++b0;
  while (b1 < a.gram_ctas && ms_first(a, b1, a.gram_ctas) < v1) ++b1;
  while (b1 > b0 + 1 && ms_first(a, b1 - 1, a.gram_ctas) >= v1) --b1;
  int exp = 126;
  for (int b = b0; b < b1; ++b) exp = min(exp, __ldg(a.part_exp + b + g));
  float s[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = 0.f;
#pragma unroll 2
  for (int b = b0; b < b1; ++b) {
    const int64_t slot = static_cast<int64_t>(b) + g;
    const int d = 2 * (exp - __ldg(a.part_exp + slot));
    const float f = d < -126 ? 0.f : pow2f(d);
    const float4* src = a.part + slot * (8 * kMsThreads) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < 2 * vecs) {
        const float4 v = __ldg(src + i * kMsThreads);
        s[4 * i] = fmaf(v.x, f, s[4 * i]);
        s[4 * i + 1] = fmaf(v.y, f, s[4 * i + 1]);
        s[4 * i + 2] = fmaf(v.z, f, s[4 * i + 2]);
        s[4 * i + 3] = fmaf(v.w, f, s[4 * i + 3]);
      }
  }
  // |u|^2 2^(2 exp) is the trace; the row's diagonal entry is the lane-th column of its quarter
  float diag = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (lane == i) diag = s[i];
  if (!mine || (warp >> 2) != (warp & 3)) diag = 0.f;
  diag = warp_sum(diag);
  if (lane == 0) ctl->red[warp] = diag;
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < kMsWarps; ++i) trace += ctl->red[i];
  const double up = ldexp(1.0, -exp);
  const double inv = 1.0 / (sqrt(trace) * up + a.eps);
  if (threadIdx.x == 0) a.inv_norm[g] = inv / a.sq;
  const float f0 = static_cast<float>(up * inv);  // (its square may be past fp32)
  const uint32_t S[2] = {smem_u32(s_hi), smem_u32(s_lo)}, P[2] = {smem_u32(p_hi), smem_u32(p_lo)},
                 Q[2] = {smem_u32(q_hi), smem_u32(q_lo)};
  const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
  auto put = [&](uint8_t* hi, uint8_t* lo, const float (&v)[32], float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= vecs) break;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = v[8 * i + j] * f;
      ms_store8(hi, lo, row, c0 + 8 * i, x);
    }
  };
  auto read = [&](uint32_t col, float (&v)[32]) {  // this thread's part of the accumulator there
    uint32_t d[32];
    tmem_ld_32x32b_x32(taddr + col, d);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(d[i]);
  };
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = s[i] * f0 * f0;
  put(s_hi, s_lo, s, kMsSs);
  uint32_t phase = 0;
  ms_publish();
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    float v[32];
    // P = a I + b S + c S^2; the first Q is the first P
    if (threadIdx.x == 0) {
      ms_mma<false, false>(tmem, S[0], S[1], S[0], S[1], a.r16, a.r16);
      mma_commit(&ctl->bar);
    }
    if (!ms_wait(ctl, phase, a.status)) break;
    if (warp_mine) {
      read(0, v);
      const float cs = a.c / (kMsSs * kMsSs);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = fmaf(cs, v[i], a.b * s[i]);
      if ((warp >> 2) == (warp & 3) && row < a.r) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (lane == i) v[i] += a.a;
      }
      put(p_hi, p_lo, v, kMsSp);
      if (k == 0) put(q_hi, q_lo, v, a.sq);
    }
    ms_publish();
    if (k == 0 && last) break;
    // Q' = P Q and T = P S (into S's images, which are read by then)
    if (threadIdx.x == 0) {
      if (k > 0) ms_mma<false, false>(tmem, P[0], P[1], Q[0], Q[1], a.r16, a.r16);
      if (!last) ms_mma<false, false>(tmem + 128, P[0], P[1], S[0], S[1], a.r16, a.r16);
      mma_commit(&ctl->bar);
    }
    if (!ms_wait(ctl, phase, a.status)) break;
    if (warp_mine && k > 0) {
      read(0, v);
      put(q_hi, q_lo, v, 1.f / kMsSp);
    }
    if (last) break;
    if (warp_mine) {
      read(128, v);
      put(s_hi, s_lo, v, kMsSt / (kMsSp * kMsSs));
    }
    ms_publish();
    // S' = T P
    if (threadIdx.x == 0) {
      ms_mma<false, false>(tmem, S[0], S[1], P[0], P[1], a.r16, a.r16);
      mma_commit(&ctl->bar);
    }
    if (!ms_wait(ctl, phase, a.status)) break;
    if (warp_mine) {
      read(0, s);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] *= 1.f / (kMsSt * kMsSp);
      put(s_hi, s_lo, s, kMsSs);
    }
    ms_publish();
  }
  __syncthreads();
  // Q's images as they are (rows past r16 are not read)
  uint4* dst = reinterpret_cast<uint4*>(a.q + static_cast<int64_t>(g) * 2 * kMsImage);
  for (int i = threadIdx.x; i < 2 * kMsImage / 16; i += kMsThreads)
    if ((i * 16 % kMsBlock) / 128 < a.r16) dst[i] = *reinterpret_cast<const uint4*>(q_hi + 16 * i);
  ms_end(tmem, 256);
}

// X of a run of units: Q times the piece (or the piece times Q), in fp32 through shared memory
// to rows of 512 bytes, so that weights and results move whole row segments.  The next
// piece's loads run beside the product and the stores.
template <typename T, bool VEC, bool OUT_VEC>
__global__ void __launch_bounds__(kMsThreads, 1) muon_apply_kernel(const __grid_constant__ MuonSmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* hi = ms_smem(smem_raw);
  uint8_t *lo = hi + kMsImage, *q_hi = hi + 2 * kMsImage;
  MsCtl* ctl = reinterpret_cast<MsCtl*>(hi + 4 * kMsImage);
  const uint32_t tmem = ms_begin(ctl, 128);
  pdl_wait();
  pdl_trigger();
  const int warp = warp_id(), lane = lane_id();
  const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
  const int64_t u0 = ms_first(a, blockIdx.x, gridDim.x), u1 = ms_first(a, blockIdx.x + 1, gridDim.x);
  uint32_t phase = 0;
  MsRaw u;
  int g = static_cast<int>(u0 / a.pieces), piece = static_cast<int>(u0 - static_cast<int64_t>(g) * a.pieces);
  int g_q = -1;
  double inv = 0.0;
  if (u0 < u1) ms_load<T, VEC, false>(a, g, piece, u);
  for (int64_t v = u0; v < u1; ++v) {
    if (g != g_q) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(g) * 2 * kMsImage);
      for (int i = threadIdx.x; i < 2 * kMsImage / 16; i += kMsThreads)
        if ((i * 16 % kMsBlock) / 128 < a.r16) *reinterpret_cast<uint4*>(q_hi + 16 * i) = __ldg(src + i);
      inv = a.inv_norm[g];
      g_q = g;
    }
    ms_form<VEC, false>(a, g, piece, u);
    const int e = ms_image(a, u.g, hi, lo, ctl->red);
    const int g_next = piece + 1 == a.pieces ? g + 1 : g, p_next = piece + 1 == a.pieces ? 0 : piece + 1;
    if (v + 1 < u1) ms_load<T, VEC, false>(a, g_next, p_next, u);
    ms_publish();
    if (threadIdx.x == 0) {
      const uint32_t h = smem_u32(hi), l = smem_u32(lo), qh = smem_u32(q_hi), ql = qh + kMsImage;
      if (a.tall) ms_mma<false, false>(tmem, h, l, qh, ql, a.r16, a.r16);
      else ms_mma<false, true>(tmem, qh, ql, h, l, 128, a.r16);
      mma_commit(&ctl->bar);
    }
    const float f = static_cast<float>(inv * ldexp(1.0, -e));
    if (!ms_wait(ctl, phase, a.status)) break;
    const int r0 = a.tall ? piece * 128 : 0, n0 = a.tall ? 0 : piece * 128;
    const int rows = min(128, a.rows - r0), cols = min(128, a.cols - n0);
    uint32_t d[32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, d);
    tmem_ld_wait();
    if (row < rows && c0 < cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4*>(hi + row * 512 + ((c0 / 4 + i) ^ (row & 7)) * 16) =
            make_float4(f * __uint_as_float(d[4 * i]), f * __uint_as_float(d[4 * i + 1]),
                        f * __uint_as_float(d[4 * i + 2]), f * __uint_as_float(d[4 * i + 3]));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int64_t base = static_cast<int64_t>(g) * a.rows * a.cols;
#pragma unroll
    for (int k = 0; k < kMsSlots; ++k) {
      const int i = warp + kMsWarps * k, col = 4 * lane;
      if (i >= rows || col >= cols) break;
      const float4 x4 = *reinterpret_cast<const float4*>(hi + i * 512 + ((lane ^ (i & 7)) * 16));
      float x[4] = {x4.x, x4.y, x4.z, x4.w};
      const int64_t at = base + static_cast<int64_t>(r0 + i) * a.cols + n0 + col;
      if constexpr (OUT_VEC) {
        if (a.w) {
          const float4 wv = load4<__nv_bfloat16>(a.w + at);
          const float wf[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = fmaf(a.keep, wf[j], -a.step * x[j]);
        }
        *reinterpret_cast<uint2*>(a.out + at) = make_uint2(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < cols) {
            if (a.w) x[j] = fmaf(a.keep, __bfloat162float(a.w[at + j]), -a.step * x[j]);
            a.out[at + j] = __float2bfloat16_rn(x[j]);
          }
      }
    }
    g = g_next;
    piece = p_next;
    __syncthreads();  // the image is written again
  }
  ms_end(tmem, 128);
}

}  // namespace moe
