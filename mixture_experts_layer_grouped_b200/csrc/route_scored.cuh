// Routing by softmax or sigmoid scores with optional bias, groups and
// renormalisation, its gradient, and the balance loss (the router of
// TransformerEngine PR "DeepSeekV3Layer", Description, DeepSeekV3MoE bullet, in
// the forms route_select_kernel does not have; the balance loss is the same PR's
// sequence-wise auxiliary loss).  Host side in route_scored_api.cuh.
//
//   score     s_e = 1 / (1 + exp(-l_e))   or   exp(l_e - max l) / sum exp(l - max l);
//             a logit of -inf or NaN is a masked expert: no score, never selected;
//   key       l_e without a bias (both scores grow strictly with the logit, so the order
//             of the logits is the order of the scores, with nothing rounded),
//             s_e + bias_e with one (-inf or NaN: never selected);
//   groups    the kept ones have the largest sum of their group_top largest keys
//             (without a bias and with group_top 2: of their largest scores);
//   gate      rsf * s_e, divided by the sum over the selected when renormalised.
//
// The selection is that of exact arithmetic as far as 64 bits resolve it: keys are
// computed in 32 bits with a known error, and a row in which two neighbours of the
// sorted keys, or the groups on both sides of the border, are nearer than that error
// is done again in 64 bits (measured at 256 experts, top 8 and a bias: under 1% of rows).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kRsWarps = 4;  // rows (warps) per block of the row kernels

struct ScoredArgs {
  const float* logits;    // [T, E] (when n_splits == 0)
  const float* partials;  // [n_splits, T, E] router GEMM partial sums (n_splits > 0)
  float* logits_out;      // [T, E] sum of the partials, in split order (n_splits > 0)
  int n_splits;
  const float* bias;      // [E] or null
  int32_t* topk_idx;      // [T, k]
  float* topk_w;          // [T, k]
  int T, E, G, g, k, size;  // size = E / G
  uint32_t size_magic;    // ceil(2^32 / size): e / size == umulhi(e, magic) for e < 1024
  float rsf;
  int score, renorm, group_top;
};

__device__ __forceinline__ float exp_k(float x) { return expf(x); }
__device__ __forceinline__ double exp_k(double x) { return exp(x); }

// Order-preserving unsigned image of a key; 0 is below every key's and means "none".
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);  // -0 and +0 are one key
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v == 0.0 ? 0.0 : v));
  return u ^ ((u >> 63) ? 0xFFFFFFFFFFFFFFFFull : 0x8000000000000000ull);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <typename K> struct KeyOf;
template <> struct KeyOf<float> { using U = uint32_t; };
template <> struct KeyOf<double> { using U = uint64_t; };

__device__ __forceinline__ uint32_t warp_max_key(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(mh) << 32) | ml;
}

template <typename K>
__device__ __forceinline__ K warp_sum(K v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// e^(l - m) with m the largest logit; 1 at the maximum, also when it is +inf.
template <typename K>
__device__ __forceinline__ K exp_below(float l, float m) {
  return l == m ? K(1) : exp_k(K(l) - K(m));
}
template <typename K>
__device__ __forceinline__ K sigmoid_k(float l) {
  return K(1) / (K(1) + exp_k(-K(l)));
}

// Share of this lane's selected score in the sum over the warp's (0 where `have` is not
// set), from the scores' logarithms: ratios of scores that no type holds stay what they are.
// log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|)).
__device__ __forceinline__ float log1p_k(float x) { return log1pf(x); }
__device__ __forceinline__ double log1p_k(double x) { return log1p(x); }
template <typename K>
__device__ __forceinline__ K selected_share(bool soft, bool have, float l) {
  K v = K(l);
  if (have && !soft) v = (v < K(0) ? v : K(0)) - log1p_k(exp_k(v < K(0) ? v : -v));
  K m = have ? v : K(-INFINITY);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const K other = __shfl_xor_sync(0xffffffffu, m, o);
    m = other > m ? other : m;
  }
  const K w = !have ? K(0) : (v == m ? K(1) : exp_k(v - m));
  const K s = warp_sum(w);
  return have ? w / s : K(0);
}

// One row by one warp; lane i holds the PER consecutive logits from i * PER on (-inf past
// the last expert, and in place of a NaN).  Returns false, without having written
// anything, when 32-bit keys cannot tell the selection (K = float only).
template <int PER, typename K>
__device__ __forceinline__ bool route_row(const ScoredArgs& a, int t, const float (&l)[PER],
                                          const float* row, K* sh) {
  using U = typename KeyOf<K>::U;
  constexpr bool kFast = sizeof(K) == 4;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const bool biased = a.bias != nullptr;
  const bool by_score = a.G > 1 && !biased && a.group_top > 1;  // group sums of scores
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  // the softmax's maximum and sum, where a score of a whole row is asked for
  float lmax = -INFINITY;
  K z = K(1), smax = K(1);
  if (soft && (biased || by_score || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < PER; ++i) lmax = fmaxf(lmax, l[i]);
    lmax = warp_max_f(lmax);
    K part = K(0);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l[i] > -INFINITY) part += exp_below<K>(l[i], lmax);
    z = warp_sum(part);
    smax = K(1) / z;
  }
  auto score_of = [&](float v) -> K {
    return soft ? exp_below<K>(v, lmax) / z : sigmoid_k<K>(v);
  };
  U key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    K v = K(-INFINITY);
    if (l[i] > -INFINITY) {
      v = K(l[i]);
      if (biased) v = score_of(l[i]) + K(__ldg(a.bias + e));
    }
    key[i] = v > K(-INFINITY) ? ordered(v) : U(0);
    if (a.G > 1 && e < a.E)
      sh[e] = by_score ? (l[i] > -INFINITY ? score_of(l[i]) : K(-INFINITY))
                       : (v > K(-INFINITY) ? v : K(-INFINITY));
  }
  // error of a 32-bit score, relative to the row's largest: the exponential's and the
  // division's roundings, and for a softmax the sum's (PER + 5 additions)
  const float eps_s = soft ? 8e-6f : 1e-6f;
  if (a.G > 1) {
    __syncwarp();
    // lpg lanes a group (one when G does not divide 32), each scanning a strided share
    // for its two largest, merged by shuffles
    const int lpg = (32 % a.G == 0) ? 32 / a.G : 1;
    const int q = lane / lpg, sub = lane - q * lpg;
    K m1 = K(-INFINITY), m2 = K(-INFINITY);
    if (q < a.G) {
      for (int e = q * a.size + sub; e < (q + 1) * a.size; e += lpg) {
        const K v = sh[e];
        if (v > m1) { m2 = m1; m1 = v; } else if (v > m2) { m2 = v; }
      }
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const K o1 = __shfl_xor_sync(kAll, m1, o);
      const K o2 = __shfl_xor_sync(kAll, m2, o);
      const K lo = m1 > o1 ? o1 : m1;
      const K s2 = m2 > o2 ? m2 : o2;
      m1 = m1 > o1 ? m1 : o1;
      m2 = lo > s2 ? lo : s2;
    }
    K gs = m1;
    if (a.group_top > 1 && m2 > K(-INFINITY)) gs += m2;
    gs = __shfl_sync(kAll, gs, (lane < a.G ? lane : 0) * lpg);
    if (lane >= a.G) gs = K(-INFINITY);
    int better = 0;
    for (int o = 0; o < a.G; ++o) {
      const K v = __shfl_sync(kAll, gs, o);
      better += (v > gs || (v == gs && o < lane)) ? 1 : 0;
    }
    const bool some = gs > K(-INFINITY);
    const bool kept = some && better < a.g;
    const uint32_t keep = __ballot_sync(kAll, kept);
    if (kFast && (biased || by_score)) {
      const uint32_t out = __reduce_max_sync(kAll, some && !kept ? ordered(float(gs)) : 0u);
      const uint32_t in = __reduce_min_sync(kAll, kept ? ordered(float(gs)) : 0xFFFFFFFFu);
      if (out != 0u) {
        const float lo = unordered(in), hi = unordered(out);
        if (!(lo - hi > 2.f * eps_s * float(smax) + 2.4e-7f * (fabsf(lo) + fabsf(hi)))) return false;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t e = static_cast<uint32_t>(lane * PER + i);
      if (e >= static_cast<uint32_t>(a.E) || !((keep >> __umulhi(e, a.size_magic)) & 1u)) key[i] = U(0);
    }
  }
  // the largest key left, the lowest expert among equal ones: experts ascend with the lane
  // and inside a lane, so the first lane of the ballot and its first maximum are the lowest
  U mine = U(0);
  int at = 0;
  auto scan = [&]() {
    mine = U(0);
    at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > mine) { mine = key[i]; at = i; }
  };
  scan();
  int sel = -1;
  U sel_key = U(0), next = U(0);
  const int rounds = a.k + ((kFast && biased) ? 1 : 0);
  for (int r = 0; r < rounds; ++r) {
    const U m = warp_max_key(mine);
    if (m == U(0)) break;
    if (r == a.k) { next = m; break; }
    const int w = __ffs(__ballot_sync(kAll, mine == m)) - 1;
    const int e = __shfl_sync(kAll, lane * PER + at, w);
    if (lane == r) { sel = e; sel_key = m; }
    if (lane == w) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == at) key[i] = U(0);
      scan();
    }
  }
  if constexpr (kFast) {
    if (biased) {
      uint32_t below = __shfl_down_sync(kAll, sel_key, 1);
      if (lane == a.k - 1 || lane == 31) below = next;
      bool close = false;
      if (lane < a.k && sel_key != 0u && below != 0u) {
        const float hi = unordered(sel_key), lo = unordered(below);
        close = !(hi - lo > eps_s * float(smax) + 1.2e-7f * (fabsf(hi) + fabsf(lo)));
      }
      if (__any_sync(kAll, close)) return false;
    }
  }
  // gates: lane j has place j
  const bool have = lane < a.k && sel >= 0;
  const float lj = have ? row[sel] : -INFINITY;
  K w = K(0);
  if (a.renorm) w = selected_share<K>(soft, have, lj);
  else if (have) w = score_of(lj);
  if (lane < a.k) {
    a.topk_idx[static_cast<int64_t>(t) * a.k + lane] = sel;
    a.topk_w[static_cast<int64_t>(t) * a.k + lane] = static_cast<float>(w * K(a.rsf));
  }
  return true;
}

template <int PER>
__device__ __noinline__ void route_row_64(const ScoredArgs& a, int t, const float* row, double* sh) {
  const int lane = threadIdx.x & 31;
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const float v = e < a.E ? row[e] : -INFINITY;
    l[i] = v > -INFINITY ? v : -INFINITY;
  }
  route_row<PER, double>(a, t, l, row, sh);
}

// A warp per row.  Floor: 4E bytes read a row (8k written); the k rounds of two warp
// reductions each are what it spends its issue slots on.
template <int PER>
__global__ void __launch_bounds__(kRsWarps * 32) route_scored_kernel(const __grid_constant__ ScoredArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[kRsWarps][PER * 32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRsWarps + w;
  if (t >= a.T) return;
  const int64_t at = static_cast<int64_t>(t) * a.E;
  const int64_t split_stride = static_cast<int64_t>(a.T) * a.E;
  const float* row = (a.n_splits > 0 ? a.logits_out : a.logits) + at;
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    float v = -INFINITY;
    if (e < a.E) {
      if (a.n_splits > 0) {
        v = a.partials[at + e];  // in split order, as route_select_kernel adds them
        for (int sp = 1; sp < a.n_splits; ++sp) v += a.partials[sp * split_stride + at + e];
        a.logits_out[at + e] = v;
      } else {
        v = row[e];
      }
    }
    l[i] = v > -INFINITY ? v : -INFINITY;  // NaN is masked like -inf
  }
  __syncwarp();  // row[sel] below may be another lane's logits_out
  if (!route_row<PER, float>(a, t, l, row, reinterpret_cast<float*>(sh[w]))) {
    __syncwarp();
    route_row_64<PER>(a, t, row, sh[w]);
  }
}

// ---------------------------------------------------------------------------
// Gradient of the gates (and of the balance loss) with respect to the logits.
// With g_j = rsf * dgate_j on the selected places, 0 elsewhere:
//   renormalised (w = s / sum over the selected):  ds_j = (g_j - sum_i g_i w_i) / sum s,
//   otherwise (w = s)                              ds_j = g_j;
//   sigmoid  dl_e = ds_e s_e (1 - s_e);   softmax  dl_e = p_e (ds_e - sum_i ds_i p_i);
// renormalised, ds_e s_e = w_e (g_e - sum_i g_i w_i), so that no sum of scores is divided by;
//   balance loss: c_e = dloss * dscore[q, e] is the gradient of s'_e = s_e / sum s, so
//   sigmoid  dl_e += s_e (1 - s_e) / Z (c_e - sum_i c_i s'_i),   softmax  += p_e (c_e - sum_i c_i p_i).
// A softmax with renormalised gates does not depend on the unselected logits: there
// sum_i ds_i p_i = 0, and w comes from the selected logits alone.
// ---------------------------------------------------------------------------
struct RouteBwdArgs {
  const float* logits;       // [T, E]
  const int32_t* topk_idx;   // [T, k]
  const float* dgate;        // [T, k]
  const float* dscore;       // [n_seq, E] or null
  const float* dloss;        // [1] or null (1)
  const int32_t* seq_offsets;  // [n_seq + 1] or null (one sequence)
  float* dlogits;            // [T, E] or null
  __nv_bfloat16* dense_b;    // the same as bf16 in rows of ld_b from column col_b, zeros to ld_b; or null
  int T, E, k, n_seq, col_b, ld_b;
  float rsf;
  int score, renorm;
};

// A row whose sigmoids sum to less than kTinySum has every logit below -69, where
// sigmoid(l) = e^l to more than 32 bits: its shares are the softmax's.  Sets s to the
// softmax's numerators, given the largest logit, and returns their sum (0 where the row is masked as a whole).
constexpr float kTinySum = 1e-30f;
template <int PER>
__device__ __forceinline__ float tiny_sigmoid_row(const float (&l)[PER], float m, float (&s)[PER]) {
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = l[i] > -INFINITY ? exp_below<float>(l[i], m) : 0.f;
    z += s[i];
  }
  return warp_sum(z);
}

// Sequence of row t: the last q with offsets[q] <= t < offsets[q + 1], -1 outside all.
__device__ __forceinline__ int sequence_of(const int32_t* off, int n_seq, int t) {
  if (!off) return 0;
  if (t < __ldg(off) || t >= __ldg(off + n_seq)) return -1;
  int lo = 0, hi = n_seq;  // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(off + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <int PER>
__global__ void __launch_bounds__(kRsWarps * 32) route_backward_kernel(const __grid_constant__ RouteBwdArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRsWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int64_t base = static_cast<int64_t>(t) * a.E;
  const float* row = a.logits + base;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  const int q = a.dscore ? sequence_of(a.seq_offsets, a.n_seq, t) : -1;
  const bool whole = q >= 0 || (soft && !a.renorm);  // scores of the whole row are needed
  float l[PER];
  float lmax = -INFINITY, z = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = -INFINITY;
  if (whole) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      const float v = e < a.E ? row[e] : -INFINITY;
      l[i] = v > -INFINITY ? v : -INFINITY;
      lmax = fmaxf(lmax, l[i]);
    }
    if (soft) lmax = warp_max_f(lmax);
  }
  // s of every expert this lane owns (softmax: numerators until z is known)
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = 0.f;
    if (l[i] > -INFINITY) s[i] = soft ? exp_below<float>(l[i], lmax) : sigmoid_k<float>(l[i]);
    z += s[i];
  }
  if (whole) z = warp_sum(z);
  bool shifted = soft;  // s holds e^(l - lmax), not the scores themselves
  if (whole && !soft && z < kTinySum) {
    shifted = true;
    lmax = warp_max_f(lmax);
    z = tiny_sigmoid_row(l, lmax, s);
  }
  const float inv_z = z > 0.f ? 1.f / z : 0.f;
  // the balance loss: c and sum c s'
  const float up = (q >= 0 && a.dloss) ? __ldg(a.dloss) : 1.f;
  const float* crow = a.dscore + static_cast<int64_t>(q >= 0 ? q : 0) * a.E;
  float csum = 0.f;
  if (q >= 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && s[i] > 0.f) csum = fmaf(up * __ldg(crow + e), s[i] * inv_z, csum);
    }
    csum = warp_sum(csum);
  }
  // the selected places: lane j holds place j; places that name the same expert add up
  int e = lane < a.k ? __ldg(a.topk_idx + static_cast<int64_t>(t) * a.k + lane) : -1;
  float lj = -INFINITY;
  if (e >= 0 && e < a.E) lj = row[e];
  const bool have = lj > -INFINITY;
  if (!have) e = -1 - lane;  // no expert: equal to no other place
  float g = have ? a.rsf * __ldg(a.dgate + static_cast<int64_t>(t) * a.k + lane) : 0.f;
  float w = 0.f;  // renormalised: the place's share; otherwise its score
  if (a.renorm) {
    w = selected_share<float>(soft, have, lj);
    const float gw = warp_sum(g * w);
    if (have) g -= gw;
  } else if (have) {
    w = soft ? exp_below<float>(lj, lmax) * inv_z : sigmoid_k<float>(lj);
  }
  const float dot = (soft && !a.renorm) ? warp_sum(g * w) : 0.f;  // sum ds p
  // every expert of the row as if it were not selected
  float* out = a.dlogits ? a.dlogits + base : nullptr;
  __nv_bfloat16* brow = a.dense_b ? a.dense_b + static_cast<int64_t>(t) * a.ld_b + a.col_b : nullptr;
  auto rest_of = [&](int ee, float lv, float sv) -> float {  // sv: sigmoid, or softmax's numerator
    float d = 0.f;
    if (lv > -INFINITY) {
      const float c = q >= 0 ? up * __ldg(crow + ee) - csum : 0.f;
      if (soft) {
        if (whole) d = sv * inv_z * (c - dot);
      } else if (q >= 0) {
        d = sv * sigmoid_k<float>(-lv) * inv_z * c;
      }
    }
    return d;
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int ee = lane + 32 * i;
    const float d = ee < a.E ? rest_of(ee, l[i], s[i]) : 0.f;
    if (out && ee < a.E) out[ee] = d;
    if (brow && ee < a.ld_b - a.col_b) brow[ee] = __float2bfloat16_rn(d);
  }
  if (brow)
    for (int ee = lane + 32 * PER; ee < a.ld_b - a.col_b; ee += 32) brow[ee] = __float2bfloat16_rn(0.f);
  // the selected ones over it (the warp's stores above come first)
  const unsigned same = __match_any_sync(kAll, e);
  float gs = g;
  if (__any_sync(kAll, have && (same & (same - 1)) != 0u)) {  // an expert named twice
    gs = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float o = __shfl_sync(kAll, g, j);
      if ((same >> j) & 1u) gs += o;
    }
  }
  __syncwarp();
  if (have && (same & ((1u << lane) - 1u)) == 0u) {
    const float sj = whole ? (shifted ? exp_below<float>(lj, lmax) : sigmoid_k<float>(lj)) : 0.f;
    float d = rest_of(e, lj, sj);
    d += soft ? gs * w : gs * w * sigmoid_k<float>(-lj);
    if (out) out[e] = d;
    if (brow) brow[e] = __float2bfloat16_rn(d);
  }
}

// ---------------------------------------------------------------------------
// Balance loss, for sequences q of rows offsets[q] .. offsets[q + 1]:
//   f_qe = E / (k n_q) * (places of q's rows that name e),   n_q = q's rows with a score,
//   P_qe = mean over those rows of s'_te = s_te / sum_e s_te,
//   loss = coef / n_seq * sum_q sum_e f_qe P_qe,
//   dscore_qe = coef / n_seq * f_qe / n_q = d loss / d s'_te for each row t of q.
// Tiles of rows never cross a sequence: tile b of the grid belongs to the sequence in
// whose run of tiles b falls (found from the offsets on the device), and each block writes
// its sums to its own place, so that every sum has one order.
// ---------------------------------------------------------------------------
constexpr int kBalWarps = 8;

struct BalanceArgs {
  const float* logits;       // [T, E]
  const int32_t* topk_idx;   // [T, k]
  const int32_t* seq_offsets;  // [n_seq + 1] or null
  float* part;               // [tiles, E] sums of s' per tile
  int32_t* part_load;        // [tiles, E]
  int32_t* part_rows;        // [tiles]
  double* seq_loss;          // [n_seq]
  int32_t* done;             // [1]
  float* loss;               // [1]
  int32_t* load;             // [n_seq, E]
  float* dscore;             // [n_seq, E]
  int T, E, k, n_seq, tiles, tile_rows;
  float coef;
  int score;
};

__device__ __forceinline__ void seq_bounds(const BalanceArgs& a, int q, int& lo, int& hi) {
  lo = 0;
  hi = a.T;
  if (a.seq_offsets) {
    lo = min(max(__ldg(a.seq_offsets + q), 0), a.T);
    hi = min(max(__ldg(a.seq_offsets + q + 1), lo), a.T);
  }
}
__device__ __forceinline__ int seq_tiles(const BalanceArgs& a, int q) {
  int lo, hi;
  seq_bounds(a, q, lo, hi);
  return (hi - lo + a.tile_rows - 1) / a.tile_rows;
}

// Sum of seq_tiles over q < n, by the whole block (every thread gets it).
__device__ __forceinline__ int tiles_before(const BalanceArgs& a, int n, int* sh) {
  int v = 0;
  for (int q = threadIdx.x; q < n; q += blockDim.x) v += seq_tiles(a, q);
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += sh[w];
  __syncthreads();
  return s;
}

template <int PER>
__global__ void __launch_bounds__(kBalWarps * 32) balance_rows_kernel(const __grid_constant__ BalanceArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sh[kBalWarps + 2];
  __shared__ int rows_ok;
  __shared__ int32_t hist[PER * 32];
  __shared__ float sums[kBalWarps][PER * 32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  // the sequence whose run of tiles holds this block
  int q = 0, first = 0;
  if (a.seq_offsets) {
    int lo = 0, hi = a.n_seq, before = 0;  // tiles of [0, lo) <= block < tiles of [0, hi)
    // sequences in steps of the block's threads: a running total, then the step that holds it
    const int b = blockIdx.x;
    q = -1;
    for (int q0 = lo; q0 < hi && q < 0; q0 += blockDim.x) {
      const int qq = q0 + threadIdx.x;
      const int n = qq < a.n_seq ? seq_tiles(a, qq) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      if (lane == 31) sh[w] = incl;
      if (threadIdx.x == 0) sh[kBalWarps] = -1;
      __syncthreads();
      int run = before;
      for (int i = 0; i < w; ++i) run += sh[i];
      const int beg = run + incl - n;
      if (n > 0 && b >= beg && b < beg + n) {
        sh[kBalWarps] = qq;
        sh[kBalWarps + 1] = beg;
      }
      for (int i = 0; i < kBalWarps; ++i) before += sh[i];
      __syncthreads();
      q = sh[kBalWarps];
      first = sh[kBalWarps + 1];
      __syncthreads();
    }
    if (q < 0) return;  // past the last tile
  }
  int lo, hi;
  seq_bounds(a, q, lo, hi);
  lo += (blockIdx.x - first) * a.tile_rows;
  hi = min(hi, lo + a.tile_rows);
  for (int i = threadIdx.x; i < PER * 32; i += blockDim.x) hist[i] = 0;
  if (threadIdx.x == 0) rows_ok = 0;
  __syncthreads();
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  int ok = 0;
  for (int t = lo + w; t < hi; t += kBalWarps) {
    const float* row = a.logits + static_cast<int64_t>(t) * a.E;
    float l[PER], s[PER], m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      const float v = e < a.E ? row[e] : -INFINITY;
      l[i] = v > -INFINITY ? v : -INFINITY;
      m = fmaxf(m, l[i]);
    }
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    if (soft) m = warp_max_f(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = 0.f;
      if (l[i] > -INFINITY) s[i] = soft ? exp_below<float>(l[i], m) : sigmoid_k<float>(l[i]);
      z += s[i];
    }
    z = warp_sum(z);
    if (!soft && z < kTinySum) z = tiny_sigmoid_row(l, warp_max_f(m), s);
    if (z > 0.f) {
      const float inv = 1.f / z;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
      ++ok;
    }
    if (lane < a.k) {
      const int e = __ldg(a.topk_idx + static_cast<int64_t>(t) * a.k + lane);
      if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) sums[w][lane + 32 * i] = acc[i];
  if (lane == 0) atomicAdd(&rows_ok, ok);
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kBalWarps; ++i) v += sums[i][e];
    a.part[at + e] = v;
    a.part_load[at + e] = hist[e];
  }
  if (threadIdx.x == 0) a.part_rows[blockIdx.x] = rows_ok;
}

// A block per sequence; the last one to finish adds the sequences' losses in order.
__global__ void __launch_bounds__(256) balance_finish_kernel(const __grid_constant__ BalanceArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sh[8];
  __shared__ double shd[8];
  __shared__ int last;
  const int q = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int first = a.seq_offsets ? tiles_before(a, q, sh) : 0;
  const int n = min(seq_tiles(a, q), max(a.tiles - first, 0));
  int rows = 0;
  for (int b = threadIdx.x; b < n; b += blockDim.x) rows += a.part_rows[first + b];
  rows = warp_sum(rows);
  __syncthreads();
  if (lane == 0) sh[w] = rows;
  __syncthreads();
  rows = 0;
  for (int i = 0; i < 8; ++i) rows += sh[i];
  const double inv_n = rows > 0 ? 1.0 / rows : 0.0;
  double mine = 0.0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    double p = 0.0;
    int64_t c = 0;
    for (int b = 0; b < n; ++b) {
      const int64_t at = static_cast<int64_t>(first + b) * a.E + e;
      p += a.part[at];
      c += a.part_load[at];
    }
    const double d = static_cast<double>(a.coef) / a.n_seq * a.E / a.k * static_cast<double>(c) *
                     inv_n * inv_n;
    mine += d * p;
    a.load[static_cast<int64_t>(q) * a.E + e] = static_cast<int32_t>(c);
    a.dscore[static_cast<int64_t>(q) * a.E + e] = static_cast<float>(d);
  }
  mine = warp_sum(mine);
  if (lane == 0) shd[w] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < 8; ++i) v += shd[i];
    a.seq_loss[q] = v;
    __threadfence();
    last = atomicAdd(a.done, 1) == a.n_seq - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < a.n_seq; i += blockDim.x) v += __ldcg(a.seq_loss + i);
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) shd[w] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    for (int i = 0; i < 8; ++i) v += shd[i];
    *a.loss = static_cast<float>(v);
  }
}

}  // namespace moe
