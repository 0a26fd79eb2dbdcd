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
// computed in 32 bits with a known error, and where two neighbours of the sorted keys, or
// the groups on both sides of the border, are nearer than that error, the keys that can
// matter there are computed again in 64 bits (at 384 experts, top 8 and a bias 2 rows in 1000).
#pragma once

#include <cfloat>

#include "common.cuh"

namespace moe {

constexpr int kRsWarps = 4;  // rows (warps) per block of the row kernels
constexpr float kTinySum = 1e-30f;  // sums of sigmoids below this lose bits in 32

struct ScoredArgs {
  const float* logits;    // [T, E] (when n_splits == 0)
  const float* partials;  // [n_splits, T, E] router GEMM partial sums (n_splits > 0)
  float* logits_out;      // [T, E] sum of the partials, in split order (n_splits > 0)
  int n_splits;
  const float* bias;      // [E] or null
  int32_t* topk_idx;      // [T, k]
  float* topk_w;          // [T, k]
  int T, E, G, g, k, size;  // size = E / G
  int lane_shift;         // log2(size / PER) where that is a whole power of two, otherwise -1
  int vec4;               // rows are whole 16-byte vectors
  uint32_t size_magic;    // ceil(2^32 / size): e / size == umulhi(e, magic) for e < 1024
  float rsf;
  int score, renorm, group_top;
};

__device__ __forceinline__ float exp_k(float x) { return expf(x); }
__device__ __forceinline__ double exp_k(double x) { return exp(x); }

// Order-preserving unsigned image of a key; 0 is below every key's and means "none".
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ordered(float v) {
  return ordered_bits(v == 0.f ? 0.f : v);  // -0 and +0 are one key
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v == 0.0 ? 0.0 : v));
  return u ^ ((u >> 63) ? 0xFFFFFFFFFFFFFFFFull : 0x8000000000000000ull);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
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

// Groups kept, as a bit mask, given the two largest keys that each of `lpg` lanes of a group
// has seen (lane / lpg is the group).  margin (or null): distance of the last kept group's
// score from the first one left out (+inf: none is left out).
template <typename K>
__device__ __forceinline__ uint32_t keep_of_tops(const ScoredArgs& a, int lane, K m1, K m2, int lpg,
                                                 float* margin) {
  constexpr unsigned kAll = 0xffffffffu;
  for (int o = 1; o < lpg; o <<= 1) {  // top 2 of two top-2 pairs
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
  const bool some = gs > K(-INFINITY), kept = some && better < a.g;
  if (margin) {
    const uint32_t out = __reduce_max_sync(kAll, some && !kept ? ordered(float(gs)) : 0u);
    const uint32_t in = __reduce_min_sync(kAll, kept ? ordered(float(gs)) : 0xFFFFFFFFu);
    if (out != 0u) *margin = unordered(in) - unordered(out);
  }
  return __ballot_sync(kAll, kept);
}

// Whether the lane's own group is kept, where every group is 2^SHIFT whole neighbouring lanes
// and m1, m2 are the lane's two largest keys.  The lanes of a group share the comparisons with
// the other groups (by shuffles: rounds of warp-wide maxima took three times as long, their
// reductions issue at a sixteenth of the rate).  margin: the last kept group's score less the
// first one's left out.
template <int SHIFT>
__device__ __forceinline__ bool own_group_kept(const ScoredArgs& a, int lane, float m1, float m2,
                                               bool want_margin, float* margin) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int lpg = 1 << SHIFT;
#pragma unroll
  for (int o = 1; o < lpg; o <<= 1) {
    const float o1 = __shfl_xor_sync(kAll, m1, o);
    const float o2 = __shfl_xor_sync(kAll, m2, o);
    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
    m1 = fmaxf(m1, o1);
  }
  const int q = lane >> SHIFT;
  float gs = m1;
  if (a.group_top > 1 && m2 > -INFINITY) gs += m2;
  if (q >= a.G) gs = -INFINITY;
  int better = 0;
#pragma unroll 2
  for (int o0 = 0; o0 < a.G; o0 += lpg) {
    const int o = o0 + (lane & (lpg - 1));
    const float v = __shfl_sync(kAll, gs, (o << SHIFT) & 31);
    better += o < a.G && (v > gs || (v == gs && o < q)) ? 1 : 0;
  }
#pragma unroll
  for (int o = 1; o < lpg; o <<= 1) better += __shfl_xor_sync(kAll, better, o);
  const bool some = gs > -INFINITY;
  if (want_margin) {
    const uint32_t first_out = __ballot_sync(kAll, some && better == a.g);
    if (first_out != 0u) {  // then the places before it are taken
      const uint32_t last_in = __ballot_sync(kAll, some && better == a.g - 1);
      *margin = __shfl_sync(kAll, gs, __ffs(last_in) - 1) - __shfl_sync(kAll, gs, __ffs(first_out) - 1);
    }
  }
  return some && better < a.g;
}

// The warp's 32 values in descending order (lane 0 the largest): a bitonic network whose
// merges start mirrored, so that the lower lane of every exchange takes the larger value.
__device__ __forceinline__ float warp_sort_desc(float v, int lane) {
  const bool low[5] = {(lane & 1) == 0, (lane & 2) == 0, (lane & 4) == 0, (lane & 8) == 0, (lane & 16) == 0};
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    float o = __shfl_xor_sync(0xffffffffu, v, (2 << k) - 1);
    v = low[k] ? fmaxf(v, o) : fminf(v, o);
#pragma unroll
    for (int j = k - 1; j >= 0; --j) {
      o = __shfl_xor_sync(0xffffffffu, v, 1 << j);
      v = low[j] ? fmaxf(v, o) : fminf(v, o);
    }
  }
  return v;
}

// The same with the keys in shared memory: lpg lanes a group (one when G does not divide
// 32), each scanning a strided share.
template <typename F>
__device__ __forceinline__ uint32_t kept_groups(const ScoredArgs& a, int lane, F key_of, float* margin) {
  using K = decltype(key_of(0));
  const int lpg = (32 % a.G == 0) ? 32 / a.G : 1;
  const int q = lane / lpg, sub = lane - q * lpg;
  K m1 = K(-INFINITY), m2 = K(-INFINITY);
  if (q < a.G) {
    for (int e = q * a.size + sub; e < (q + 1) * a.size; e += lpg) {
      const K v = key_of(e);
      if (v > m1) { m2 = m1; m1 = v; } else if (v > m2) { m2 = v; }
    }
  }
  return keep_of_tops(a, lane, m1, m2, lpg, margin);
}

// A softmax's sum over the row and a score, in 64 bits: calls and loops, not unrolled, since
// what a rare row pays for is mostly the instructions' way into the SM.
__device__ __noinline__ double sum_64(const float* row, int E, int lane, float lmax) {
  double z = 0.0;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const float v = row[e];
    if (v > -INFINITY) z += exp_below<double>(v, lmax);
  }
  return warp_sum(z);
}
__device__ __noinline__ double score_64(bool soft, float l, float lmax, double z) {
  const double x = exp(soft ? (l == lmax ? 0.0 : static_cast<double>(l) - lmax) : -static_cast<double>(l));
  return soft ? x / z : 1.0 / (1.0 + x);
}

// One row in 64 bits by one warp, for the rows with more candidates than route_row holds (many
// equal keys) and those of groups that are not whole lanes and too near each other:
// lane i holds the PER consecutive logits from i * PER on.  k rounds of a warp maximum.
template <int PER>
__device__ __noinline__ void route_row_64(const ScoredArgs& a, int t, const float* row, double* sh) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const bool biased = a.bias != nullptr;
  const bool by_score = a.G > 1 && !biased && a.group_top > 1;  // group sums of scores
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  float l[PER];
  float lmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const float v = e < a.E ? row[e] : -INFINITY;
    l[i] = v > -INFINITY ? v : -INFINITY;  // NaN is masked like -inf
    lmax = fmaxf(lmax, l[i]);
  }
  lmax = warp_max_f(lmax);
  double z = 1.0;
  if (soft) {
    z = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l[i] > -INFINITY) z += exp_below<double>(l[i], lmax);
    z = warp_sum(z);
  }
  auto score_of = [&](float v) -> double {
    return soft ? exp_below<double>(v, lmax) / z : sigmoid_k<double>(v);
  };
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    double v = -INFINITY;
    if (l[i] > -INFINITY) {
      v = l[i];
      if (biased) v = score_of(l[i]) + static_cast<double>(__ldg(a.bias + e));
    }
    key[i] = v > -INFINITY ? ordered(v) : 0ull;
    if (a.G > 1 && e < a.E)
      sh[e] = by_score ? (l[i] > -INFINITY ? score_of(l[i]) : -INFINITY) : (v > -INFINITY ? v : -INFINITY);
  }
  if (a.G > 1) {
    __syncwarp();
    const uint32_t keep = kept_groups(a, lane, [&](int e) { return sh[e]; }, nullptr);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t e = static_cast<uint32_t>(lane * PER + i);
      if (e >= static_cast<uint32_t>(a.E) || !((keep >> __umulhi(e, a.size_magic)) & 1u)) key[i] = 0ull;
    }
  }
  // the largest key left, the lowest expert among equal ones: experts ascend with the lane
  // and inside a lane, so the first lane of the ballot and its first maximum are the lowest
  uint64_t mine = 0ull;
  int at = 0;
  auto scan = [&]() {
    mine = 0ull;
    at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > mine) { mine = key[i]; at = i; }
  };
  scan();
  int sel = -1;
  for (int r = 0; r < a.k; ++r) {
    const uint64_t m = warp_max_key(mine);
    if (m == 0ull) break;
    const int w = __ffs(__ballot_sync(kAll, mine == m)) - 1;
    const int e = __shfl_sync(kAll, lane * PER + at, w);
    if (lane == r) sel = e;
    if (lane == w) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == at) key[i] = 0ull;
      scan();
    }
  }
  const bool have = lane < a.k && sel >= 0;
  const float lj = have ? row[sel] : -INFINITY;
  double w = 0.0;
  if (a.renorm) w = selected_share<double>(soft, have, lj);
  else if (have) w = score_of(lj);
  if (lane < a.k) {
    a.topk_idx[static_cast<int64_t>(t) * a.k + lane] = sel;
    a.topk_w[static_cast<int64_t>(t) * a.k + lane] = static_cast<float>(w * static_cast<double>(a.rsf));
  }
}

// 2^x and 1 / x from the hardware (2^-22 and 2^-23 of the result); no result is subnormal.
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// e^x and 1 / (1 + e^-x) from them, for keys alone.  The exponential's argument's rounding
// adds |x| 2^-24, so a sigmoid is off by at most
// s (1 - s) (2^-22 + |x| 2^-24) + s (2^-23 + 2^-24) < 2.6e-7.
__device__ __forceinline__ float exp_fast(float x) { return ex2_fast(x * 1.4426950408889634f); }
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.f + exp_fast(-x)); }

constexpr int kRsCand = 64;  // candidates of a row

// Top k: the k-th largest of the lanes' maxima is at most the k-th largest key, so the keys
// from it on (less their error, with a bias) are few and hold the selection; they are gathered
// through shared memory, one or two a lane, and each finds its rank by comparing itself to all.
// That takes about half the instructions of k rounds of maximum and removal.
//
// Keys nearer to each other than their error: 64 bits for the two largest of each lane (groups)
// or for the candidates alone.  (The whole row in 64 bits: 17 us for 1024 rows of 384 logits,
// in nearly every batch of which there is such a row, against 8.)
//
// One row in 32 bits by one warp; lane i holds the PER consecutive logits from i * PER on
// (-inf past the last expert, and in place of a NaN).  Returns false, without having written
// anything, where it cannot tell the selection.
// SOFT, BIASED: the form, 0 or 1, or -1 where it is asked for row by row.
template <int PER, int SOFT, int BIASED>
__device__ __forceinline__ bool route_row(const ScoredArgs& a, int t, const float (&l)[PER],
                                          const float (&bias)[PER], float bias_max, const float* row,
                                          float* sh) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const bool biased = BIASED < 0 ? a.bias != nullptr : BIASED == 1;
  const bool soft = SOFT < 0 ? a.score == MOE_SCORE_SOFTMAX : SOFT == 1;
  const bool by_score = !biased && a.G > 1 && a.group_top > 1;
  // the softmax's maximum and sum, where a score of the whole row is asked for
  float lmax = -INFINITY, z = 1.f, smax = 1.f;
  if (soft && (biased || by_score || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < PER; ++i) lmax = fmaxf(lmax, l[i]);
    lmax = warp_max_f(lmax);
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l[i] > -INFINITY) part += l[i] == lmax ? 1.f : exp_fast(l[i] - lmax);
    z = warp_sum(part);
    smax = 1.f / z;
  }
  auto key_score = [&](float v) -> float {
    return soft ? (v == lmax ? 1.f : exp_fast(v - lmax)) * smax : sigmoid_fast(v);
  };
  // error of such a score, doubled, relative to the row's largest: the exponential's and the
  // division's roundings, and for a softmax the sum's (PER + 5 additions)
  const float eps = (soft ? 8e-6f : 1e-6f) * smax;
  // of a difference of two keys: the score's, and the roundings of sums with the bias
  const float near = eps + 2.4e-7f * (smax + bias_max);
  float key[PER];  // -inf: none (a bias that takes an expert out is -inf)
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = biased ? (l[i] > -INFINITY ? key_score(l[i]) + bias[i] : -INFINITY) : l[i];
  float top = -INFINITY, second = -INFINITY;  // the lane's largest
  bool kept = true;                           // its group is
  if (a.G > 1) {
    float margin = INFINITY;
    if (a.lane_shift >= 0) {  // a group is 2^lane_shift whole lanes
      if (by_score) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float v = l[i] > -INFINITY ? key_score(l[i]) : -INFINITY;
          second = fmaxf(second, fminf(top, v));
          top = fmaxf(top, v);
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          second = fmaxf(second, fminf(top, key[i]));
          top = fmaxf(top, key[i]);
        }
      }
      const bool border = biased || by_score;
      switch (a.lane_shift) {
        case 0: kept = own_group_kept<0>(a, lane, top, second, border, &margin); break;
        case 1: kept = own_group_kept<1>(a, lane, top, second, border, &margin); break;
        case 2: kept = own_group_kept<2>(a, lane, top, second, border, &margin); break;
        case 3: kept = own_group_kept<3>(a, lane, top, second, border, &margin); break;
        default: kept = own_group_kept<4>(a, lane, top, second, border, &margin); break;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane * PER + i < a.E)
          sh[lane * PER + i] = by_score && key[i] > -INFINITY ? key_score(l[i]) : key[i];
      __syncwarp();
      const uint32_t keep = kept_groups(a, lane, [&](int e) { return sh[e]; }, &margin);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t e = static_cast<uint32_t>(lane * PER + i);
        if (e >= static_cast<uint32_t>(a.E) || !((keep >> __umulhi(e, a.size_magic)) & 1u)) key[i] = -INFINITY;
      }
    }
    // a group has one or two keys
    if ((biased || by_score) && !(margin > (a.group_top > 1 ? 2.f : 1.f) * near)) {
      if (a.lane_shift < 0) return false;
      const float from = (a.group_top > 1 ? second : top) - near;
      uint32_t again = 0u;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float v = by_score && key[i] > -INFINITY ? key_score(l[i]) : key[i];
        again |= v > -INFINITY && v >= from ? 1u << i : 0u;
      }
      const double z64 = soft ? sum_64(row, a.E, lane, lmax) : 1.0;
      double m1 = -INFINITY, m2 = -INFINITY;
      for (; again != 0u; again &= again - 1) {
        const int e = lane * PER + __ffs(again) - 1;
        const double v = score_64(soft, row[e], lmax, z64) + (biased ? static_cast<double>(__ldg(a.bias + e)) : 0.0);
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      __syncwarp();
      kept = (keep_of_tops<double>(a, lane, m1, m2, 1 << a.lane_shift, nullptr) >> (lane >> a.lane_shift)) & 1u;
    }
  }
  // a lower bound of the last key needed, from the lanes' maxima
  if (a.G == 1 || by_score || a.lane_shift < 0) {  // (otherwise the lane's top it is)
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, key[i]);
  }
  const float ranked = warp_sort_desc(kept ? top : -INFINITY, lane);
  float bound = __shfl_sync(kAll, ranked, a.k - 1);
  if (biased) bound -= near;
  bound = fmaxf(bound, -FLT_MAX);  // (none is below)
  uint32_t in = 0u;  // a bit for each candidate
#pragma unroll
  for (int i = 0; i < PER; ++i) in |= key[i] >= bound ? 1u << i : 0u;
  if (!kept) in = 0u;
  const int mine_in = __popc(in);
  int at = mine_in;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, at, o);
    if (lane >= o) at += v;
  }
  const int n = __shfl_sync(kAll, at, 31);
  if (n > kRsCand) return false;  // many equal keys
  // gathered in the order of the experts, as (key, expert)
  uint2* cand = reinterpret_cast<uint2*>(sh);
  uint32_t* keys = reinterpret_cast<uint32_t*>(cand + kRsCand);
  uint2* slot = cand + at - mine_in;
  if (in != 0u) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((in >> i) & 1u) *slot++ = make_uint2(__float_as_uint(key[i]), lane * PER + i);
  }
  __syncwarp();
  uint2 mine[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = lane + 32 * h;
    if (c < n) {
      mine[h] = cand[c];
      mine[h].x = ordered_bits(__fadd_rn(__uint_as_float(mine[h].x), 0.f));  // -0 and +0 are one key
    }
    if (h == 0 || n > 32) keys[c] = mine[h].x;  // (0 past the last one)
  }
  __syncwarp();
  // the rank of a candidate: larger keys, and equal ones before it
  uint2* sorted = cand;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = lane + 32 * h;
    if (h == 1 && n <= 32) break;
    int rank = 0;
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(keys + j);
      rank += o.x > mine[h].x - (j < c ? 1u : 0u) ? 1 : 0;
      rank += o.y > mine[h].x - (j + 1 < c ? 1u : 0u) ? 1 : 0;
      rank += o.z > mine[h].x - (j + 2 < c ? 1u : 0u) ? 1 : 0;
      rank += o.w > mine[h].x - (j + 3 < c ? 1u : 0u) ? 1 : 0;
    }
    if (c < n) sorted[rank] = mine[h];
  }
  __syncwarp();
  const uint2 got = lane < min(n, a.k) ? sorted[lane] : make_uint2(0u, 0u);
  int sel = got.x != 0u ? static_cast<int>(got.y) : -1;
  if (biased) {
    bool close = false;
    if (sel >= 0 && lane + 1 < n) {
      const float hi = unordered(got.x);
      const float lo = unordered(sorted[lane + 1].x);
      close = !(hi - lo > eps + 1.2e-7f * (fabsf(hi) + fabsf(lo)));
    }
    if (__any_sync(kAll, close)) {
      const double z64 = soft ? sum_64(row, a.E, lane, lmax) : 1.0;
      __syncwarp();  // sorted and keys are read
      double* keys64 = reinterpret_cast<double*>(cand);
      int* order = reinterpret_cast<int*>(keys);
      double v[2] = {0.0, 0.0};
      for (int c = lane, h = 0; c < n; c += 32, ++h) {
        const int e = static_cast<int>(h == 0 ? mine[0].y : mine[1].y);
        const double x = score_64(soft, row[e], lmax, z64) + static_cast<double>(__ldg(a.bias + e));
        if (h == 0) v[0] = x; else v[1] = x;
        keys64[c] = x;
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += keys64[j] > v[h] || (keys64[j] == v[h] && j < c) ? 1 : 0;
        if (c < n) order[rank] = static_cast<int>(mine[h].y);
      }
      __syncwarp();
      sel = lane < min(n, a.k) ? order[lane] : -1;
    }
  }
  // gates: lane j has place j
  const bool have = sel >= 0;
  const float lj = have ? row[sel] : -INFINITY;
  float w = 0.f;
  if (have && !(soft && a.renorm))
    w = soft ? exp_below<float>(lj, lmax) * smax : __fdividef(1.f, 1.f + expf(-lj));
  if (a.renorm) {
    const float sum = soft ? 0.f : warp_sum(w);
    if (sum >= kTinySum) w = __fdividef(w, sum);
    else w = selected_share<float>(soft, have, lj);
  }
  if (lane < a.k) {
    a.topk_idx[static_cast<int64_t>(t) * a.k + lane] = sel;
    a.topk_w[static_cast<int64_t>(t) * a.k + lane] = w * a.rsf;
  }
  return true;
}

// A warp per row, rows in a grid stride with the next row's logits on their way.
// Floor: 4E bytes read a row (8k written); instruction issue is what it spends its time on
// (65536 x 256, top 8 with a bias and groups: 64 us, 1.1 TB/s, 770 instructions a row).
template <int PER, int SOFT, int BIASED>
__global__ void __launch_bounds__(kRsWarps * 32, PER <= 8 ? 8 : (PER <= 12 ? 6 : 1)) route_scored_kernel(const __grid_constant__ ScoredArgs a) {
  pdl_wait();
  pdl_trigger();
  // the fp32 row's group scores or candidates and their sorted copy, or the 64-bit row's scores
  __shared__ double sh[kRsWarps][PER * 32 > 2 * kRsCand ? PER * 32 : 2 * kRsCand];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t split_stride = static_cast<int64_t>(a.T) * a.E;
  const int stride = gridDim.x * kRsWarps;
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const float b = BIASED != 0 && a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
    bias[i] = fmaxf(b, -INFINITY);  // NaN takes an expert out like -inf
  }
  float bias_max = 0.f;  // of the finite ones
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (fabsf(bias[i]) < INFINITY) bias_max = fmaxf(bias_max, fabsf(bias[i]));
  if (BIASED != 0) bias_max = warp_max_f(bias_max);
  auto fetch = [&](int t, float (&l)[PER]) {
    const int64_t at = static_cast<int64_t>(t) * a.E;
    const float* src = (a.n_splits > 0 ? a.partials : a.logits) + at;
    if (PER % 4 == 0 && a.vec4) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const int e = lane * PER + i;
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < a.E) v = *reinterpret_cast<const float4*>(src + e);
        l[i] = v.x;
        l[i + 1] = v.y;
        l[i + 2] = v.z;
        l[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i;
        l[i] = e < a.E ? src[e] : -INFINITY;
      }
    }
    if (a.n_splits > 0) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i;
        if (e < a.E)  // in split order, as route_select_kernel adds them
          for (int sp = 1; sp < a.n_splits; ++sp) l[i] += a.partials[sp * split_stride + at + e];
      }
    }
  };
  int t = blockIdx.x * kRsWarps + w;
  float l[PER], next[PER];
  if (t < a.T) fetch(t, l);
  for (; t < a.T; t += stride) {
    if (t + stride < a.T) fetch(t + stride, next);
    const int64_t at = static_cast<int64_t>(t) * a.E;
    const float* row = (a.n_splits > 0 ? a.logits_out : a.logits) + at;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (a.n_splits > 0 && e < a.E) a.logits_out[at + e] = l[i];
      l[i] = fmaxf(l[i], -INFINITY);  // NaN is masked like -inf
    }
    __syncwarp();  // row[sel] may be another lane's logits_out
    if (!route_row<PER, SOFT, BIASED>(a, t, l, bias, bias_max, row, reinterpret_cast<float*>(sh[w]))) {
      __syncwarp();
      route_row_64<PER>(a, t, row, sh[w]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = next[i];
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
  int rows;                  // a warp's run
  float rsf;
  int score, renorm;
};

// Experts of a lane, in a row of 32 * PER: every 32nd one, or (VEC: rows of whole 16-byte
// vectors) four neighbours in every 128.
template <int PER, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : lane + 32 * i;
}
template <int PER, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float fill, float (&v)[PER]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int e = expert_of<PER, VEC>(lane, i);
      float4 x = make_float4(fill, fill, fill, fill);
      if (e < E) x = __ldg(reinterpret_cast<const float4*>(row + e));
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = expert_of<PER, VEC>(lane, i);
      v[i] = e < E ? __ldg(row + e) : fill;
    }
  }
}

// sigmoid(l) and 1 - sigmoid(l), each to its own precision: with q = exp(-|l|), 1 / (1 + q)
// is the larger of the two and q / (1 + q) the smaller (0 at -inf).
__device__ __forceinline__ void sigmoid_both(float l, float& s, float& t) {
  const float q = ex2_fast(fabsf(l) * -1.4426950408889634f), r = rcp_fast(1.f + q), o = q * r;
  s = l >= 0.f ? r : o;
  t = l >= 0.f ? o : r;
}

// s = e^(l - max l) of a row, and its sum (0 where the row is masked as a whole); lmax: the
// largest logit.  l has -inf in place of a NaN.
template <int PER>
__device__ __forceinline__ float softmax_of_row(const float (&l)[PER], float (&s)[PER], float& lmax) {
  lmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) lmax = fmaxf(lmax, l[i]);
  lmax = warp_max_f(lmax);
  float z = 0.f;
  if (fabsf(lmax) < INFINITY) {
    const float c = 1.4426950408889634f, m = lmax * c;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = ex2_fast(fmaf(l[i], c, -m));
      z += s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = l[i] == lmax && lmax > -INFINITY ? 1.f : 0.f;
      z += s[i];
    }
  }
  return warp_sum(z);
}

// Scores of a row up to a common factor: l (NaN: -inf) -> s, and t = 1 - sigmoid (sigmoid
// only).  Returns the sum of s over the row, 0 where it is masked as a whole; shifted: s is
// e^(l - lmax).
// A row whose sigmoids sum to less than kTinySum has every logit below -69, where
// sigmoid(l) = e^l to more than 32 bits: its shares are the softmax's.
template <int PER>
__device__ __forceinline__ float scores_of_row(bool soft, float (&l)[PER], float (&s)[PER], float (&t)[PER],
                                               float& lmax, bool& shifted) {
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = fmaxf(l[i], -INFINITY);
  if (!soft) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      sigmoid_both(l[i], s[i], t[i]);
      z += s[i];
    }
    z = warp_sum(z);
    shifted = false;
    if (z >= kTinySum) return z;
  }
  shifted = true;
  return softmax_of_row<PER>(l, s, lmax);
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

// A warp for a run of `rows` neighbouring rows: the sequence's coefficients stay in registers
// from row to row.  Floor: 4E bytes read (where whole rows are needed) and 4E written a row;
// instruction issue is what it spends its time on (32768 x 384, top 8, with the balance
// loss's part: 32 us, 3.3 TB/s; a row a warp: 34).
template <int PER, bool VEC>
__global__ void __launch_bounds__(kRsWarps * 32, PER <= 12 ? 8 : 1) route_backward_kernel(const __grid_constant__ RouteBwdArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRsWarps + (threadIdx.x >> 5)) * a.rows;
  const int t_end = static_cast<int>(min(static_cast<int64_t>(a.T), t0 + a.rows));
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  const float up = a.dscore && a.dloss ? __ldg(a.dloss) : 1.f;
  float c[PER];
  int q = -1, q_end = static_cast<int>(t0);  // q: the sequence of the rows before q_end
  for (int t = static_cast<int>(t0); t < t_end; ++t) {
    const int64_t base = static_cast<int64_t>(t) * a.E;
    const float* row = a.logits + base;
    // the selected places: lane j holds place j
    int e = lane < a.k ? __ldg(a.topk_idx + static_cast<int64_t>(t) * a.k + lane) : -1;
    const float dg = lane < a.k ? __ldg(a.dgate + static_cast<int64_t>(t) * a.k + lane) : 0.f;
    if (a.dscore && t >= q_end) {
      q = sequence_of(a.seq_offsets, a.n_seq, t);
      q_end = q < 0 ? t + 1 : (a.seq_offsets ? __ldg(a.seq_offsets + q + 1) : a.T);
      if (q >= 0) load_row<PER, VEC>(a.dscore + static_cast<int64_t>(q) * a.E, a.E, lane, 0.f, c);
    }
    const bool whole = q >= 0 || (soft && !a.renorm);  // scores of the whole row are needed
    float l[PER], s[PER], t1[PER];
    float lmax = -INFINITY, z = 0.f;
    bool shifted = soft;
    if (whole) load_row<PER, VEC>(row, a.E, lane, -INFINITY, l);
    float lj = -INFINITY;
    if (e >= 0 && e < a.E) lj = __ldg(row + e);
    const bool have = lj > -INFINITY;
    if (!have) e = -1 - lane;  // no expert: equal to no other place
    if (whole) z = scores_of_row<PER>(soft, l, s, t1, lmax, shifted);
    const float inv_z = z > 0.f ? 1.f / z : 0.f;
    float csum = 0.f;  // sum c s'
    if (q >= 0) {
#pragma unroll
      for (int i = 0; i < PER; ++i) csum = fmaf(c[i], s[i], csum);
      csum = warp_sum(csum) * inv_z;
    }
    float g = have ? a.rsf * dg : 0.f;
    float sj = 0.f, tj = 0.f;  // the place's sigmoid and 1 - sigmoid
    if (!soft && have) sigmoid_both(lj, sj, tj);
    const float mine = shifted ? (have ? exp_below<float>(lj, lmax) : 0.f) : sj;
    float w = 0.f;       // renormalised: the place's share; otherwise its score
    uint32_t same = 0u;  // places that name this one's expert
    if (a.renorm) {
      const float sum = soft ? 0.f : warp_sum(sj);
      if (sum >= kTinySum) w = __fdividef(sj, sum);
      else w = selected_share<float>(soft, have, lj);
      // g_j - sum_i g_i w_i as sum_i w_i (g_j - g_i): a share near one does not cancel, and a
      // single place's gradient is zero
      float d = 0.f;
#pragma unroll 4
      for (int i = 0; i < a.k; ++i) {
        d = fmaf(__shfl_sync(kAll, w, i), g - __shfl_sync(kAll, g, i), d);
        same |= __shfl_sync(kAll, e, i) == e ? 1u << i : 0u;
      }
      g = have ? d : 0.f;
    } else {
      if (have) w = soft ? mine * inv_z : sj;
#pragma unroll 4
      for (int i = 0; i < a.k; ++i) same |= __shfl_sync(kAll, e, i) == e ? 1u << i : 0u;
    }
    const float dot = (soft && !a.renorm) ? warp_sum(g * w) : 0.f;  // sum ds p
    // every expert of the row as if it were not selected
    if (q >= 0) {
      const float f = inv_z * up, h = inv_z * fmaf(up, csum, dot);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        s[i] *= fmaf(f, c[i], -h);
        if (!soft) s[i] *= t1[i];
      }
    } else {  // a softmax, or nothing
      const float h = whole ? inv_z * -dot : 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) s[i] = whole ? s[i] * h : 0.f;
    }
    float* out = a.dlogits ? a.dlogits + base : nullptr;
    __nv_bfloat16* brow = a.dense_b ? a.dense_b + static_cast<int64_t>(t) * a.ld_b + a.col_b : nullptr;
    if (out) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int ee = expert_of<PER, VEC>(lane, i);
        if constexpr (VEC) {
          if (i % 4 == 0 && ee < a.E)
            *reinterpret_cast<float4*>(out + ee) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
        } else {
          if (ee < a.E) out[ee] = s[i];
        }
      }
    }
    if (brow) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int ee = expert_of<PER, VEC>(lane, i);
        if (ee < a.ld_b - a.col_b) brow[ee] = __float2bfloat16_rn(ee < a.E ? s[i] : 0.f);
      }
      for (int ee = lane + 32 * PER; ee < a.ld_b - a.col_b; ee += 32) brow[ee] = __float2bfloat16_rn(0.f);
    }
    // the selected ones over it (the warp's stores above come first); places that name the
    // same expert add up
    float gs = g;
    if (__any_sync(kAll, have && (same & (same - 1u)) != 0u)) {
      gs = 0.f;
      for (int i = 0; i < a.k; ++i) {
        const float gi = __shfl_sync(kAll, g, i);
        if ((same >> i) & 1u) gs += gi;
      }
    }
    __syncwarp();
    if (have && __ffs(same) - 1 == lane) {
      float d = 0.f;
      if (whole) d = mine * inv_z * ((q >= 0 ? up * (__ldg(a.dscore + static_cast<int64_t>(q) * a.E + e) - csum) : 0.f) - dot);
      d = fmaf(gs, w, d);
      if (!soft) d *= tj;
      if (out) out[e] = d;
      if (brow) brow[e] = __float2bfloat16_rn(d);
    }
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
  double* seq_loss;          // [n_seq, e_blocks]
  int32_t* done;             // [1]
  float* loss;               // [1]
  int32_t* load;             // [n_seq, E]
  float* dscore;             // [n_seq, E]
  int T, E, k, n_seq, tiles, tile_rows, e_blocks;
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

// Sum of seq_tiles over q < n, by the whole block (every thread gets it); at most a.tiles, as
// it is for ascending offsets, whatever the offsets are.
__device__ __forceinline__ int tiles_before(const BalanceArgs& a, int n, int* sh) {
  int64_t all = 0;
  for (int q = threadIdx.x; q < n; q += blockDim.x) all += seq_tiles(a, q);
  const int v = static_cast<int>(min(warp_sum(all), static_cast<int64_t>(a.tiles)));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s = min(s + sh[w], a.tiles);
  __syncthreads();
  return s;
}

// Floor: 4E + 4k bytes read a row.  Each warp has the next row's logits on their way.
// (65536 x 256: 17 us, 4.1 TB/s; issue slots half used, the rest waits for loads and sums.)
template <int PER, bool VEC>
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
  // (inside the sequence whatever the offsets are)
  lo = max(lo, lo + (static_cast<int>(blockIdx.x) - first) * a.tile_rows);
  hi = min(hi, lo + a.tile_rows);
  for (int i = threadIdx.x; i < PER * 32; i += blockDim.x) hist[i] = 0;
  if (threadIdx.x == 0) rows_ok = 0;
  __syncthreads();
  float acc[PER], l[PER], next[PER], s[PER], t1[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  int ok = 0;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  int t = lo + w;
  int pick = -1, pick_next = -1;
  auto fetch = [&](int r, float (&v)[PER], int& p) {
    load_row<PER, VEC>(a.logits + static_cast<int64_t>(r) * a.E, a.E, lane, -INFINITY, v);
    p = lane < a.k ? __ldg(a.topk_idx + static_cast<int64_t>(r) * a.k + lane) : -1;
  };
  if (t < hi) fetch(t, l, pick);
  for (; t < hi; t += kBalWarps) {
    if (t + kBalWarps < hi) fetch(t + kBalWarps, next, pick_next);
    float lmax;
    bool shifted;
    const float z = scores_of_row<PER>(soft, l, s, t1, lmax, shifted);
    if (z > 0.f) {
      const float inv = 1.f / z;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
      ++ok;
    }
    if (pick >= 0 && pick < a.E) atomicAdd(&hist[pick], 1);
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = next[i];
    pick = pick_next;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) sums[w][expert_of<PER, VEC>(lane, i)] = acc[i];
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

// A block per sequence and 64 experts, eight threads an expert over the sequence's tiles; the
// last block to finish adds the blocks' losses in order.  Latency: about 5 us.
constexpr int kBalExperts = 64, kBalSlices = 8;
__global__ void __launch_bounds__(kBalExperts * kBalSlices) balance_finish_kernel(const __grid_constant__ BalanceArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = kBalExperts * kBalSlices / 32;
  __shared__ int sh[kWarps];
  __shared__ double shd[kBalSlices][kBalExperts];
  __shared__ int shc[kBalSlices][kBalExperts];
  __shared__ int last;
  const int q = blockIdx.x / a.e_blocks, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int first = a.seq_offsets ? tiles_before(a, q, sh) : 0;
  const int n = min(seq_tiles(a, q), max(a.tiles - first, 0));
  int rows = 0;
  for (int b = threadIdx.x; b < n; b += blockDim.x) rows += a.part_rows[first + b];
  rows = warp_sum(rows);
  __syncthreads();
  if (lane == 0) sh[w] = rows;
  const int el = threadIdx.x % kBalExperts, sl = threadIdx.x / kBalExperts;
  const int e = (blockIdx.x - q * a.e_blocks) * kBalExperts + el;
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = sl; b < n; b += kBalSlices) {
      const int64_t at = static_cast<int64_t>(first + b) * a.E + e;
      p += a.part[at];
      c += a.part_load[at];
    }
  }
  shd[sl][el] = p;
  shc[sl][el] = c;
  __syncthreads();
  rows = 0;
  for (int i = 0; i < kWarps; ++i) rows += sh[i];
  const double inv_n = rows > 0 ? 1.0 / rows : 0.0;
  if (sl == 0) {
    for (int i = 1; i < kBalSlices; ++i) {
      p += shd[i][el];
      c += shc[i][el];
    }
    const double d = static_cast<double>(a.coef) / a.n_seq * a.E / a.k * c * inv_n * inv_n;
    if (e < a.E) {
      a.load[static_cast<int64_t>(q) * a.E + e] = c;
      a.dscore[static_cast<int64_t>(q) * a.E + e] = static_cast<float>(d);
    }
    shd[0][el] = d * p;
  }
  __syncthreads();
  if (w == 0) {
    const double v = warp_sum(shd[0][lane] + shd[0][lane + 32]);
    if (lane == 0) {
      a.seq_loss[blockIdx.x] = v;
      __threadfence();
      last = atomicAdd(a.done, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += blockDim.x) v += __ldcg(a.seq_loss + i);
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) shd[0][w] = v;
  __syncthreads();
  if (w == 0) {
    v = warp_sum(lane < kWarps ? shd[0][lane] : 0.0);
    if (lane == 0) *a.loss = static_cast<float>(v);
  }
}

}  // namespace moe
