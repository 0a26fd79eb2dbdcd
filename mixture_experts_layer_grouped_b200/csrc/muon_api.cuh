// Host side of the orthogonalised updates (part of moe_api.cu's translation unit): the
// workspace layout, the launches and the C ABI calls of include/moe_b200.h's Muon section.
// The kernels are in muon.cuh and muon_small.cuh.
#pragma once

namespace {

struct MuonLayout {
  size_t status, counters, part, x[2][2], a[2], b[2], diag[2], partial, total;  // [buffer][hi, lo], [hi, lo]
  int r, ld, ldr, chunk, chunks;
  int64_t units;  // of all steps
  int tile, sym_n, sym_tiles, app_n, app_tiles, k_gram, k_r, splits, sums, n_counters;
};

// What the steps can reach from singular values in [0, 1], interval by interval: with
// x = sigma^2 in [0, R^2], the extremes of f(sigma) = sigma (a + b x + c x^2), of a + b x + c x^2
// and of b x + c x^2 lie at the interval's end or where their derivatives vanish.
struct MuonBounds {
  bool ok;      // inside what the fp16 scales hold: |f| < 1.9, |b x + c x^2| < 7.9
  double p, q;  // the largest |a + b x + c x^2|, and the product of the steps'
};

MuonBounds muon_bounds(const moe_muon_config& cfg) {
  const double a = cfg.a, b = cfg.b, c = cfg.c;
  MuonBounds r{true, 0.0, 1.0};
  double X = 1.0;  // R^2
  for (int s = 0; s < cfg.steps; ++s) {
    double at[6] = {0.0, X, 0.0, 0.0, 0.0, 0.0};
    int n = 2;
    auto add = [&](double x) { if (x > 0.0 && x < X) at[n++] = x; };
    if (c != 0.0) {
      add(-b / (2.0 * c));  // of the polynomial itself
      const double d = 9.0 * b * b - 20.0 * a * c;
      if (d >= 0.0) {
        add((-3.0 * b + std::sqrt(d)) / (10.0 * c));
        add((-3.0 * b - std::sqrt(d)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      add(-a / (3.0 * b));
    }
    double next = 0.0, most = 0.0;
    for (int i = 0; i < n; ++i) {
      const double x = at[i], poly = b * x + c * x * x, f = (a + poly) * std::sqrt(x);
      if (!(std::fabs(poly) < 7.9) || !(std::fabs(f) < 1.9)) r.ok = false;
      next = std::fmax(next, std::fabs(f));
      most = std::fmax(most, std::fabs(a + poly));
    }
    if (!r.ok) break;
    r.p = std::fmax(r.p, most);
    r.q *= most;
    X = next * next;
  }
  return r;
}

// Products of hi and lo parts for matrices of at most 128 rows or columns.
bool muon_split(const moe_muon_config& c) { return c.rows <= 128 || c.cols <= 128; }

// The r x r form (muon_small.cuh) where one extent is at most 128 and Q stays small: its
// 22 bits are then 2^-22 * 1024 of the result or better.
bool muon_small(const moe_muon_config& c) {
  if (!muon_split(c)) return false;
  const MuonBounds m = muon_bounds(c);
  return m.q <= 1024.0 && m.p <= 15.0;
}

struct MuonSmallLayout {
  size_t status, part, part_exp, q, inv_norm, total;
  int pieces, gram_ctas;
};

MuonSmallLayout muon_small_layout(const moe_muon_config& c) {
  MuonSmallLayout L;
  const size_t G = c.groups;
  const int n = c.rows > c.cols ? c.rows : c.cols;
  L.pieces = (n + 127) / 128;
  // CTAs of the sums: one round of the GPU, at most kMsMaxParts a matrix (one CTA adds them up)
  const int64_t units = static_cast<int64_t>(c.groups) * L.pieces;
  int64_t ctas = static_cast<int64_t>(c.groups) * kMsMaxParts;
  if (ctas > 148) ctas = 148;
  if (ctas > units) ctas = units;
  L.gram_ctas = static_cast<int>(ctas);
  const size_t slots = G + L.gram_ctas;
  size_t o = 0;
  L.status = o; o = align_up(o + 4);
  L.part = o; o = align_up(o + slots * 8 * kMsThreads * 16);
  L.part_exp = o; o = align_up(o + slots * 4);
  L.q = o; o = align_up(o + G * 2 * kMsImage);
  L.inv_norm = o; o = align_up(o + G * 8);
  L.total = o;
  return L;
}

MuonLayout muon_layout(const moe_muon_config& c) {
  MuonLayout L;
  const size_t G = c.groups;
  const int64_t n = static_cast<int64_t>(c.rows) * c.cols;
  L.r = c.rows < c.cols ? c.rows : c.cols;
  L.ld = (c.cols + 7) / 8 * 8;
  L.ldr = (L.r + 7) / 8 * 8;
  // at most 1024 partial sums a matrix: a CTA has whole runs of 1024 elements, of 4096 (four
  // vector accesses in flight) where the GPU is full anyway (5 x [333, 215]: 140 -> 133 us)
  const int64_t part = (n + 1023) / 1024, unit = part > 2048 ? 4096 : 1024;
  const int64_t chunk = (part + unit - 1) / unit * unit;
  L.chunk = static_cast<int>(chunk);
  L.chunks = static_cast<int>((n + chunk - 1) / chunk);
  const bool split = muon_split(c);
  // 256 x 256 tiles by CTA pairs, which read half as much per product, where they fill the GPU
  // and are not mostly edge: 128 x 128 tiles of one CTA where there are at most three of them
  // for one of the large.  (Small against large: three each at 64 x [384, 2048] 1.24 and 1.33 ms,
  // 2.8 at 8 x [640, 640] 0.17 and 0.20; 3.4 at 16 x [1300, 1300] 1.73 and 1.43, four at
  // 16 x [1024, 1024] 0.71 and 0.57.)
  auto tiles = [&](int v) { return (v + L.tile - 1) / L.tile; };
  L.tile = 128;
  const int64_t small = static_cast<int64_t>(tiles(c.rows)) * tiles(c.cols);
  L.tile = 256;
  const int64_t large = static_cast<int64_t>(tiles(c.rows)) * tiles(c.cols);
  if (split || static_cast<int64_t>(G) * large < 74 || small <= 3 * large) L.tile = 128;
  L.sym_n = tiles(L.r);
  L.sym_tiles = L.sym_n * (L.sym_n + 1) / 2;
  L.app_n = tiles(c.cols);
  L.app_tiles = tiles(c.rows) * L.app_n;
  L.k_gram = ((c.rows <= c.cols ? c.cols : c.rows) + kNsBK - 1) / kNsBK;
  L.k_r = (L.r + kNsBK - 1) / kNsBK;
  // Gram tiles that leave most of the GPU idle are split along the contraction (at least
  // four 64-wide steps a part); a unit for each 32 columns of a warp's half tile adds them up
  const int64_t ctas = L.tile == 128 ? 148 : 74, gram = static_cast<int64_t>(c.groups) * L.sym_tiles;
  int64_t parts = gram < ctas ? ctas / gram : 1;
  if (parts > kNsMaxSplits) parts = kNsMaxSplits;
  if (parts > L.k_gram / 4) parts = L.k_gram / 4;
  L.splits = parts < 1 ? 1 : static_cast<int>(parts);
  L.sums = L.splits > 1 ? L.tile / 64 : 0;
  // claims; finished warps a matrix and product; left parts a Gram tile
  L.n_counters = static_cast<int>(1 + G * 3 * c.steps + (L.splits > 1 ? G * L.sym_tiles : 0));
  const size_t xb = G * static_cast<size_t>(c.rows) * L.ld * 2;
  const size_t ab = G * static_cast<size_t>(L.r) * L.ldr * 2;
  L.units = static_cast<int64_t>(c.groups) * c.steps *
            (static_cast<int64_t>(L.sym_tiles) * (L.splits + L.sums + 1) + L.app_tiles);
  size_t o = 0;
  L.status = o; o = align_up(o + 4);
  L.counters = o; o = align_up(o + static_cast<size_t>(L.n_counters) * 4);
  L.part = o; o = align_up(o + G * L.chunks * 8);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) { L.x[i][j] = o; o = align_up(o + xb); }
  for (int j = 0; j < 2; ++j) {
    L.a[j] = o; o = align_up(o + (j == 0 || split ? ab : 0));
    L.b[j] = o; o = align_up(o + (j == 0 || split ? ab : 0));
  }
  for (int j = 0; j < 2; ++j) { L.diag[j] = o; o = align_up(o + G * L.r * 4); }
  L.partial = o;
  o = align_up(o + G * L.sym_tiles * (L.splits > 1 ? L.splits : 0) * static_cast<size_t>(L.tile) * L.tile * 4);
  L.total = o;
  return L;
}

moe_status check_muon(const moe_muon_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->groups < 1 || c->rows < 1 || c->cols < 1 || c->steps < 1 || c->steps > 64)
    return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !(c->eps < 1.f)) return MOE_ERR_INVALID_ARG;
  if (c->groups > 65535) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->rows) * ((static_cast<int64_t>(c->cols) + 7) / 8 * 8) > (int64_t(1) << 30))
    return MOE_ERR_UNSUPPORTED;
  if (!muon_bounds(*c).ok) return MOE_ERR_UNSUPPORTED;
  if (!muon_small(*c) && muon_layout(*c).units > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// [groups, rows, inner] of 16-bit elements with row length ld: boxes of box_cols x box_rows,
// swizzled over the 128 or 64 bytes of a box row.
moe_status make_ns_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows,
                       uint64_t groups, uint64_t ld, uint32_t box_rows, uint32_t box_cols) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MOE_ERR_CUDA;
  cuuint64_t dims[3] = {inner, rows, groups};
  cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "moe_b200: cuTensorMapEncodeTiled (muon) failed (%d)\n", static_cast<int>(r));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// Persistent CTAs (pairs: clusters of two), as many as the units or the GPU has.
template <bool TALL, bool PAIR, bool SPLIT>
moe_status launch_ns(const NsParams& p, cudaStream_t s) {
  auto kern = ns_steps_kernel<TALL, PAIR, SPLIT>;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmemBytes));
  int ctas = sm_count() / (PAIR ? 2 : 1);
  // no more than one product of the whole stack keeps busy: a CTA that meets every product
  // has its instructions at hand (5 x [333, 215]: 199 us with 74 pairs, 195 with 10)
  const int64_t most = static_cast<int64_t>(p.groups) * std::max(p.sym_tiles * p.splits, p.app_tiles);
  if (most < ctas) ctas = static_cast<int>(most);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.gridDim = dim3(PAIR ? 2 * ctas : ctas);
  cfg.blockDim = dim3(kNsThreads);
  cfg.dynamicSmemBytes = kNsSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  MOE_CUDA(cudaLaunchKernelEx(&cfg, kern, p));
  return launch_check();
}

struct MuonArgs {
  const void* grad;
  bool grad_bf16;
  const float* mom_in;
  float* mom_out;
  float beta;
  bool nesterov;
  const __nv_bfloat16* w;
  __nv_bfloat16* out;
  float keep, step;
};

// All steps' products on tiles of one CTA or of a pair.
template <bool PAIR, bool SPLIT>
moe_status ns_steps(const moe_muon_config& c, const MuonArgs& u, const MuonLayout& L, uint8_t* b,
                    cudaStream_t s) {
  const bool wide = c.rows <= c.cols;
  const uint64_t G = c.groups, rows = c.rows, cols = c.cols, r = L.r;
  NsParams p;
  memset(&p, 0, sizeof(p));
  for (int j = 0; j < 2; ++j) {
    for (int i = 0; i < 2; ++i) {
      const void* x = b + L.x[i][j];
      MOE_TRY(make_ns_map(&p.x_gram[i][j], x, cols, rows, G, L.ld, wide ? 128 : 64, 64));
      MOE_TRY(make_ns_map(&p.x_apply[i][j], x, cols, rows, G, L.ld, wide ? 64 : 128, 64));
      MOE_TRY(make_ns_map(&p.x_blk[i][j], x, cols, rows, G, L.ld, 32, 32));
      const void* ab = b + (i == 0 ? L.a[j] : L.b[j]);
      if (!SPLIT && j) {  // A and B have no lo part there: not read
        p.ab_op[i][j] = p.ab_op[i][0];
        p.ab_blk[i][j] = p.ab_blk[i][0];
        continue;
      }
      MOE_TRY(make_ns_map(&p.ab_op[i][j], ab, r, r, G, L.ldr, 128, 64));
      MOE_TRY(make_ns_map(&p.ab_blk[i][j], ab, r, r, G, L.ldr, 32, 32));
      if (j == 0) MOE_TRY(make_ns_map(&p.ab_mir[i], ab, r, r, G, L.ldr, 64, 64));
    }
  }
  p.tma_out = c.cols % 8 == 0 && aligned16(u.out) && aligned16(u.w) ? 1 : 0;
  p.out_map = p.w_map = p.x_blk[0][0];  // not read without tma_out
  if (p.tma_out) {
    MOE_TRY(make_ns_map(&p.out_map, u.out, cols, rows, G, cols, 32, 32));
    if (u.w) MOE_TRY(make_ns_map(&p.w_map, u.w, cols, rows, G, cols, 32, 32));
  }
  p.groups = c.groups;
  p.rows = c.rows;
  p.cols = c.cols;
  p.r = L.r;
  p.steps = c.steps;
  p.sym_tiles = L.sym_tiles;
  p.sym_n = L.sym_n;
  p.app_tiles = L.app_tiles;
  p.app_n = L.app_n;
  p.k_gram = L.k_gram;
  p.k_r = L.k_r;
  p.splits = L.splits;
  p.sums = L.sums;
  p.total = static_cast<int32_t>(L.units);
  int32_t* counters = reinterpret_cast<int32_t*>(b + L.counters);
  p.unit_counter = counters;
  p.done = counters + 1;
  p.split_done = p.done + static_cast<size_t>(c.groups) * 3 * c.steps;
  p.partial = reinterpret_cast<float4*>(b + L.partial);
  for (int j = 0; j < 2; ++j) p.diag[j] = reinterpret_cast<float*>(b + L.diag[j]);
  p.out = u.out;
  p.w = u.w;
  p.a = c.a;
  p.b = c.b;
  p.c = c.c;
  p.keep = u.keep;
  p.step = u.step;
  p.status = status_ptr(b);
  return wide ? launch_ns<false, PAIR, SPLIT>(p, s) : launch_ns<true, PAIR, SPLIT>(p, s);
}

template <typename K>
moe_status launch_ms(K kern, dim3 grid, int smem, cudaStream_t s, const MuonSmallArgs& a) {
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  MOE_TRY(launch_pdl(kern, grid, dim3(kMsThreads), smem, s, a));
  return launch_check();
}

moe_status muon_small_run(const moe_muon_config& c, const MuonArgs& u, void* ws, cudaStream_t s) {
  const MuonSmallLayout L = muon_small_layout(c);
  uint8_t* b = static_cast<uint8_t*>(ws);
  MuonSmallArgs a;
  memset(&a, 0, sizeof(a));
  a.grad = u.grad;
  a.mom_in = u.mom_in;
  a.mom_out = u.mom_out;
  a.w = u.w;
  a.out = u.out;
  a.part = reinterpret_cast<float4*>(b + L.part);
  a.part_exp = reinterpret_cast<int32_t*>(b + L.part_exp);
  a.q = b + L.q;
  a.inv_norm = reinterpret_cast<double*>(b + L.inv_norm);
  a.rows = c.rows;
  a.cols = c.cols;
  a.tall = c.rows > c.cols ? 1 : 0;
  a.r = a.tall ? c.cols : c.rows;
  a.r16 = (a.r + 15) / 16 * 16;
  a.pieces = L.pieces;
  a.units = static_cast<int64_t>(c.groups) * L.pieces;
  a.gram_ctas = L.gram_ctas;
  a.steps = c.steps;
  a.nesterov = u.nesterov ? 1 : 0;
  a.beta = u.beta;
  a.a = c.a;
  a.b = c.b;
  a.c = c.c;
  a.eps = c.eps;
  a.keep = u.keep;
  a.step = u.step;
  a.sq = std::exp2(std::floor(std::log2(60000.0 / std::fmax(muon_bounds(c).q, 1.0))));
  a.status = status_ptr(b);
  const bool vec = c.cols % 4 == 0 && aligned16(u.grad) && aligned16(u.mom_in) && aligned16(u.mom_out);
  const bool out_vec = c.cols % 4 == 0 && aligned16(u.out) && aligned16(u.w);
  const dim3 grid(static_cast<unsigned>(L.gram_ctas));
  const dim3 agrid(static_cast<unsigned>(a.units < sm_count() ? a.units : sm_count()));
  auto run = [&](auto gram, auto apply) -> moe_status {
    MOE_TRY(launch_ms(gram, grid, kMsGramSmem, s, a));
    MOE_TRY(launch_ms(muon_chain_kernel, dim3(c.groups), kMsChainSmem, s, a));
    return launch_ms(apply, agrid, kMsApplySmem, s, a);
  };
  using bf = __nv_bfloat16;
  if (u.grad_bf16) {
    if (vec) return out_vec ? run(muon_gram_kernel<bf, true>, muon_apply_kernel<bf, true, true>)
                            : run(muon_gram_kernel<bf, true>, muon_apply_kernel<bf, true, false>);
    return run(muon_gram_kernel<bf, false>, muon_apply_kernel<bf, false, false>);
  }
  if (vec) return out_vec ? run(muon_gram_kernel<float, true>, muon_apply_kernel<float, true, true>)
                          : run(muon_gram_kernel<float, true>, muon_apply_kernel<float, true, false>);
  return run(muon_gram_kernel<float, false>, muon_apply_kernel<float, false, false>);
}

moe_status muon_run(const moe_muon_config& c, const MuonArgs& u, void* ws, cudaStream_t s) {
  if (muon_small(c)) return muon_small_run(c, u, ws, s);
  const MuonLayout L = muon_layout(c);
  uint8_t* b = static_cast<uint8_t*>(ws);
  MuonInArgs a;
  memset(&a, 0, sizeof(a));
  a.grad = u.grad;
  a.mom_in = u.mom_in;
  a.mom_out = u.mom_out;
  a.part = reinterpret_cast<double*>(b + L.part);
  a.hi = reinterpret_cast<__half*>(b + L.x[0][0]);
  a.lo = reinterpret_cast<__half*>(b + L.x[0][1]);
  a.n = static_cast<int64_t>(c.rows) * c.cols;
  a.cols = c.cols;
  a.ld = L.ld;
  a.chunk = L.chunk;
  a.chunks = L.chunks;
  a.nesterov = u.nesterov ? 1 : 0;
  a.beta = u.beta;
  a.eps = c.eps;
  a.counters = reinterpret_cast<int32_t*>(b + L.counters);
  a.n_counters = L.n_counters;
  // vectors of four where no vector crosses a row or a matrix's alignment
  const bool vec = c.cols % 4 == 0 && aligned16(u.grad) && aligned16(u.mom_in) && aligned16(u.mom_out);
  const dim3 grid(static_cast<unsigned>(L.chunks), static_cast<unsigned>(c.groups)), block(256);
  auto in = [&](auto norm, auto scale) -> moe_status {
    MOE_TRY(launch_pdl(norm, grid, block, 0, s, a));
    MOE_TRY(launch_check());
    MOE_TRY(launch_pdl(scale, grid, block, 0, s, a));
    return launch_check();
  };
  if (u.grad_bf16)
    MOE_TRY(vec ? in(muon_norm_kernel<__nv_bfloat16, true>, muon_scale_kernel<__nv_bfloat16, true>)
                : in(muon_norm_kernel<__nv_bfloat16, false>, muon_scale_kernel<__nv_bfloat16, false>));
  else
    MOE_TRY(vec ? in(muon_norm_kernel<float, true>, muon_scale_kernel<float, true>)
                : in(muon_norm_kernel<float, false>, muon_scale_kernel<float, false>));
  if (muon_split(c)) return ns_steps<false, true>(c, u, L, b, s);
  return L.tile == 256 ? ns_steps<true, false>(c, u, L, b, s) : ns_steps<false, false>(c, u, L, b, s);
}

size_t muon_bytes(const moe_muon_config& c) {
  return muon_small(c) ? muon_small_layout(c).total : muon_layout(c).total;
}

moe_status check_muon_call(const moe_muon_config* cfg, const void* grad, int32_t grad_dtype,
                           void* ws, size_t bytes) {
  MOE_TRY(check_muon(cfg));
  if (!grad || (grad_dtype != MOE_GRAD_FP32 && grad_dtype != MOE_GRAD_BF16)) return MOE_ERR_INVALID_ARG;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % kAlign) return MOE_ERR_INVALID_ARG;
  if (bytes < muon_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_muon_workspace_size(const moe_muon_config* cfg, size_t* bytes) {
  MOE_TRY(check_muon(cfg));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = muon_bytes(*cfg);
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_muon_config* cfg, const void* g, int32_t g_dtype, void* out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  MOE_TRY(check_muon_call(cfg, g, g_dtype, workspace, workspace_bytes));
  if (!out) return MOE_ERR_INVALID_ARG;
  MuonArgs u;
  memset(&u, 0, sizeof(u));
  u.grad = g;
  u.grad_bf16 = g_dtype == MOE_GRAD_BF16;
  u.out = static_cast<__nv_bfloat16*>(out);
  return muon_run(*cfg, u, workspace, static_cast<cudaStream_t>(stream));
}

moe_status moe_muon_step(const moe_muon_config* cfg, const void* grad, int32_t grad_dtype,
                         const float* momentum_in, float* momentum_out, float beta,
                         int32_t nesterov, const void* w_in, void* w_out, float step, float decay,
                         void* workspace, size_t workspace_bytes, void* stream) {
  MOE_TRY(check_muon_call(cfg, grad, grad_dtype, workspace, workspace_bytes));
  if (!momentum_in || !momentum_out || !w_in || !w_out) return MOE_ERR_INVALID_ARG;
  if (!(beta >= 0.f && beta < 1.f) || (nesterov != 0 && nesterov != 1)) return MOE_ERR_INVALID_ARG;
  MuonArgs u;
  u.grad = grad;
  u.grad_bf16 = grad_dtype == MOE_GRAD_BF16;
  u.mom_in = momentum_in;
  u.mom_out = momentum_out;
  u.beta = beta;
  u.nesterov = nesterov != 0;
  u.w = static_cast<const __nv_bfloat16*>(w_in);
  u.out = static_cast<__nv_bfloat16*>(w_out);
  u.keep = 1.f - decay;
  u.step = step;
  return muon_run(*cfg, u, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
