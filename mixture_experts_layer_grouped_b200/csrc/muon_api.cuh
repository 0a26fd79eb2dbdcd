// Host side of the orthogonalised updates (part of moe_api.cu's translation unit): the
// workspace layout, the launches and the C ABI calls of include/moe_b200.h's Muon section.
// The kernels are in muon.cuh.
#pragma once

namespace {

struct MuonLayout {
  size_t status, part, x[2][2], a[2], b[2], da, db, total;  // [buffer][hi, lo], [hi, lo]
  int r, ld, ldr, chunk, chunks;
};

// One-CTA tiles and products of hi and lo parts for matrices of at most 128 rows or columns.
bool muon_split(const moe_muon_config& c) { return c.rows <= 128 || c.cols <= 128; }

MuonLayout muon_layout(const moe_muon_config& c) {
  MuonLayout L;
  const size_t G = c.groups;
  const int64_t n = static_cast<int64_t>(c.rows) * c.cols;
  L.r = c.rows < c.cols ? c.rows : c.cols;
  L.ld = (c.cols + 7) / 8 * 8;
  L.ldr = (L.r + 7) / 8 * 8;
  // at most 256 partial sums a matrix, each of at least 4096 elements
  int64_t chunk = ((n + 255) / 256 + 1023) / 1024 * 1024;
  if (chunk < 4096) chunk = 4096;
  L.chunk = static_cast<int>(chunk);
  L.chunks = static_cast<int>((n + chunk - 1) / chunk);
  const size_t xb = G * static_cast<size_t>(c.rows) * L.ld * 2;
  const size_t ab = G * static_cast<size_t>(L.r) * L.ldr * 2;
  size_t o = 0;
  L.status = o; o = align_up(o + 4);
  L.part = o; o = align_up(o + G * L.chunks * 8);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) { L.x[i][j] = o; o = align_up(o + xb); }
  const bool split = muon_split(c);
  for (int j = 0; j < 2; ++j) {
    L.a[j] = o; o = align_up(o + (j == 0 || split ? ab : 0));
    L.b[j] = o; o = align_up(o + (j == 0 || split ? ab : 0));
  }
  L.da = o; o = align_up(o + G * L.r * 4);
  L.db = o; o = align_up(o + G * L.r * 4);
  L.total = o;
  return L;
}

// The largest |singular value| that the steps can reach from [0, 1], and the largest
// |b x + c x^2| on the way, must stay inside what the fp16 scales hold.
bool muon_bounded(const moe_muon_config& c) {
  const int kPoints = 4096;
  double R = 1.0;
  for (int s = 0; s < c.steps; ++s) {
    double next = 0.0;
    for (int i = 0; i <= kPoints; ++i) {
      const double v = R * i / kPoints, x = v * v;
      const double poly = static_cast<double>(c.b) * x + static_cast<double>(c.c) * x * x;
      const double y = (c.a + poly) * v;
      if (!(poly > -7.9 && poly < 7.9)) return false;
      if (!(y > -1.9 && y < 1.9)) return false;
      next = y < 0 ? (-y > next ? -y : next) : (y > next ? y : next);
    }
    R = next;
  }
  return true;
}

moe_status check_muon(const moe_muon_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->groups < 1 || c->rows < 1 || c->cols < 1 || c->steps < 1 || c->steps > 64)
    return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !(c->eps < 1.f)) return MOE_ERR_INVALID_ARG;
  if (c->groups > 65535) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->rows) * ((static_cast<int64_t>(c->cols) + 7) / 8 * 8) > (int64_t(1) << 30))
    return MOE_ERR_UNSUPPORTED;
  if (!muon_bounded(*c)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// [groups, rows, inner] fp16 with row length ld: boxes of 64 elements x box_rows rows.
moe_status make_ns_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows,
                       uint64_t groups, uint64_t ld, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return MOE_ERR_CUDA;
  cuuint64_t dims[3] = {inner, rows, groups};
  cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "moe_b200: cuTensorMapEncodeTiled (muon) failed (%d)\n", static_cast<int>(r));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

template <int MODE, bool A_MN, bool B_MN, bool PAIR, bool LAST>
moe_status launch_ns(const NsParams& p, cudaStream_t s) {
  auto kern = ns_gemm_kernel<MODE, A_MN, B_MN, PAIR, LAST>;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmemBytes));
  int ctas = sm_count() / (PAIR ? 2 : 1);
  if (p.total < ctas) ctas = p.total;
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

// The steps' three products on tiles of one CTA or of a pair.
template <bool PAIR>
moe_status ns_steps(const moe_muon_config& c, const MuonArgs& u, const MuonLayout& L, uint8_t* b,
                    cudaStream_t s) {
  constexpr int TILE = PAIR ? 256 : 128;
  const bool wide = c.rows <= c.cols;
  const int r = L.r;
  const uint64_t G = c.groups, rows = c.rows, cols = c.cols;
  auto float_at = [&](size_t off) { return reinterpret_cast<float*>(b + off); };
  auto half_at = [&](size_t off) { return reinterpret_cast<__half*>(b + off); };
  auto tiles = [](int n) { return (n + TILE - 1) / TILE; };
  const int rt = tiles(r);
  NsParams sym;
  memset(&sym, 0, sizeof(sym));
  sym.M = sym.N = r;
  sym.n_tiles = rt;
  sym.per_group = rt * (rt + 1) / 2;
  sym.total = c.groups * sym.per_group;
  sym.ld = L.ldr;
  sym.stride = static_cast<int64_t>(r) * L.ldr;
  sym.status = status_ptr(b);
  for (int k = 0; k < c.steps; ++k) {
    const int in = k & 1;
    // A = X X^T or X^T X
    NsParams g = sym;
    const uint32_t box = wide ? 128 : 64;
    MOE_TRY(make_ns_map(&g.a, b + L.x[in][0], cols, rows, G, L.ld, box));
    MOE_TRY(make_ns_map(&g.a_lo, b + L.x[in][1], cols, rows, G, L.ld, box));
    g.b = g.a;
    g.b_lo = g.a_lo;
    g.ksteps = ((wide ? c.cols : c.rows) + kNsBK - 1) / kNsBK;
    g.out_hi = half_at(L.a[0]);
    g.out_lo = half_at(L.a[1]);
    g.out_diag = float_at(L.da);
    g.alpha = kNsSa / (kNsSx * kNsSx);
    if (wide) MOE_TRY((launch_ns<kNsGram, false, false, PAIR, false>(g, s)));
    else MOE_TRY((launch_ns<kNsGram, true, true, PAIR, false>(g, s)));
    // B = b A + c A^2
    NsParams q = sym;
    MOE_TRY(make_ns_map(&q.a, b + L.a[0], r, r, G, L.ldr, 128));
    MOE_TRY(make_ns_map(&q.a_lo, b + L.a[1], r, r, G, L.ldr, 128));
    q.b = q.a;
    q.b_lo = q.a_lo;
    q.ksteps = (r + kNsBK - 1) / kNsBK;
    q.in_hi = half_at(L.a[0]);
    q.in_lo = half_at(L.a[1]);
    q.in_diag = float_at(L.da);
    q.out_hi = half_at(L.b[0]);
    q.out_lo = half_at(L.b[1]);
    q.out_diag = float_at(L.db);
    q.alpha = c.c * kNsSb / (kNsSa * kNsSa);
    q.beta = c.b * kNsSb / kNsSa;
    MOE_TRY((launch_ns<kNsPoly, false, false, PAIR, false>(q, s)));
    // X' = a X + B X or a X + X B
    NsParams x;
    memset(&x, 0, sizeof(x));
    x.M = c.rows;
    x.N = c.cols;
      x.n_tiles = tiles(c.cols);
    x.per_group = tiles(c.rows) * x.n_tiles;
    x.total = c.groups * x.per_group;
    x.ksteps = q.ksteps;
    x.ld = L.ld;
    x.stride = static_cast<int64_t>(c.rows) * L.ld;
    x.in_hi = half_at(L.x[in][0]);
    x.in_lo = half_at(L.x[in][1]);
    x.out_hi = half_at(L.x[in ^ 1][0]);
    x.out_lo = half_at(L.x[in ^ 1][1]);
    x.in_diag = float_at(L.db);
    x.alpha = 1.f / kNsSb;
    x.beta = c.a;
    x.diag_scale = 1.f / kNsSb;
    x.tall = wide ? 0 : 1;
    x.status = status_ptr(b);
    x.out = u.out;
    x.w = u.w;
    x.keep = u.keep;
    x.step = u.step;
    const bool last = k + 1 == c.steps;
    CUtensorMap bm[2], xm[2];
    for (int j = 0; j < 2; ++j) {
      MOE_TRY(make_ns_map(&bm[j], b + L.b[j], r, r, G, L.ldr, 128));
      MOE_TRY(make_ns_map(&xm[j], b + L.x[in][j], cols, rows, G, L.ld, wide ? 64 : 128));
    }
    x.a = wide ? bm[0] : xm[0];
    x.a_lo = wide ? bm[1] : xm[1];
    x.b = wide ? xm[0] : bm[0];
    x.b_lo = wide ? xm[1] : bm[1];
    if (wide) {
      if (last) MOE_TRY((launch_ns<kNsApply, false, true, PAIR, true>(x, s)));
      else MOE_TRY((launch_ns<kNsApply, false, true, PAIR, false>(x, s)));
    } else {
      if (last) MOE_TRY((launch_ns<kNsApply, false, false, PAIR, true>(x, s)));
      else MOE_TRY((launch_ns<kNsApply, false, false, PAIR, false>(x, s)));
    }
  }
  return MOE_OK;
}

moe_status muon_run(const moe_muon_config& c, const MuonArgs& u, void* ws, cudaStream_t s) {
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
  return muon_split(c) ? ns_steps<false>(c, u, L, b, s) : ns_steps<true>(c, u, L, b, s);
}

moe_status check_muon_call(const moe_muon_config* cfg, const void* grad, int32_t grad_dtype,
                           void* ws, size_t bytes) {
  MOE_TRY(check_muon(cfg));
  if (!grad || (grad_dtype != MOE_GRAD_FP32 && grad_dtype != MOE_GRAD_BF16)) return MOE_ERR_INVALID_ARG;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % kAlign) return MOE_ERR_INVALID_ARG;
  if (bytes < muon_layout(*cfg).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_muon_workspace_size(const moe_muon_config* cfg, size_t* bytes) {
  MOE_TRY(check_muon(cfg));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = muon_layout(*cfg).total;
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
