// Host side of the scored router, its gradient and the balance loss (part of moe_api.cu's
// translation unit).  The kernels are in route_scored.cuh.
#pragma once

namespace {

// Dispatch on the logits a lane holds: f(std::integral_constant<int, PER>).
template <typename F>
moe_status by_experts(int E, F f) {
  const int per = (E + 31) / 32;
  if (per <= 1) return f(std::integral_constant<int, 1>());
  if (per <= 2) return f(std::integral_constant<int, 2>());
  if (per <= 4) return f(std::integral_constant<int, 4>());
  if (per <= 8) return f(std::integral_constant<int, 8>());
  if (per <= 12) return f(std::integral_constant<int, 12>());
  if (per <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

moe_status check_router(const moe_router* r) {
  if (!r) return MOE_ERR_INVALID_ARG;
  if (r->score != MOE_SCORE_SIGMOID && r->score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
  if (r->renormalize != 0 && r->renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (r->group_top != 1 && r->group_top != 2) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status do_route_scored(const moe_config& c, const moe_router& r, const void* x,
                           const void* w_router, const float* bias, const float* logits_in,
                           float* logits_out, int32_t* topk_idx, float* topk_w, void* ws,
                           cudaStream_t s) {
  ScoredArgs a;
  memset(&a, 0, sizeof(a));
  if (logits_in) {
    a.logits = logits_in;
  } else {
    MOE_TRY(router_gemm(c, x, w_router, ws, s, &a.partials, &a.n_splits));
    a.logits_out = logits_out;
  }
  a.bias = bias;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.T = c.T;
  a.E = c.E;
  a.G = c.n_group;
  a.g = c.topk_group;
  a.k = c.top_k;
  a.size = c.E / c.n_group;
  a.size_magic = static_cast<uint32_t>(((1ull << 32) + a.size - 1) / a.size);
  a.rsf = c.routed_scaling_factor;
  a.score = r.score;
  a.renorm = r.renormalize;
  a.group_top = r.group_top;
  a.vec4 = c.E % 4 == 0 && aligned16(a.n_splits > 0 ? a.partials : a.logits) ? 1 : 0;
  return by_experts(c.E, [&](auto per) -> moe_status {
    constexpr int PER = decltype(per)::value;
    const int lanes = a.size % PER == 0 ? a.size / PER : 0;
    a.lane_shift = -1;
    if (lanes > 0 && (lanes & (lanes - 1)) == 0)
      for (a.lane_shift = 0; (1 << a.lane_shift) < lanes;) ++a.lane_shift;
    // the form is compiled in where rows are short enough that its branches show
    auto kern = route_scored_kernel<PER, -1, -1>;
    if constexpr (PER == 8 || PER == 12) {
      kern = r.score == MOE_SCORE_SOFTMAX
                 ? (bias ? route_scored_kernel<PER, 1, 1> : route_scored_kernel<PER, 1, 0>)
                 : (bias ? route_scored_kernel<PER, 0, 1> : route_scored_kernel<PER, 0, 0>);
    }
    const int want = (c.T + kRsWarps - 1) / kRsWarps, most = sm_count() * 8;
    MOE_TRY(launch_pdl(kern, dim3(want < most ? want : most), dim3(kRsWarps * 32), 0, s, a));
    return launch_check();
  });
}

// What the balance loss adds to the router's gradient (dscore null: nothing).
struct BalanceGrad {
  const float* dscore;
  const int32_t* seq_offsets;
  int32_t n_seq;
  const float* dloss;
};

moe_status do_route_backward(const moe_config& c, const moe_router& r, const float* logits,
                             const int32_t* topk_idx, const float* dgate, const BalanceGrad& bal,
                             float* dlogits, __nv_bfloat16* dense_b, int col_b, int ld_b,
                             cudaStream_t s) {
  RouteBwdArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.dgate = dgate;
  a.dscore = bal.dscore;
  a.dloss = bal.dloss;
  a.seq_offsets = bal.seq_offsets;
  a.n_seq = bal.n_seq;
  a.dlogits = dlogits;
  a.dense_b = dense_b;
  a.col_b = col_b;
  a.ld_b = ld_b;
  a.T = c.T;
  a.E = c.E;
  a.k = c.top_k;
  a.rsf = c.routed_scaling_factor;
  a.score = r.score;
  a.renorm = r.renormalize;
  const bool vec = c.E % 4 == 0 && aligned16(logits) && aligned16(dlogits) && aligned16(bal.dscore);
  return by_experts(c.E, [&](auto per) -> moe_status {
    constexpr int PER = decltype(per)::value;
    auto kern = route_backward_kernel<PER, false>;
    if constexpr (PER % 4 == 0) {
      if (vec) kern = route_backward_kernel<PER, true>;
    }
    // one wave of 32 warps an SM, equal runs
    const int blocks = (c.T + kRsWarps - 1) / kRsWarps, wave = 8 * sm_count();
    a.rows = (blocks + wave - 1) / wave;
    const int warps = (c.T + a.rows - 1) / a.rows;
    MOE_TRY(launch_pdl(kern, dim3((warps + kRsWarps - 1) / kRsWarps), dim3(kRsWarps * 32), 0, s, a));
    return launch_check();
  });
}

moe_status check_balance_grad(const BalanceGrad& b) {
  if (b.dscore && b.n_seq < 1) return MOE_ERR_INVALID_ARG;
  if (b.dscore && !b.seq_offsets && b.n_seq != 1) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct BalanceLayout {
  size_t part, part_load, part_rows, seq_loss, done, total;
  int tiles, tile_rows;
};

BalanceLayout balance_layout(const moe_config& c, int32_t n_seq) {
  BalanceLayout L;
  // rows a block: one a warp until the blocks fill the GPU, at most 128
  int rows = (c.T / 148 + kBalWarps - 1) / kBalWarps * kBalWarps;
  L.tile_rows = rows < kBalWarps ? kBalWarps : (rows > 128 ? 128 : rows);
  L.tiles = static_cast<int>((static_cast<int64_t>(c.T) + L.tile_rows - 1) / L.tile_rows) + n_seq;
  const size_t n = static_cast<size_t>(L.tiles) * c.E * 4;
  size_t o = 0;
  L.part = o; o = align_up(o + n);
  L.part_load = o; o = align_up(o + n);
  L.part_rows = o; o = align_up(o + static_cast<size_t>(L.tiles) * 4);
  L.seq_loss = o;
  o = align_up(o + static_cast<size_t>(n_seq) * ((c.E + kBalExperts - 1) / kBalExperts) * 8);
  L.done = o; o = align_up(o + 4);
  L.total = o;
  return L;
}

moe_status check_balance(const moe_config* c, int32_t n_seq) {
  MOE_TRY(check_config(c));
  if (n_seq < 1) return MOE_ERR_INVALID_ARG;
  if (n_seq > (1 << 20) || c->T > (1 << 28)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_scored(const moe_config* cfg, const moe_router* router, const void* x,
                            const void* w_router, const float* bias, const float* logits_in,
                            float* logits_out, int32_t* topk_idx, float* topk_w, void* workspace,
                            size_t workspace_bytes, void* stream) {
  MOE_TRY(check_config(cfg));
  MOE_TRY(check_router(router));
  if (!topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!logits_in) {
    MOE_TRY(check_ws(*cfg, workspace, workspace_bytes));
    if (!x || !w_router || !logits_out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w_router)) return MOE_ERR_INVALID_ARG;
  }
  return do_route_scored(*cfg, *router, x, w_router, bias, logits_in, logits_out, topk_idx, topk_w,
                         workspace, static_cast<cudaStream_t>(stream));
}

moe_status moe_forward_scored(const moe_config* cfg, const moe_router* router, const moe_weights* w,
                              const void* w_router, const float* bias, const void* x, void* y,
                              int32_t xy_on_host, void* workspace, size_t workspace_bytes,
                              void* stream) {
  MOE_TRY(check_router(router));
  return forward_layer(cfg, router, w, w_router, bias, x, y, xy_on_host, workspace,
                       workspace_bytes, stream);
}

moe_status moe_route_backward(const moe_config* cfg, const moe_router* router, const float* logits,
                              const int32_t* topk_idx, const float* dgate, const float* dscore,
                              const int32_t* seq_offsets, int32_t n_seq, const float* dloss,
                              float* dlogits, void* stream) {
  MOE_TRY(check_config(cfg));
  MOE_TRY(check_router(router));
  if (!logits || !topk_idx || !dgate || !dlogits) return MOE_ERR_INVALID_ARG;
  const BalanceGrad b{dscore, seq_offsets, n_seq, dloss};
  MOE_TRY(check_balance_grad(b));
  return do_route_backward(*cfg, *router, logits, topk_idx, dgate, b, dlogits, nullptr, 0, 0,
                           static_cast<cudaStream_t>(stream));
}

moe_status moe_balance_workspace_size(const moe_config* cfg, int32_t n_seq, size_t* bytes) {
  MOE_TRY(check_balance(cfg, n_seq));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = balance_layout(*cfg, n_seq).total;
  return MOE_OK;
}

moe_status moe_balance_loss(const moe_config* cfg, const moe_router* router, const float* logits,
                            const int32_t* topk_idx, const int32_t* seq_offsets, int32_t n_seq,
                            float coef, float* loss, int32_t* load, float* dscore, void* workspace,
                            size_t workspace_bytes, void* stream) {
  MOE_TRY(check_balance(cfg, n_seq));
  MOE_TRY(check_router(router));
  if (!logits || !topk_idx || !loss || !load || !dscore) return MOE_ERR_INVALID_ARG;
  if (!seq_offsets && n_seq != 1) return MOE_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign) return MOE_ERR_INVALID_ARG;
  const BalanceLayout L = balance_layout(*cfg, n_seq);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  uint8_t* b = static_cast<uint8_t*>(workspace);
  BalanceArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.seq_offsets = seq_offsets;
  a.part = reinterpret_cast<float*>(b + L.part);
  a.part_load = reinterpret_cast<int32_t*>(b + L.part_load);
  a.part_rows = reinterpret_cast<int32_t*>(b + L.part_rows);
  a.seq_loss = reinterpret_cast<double*>(b + L.seq_loss);
  a.done = reinterpret_cast<int32_t*>(b + L.done);
  a.loss = loss;
  a.load = load;
  a.dscore = dscore;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->top_k;
  a.n_seq = n_seq;
  a.tile_rows = L.tile_rows;
  a.tiles = seq_offsets ? L.tiles : (cfg->T + L.tile_rows - 1) / L.tile_rows;
  a.coef = coef;
  a.score = router->score;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = cfg->E % 4 == 0 && aligned16(logits);
  MOE_TRY(by_experts(cfg->E, [&](auto per) -> moe_status {
    constexpr int PER = decltype(per)::value;
    auto kern = balance_rows_kernel<PER, false>;
    if constexpr (PER % 4 == 0) {
      if (vec) kern = balance_rows_kernel<PER, true>;
    }
    MOE_TRY(launch_pdl(kern, dim3(a.tiles), dim3(kBalWarps * 32), 0, s, a));
    return launch_check();
  }));
  a.e_blocks = (cfg->E + kBalExperts - 1) / kBalExperts;
  MOE_TRY(launch_pdl(balance_finish_kernel, dim3(n_seq * a.e_blocks),
                     dim3(kBalExperts * kBalSlices), 0, s, a));
  return launch_check();
}

}  // extern "C"
