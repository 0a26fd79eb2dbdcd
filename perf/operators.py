"""The layer's training operators, measured: routing by softmax or sigmoid scores, its gradient,
the balance loss, and the orthogonalised (Muon) update of stacked matrices.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes a
case's inputs on the GPU, ``run`` makes one pass (plain torch operations, or the library's calls
where ``own`` is set), ``exact`` computes the same in 64 bits from the definitions, and ``work``
counts the bytes and operations that a pass cannot do without.
"""

import math

import torch

own = False

SIGMOID, SOFTMAX = 0, 1
NS = (3.4445, -4.7750, 2.0315)  # the quintic's coefficients
EPS = 1e-7
BETA, STEP, DECAY = 0.95, 0.02, 0.002
COEF = 1e-3
RSF = 2.5


def _route(name, T, E, k, score, renorm, groups=1, kept=1, top=1, bias=True, masked=False):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, renorm=renorm, groups=groups,
                kept=kept, top=top, bias=bias, masked=masked)


def _back(name, T, E, k, score, renorm, seqs=0, masked=False):
    """seqs > 0: the balance loss's gradient over so many sequences is added."""
    return dict(name=name, op="back", T=T, E=E, k=k, score=score, renorm=renorm, seqs=seqs,
                masked=masked)


def _balance(name, T, E, k, score, seqs, masked=False):
    return dict(name=name, op="balance", T=T, E=E, k=k, score=score, seqs=seqs, masked=masked)


def _ortho(name, G, M, N, grad, momentum, rank):
    """momentum: the whole optimiser step (momentum, update, weights); without it the
    orthogonalised matrix alone.  rank: rows that the gradient is summed over."""
    return dict(name=name, op="muon" if momentum else "ortho", G=G, M=M, N=N, grad=grad, rank=rank)


def listed():
    return [
        # one token of a serving step: latency alone
        _route("route one token", 1, 256, 8, SOFTMAX, True, bias=False),
        # a serving batch of the 384-expert geometry with groups kept by their best expert
        _route("route serving batch", 1024, 384, 6, SOFTMAX, False, 8, 4, 1),
        # a long prefill, aux-loss-free bias and top-2 groups
        _route("route prefill", 65536, 256, 8, SIGMOID, True, 8, 4, 2),
        # a training micro-batch of the 64-expert layer
        _back("route gradient 64 experts", 2048, 64, 6, SOFTMAX, False),
        # a long batch of the 384-expert geometry, packed sequences, balance loss
        _back("route gradient with balance", 32768, 384, 8, SIGMOID, True, seqs=24),
        # the 64-expert layer's micro-batch as one sequence
        _balance("balance one sequence", 2048, 64, 6, SIGMOID, 1),
        # a long batch of packed sequences of many lengths
        _balance("balance packed", 65536, 256, 8, SOFTMAX, 40),
        # the tiny layer's experts: one tile a matrix
        _ortho("orthogonalize tiny experts", 16, 128, 256, "float32", False, 16),
        # odd sizes, bf16 gradients
        _ortho("muon odd sizes", 5, 333, 215, "bfloat16", True, 90),
        # the 384-expert geometry's router weight: one wide matrix
        _ortho("muon router weight", 1, 384, 7168, "float32", True, 4096),
        # the 64-expert layer's down projections (taller than wide)
        _ortho("muon 64 experts down", 64, 2048, 1024, "float32", True, 192),
        # a slice of the 256-expert layer's up projections
        _ortho("muon 32 experts up", 32, 2048, 4096, "bfloat16", True, 96),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "back", "balance", "ortho", "muon"])
    if op in ("ortho", "muon"):
        while True:
            M, N, G = _log(rng, 1, 4096), _log(rng, 1, 7168), _log(rng, 1, 64)
            r, n = min(M, N), max(M, N)
            if G * (3.0 * r * r * n + float(r) ** 3) <= 32 * 5.8e10 and G * M * N <= 2.6e8:
                break
        c = _ortho("", G, M, N, rng.choice(["float32", "bfloat16"]), op == "muon",
                   _log(rng, 1, 512))
        del c["name"]
        return c
    T = _log(rng, 1, 65536)
    groups = rng.choice([1, 1, 4, 8])
    E = groups * max(2, _log(rng, 8, 384) // groups)
    if T * E > 32768 * 384:
        T = 32768 * 384 // E
    score, renorm = rng.choice([SIGMOID, SOFTMAX]), rng.random() < 0.5
    masked = rng.random() < 0.25
    kept = rng.randint(max(1, groups // 2), groups)
    k = rng.randint(1, min(12, kept * (E // groups)))
    if op == "route":
        c = _route("", T, E, k, score, renorm, groups, kept, rng.choice([1, 2]),
                   rng.random() < 0.7, masked)
    elif op == "back":
        c = _back("", T, E, k, score, renorm, rng.choice([0, 1, _log(rng, 1, 64)]), masked)
    else:
        c = _balance("", T, E, k, score, _log(rng, 1, 64), masked)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _logits(case, g):
    """Router logits as a trained router's: standard normal with experts of different mean."""
    T, E = case["T"], case["E"]
    x = torch.randn(T, E, generator=g, device="cuda")
    x += 0.5 * torch.randn(E, generator=g, device="cuda")
    if case["masked"]:  # experts switched off for some tokens, and padded rows with none left
        x[torch.rand(T, E, generator=g, device="cuda") < 0.3] = -math.inf
        x[torch.rand(T, generator=g, device="cuda") < 0.05] = -math.inf
    return x


def _selected(x, k):
    """k experts of each row by logit, -1 where fewer are left (made input, not measured)."""
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] > -math.inf, i[:, :k], -1).to(torch.int32).contiguous()


def _offsets(case, g):
    """Offsets of ragged sequences that fill the batch, on the device."""
    S, T = case["seqs"], case["T"]
    w = torch.rand(S, generator=g, device="cuda", dtype=torch.float64) + 0.05
    cut = (torch.cumsum(w, 0) / w.sum() * T).round().to(torch.int32)
    cut[-1] = T
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cut]).contiguous()


def _matrices(case, g):
    """Gradients as a layer's backward makes them: sums of outer products over a group's rows,
    with rows and columns of different size."""
    G, M, N, r = case["G"], case["M"], case["N"], case["rank"]
    a = torch.randn(G, M, r, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(G, r, N, generator=g, device="cuda").to(torch.bfloat16)
    a *= torch.exp(0.5 * torch.randn(G, M, 1, generator=g, device="cuda")).to(torch.bfloat16)
    x = torch.matmul(a, b).float() * (1e-3 / math.sqrt(r))
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    op = case["op"]
    if op in ("ortho", "muon"):
        G, M, N = case["G"], case["M"], case["N"]
        dt = getattr(torch, case["grad"])
        st["grad"] = _matrices(case, g).to(dt)
        st["out"] = torch.empty(G, M, N, dtype=torch.bfloat16, device="cuda")
        if op == "muon":
            # a momentum of many steps: full rank, with rows of different size
            m = torch.randn(G, M, N, generator=g, device="cuda")
            m *= 5e-3 * torch.exp(0.5 * torch.randn(G, M, 1, generator=g, device="cuda"))
            st["momentum"], st["momentum_out"] = m, torch.empty(G, M, N, **f32)
            st["w"] = (torch.randn(G, M, N, generator=g, device="cuda") / math.sqrt(N)).to(
                torch.bfloat16)
        if own:
            import mixture_experts_layer_grouped_b200 as moe
            st["cfg"] = moe.MoEMuonConfig(groups=G, rows=M, cols=N, steps=5, a=NS[0], b=NS[1],
                                          c=NS[2], eps=EPS)
            st["ws"] = moe.binding.new_workspace(moe.moe_muon_workspace_size(st["cfg"]))
        return st
    T, E, k = case["T"], case["E"], case["k"]
    st["logits"] = _logits(case, g)
    if op == "route":
        st["bias"] = (torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1
                      if case["bias"] else None)
        st["idx"], st["w"] = torch.empty(T, k, **i32), torch.empty(T, k, **f32)
    else:
        st["idx"] = _selected(st["logits"], k)
        st["offsets"] = _offsets(case, g) if case["seqs"] else None
    if op == "back":
        st["dgate"] = torch.randn(T, k, generator=g, device="cuda")
        st["dlogits"] = torch.empty(T, E, **f32)
        st["dscore"] = (torch.rand(case["seqs"], E, generator=g, device="cuda") * 1e-2
                        if case["seqs"] else None)
    if op == "balance":
        S = case["seqs"]
        st["loss"] = torch.empty(1, **f32)
        st["load"], st["dscore"] = torch.empty(S, E, **i32), torch.empty(S, E, **f32)
    if own:
        import mixture_experts_layer_grouped_b200 as moe
        st["cfg"] = moe.MoEConfig(T=T, H=128, I=128, E=E, n_group=case.get("groups", 1),
                                  topk_group=case.get("kept", 1), top_k=k, I_shared=0,
                                  routed_scaling_factor=RSF, dtype=0, pad_multiple=8)
        st["router"] = moe.MoERouter(score=case["score"], renormalize=int(case["renorm"])
                                     if "renorm" in case else 1, group_top=case.get("top", 1))
        if op == "balance":
            st["ws"] = moe.binding.new_workspace(
                moe.moe_balance_workspace_size(st["cfg"], case["seqs"]))
    return st


# -------------------------------------------------------------------------------- plain forms
def _scores(x, score):
    """Scores in 64 bits: a place at -inf has none."""
    x = x.double()
    if score == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(dim=1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - torch.where(m > -math.inf, m, 0.0)), 0.0)
    z = e.sum(dim=1, keepdim=True)
    return e / torch.where(z > 0, z, 1.0)


def _gates(s, idx, renorm):
    """Gates of the selected places in 64 bits, 0 where there is none."""
    v = torch.where(idx >= 0, torch.gather(s, 1, idx.clamp(min=0).long()), 0.0)
    if renorm:
        z = v.sum(dim=1, keepdim=True)
        v = v / torch.where(z > 0, z, 1.0)
    return v * RSF


def _plain_route(st):
    c, x, bias = st["case"], st["logits"], st["bias"]
    T, E, G = c["T"], c["E"], c["groups"]
    s = _scores(x, c["score"])  # in 64 bits: near a border 32 would choose another expert
    key = x.double()
    if bias is not None:
        key = torch.where(x > -math.inf, s + bias.double(), -math.inf)
    if G > 1:
        size = E // G
        by = key if bias is not None or c["top"] == 1 else torch.where(x > -math.inf, s, -math.inf)
        best = torch.sort(by.view(T, G, size), dim=2, descending=True)[0][:, :, : c["top"]]
        some = best[:, :, 0] > -math.inf
        score = torch.where(best > -math.inf, best, 0.0).sum(dim=2)
        score = torch.where(some, score, -math.inf)
        keep = torch.sort(score, dim=1, descending=True, stable=True)[1][:, : c["kept"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        key = torch.where(kept.repeat_interleave(size, dim=1), key, -math.inf)
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    idx = torch.where(v[:, : c["k"]] > -math.inf, i[:, : c["k"]], -1)
    return {"idx": idx.to(torch.int32), "gate": _gates(s, idx, c["renorm"]).float()}


def _sequence_of(offsets, T):
    return torch.searchsorted(offsets[1:].contiguous(),
                              torch.arange(T, device=offsets.device, dtype=torch.int32), right=True)


def _plain_back(st):
    c, x, idx = st["case"], st["logits"], st["idx"]
    s = _scores(x, c["score"]).float()
    off = 1.0 / (1.0 + torch.exp(x))  # 1 - sigmoid
    have = idx >= 0
    at = idx.clamp(min=0).long()
    g = torch.where(have, st["dgate"], 0.0) * RSF
    v = torch.where(have, torch.gather(s, 1, at), 0.0)
    if c["renorm"]:
        z = v.sum(dim=1, keepdim=True)
        z = torch.where(z > 0, z, 1.0)
        g = torch.where(have, (g - (g * v / z).sum(dim=1, keepdim=True)) / z, 0.0)
    ds = torch.zeros_like(s).scatter_add_(1, at, g)
    if c["score"] == SIGMOID:
        d = ds * s * off
    else:
        d = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    if c["seqs"]:
        e = st["dscore"][_sequence_of(st["offsets"], c["T"])]
        z = s.sum(dim=1, keepdim=True)
        z = torch.where(z > 0, z, 1.0)
        h = e - (e * s).sum(dim=1, keepdim=True) / z
        d = d + (h * s * off / z if c["score"] == SIGMOID else h * s)
    return {"dlogits": d}


def _plain_balance(st):
    c, idx = st["case"], st["idx"]
    T, E, S = c["T"], c["E"], c["seqs"]
    s = _scores(st["logits"], c["score"])
    z = s.sum(dim=1, keepdim=True)
    seq = _sequence_of(st["offsets"], T)
    f64 = dict(dtype=torch.float64, device=s.device)
    share = torch.zeros(S, E, **f64).index_add_(0, seq, s / torch.where(z > 0, z, 1.0))
    rows = torch.zeros(S, **f64).index_add_(0, seq, (z[:, 0] > 0).double())
    place = (seq[:, None] * E + idx.clamp(min=0))[idx >= 0]
    load = torch.zeros(S * E, **f64).index_add_(0, place, torch.ones(len(place), **f64)).view(S, E)
    n = torch.where(rows > 0, rows, 1.0)[:, None]
    d = COEF / S * E / c["k"] * load / n / n
    return {"loss": (d * share).sum().float().view(1), "load": load.to(torch.int32),
            "dscore": d.float()}


def _newton_schulz(u):
    """In 32 bits, on the side with fewer rows."""
    tall = u.shape[1] > u.shape[2]
    x = u.mT if tall else u
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(5):
        a = torch.matmul(x, x.mT)
        x = NS[0] * x + torch.matmul(NS[1] * a + NS[2] * torch.matmul(a, a), x)
    return x.mT if tall else x


def _plain_ortho(st):
    return {"update": _newton_schulz(st["grad"].float()).to(torch.bfloat16).contiguous()}


def _plain_muon(st):
    g = st["grad"].float()
    m = BETA * st["momentum"] + g
    x = _newton_schulz(g + BETA * m)
    return {"momentum": m, "w": ((1 - DECAY) * st["w"].float() - STEP * x).to(torch.bfloat16)}


# ------------------------------------------------------------------------------------- passes
def _own(st):
    import mixture_experts_layer_grouped_b200 as moe
    op = st["case"]["op"]
    if op == "route":
        moe.moe_route_scored(st["cfg"], st["router"], st["idx"], st["w"], bias=st["bias"],
                             logits_in=st["logits"])
        return {"idx": st["idx"], "gate": st["w"]}
    if op == "back":
        moe.moe_route_backward(st["cfg"], st["router"], st["logits"], st["idx"], st["dgate"],
                               st["dlogits"], dscore=st["dscore"], seq_offsets=st["offsets"])
        return {"dlogits": st["dlogits"]}
    if op == "balance":
        moe.moe_balance_loss(st["cfg"], st["router"], st["logits"], st["idx"], COEF, st["loss"],
                             st["load"], st["dscore"], st["ws"], seq_offsets=st["offsets"])
        return {"loss": st["loss"], "load": st["load"], "dscore": st["dscore"]}
    if op == "ortho":
        moe.moe_orthogonalize(st["cfg"], st["grad"], st["out"], st["ws"])
        return {"update": st["out"]}
    moe.moe_muon_step(st["cfg"], st["grad"], st["momentum"], st["momentum_out"], st["w"],
                      st["out"], st["ws"], beta=BETA, nesterov=True, step=STEP, decay=DECAY)
    return {"momentum": st["momentum_out"], "w": st["out"]}


_PLAIN = {"route": _plain_route, "back": _plain_back, "balance": _plain_balance,
          "ortho": _plain_ortho, "muon": _plain_muon}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    if case["op"] in ("ortho", "muon"):
        G, r, n = case["G"], min(case["M"], case["N"]), max(case["M"], case["N"])
        each = (2 if case["grad"] == "bfloat16" else 4) + (12 if case["op"] == "muon" else 2)
        # the two symmetric products need half of their entries
        flops = 5.0 * G * (float(r) * r * n + float(r) ** 3 + 2.0 * r * r * n)
        return {"bytes": float(G) * r * n * each, "flops": flops}
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        return {"bytes": 4.0 * T * E + 4.0 * E * case["bias"] + 8.0 * T * k, "flops": 8.0 * T * E}
    S = case["seqs"]
    if case["op"] == "back":
        return {"bytes": 8.0 * T * E + 8.0 * T * k + 4.0 * S * E, "flops": 12.0 * T * E}
    return {"bytes": 4.0 * T * E + 4.0 * T * k + 8.0 * S * E, "flops": 8.0 * T * E}


# ------------------------------------------------------------------- 64 bits, from definitions
def _exact_scores(x, score):
    if score == SIGMOID:
        return torch.sigmoid(x)
    p = torch.softmax(torch.where(torch.isneginf(x).all(dim=1, keepdim=True), 0.0, x), dim=1)
    return torch.where(torch.isneginf(x), 0.0, p)


def _exact_gates(s, idx, renorm):
    one = torch.nn.functional.one_hot((idx + 1).long(), s.shape[1] + 1)[:, :, 1:].to(s.dtype)
    v = torch.einsum("tke,te->tk", one, s)
    if renorm:
        z = v.sum(dim=1)
        v = torch.where((z > 0)[:, None], v / torch.where(z > 0, z, 1.0)[:, None], 0.0)
    return RSF * v


def _exact_select(x, s, bias, c):
    """One expert after another: the largest key left, the first of equal ones."""
    T, E, G = c["T"], c["E"], c["groups"]
    dead = torch.isneginf(x)
    key = x.clone() if bias is None else torch.where(dead, -math.inf, s + bias.double())
    if G > 1:
        by = key if bias is not None or c["top"] == 1 else torch.where(dead, -math.inf, s)
        left, score = by.reshape(T, G, -1).clone(), torch.zeros(T, G, dtype=x.dtype, device=x.device)
        for j in range(c["top"]):
            m = left.amax(dim=2)
            score += torch.where(torch.isneginf(m), 0.0 if j else -math.inf, m)
            first = (left == m[:, :, None]).int().cumsum(dim=2) == 1
            left[first & (left == m[:, :, None])] = -math.inf
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        for _ in range(c["kept"]):
            open_ = torch.where(keep, -math.inf, score)
            hit = (open_ == open_.amax(dim=1, keepdim=True)) & ~keep
            keep |= hit & (hit.int().cumsum(dim=1) == 1)
        key = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    idx = []
    for _ in range(c["k"]):
        m = key.amax(dim=1, keepdim=True)
        hit = (key == m) & (m > -math.inf)
        hit &= hit.int().cumsum(dim=1) == 1
        idx.append(torch.where(hit.any(dim=1), hit.int().argmax(dim=1), -1))
        key = torch.where(hit, -math.inf, key)
    return torch.stack(idx, dim=1)


def _exact_share(s):
    z = s.sum(dim=1, keepdim=True)
    return torch.where(z > 0, s / torch.where(z > 0, z, 1.0), 0.0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("ortho", "muon"):
        u = st["grad"].double()
        if case["op"] == "muon":
            m = BETA * st["momentum"].double() + u
            u = u + BETA * m
        u /= torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + EPS
        # X5 = Q X0 with Q a polynomial of S = X0 X0^T (of X0^T X0 from the other side)
        tall = case["M"] > case["N"]
        p = u.mT @ u if tall else u @ u.mT
        one = torch.eye(p.shape[1], dtype=p.dtype, device=p.device)
        q = None
        for _ in range(5):
            f = NS[0] * one + NS[1] * p + NS[2] * (p @ p)
            q = f if q is None else f @ q
            p = f @ p @ f
        x = u @ q if tall else q @ u
        if case["op"] == "ortho":
            return {"update": x}
        return {"momentum": m, "w": (1 - DECAY) * st["w"].double() - STEP * x}
    x = st["logits"].double()
    c, E, k = case, case["E"], case["k"]
    if case["op"] == "route":
        s = _exact_scores(x, c["score"])
        idx = _exact_select(x, s, st["bias"], c)
        return {"idx": None, "gate": _exact_gates(s, idx, c["renorm"])}
    seq = None
    if c["seqs"]:
        at = torch.arange(c["T"], device=x.device)
        seq = (at[:, None] >= st["offsets"][None, 1:-1]).sum(dim=1)
    if case["op"] == "back":
        dead = torch.isneginf(x)
        x = torch.where(dead, -1e4, x).requires_grad_()
        s = torch.where(dead, 0.0, _exact_scores(x, c["score"]))
        total = (_exact_gates(s, st["idx"], c["renorm"]) * st["dgate"].double()).sum()
        if seq is not None:
            total = total + (_exact_share(s) * st["dscore"].double()[seq]).sum()
        total.backward()
        return {"dlogits": torch.where(dead, 0.0, x.grad)}
    s = _exact_scores(x, c["score"])
    S = c["seqs"]
    loss, d = 0.0, []
    for q in range(S):
        mine = s[seq == q]
        n = max(1, int((mine.sum(dim=1) > 0).sum()))
        chosen = st["idx"][seq == q].flatten()
        f = torch.bincount(chosen[chosen >= 0].long(), minlength=E).double() * E / (k * n)
        d.append(COEF / S * f / n)
        loss += float((d[-1] * _exact_share(mine).sum(dim=0)).sum())
    return {"loss": torch.tensor([loss], dtype=torch.float64), "load": None,
            "dscore": torch.stack(d)}
