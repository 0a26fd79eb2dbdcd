"""The scored router, its gradient and the balance loss on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, the largest relative rounding of fp32):
* gates: exponential 2u, sum of E <= 1024 scores by 32 + 5 additions 37u, division, product
  and the last rounding 4u; renormalised the selected ones' sum 5u more: under 64u relative;
* dlogits: a product of scores (64u each, two of them) and of differences of sums of at most
  32 + 5 terms bounded by rsf max|dgate| (and by max|c| for the balance part): under 256u of
  that bound;
* loss and dscore: rows' shares 64u, fp32 sums of at most 16 rows a warp and 8 warps 24u, the
  rest in 64 bits: under 96u relative; dscore is computed in 64 bits: u."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import train_oracle as TO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RSF = 2.5


@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_grouped_b200 as M
    M.lib()
    return M


def config(M, T, E, k, G=1, g=1, rsf=RSF):
    return M.MoEConfig(T=T, H=128, I=128, E=E, n_group=G, topk_group=g, top_k=k, I_shared=0,
                       routed_scaling_factor=rsf, dtype=0, pad_multiple=8)


def logits_of(T, E, seed, mask=0.0, empty=0.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * scale
    x[torch.rand(T, E, generator=g) < mask] = -float("inf")
    x[torch.rand(T, generator=g) < empty] = -float("inf")
    return x


def route(M, c, r, x, bias=None, stream=None):
    x = x.cuda()
    idx = torch.full((c.T, c.top_k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((c.T, c.top_k), float("nan"), device="cuda")
    M.moe_route_scored(c, r, idx, w, logits_in=x, bias=None if bias is None else bias.cuda(),
                       stream=stream)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_route(M, T, E, k, G, g, score, renorm, top, bias, x, rsf=RSF):
    c = config(M, T, E, k, G, g, rsf)
    idx, w = route(M, c, M.MoERouter(score, renorm, top), x, bias)
    ref_i, ref_w = TO.route(x.numpy(), None if bias is None else bias.numpy(), G, g, k, score,
                            renorm, top, rsf)
    assert np.array_equal(idx, ref_i)
    assert np.all(np.abs(w - ref_w) <= 64 * U * np.abs(ref_w) + 1e-37)


SHAPES = [  # T, E, k, G, g
    (1, 2, 1, 1, 1), (1, 256, 8, 1, 1), (3, 17, 5, 1, 1), (37, 16, 4, 4, 2), (65, 60, 6, 3, 2),
    (50, 64, 6, 8, 4), (33, 100, 32, 1, 1), (40, 256, 8, 8, 4), (21, 384, 6, 8, 4),
    (9, 390, 12, 5, 5), (5, 1024, 32, 32, 16), (7, 96, 3, 32, 2), (11, 33, 33 - 1, 1, 1),
]


@pytest.mark.parametrize("T,E,k,G,g", SHAPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_route_matches_oracle(M, T, E, k, G, g, score, biased):
    gen = torch.Generator().manual_seed(E + k)
    bias = torch.rand(E, generator=gen) * 0.2 - 0.1 if biased else None
    for n, (renorm, top) in enumerate([(0, 1), (1, 2), (1, 1), (0, 2)]):
        check_route(M, T, E, k, G, g, score, renorm, top, bias, logits_of(T, E, 10 * E + n))
        check_route(M, T, E, k, G, g, score, renorm, top, bias,
                    logits_of(T, E, 7 * E + n, mask=0.4, empty=0.2))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route_edges(M, score, renorm):
    """Rows with nothing left, the type's lowest value, infinities, NaN, ties, far logits."""
    inf, low = float("inf"), torch.finfo(torch.float32).min
    E = 8
    x = torch.tensor([
        [-inf] * E, [float("nan")] * E, [low] * E, [0.0] * E, [low] * 7 + [1.0],
        [inf, 1, inf, 0, -inf, float("nan"), 2, 3], [-200.0] * 4 + [-210.0] * 4,
        [300.0, 200, 100, 0, -100, -200, -300, -400], [-0.0, 0.0, -0.0, 0.0, 1, 1, -inf, 1],
        [-95.0, -96, -97, -98, -99, -100, -101, -102]])
    check_route(M, len(x), E, 3, 1, 1, score, renorm, 1, None, x)
    check_route(M, len(x), E, 3, 4, 2, score, renorm, 1, None, x)
    bias = torch.zeros(E)
    check_route(M, len(x), E, 3, 1, 1, score, renorm, 1, bias, x)
    bias = torch.tensor([0, -inf, float("nan"), 0.5, inf, 0, -1e30, -100])
    check_route(M, len(x), E, 4, 1, 1, score, renorm, 1, bias, x)
    check_route(M, len(x), E, 4, 2, 1, score, renorm, 2, bias, x)


def check_selection(M, T, E, k, G, g, score, top, bias, x):
    """The selection is the one of the keys' 64-bit values, where these differ by more than 64
    bits hold of them: a score there has the roundings of E additions, one division and two
    exponentials, (E + 8) 2^-53 of itself, which a key or a group's sum of two at most doubles.
    (32-bit keys would be off by 2^-24 of the scores, 2^29 / (2 E + 16) times as much.)"""
    idx, _ = route(M, config(M, T, E, k, G, g), M.MoERouter(score, 1, top), x, bias)
    for t in range(T):
        s = TO.scores(x[t].numpy(), score)
        d = 4 * (E + 8) * 2.0 ** -53 * s.max()
        key = s + (0.0 if bias is None else bias.numpy().astype(np.float64))
        total = np.array([sum(sorted(v)[::-1][:top]) for v in key.reshape(G, -1)])
        border = np.sort(total)[::-1][g - 1]
        mine = idx[t]
        assert len(set(mine)) == k and mine.min() >= 0
        assert np.all(np.diff(key[mine]) <= d)
        assert np.all(total[mine // (E // G)] >= border - d)
        sure = [e for e in range(E) if total[e // (E // G)] > border + d and e not in mine]
        assert all(key[e] <= key[mine[-1]] + d for e in sure)


@pytest.mark.parametrize("score", [0, 1])
def test_route_near_ties_are_decided_in_64_bits(M, score):
    """Keys one part in 1e9 apart, which 32-bit scores cannot tell apart: two experts whose
    biases make up for their scores up to a few roundings of the bias."""
    gen = torch.Generator().manual_seed(5)
    T, E = 200, 32
    x = torch.randn(T, E, generator=gen)
    x[:, 1:] = x[:, :1] + torch.arange(1, E) * 2.0 ** -20
    bias = torch.zeros(E)
    for t in range(4):
        s = np.stack([TO.scores(r, score) for r in x.numpy()])
        bias = torch.from_numpy((s[t].max() - s[t]).astype(np.float32))
        check_selection(M, T, E, 8, 1, 1, score, 1, bias, x)
        check_selection(M, T, E, 8, 8, 3, score, 2, bias, x)


@pytest.mark.parametrize("E,G,g", [(48, 1, 1), (64, 8, 4), (256, 8, 3), (384, 8, 4), (512, 16, 8)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_many_near_ties(M, E, G, g, score):
    """The same with several experts a lane, and with more than 32 keys within the error of
    the last one selected."""
    T = 40
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(E))
    x[:, 1:] = x[:, :1] + torch.arange(1, E) * 2.0 ** -20
    far = torch.arange(E) % 7 != 0  # the others stay near each other
    s = np.stack([TO.scores(r, score) for r in x.numpy()])
    bias = torch.from_numpy((s[3].max() - s[3]).astype(np.float32))
    for top in (1, 2):
        check_selection(M, T, E, 8, G, g, score, top, bias, x)
        check_selection(M, T, E, 8, G, g, score, top, bias - 0.01 * far, x)


@pytest.mark.parametrize("E,G,g", [(32, 8, 4), (256, 8, 4), (384, 8, 4), (60, 6, 3)])
def test_route_groups_with_near_sums(M, E, G, g):
    """No bias and groups by two scores: sigmoid(d) + sigmoid(-d) = 1 for every d, so groups
    whose best logits are d and a hair more than -d differ by that hair alone."""
    T, size = 64, E // G
    gen = torch.Generator().manual_seed(E)
    x = torch.full((T, G, size), -8.0) - torch.rand(T, G, size, generator=gen)
    d = (torch.rand(T, G, generator=gen) * 64).round() / 64
    hair = torch.randint(0, 64, (T, G), generator=gen) * 2.0 ** -24
    x[:, :, 1] = d
    x[:, :, size - 1] = -d + hair * (d > 0.3)
    check_selection(M, T, E, 4, G, g, 0, 2, None, x.reshape(T, E).contiguous())


@pytest.mark.parametrize("score", [0, 1])
def test_gradient_where_one_share_is_nearly_all(M, score):
    """Renormalised: a single place's gate is a constant, its gradient zero; of two places far
    apart both gradients keep their relative precision (w1 w2 (g1 - g2): two shares of 64u,
    a difference and products of a few u, under 256u)."""
    T, E = 6, 48
    x = logits_of(T, E, 3)
    r = M.MoERouter(score, 1, 1)
    out = torch.full((T, E), float("nan"), device="cuda")
    M.moe_route_backward(config(M, T, E, 1), r, x.cuda(), x.argmax(1, keepdim=True).int().cuda(),
                         torch.randn(T, 1).cuda(), out)
    assert torch.count_nonzero(out) == 0
    x[:, 7], x[:, 11] = 3.0, -torch.arange(T) * 3.0
    idx = np.tile([7, 11], (T, 1))
    dgate = torch.tensor([[1.0, -0.5]] * T)
    M.moe_route_backward(config(M, T, E, 2), r, x.cuda(), torch.from_numpy(idx).int().cuda(),
                         dgate.cuda(), out)
    ref = TO.route_backward(x.numpy(), idx, dgate.numpy(), score, 1, RSF)
    got = out.cpu().numpy()
    assert np.all(np.abs(got - ref)[:, [7, 11]] <= 256 * U * np.abs(ref)[:, [7, 11]])
    assert np.count_nonzero(got) == 2 * T


@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (5, 16, 4), (33, 60, 6), (40, 384, 8),
                                   (3, 1024, 32), (19, 257, 12)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("seqs", [0, 1, 3])
def test_gradient_matches_oracle(M, T, E, k, score, renorm, seqs):
    c, r = config(M, T, E, k), M.MoERouter(score, renorm, 1)
    x = logits_of(T, E, T + E, mask=0.2, empty=0.1)
    idx, _ = TO.route(x.numpy(), None, 1, 1, k, score, renorm, 1, RSF)
    gen = torch.Generator().manual_seed(1)
    dgate = torch.randn(T, k, generator=gen)
    off = {0: None, 1: None, 3: [0, T // 3, T // 3, T - T // 4]}[seqs]
    dscore = torch.rand(seqs, E, generator=gen) if seqs else None
    dloss = torch.tensor([1.5]) if seqs == 3 else None
    out = torch.full((T, E), float("nan"), device="cuda")
    cu = lambda t: None if t is None else t.cuda()
    M.moe_route_backward(c, r, x.cuda(), torch.from_numpy(idx).int().cuda(), dgate.cuda(), out,
                         dscore=cu(dscore), dloss=cu(dloss),
                         seq_offsets=None if off is None else torch.tensor(off).int().cuda())
    torch.cuda.synchronize()
    ref = TO.route_backward(x.numpy(), idx, dgate.numpy(), score, renorm, RSF,
                            None if dscore is None else dscore.numpy(), off,
                            1.5 if dloss is not None else 1.0)
    bound = RSF * dgate.abs().max().item() + (1.5 if dscore is not None else 0.0)
    assert np.all(np.abs(out.cpu().numpy() - ref) <= 256 * U * bound)


def test_gradient_of_repeated_and_bad_places(M):
    """An expert named twice gets both places' gradient; places outside [0, E) and masked
    experts get none."""
    T, E, k = 4, 16, 4
    c = config(M, T, E, k)
    x = logits_of(T, E, 3)
    x[2, 5] = -float("inf")
    idx = np.array([[3, 3, 1, 0], [-1, 2, 16, -7], [5, 5, 4, 4], [9, 9, 9, 9]])
    dgate = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    for score in (0, 1):
        for renorm in (0, 1):
            out = torch.empty(T, E, device="cuda")
            M.moe_route_backward(c, M.MoERouter(score, renorm, 1), x.cuda(),
                                 torch.from_numpy(idx).int().cuda(), dgate.cuda(), out)
            ref = TO.route_backward(x.numpy(), idx, dgate.numpy(), score, renorm, RSF)
            assert np.all(np.abs(out.cpu().numpy() - ref) <=
                          256 * U * RSF * dgate.abs().max().item())


@pytest.mark.parametrize("T,E,k,off", [
    (1, 2, 1, None), (7, 16, 4, None), (300, 64, 6, None), (97, 60, 6, [0, 0, 5, 97]),
    (256, 384, 8, [3, 40, 41, 41, 200]), (64, 257, 3, list(range(65))), (9, 1024, 32, [0, 0, 0]),
    (2100, 33, 5, [0, 1000, 1001, 2100])])
@pytest.mark.parametrize("score", [0, 1])
def test_balance_matches_oracle(M, T, E, k, off, score):
    c, r = config(M, T, E, k), M.MoERouter(score, 1, 1)
    x = logits_of(T, E, E, mask=0.1, empty=0.1)
    idx, _ = TO.route(x.numpy(), None, 1, 1, k, score, 1, 1, RSF)
    S = 1 if off is None else len(off) - 1
    loss = torch.full((1,), float("nan"), device="cuda")
    load = torch.full((S, E), -5, dtype=torch.int32, device="cuda")
    dscore = torch.full((S, E), float("nan"), device="cuda")
    ws = torch.full((M.moe_balance_workspace_size(c, S),), 255, dtype=torch.uint8, device="cuda")
    args = (c, r, x.cuda(), torch.from_numpy(idx).int().cuda(), 0.01, loss, load, dscore, ws)
    o = None if off is None else torch.tensor(off).int().cuda()
    M.moe_balance_loss(*args, seq_offsets=o)
    ref = TO.balance(x.numpy(), idx, score, k, 0.01, off)
    assert np.array_equal(load.cpu().numpy(), ref[1])
    assert abs(loss.item() - ref[0]) <= 96 * U * ref[0]
    assert np.all(np.abs(dscore.cpu().numpy() - ref[2]) <= 2 * U * np.abs(ref[2]))
    first = loss.clone()
    M.moe_balance_loss(*args, seq_offsets=o)
    assert torch.equal(loss, first)  # the same bits every time


def test_balance_offsets_outside_the_batch_are_clamped(M):
    """Offsets past T or descending are the caller's mistake; nothing outside is touched."""
    T, E, k = 40, 16, 2
    c, r = config(M, T, E, k), M.MoERouter(1, 1, 1)
    x = logits_of(T, E, 1)
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    out = [torch.empty(1, device="cuda"), torch.empty(3, E, dtype=torch.int32, device="cuda"),
           torch.empty(3, E, device="cuda")]
    ws = M.binding.new_workspace(M.moe_balance_workspace_size(c, 3))
    for off in ([0, 30, 20, 4000], [-5, 10, 10, 40]):
        M.moe_balance_loss(c, r, x.cuda(), idx, 0.1, *out, ws,
                           seq_offsets=torch.tensor(off).int().cuda())
        torch.cuda.synchronize()


def test_capture_replay_and_streams(M):
    """Routing, balance loss and gradient captured once and replayed on new inputs; and on
    another stream than the current one."""
    T, E, k = 70, 64, 6
    c, r = config(M, T, E, k, 8, 4), M.MoERouter(1, 0, 1)
    x = torch.empty(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, dgate = torch.empty(T, k, device="cuda"), torch.randn(T, k, device="cuda")
    loss, load = torch.empty(1, device="cuda"), torch.empty(1, E, dtype=torch.int32, device="cuda")
    dscore, dl = torch.empty(1, E, device="cuda"), torch.empty(T, E, device="cuda")
    ws = M.binding.new_workspace(M.moe_balance_workspace_size(c, 1))

    def step():
        M.moe_route_scored(c, r, idx, w, logits_in=x)
        M.moe_balance_loss(c, r, x, idx, 0.01, loss, load, dscore, ws)
        M.moe_route_backward(c, r, x, idx, dgate, dl, dscore=dscore)

    x.copy_(logits_of(T, E, 0))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(logits_of(T, E, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, w, loss, load, dscore, dl)]
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        for a, b in zip(got, (idx, w, loss, load, dscore, dl)):
            assert torch.equal(a, b)
        ref_i, _ = TO.route(x.cpu().numpy(), None, 8, 4, k, 1, 0, 1, RSF)
        assert np.array_equal(idx.cpu().numpy(), ref_i)


def test_route_from_tokens_uses_the_router_gemm(M):
    """x and W_r given: the logits are moe_route's bit for bit, and the selection theirs."""
    import synth
    cfg = synth.get_config("mid_bf16_shared_T2048")
    c = M.config_from_shape(cfg)
    x = synth.gen_x(cfg, "cuda")
    w_r, bias = synth.gen_router(cfg, "cuda")
    nb, _ = M.moe_workspace_size(c)
    ws = M.binding.new_workspace(nb)
    T, E, k = cfg.T, cfg.E, cfg.top_k
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    l0, l1 = new(T, E), new(T, E)
    i0, i1 = new(T, k, dt=torch.int32), new(T, k, dt=torch.int32)
    w0, w1 = new(T, k), new(T, k)
    M.moe_route(c, x, w_r, bias, i0, w0, ws, logits_out=l0)
    M.moe_route_scored(c, M.MoERouter(0, 1, 2), i1, w1, x=x, w_router=w_r, bias=bias,
                       workspace=ws, logits_out=l1)
    torch.cuda.synchronize()
    assert M.moe_get_device_status(ws) == 0
    assert torch.equal(l0, l1)
    ref_i, ref_w = TO.route(l1.cpu().numpy(), bias.cpu().numpy(), cfg.n_group, cfg.topk_group, k,
                            0, True, 2, cfg.rsf)
    assert np.array_equal(i1.cpu().numpy(), ref_i)
    assert np.all(np.abs(w1.cpu().numpy() - ref_w) <= 64 * U * ref_w)
