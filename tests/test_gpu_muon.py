"""The orthogonalised update on the GPU against the fp64 oracle.

Tolerance of X, relative in the Frobenius norm.  The products see X, A and B = b A + c A^2
rounded to fp16: at most 2^-11 relative a value, 2^-11 / sqrt(3) = 2.8e-4 rms over evenly
spread remainders of the worst binade, 2e-4 over a binade.  One step's error in B X, with
|B| <= 2.81 and |X| <= 1.21: the rounding of X reaches it through b A X and c A^2 X three and
five times (factors 3 |b| and 5 |c| on a value of A near 1, partly cancelling: b + c A is
negative over the whole range), of A through b and 2 c A, of B once: about
2e-4 * sqrt((3 * 4.8 - 5 * 2.0)^2 + (4.8 - 2 * 2.0)^2 + 2.8^2) = 1.1e-3 on the directions whose
singular values are near 1, and less on the others; a step passes an earlier error on by
p'(sigma) <= 1 there, so five steps give at most 1.1e-3 sqrt(5) = 2.5e-3.  The bf16 result
adds 2^-8 / sqrt(3) = 2.3e-3 rms at most: 3.4e-3 in all, checked as 4e-3.  Weights and
momentum: bf16's half step 2^-8 of the value and 4e-3 of step |X|; one fused fp32 rounding."""

import numpy as np
import pytest
import torch

from oracle import train_oracle as TO

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
TOL = 4e-3


@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_grouped_b200 as M
    M.lib()
    return M


def config(M, G, R, C, steps=5):
    return M.MoEMuonConfig(groups=G, rows=R, cols=C, steps=steps, a=NS[0], b=NS[1], c=NS[2],
                           eps=1e-7)


def grads(G, R, C, seed, rank=None, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    if rank is None:
        return torch.randn(G, R, C, generator=g) * scale
    return torch.randn(G, R, rank, generator=g) @ torch.randn(G, rank, C, generator=g) * scale


def ortho(M, c, g, out=None, ws=None):
    out = torch.empty(c.groups, c.rows, c.cols, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = M.binding.new_workspace(M.moe_muon_workspace_size(c)) if ws is None else ws
    M.moe_orthogonalize(c, g.cuda(), out, ws)
    torch.cuda.synchronize()
    assert M.moe_get_device_status(ws) == 0
    return out


def check(got, g, steps=5):
    for x, u in zip(got.double().cpu().numpy(), g.double().numpy()):
        ref = TO.orthogonalize(u, steps, *NS, 1e-7)
        assert np.linalg.norm(x - ref) <= TOL * np.linalg.norm(ref) + 1e-30


SHAPES = [  # groups, rows, cols
    (1, 1, 1), (3, 1, 7), (2, 5, 1), (2, 8, 8), (3, 17, 130), (2, 130, 17), (2, 128, 256),
    (2, 256, 128), (1, 129, 64), (2, 64, 129), (1, 200, 333), (2, 300, 130), (3, 256, 512),
    (1, 512, 257), (1, 130, 1100), (1, 1100, 131), (40, 136, 136), (1, 384, 2056), (2, 515, 515),
    # tiles of CTA pairs: one a matrix, several with a mirrored one, split along the contraction
    (80, 136, 136), (80, 150, 132), (20, 500, 512), (20, 512, 505), (10, 505, 1100), (10, 1100, 505),
]


@pytest.mark.parametrize("G,R,C", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_matches_oracle(M, G, R, C, dtype):
    g = grads(G, R, C, R + C).to(dtype)
    check(ortho(M, config(M, G, R, C), g), g)


@pytest.mark.parametrize("R,C,rank", [(256, 512, 1), (256, 512, 40), (300, 200, 7), (128, 128, 3)])
def test_rank_deficient_gradients(M, R, C, rank):
    """Few rows behind a gradient: the directions it does not have must stay empty."""
    g = grads(2, R, C, rank, rank=rank)
    check(ortho(M, config(M, 2, R, C), g), g)


def test_wide_spectra_and_magnitudes(M):
    """Singular values over six decades; rows and columns of very different size; gradients
    far below and above 1."""
    g = torch.Generator().manual_seed(0)
    q = torch.linalg.qr(torch.randn(200, 200, generator=g))[0]
    p = torch.linalg.qr(torch.randn(320, 200, generator=g))[0]
    s = 10.0 ** -torch.linspace(0, 6, 200)
    x = torch.stack([(q * s) @ p.T, torch.randn(200, 320, generator=g) *
                     torch.exp(2 * torch.randn(200, 1, generator=g)) *
                     torch.exp(2 * torch.randn(1, 320, generator=g)),
                     torch.randn(200, 320, generator=g) * 1e30,
                     torch.randn(200, 320, generator=g) * 1e-4])
    check(ortho(M, config(M, 4, 200, 320), x), x)


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_other_step_counts(M, steps):
    g = grads(2, 140, 260, steps)
    check(ortho(M, config(M, 2, 140, 260, steps), g), g, steps)


def test_zero_and_bad_matrices_stay_by_themselves(M):
    """A zero matrix (an expert no token picked) stays zero, a NaN and an infinity stay in
    their own matrices."""
    for R, C in ((140, 200), (64, 100)):
        g = grads(5, R, C, 1)
        g[1] = 0
        g[2, 3, 4] = float("nan")
        g[3, 5, 6] = float("inf")
        x = ortho(M, config(M, 5, R, C), g)
        assert not x[1].any()
        assert torch.isnan(x[2]).any() and torch.isnan(x[3]).any()
        check(x[[0, 4]], g[[0, 4]])


@pytest.mark.parametrize("G,R,C", [(2, 128, 256), (3, 33, 65), (2, 300, 144), (1, 1, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nesterov", [False, True])
def test_step_matches_oracle(M, G, R, C, dtype, nesterov):
    c = config(M, G, R, C)
    g = grads(G, R, C, 1, scale=1e-3).to(dtype)
    m = grads(G, R, C, 2, scale=1e-2)
    w = (grads(G, R, C, 3) * 0.05).bfloat16()
    mo = torch.empty(G, R, C, device="cuda")
    wo = torch.empty(G, R, C, dtype=torch.bfloat16, device="cuda")
    ws = M.binding.new_workspace(M.moe_muon_workspace_size(c))
    args = dict(beta=0.9, nesterov=nesterov, step=0.02, decay=0.01)
    M.moe_muon_step(c, g.cuda(), m.cuda(), mo, w.cuda(), wo, ws, **args)
    torch.cuda.synchronize()
    rm, rw = TO.muon_step(g.double().numpy(), m.double().numpy(), w.double().numpy(), 0.9,
                          nesterov, 0.02, 0.01, 5, *NS, 1e-7)
    # beta and 1 - decay are fp32 numbers: 2^-24 relative each beside the roundings
    assert np.all(np.abs(mo.cpu().numpy() - rm) <= 2.0 ** -22 * (0.9 * np.abs(m.numpy()) + np.abs(g.float().numpy())))
    off = np.abs(wo.double().cpu().numpy() - rw)
    x = np.linalg.norm((rw - 0.99 * w.double().numpy()).reshape(G, -1), axis=1)
    rest = np.linalg.norm(np.maximum(off - 2.0 ** -8 * np.abs(rw), 0).reshape(G, -1), axis=1)
    assert np.all(rest <= TOL * x + 1e-30)
    # in place, the same bits
    m2, w2 = m.cuda(), w.cuda()
    M.moe_muon_step(c, g.cuda(), m2, m2, w2, w2, ws, **args)
    assert torch.equal(m2, mo) and torch.equal(w2, wo)
    assert M.moe_get_device_status(ws) == 0


def test_rows_behind_the_matrices_are_untouched(M):
    for R, C in ((130, 70), (70, 133), (300, 257)):
        c = config(M, 1, R, C)
        buf = torch.full((2, R, C), 7.0, dtype=torch.bfloat16, device="cuda")
        ortho(M, c, grads(1, R, C, 0), out=buf[0])
        assert (buf[1] == 7.0).all()


def test_unaligned_pointers(M):
    """Tensors that start two or four bytes off a 16-byte boundary."""
    G, R, C = 1, 64, 96
    c = config(M, G, R, C)
    g = grads(G, R, C, 4)
    m, w = grads(G, R, C, 5), grads(G, R, C, 6).bfloat16()
    n = R * C

    def off(t):
        b = torch.empty(n + 1, dtype=t.dtype, device="cuda")[1:].view(G, R, C)
        return b.copy_(t)

    ws = M.binding.new_workspace(M.moe_muon_workspace_size(c))
    res = []
    for f in (lambda t: t.cuda(), off):
        mo, wo = f(torch.zeros_like(m)), f(torch.zeros_like(w))
        M.moe_muon_step(c, f(g), f(m), mo, f(w), wo, ws)
        res.append((mo.cpu(), wo.cpu()))
    assert torch.equal(res[0][0], res[1][0])
    # the norm's partial sums may have another order there: at most one bf16 step apart
    assert (res[0][1].float() - res[1][1].float()).abs().max() <= 2.0 ** -7 * w.float().abs().max()


def test_capture_replay_and_second_stream(M):
    c = config(M, 2, 140, 300)
    ws, ws2 = (M.binding.new_workspace(M.moe_muon_workspace_size(c)) for _ in range(2))
    g = torch.empty(2, 140, 300, device="cuda")
    out, out2 = (torch.empty(2, 140, 300, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.copy_(grads(2, 140, 300, 0))
    M.moe_orthogonalize(c, g, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_orthogonalize(c, g, out, ws)
    side = torch.cuda.Stream()
    for seed in (1, 2):
        g.copy_(grads(2, 140, 300, seed))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):  # at the same time, with a workspace of its own
            M.moe_orthogonalize(c, g, out2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
        check(out, g.cpu())


def test_layer_gradients_are_orthogonalised(M):
    """A larger stack in the layer's own shapes: up and down projections of its experts."""
    for R, C in ((1024, 2048), (2048, 1024)):
        g = grads(4, R, C, R, rank=192, scale=1e-3)
        check(ortho(M, config(M, 4, R, C), g), g)
