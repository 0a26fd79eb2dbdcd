"""The training operators together, as a training step uses them: the scored router, the
balance loss, the layer's backward and the Muon update, on the layer's own classes.

Tolerance of the layer's results: relative Frobenius 1e-2, as for moe_backward; of the router's
fp32 gradients given the layer's own dgate: 256 roundings of 2^-24 of the largest term."""

import numpy as np
import pytest
import torch

import synth
from moe_testlib import f64, rel_frob, weights_dict
from oracle import moe_oracle as O
from oracle import train_oracle as TO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_grouped_b200 as M
    M.lib()
    return M


def shape(**kw):
    return synth.get_config("tiny_bf16_T64").scaled(pad_multiple=64, **kw)


def oracle_layer(cfg, h, idx, w):
    """y of the layer for given places and gates (rounding off), and each place's output."""
    T, H = h["x"].shape
    out = np.zeros((T, cfg.top_k, H))
    y = np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(idx[t]):
            if e >= 0:
                x = h["x"][t][None]
                out[t, j] = (O.swiglu(x @ h["w1"][e].T, x @ h["w3"][e].T) @ h["w2"][e].T)[0]
                y[t] += w[t, j] * out[t, j]
    if cfg.I_shared:
        y += O.swiglu(h["x"] @ h["ws1"].T, h["x"] @ h["ws3"].T) @ h["ws2"].T
    return y, out


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_forward_scored_matches_oracle(M, score, renorm, biased):
    cfg = shape(T=70, I_shared=128)
    d = synth.gen_all(cfg, "cuda")
    c, r = M.config_from_shape(cfg), M.MoERouter(score, renorm, 2)
    layer = M.MoELayer(c, weights_dict(d), d["w_router"], d["bias"] if biased else None, router=r)
    y = layer.forward(d["x"])
    host = layer.forward(d["x"].cpu().pin_memory())
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    assert torch.equal(y.cpu(), host)
    h = {k: f64(v) for k, v in d.items()}
    idx, w = TO.route(h["x"] @ h["w_router"].T, h["bias"] if biased else None, cfg.n_group,
                      cfg.topk_group, cfg.top_k, score, renorm, 2, cfg.rsf)
    assert rel_frob(f64(y), oracle_layer(cfg, h, idx, w)[0]) <= 1e-2


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("shared", [0, 128])
def test_train_layer_gradients(M, score, renorm, shared):
    """dgate, dlogits (gates and balance loss), dx and dW_r of the layer's two classes' calls."""
    cfg = shape(T=70, I_shared=shared)
    d = synth.gen_all(cfg, "cuda")
    c, r = M.config_from_shape(cfg), M.MoERouter(score, renorm, 1)
    coef, off = 0.5, torch.tensor([0, 30, 30, 66], dtype=torch.int32, device="cuda")
    layer = M.MoETrainLayer(c, weights_dict(d), d["w_router"], None, router=r, balance_coef=coef)
    layer.forward(d["x"], seq_offsets=off)
    dy = synth.gen_dy(cfg, "cuda")
    g = layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    h = {k: f64(v) for k, v in d.items()}
    logits = layer.saved["logits"].cpu().numpy()
    idx, w = TO.route(logits, None, cfg.n_group, cfg.topk_group, cfg.top_k, score, renorm, 1,
                      cfg.rsf)
    assert np.array_equal(layer.saved["topk_idx"].cpu().numpy(), idx)
    loss, load, dscore = TO.balance(logits, idx, score, cfg.top_k, coef, off.tolist())
    assert abs(layer.balance["loss"].item() - loss) <= 96 * U * loss
    assert np.array_equal(layer.balance["load"].cpu().numpy(), load)
    _, out = oracle_layer(cfg, h, idx, w)
    assert rel_frob(f64(g["dgate"]), np.einsum("th,tjh->tj", f64(dy), out)) <= 1e-2
    dgate = g["dgate"].cpu().numpy()
    ref = TO.route_backward(logits, idx, dgate, score, renorm, cfg.rsf,
                            layer.balance["dscore"].cpu().numpy(), off.tolist())
    assert np.all(np.abs(g["dlogits"].cpu().numpy() - ref) <=
                  256 * U * (cfg.rsf * np.abs(dgate).max() + layer.balance["dscore"].max().item()))
    assert rel_frob(f64(g["dw_router"]), ref.T @ h["x"]) <= 1e-2
    dx = ref @ h["w_router"]
    for t in range(cfg.T):
        for j, e in enumerate(idx[t]):
            dx[t] += O.expert_backward(h["x"][t][None], h["w1"][e], h["w3"][e], h["w2"][e],
                                       w[t, j] * f64(dy)[t][None])[0][0]
    if shared:
        dx += O.expert_backward(h["x"], h["ws1"], h["ws3"], h["ws2"], f64(dy))[0]
    assert rel_frob(f64(g["dx"]), dx) <= 1e-2


def test_sigmoid_router_equals_the_plain_layer(M):
    """Sigmoid, renormalised, top-2 groups is moe_route's router: the scored layer's results
    are the plain layer's up to fp32 roundings of the gates."""
    cfg = shape(I_shared=128)
    d = synth.gen_all(cfg, "cuda")
    c = M.config_from_shape(cfg)
    dy = synth.gen_dy(cfg, "cuda")
    res = []
    for r in (None, M.MoERouter(0, 1, 2)):
        layer = M.MoETrainLayer(c, weights_dict(d), d["w_router"], d["bias"], router=r)
        y = layer.forward(d["x"])
        res.append((y, layer.backward(dy), layer.saved["topk_idx"].clone()))
    assert torch.equal(res[0][2], res[1][2])
    assert rel_frob(f64(res[1][0]), f64(res[0][0])) <= 1e-3
    for key in res[0][1]:
        assert rel_frob(f64(res[1][1][key]), f64(res[0][1][key])) <= 2e-3, key


def test_masked_tokens_pass_the_layer(M):
    """A token without a selectable expert (its logits are NaN) gets the shared expert's output
    alone, reports its dropped places, and leaves the other tokens as they were."""
    cfg = shape(I_shared=128)
    d = synth.gen_all(cfg, "cuda")
    c, r = M.config_from_shape(cfg), M.MoERouter(1, 1, 1)
    layer = M.MoETrainLayer(c, weights_dict(d), d["w_router"], None, router=r, balance_coef=0.1)
    y0 = layer.forward(d["x"]).clone()
    assert layer.device_status() == 0
    bad = d["w_router"].clone()
    bad[2:] = float("nan")  # two experts are left, in one group, of top_k 4
    layer.w_router = bad
    y1 = layer.forward(d["x"])
    torch.cuda.synchronize()
    idx = layer.saved["topk_idx"].cpu().numpy()
    assert set(idx[:, :2].flatten()) == {0, 1} and (idx[:, 2:] == -1).all()
    assert layer.device_status() == 4
    h = {k: f64(v) for k, v in d.items()}
    ref = oracle_layer(cfg, h, idx, layer.saved["topk_w"].cpu().numpy().astype(np.float64))[0]
    assert rel_frob(f64(y1), ref) <= 1e-2 and torch.isfinite(y0).all()


@pytest.mark.parametrize("dtype", ["mxfp8", "nvfp4"])
def test_block_scaled_layers_take_the_router(M, dtype):
    """The scored router in the block-scaled layers: the plain layer's results where the two
    routers are the same (up to fp32 roundings of the gates)."""
    cfg = synth.get_config("tiny_bf16_T64").scaled(dtype=dtype, H=256, I=256, I_shared=256,
                                                    pad_multiple=128)
    d = synth.gen_all(cfg, "cuda")
    c = M.config_from_shape(cfg)
    ys = [M.MoELayer(c, weights_dict(d), d["w_router"], d["bias"], router=r).forward(d["x"])
          for r in (None, M.MoERouter(0, 1, 2))]
    assert rel_frob(f64(ys[1]), f64(ys[0])) <= 1e-3


def test_captured_steps_of_different_sequences(M):
    """Two captured training steps of one layer, with one and with three sequences, replayed in
    turn: each gives what the eager step gives, the loss and the gradients among them."""
    cfg = shape()
    d = synth.gen_all(cfg, "cuda")
    c, r = M.config_from_shape(cfg), M.MoERouter(0, 1, 1)
    layer = M.MoETrainLayer(c, weights_dict(d), d["w_router"], None, router=r, balance_coef=0.3)
    dy = synth.gen_dy(cfg, "cuda")
    offs = [None, torch.tensor([0, 20, 20, 60], dtype=torch.int32, device="cuda")]
    out = torch.empty_like(d["x"])

    def step(off):
        layer.forward(d["x"], out=out, seq_offsets=off)
        g = layer.backward(dy)
        return {**g, "loss": layer.balance["loss"], "load": layer.balance["load"], "y": out}

    eager = [{k: v.clone() for k, v in step(off).items()} for off in offs]
    graphs, held = [], []
    for off in offs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(step(off))
    for i in (0, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        for k, v in eager[i].items():
            assert rel_frob(f64(held[i][k]), f64(v)) <= 1e-6, k
        assert torch.equal(held[i]["load"], eager[i]["load"])
    assert layer.device_status() == 0
    del graphs


@pytest.mark.parametrize("shared", [0, 128])
def test_training_steps_with_muon(M, shared):
    """Forward, balance loss, backward, Muon on every weight, and the next forward with the
    new weights; the updated weights against the oracle given the same gradients."""
    cfg = shape(I_shared=shared)
    d = synth.gen_all(cfg, "cuda")
    c, r = M.config_from_shape(cfg), M.MoERouter(1, 1, 1)
    weights = weights_dict(d)
    layer = M.MoETrainLayer(c, weights, d["w_router"], None, router=r, balance_coef=0.01)
    params = dict(weights, w_router=d["w_router"])
    opt = M.MoEMuon(params, decay=0.1)
    ns = (3.4445, -4.7750, 2.0315)
    ys = []
    for it in range(2):
        ys.append(layer.forward(d["x"]).clone())
        g = layer.backward(synth.gen_dy(cfg, "cuda"))
        before = {k: f64(v).copy() for k, v in params.items()}
        mom = {k: f64(v).copy() for k, v in opt.momentum.items()}
        opt.step(g, 0.05)
        layer.update_weights(weights, d["w_router"])
        torch.cuda.synchronize()
        assert opt.device_status() == 0 and layer.device_status() == 0
        for k, v in params.items():
            sh = before[k].shape if before[k].ndim == 3 else (1,) + before[k].shape
            step = 0.05 * max(1.0, sh[1] / sh[2]) ** 0.5
            m, w = TO.muon_step(f64(g["d" + k]).reshape(sh), mom[k].reshape(sh),
                                before[k].reshape(sh), 0.95, True, step, 0.005, 5, *ns, 1e-7)
            assert rel_frob(f64(opt.momentum[k]).reshape(sh), m) <= 1e-6, k
            off = np.maximum(np.abs(f64(v).reshape(sh) - w) - 2.0 ** -8 * np.abs(w), 0)
            moved = np.linalg.norm(w - 0.995 * before[k].reshape(sh))
            assert np.linalg.norm(off) <= 4e-3 * moved, k
    # the layer runs on the new weights
    fresh = M.MoETrainLayer(c, weights, d["w_router"], None, router=r)
    assert torch.equal(layer.forward(d["x"]), fresh.forward(d["x"]))
    assert not torch.equal(ys[0], ys[1])
    with pytest.raises(ValueError):
        M.MoETrainLayer(c, weights, d["w_router"], d["bias"], balance_coef=0.1)
