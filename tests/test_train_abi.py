"""Refusals of the scored router, the balance loss and the Muon calls: every case below fails
validation on the host, before the first CUDA call."""

import ctypes

import pytest
import torch

import synth

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def M():
    import mixture_experts_layer_grouped_b200 as M
    from mixture_experts_layer_grouped_b200 import build
    build.build()
    return M


def _cfg(M, **kw):
    return M.config_from_shape(synth.get_config("tiny_bf16_T64").scaled(**kw))


def _size(M, fn, *args):
    n = ctypes.c_size_t()
    return getattr(M.lib(), fn)(*args, ctypes.byref(n)), n.value


@pytest.mark.parametrize("router", [(2, 1, 1), (-1, 1, 1), (0, 2, 1), (1, 1, 0), (1, 1, 3)])
def test_router_options_are_checked(M, router):
    c, r = _cfg(M), M.MoERouter(*router)
    b = ctypes.byref
    assert M.lib().moe_route_scored(b(c), b(r), None, None, None, FAKE, None, FAKE, FAKE, None, 0,
                                    None) == 1
    assert M.lib().moe_route_backward(b(c), b(r), FAKE, FAKE, FAKE, None, None, 1, None, FAKE,
                                      None) == 1
    assert M.lib().moe_balance_loss(b(c), b(r), FAKE, FAKE, None, 1, 0.1, FAKE, FAKE, FAKE, FAKE,
                                    1 << 30, None) == 1


def test_route_scored_rejects(M):
    lib, b = M.lib(), ctypes.byref
    c, r = _cfg(M), M.MoERouter(1, 1, 1)
    nb, _ = M.moe_workspace_size(c)
    call = lambda c=c, r=b(r), x=FAKE, w=FAKE, li=None, lo=FAKE, idx=FAKE, gates=FAKE, ws=FAKE, n=nb: (
        lib.moe_route_scored(b(c), r, x, w, None, li, lo, idx, gates, ws, n, None))
    assert call(r=None) == 1
    assert call(idx=None) == 1 and call(gates=None) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(lo=None) == 1
    assert call(x=ctypes.c_void_p((1 << 20) + 4)) == 1
    assert call(ws=None) == 1 and call(n=16) == 3
    assert call(c=_cfg(M, top_k=40)) == 2


def test_route_backward_rejects(M):
    lib, b = M.lib(), ctypes.byref
    c, r = _cfg(M), M.MoERouter(1, 1, 1)
    ok = dict(l=FAKE, i=FAKE, g=FAKE, ds=None, off=None, n=1, d=FAKE)

    def call(**kw):
        v = {**ok, **kw}
        return lib.moe_route_backward(b(c), b(r), v["l"], v["i"], v["g"], v["ds"], v["off"], v["n"],
                                      None, v["d"], None)

    for key in ("l", "i", "g", "d"):
        assert call(**{key: None}) == 1
    assert call(ds=FAKE, n=0) == 1
    assert call(ds=FAKE, n=2) == 1  # several sequences need their offsets


def test_balance_rejects(M):
    lib, b = M.lib(), ctypes.byref
    c, r = _cfg(M), M.MoERouter(0, 1, 1)
    code, nb = _size(M, "moe_balance_workspace_size", b(c), 4)
    assert code == 0 and nb > 0
    assert _size(M, "moe_balance_workspace_size", b(c), 0)[0] == 1
    assert _size(M, "moe_balance_workspace_size", b(c), 1 << 21)[0] == 2
    assert lib.moe_balance_workspace_size(b(c), 1, None) == 1
    call = lambda off=FAKE, n=4, loss=FAKE, ws=FAKE, nb=nb: lib.moe_balance_loss(
        b(c), b(r), FAKE, FAKE, off, n, 0.1, loss, FAKE, FAKE, ws, nb, None)
    assert call(loss=None) == 1 and call(ws=None) == 1
    assert call(off=None) == 1
    assert call(nb=16) == 3
    assert call(ws=ctypes.c_void_p((1 << 20) + 8)) == 1


def _muon(M, **kw):
    v = dict(groups=2, rows=64, cols=32, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7)
    v.update(kw)
    return M.MoEMuonConfig(**v)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=0), 1), (dict(rows=0), 1), (dict(cols=-3), 1), (dict(steps=0), 1),
    (dict(steps=65), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(groups=65536), 2), (dict(rows=1 << 15, cols=(1 << 15) + 1), 2),
    (dict(a=20.0), 2),               # singular values grow past what fp16 holds
    (dict(a=float("nan")), 2), (dict(b=-40.0, c=38.0), 2),
    (dict(), 0), (dict(a=1.5, b=-0.5, c=0.0, steps=64), 0), (dict(a=2.0, b=-1.5, c=0.5), 0)])
def test_muon_config_is_checked(M, kw, code):
    assert _size(M, "moe_muon_workspace_size", ctypes.byref(_muon(M, **kw)))[0] == code


def test_muon_calls_reject(M):
    lib, b = M.lib(), ctypes.byref
    c = _muon(M)
    nb = M.moe_muon_workspace_size(c)
    assert lib.moe_orthogonalize(b(c), None, 0, FAKE, FAKE, nb, None) == 1
    assert lib.moe_orthogonalize(b(c), FAKE, 2, FAKE, FAKE, nb, None) == 1
    assert lib.moe_orthogonalize(b(c), FAKE, 0, None, FAKE, nb, None) == 1
    assert lib.moe_orthogonalize(b(c), FAKE, 0, FAKE, None, nb, None) == 1
    assert lib.moe_orthogonalize(b(c), FAKE, 0, FAKE, FAKE, nb - 1, None) == 3
    step = lambda m=FAKE, mo=FAKE, beta=0.9, nest=1, w=FAKE, wo=FAKE: lib.moe_muon_step(
        b(c), FAKE, 0, m, mo, beta, nest, w, wo, 0.1, 0.0, FAKE, nb, None)
    assert step(m=None) == 1 and step(mo=None) == 1 and step(w=None) == 1 and step(wo=None) == 1
    assert step(beta=1.0) == 1 and step(beta=-0.1) == 1 and step(beta=float("nan")) == 1
    assert step(nest=2) == 1


def test_binding_checks_shapes_and_devices(M):
    """Host tensors, other shapes, other types and other layouts are a ValueError before any
    C call."""
    c, r = _cfg(M), M.MoERouter(1, 1, 1)
    T, E, k = c.T, c.E, c.top_k
    x, idx, w = torch.zeros(T, E), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    with pytest.raises(ValueError):
        M.moe_route_scored(c, r, idx, w, logits_in=x)
    with pytest.raises(ValueError, match="of shape"):
        M.moe_route_scored(c, r, idx, w, logits_in=x[:-1])
    with pytest.raises(ValueError, match="of shape"):
        M.moe_route_backward(c, r, x[:, 1:], idx, w, x)
    with pytest.raises(ValueError, match="offsets"):
        M.moe_balance_loss(c, r, x, idx, 0.1, w, idx, w, x, seq_offsets=torch.zeros(1))
    m = _muon(M)
    g = torch.zeros(2, 64, 32)
    with pytest.raises(ValueError):
        M.moe_orthogonalize(m, g, g, g)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        M.moe_orthogonalize(m, g.half(), g, g)
    with pytest.raises(ValueError, match="of shape"):
        M.moe_orthogonalize(m, g.mT, g, g)
