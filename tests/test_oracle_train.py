"""Pins of the oracle's scored router, balance loss and orthogonalised update."""

import itertools

import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import train_oracle as TO

NS = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_is_the_best_of_all_choices(kind, biased, group_top):
    """Every set of kept groups and every ordered choice of experts, by enumeration."""
    rng = np.random.default_rng(3)
    for _ in range(20):
        E, G, g, k = 8, 4, 2, 3
        l = rng.normal(size=E)
        bias = rng.normal(size=E) * 0.2 if biased else None
        s = np.exp(l) / np.exp(l).sum() if kind else 1 / (1 + np.exp(-l))
        key = l if bias is None else s + bias
        by = s if bias is None and group_top == 2 else key

        kept = max(itertools.combinations(range(G), g),
                   key=lambda c: sum(sum(sorted(by[2 * q: 2 * q + 2])[::-1][:group_top])
                                     for q in c))
        # the ordered choice whose first key is largest, then its second, ...
        want = max(itertools.permutations([e for q in kept for e in (2 * q, 2 * q + 1)], k),
                   key=lambda p: tuple(key[list(p)]))
        idx, w = TO.route_row(l, bias, G, g, k, kind, False, group_top, 2.5)
        assert idx.tolist() == list(want)
        assert np.allclose(w, 2.5 * s[idx], rtol=1e-14)


def test_sigmoid_form_is_the_layer_router():
    """Sigmoid, bias, top-2 groups, renormalised: the layer oracle's own route()."""
    rng = np.random.default_rng(0)
    import synth
    cfg = synth.get_config("tiny_bf16_T64")
    l = rng.normal(size=(64, cfg.E))
    bias = rng.uniform(-0.1, 0.1, cfg.E)
    r = O.route(l, bias, cfg.n_group, cfg.topk_group, cfg.top_k, cfg.rsf)
    idx, w = TO.route(l, bias, cfg.n_group, cfg.topk_group, cfg.top_k, 0, True, 2, cfg.rsf)
    assert np.array_equal(idx, r["idx"])
    assert np.allclose(w, r["w"], rtol=1e-13)


def test_masks_and_ties():
    inf = np.inf
    l = np.array([1.0, -inf, np.nan, 1.0, 0.5])
    idx, w = TO.route_row(l, None, 1, 1, 4, 1, True, 1, 1.0)
    assert idx.tolist() == [0, 3, 4, -1] and w[3] == 0 and np.isclose(w.sum(), 1)
    idx, w = TO.route_row(np.full(4, -inf), None, 1, 1, 2, 1, True, 1, 1.0)
    assert idx.tolist() == [-1, -1] and not w.any()
    idx, w = TO.route_row([0.0, inf, 1.0], None, 1, 1, 2, 1, False, 1, 1.0)
    assert idx.tolist() == [1, 2] and w.tolist() == [1.0, 0.0]
    idx, _ = TO.route_row([1.0, 2.0, 3.0], [0, 0, -inf], 1, 1, 3, 0, True, 1, 1.0)
    assert idx.tolist() == [1, 0, -1]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_by_differences(kind, renorm):
    rng = np.random.default_rng(1)
    T, E, k, rsf, coef = 5, 6, 2, 2.5, 0.7
    l = rng.normal(size=(T, E))
    l[1, 2] = -np.inf
    idx, _ = TO.route(l, None, 1, 1, k, kind, renorm, 1, rsf)
    dgate = rng.normal(size=(T, k))
    off = [0, 2, 2, 4]  # an empty sequence, and a row outside
    _, _, dscore = TO.balance(l, idx, kind, k, coef, off)

    def total(x):
        gates = np.stack([TO.gates_row(x[t], idx[t], kind, renorm, rsf)
                          for t in range(T)])
        return np.sum(gates * dgate) + 1.5 * TO.balance(x, idx, kind, k, coef, off)[0]

    d = TO.route_backward(l, idx, dgate, kind, renorm, rsf, dscore, off, 1.5)
    for t, e in itertools.product(range(T), range(E)):
        if l[t, e] == -np.inf:
            assert d[t, e] == 0
            continue
        p, m = l.copy(), l.copy()
        p[t, e] += 1e-5
        m[t, e] -= 1e-5
        # central differences: error ~ h^2 f''' / 6 ~ 1e-10, rounding ~ 1e-16 / 1e-5
        assert abs(d[t, e] - (total(p) - total(m)) / 2e-5) < 1e-8


def test_ratios_of_scores_below_64_bits():
    """exp(-2000) is no number in 64 bits; the renormalised gates and shares still are."""
    for kind in (0, 1):
        idx, w = TO.route_row([-2000.0, -2001.0, -2001.0], None, 1, 1, 2, kind, True, 1, 1.0)
        assert idx.tolist() == [0, 1] and np.allclose(w, np.array([1, np.exp(-1)]) / (1 + np.exp(-1)))
    w = TO.gates_row([0.0, -2000.0, -2001.0], [1, 2], 1, True, 1.0)
    assert np.allclose(w, np.array([1, np.exp(-1)]) / (1 + np.exp(-1)))


def test_balance_of_even_load_is_coef():
    """With f = 1 for every expert, sum f P = sum P = 1."""
    E, k = 4, 2
    idx = np.array([[0, 1], [2, 3]])
    loss, load, _ = TO.balance(np.random.default_rng(0).normal(size=(2, E)), idx, 1, k, 0.3)
    assert np.isclose(loss, 0.3) and load.tolist() == [[1, 1, 1, 1]]


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 4)])
def test_orthogonalize_acts_on_the_singular_values(shape):
    rng = np.random.default_rng(2)
    g = rng.normal(size=shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    for _ in range(5):
        s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
    assert np.allclose(TO.orthogonalize(g, 5, *NS, 1e-7), (u * s) @ vt, atol=1e-12)
