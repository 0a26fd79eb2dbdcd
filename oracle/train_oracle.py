"""CPU oracle of the scored router, its gradient, the balance loss and the orthogonalised
update -- TEST INFRASTRUCTURE ONLY.

Plain fp64 numpy statements of include/moe_b200.h's definitions, one row or one matrix at a
time; they share no code with the CUDA kernels.  Pinned on the CPU by brute force, central
finite differences and the closed form by singular values.
"""

import numpy as np

SIGMOID, SOFTMAX = 0, 1


def scores(l, kind):
    """Scores of one row; a logit of -inf or NaN has none (0)."""
    l = np.asarray(l, np.float64)
    ok = l > -np.inf
    s = np.zeros_like(l)
    if not ok.any():
        return s
    if kind == SIGMOID:
        with np.errstate(over="ignore"):
            s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        return s
    m = l[ok].max()
    with np.errstate(invalid="ignore"):
        e = np.where(l[ok] == m, 1.0, np.exp(l[ok] - m))
    s[ok] = e / e.sum()
    return s


def log_scores(l, kind):
    """Logarithms of scores() up to a constant of the row: ratios of scores that are too small
    for 64 bits stay what they are."""
    l = np.asarray(l, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        v = l if kind == SOFTMAX else -np.logaddexp(0.0, -l)
    return np.where(l > -np.inf, v, -np.inf)


def shares(v):
    """exp(v) / sum exp(v); zeros where nothing is above -inf."""
    v = np.asarray(v, np.float64)
    m = v.max() if len(v) else -np.inf
    if m == -np.inf:
        return np.zeros_like(v)
    with np.errstate(invalid="ignore"):
        e = np.where(v == m, 1.0, np.exp(v - m))
    return e / e.sum()


def route_row(l, bias, G, g, k, kind, renorm, group_top, rsf):
    """(indices, gates) of one row; index -1 and gate 0 where nothing is left to select."""
    l = np.asarray(l, np.float64)
    E = len(l)
    s = scores(l, kind)
    ok = l > -np.inf
    key = l.copy() if bias is None else s + np.asarray(bias, np.float64)
    ok &= key > -np.inf
    if G > 1:
        by = s if bias is None and group_top == 2 else key
        total = []
        for q in range(G):
            mine = sorted((by[e] for e in range(q * E // G, (q + 1) * E // G) if ok[e]),
                          reverse=True)[:group_top]
            total.append(sum(mine) if mine else -np.inf)
        order = sorted(range(G), key=lambda q: (-total[q], q))
        kept = {q for q in order[:g] if total[q] > -np.inf}
        ok &= np.array([e // (E // G) in kept for e in range(E)])
    best = sorted((e for e in range(E) if ok[e]), key=lambda e: (-key[e], e))[:k]
    idx = np.full(k, -1, np.int64)
    idx[: len(best)] = best
    return idx, gates_row(l, idx, kind, renorm, rsf)


def gates_row(l, idx, kind, renorm, rsf):
    E, some = len(l), [0 <= e < len(l) for e in idx]
    if renorm:
        v = log_scores(l, kind)
        return rsf * shares([v[e] if ok else -np.inf for e, ok in zip(idx, some)])
    s = scores(l, kind)
    return rsf * np.array([s[e] if ok else 0.0 for e, ok in zip(idx, some)])


def route(logits, bias, G, g, k, kind, renorm, group_top, rsf):
    rows = [route_row(l, bias, G, g, k, kind, renorm, group_top, rsf) for l in logits]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def sequence_of(offsets, T):
    """The sequence of each row, -1 outside all."""
    q = np.full(T, -1)
    for i in range(len(offsets) - 1):
        q[offsets[i]:offsets[i + 1]] = i
    return q


def route_backward(logits, idx, dgate, kind, renorm, rsf, dscore=None, offsets=None, dloss=1.0):
    """dlogits of sum(gates * dgate), plus those of the balance loss given its dscore."""
    T, E = logits.shape
    out = np.zeros((T, E))
    seq = sequence_of([0, T] if offsets is None else offsets, T)
    for t in range(T):
        s, v = scores(logits[t], kind), log_scores(logits[t], kind)
        dlog = np.zeros(E)  # with respect to the scores' logarithms
        at = [(j, e) for j, e in enumerate(idx[t]) if 0 <= e < E and v[e] > -np.inf]
        g = np.array([rsf * float(dgate[t, j]) for j, _ in at])
        w = shares([v[e] for _, e in at]) if renorm else np.array([s[e] for _, e in at])
        for (j, e), gj, wj in zip(at, g, w):
            dlog[e] += wj * (gj - (np.sum(g * w) if renorm else 0.0))
        if dscore is not None and seq[t] >= 0:
            c = dloss * np.asarray(dscore[seq[t]], np.float64)
            p = shares(v)
            dlog += p * (c - np.sum(c * p))
        # d log s_e / d l_e: 1 - s_e, or for the softmax delta - p
        out[t] = dlog * (1 - s) if kind == SIGMOID else dlog - s * np.sum(dlog)
    return out


def balance(logits, idx, kind, k, coef, offsets=None):
    """(loss, load [S, E], dscore [S, E])."""
    T, E = logits.shape
    offsets = [0, T] if offsets is None else offsets
    S = len(offsets) - 1
    loss, load, d = 0.0, np.zeros((S, E), np.int64), np.zeros((S, E))
    for q in range(S):
        P, n = np.zeros(E), 0
        for t in range(offsets[q], offsets[q + 1]):
            v = log_scores(logits[t], kind)
            if v.max() > -np.inf:
                P += shares(v)
                n += 1
            for e in idx[t]:
                if 0 <= e < E:
                    load[q, e] += 1
        if n:
            f = E / (k * n) * load[q]
            d[q] = coef / S * f / n
            loss += coef / S * np.sum(f * P / n)
    return loss, load, d


def orthogonalize(u, steps, a, b, c, eps):
    """One matrix through the Newton-Schulz steps."""
    x = np.asarray(u, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt(np.sum(x * x)) + eps)
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.T if tall else x


def muon_step(grad, m, w, beta, nesterov, step, decay, steps, a, b, c, eps):
    """(m', w') of a stack of matrices."""
    m = beta * np.asarray(m, np.float64) + grad
    u = grad + beta * m if nesterov else m
    x = np.stack([orthogonalize(v, steps, a, b, c, eps) for v in u])
    return m, (1 - decay) * w - step * x
