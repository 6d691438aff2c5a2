"""CPU pins of the routing oracle, and the host checks of the routing calls."""

import ctypes
import math

import numpy as np
import pytest
import torch

from fp4_fake_quant_amd import _lib
from oracle import route

INF = math.inf


def by_hand(x, k, scoring, bias, n_group, topk_group, rule, renorm, scale):
    E = len(x)
    if scoring == "sigmoid":
        s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in x]
    else:
        m = max(x)
        e = [math.exp(v - m) if v > -INF else 0.0 for v in x]
        s = [v / math.fsum(e) for v in e]
    key = [(s[i] + bias[i]) if x[i] > -INF else -INF for i in range(E)]
    size = E // n_group
    gs = []
    for g in range(n_group):
        own = sorted((v for v in key[g * size:(g + 1) * size] if v > -INF), reverse=True)
        gs.append(sum(own[:2 if rule == "top2" else 1]) if own else -INF)
    kept = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
    pool = [i for i in range(E) if i // size in kept and key[i] > -INF]
    best = sorted(pool, key=lambda i: (-key[i], i))[:k]
    u = [s[i] for i in best]
    if renorm and u:
        u = [v / math.fsum(u) for v in u]
    return best + [-1] * (k - len(best)), [v * scale for v in u] + [0.0] * (k - len(best))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group,rule", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2"), (12, 5, "top2")])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_by_hand(scoring, n_group, topk_group, rule, renorm):
    rng = np.random.default_rng(n_group + renorm)
    x = np.round(rng.standard_normal((40, 12)) * 3) / 2            # many ties
    x[3, 2:9] = -INF
    x[4, 1:] = -INF
    bias = np.round(rng.standard_normal(12) * 2) / 8
    for b in (None, bias):
        idx, w = route.route(x, 5, scoring, b, n_group, topk_group, rule, renorm, 1.5)
        for t in range(40):
            hi, hw = by_hand(x[t], 5, scoring, np.zeros(12) if b is None else b, n_group, topk_group, rule, renorm, 1.5)
            assert idx[t].tolist() == hi
            assert np.allclose(w[t], hw, rtol=1e-12, atol=1e-15)
    idx, w = route.route(np.full((1, 12), -INF), 5, scoring, None, n_group, topk_group, rule, renorm, 1.0)
    assert np.all(idx == -1) and not w.any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(scoring, renorm):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 9))
    idx = np.stack([rng.permutation(9)[:4] for _ in range(6)]).astype(np.int32)
    idx[0, 2] = -1
    idx[1] = -1
    idx[2, 1] = idx[2, 0]                                          # an index given twice
    dw = rng.standard_normal((6, 4))
    got, mag = route.backward(x, idx, dw, scoring, renorm, 2.0)
    h = 1e-5
    for e in range(9):
        d = np.zeros_like(x)
        d[:, e] = h
        diff = ((route.weights_of(x + d, idx, scoring, renorm, 2.0) - route.weights_of(x - d, idx, scoring, renorm, 2.0)) * dw).sum(1) / (2 * h)
        assert np.allclose(got[:, e], diff, rtol=0, atol=1e-8)     # h^2 times a third derivative of order 1
    assert np.all(np.abs(got) <= mag + 1e-15)


@pytest.mark.parametrize("x", [-40.0, -9.0, 0.5, 8.0, 20.0, 37.0, 60.0, 300.0])
def test_sigmoid_gradient_closed_form(x):
    """s (1 - s) = 1 / (2 + 2 cosh x), also where 1 - s is below the rounding of s; over its sum with
    a second choice of score 1/2, the derivative by hand."""
    both, one = np.array([[x, 0.0, -1.0]]), np.ones((1, 1))
    d, mag = route.backward(both, np.zeros((1, 1), np.int32), one, "sigmoid", False, 1.0)
    assert np.allclose(d[0], [1 / (2 + 2 * math.cosh(x)), 0, 0], rtol=1e-13, atol=0) and np.all(mag >= np.abs(d))
    d, _ = route.backward(both, np.array([[0, 1]], np.int32), np.array([[1.0, 0.0]]), "sigmoid", True, 1.0)
    s = 1 / (1 + math.exp(-x))                               # w = s / (s + 1/2): dw/ds = (1/2) / (s + 1/2)^2
    assert np.allclose(d[0, 0], 0.5 / (s + 0.5) ** 2 / (2 + 2 * math.cosh(x)), rtol=1e-12, atol=0)


@pytest.mark.parametrize("at", [-30.0, -89.0, -800.0, -1e6])
def test_low_sigmoid_scores(at):
    """Far below zero a sigmoid is exp(x), so its shares are a softmax's, however small the scores."""
    x = np.array([[0.0, -1.0, 2.0, -3.0]]) + at
    idx, w = route.route(x, 3, "sigmoid")
    e = np.exp(np.array([2.0, 0.0, -1.0]))
    assert idx.tolist() == [[2, 0, 1]] and np.allclose(w[0], e / e.sum(), rtol=1e-12, atol=0)
    p, g = e / e.sum(), np.array([0.5, -1.0, 2.0])
    d, _ = route.backward(x, idx, g[None], "sigmoid", True, 1.0)
    assert np.allclose(d[0, [2, 0, 1]], p * (g - (g * p).sum()), rtol=1e-11, atol=0) and d[0, 3] == 0


def test_refusals():
    L = _lib.lib()
    p = 0x10000000

    def call(back=False, idx=p + 0x100000, w=p + 0x200000, dl=p + 0x300000, ldd=64, **kw):
        d = _lib.RouteDesc()
        base = dict(logits=p, tokens=10, ld=64, bias=None, scale=1.0, logits_bf16=0, experts=64, k=8, scoring=0, renorm=1,
                    n_group=1, topk_group=1, group_rule=0)
        for key, v in dict(base, **kw).items():
            setattr(d, key, v)
        if back:
            return L.qf_moe_route_backward(ctypes.byref(d), ctypes.c_void_p(idx) if idx else None,
                                           ctypes.c_void_p(w) if w else None, ctypes.c_void_p(dl) if dl else None, ldd, None)
        return L.qf_moe_route(ctypes.byref(d), ctypes.c_void_p(idx) if idx else None, ctypes.c_void_p(w) if w else None, None)

    for back in (False, True):
        assert call(back, tokens=0) == 0
        assert call(back, experts=0) == 2 and call(back, experts=1025, ld=1025) == 2 and call(back, ld=63) == 2
        assert call(back, tokens=-1) == 2 and call(back, tokens=1 << 30) == 2
        assert call(back, tokens=(1 << 26) + 1) == 2         # one launch holds no more rows
        assert call(back, k=0) == 7 and call(back, k=33) == 7 and call(back, experts=4, k=5) == 7
        assert call(back, scoring=2) == 7 and call(back, renorm=2) == 7 and call(back, logits_bf16=2) == 7
        assert call(back, scale=float("nan")) == 7 and call(back, scale=INF) == 7
        assert call(back, logits=None) == 1 and call(back, idx=None) == 1 and call(back, w=None) == 1
        assert call(back, logits=p + 2) == 3 and call(back, idx=p + 2) == 3 and call(back, w=p + 2) == 3
        assert call(back, logits=p + 1, logits_bf16=1) == 3
    assert call(n_group=3) == 7 and call(n_group=65, experts=65, ld=65) == 7 and call(n_group=8, topk_group=9) == 7
    assert call(n_group=8, topk_group=0) == 7 and call(n_group=0) == 7 and call(n_group=16, topk_group=1, k=5) == 7
    assert call(group_rule=2) == 7 and call(bias=p + 2) == 3
    assert call(True, dl=None) == 1 and call(True, ldd=63) == 2 and call(True, dl=p + 2) == 3
    assert L.qf_moe_route(None, None, None, None) == 1


def test_every_finite_scale_is_taken():
    L = _lib.lib()
    p, most = 0x10000000, float(np.finfo(np.float32).max)
    for scale, want in ((most, 0), (-most, 0), (3.3e38, 0), (0.0, 0), (INF, 7), (-INF, 7), (float("nan"), 7)):
        d = _lib.RouteDesc(p, 0, 8, None, scale, 0, 8, 2, 0, 1, 1, 1, 0)
        assert L.qf_moe_route(ctypes.byref(d), p, p, None) == want
        assert L.qf_moe_route_backward(ctypes.byref(d), p, p, p, 8, None) == want


def test_binding_refuses_host_tensors():
    import fp4_fake_quant_amd as fq
    with pytest.raises(TypeError):
        fq.qf_moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        fq.qf_moe_route(torch.zeros(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        fq.qf_moe_route(torch.zeros(2, 8), 2, scoring="relu")
