"""The gated activation and its gradient on the GPU where a factor is infinite, NaN, or past the range."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8
from oracle import primitives as prim
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu
f32 = prim.bf16_to_f32
INF = float("inf")


def bits(a):
    return prim.f32_to_bf16(np.asarray(a, np.float32))


def same_non_finite(got, want):
    """NaN where want is NaN, and its infinities with their signs."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))


GATES = [INF, -INF, float("nan"), 3.38e38, -3.38e38, 100.0, 2.0, 0.0, -0.0, -2.0, -80.0]
UPS = [1.5, -2.0, 0.0, INF, -INF, float("nan")]


def grid(cols):
    """[gates x ups] rows with one pair each, zeros elsewhere: the first column of g and of u."""
    g, u = (v.reshape(-1) for v in np.meshgrid(GATES, UPS, indexing="ij"))
    h = np.zeros((g.size, 2 * cols))
    h[:, 0], h[:, cols] = g, u
    return h


@pytest.mark.parametrize("cols", [16, 144])
def test_activation_of_infinities(cols):
    h = grid(cols)
    y = torch.full((h.shape[0], cols), 7.0, dtype=torch.bfloat16, device="cuda")
    _, scales = fq.qf_swiglu_quant_fp8(dev(bits(h)), y=y)
    with np.errstate(all="ignore"):
        a = fp8.swiglu(f32(bits(h)))
    # products past the range of fp32 are infinite as bf16 (and of a block with one the scale is NaN)
    a = np.where(np.abs(a) >= 2.0 ** 128, np.copysign(INF, a), a)
    same_non_finite(f32(host(y)), a)
    assert not f32(host(y))[:, 1:].any()
    s = scales.cpu().numpy()
    assert np.array_equal(np.isnan(s[0]), ~np.isfinite(a[:, 0])) and not s[1:].any()


@pytest.mark.parametrize("cols", [8, 136])
@pytest.mark.parametrize("da", [1.0, -3.0, 0.0, INF, -INF, float("nan")])
def test_gradient_of_infinities(cols, da):
    h = grid(cols)
    d = np.zeros((h.shape[0], cols))
    d[:, 0] = da
    got = f32(host(fq.qf_swiglu_backward(dev(bits(h)), dev(bits(d)))))
    hf, df = f32(bits(h)), f32(bits(d))
    with np.errstate(all="ignore"):
        want = fp8.swiglu_backward(hf, df)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(INF, want), want)
    same_non_finite(got[:, [0, cols]], want[:, [0, cols]])
    rest = np.delete(got, [0, cols], 1)
    assert not rest.any()


def test_gradient_past_the_range():
    """da u passes fp32's range, the gradient does not."""
    cols = 16
    g = np.array([-85.0, -80, -60, -40, -20, -1.28, 0, 5, 200])
    pairs = [(1e30, 1e30), (-3e38, 2e5), (2.0, 3e38), (1e-30, -3e38), (3e38, 1e-38), (3.38e38, 1.0), (1e25, 1e15)]
    rows = [(a, b, c) for a in g for b, c in pairs]
    h, d = np.zeros((len(rows), 2 * cols)), np.zeros((len(rows), cols))
    for i, (a, b, c) in enumerate(rows):
        h[i, 0], h[i, cols], d[i, 0] = a, c, b
    got = f32(host(fq.qf_swiglu_backward(dev(bits(h)), dev(bits(d))))).astype(np.float64)[:, 0]
    hf, df = f32(bits(h)).astype(np.float64), f32(bits(d)).astype(np.float64)
    want = fp8.swiglu_backward(hf, df)[:, 0]
    # the sigmoid is off by at most 16 2^-24 of itself or by 2^-119, 1 + g (1 - s) by 20 2^-24 of 1 + |g|, and two products follow
    g, p = hf[:, 0], np.abs(df[:, 0] * hf[:, cols])
    off = (64 * 2.0 ** -24 * fp8.sigmoid(g) + 2.0 ** -119) * p * (1 + np.abs(g))
    top = 2.0 ** 128 * (1 - 2.0 ** -9)              # what is larger rounds to an infinity
    keep = np.abs(want) + off < top * (1 - 2.0 ** -8)
    assert keep.sum() > 40 and np.any(keep & (p > top))
    err = np.abs(got - want)
    assert np.all((err <= 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * off + 2.0 ** -134)[keep]), np.argwhere(~(err <= off) & keep)
    past = np.abs(want) - off > top * (1 + 2.0 ** -8)
    assert past.any() and np.array_equal(got[past], np.copysign(INF, want[past]))


@pytest.mark.parametrize("u", [INF, -INF])
@pytest.mark.parametrize("da", [1e-38, -2.0 ** -133, 3e38])
def test_gradient_of_an_infinite_factor(u, da):
    """An infinite u or da against a small other factor and a small sigmoid: the formula's infinity, no NaN."""
    cols = 16
    g = np.array([-85.0, -60, -20, -2, 0, 2, 200])
    h, d = np.zeros((2 * g.size, 2 * cols)), np.zeros((2 * g.size, cols))
    h[:, 0] = np.tile(g, 2)
    h[:, cols] = np.repeat([u, da], g.size)
    d[:, 0] = np.repeat([da, u], g.size)
    got = f32(host(fq.qf_swiglu_backward(dev(bits(h)), dev(bits(d)))))
    with np.errstate(all="ignore"):
        want = fp8.swiglu_backward(f32(bits(h)), f32(bits(d)))
    assert np.isinf(want[:, 0]).all()
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(INF, want), want)
    same_non_finite(got, want)
