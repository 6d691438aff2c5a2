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
