"""CPU pins of the AdamW oracle and the host checks of qf_adamw_step."""

import ctypes

import numpy as np
import pytest
import torch

from fp4_fake_quant_amd import _lib
from oracle import adamw

U = 2.0 ** -24


def bounds64(p, g, m, v, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    """Bounds of |fp32 - float64| for p', m', v' by counting roundings of relative size U.

    g*s: 1.  m': factor, product and sum of each term (3), g (1), a decoded m (1): 5 of
    Sm = b1|m| + (1-b1)|g|.  v': factor, two products, sum (4), g twice (2), a decoded v (3): at
    most 9 of v', 4.5 of its root, plus the root's own: 5.5.  root factor and product: 7.5, eps
    and sum: 9.5 of the divisor.  quotient, size factor and product: 3.  Together 5 + 9.5 + 3 <
    18 of lr_t Sm / d.  p: factor, product, difference: 3 of |p| and 1 of the update.  One more
    of each covers the products of these terms.
    """
    p, g, m, v = (np.abs(np.asarray(x, np.float64)) for x in (p, g, m, v))
    g = g * grad_scale
    sm = beta1 * m + (1 - beta1) * g
    v64 = beta2 * v + (1 - beta2) * g * g
    d = np.sqrt(v64 / (1 - beta2 ** step)) + eps
    upd = lr / (1 - beta1 ** step) * sm / d
    return 4 * U * p + 20 * U * upd, 6 * U * sm, 10 * U * v64


def draw(n, seed, g_bf16=False):
    rng = np.random.default_rng(seed)
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    size = 2e-4 * np.exp(1.5 * rng.standard_normal(n))
    g = (rng.standard_normal(n) * size).astype(np.float32)
    if g_bf16:
        g = torch.from_numpy(g).bfloat16().float().numpy()
    m = (rng.standard_normal(n) * 0.3 * size).astype(np.float32)
    r = (np.abs(rng.standard_normal(n)) * 0.1 * size).astype(np.float32)
    return p, g, m, r


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 6])
@pytest.mark.parametrize("wd,gs", [(0.0, 1.0), (0.1, 0.37)])
def test_fp32_against_float64(step, wd, gs):
    p, g, m, r = draw(5000, step)
    if step == 1:
        m[:], r[:] = 0, 0
    g[:50] = 0
    v = r * r
    got = adamw.step32(p, g, m, v, 1e-3, step, weight_decay=wd, grad_scale=gs)
    want = adamw.step64(p, g, m, v, 1e-3, step, weight_decay=wd, grad_scale=float(np.float32(gs)))
    for a, b, tol in zip(got, want, bounds64(p, g, m, v, 1e-3, step, weight_decay=wd, grad_scale=gs)):
        assert np.all(np.abs(a - b) <= tol + 1e-44)


def test_e4m3_values():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(adamw.e4m3_values(), want, equal_nan=True)


def test_stochastic_rounding_neighbours_and_mean():
    """Every rounding lands on one of the two codes around y, and over all 65536 random numbers
    the mean is y to one part in 65536 of the step."""
    rng = np.random.default_rng(3)
    vals = adamw.e4m3_values()[:0x7F].astype(np.float64)
    ys = np.concatenate([vals[1:], rng.uniform(0, 448, 40), rng.uniform(0, 2.0 ** -6, 40), 2.0 ** rng.uniform(-12, 8, 40)])
    rnd = np.arange(65536, dtype=np.uint32)
    for y in ys.astype(np.float32):
        x = np.full(65536 * 2, y, np.float32)
        x[::256] = 448                       # a block whose scale is exactly 1
        pos = np.arange(x.size) % 256 != 0
        r = np.zeros(x.size, np.uint32)
        r[pos] = np.resize(rnd, pos.sum())
        codes, scales = adamw.encode(x, r, False)
        assert np.all(scales == np.float32(448) * np.float32(1 / 448))
        got = vals[codes[pos][:65536]]
        lo = vals[vals <= y].max()
        hi = vals[vals >= y].min()
        assert set(np.unique(got)) <= {lo, hi}
        assert abs(got.mean() - y) <= (hi - lo) * 2.0 ** -16 + float(y) * U


def test_encode_edges():
    x = np.zeros(600, np.float32)
    x[300] = 2.0 ** -101                     # block 1: below the smallest scaled maximum
    x[512] = -7.0
    x[513] = 1e-9
    for lift in (False, True):
        codes, scales = adamw.encode(x, np.zeros(600, np.uint32), lift)
        assert scales[0] == 0 and scales[1] == 0 and not codes[:512].any()
        assert codes[512] == 0x80 | 0x7E and codes[513] == int(lift)
        assert scales.size == 3


def test_refusals():
    L = _lib.lib()

    def call(n=1, bits=32, **kw):
        t = (_lib.AdamwTensor * 1)()
        for k, a in zip(("p", "g", "m", "v", "m_scale", "v_scale"), range(6)):
            setattr(t[0], k, 0x10000000 + a * 0x100000)
        t[0].n = 0
        h = _lib.AdamwHyper(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None, None, 0)
        for k, v in kw.items():
            setattr(h if hasattr(h, k) else t[0], k, v)
        return L.qf_adamw_step(ctypes.byref(t), n, bits, ctypes.byref(h), None)

    assert call() == 0 and call(n=0) == 0                # nothing to do
    assert call(bits=16) == 7 and call(n=-1) == 7
    nan = float("nan")
    for k in ("beta1", "beta2"):
        assert call(**{k: 1.0}) == 7 and call(**{k: -0.1}) == 7 and call(**{k: nan}) == 7
    assert call(eps=-1.0) == 7 and call(eps=nan) == 7 and call(lr=nan) == 7 and call(lr=-1.0) == 7
    assert call(step=0) == 7 and call(weight_decay=nan) == 7 and call(weight_decay=-0.1) == 7 and call(g_bf16=2) == 7
    assert call(d_step=0x10000004) == 3 and call(d_lr=0x10000002) == 3 and call(d_skip=0x10000001) == 3
    t = (_lib.AdamwTensor * 1)()
    h = _lib.AdamwHyper(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None, None, 0)

    def sized(bits=32, **kw):
        for i, k in enumerate(("p", "g", "m", "v", "m_scale", "v_scale")):
            setattr(t[0], k, 0x10000000 + i * 0x100000)
        t[0].p16, t[0].n, t[0].g_bf16, t[0].weight_decay = None, 100, 0, 0.0
        for k, v in kw.items():
            setattr(t[0], k, v)
        return L.qf_adamw_step(ctypes.byref(t), 1, bits, ctypes.byref(h), None)

    for k in ("p", "g", "m", "v"):
        assert sized(**{k: None}) == 1 and sized(**{k: 0x10000008}) == 3
    assert sized(p16=0x10000008) == 3
    assert sized(8, m_scale=None) == 1 and sized(8, v_scale=0x10000002) == 3
    assert sized(n=-1) == 2 and sized(n=1 << 31) == 2
    assert L.qf_adamw_step(None, 1, 32, ctypes.byref(h), None) == 1
    assert L.qf_adamw_step(ctypes.byref(t), 1, 32, None, None) == 1


def test_table_refusals():
    L = _lib.lib()
    t = (_lib.AdamwTensor * 3)()
    for i in range(3):
        for j, k in enumerate(("p", "g", "m", "v", "m_scale", "v_scale")):
            setattr(t[i], k, 0x10000000 + (8 * i + j) * 0x100000)
        t[i].n, t[i].g_bf16 = 5000 * i, i % 2
    need = L.qf_adamw_table_bytes(3)
    buf = (ctypes.c_uint8 * need)()
    plan = _lib.AdamwPlan()
    assert L.qf_adamw_table_bytes(0) == 0 and L.qf_adamw_table_bytes(-1) == 0 and need > 0
    assert L.qf_adamw_table(ctypes.byref(t), 3, 8, buf, need, ctypes.byref(plan)) == 0
    # the empty tensor is left out; 5000 and 10000 elements in workgroups of 2048
    assert list(plan.tensors) == [1, 1] and list(plan.workgroups) == [5, 3] and plan.capacity == 3
    assert L.qf_adamw_table(ctypes.byref(t), 3, 8, buf, need - 1, ctypes.byref(plan)) == 4
    assert L.qf_adamw_table(ctypes.byref(t), 3, 9, buf, need, ctypes.byref(plan)) == 7
    assert L.qf_adamw_table(None, 3, 8, buf, need, ctypes.byref(plan)) == 1
    assert L.qf_adamw_table(ctypes.byref(t), 3, 8, None, need, ctypes.byref(plan)) == 1
    assert L.qf_adamw_table(ctypes.byref(t), 3, 8, buf, need, None) == 1
    t[1].m = 0x10000008
    assert L.qf_adamw_table(ctypes.byref(t), 3, 8, buf, need, ctypes.byref(plan)) == 3
    h = _lib.AdamwHyper(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None, None, 0)
    d = ctypes.c_void_p(0x20000000)
    empty = _lib.AdamwPlan(8, 0, (0, 0), (0, 0))
    assert L.qf_adamw_step_table(ctypes.byref(empty), None, ctypes.byref(h), None) == 0
    assert L.qf_adamw_step_table(None, d, ctypes.byref(h), None) == 1
    assert L.qf_adamw_step_table(ctypes.byref(empty), d, None, None) == 1
    assert L.qf_adamw_step_table(ctypes.byref(_lib.AdamwPlan(8, 2, (1, 1), (1, 1))), None, ctypes.byref(h), None) == 1
    for bad in (_lib.AdamwPlan(7, 2, (1, 1), (1, 1)), _lib.AdamwPlan(8, 1, (1, 1), (1, 1)), _lib.AdamwPlan(8, 2, (-1, 1), (1, 1))):
        assert L.qf_adamw_step_table(ctypes.byref(bad), d, ctypes.byref(h), None) == 7
    assert L.qf_adamw_step_table(ctypes.byref(_lib.AdamwPlan(8, 2, (1, 1), (1, 1))), ctypes.c_void_p(0x20000004),
                                 ctypes.byref(h), None) == 3
    h.step = 0
    assert L.qf_adamw_step_table(ctypes.byref(empty), None, ctypes.byref(h), None) == 7


def test_binding_refusals():
    import fp4_fake_quant_amd as fq
    cpu = dict(p=torch.zeros(8), g=torch.zeros(8), m=torch.zeros(8), v=torch.zeros(8))
    with pytest.raises(TypeError):
        fq.AdamwBatch([cpu])                             # tensors of the host
    with pytest.raises(ValueError):
        fq.AdamwBatch([], state_bits=16)
    with pytest.raises(ValueError):
        fq.adamw_state(8, state_bits=4, device="cpu")
    s = fq.adamw_state(257, state_bits=8, device="cpu")
    assert s["m"].shape == (257,) and s["m_scale"].shape == (2,) and not s["v"].any()


def test_table_refuses_more_than_a_launch():
    """2^24 workgroups of 256 lanes are past the 32-bit size of a launch."""
    L = _lib.lib()
    most = (1 << 31) - 1                                     # elements of a tensor: 2^21 workgroups with fp32 states
    for bits, n, chunk in ((32, 8, 1024), (8, 16, 2048)):
        t = (_lib.AdamwTensor * n)()
        for i in range(n):
            for j, k in enumerate(("p", "g", "m", "v", "m_scale", "v_scale")):
                setattr(t[i], k, 0x10000000 + j * 0x100000)
            t[i].n = most
        buf = (ctypes.c_uint8 * L.qf_adamw_table_bytes(n))()
        plan = _lib.AdamwPlan()
        assert L.qf_adamw_table(ctypes.byref(t), n, bits, buf, len(buf), ctypes.byref(plan)) == 2
        t[n - 1].n = most - chunk
        assert L.qf_adamw_table(ctypes.byref(t), n, bits, buf, len(buf), ctypes.byref(plan)) == 0
        assert plan.workgroups[0] == (1 << 24) - 1
        t[0].g_bf16, t[n - 1].n = 1, most                    # a launch per gradient type
        assert L.qf_adamw_table(ctypes.byref(t), n, bits, buf, len(buf), ctypes.byref(plan)) == 0
