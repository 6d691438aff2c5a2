"""Rows into expert order and back on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8, rows
from oracle import primitives as prim
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu
f32 = prim.bf16_to_f32


def bf(rng, shape, scale=1.0):
    return prim.f32_to_bf16((rng.standard_normal(shape) * scale).astype(np.float32))


def strided(bits, pad, fill=float("nan")):
    """bits on the GPU in rows that are `pad` elements longer."""
    full = torch.full((bits.shape[0], bits.shape[1] + pad), fill, dtype=torch.bfloat16, device="cuda")
    view = full[:, :bits.shape[1]]
    view.copy_(dev(bits))
    return full, view


def ids_of(rng, T, k, E, none):
    ids = rng.integers(0, E, T * k).astype(np.int32)
    return np.where(rng.random(T * k) < none, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], T * k), ids).astype(np.int32)


def plan_of(ids, E):
    plan = fq.qf_row_plan(torch.from_numpy(ids).cuda(), E, positions=True)
    offsets, order, tiles = rows.plan(ids, E)
    assert np.array_equal(plan.order.cpu().numpy(), order) and np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.positions.cpu().numpy(), fp8.positions(order))
    assert np.array_equal(plan.tiles.cpu().numpy(), tiles)
    return plan, offsets, order


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 512, 2049, 16384, 16385, 131073])
@pytest.mark.parametrize("E", [1, 3, 128, 1024])
def test_positions(n, E):
    rng = np.random.default_rng(n + E)
    plan_of(ids_of(rng, n, 1, E, 0.2), E)


def test_positions_into_a_kept_plan():
    rng = np.random.default_rng(0)
    a, b = (torch.from_numpy(ids_of(rng, 50, 2, 7, 0.1)).cuda() for _ in range(2))
    plan = fq.qf_row_plan(a, 7, positions=True)
    want = fq.qf_row_plan(b, 7, positions=True)
    fq.qf_row_plan(b, 7, plan=plan)
    assert torch.equal(plan.positions, want.positions) and torch.equal(plan.order, want.order)
    with pytest.raises(ValueError):
        fq.qf_row_plan(b, 7, plan=fq.qf_row_plan(a, 7), positions=True)


CASES = [(1, 1, 8, 1, 0.0), (1, 8, 16, 4, 0.0), (3, 2, 40, 2, 0.3), (7, 8, 2048, 128, 0.0), (64, 6, 136, 5, 0.1), (33, 3, 1032, 9, 0.5),
         (257, 1, 4096, 3, 0.05), (100, 32, 72, 200, 0.9), (40, 8, 264, 16, 1.1), (500, 5, 24, 1024, 0.0), (5, 40, 512, 3, 0.1)]


@pytest.mark.parametrize("T,k,H,E,none", CASES)
def test_dispatch(T, k, H, E, none):
    rng = np.random.default_rng(T + H)
    ids = ids_of(rng, T, k, E, none)
    plan, _, order = plan_of(ids, E)
    for per in (1, k, T * k):                                        # rows of x that share one
        x = bf(rng, (-(-T * k // per), H))
        full, view = strided(x, 8 if H % 16 else 0)
        ofull, out = strided(bf(rng, (T * k, H)), 16)
        before = host(out)
        assert fq.qf_moe_dispatch(view, plan, per, out=out) is out
        got = host(out)
        live = order >= 0
        assert np.array_equal(got[live], x[order[live] // per])
        assert np.array_equal(got[~live], before[~live]) and bool(ofull[:, H:].isnan().all())


@pytest.mark.parametrize("n,per", [(10, 4), (100, 33), (70, 16), (33, 17), (5, 1000)])
def test_dispatch_of_a_last_row_with_fewer(n, per):
    rng = np.random.default_rng(n)
    plan, _, order = plan_of(ids_of(rng, n, 1, 3, 0.2), 3)
    x, live = bf(rng, (-(-n // per), 144)), order >= 0
    out = torch.full((n, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.qf_moe_dispatch(dev(x), plan, per, out=out)
    assert np.array_equal(host(out)[live], x[order[live] // per]) and bool((out[torch.from_numpy(~live).cuda()] == 7).all())
    c, s = fq.qf_quant_fp8(dev(x), plan=plan, rows_per_x=per)
    codes, scales = fp8.quant_rows(f32(x)[order[live] // per])
    assert np.array_equal(c.cpu().numpy()[live], codes) and np.array_equal(s.cpu().numpy()[:, live], scales)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,H,E,none", CASES)
def test_combine(T, k, H, E, none, weighted):
    rng = np.random.default_rng(T + H + 1)
    plan, offsets, order = plan_of(ids_of(rng, T, k, E, none), E)
    R = bf(rng, (T * k, H))
    R[offsets[-1]:] = 0x7FC0                                         # what lies behind the last group is not read
    _, r = strided(R, 8)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else np.ones((T, k), np.float32)
    pos = fp8.positions(order)
    wd = torch.from_numpy(w.copy())
    wd.view(-1)[torch.from_numpy(pos < 0)] = float("nan")            # a row in no group adds nothing, whatever its weight
    yfull, Y = strided(bf(rng, (T, H)), 8)
    got = host(fq.qf_moe_combine(r, plan, wd.cuda() if weighted else None, k=k, Y=Y))
    y, P = fp8.combine(f32(R), pos, w)
    err = np.abs(f32(got).astype(np.float64) - y)
    assert np.all(err <= 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * fp8.gamma(k) * P)
    assert bool(yfull[:, H:].isnan().all())
    assert np.array_equal(host(fq.qf_moe_combine(r, plan, wd.cuda() if weighted else None, k=k)), got)


@pytest.mark.parametrize("T,k,H,E,none", CASES)
def test_combine_backward(T, k, H, E, none):
    rng = np.random.default_rng(T + H + 2)
    plan, offsets, order = plan_of(ids_of(rng, T, k, E, none), E)
    R, dY = bf(rng, (T * k, H)), bf(rng, (T, H))
    R[offsets[-1]:] = 0x7FC0
    w = rng.standard_normal((T, k)).astype(np.float32)
    wd = torch.from_numpy(w).cuda()
    pos = fp8.positions(order)
    dR, dW, P = fp8.combine_backward(f32(dY), f32(R), pos, w)
    _, r = strided(R, 8)
    _, dy = strided(dY, 24)
    ofull, out = strided(bf(rng, (T * k, H)), 8)
    before = host(out)
    got, gw = fq.qf_moe_combine_backward(dy, r, plan, wd, d_rows=out)
    n = offsets[-1]
    got_h = host(got)
    assert np.all(np.abs(f32(got_h[:n]).astype(np.float64) - dR[:n]) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(dR[:n]))
    assert np.array_equal(got_h[n:], before[n:]) and bool(ofull[:, H:].isnan().all())
    gw_h = gw.cpu().numpy()
    assert np.all(np.abs(gw_h - dW) <= fp8.gamma(H) * P) and np.all(gw_h.reshape(-1)[pos < 0] == 0)
    only_r, none_w = fq.qf_moe_combine_backward(dy, None, plan, wd, want=(True, False))
    none_r, only_w = fq.qf_moe_combine_backward(dy, r, plan, wd, want=(False, True))
    assert none_w is None and none_r is None and np.array_equal(host(only_r)[:n], got_h[:n]) and torch.equal(only_w, gw)
    ones, _ = fq.qf_moe_combine_backward(dy, r, plan, k=k, want=(True, False))
    live = order >= 0
    assert np.array_equal(host(ones)[live], dY[order[live] // k])


def test_infinities_stay_in_their_rows():
    rng = np.random.default_rng(9)
    T, k, H, E = 6, 2, 64, 3
    ids = ids_of(rng, T, k, E, 0.0)
    plan, _, order = plan_of(ids, E)
    pos = fp8.positions(order)
    R = bf(rng, (T * k, H))
    R[pos[4], 5], R[pos[7], 6] = 0x7F80, 0x7FC0
    w = torch.rand(T, k, device="cuda") + 0.5
    y = fq.qf_moe_combine(dev(R), plan, w).float().cpu().numpy()
    bad = ~np.isfinite(y)
    assert bad.sum() == 2 and np.isposinf(y[2, 5]) and np.isnan(y[3, 6])
    dr, dw = fq.qf_moe_combine_backward(dev(bf(rng, (T, H))), dev(R), plan, w)
    assert bool(torch.isfinite(dr).all())
    assert sorted(np.flatnonzero(~np.isfinite(dw.cpu().numpy().reshape(-1)))) == [4, 7]


def test_far_rows():
    """Row offsets past 2^31 elements."""
    T, k, H = 2, 1, 8
    ld = 1 << 22
    big = torch.empty((520, ld), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((520,), 0, dtype=torch.int32, device="cuda")
    plan = fq.qf_row_plan(ids, 1, positions=True)
    x = torch.randn(520, H, device="cuda").bfloat16()
    out = big[:, :H]
    fq.qf_moe_dispatch(x, plan, out=out)
    assert torch.equal(out, x)
    assert torch.equal(fq.qf_moe_combine(out, plan, k=1), x)
    dr, dw = fq.qf_moe_combine_backward(x, out, plan, k=1, d_rows=out)
    assert torch.equal(dr, x)


def test_refusals():
    ids = torch.zeros(8, dtype=torch.int32, device="cuda")
    plan, bare = fq.qf_row_plan(ids, 2, positions=True), fq.qf_row_plan(ids, 2)
    x, r, w = (torch.zeros(s, dtype=t, device="cuda") for s, t in (((4, 16), torch.bfloat16), ((8, 16), torch.bfloat16), ((4, 2), torch.float32)))
    for f in (lambda: fq.qf_moe_dispatch(x, plan, 3), lambda: fq.qf_moe_dispatch(x, plan, 0), lambda: fq.qf_moe_dispatch(x, plan, 2, out=x),
              lambda: fq.qf_moe_combine(r, bare, w), lambda: fq.qf_moe_dispatch(x, bare, 2), lambda: fq.qf_moe_combine(r, plan), lambda: fq.qf_moe_combine(r, plan, k=3),
              lambda: fq.qf_moe_combine(x, plan, w), lambda: fq.qf_moe_combine(r, plan, w.t()), lambda: fq.qf_moe_combine(r, plan, w, k=4),
              lambda: fq.qf_moe_combine(r, plan, w, Y=r), lambda: fq.qf_moe_combine_backward(r, r, plan, w),
              lambda: fq.qf_moe_combine_backward(x, x, plan, w), lambda: fq.qf_moe_combine_backward(x, r, plan, w, d_rows=x),
              lambda: fq.qf_moe_combine_backward(x, r, plan, w, d_weights=w.double())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fq.qf_moe_dispatch(x.float(), plan, 2), lambda: fq.qf_moe_dispatch(x, ids, 2), lambda: fq.qf_moe_combine(r.cpu(), plan, w)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(fq.QFError):
        fq.qf_moe_dispatch(x[:, :12], plan, 2)
