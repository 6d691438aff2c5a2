"""CPU pins of the row plan and adapter oracles, and the host checks of qf_row_plan and
qf_lora_apply."""

import ctypes

import numpy as np
import pytest
import torch

from fp4_fake_quant_amd import _lib
from oracle import rows


def P(v):
    return ctypes.c_void_p(v) if v else None


@pytest.mark.parametrize("n,n_ids", [(0, 3), (1, 1), (33, 1), (200, 7), (500, 300)])
def test_plan_row_by_row(n, n_ids):
    rng = np.random.default_rng(n)
    ids = rng.integers(-1, n_ids + 1, n)
    offsets, order, tiles = rows.plan(ids, n_ids)
    kept = int(offsets[-1])
    assert kept == sum(0 <= i < n_ids for i in ids) and np.all(order[kept:] == -1)
    assert sorted(order[:kept].tolist()) == [i for i in range(n) if 0 <= ids[i] < n_ids]
    pairs = [(ids[i], i) for i in order[:kept]]
    assert pairs == sorted(pairs)
    seen = []
    for e, f in tiles:
        if e >= 0:
            c = min(rows.TILE, offsets[e + 1] - f)
            assert c > 0 and np.all(ids[order[f:f + c]] == e)
            seen += list(range(f, f + c))
    assert seen == list(range(kept))
    assert len(tiles) == _lib.lib().qf_row_plan_tiles(n, n_ids)


def test_apply_row_by_row():
    rng = np.random.default_rng(0)
    X, A, B = rng.standard_normal((4, 16)), rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 5, 2))
    ids, scale = np.array([0, 2, -1, 1, 2, 3, 0, 0]), np.array([0.5, -1.0, 2.0])
    Y = rng.standard_normal((8, 5))
    out, P_, _ = rows.apply(X, A, B, ids, Y, scale, 2)
    for i, e in enumerate(ids):
        want = Y[i] + (scale[e] * B[e] @ (A[e] @ X[i // 2]) if 0 <= e < 3 else 0)
        assert np.allclose(out[i], want, rtol=1e-13, atol=1e-13)
        assert (P_[i] > 0).all() == (0 <= e < 3)


def test_row_plan_refusals():
    L = _lib.lib()
    ids, off, order, tiles, ws = (P(0x10000000 + k * 0x100000) for k in range(5))
    ok = dict(ids=ids, n=100, n_ids=8, off=off, order=order, tiles=tiles, ws=None, wsb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return L.qf_row_plan(a["ids"], a["n"], a["n_ids"], a["off"], a["order"], a["tiles"], a["ws"], a["wsb"], None)
    assert call(n=-1) == 2 and call(n=1 << 30) == 2
    assert call(n_ids=0) == 7 and call(n_ids=1025) == 7
    for k in ("ids", "off", "order", "tiles"):
        assert call(**{k: None}) == 1
        assert call(**{k: P(0x10000002)}) == 3
    assert call(tiles=P(0x10000004)) == 3
    need = L.qf_row_plan_workspace(100000, 8)
    assert need > 0 and L.qf_row_plan_workspace(4096, 8) == 0
    assert call(n=100000) == 4 and call(n=100000, ws=ws, wsb=need - 1) == 4
    assert call(n=100000, ws=P(0x10000004), wsb=need) == 3
    assert L.qf_row_plan_workspace(5, 0) == 0 and L.qf_row_plan_tiles(-1, 4) == 0 and L.qf_row_plan_tiles(5, 1025) == 0


def test_lora_apply_refusals():
    L = _lib.lib()
    X, A, B, S, ids, Y, ws, off, order, tiles = (P(0x10000000 + k * 0x100000) for k in range(10))
    ok = dict(X=X, ldx=64, per=1, A=A, B=B, S=S, E=4, ids=ids, Y=Y, ldy=40, rows=10, N=40, K=64, r=8, ws=ws, wsb=1 << 30,
              off=off, order=order, tiles=tiles, n_ids=4)

    def call(planned=False, **kw):
        a = dict(ok, **kw)
        tail = (a["Y"], a["ldy"], a["rows"], a["N"], a["K"], a["r"], a["ws"], a["wsb"], None)
        head = (a["X"], a["ldx"], a["per"], a["A"], a["B"], a["S"], a["E"])
        if planned:
            return L.qf_lora_apply_planned(*head, a["off"], a["order"], a["tiles"], a["n_ids"], *tail)
        return L.qf_lora_apply(*head, a["ids"], *tail)

    for planned in (False, True):
        c = lambda **kw: call(planned, **kw)  # noqa: E731
        assert c(rows=0) == 0
        assert c(r=0) == 7 and c(r=129) == 7 and c(E=0) == 7 and c(E=1025) == 7 and c(per=0) == 7
        assert c(rows=-1) == 2 and c(rows=1 << 24) == 2 and c(K=0) == 2 and c(K=60) == 2 and c(N=0) == 2
        assert c(ldx=56) == 2 and c(ldy=39) == 2 and c(K=1 << 22, ldx=1 << 22) == 2
        for k in ("X", "A", "B", "Y"):
            assert c(**{k: None}) == 1
        assert c(X=P(0x10000008)) == 3 and c(A=P(0x10000008)) == 3 and c(ldx=68) == 3 and c(B=P(0x10000001)) == 3
        assert c(Y=P(0x10000001)) == 3 and c(S=P(0x10000002)) == 3
        rows = 10 if planned else 1000                     # few rows without a plan need no workspace
        need = L.qf_lora_apply_workspace(rows, 64, 8, 4, int(planned))
        assert need > 0 and c(rows=rows, ws=None) == 4 and c(rows=rows, wsb=need - 1) == 4
        assert c(rows=rows, ws=P(0x10000008)) == 3
    for r, few in ((8, 256), (16, 256), (17, 240), (32, 128), (64, 64), (65, 0), (128, 0)):
        assert L.qf_lora_apply_workspace(few, 64, r, 4, 0) == 0 and L.qf_lora_apply_workspace(few + 1, 64, r, 4, 0) > 0
    assert call(ids=None) == 1 and call(ids=P(0x10000002)) == 3
    for k in ("off", "order", "tiles"):
        assert call(True, **{k: None}) == 1 and call(True, **{k: P(0x10000002)}) == 3
    assert call(True, n_ids=5) == 7 and call(True, n_ids=0) == 7
    assert L.qf_lora_apply_workspace(10, 60, 8, 4, 0) == 0 and L.qf_lora_apply_workspace(10, 64, 200, 4, 0) == 0


def test_rows_per_x_has_no_upper_limit():
    """X of one row serves any number of rows of Y."""
    L = _lib.lib()
    X, A, B, ids, Y, off, order, tiles = (P(0x10000000 + k * 0x100000) for k in range(8))
    for per in (1, 1 << 24, (1 << 24) + 1, 1 << 40, (1 << 63) - 1):
        assert L.qf_lora_apply(X, 64, per, A, B, None, 4, ids, Y, 40, 0, 40, 64, 8, None, 0, None) == 0
        assert L.qf_lora_apply_planned(X, 64, per, A, B, None, 4, off, order, tiles, 4, Y, 40, 0, 40, 64, 8, None, 0, None) == 0


def test_binding_refuses_host_tensors():
    import fp4_fake_quant_amd as fq
    with pytest.raises(TypeError):
        fq.qf_row_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        fq.qf_row_plan(torch.zeros(4, dtype=torch.int64), 2)
    z = torch.zeros(1, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fq.qf_lora_apply(z.view(1, 1), z.view(1, 1, 1), z.view(1, 1, 1), torch.zeros(1, dtype=torch.int32), z.view(1, 1))


def test_binding_refuses_a_plan_for_ids():
    """A plan's arrays must not reach the entry point that takes ids."""
    import torch
    import fp4_fake_quant_amd as fq
    X, A = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    B, Y = torch.zeros((2, 40, 8), dtype=torch.bfloat16), torch.zeros((4, 40), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="qf_lora_apply_planned"):
        fq.qf_lora_apply(X, A, B, fq.RowPlan(4, 2, "cpu"), Y)
    with pytest.raises(TypeError, match="RowPlan"):
        fq.qf_lora_apply_planned(X, A, B, torch.zeros(4, dtype=torch.int32), Y)
