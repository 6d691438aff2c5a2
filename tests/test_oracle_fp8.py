"""Pins of the 8-bit oracle, and the refusals of the 8-bit and row entry points (CPU)."""

import ctypes

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from fp4_fake_quant_amd import _lib
from oracle import fp8, rows
from oracle import primitives as prim


def test_values_and_codes_against_torch():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, fp8.VALUES, equal_nan=True)
    y = prim.bf16_to_f32(np.arange(65536, dtype=np.uint16))
    y = np.clip(y[np.isfinite(y)], -448, 448)
    grid = fp8.VALUES[:127]
    mid = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    y = np.concatenate([y, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(500)), -mid])
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(y), want)


def test_codes_are_nearest():
    y = np.linspace(-448, 448, 20001).astype(np.float32)
    got = fp8.VALUES[fp8.encode(y)]
    best = np.abs(fp8.VALUES[np.r_[0:127, 128:255]][None, :] - y.astype(np.float64)[:, None]).min(1)
    assert np.array_equal(np.abs(got - y.astype(np.float64)), best)


def test_blocks():
    rng = np.random.default_rng(3)
    x = prim.bf16_to_f32(prim.f32_to_bf16((rng.standard_normal((300, 400)) * np.exp(rng.standard_normal((300, 1)))).astype(np.float32)))
    x[5] = 0
    x[7, :128] = 1e-31                                 # below 2^-100
    codes, scales = fp8.quant_rows(x)
    assert np.all(scales[:, 5] == 0) and scales[0, 7] == 0 and not codes[7, :128].any()
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * np.repeat(scales.T, 128, 1)[:, :400]) * (1 + 2.0 ** -20)
    keep = np.abs(x) >= 1e-30
    assert np.all((np.abs(fp8.dequant_rows(codes, scales) - x) <= step)[keep])
    # the largest element of a live block keeps its value up to the scale's rounding
    top = np.abs(fp8.dequant_rows(codes, scales))[:, :128].max(1)
    live = np.abs(x[:, :128]).max(1) > 1e-30
    assert np.allclose(top[live], np.abs(x[:, :128]).max(1)[live], rtol=2.0 ** -23)
    # tiles: one block over the tile's flattened elements; the transpose has the same values
    c, s = fp8.quant_tiles(x)
    ct, st = fp8.quant_tiles(np.ascontiguousarray(x.T))
    assert np.array_equal(c.T, ct) and np.array_equal(s.T, st)
    flat, fs = fp8.scale_of(np.abs(x[128:256, 256:384]).max())
    assert s[1, 2] == flat
    assert np.array_equal(c[128:256, 256:384], fp8.encode(x[128:256, 256:384] * fs))
    # panels: groups of 130, 0, 1 and 169 rows take 2, 0, 1 and 2
    off = [0, 130, 130, 131, 300]
    assert fp8.panel_blocks(off) == [(0, 0, 128), (0, 128, 2), (2, 130, 1), (3, 131, 128), (3, 259, 41)]
    pc, ps = fp8.quant_panels(x, off)
    back = fp8.dequant_panels(pc, ps)
    for i, (_, r, n) in enumerate(fp8.panel_blocks(off)):
        for col in (0, 399):
            c1, s1 = fp8.quant_rows(x[r:r + n, col][None, :])
            assert np.array_equal(pc[i, col, :n], c1[0]) and ps[i, col] == s1[0, 0]
        assert not back[i, n:].any()


def test_product_by_blocks():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((5, 300)).astype(np.float32), rng.standard_normal((200, 300)).astype(np.float32)
    xc, xs = fp8.quant_rows(x)
    wc, ws = fp8.quant_tiles(w)
    y, P = fp8.product(xc, xs, wc, ws)
    want = np.zeros((5, 200))
    for b in range(3):
        part = fp8.VALUES[xc[:, 128 * b:128 * b + 128]] @ fp8.VALUES[wc[:, 128 * b:128 * b + 128]].T
        want += part * xs[b][:, None] * np.repeat(ws[:, b], 128)[:200][None, :]
    assert np.allclose(y, want, rtol=1e-12, atol=1e-12 * P.max())


def test_block_sums_bound_catches():
    """Blocks in pairs that cancel, codes of 0, 1, 1.5 and 2: sums in fp32 pass; one term lost, sums held in bf16, or a
    block counted with another one's scale do not."""
    rng = np.random.default_rng(6)
    codes = np.array([0x00, 0x38, 0x3C, 0x40, 0xB8, 0xBC, 0xC0], np.uint8)
    M, N, pairs = 9, 11, 16
    pick = lambda *shape: fp8.VALUES[codes[rng.integers(0, 7, shape)]]
    a, b = pick(M, pairs, 128), pick(N, pairs, 128)
    x = np.concatenate([np.stack([a, -a], 2).reshape(M, -1), pick(M, 16)], 1)
    w = np.concatenate([np.stack([b, b], 2).reshape(N, -1), pick(N, 16)], 1)
    sx = np.exp(np.concatenate([np.repeat(rng.standard_normal((pairs, M)), 2, 0), rng.standard_normal((1, M))])).astype(np.float32)
    sw = np.exp(np.concatenate([np.repeat(rng.standard_normal(pairs), 2), rng.standard_normal(1)])).astype(np.float32)
    blocks = 2 * pairs + 1
    cut = [slice(128 * i, 128 * i + 128) for i in range(blocks)]
    P = np.stack([x[:, c] @ w[:, c].T for c in cut])
    t = P * (sx.astype(np.float64) * sw.astype(np.float64)[:, None])[:, :, None]
    y, S = t.sum(0), np.abs(t).sum(0)

    def fails(P, hold=lambda v: v, s=(sx * sw[:, None]).astype(np.float32)):
        acc = np.zeros((M, N), np.float32)
        for i in range(blocks):
            acc = hold((acc + (P[i].astype(np.float32) * s[i][:, None])).astype(np.float32))
        got = prim.bf16_to_f32(prim.f32_to_bf16(acc)).astype(np.float64)
        return np.mean(~(np.abs(got - y) <= fp8.block_sums_bound(y, S, 2 * blocks)))

    assert fails(P) == 0                               # (a product and a sum each rounded: two a block)
    bound = fp8.block_sums_bound(y, S, 2 * blocks)
    for k in (0, 128 * 5 + 77, x.shape[1] - 1):
        lost, term = P.copy(), np.outer(x[:, k], w[:, k])
        lost[k // 128] -= term
        # the rounded rest is off from y by the term, less its own bound, at most the term's 2^-8 more than y's
        seen = np.mean(np.abs(term * sx[k // 128][:, None] * float(sw[k // 128])) * (1 - 2.0 ** -7) > 2 * bound)
        assert fails(lost) >= seen > 0.3
    # (one result outside is enough for a test to fail)
    assert fails(P, hold=lambda v: prim.bf16_to_f32(prim.f32_to_bf16(v))) > 0
    assert fails(P, s=(sx * np.roll(sw, 1)[:, None]).astype(np.float32)) > 0


def test_gradients_against_differences():
    rng = np.random.default_rng(5)
    h, da = rng.standard_normal((4, 12)) * 3, rng.standard_normal((4, 6))
    g = fp8.swiglu_backward(h, da)
    for i in range(4):
        for j in range(12):
            d = np.zeros_like(h)
            d[i, j] = 1e-5
            diff = ((fp8.swiglu(h + d) - fp8.swiglu(h - d)) * da).sum() / 2e-5
            assert abs(diff - g[i, j]) < 1e-7 * max(1, abs(diff))
    ids = np.array([2, 0, -1, 1, 2, 2], np.int32)
    pos = fp8.positions(rows.plan(ids, 3)[1])
    R, w, dY = rng.standard_normal((6, 5)), rng.random((3, 2)), rng.standard_normal((3, 5))
    dR, dW, _ = fp8.combine_backward(dY, R, pos, w)
    for p in range(6):
        d = np.zeros_like(R)
        d[p, 3] = 1e-5
        diff = ((fp8.combine(R + d, pos, w)[0] - fp8.combine(R - d, pos, w)[0]) * dY).sum() / 2e-5
        assert abs(diff - dR[p, 3]) < 1e-8
    for t in range(3):
        for j in range(2):
            d = np.zeros_like(w)
            d[t, j] = 1e-5
            diff = ((fp8.combine(R, pos, w + d)[0] - fp8.combine(R, pos, w - d)[0]) * dY).sum() / 2e-5
            assert abs(diff - dW[t, j]) < 1e-8


def test_positions():
    ids = np.array([3, -1, 0, 3, 9, 0, 1], np.int32)
    order = rows.plan(ids, 4)[1]
    pos = fp8.positions(order)
    for i, p in enumerate(pos):
        assert (p < 0) == (ids[i] not in range(4)) and (p < 0 or order[p] == i)


# ------------------------------------------------------------------ refusals ----
A = 0x10000000                    # addresses that no call may touch
NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 7


def call(name, good, **bad):
    order = {"dispatch": "X ldx per pos n H out ldo", "combine": "R ldr pos w T k H Y ldy",
             "combine_backward": "dY lddy R ldr pos w T k H dR lddr dW",
             "quant_fp8": "x ldx rows cols pos per used codes ldc scales lds",
             "quant_fp8_panels": "x ldx rows cols order per offsets n_ids codes scales",
             "quant_fp8_tiles": "x ldx count rows cols codes scales codes_t scales_t",
             "swiglu_quant_fp8": "x ldx rows cols used codes ldc scales lds y ldy",
             "swiglu_backward": "x ldx da ldda rows cols used dh lddh",
             "gemm_fp8": "Xc ldx Xs ldxs Wc ldw Ws Y ldy M N K",
             "gemm_fp8_grouped": "Xc ldx Xs ldxs Wc ldw Ws offsets tiles n_ids Y ldy M N K",
             "gemm_fp8_wgrad": "Dc Ds Xc Xs offsets n_ids rows dW N K"}[name].split()
    v = dict(good, **bad)
    prefix = "qf_moe_" if name in ("dispatch", "combine", "combine_backward") else "qf_"
    f = getattr(_lib.lib(), prefix + name)
    args = [ctypes.c_void_p(v[o]) if t is ctypes.c_void_p else v[o] for o, t in zip(order, f.argtypes)]
    assert len(order) + 1 == len(f.argtypes)
    return f(*args, None)


DISPATCH = dict(X=A, ldx=64, per=2, pos=A, n=8, H=64, out=A, ldo=64)
COMBINE = dict(R=A, ldr=64, pos=A, w=A, T=4, k=2, H=64, Y=A, ldy=64, dY=A, lddy=64, dR=A, lddr=64, dW=A)
QUANT = dict(x=A, ldx=64, rows=8, cols=64, pos=0, per=1, used=0, codes=A, ldc=64, scales=A, lds=8, y=0, ldy=64)
GATE = dict(QUANT, ldx=128)
PANELS = dict(x=A, ldx=64, rows=8, cols=64, order=0, per=1, offsets=A, n_ids=3, codes=A, scales=A)
TILES = dict(x=A, ldx=64, count=2, rows=32, cols=64, codes=A, scales=A, codes_t=A, scales_t=A)
BACK = dict(x=A, ldx=128, da=A, ldda=64, rows=8, cols=64, used=0, dh=A, lddh=128)
GEMM = dict(Xc=A, ldx=64, Xs=A, ldxs=8, Wc=A, ldw=64, Ws=A, Y=A, ldy=32, M=8, N=32, K=64, offsets=A, tiles=A, n_ids=2)
WGRAD = dict(Dc=A, Ds=A, Xc=A, Xs=A, offsets=A, n_ids=2, rows=8, dW=A, N=32, K=64)


@pytest.mark.parametrize("name,good,bad,want", [
    ("dispatch", DISPATCH, dict(X=0), NULL), ("dispatch", DISPATCH, dict(pos=0), NULL), ("dispatch", DISPATCH, dict(out=0), NULL),
    ("dispatch", DISPATCH, dict(H=60), SHAPE), ("dispatch", DISPATCH, dict(H=0), SHAPE), ("dispatch", DISPATCH, dict(ldx=56), SHAPE),
    ("dispatch", DISPATCH, dict(ldo=56), SHAPE), ("dispatch", DISPATCH, dict(n=-1), SHAPE), ("dispatch", DISPATCH, dict(n=1 << 30), SHAPE),
    ("dispatch", DISPATCH, dict(H=1 << 22, ldx=1 << 22, ldo=1 << 22), SHAPE), ("dispatch", DISPATCH, dict(per=0), ARG),
    ("dispatch", DISPATCH, dict(X=A + 8), ALIGN), ("dispatch", DISPATCH, dict(ldx=68), ALIGN), ("dispatch", DISPATCH, dict(ldo=68), ALIGN),
    ("dispatch", DISPATCH, dict(pos=A + 2), ALIGN), ("dispatch", DISPATCH, dict(out=A + 8), ALIGN),
    ("combine", COMBINE, dict(R=0), NULL), ("combine", COMBINE, dict(pos=0), NULL), ("combine", COMBINE, dict(Y=0), NULL),
    ("combine", COMBINE, dict(k=0), ARG), ("combine", COMBINE, dict(T=-1), SHAPE), ("combine", COMBINE, dict(T=1 << 29, k=2), SHAPE),
    ("combine", COMBINE, dict(k=1 << 40), ARG), ("combine", COMBINE, dict(H=12), SHAPE), ("combine", COMBINE, dict(ldr=56), SHAPE),
    ("combine", COMBINE, dict(ldy=56), SHAPE), ("combine", COMBINE, dict(ldy=66), ALIGN), ("combine", COMBINE, dict(w=A + 2), ALIGN),
    ("combine", COMBINE, dict(R=A + 2), ALIGN), ("combine", COMBINE, dict(pos=A + 1), ALIGN),
    ("combine_backward", COMBINE, dict(dY=0), NULL), ("combine_backward", COMBINE, dict(R=0), NULL),
    ("combine_backward", COMBINE, dict(pos=0), NULL), ("combine_backward", COMBINE, dict(lddr=56), SHAPE),
    ("combine_backward", COMBINE, dict(ldr=56), SHAPE), ("combine_backward", COMBINE, dict(dW=A + 2), ALIGN),
    ("combine_backward", COMBINE, dict(dR=A + 2), ALIGN), ("combine_backward", COMBINE, dict(k=-3), ARG),
    ("quant_fp8", QUANT, dict(x=0), NULL), ("quant_fp8", QUANT, dict(codes=0), NULL), ("quant_fp8", QUANT, dict(scales=0), NULL),
    ("quant_fp8", QUANT, dict(cols=56), SHAPE), ("quant_fp8", QUANT, dict(cols=0), SHAPE), ("quant_fp8", QUANT, dict(lds=7), SHAPE),
    ("quant_fp8", QUANT, dict(ldc=48), SHAPE), ("quant_fp8", QUANT, dict(ldc=72), ALIGN), ("quant_fp8", QUANT, dict(ldx=66), ALIGN),
    ("quant_fp8", QUANT, dict(rows=-1), SHAPE), ("quant_fp8", QUANT, dict(pos=A, per=0), ARG), ("quant_fp8", QUANT, dict(codes=A + 8), ALIGN),
    ("quant_fp8", QUANT, dict(used=A + 2), ALIGN), ("quant_fp8", QUANT, dict(scales=A + 2), ALIGN),
    ("quant_fp8_panels", PANELS, dict(x=0), NULL), ("quant_fp8_panels", PANELS, dict(codes=0), NULL), ("quant_fp8_panels", PANELS, dict(cols=60), SHAPE),
    ("quant_fp8_panels", PANELS, dict(n_ids=0), ARG), ("quant_fp8_panels", PANELS, dict(n_ids=1025), ARG),
    ("quant_fp8_panels", PANELS, dict(offsets=0), ARG), ("quant_fp8_panels", PANELS, dict(order=A, per=0), ARG),
    ("quant_fp8_panels", PANELS, dict(offsets=A + 2), ALIGN), ("quant_fp8_panels", PANELS, dict(codes=A + 4), ALIGN),
    ("quant_fp8_tiles", TILES, dict(x=0), NULL), ("quant_fp8_tiles", TILES, dict(codes=0), ARG), ("quant_fp8_tiles", TILES, dict(scales_t=0), ARG),
    ("quant_fp8_tiles", TILES, dict(codes=0, scales=0, codes_t=0, scales_t=0), NULL), ("quant_fp8_tiles", TILES, dict(rows=24), SHAPE),
    ("quant_fp8_tiles", TILES, dict(cols=56), SHAPE), ("quant_fp8_tiles", TILES, dict(count=1025), ARG), ("quant_fp8_tiles", TILES, dict(count=-1), SHAPE),
    ("quant_fp8_tiles", TILES, dict(codes_t=A + 8), ALIGN), ("quant_fp8_tiles", TILES, dict(rows=1 << 22), SHAPE),
    ("swiglu_quant_fp8", GATE, dict(ldx=112), SHAPE), ("swiglu_quant_fp8", GATE, dict(x=0), NULL), ("swiglu_quant_fp8", GATE, dict(y=A, ldy=56), SHAPE),
    ("swiglu_quant_fp8", GATE, dict(y=A + 2), ALIGN), ("swiglu_quant_fp8", GATE, dict(y=A, ldy=68), ALIGN),
    ("swiglu_backward", BACK, dict(x=0), NULL), ("swiglu_backward", BACK, dict(da=0), NULL), ("swiglu_backward", BACK, dict(dh=0), NULL),
    ("swiglu_backward", BACK, dict(ldx=120), SHAPE), ("swiglu_backward", BACK, dict(lddh=120), SHAPE), ("swiglu_backward", BACK, dict(cols=12), SHAPE),
    ("swiglu_backward", BACK, dict(ldda=68), ALIGN), ("swiglu_backward", BACK, dict(used=A + 1), ALIGN),
    *[(n, GEMM, b, w) for n in ("gemm_fp8", "gemm_fp8_grouped") for b, w in (
        (dict(Xc=0), NULL), (dict(Xs=0), NULL), (dict(Wc=0), NULL), (dict(Ws=0), NULL), (dict(Y=0), NULL), (dict(K=56), SHAPE), (dict(K=0), SHAPE),
        (dict(ldx=48), SHAPE), (dict(ldw=48), SHAPE), (dict(ldxs=7), SHAPE), (dict(ldy=31), SHAPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE),
        (dict(N=1 << 22, ldy=1 << 22), SHAPE), (dict(ldx=72), ALIGN), (dict(ldw=72), ALIGN), (dict(Xc=A + 8), ALIGN), (dict(Wc=A + 4), ALIGN),
        (dict(Y=A + 1), ALIGN), (dict(Xs=A + 2), ALIGN), (dict(M=(1 << 30) - 1, ldxs=1 << 30), SHAPE))],
    ("gemm_fp8_grouped", GEMM, dict(offsets=0), NULL), ("gemm_fp8_grouped", GEMM, dict(tiles=0), NULL), ("gemm_fp8_grouped", GEMM, dict(n_ids=0), ARG),
    ("gemm_fp8_grouped", GEMM, dict(n_ids=1025), ARG), ("gemm_fp8_grouped", GEMM, dict(tiles=A + 4), ALIGN),
    ("gemm_fp8_wgrad", WGRAD, dict(Dc=0), NULL), ("gemm_fp8_wgrad", WGRAD, dict(dW=0), NULL), ("gemm_fp8_wgrad", WGRAD, dict(N=30), SHAPE),
    ("gemm_fp8_wgrad", WGRAD, dict(K=60), SHAPE), ("gemm_fp8_wgrad", WGRAD, dict(offsets=0), ARG), ("gemm_fp8_wgrad", WGRAD, dict(dW=A + 8), ALIGN),
    ("gemm_fp8_wgrad", WGRAD, dict(rows=-1), SHAPE), ("gemm_fp8_wgrad", WGRAD, dict(N=1 << 21, K=1 << 21), SHAPE),
])
def test_refusals(name, good, bad, want):
    assert call(name, good, **bad) == want


@pytest.mark.parametrize("name,good,none", [
    ("dispatch", DISPATCH, dict(n=0, X=0)), ("combine", COMBINE, dict(T=0, R=0)), ("combine_backward", COMBINE, dict(T=0)),
    ("combine_backward", COMBINE, dict(dR=0, dW=0)), ("quant_fp8", QUANT, dict(rows=0)), ("quant_fp8_panels", PANELS, dict(rows=0)),
    ("quant_fp8_tiles", TILES, dict(count=0)), ("quant_fp8_tiles", TILES, dict(rows=0)), ("swiglu_quant_fp8", GATE, dict(rows=0)),
    ("swiglu_backward", BACK, dict(rows=0)), ("gemm_fp8", GEMM, dict(M=0)), ("gemm_fp8", GEMM, dict(N=0)), ("gemm_fp8_grouped", GEMM, dict(M=0)),
    ("gemm_fp8_wgrad", WGRAD, dict(N=0)), ("gemm_fp8_wgrad", WGRAD, dict(K=0))])
def test_nothing_to_do(name, good, none):
    assert call(name, good, **none) == 0


def test_panels_bound():
    f = _lib.lib().qf_fp8_panels
    assert f(0, 1) == 0 and f(1, 1) == 1 and f(129, 1) == 2 and f(129, 5) == 7 and f(3, 1024) == 4
    assert f(-1, 1) == 0 and f(1, 0) == 0 and f(1, 1025) == 0 and f(1 << 30, 1) == 0
    rng = np.random.default_rng(0)
    for _ in range(200):
        n, e = int(rng.integers(0, 2000)), int(rng.integers(1, 60))
        off = rows.plan(rng.integers(-1, e, n).astype(np.int32), e)[0]
        assert len(fp8.panel_blocks(off)) <= f(n, e)


def test_binding_strides_and_counts():
    """Scales that share one row of memory have a row stride below their rows, which the entry points
    refuse; a count that does not fit the C argument is refused before it wraps around."""
    assert fq._scales(torch.empty(3, 8), "scales", 3, 8) == 8
    assert fq._scales(torch.empty(3, 12)[:, :8], "scales", 3, 8) == 12
    assert fq._scales(torch.empty(1, 8), "scales", 1, 8) >= 8
    shared = fq._scales(torch.empty(1, 8).expand(3, 8), "scales", 3, 8)
    assert shared < 8
    assert call("quant_fp8", QUANT, lds=shared) == SHAPE
    assert call("gemm_fp8", GEMM, ldxs=shared) == SHAPE and call("gemm_fp8_grouped", GEMM, ldxs=shared) == SHAPE
    fq._x_rows(1, 5, 1000)
    for bad in (0, -1, 1 << 62, (1 << 64) + 1):
        with pytest.raises(ValueError):
            fq._x_rows(1, 5, bad)
