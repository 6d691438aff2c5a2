"""8-bit blocks of 128, the gated activation and the products on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8, rows
from oracle import primitives as prim
from tests.gpu_util import dev, host
from tests.test_gpu_moe_rows import bf, ids_of, plan_of, strided

pytestmark = pytest.mark.gpu
f32 = prim.bf16_to_f32


def spread(rng, shape):
    """bf16 rows and columns of different sizes, with zeros and a row of tiny values."""
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal((shape[0], 1))) * np.exp(rng.standard_normal((1, shape[1])))
    x[rng.random(shape) < 0.02] = 0
    if shape[0] > 3:
        x[2] = 0
        x[3] *= 1e-34
    return prim.f32_to_bf16(x.astype(np.float32))


def padded(shape, pad, fill):
    full = torch.full((shape[0], shape[1] + pad), fill, dtype=torch.uint8, device="cuda")
    return full, full[:, :shape[1]]


def within(got, want, bound):
    err = np.abs(got.astype(np.float64) - want)
    bad = np.argwhere(~(err <= bound))
    i = tuple(bad[0]) if len(bad) else None
    assert i is None, f"{len(bad)} outside, first {i}: {got[i]!r} for {want[i]!r}, bound {bound[i]!r}"


def same(got, want):
    return np.array_equal(got.cpu().numpy(), want)


# ---------------------------------------------------------------- quantizers ----
ROWS = [(1, 16), (1, 4096), (3, 48), (7, 128), (31, 144), (32, 256), (33, 2064), (64, 4096), (130, 1040), (1000, 272), (2100, 16)]


@pytest.mark.parametrize("n,cols", ROWS)
def test_quant_rows(n, cols):
    rng = np.random.default_rng(n + cols)
    x = spread(rng, (n, cols))
    _, xd = strided(x, 8)
    codes, scales = fp8.quant_rows(f32(x))
    c, s = fq.qf_quant_fp8(xd)
    assert same(c, codes) and same(s, scales)
    cfull, c = padded((n, cols), 32, 0x55)
    sfull = torch.full((scales.shape[0], n + 3), 7.0, device="cuda")
    fq.qf_quant_fp8(xd, codes=c, scales=sfull[:, :n])
    assert same(c, codes) and same(sfull[:, :n], scales)
    assert bool((cfull[:, cols:] == 0x55).all()) and bool((sfull[:, n:] == 7).all())


def test_every_bf16_value():
    """Blocks that hold every finite bf16 against a few largest magnitudes."""
    v = np.arange(65536, dtype=np.uint16)
    v = v[np.isfinite(f32(v))]
    x = np.zeros((4, -(-v.size // 120) * 128), np.uint16)
    for i, top in enumerate((0x7F7F, 0x3F80, 0x0D80, 0x43E1)):
        keep = v[(v & 0x7FFF) <= top]
        pad = np.zeros(-(-keep.size // 120) * 120, np.uint16)
        pad[:keep.size] = keep
        part = np.concatenate([pad.reshape(-1, 120), np.full((pad.size // 120, 8), top, np.uint16)], 1).reshape(-1)
        x[i, :part.size] = part
    codes, scales = fp8.quant_rows(f32(x))
    c, s = fq.qf_quant_fp8(dev(x))
    assert same(c, codes) and same(s, scales)


@pytest.mark.parametrize("T,k,cols,E,none", [(5, 2, 160, 3, 0.2), (64, 8, 512, 16, 0.1), (300, 3, 272, 40, 0.0), (9, 4, 128, 1024, 1.1)])
def test_quant_rows_in_expert_order(T, k, cols, E, none):
    rng = np.random.default_rng(T)
    plan, offsets, order = plan_of(ids_of(rng, T, k, E, none), E)
    n, used = T * k, int(offsets[-1])
    x = spread(rng, (T, cols))
    cfull, c = padded((n, cols), 16, 0x33)
    s = torch.full((fp8.blocks_of(cols), n), 5.0, device="cuda")
    fq.qf_quant_fp8(dev(x), plan=plan, rows_per_x=k, codes=c, scales=s)
    codes, scales = fp8.quant_rows(f32(x)[order[:used] // k])
    assert same(c[:used], codes) and same(s[:, :used], scales)
    assert bool((c[used:] == 0x33).all()) and bool((s[:, used:] == 5).all())
    # rows that are in that order already: the rest is left alone
    y = spread(rng, (n, cols))
    c.fill_(0x44)
    s.fill_(6.0)
    fq.qf_quant_fp8(dev(y), plan=plan, codes=c, scales=s)
    codes, scales = fp8.quant_rows(f32(y)[:used])
    assert same(c[:used], codes) and same(s[:, :used], scales)
    assert bool((c[used:] == 0x44).all()) and bool((s[:, used:] == 6).all())


@pytest.mark.parametrize("T,k,cols,E,none", [(1, 1, 8, 1, 0.0), (5, 2, 160, 3, 0.2), (64, 8, 520, 16, 0.1), (300, 3, 272, 40, 0.0), (100, 4, 136, 1000, 0.1),
                                             (9, 4, 128, 1024, 1.1), (513, 2, 128, 2, 0.0)])
def test_quant_panels(T, k, cols, E, none):
    rng = np.random.default_rng(T + 1)
    plan, offsets, order = plan_of(ids_of(rng, T, k, E, none), E)
    n, used = T * k, int(offsets[-1])
    for gather in (False, True):
        x = spread(rng, (T if gather else n, cols))
        if not gather:
            x[used:] = 0x7FC0
        _, xd = strided(x, 8)
        panels = fq.qf_fp8_panels(n, E)
        c = torch.full((panels, cols, 128), 0x11, dtype=torch.uint8, device="cuda")
        s = torch.full((panels, cols), 3.0, device="cuda")
        fq.qf_quant_fp8_panels(xd, plan=plan, rows_per_x=k if gather else None, codes=c, scales=s)
        codes, scales = fp8.quant_panels(f32(x)[order[:used] // k] if gather else f32(x), offsets)
        m = codes.shape[0]
        assert same(c[:m], codes) and same(s[:m], scales)
        assert bool((c[m:] == 0x11).all()) and bool((s[m:] == 3).all())


@pytest.mark.parametrize("n,cols", [(1, 8), (127, 136), (128, 128), (300, 264)])
def test_quant_panels_of_all_rows(n, cols):
    x = spread(np.random.default_rng(n), (n, cols))
    c, s = fq.qf_quant_fp8_panels(dev(x))
    codes, scales = fp8.quant_panels(f32(x), [0, n])
    assert same(c, codes) and same(s, scales)


@pytest.mark.parametrize("count,n,cols", [(1, 16, 16), (3, 128, 128), (2, 144, 272), (1, 400, 1040), (5, 32, 528)])
def test_quant_tiles(count, n, cols):
    rng = np.random.default_rng(n)
    x = np.stack([spread(rng, (n, cols)) for _ in range(count)])
    full = torch.full((count, n, cols + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    full[:, :, :cols] = dev(x.reshape(-1, cols)).view(count, n, cols)
    for xd in (full[:, :, :cols], full[:, :, :cols].contiguous()):
        c, s, ct, st = fq.qf_quant_fp8_tiles(xd, transpose=True)
        for e in range(count):
            codes, scales = fp8.quant_tiles(f32(x[e]))
            assert same(c[e], codes) and same(s[e], scales) and same(ct[e], codes.T) and same(st[e], scales.T)
    c2, s2 = fq.qf_quant_fp8_tiles(full[0, :, :cols])
    assert torch.equal(c2, c[0]) and torch.equal(s2, s[0])


def test_tiles_of_odd_rows():
    x = spread(np.random.default_rng(1), (131, 48))
    c, s = fq.qf_quant_fp8_tiles(dev(x))
    codes, scales = fp8.quant_tiles(f32(x))
    assert same(c, codes) and same(s, scales)
    with pytest.raises(fq.QFError):
        fq.qf_quant_fp8_tiles(dev(x), transpose=True)


def test_quant_non_finite():
    """A NaN or an infinity makes its block's scale NaN and leaves the others alone."""
    rng = np.random.default_rng(2)
    x = bf(rng, (40, 384))
    x[3, 130], x[17, 0], x[39, 383] = 0x7F80, 0xFFC1, 0xFF80
    good = x.copy()
    good[[3, 17, 39], [130, 0, 383]] = 0
    c, s = fq.qf_quant_fp8(dev(x))
    codes, scales = fp8.quant_rows(f32(good))
    want = np.zeros((3, 40), bool)
    want[[1, 0, 2], [3, 17, 39]] = True
    assert np.array_equal(np.isnan(s.cpu().numpy()), want) and np.array_equal(s.cpu().numpy()[~want], scales[~want])
    mask = np.repeat(want.T, 128, 1)
    assert np.array_equal(c.cpu().numpy()[~mask], codes[~mask])
    _, s = fq.qf_quant_fp8_panels(dev(x))
    assert np.array_equal(np.flatnonzero(np.isnan(s.cpu().numpy()[0])), [0, 130, 383])
    _, s, _, st = fq.qf_quant_fp8_tiles(dev(x[:32]), transpose=True)
    assert np.array_equal(np.isnan(s.cpu().numpy()), [[True, True, False]]) and torch.equal(s.t().isnan(), st.isnan())


# ---------------------------------------------------------- gated activation ----
GATED = [(1, 16), (3, 128), (33, 144), (65, 2064), (200, 512)]


def gate_input(rng, n, cols):
    h = rng.standard_normal((n, 2 * cols)) * np.exp(rng.standard_normal((n, 1)))
    h[:, :cols] *= 4
    h[:, 0], h[:, 1] = rng.choice([-95, -88, -60, 60, 95, 300, -300], n), 0
    return prim.f32_to_bf16(h.astype(np.float32))


def act_error(h, a):
    """How far the held fp32 product may be off."""
    return 16 * 2.0 ** -24 * np.abs(a) + 2.0 ** -119 * np.abs(h[:, h.shape[1] // 2:])


@pytest.mark.parametrize("n,cols", GATED)
def test_swiglu_quant(n, cols):
    rng = np.random.default_rng(n + cols)
    h = gate_input(rng, n, cols)
    _, hd = strided(h, 16)
    yfull, y = strided(bf(rng, (n, cols)), 8)
    c, s = fq.qf_swiglu_quant_fp8(hd, y=y)
    hf = f32(h).astype(np.float64)
    a = fp8.swiglu(hf)
    off = act_error(hf, a)
    within(f32(host(y)), a, 2.0 ** -8 * np.abs(a) + (1 + 2.0 ** -8) * off + 2.0 ** -134)
    assert bool(yfull[:, cols:].isnan().all())
    c, s = c.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    for b in range(s.shape[0]):
        part = slice(128 * b, 128 * b + 128)
        top = np.abs(a[:, part]).max(1)
        within(s[b], top / 448, 20 * 2.0 ** -24 * top / 448)
    deq = fp8.dequant_rows(c, s)
    # half a step of the code, and what the scaled value was off by
    step = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * np.repeat(s.T, 128, 1)[:, :cols]) * (1 + 2.0 ** -10)
    within(deq, a, step + off)
    c2, s2 = fq.qf_swiglu_quant_fp8(hd)
    assert same(c2, c) and np.array_equal(s2.cpu().numpy(), s.astype(np.float32))


def test_gate_at_every_value():
    """The held product at every finite bf16 gate, read off the scale of a block with one element."""
    v = np.arange(65536, dtype=np.uint16)
    v = v[np.isfinite(f32(v))]
    h = np.zeros((v.size, 32), np.uint16)
    h[:, 0], h[:, 16] = v, prim.f32_to_bf16(np.float32([1.5]))[0]
    _, s = fq.qf_swiglu_quant_fp8(dev(h))
    a = np.abs(fp8.swiglu(f32(h).astype(np.float64))[:, 0])
    top = s.cpu().numpy()[0].astype(np.float64) * 448
    # a, the division and the scale's own rounding; values that the block drops, or past the range of fp32
    keep = (a >= 2.0 ** -99) & (a < 2.0 ** 127)
    within(top[keep], a[keep], 16 * 2.0 ** -24 * a[keep] + 2.0 ** -119 * 1.5 + 2.0 ** -23 * a[keep])
    assert np.all(top[a < 2.0 ** -101] == 0)


@pytest.mark.parametrize("n,cols", GATED + [(5, 24)])
def test_swiglu_backward(n, cols):
    rng = np.random.default_rng(n + cols + 1)
    h, da = gate_input(rng, n, cols), bf(rng, (n, cols))
    _, hd = strided(h, 8)
    _, dd = strided(da, 8)
    ofull, out = strided(bf(rng, (n, 2 * cols)), 8)
    got = f32(host(fq.qf_swiglu_backward(hd, dd, dh=out))).astype(np.float64)
    hf, df = f32(h).astype(np.float64), f32(da).astype(np.float64)
    g, u = hf[:, :cols], hf[:, cols:]
    want = fp8.swiglu_backward(hf, df)
    off = 32 * 2.0 ** -24 * np.concatenate([np.abs(df * u) * (1 + np.abs(g)), np.abs(df * g)], 1)
    within(got, want, 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * off + 2.0 ** -119 * np.abs(np.concatenate([df * u, df], 1)))
    assert bool(ofull[:, 2 * cols:].isnan().all())


def test_gate_leaves_rows_behind_the_last_group():
    rng = np.random.default_rng(7)
    plan, offsets, _ = plan_of(ids_of(rng, 40, 2, 5, 0.4), 5)
    used = int(offsets[-1])
    h, da = gate_input(rng, 80, 64), bf(rng, (80, 64))
    c = torch.full((80, 64), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 80), 4.0, device="cuda")
    y = torch.full((80, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    fq.qf_swiglu_quant_fp8(dev(h), plan=plan, y=y, codes=c, scales=s)
    c2, s2 = fq.qf_swiglu_quant_fp8(dev(h))
    assert torch.equal(c[:used], c2[:used]) and torch.equal(s[:, :used], s2[:, :used])
    assert bool((c[used:] == 9).all()) and bool((s[:, used:] == 4).all()) and bool((y[used:] == 2).all())
    dh = torch.full((80, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.qf_swiglu_backward(dev(h), dev(da), plan=plan, dh=dh)
    assert torch.equal(dh[:used], fq.qf_swiglu_backward(dev(h), dev(da))[:used]) and bool((dh[used:] == 3).all())


# ------------------------------------------------------------------ products ----
def codes_of(rng, shape):
    """Every code but the NaNs, with a share of zeros."""
    c = rng.integers(0, 127, shape) + 128 * rng.integers(0, 2, shape)
    return np.where(rng.random(shape) < 0.05, 0, c).astype(np.uint8)


def scales_of(rng, shape):
    return np.exp(rng.standard_normal(shape)).astype(np.float32)


def put(codes, pad):
    """codes on the GPU in longer rows, NaN codes behind each row's end."""
    full = torch.full((codes.shape[0], codes.shape[1] + pad), 0x7F, dtype=torch.uint8, device="cuda")
    full[:, :codes.shape[1]] = torch.from_numpy(codes).cuda()
    return full[:, :codes.shape[1]]


def check_product(got, y, P, L):
    within(f32(host(got)), y, fp8.product_bound(y, P, L))


GEMM = [(1, 1, 16), (1, 5, 128), (3, 17, 144), (16, 16, 1040), (17, 48, 256), (33, 130, 272), (64, 128, 128), (65, 129, 4112), (128, 128, 256),
        (129, 260, 400), (257, 300, 640), (300, 1000, 1040), (513, 770, 2064), (1, 6144, 512), (7, 2000, 4096), (61, 3000, 1040), (256, 256, 112),
        (1024, 520, 96), (1500, 1300, 272), (2, 100, 14336), (200, 4096, 144)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm(M, N, K):
    rng = np.random.default_rng(M + N + K)
    xc, wc = codes_of(rng, (M, K)), codes_of(rng, (N, K))
    nb = fp8.blocks_of(K)
    xs, ws = scales_of(rng, (nb, M)), scales_of(rng, (fp8.blocks_of(N), nb))
    y, P = fp8.product(xc, xs, wc, ws)
    t = lambda a: torch.from_numpy(a).cuda()
    Y = fq.qf_gemm_fp8(t(xc), t(xs), t(wc), t(ws))
    check_product(Y, y, P, K)
    assert torch.equal(fq.qf_gemm_fp8(t(xc), t(xs), t(wc), t(ws)), Y)
    # long rows with NaN codes behind them, strided scales, an output inside a larger one
    xsf = torch.full((nb, M + 5), float("nan"), device="cuda")
    xsf[:, :M] = t(xs)
    full = torch.full((M + 1, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.qf_gemm_fp8(put(xc, 48), xsf[:, :M], put(wc, 16), t(ws), Y=full[:M, :N])
    assert torch.equal(full[:M, :N], Y) and bool((full[M:] == 7).all()) and bool((full[:, N:] == 7).all())


@pytest.mark.parametrize("M,N,K", [(4200, 4100, 144), (4097, 4104, 16), (2100, 8200, 400)])
def test_gemm_large_tiles(M, N, K):
    test_gemm(M, N, K)


def test_gemm_far_rows():
    """Codes and results whose offsets pass 2^31."""
    rng = np.random.default_rng(3)
    M, N, K, ld = 40000, 264, 48, 1 << 16
    x, y = torch.zeros((M, ld), dtype=torch.uint8, device="cuda"), torch.zeros((M, ld), dtype=torch.bfloat16, device="cuda")
    xc = torch.from_numpy(codes_of(rng, (M, K))).cuda()
    x[:, :K] = xc
    xs, wc, ws = (torch.from_numpy(v).cuda() for v in (scales_of(rng, (1, M)), codes_of(rng, (N, K)), scales_of(rng, (3, 1))))
    want = fq.qf_gemm_fp8(xc, xs, wc, ws)
    fq.qf_gemm_fp8(x[:, :K], xs, wc, ws, Y=y[:, :N])
    assert torch.equal(y[:, :N], want)
    last = slice(M - 300, M)
    Y, P = fp8.product(xc[last].cpu().numpy(), xs[:, last].cpu().numpy(), wc.cpu().numpy(), ws.cpu().numpy())
    check_product(want[last], Y, P, K)
    q = fq.qf_quant_fp8(y[:, :N // 16 * 16])
    assert torch.equal(q[0], fq.qf_quant_fp8(want[:, :N // 16 * 16].contiguous())[0])


@pytest.mark.parametrize("M", [3, 40, 200])
def test_gemm_nan_stays_in_its_rows(M):
    rng = np.random.default_rng(M)
    N, K = 300, 400
    xc, wc = codes_of(rng, (M, K)), codes_of(rng, (N, K))
    xs, ws = scales_of(rng, (4, M)), scales_of(rng, (3, 4))
    xs[2, M - 2], ws[1, 3] = np.nan, np.nan
    t = lambda a: torch.from_numpy(a).cuda()
    bad = ~torch.isfinite(fq.qf_gemm_fp8(t(xc), t(xs), t(wc), t(ws)).float()).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[M - 2], want[:, 128:256] = True, True
    assert np.array_equal(bad, want)


GROUPED = [(1, 1, 1, 8, 16, 0.0), (5, 2, 3, 40, 160, 0.2), (61, 8, 128, 136, 256, 0.0), (64, 8, 16, 520, 272, 0.1), (300, 3, 5, 300, 400, 0.0),
           (100, 4, 1000, 72, 144, 0.1), (9, 4, 1024, 24, 32, 1.1), (700, 2, 2, 264, 640, 0.0), (1, 8, 8, 1536, 2048, 0.0), (400, 8, 6, 384, 128, 0.5),
           (31, 1, 1, 1000, 1040, 0.0), (1500, 2, 5, 4700, 144, 0.1), (2000, 2, 70, 2100, 272, 0.0), (26000, 1, 1024, 40, 32, 0.0),
           (3000, 1, 100, 264, 48, 0.3)]


@pytest.mark.parametrize("T,k,E,N,K,none", GROUPED)
def test_gemm_grouped(T, k, E, N, K, none):
    rng = np.random.default_rng(T + N)
    plan, offsets, _ = plan_of(ids_of(rng, T, k, E, none), E)
    n, used, nb = T * k, int(offsets[-1]), fp8.blocks_of(K)
    xc, wc = codes_of(rng, (n, K)), codes_of(rng, (E, N, K))
    xs, ws = scales_of(rng, (nb, n)), scales_of(rng, (E, fp8.blocks_of(N), nb))
    xc[used:], xs[:, used:] = 0x7F, np.nan
    full = torch.full((n, N + 4), 7.0, dtype=torch.bfloat16, device="cuda")
    t = lambda a: torch.from_numpy(a).cuda()
    fq.qf_gemm_fp8_grouped(put(xc, 16), t(xs), t(wc), t(ws), plan, Y=full[:, :N])
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            y, P = fp8.product(xc[lo:hi], xs[:, lo:hi], wc[e], ws[e])
            check_product(full[lo:hi, :N], y, P, K)
    assert bool((full[used:] == 7).all()) and bool((full[:, N:] == 7).all())


@pytest.mark.parametrize("T", [6, 900])
def test_gemm_grouped_one_group_is_the_dense_product(T):
    rng = np.random.default_rng(T)
    plan, _, _ = plan_of(np.zeros(T, np.int32), 1)
    t = lambda a: torch.from_numpy(a).cuda()
    xc, wc, xs, ws = codes_of(rng, (T, 272)), codes_of(rng, (200, 272)), scales_of(rng, (3, T)), scales_of(rng, (2, 3))
    y, P = fp8.product(xc, xs, wc, ws)
    check_product(fq.qf_gemm_fp8(t(xc), t(xs), t(wc), t(ws)), y, P, 272)
    check_product(fq.qf_gemm_fp8_grouped(t(xc), t(xs), t(wc)[None], t(ws)[None], plan), y, P, 272)


WGRAD = [(1, 1, 1, 8, 8, 0.0), (5, 2, 3, 40, 160, 0.2), (64, 8, 16, 136, 264, 0.1), (300, 3, 5, 520, 272, 0.0), (100, 4, 100, 72, 48, 0.1), (9, 4, 1024, 8, 16, 1.1),
         (700, 2, 2, 264, 128, 0.0), (1000, 2, 45, 640, 648, 0.1), (40, 1, 70, 512, 520, 0.1)]


@pytest.mark.parametrize("T,k,E,N,K,none", WGRAD)
def test_wgrad(T, k, E, N, K, none):
    rng = np.random.default_rng(T + N + 3)
    plan, offsets, _ = plan_of(ids_of(rng, T, k, E, none), E)
    panels = fq.qf_fp8_panels(T * k, E)
    dc, xc = codes_of(rng, (panels, N, 128)), codes_of(rng, (panels, K, 128))
    ds, xs = scales_of(rng, (panels, N)), scales_of(rng, (panels, K))
    blocks = fp8.panel_blocks(offsets)
    dc[len(blocks):], ds[len(blocks):], xs[len(blocks):] = 0x7F, np.nan, np.nan
    t = lambda a: torch.from_numpy(a).cuda()
    args = t(dc), t(ds), t(xc), t(xs)
    got = fq.qf_gemm_fp8_wgrad(*args, plan)
    m = len(blocks)
    D, X = fp8.dequant_panels(dc[:m], ds[:m]), fp8.dequant_panels(xc[:m], xs[:m])
    DM, XM = fp8.panels_magnitudes(dc[:m], ds[:m]), fp8.panels_magnitudes(xc[:m], xs[:m])
    for e in range(E):
        at = [i for i, b in enumerate(blocks) if b[0] == e]
        y, P = np.zeros((N, K)), np.zeros((N, K))
        for i in at:
            y += D[i].T @ X[i]
            P += DM[i].T @ XM[i]
        check_product(got[e], y, P, 128 * len(at))
    assert torch.equal(fq.qf_gemm_fp8_wgrad(*args, plan, dW=torch.full_like(got, 7)), got)


def test_wgrad_of_all_rows():
    rng = np.random.default_rng(8)
    x, d = bf(rng, (300, 72)), bf(rng, (300, 40))
    got = fq.qf_gemm_fp8_wgrad(*fq.qf_quant_fp8_panels(dev(d)), *fq.qf_quant_fp8_panels(dev(x)))
    qd, qx = (fp8.quant_panels(f32(v), [0, 300]) for v in (d, x))
    D, X = (fp8.dequant_panels(*q).reshape(384, -1) for q in (qd, qx))
    DM, XM = (fp8.panels_magnitudes(*q).reshape(384, -1) for q in (qd, qx))
    check_product(got, D.T @ X, DM.T @ XM, 384)
    assert got.shape == (40, 72)


def test_no_rows():
    z = lambda *s, t=torch.uint8: torch.empty(s, dtype=t, device="cuda")
    plan = fq.qf_row_plan(z(0, t=torch.int32), 3, positions=True)
    dW = fq.qf_gemm_fp8_wgrad(z(0, 16, 128), z(0, 16, t=torch.float32), z(0, 8, 128), z(0, 8, t=torch.float32), plan)
    assert dW.shape == (3, 16, 8) and not dW.any()
    assert fq.qf_gemm_fp8_grouped(z(0, 32), z(1, 0, t=torch.float32), z(3, 16, 32), z(3, 1, 1, t=torch.float32), plan).shape == (0, 16)
    c, s = fq.qf_quant_fp8(z(0, 32, t=torch.bfloat16), plan=plan, rows_per_x=1)
    assert c.shape == (0, 32) and s.shape == (1, 0)
    assert fq.qf_moe_combine(z(0, 32, t=torch.bfloat16), plan, k=4).shape == (0, 32)


def test_another_stream():
    """Calls follow torch's current stream."""
    rng = np.random.default_rng(11)
    x, w = dev(bf(rng, (200, 512))), dev(bf(rng, (256, 512)))
    want = fq.qf_gemm_fp8(*fq.qf_quant_fp8(x), *fq.qf_quant_fp8_tiles(w))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = big @ big * 1e-2
        late = torch.where(big[:200, :512].isnan() | True, x, x)      # ready only behind the products
        got = fq.qf_gemm_fp8(*fq.qf_quant_fp8(late), *fq.qf_quant_fp8_tiles(w))
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")
    f, b = torch.float32, torch.bfloat16
    plan = fq.qf_row_plan(z(8, t=torch.int32), 2, positions=True)
    X, Xs, W, Ws = z(8, 64), z(1, 8, t=f), z(32, 64), z(1, 1, t=f)
    bare = fq.qf_row_plan(z(8, t=torch.int32), 2)
    for call in (lambda: fq.qf_quant_fp8(z(8, 64, t=b), rows_per_x=1), lambda: fq.qf_quant_fp8(z(8, 64, t=b), plan=bare, rows_per_x=1),
                 lambda: fq.qf_quant_fp8(z(7, 64, t=b), plan=plan),
                 lambda: fq.qf_quant_fp8(z(8, 64, t=b), plan=plan, rows_per_x=2), lambda: fq.qf_quant_fp8(z(8, 64, t=b), codes=z(8, 63)),
                 lambda: fq.qf_quant_fp8(z(8, 64, t=b), scales=z(8, 1, t=f)), lambda: fq.qf_quant_fp8_panels(z(7, 64, t=b), plan=plan),
                 lambda: fq.qf_quant_fp8_panels(z(8, 64, t=b), codes=z(2, 64, 128), plan=plan), lambda: fq.qf_quant_fp8_tiles(z(8, t=b)),
                 lambda: fq.qf_quant_fp8_tiles(z(2, 32, 64, t=b).transpose(0, 1)), lambda: fq.qf_quant_fp8_tiles(z(32, 64, t=b), codes_t=z(64, 32)),
                 lambda: fq.qf_swiglu_quant_fp8(z(8, 63, t=b)), lambda: fq.qf_swiglu_quant_fp8(z(7, 64, t=b), plan=plan),
                 lambda: fq.qf_swiglu_quant_fp8(z(8, 64, t=b), y=z(8, 64, t=b)), lambda: fq.qf_swiglu_backward(z(8, 64, t=b), z(8, 64, t=b)),
                 lambda: fq.qf_gemm_fp8(X, Xs, z(32, 48), Ws), lambda: fq.qf_gemm_fp8(X, z(1, 7, t=f), W, Ws), lambda: fq.qf_gemm_fp8(X, Xs, W, z(1, 2, t=f)),
                 lambda: fq.qf_gemm_fp8(X, Xs, W, Ws, Y=z(8, 33, t=b)), lambda: fq.qf_gemm_fp8_grouped(X, Xs, W, Ws, plan),
                 lambda: fq.qf_gemm_fp8_grouped(X, Xs, z(3, 32, 64), z(3, 1, 1, t=f), plan),
                 lambda: fq.qf_gemm_fp8_grouped(z(7, 64), z(1, 7, t=f), z(2, 32, 64), z(2, 1, 1, t=f), plan),
                 lambda: fq.qf_gemm_fp8_wgrad(z(1, 8, 128), z(1, 8, t=f), z(1, 8, 128), z(1, 8, t=f), plan),
                 lambda: fq.qf_gemm_fp8_wgrad(z(1, 8, 128), z(1, 8, t=f), z(1, 8, 128), z(1, 7, t=f)),
                 lambda: fq.qf_gemm_fp8_wgrad(z(1, 8, 128), z(1, 8, t=f), z(1, 8, 128), z(1, 8, t=f), dW=z(8, 8, t=f))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.qf_quant_fp8(z(8, 64, t=f)), lambda: fq.qf_gemm_fp8(X.view(torch.int8), Xs, W, Ws), lambda: fq.qf_gemm_fp8(X.cpu(), Xs, W, Ws)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fq.qf_quant_fp8(z(8, 24, t=b)), lambda: fq.qf_gemm_fp8(z(8, 24), Xs, z(32, 24), Ws)):
        with pytest.raises(fq.QFError):
            call()
