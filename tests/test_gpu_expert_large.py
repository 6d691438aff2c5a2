"""Row and 8-bit operators at sizes whose outputs are stored past the caches (another form of each kernel):
the same bits as in pieces that are not, or as the formula where it leaves no choice.  Panels in larger buffers."""

import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8

pytestmark = pytest.mark.gpu
MIB = 1 << 20


def randn(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()


def plan_of(seed, n, E):
    ids = torch.randint(-1, E, (n,), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(seed))
    plan = fq.qf_row_plan(ids, E, positions=True)
    return plan, int(plan.offsets[E]), plan.order.long()


def cuts(n, piece):
    return [slice(a, min(a + piece, n)) for a in range(0, n, piece)]


def test_dispatch_and_gradients():
    T, k, H = 9001, 3, 4400
    plan, n, order = plan_of(1, T * k, 7)
    assert T * k * H * 2 > 224 * MIB
    x, w = randn(2, T, H), torch.rand(T, k, device="cuda")
    out = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.qf_moe_dispatch(x, plan, k, out=out)
    assert torch.equal(out[:n], x[order[:n] // k]) and bool((out[n:] == 7).all())
    dr = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    dr, dw = fq.qf_moe_combine_backward(x, out, plan, w, d_rows=dr)
    assert torch.equal(dr[:n], (w.view(-1)[order[:n], None] * x[order[:n] // k].float()).bfloat16()) and bool((dr[n:] == 7).all())
    some = order[:n:97]
    rows = x[some // k].double()
    want, P = (rows * rows).sum(1), (rows * rows).sum(1)
    assert bool(((dw.view(-1)[some] - want).abs() <= fp8.gamma(H) * P).all())
    assert bool((dw.view(-1)[plan.positions < 0] == 0).all()) and int((plan.positions < 0).sum()) == T * k - n


def test_combine():
    T, k, H = 8300, 3, 4104
    assert T * H * 2 > 64 * MIB
    plan, n, order = plan_of(3, T * k, 5)
    r, w = randn(4, T * k, H), torch.randn(T, k, device="cuda")
    got = fq.qf_moe_combine(r, plan, w)
    place = plan.positions.view(T, k)
    some = torch.arange(0, T, 13, device="cuda")
    p = place[some].long()
    term = torch.where((p >= 0)[..., None], w[some].double()[..., None] * r[p.clamp(min=0)].double(), 0.0)
    y, P = term.sum(1), term.abs().sum(1)
    # k multiply-adds of fp32, then half a step of bf16
    assert bool(((got[some].double() - y).abs() <= 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * fp8.gamma(k) * P).all())


def test_quantization():
    n, cols = 17000, 4112
    assert n * cols > 64 * MIB
    x = randn(5, n, cols)
    codes, scales = fq.qf_quant_fp8(x)
    for s in cuts(n, 6000):
        c, v = fq.qf_quant_fp8(x[s])
        assert torch.equal(codes[s], c) and torch.equal(scales[:, s], v)
    pc, ps = fq.qf_quant_fp8_panels(x)
    for s in cuts(n, 6016):
        c, v = fq.qf_quant_fp8_panels(x[s])
        b = slice(s.start // 128, s.start // 128 + c.shape[0])
        assert torch.equal(pc[b], c) and torch.equal(ps[b], v)
    # rows into the order of groups
    plan, m, order = plan_of(6, 3 * n, 9)
    gc, gs = fq.qf_quant_fp8(x, plan=plan, rows_per_x=3)
    assert torch.equal(gc[:m], codes[order[:m] // 3]) and torch.equal(gs[:, :m], scales[:, order[:m] // 3])


def test_gate():
    n, cols = 16500, 4112
    assert n * cols > 64 * MIB
    h, da = randn(7, n, 2 * cols), randn(8, n, cols)
    y = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    codes, scales = fq.qf_swiglu_quant_fp8(h, y=y)
    dh = fq.qf_swiglu_backward(h, da)
    for s in cuts(n, 6000):
        part = torch.empty(h[s].shape[0], cols, dtype=torch.bfloat16, device="cuda")
        c, v = fq.qf_swiglu_quant_fp8(h[s], y=part)
        assert torch.equal(codes[s], c) and torch.equal(scales[:, s], v) and torch.equal(y[s], part)
        assert torch.equal(dh[s], fq.qf_swiglu_backward(h[s], da[s]))


def test_products():
    M, N, K = 28711, 4104, 272
    assert M * N * 2 > 224 * MIB
    xc, xs = fq.qf_quant_fp8(randn(9, M, K))
    wc, ws = fq.qf_quant_fp8_tiles(randn(10, 1, N, K))
    full = torch.full((M + 1, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = fq.qf_gemm_fp8(xc, xs, wc[0], ws[0], Y=full[:M, :N])
    assert bool((full[M:] == 7).all()) and bool((full[:, N:] == 7).all())
    for s in cuts(M, 9000):
        assert torch.equal(Y[s], fq.qf_gemm_fp8(xc[s], xs[:, s], wc[0], ws[0]))
    plan = fq.qf_row_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(fq.qf_gemm_fp8_grouped(xc, xs, wc, ws, plan), Y)


def test_weight_gradients():
    n, N, K = 300, 10840, 10848
    assert N * K * 2 > 224 * MIB
    dc, ds = fq.qf_quant_fp8_panels(randn(11, n, N))
    xc, xs = fq.qf_quant_fp8_panels(randn(12, n, K))
    dW = fq.qf_gemm_fp8_wgrad(dc, ds, xc, xs)
    for s in cuts(N, 4000):
        assert torch.equal(dW[s], fq.qf_gemm_fp8_wgrad(dc[:, s].contiguous(), ds[:, s].contiguous(), xc, xs))


@pytest.mark.parametrize("n,E", [(1, 1), (130, 1), (300, 4)])
def test_more_panels_than_needed(n, E):
    """Panels in larger buffers, what lies behind the last (NaN) neither written nor read."""
    ids = torch.zeros(n, dtype=torch.int32, device="cuda") if E == 1 else (torch.arange(n, device="cuda") % E).int()
    plan = fq.qf_row_plan(ids, E, positions=True)
    need = fq.qf_fp8_panels(n, E)
    d, x = randn(13, n, 48), randn(14, n, 80)
    panels, want = [], []
    for t, extra in ((d, 1), (x, 3)):
        codes = torch.full((need + extra, t.shape[1], 128), 0x7F, dtype=torch.uint8, device="cuda")
        scales = torch.full((need + extra, t.shape[1]), float("nan"), device="cuda")
        panels += fq.qf_quant_fp8_panels(t, plan=plan, codes=codes, scales=scales)
        want += fq.qf_quant_fp8_panels(t, plan=plan)
        assert bool((codes[need:] == 0x7F).all()) and bool(scales[need:].isnan().all())
    dW = fq.qf_gemm_fp8_wgrad(*panels, plan)
    assert torch.equal(dW, fq.qf_gemm_fp8_wgrad(*want, plan)) and not bool(dW.isnan().any())
    with pytest.raises(ValueError):
        fq.qf_gemm_fp8_wgrad(panels[0][:need - 1], *panels[1:], plan)
    with pytest.raises(ValueError):
        fq.qf_quant_fp8_panels(d, plan=plan, codes=panels[0][:need - 1])
    with pytest.raises(ValueError):
        fq.qf_gemm_fp8_wgrad(*panels)
