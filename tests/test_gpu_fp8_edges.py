"""Edges of the 8-bit operators on the GPU: what a NaN or an infinity reaches."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8
from tests.test_gpu_fp8 import codes_of, scales_of

pytestmark = pytest.mark.gpu


def gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def not_finite(t):
    return ~torch.isfinite(t.float()).cpu().numpy()


# ------------------------------------------ products of many tiles ----
# more tiles of outputs than workgroups, in tiles of 256 (at least 1024 of 128 x 128) and of 128
@pytest.mark.parametrize("E,N,K", [(45, 640, 648), (150, 256, 384), (70, 512, 520)])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("rows", [100, 300])
def test_wgrad_keeps_a_scale_in_its_row_or_column(E, N, K, value, rows):
    """A column of X and a row of dY of two groups: their weight gradients' column and row alone."""
    rng = np.random.default_rng(E + rows)
    n = E * rows
    plan = fq.qf_row_plan((torch.arange(n, device="cuda") % E).int(), E)
    offsets = [rows * e for e in range(E + 1)]
    blocks = fp8.panel_blocks(offsets)
    panels = fq.qf_fp8_panels(n, E)
    dc, xc = gpu(codes_of(rng, (panels, N, 128)), codes_of(rng, (panels, K, 128)))
    ds, xs = scales_of(rng, (panels, N)), scales_of(rng, (panels, K))
    last = {e: i for i, (e, _, _) in enumerate(blocks)}
    clean = fq.qf_gemm_fp8_wgrad(dc, *gpu(ds), xc, *gpu(xs), plan)
    assert not not_finite(clean).any()
    for of_x, e, at in ((True, 0, 5), (True, E // 2, K - 1), (False, 1, 3), (False, E // 2, N - 1), (True, E - 1, 0)):
        (xs if of_x else ds)[last[e], at] = value
    got = fq.qf_gemm_fp8_wgrad(dc, *gpu(ds), xc, *gpu(xs), plan)
    want = np.zeros((E, N, K), bool)
    want[0, :, 5] = want[E // 2, :, K - 1] = want[E - 1, :, 0] = True
    want[1, 3] = want[E // 2, N - 1] = True
    assert np.array_equal(not_finite(got), want)
    assert torch.equal(torch.where(torch.from_numpy(want).cuda(), clean, got), clean)


@pytest.mark.parametrize("M,N,K", [(4200, 4100, 144), (2000, 2052, 272)])
@pytest.mark.parametrize("grouped", [False, True])
def test_product_keeps_a_scale_in_its_row_or_tile(M, N, K, grouped):
    rng = np.random.default_rng(M)
    nb, E = fp8.blocks_of(K), 3 if grouped else 1
    plan = fq.qf_row_plan((torch.arange(M, device="cuda") * E // M).int(), E)
    xc, wc = gpu(codes_of(rng, (M, K)), codes_of(rng, (E, N, K)))
    xs, ws = scales_of(rng, (nb, M)), scales_of(rng, (E, fp8.blocks_of(N), nb))

    def run():
        a, b = gpu(xs, ws)
        return fq.qf_gemm_fp8_grouped(xc, a, wc, b, plan) if grouped else fq.qf_gemm_fp8(xc, a, wc[0], b[0])

    clean = run()
    xs[nb - 1, 17], xs[0, M - 5], ws[E - 1, 1, nb - 1], ws[0, -1, 0] = np.nan, np.inf, np.nan, np.inf
    got = run()
    off = plan.offsets.cpu().numpy()
    want = np.zeros((M, N), bool)
    want[[17, M - 5]] = True
    want[off[E - 1]:, 128:256] = True
    want[:off[1], N // 128 * 128:] = True
    assert np.array_equal(not_finite(got), want)
    assert torch.equal(torch.where(torch.from_numpy(want).cuda(), clean, got), clean)


# --------------------------------------------------- matrices of one row ----
@pytest.mark.parametrize("count", [1, 3, 130])
def test_tiles_of_single_rows(count):
    """Matrices of one row, whose stride says nothing: any that lie one after another."""
    x = torch.randn(count, 144, device="cuda").bfloat16()
    want = [fp8.quant_tiles(x[e:e + 1].float().cpu().numpy()) for e in range(count)]
    for v in (x[:, None], x.as_strided((count, 1, 144), (144, 1 << 20, 1)), x[None].transpose(0, 1)):
        c, s = fq.qf_quant_fp8_tiles(v)
        assert c.shape == (count, 1, 144) and s.shape == (count, 1, 2)
        for e in range(count):
            assert np.array_equal(c[e].cpu().numpy(), want[e][0]) and np.array_equal(s[e].cpu().numpy(), want[e][1])


def test_tiles_of_single_rows_apart():
    """Single rows with room between them: the row stride is the matrices'."""
    full = torch.full((5, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    full[:, :144] = torch.randn(5, 144, device="cuda").bfloat16()
    c, s = fq.qf_quant_fp8_tiles(full[:, None, :144])
    c2, s2 = fq.qf_quant_fp8_tiles(full[:, :144].contiguous()[:, None])
    assert torch.equal(c, c2) and torch.equal(s, s2)
    with pytest.raises(ValueError):
        fq.qf_quant_fp8_tiles(full.view(5, 10, 16)[:, :9].transpose(0, 1))


def test_tiles_without_rows():
    c, s, ct, st = fq.qf_quant_fp8_tiles(torch.empty(3, 0, 64, dtype=torch.bfloat16, device="cuda"), transpose=True)
    assert c.shape == (3, 0, 64) and s.shape == (3, 0, 1) and ct.shape == (3, 64, 0) and st.shape == (3, 1, 0)
