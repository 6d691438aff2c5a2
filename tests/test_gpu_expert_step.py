"""A mixture's experts in 8 bits, forward and backward, as a training step runs them: routing, row
plan, dispatch with quantization, gate/up product, gated activation, down product, combine; then the
gradients of the routing weights, the tokens and the experts' weights, AdamW on the latter.  Every
step against the oracle from the operands that it was given, eager and captured."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import fp8
from oracle import primitives as prim
from tests.gpu_util import dev, host
from tests.test_gpu_fp8 import act_error, check_product, within
from tests.test_gpu_moe_rows import bf

pytestmark = pytest.mark.gpu
f32 = prim.bf16_to_f32


class Step:
    """The step's tensors, kept so that a captured graph finds them where they were."""

    def __init__(self, T, k, E, H, I, seed, masked):
        rng = np.random.default_rng(seed)
        self.T, self.k, self.E, self.H, self.I = T, k, E, H, I
        self.x, self.dy = dev(bf(rng, (T, H))), dev(bf(rng, (T, H)))
        self.logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
        if masked:                                   # tokens that nobody takes, an expert that takes nobody
            self.logits[:2] = -float("inf")
            self.logits[:, 1] = -float("inf")
        self.w1 = dev(bf(rng, (E * 2 * I, H), H ** -0.5)).view(E, 2 * I, H)
        self.w2 = dev(bf(rng, (E * H, I), I ** -0.5)).view(E, H, I)
        self.p1, self.p2 = self.w1.float(), self.w2.float()
        n, z = T * k, lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
        self.h, self.a, self.r, self.dr, self.dh, self.da, self.dxs = (z(n, c) for c in (2 * I, I, H, H, 2 * I, I, H))
        self.dw1, self.dw2 = z(E, 2 * I, H), z(E, H, I)
        self.plan = None
        self.batch = None

    def forward(self):
        s = self
        s.idx, s.w = fq.qf_moe_route(s.logits, s.k)
        s.plan = fq.qf_row_plan(s.idx, s.E, plan=s.plan, positions=True)
        s.q1, s.q2 = fq.qf_quant_fp8_tiles(s.w1, transpose=True), fq.qf_quant_fp8_tiles(s.w2, transpose=True)
        s.qx = fq.qf_quant_fp8(s.x, plan=s.plan, rows_per_x=s.k)
        fq.qf_gemm_fp8_grouped(*s.qx, *s.q1[:2], s.plan, Y=s.h)
        s.qa = fq.qf_swiglu_quant_fp8(s.h, plan=s.plan, y=s.a)
        fq.qf_gemm_fp8_grouped(*s.qa, *s.q2[:2], s.plan, Y=s.r)
        s.y = fq.qf_moe_combine(s.r, s.plan, s.w)

    def backward(self):
        s = self
        _, s.dw = fq.qf_moe_combine_backward(s.dy, s.r, s.plan, s.w, d_rows=s.dr)
        s.dlogits = fq.qf_moe_route_backward(s.logits, s.idx, s.dw)
        s.qdr = fq.qf_quant_fp8(s.dr, plan=s.plan)
        fq.qf_gemm_fp8_grouped(*s.qdr, *s.q2[2:], s.plan, Y=s.da)
        fq.qf_swiglu_backward(s.h, s.da, plan=s.plan, dh=s.dh)
        s.qdh = fq.qf_quant_fp8(s.dh, plan=s.plan)
        fq.qf_gemm_fp8_grouped(*s.qdh, *s.q1[2:], s.plan, Y=s.dxs)
        s.dx = fq.qf_moe_combine(s.dxs, s.plan, k=s.k)
        s.pdr, s.pa = fq.qf_quant_fp8_panels(s.dr, plan=s.plan), fq.qf_quant_fp8_panels(s.a, plan=s.plan)
        s.pdh, s.px = fq.qf_quant_fp8_panels(s.dh, plan=s.plan), fq.qf_quant_fp8_panels(s.x, plan=s.plan, rows_per_x=s.k)
        fq.qf_gemm_fp8_wgrad(*s.pdr, *s.pa, s.plan, dW=s.dw2)
        fq.qf_gemm_fp8_wgrad(*s.pdh, *s.px, s.plan, dW=s.dw1)

    def update(self):
        if self.batch is None:
            self.batch = fq.AdamwBatch([dict(p=p.view(-1), g=g.view(-1), p16=w.view(-1), **fq.adamw_state(p.numel()))
                                        for p, g, w in ((self.p1, self.dw1, self.w1), (self.p2, self.dw2, self.w2))])
        fq.qf_adamw_step(self.batch, 1e-3, 1)

    def outputs(self):
        return [self.y, self.dx, self.dlogits, self.dw1, self.dw2, self.h[:self.used], self.da[:self.used]]

    @property
    def used(self):
        return int(self.plan.offsets[-1])


def codes(q, n=None):
    c, s = (t.cpu().numpy() for t in q[:2])
    return (c, s) if n is None else (c[:n], s[:, :n])


SIZES = [(1, 1, 2, 32, 16, False), (7, 2, 8, 160, 48, True), (70, 4, 5, 256, 144, True), (300, 2, 3, 400, 128, False)]


@pytest.mark.parametrize("T,k,E,H,I,masked", SIZES)
def test_every_step(T, k, E, H, I, masked):
    s = Step(T, k, E, H, I, T, masked)
    s.forward()
    s.backward()
    n, off, order, w = s.used, s.plan.offsets.cpu().numpy(), s.plan.order.cpu().numpy(), s.w.cpu().numpy()
    pos = fp8.positions(order)
    x, dy = f32(host(s.x)), f32(host(s.dy))
    h, a, r, dr, da, dh, dxs = (f32(host(t)) for t in (s.h, s.a, s.r, s.dr, s.da, s.dh, s.dxs))

    # quantized operands
    def same(got, want):
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    same(codes(s.qx, n), fp8.quant_rows(x[order[:n] // k]))
    same(codes(s.qdr, n), fp8.quant_rows(dr[:n]))
    same(codes(s.qdh, n), fp8.quant_rows(dh[:n]))
    panels = {}
    for name, q, m in (("dr", s.pdr, dr), ("a", s.pa, a), ("dh", s.pdh, dh), ("x", s.px, x[np.maximum(order, 0) // k])):
        panels[name] = fp8.quant_panels(m[:n], off)
        count = panels[name][0].shape[0]
        assert np.array_equal(q[0].cpu().numpy()[:count], panels[name][0]) and np.array_equal(q[1].cpu().numpy()[:count], panels[name][1])

    # products of the rows: forward with the weights, backward with their transpose
    for q, wq, got, K in ((s.qx, s.q1[:2], s.h, H), (s.qa, s.q2[:2], s.r, I), (s.qdr, s.q2[2:], s.da, H), (s.qdh, s.q1[2:], s.dxs, 2 * I)):
        c, sc = codes(q, n)
        wc, ws = codes(wq)
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            if off[e + 1] > off[e]:
                check_product(got[rows], *fp8.product(c[rows], sc[:, rows], wc[e], ws[e]), K)
    # gated activation
    hf = h[:n].astype(np.float64)
    act = fp8.swiglu(hf)
    within(a[:n], act, 2.0 ** -8 * np.abs(act) + (1 + 2.0 ** -8) * act_error(hf, act) + 2.0 ** -134)
    want = fp8.swiglu_backward(hf, da[:n])
    g, u, d = hf[:, :I], hf[:, I:], da[:n].astype(np.float64)
    within(dh[:n], want, 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 32 * 2.0 ** -24 *
           np.concatenate([np.abs(d * u) * (1 + np.abs(g)), np.abs(d * g)], 1) + 2.0 ** -119 * np.abs(np.concatenate([d * u, d], 1)))
    # rows back to tokens
    for got, m, wt in ((s.y, r, w), (s.dx, dxs, np.ones_like(w))):
        y, P = fp8.combine(m, pos, wt)
        within(f32(host(got)), y, 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * fp8.gamma(k) * P)
    wdr, wdw, P = fp8.combine_backward(dy, r, pos, w)
    within(dr[:n], wdr[:n], (2.0 ** -8 + 2.0 ** -22) * np.abs(wdr[:n]))
    within(s.dw.cpu().numpy(), wdw, fp8.gamma(H) * P)
    # weight gradients
    for got, dn, xn, N, K in ((s.dw2, "dr", "a", H, I), (s.dw1, "dh", "x", 2 * I, H)):
        D, X = fp8.dequant_panels(*panels[dn]), fp8.dequant_panels(*panels[xn])
        DM, XM = fp8.panels_magnitudes(*panels[dn]), fp8.panels_magnitudes(*panels[xn])
        blocks = fp8.panel_blocks(off)
        for e in range(E):
            at = [i for i, b in enumerate(blocks) if b[0] == e]
            y, P = sum((D[i].T @ X[i] for i in at), np.zeros((N, K))), sum((DM[i].T @ XM[i] for i in at), np.zeros((N, K)))
            check_product(got[e], y, P, 128 * len(at))
    # a token without an expert, and an expert without a token
    if masked:
        assert not s.y[:2].any() and not s.dx[:2].any() and not s.dw1[1].any() and not s.dw2[1].any()
    # rows behind the last group are zeros still
    for t in (s.h, s.a, s.r, s.dr, s.da, s.dh, s.dxs):
        assert not t[n:].any()
    before = s.w1.clone()
    s.update()
    assert not torch.equal(s.w1, before) and torch.equal(s.w1, s.p1.bfloat16()) and bool(torch.isfinite(s.p1).all())


@pytest.mark.parametrize("T,k,E,H,I,masked", SIZES[1:])
def test_captured(T, k, E, H, I, masked):
    """Replays with other inputs equal eager steps, bit for bit, with eager work in between."""
    s = Step(T, k, E, H, I, T + 1, masked)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.forward()
        s.backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.forward()
        s.backward()
    for seed in range(4):
        other = Step(T, k, E, H, I, T + 10 + seed, masked)
        for name in ("x", "dy", "logits", "w1", "w2"):
            getattr(s, name).copy_(getattr(other, name))
        g.replay()
        other.forward()
        other.backward()
        torch.cuda.synchronize()
        assert s.used == other.used
        for i, (got, want) in enumerate(zip(s.outputs(), other.outputs())):
            assert torch.equal(got, want), f"output {i}, seed {seed}"


def test_two_streams_at_once():
    """Steps on two streams do not see each other (no call keeps a workspace)."""
    steps = [Step(300, 2, 3, 400, 128, 50 + i, i == 1) for i in range(2)]
    for s in steps:
        s.forward()
        s.backward()
    torch.cuda.synchronize()
    want = [[t.clone() for t in s.outputs()] for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.forward()
                s.backward()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for got, ref in zip(s.outputs(), w):
            assert torch.equal(got, ref)
