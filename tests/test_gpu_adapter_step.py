"""Routing, row plan, per-request adapters, merge, adapter gradients and AdamW together, as a
training step of a mixture's adapters uses them: tokens are routed; the unmerged adapters of the
chosen experts are applied to their (token, expert) rows; the merged experts are quantized;
the adapters' gradients update fp32 masters, whose bf16 copies are the adapters of the next
step; the router gets its gradient.  Every stage is checked against the oracle, and the whole
step, captured in a graph, gives the bits of the eager step on every replay.
"""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import adamw, lora, nvfp4, route, rows
from oracle import primitives as prim
from tests.gpu_util import dev, host, u8

pytestmark = pytest.mark.gpu
E, R, ROWS, COLS, T, K = 6, 4, 72, 96, 70, 2
LR = 1e-2


class Step:
    def __init__(self, state_bits):
        rng = np.random.default_rng(3)
        f = lambda shape, s: torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).cuda()  # noqa: E731
        self.bits = state_bits
        self.W = f((E, ROWS, COLS), 0.02).bfloat16()
        self.pA, self.pB = f((E, R, COLS), 0.1), f((E, ROWS, R), 0.1)
        self.A, self.B = self.pA.bfloat16(), self.pB.bfloat16()
        self.X, self.logits = f((T, COLS), 1.0).bfloat16(), f((T, E), 1.0)
        self.Y0 = f((T * K, ROWS), 1.0).bfloat16()
        self.G = f((E, ROWS, COLS), 1.0).bfloat16()
        self.dw = f((T, K), 1.0)
        self.bias = f((E,), 0.05)
        self.Y = torch.empty_like(self.Y0)
        self.idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
        self.w = torch.empty((T, K), device="cuda")
        self.dlogits = torch.empty_like(self.logits)
        self.plan = fq.RowPlan(T * K, E, "cuda")
        self.y = torch.empty_like(self.W)
        self.codes = torch.empty((E, ROWS, COLS // 2), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty((E, ROWS, COLS // 16), dtype=torch.uint8, device="cuda")
        self.ts = torch.empty(E, device="cuda")
        self.dA, self.dB = torch.empty_like(self.pA), torch.empty_like(self.pB)
        self.ex = fq.LoraExperts([dict(W=self.W, A=self.A, B=self.B, group=0, y=self.y, codes=self.codes,
                                       scales=self.scales, G=self.G, dA=self.dA, dB=self.dB)])
        self.sA, self.sB = fq.adamw_state(self.pA.numel(), state_bits), fq.adamw_state(self.pB.numel(), state_bits)
        self.batch = fq.AdamwBatch([dict(p=self.pA.view(-1), g=self.dA.view(-1), p16=self.A.view(-1), weight_decay=0.1, **self.sA),
                                    dict(p=self.pB.view(-1), g=self.dB.view(-1), p16=self.B.view(-1), **self.sB)], state_bits)
        self.d_step = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.ws1 = torch.empty(max(fq.qf_lora_apply_workspace(T * K, COLS, R, E, True), 1), dtype=torch.uint8, device="cuda")
        self.ws2 = torch.empty(max(self.ex.workspace_bytes, 4), dtype=torch.uint8, device="cuda")

    def run(self):
        fq.qf_moe_route(self.logits, K, scoring="sigmoid", bias=self.bias, indices=self.idx, weights=self.w)
        fq.qf_row_plan(self.idx, E, plan=self.plan)
        self.Y.copy_(self.Y0)
        fq.qf_lora_apply_planned(self.X, self.A, self.B, self.plan, self.Y, rows_per_x=K, ws=self.ws1)
        fq.qf_moe_route_backward(self.logits, self.idx, self.dw, scoring="sigmoid", d_logits=self.dlogits)
        fq.qf_lora_experts_merge_tensor_scale_nvfp4(self.ex, E, self.ts, None, self.ws2)
        fq.qf_lora_experts_merge_qdq_pack_nvfp4(self.ex, self.ts)
        fq.qf_lora_experts_adapter_grads(self.ex, False, self.ws2)
        self.d_step.add_(1)
        fq.qf_adamw_step(self.batch, LR, 1, d_step=self.d_step, seed=11)

    def tensors(self):
        return dict(idx=self.idx, w=self.w, offsets=self.plan.offsets, order=self.plan.order, tiles=self.plan.tiles, Y=self.Y,
                    dlogits=self.dlogits, y=self.y, codes=self.codes, scales=self.scales, ts=self.ts, dA=self.dA, dB=self.dB,
                    pA=self.pA, pB=self.pB, A=self.A, B=self.B, **{"A" + k: v for k, v in self.sA.items()},
                    **{"B" + k: v for k, v in self.sB.items()})


def np32(t):
    return t.detach().float().cpu().numpy()


@pytest.mark.parametrize("bits", [32, 8])
def test_step_against_the_oracle(bits):
    s = Step(bits)
    states = {}
    for p, st in (("A", s.sA), ("B", s.sB)):
        states[p] = [u8(v) if v.dtype == torch.uint8 else np32(v) for v in
                     ((st["m"], st["m_scale"], st["v"], st["v_scale"]) if bits == 8 else (st["m"], st["v"]))]
    for step in (1, 2, 3):
        before = {k: v.clone() for k, v in dict(A=s.A, B=s.B, pA=s.pA, pB=s.pB).items()}
        s.run()
        ri, rw = route.route(np32(s.logits), K, "sigmoid", np32(s.bias))
        assert np.array_equal(s.idx.cpu().numpy(), ri) and np.allclose(np32(s.w), rw, rtol=1e-5, atol=0)
        ids = ri.reshape(-1)
        for got, want in zip((s.plan.offsets, s.plan.order, s.plan.tiles), rows.plan(ids, E)):
            assert np.array_equal(got.cpu().numpy(), want)
        y, P, y0 = rows.apply(np32(s.X), np32(before["A"]), np32(before["B"]), ids, np32(s.Y0), None, K)
        assert np.all(np.abs(np32(s.Y) - y) <= rows.apply_bound(y, P, y0, COLS, R))
        d, mag = route.backward(np32(s.logits), ri, np32(s.dw), "sigmoid", True, 1.0)
        assert np.all(np.abs(np32(s.dlogits) - d) <= 304 * 2.0 ** -24 * mag)
        for e in range(E):
            M = lora.merge(host(s.W[e]), host(before["A"][e]), host(before["B"][e]))
            ts = nvfp4.tensor_scale([M])
            codes, S = nvfp4.quantize(M, ts)
            pc, ps = nvfp4.pack(codes, S)
            assert np.array_equal(u8(s.codes[e]), pc) and np.array_equal(u8(s.scales[e]), ps)
            assert np.array_equal(host(s.y[e]), nvfp4.dequantize(codes, S, ts))
        for p, master, g, wd in (("A", before["pA"], s.dA, 0.1), ("B", before["pB"], s.dB, 0.0)):
            n = master.numel()
            if bits == 8:
                out = adamw.step8(np32(master).reshape(-1), np32(g).reshape(-1), *states[p], LR, step, 11, weight_decay=wd)
            else:
                out = adamw.step32(np32(master).reshape(-1), np32(g).reshape(-1), *states[p], LR, step, weight_decay=wd)
            states[p] = list(out[1:])
            new = s.pA if p == "A" else s.pB
            assert np.array_equal(np32(new).reshape(-1), out[0]) and n == out[0].size
            assert np.array_equal(host(s.A if p == "A" else s.B).reshape(-1), prim.f32_to_bf16(out[0]))
        assert not torch.equal(before["A"], s.A)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_the_eager_one(bits):
    eager, graphed = Step(bits), Step(bits)
    first = {k: v.clone() for k, v in graphed.tensors().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.run()                                    # first calls outside the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.run()
    for k, v in graphed.tensors().items():
        v.copy_(first[k])
    graphed.d_step.zero_()
    for seed in range(4):
        rng = np.random.default_rng(seed)
        for name, shape in (("logits", (T, E)), ("dw", (T, K))):
            x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
            getattr(eager, name).copy_(x)
            getattr(graphed, name).copy_(x)
        eager.run()
        g.replay()
        torch.cuda.synchronize()
        for (k, a), b in zip(eager.tensors().items(), graphed.tensors().values()):
            assert torch.equal(a, b), f"replay {seed}: {k}"
