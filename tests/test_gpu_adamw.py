"""qf_adamw_step on the GPU: bit for bit the stated fp32 sequence, and within counted roundings
of the float64 formula."""

import gc
import weakref

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import adamw
from oracle import primitives as P
from tests.gpu_util import first_mismatch, host
from tests.test_oracle_adamw import bounds64, draw

pytestmark = pytest.mark.gpu
SIZES = [1, 2, 3, 4, 5, 63, 64, 255, 256, 257, 1023, 4095, 4096, 4097, 70001]


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def down(t):
    return t.detach().cpu().numpy()


def make(n, seed, bits, g_bf16, copy=True, fresh=False, wd=0.0):
    """(device item, host copies) of one tensor."""
    p, g, m, r = draw(n, seed, g_bf16)
    h = dict(p=p, g=g, wd=wd)
    it = dict(p=up(p), g=up(g).bfloat16() if g_bf16 else up(g), weight_decay=wd)
    if fresh:
        m[:], r[:] = 0, 0
    if bits == 8:
        zero = np.zeros(n, np.uint32)
        h["mc"], h["ms"] = adamw.encode(m, zero, False)
        h["vc"], h["vs"] = adamw.encode(r, zero, True)
        it.update(m=up(h["mc"]), m_scale=up(h["ms"]), v=up(h["vc"]), v_scale=up(h["vs"]))
    else:
        h["m"], h["v"] = m, r * r
        it.update(m=up(m), v=up(h["v"]))
    if copy:
        it["p16"] = torch.full((n,), -7.0, dtype=torch.bfloat16, device="cuda")
    return it, h


def want(h, bits, lr, step, seed=0, **kw):
    if bits == 8:
        return adamw.step8(h["p"], h["g"], h["mc"], h["ms"], h["vc"], h["vs"], lr, step, seed, weight_decay=h["wd"], **kw)
    return adamw.step32(h["p"], h["g"], h["m"], h["v"], lr, step, weight_decay=h["wd"], **kw)


def names(bits):
    return ("p", "m", "m_scale", "v", "v_scale") if bits == 8 else ("p", "m", "v")


def same(it, w, bits, what):
    for k, b in zip(names(bits), w):
        a = down(it[k])
        b = np.asarray(b)
        a, b = a.view(np.uint8 if a.dtype == np.uint8 else np.uint32), b.view(np.uint8 if b.dtype == np.uint8 else np.uint32)
        assert np.array_equal(a, b), f"{what} {k}: {first_mismatch(a, b)}"
    if it.get("p16") is not None:
        assert np.array_equal(host(it["p16"]), P.f32_to_bf16(np.asarray(w[0]))), f"{what} p16"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_bf16", [False, True])
def test_sizes_bit_exact(bits, g_bf16):
    """Every size in one call (partial lanes, blocks and workgroups), two steps in a row."""
    made = [make(n, n, bits, g_bf16, copy=n % 2 == 1, wd=0.1 * (n % 3)) for n in SIZES]
    batch = fq.AdamwBatch([it for it, _ in made], state_bits=bits)
    grads = [it["g"].clone() for it, _ in made]
    for step in (3, 4):
        fq.qf_adamw_step(batch, 1e-3, step, seed=99)
        for (it, h), n in zip(made, SIZES):
            w = want(h, bits, 1e-3, step, 99)
            same(it, w, bits, f"n={n} step {step}")
            h.update(zip(("p", "mc", "ms", "vc", "vs") if bits == 8 else ("p", "m", "v"), w))
    for (it, _), g in zip(made, grads):
        assert torch.equal(it["g"], g)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_mixed_gradients(bits):
    """131 tensors with both gradient types and an empty one: several launches of each type."""
    made = [make(1 + 37 * i % 1500, 1000 + i, bits, i % 3 == 0, copy=i % 4 == 0, wd=0.05 * (i % 2)) for i in range(130)]
    empty = dict(p=torch.empty(0, device="cuda"), g=torch.empty(0, device="cuda"), **fq.adamw_state(0, bits))
    batch = fq.AdamwBatch([it for it, _ in made[:60]] + [empty] + [it for it, _ in made[60:]], state_bits=bits)
    fq.qf_adamw_step(batch, 2e-4, 17, beta1=0.8, beta2=0.95, eps=1e-6, seed=5)
    for i, (it, h) in enumerate(made):
        same(it, want(h, bits, 2e-4, 17, 5, beta1=0.8, beta2=0.95, eps=1e-6), bits, f"tensor {i}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [9, 64, 65, 130, 4200])
def test_table_and_host_descriptors_agree(bits, count):
    """The table's one launch against the descriptors in the arguments, for counts around the
    lookup's 64 lanes and its third level."""
    def items():
        rng = np.random.default_rng(count)
        flat = {k: torch.from_numpy(rng.standard_normal(count * 512).astype(np.float32)).cuda() for k in ("p", "g")}
        out = []
        for i in range(count):
            n = int(rng.integers(0, 500))
            it = {k: flat[k][512 * i:512 * i + n] for k in ("p", "g")}
            if i % 5 == 0:
                it["g"] = it["g"].bfloat16()
            it.update({k: torch.zeros_like(v) for k, v in fq.adamw_state(n, bits).items()})
            out.append(dict(it, weight_decay=0.1 * (i % 2)))
        return out
    a, b = items(), items()
    ba, bb = fq.AdamwBatch(a, bits), fq.AdamwBatch(b, bits)
    assert ba.table is not None
    bb.table = None                                      # through qf_adamw_step
    for step in (1, 2):
        fq.qf_adamw_step(ba, 1e-3, step, seed=8)
        fq.qf_adamw_step(bb, 1e-3, step, seed=8)
    for x, y in zip(a, b):
        for k in names(bits):
            assert torch.equal(x[k], y[k])


@pytest.mark.parametrize("bits", [32, 8])
def test_against_float64(bits):
    n, lr, step, gs = 50000, 1e-3, 12, 0.25
    it, h = make(n, 7, bits, False, wd=0.1)
    if bits == 8:
        m, r = adamw.decode(h["mc"], h["ms"]).astype(np.float64), adamw.decode(h["vc"], h["vs"]).astype(np.float64)
        v = r * r
    else:
        m, v = h["m"], h["v"]
    p64, m64, v64 = adamw.step64(h["p"], h["g"], m, v, lr, step, weight_decay=0.1, grad_scale=gs)
    tp, tm, tv = bounds64(h["p"], h["g"], m, v, lr, step, weight_decay=0.1, grad_scale=gs)
    fq.qf_adamw_step(fq.AdamwBatch([it], state_bits=bits), lr, step, seed=1, d_grad_scale=torch.full((1,), gs, device="cuda"))
    assert np.all(np.abs(down(it["p"]) - p64) <= tp)
    if bits == 32:
        assert np.all(np.abs(down(it["m"]) - m64) <= tm) and np.all(np.abs(down(it["v"]) - v64) <= tv)
        return
    for k, x, tol in (("m", m64, tm), ("v", np.sqrt(v64), tv / np.maximum(np.sqrt(v64), 1e-300))):
        dec = adamw.decode(down(it[k]), down(it[k + "_scale"])).astype(np.float64)
        sc = np.repeat(down(it[k + "_scale"]).astype(np.float64), 256)[:n]
        step8 = np.maximum(2.0 ** -3 * np.abs(x), 2.0 ** -9 * sc)          # at most one E4M3 step
        assert np.all(np.abs(dec - x) <= step8 * (1 + 8 * 2.0 ** -24) + tol + 4 * 2.0 ** -24 * np.abs(x))
        # unbiased: n roundings, each within one step: the mean error is below 5 / (2 sqrt(n)) steps
        if k == "m":
            assert abs(np.mean((dec - x) / step8)) < 2.5 / np.sqrt(n)


def test_device_scalars_and_skip():
    it, h = make(5000, 11, 32, False)
    batch = fq.AdamwBatch([it])
    d_lr = torch.full((1,), 0.5, device="cuda")
    d_step = torch.full((1,), 9, dtype=torch.int64, device="cuda")
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    before = {k: it[k].clone() for k in ("p", "m", "v", "p16")}
    fq.qf_adamw_step(batch, 1e-3, 1, d_lr=d_lr, d_step=d_step, d_skip=skip)
    for k, b in before.items():
        assert torch.equal(it[k], b)
    skip.zero_()
    fq.qf_adamw_step(batch, 1e-3, 1, d_lr=d_lr, d_step=d_step, d_skip=skip)
    same(it, want(h, 32, 0.5, 9), 32, "device scalars")


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_replays(bits):
    """A captured step follows the device step number on every replay."""
    it, h = make(9001, 21, bits, True)
    batch = fq.AdamwBatch([it], state_bits=bits)
    d_step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        d_step.add_(1)
        fq.qf_adamw_step(batch, 1e-3, 1, d_step=d_step, seed=3)
    keep = {k: v.clone() for k, v in it.items() if isinstance(v, torch.Tensor)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for k, v in keep.items():
        it[k].copy_(v)
    d_step.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 2, 3):
        g = draw(9001, 50 + i, True)[1]
        it["g"].copy_(up(g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        h["g"] = g
        w = want(h, bits, 1e-3, i, 3)
        same(it, w, bits, f"replay {i}")
        h.update(zip(("p", "mc", "ms", "vc", "vs") if bits == 8 else ("p", "m", "v"), w))


def test_grouping_does_not_change_results():
    a = [make(n, n, 8, False) for n in (300, 4099, 17)]
    b = [make(n, n, 8, False) for n in (300, 4099, 17)]
    fq.qf_adamw_step(fq.AdamwBatch([it for it, _ in a], 8), 1e-3, 2, seed=4)
    for it, _ in reversed(b):
        fq.qf_adamw_step(fq.AdamwBatch([it], 8), 1e-3, 2, seed=4)
    for (x, _), (y, _) in zip(a, b):
        for k in names(8):
            assert torch.equal(x[k], y[k])


def test_table_outlives_a_step_on_another_stream():
    """A batch dropped while its step waits on another stream: the table's memory is not given out again."""
    made = [make(300 + i, i, 32, False) for i in range(20)]
    batch = fq.AdamwBatch([it for it, _ in made])
    at, size = batch.table.data_ptr(), batch.table.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                    # cycles; the step is queued behind it
        fq.qf_adamw_step(batch, 1e-3, 2)
    busy = not side.query()
    del batch
    fresh = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert busy and all(t.data_ptr() != at for t in fresh)
    torch.cuda.synchronize()
    for it, h in made:
        same(it, want(h, 32, 1e-3, 2), 32, "side stream")


@pytest.mark.parametrize("bits", [32, 8])
def test_shared_and_overlapping_tensors_are_refused(bits):
    """Two tensors of a batch run at the same time: no state, weight or copy may serve both."""
    a, b = (make(512, i, bits, False)[0] for i in (1, 2))
    fq.AdamwBatch([a, b], bits)
    for k in ("p", "m", "v", "p16") + (("m_scale", "v_scale") if bits == 8 else ()):
        with pytest.raises(ValueError, match="overlap"):
            fq.AdamwBatch([a, dict(b, **{k: a[k]})], bits)
    both = torch.zeros(768, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        fq.AdamwBatch([dict(a, p=both[:512]), dict(b, p=both[256:])], bits)
    with pytest.raises(ValueError, match="overlap"):
        fq.AdamwBatch([dict(a, p16=a["p"].view(torch.bfloat16)[:512])], bits)
    fq.AdamwBatch([a, dict(b, g=a["g"])], bits)          # only read
    empty = dict(p=a["p"][:0], g=a["g"][:0], m=a["m"][:0], v=a["v"][:0])
    if bits == 8:
        empty.update(m_scale=a["m_scale"][:0], v_scale=a["v_scale"][:0])
    fq.AdamwBatch([a, empty, empty], bits)


@pytest.mark.parametrize("count", [1, 12])
def test_batch_holds_its_tensors(count):
    """A caller that puts other tensors into its dicts (new gradients) leaves the batch's alive."""
    made = [make(300 + i, i, 32, False) for i in range(count)]
    batch = fq.AdamwBatch([it for it, _ in made])
    refs = [weakref.ref(it[k]) for it, _ in made for k in ("p", "g", "m", "v", "p16")]
    kept = [dict(it) for it, _ in made]
    for it, _ in made:
        it.clear()
    held = [{k: batch.items[i][k] for k in k0} for i, k0 in enumerate(kept)]
    assert all(a[k] is b[k] for a, b in zip(kept, held) for k in a)
    del kept, held, it
    gc.collect()
    assert all(r() is not None for r in refs)
    fq.qf_adamw_step(batch, 1e-3, 2)
    for it, (_, h) in zip(batch.items, made):
        same(it, want(h, 32, 1e-3, 2), 32, "held")


def test_binding_checks():
    it, _ = make(64, 1, 32, False)
    with pytest.raises(ValueError):
        fq.AdamwBatch([it, it])                                  # the same tensor twice
    with pytest.raises(ValueError):
        fq.AdamwBatch([dict(it, m=it["m"][:63])])
    with pytest.raises(ValueError):
        fq.AdamwBatch([it], state_bits=8)                        # fp32 moments
    with pytest.raises(TypeError):
        fq.AdamwBatch([dict(it, g=it["g"].half())])
    with pytest.raises(TypeError):
        fq.qf_adamw_step(fq.AdamwBatch([it]), 1e-3, 1, d_step=torch.zeros(1, device="cuda"))
    with pytest.raises(fq.QFError):
        fq.qf_adamw_step(fq.AdamwBatch([it]), 1e-3, 0)
    big = torch.zeros(68, device="cuda")
    with pytest.raises(fq.QFError):                              # 4-byte aligned weights
        fq.qf_adamw_step(fq.AdamwBatch([dict(it, p=big[1:65])]), 1e-3, 1)
