"""qf_moe_route and its gradient on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import route

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")


def logits(T, E, seed, bf16, scale=1.5):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)) * scale).float()
    return x.bfloat16().cuda() if bf16 else x.cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


def spread(x):
    """Largest distance of a row's unmasked logits."""
    f = np.where(np.isfinite(x), x, np.nan)
    with np.errstate(all="ignore"):
        return np.nan_to_num(np.nanmax(f, 1) - np.nanmin(f, 1)) if x.size else np.zeros(0)


def check(x, k, scoring, renorm=True, scale=1.0, **kw):
    bias = kw.get("bias")
    idx, w = fq.qf_moe_route(x, k, scoring=scoring, renorm=renorm, scale=scale, **kw)
    ref = dict(kw, bias=np64(bias) if bias is not None else None)
    xi = np64(x)
    ri, rw = route.route(xi, k, scoring, renorm=renorm, scale=scale, **ref)
    got = idx.cpu().numpy()
    assert np.array_equal(got, ri), f"{(got != ri).any(1).sum()} rows choose differently"
    D = spread(xi)[:, None] if scoring == "softmax" else 0.0
    assert np.all(np.abs(np64(w) - rw) <= (2 * D + 60) * U * np.abs(rw) + 1e-37)
    return idx, w


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 3, 2), (33, 60, 6), (5, 64, 32), (300, 127, 4), (17, 128, 20),
                                   (40, 160, 6), (65, 256, 8), (9, 257, 9), (12, 512, 10), (6, 1000, 32), (3, 1024, 17)])
def test_plain(T, E, k, scoring, bf16):
    x = logits(T, E, T * E, bf16)
    check(x, k, scoring, renorm=True)
    check(x, k, scoring, renorm=False, scale=2.5)
    bias = torch.from_numpy(np.random.default_rng(E).standard_normal(E) * 0.1).float().cuda()
    check(x, k, scoring, renorm=True, bias=bias, scale=0.5)
    check(x, k, scoring, renorm=False, bias=bias)


@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("E,G,kept,k", [(256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 2, 8), (64, 64, 5, 5), (1024, 32, 7, 16),
                                        (10, 5, 2, 3), (96, 3, 3, 7), (512, 2, 1, 32)])
def test_groups(E, G, kept, k, rule):
    for scoring in ("softmax", "sigmoid"):
        for bf16 in (False, True):
            x = logits(150, E, E + G, bf16)
            bias = torch.from_numpy(np.random.default_rng(G).standard_normal(E) * 0.1).float().cuda()
            kw = dict(n_group=G, topk_group=kept, group_rule=rule)
            check(x, k, scoring, **kw)
            check(x, k, scoring, bias=bias, renorm=False, **kw)


@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("E,G,kept,k", [(300, 4, 2, 8), (384, 8, 3, 8), (510, 5, 2, 32), (513, 3, 2, 9), (1000, 8, 3, 16),
                                        (1001, 7, 3, 9), (1024, 64, 30, 32), (1023, 33, 4, 31)])
def test_many_experts_in_groups_of_any_size(E, G, kept, k, rule):
    for scoring in ("softmax", "sigmoid"):
        for bf16 in (False, True):
            x = logits(70, E, E + G, bf16)
            bias = torch.from_numpy(np.random.default_rng(G).standard_normal(E) * 0.1).float().cuda()
            kw = dict(n_group=G, topk_group=kept, group_rule=rule)
            check(x, k, scoring, **kw)
            check(x, k, scoring, bias=bias, renorm=False, **kw)


@pytest.mark.parametrize("E,G", [(64, 4), (256, 8), (512, 4), (1000, 8)])
def test_groups_of_an_unaligned_view(E, G):
    for bf16 in (False, True):
        x = torch.full((40, E + 5), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")[:, 1:E + 1]
        x.copy_(logits(40, E, E, bf16))
        bias = torch.from_numpy(np.random.default_rng(G).standard_normal(E) * 0.1).float().cuda()
        for rule in ("max", "top2"):
            check(x, 6, "softmax", n_group=G, topk_group=2, group_rule=rule)
            check(x, 6, "sigmoid", bias=bias, n_group=G, topk_group=2, group_rule=rule)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(n_group=4, topk_group=2, group_rule="top2"), dict(n_group=4, topk_group=2)])
def test_ties_and_masks(scoring, groups):
    """Few distinct values (ties of experts and of groups); masked experts, groups and rows.  The
    values are off the half-integers (sigmoid(x) + sigmoid(-x) = 1 for every x) and the biases of
    ranked pairs generic, so that no two different sums are equal but for rounding."""
    rng = np.random.default_rng(9)
    v = np.round(rng.standard_normal((64, 32)) * 2) / 2 + 0.3
    v[3] = 1.25
    v[4, :] = -INF
    v[5, 1:] = -INF
    v[6, :24] = -INF
    v[7, ::2] = -INF
    v[8, 3:30] = -INF
    x = torch.from_numpy(v).float().cuda()
    bias = rng.standard_normal(32) * 2
    bias = torch.from_numpy((bias if groups.get("group_rule") == "top2" else np.round(bias)) / 16).float().cuda()
    off = bias.clone()
    off[5:12] = -INF                                     # experts taken out by their bias
    for t in (x, x.bfloat16()):
        for renorm in (True, False):
            check(t, 6, scoring, renorm=renorm, **groups)
            check(t, 6, scoring, renorm=renorm, bias=torch.zeros(32, device="cuda"), **groups)
            check(t, 6, scoring, renorm=renorm, bias=bias, **groups)
            check(t, 6, scoring, renorm=renorm, bias=off, **groups)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_rule="top2")])
def test_zeros_of_both_signs_tie(scoring, groups):
    """+0 and -0 are one value (a clipped or masked router gives both): the lower index comes first."""
    rng = np.random.default_rng(12)
    v = np.where(rng.integers(0, 2, (200, 64)) == 1, 0.0, -0.0)
    v[100:] = np.where(rng.integers(0, 4, (100, 64)) == 0, rng.standard_normal((100, 64)), v[100:])
    x = torch.from_numpy(v).float().cuda()
    bias = torch.where(torch.arange(64) % 3 == 0, 0.0, -0.0).cuda()
    for t in (x, x.bfloat16()):
        check(t, 8, scoring, **groups)
        check(t, 8, scoring, bias=bias, **groups)


def test_near_ties_are_decided_in_64_bits():
    """Biased scores that differ by less than an fp32 rounding."""
    T, E = 2000, 64
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((T, E))).float()
    s = 1.0 / (1.0 + torch.exp(-x[0].double()))
    bias = (0.75 - s).float()                            # every expert of row 0 at 0.75 within an fp32 step
    x[1::2] = x[0]
    x[1::2] += torch.from_numpy(rng.integers(-3, 4, (T // 2, E)) * 2.0 ** -22).float()
    check(x.cuda(), 8, "sigmoid", bias=bias.cuda())
    check(x.cuda(), 8, "sigmoid", bias=bias.cuda(), n_group=8, topk_group=3, group_rule="top2")
    check(x.cuda(), 8, "softmax", bias=bias.cuda())


def test_extreme_logits():
    """Far apart logits; the weights of chosen experts that softmax alone would underflow."""
    rng = np.random.default_rng(6)
    v = rng.standard_normal((50, 40)) * 60
    x = torch.from_numpy(v).float().cuda()
    bias = torch.zeros(40, device="cuda")
    bias[:4] = -5.0                                      # sends away from the largest scores
    check(x, 4, "softmax")
    check(x, 4, "softmax", bias=bias)
    check(x.clamp(-80, 30), 4, "sigmoid")


def test_low_sigmoid_scores_of_groups():
    """Groups ranked by sums of scores down to the end of 64 bits: distinct logits, distinct sums."""
    rng = np.random.default_rng(15)
    v = np.stack([rng.permutation(np.arange(-738, -738 + 24)) for _ in range(100)]).astype(np.float64)
    x = torch.from_numpy(v).float().cuda()
    for rule in ("top2", "max"):
        check(x, 5, "sigmoid", n_group=6, topk_group=2, group_rule=rule)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_poisoned_rows(scoring):
    """A NaN or plus infinity shows in its own row alone."""
    x = logits(9, 48, 2, False)
    clean_i, clean_w = fq.qf_moe_route(x, 5, scoring=scoring)
    y = x.clone()
    y[2, 47], y[5, 0] = float("nan"), INF
    for kw in (dict(), dict(bias=torch.zeros(48, device="cuda")), dict(n_group=4, topk_group=2, group_rule="top2")):
        base_i, base_w = fq.qf_moe_route(x, 5, scoring=scoring, **kw)
        i, w = fq.qf_moe_route(y, 5, scoring=scoring, **kw)
        for t in range(9):
            if t in (2, 5):
                assert bool((i[t] == -1).all()) and bool(w[t].isnan().all())
            else:
                assert torch.equal(i[t], base_i[t]) and torch.equal(w[t], base_w[t])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_poisoned_bias(scoring, bad):
    """A NaN or plus infinity in the bias shows in every row, also in those that mask its expert."""
    for E, groups in ((48, dict()), (48, dict(n_group=4, topk_group=2)), (45, dict(n_group=3, topk_group=2, group_rule="top2")),
                      (300, dict(n_group=4, topk_group=2))):
        x = logits(8, E, 2, False)
        bias = torch.zeros(E, device="cuda")
        x[::2, E - 2] = -INF
        x[5] = -INF
        clean_i, _ = fq.qf_moe_route(x, 5, scoring=scoring, bias=bias, **groups)
        assert bool((clean_i[5] == -1).all()) and bool((clean_i[:5] >= 0).all())
        bias[E - 2] = bad
        for t in (x, x.bfloat16()):
            i, w = fq.qf_moe_route(t, 5, scoring=scoring, bias=bias, **groups)
            assert bool((i == -1).all()) and bool(w.isnan().all())
        bias[E - 2] = -INF
        i, w = fq.qf_moe_route(x, 5, scoring=scoring, bias=bias, **groups)
        assert not bool((i == E - 2).any()) and bool(w.isfinite().all()) and bool((i[:5] >= 0).all())


def check_backward(x, idx, dw, scoring, renorm, scale, **kw):
    got = fq.qf_moe_route_backward(x, idx, dw, scoring=scoring, renorm=renorm, scale=scale, **kw)
    xi = np64(x)
    ref, mag = route.backward(xi, idx.cpu().numpy(), np64(dw), scoring, renorm, scale)
    D = spread(xi)[:, None] if scoring == "softmax" else 0.0
    # every factor within (2 D + 60) U of its value, at most four of them in a term, sums of
    # up to 32 chosen terms and the row's; then one rounding to the output's type
    tol = (4 * (2 * D + 60) + 64) * U * mag + 1e-37
    if x.dtype == torch.bfloat16:
        tol = 2.0 ** -8 * (np.abs(ref) + tol) + tol
    assert np.all(np.abs(np64(got) - ref) <= tol)
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (70, 128, 8), (33, 129, 6), (9, 256, 32), (4, 1024, 12)])
def test_backward(T, E, k, scoring, renorm, bf16):
    x = logits(T, E, E, bf16)
    dw = torch.from_numpy(np.random.default_rng(T).standard_normal((T, k))).float().cuda()
    idx, _ = fq.qf_moe_route(x, k, scoring=scoring)
    check_backward(x, idx, dw, scoring, renorm, 1.5)
    if T > 3:
        idx[1] = -1                                      # no expert at all
        idx[2, 0] = -1
        idx[3, 0], idx[3, k - 1] = E + 5, -2 ** 31
        check_backward(x, idx, dw, scoring, renorm, 1.0)
        if k > 1:
            idx[0, 1] = idx[0, 0]                        # the same index twice
            check_backward(x, idx, dw, scoring, renorm, 1.0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(scoring, renorm):
    """Central differences of the forward's own weights (its fp32 error is U-sized, the step 2^-6)."""
    T, E, k = 6, 24, 4
    x = logits(T, E, 77, False)
    dw = torch.from_numpy(np.random.default_rng(78).standard_normal((T, k))).float().cuda()
    idx, _ = fq.qf_moe_route(x, k, scoring=scoring, renorm=renorm)
    got = np64(fq.qf_moe_route_backward(x, idx, dw, scoring=scoring, renorm=renorm))
    h = 2.0 ** -6

    def loss(y):
        i, w = fq.qf_moe_route(y, k, scoring=scoring, renorm=renorm)
        # weights matched by expert: a small step may reorder the same choice
        full = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, i.long(), w.double())
        return (full.gather(1, idx.long()) * dw.double()).sum(1), torch.equal(i.sort(1).values, idx.sort(1).values)
    for e in range(E):
        d = torch.zeros_like(x)
        d[:, e] = h
        (a, same_a), (b, same_b) = loss(x + d), loss(x - d)
        if not (same_a and same_b):
            continue                                     # the choice itself changed
        diff = np64((a - b) / (2 * h))
        # |third derivative| of a weight <= 1, so h^2 / 6 sum |dw|; fp32 weights: 100 U / h each
        tol = (h * h / 6 + 2 * 100 * U / h) * np64(dw.abs().sum(1))
        assert np.all(np.abs(got[:, e] - diff) <= tol)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_backward_of_a_lone_choice_is_zero(scoring, bf16):
    """Over its own sum a single weight is constant: no rounding may leave a gradient for an optimizer to scale up."""
    x = logits(400, 43, 8, bf16)
    dw = torch.from_numpy(np.random.default_rng(3).standard_normal((400, 1))).float().cuda()
    idx, _ = fq.qf_moe_route(x, 1, scoring=scoring)
    assert int(fq.qf_moe_route_backward(x, idx, dw, scoring=scoring).count_nonzero()) == 0
    three = torch.cat([idx, torch.full_like(idx, -1), torch.full_like(idx, -1)], 1)
    assert int(fq.qf_moe_route_backward(x, three, dw.repeat(1, 3), scoring=scoring).count_nonzero()) == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_confident_choices(renorm, bf16):
    """1 - s keeps its digits where s is near 1, under the bound of every other gradient: chosen
    logits up to 80, where s rounds to 1, beside ones near 0 and down to -80."""
    for top in (7.0, 8.0, 10.0, 12.0, 15.0, 16.0, 17.0, 20.0, 30.0, 40.0, 80.0):
        x = logits(40, 32, int(top), False, scale=0.25)
        x[:, 3] += top
        x[::2, 17] += top
        x[::3, 30] -= top
        x = x.bfloat16() if bf16 else x
        idx, _ = fq.qf_moe_route(x, 6, scoring="sigmoid", renorm=renorm)
        idx[::3, 5] = 30                                 # the lowest logit, chosen
        dw = torch.from_numpy(np.random.default_rng(int(top)).standard_normal((40, 6))).float().cuda()
        got = check_backward(x, idx, dw, "sigmoid", renorm, 1.5)
        assert bool((got[:, 3] != 0).all())              # as in the formula


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("at", [-15.0, -19.0, -21.0, -50.0, -80.0, -89.0, -95.0, -100.0, -200.0, -700.0, -5000.0, -1e30])
def test_low_sigmoid_scores(at, renorm):
    """Scores below fp32's range: their weights over their sum are those of the formula, and so is
    the gradient; the plain ones vanish as the formula's do."""
    T, E, k = 60, 48, 5
    x = logits(T, E, 11, False) + at
    x[::4, 7] = at / 2                                   # rows with one far larger choice
    x[1::8, 3:] = at - 70                                # and with far smaller ones
    x[5::8, 3:] = at - 90
    x[2::4, 9:] = -INF
    dw = torch.from_numpy(np.random.default_rng(12).standard_normal((T, k))).float().cuda()
    for t in (x, x.bfloat16()):
        xi = np64(t)
        idx, w = fq.qf_moe_route(t, k, scoring="sigmoid", renorm=renorm, scale=2.0)
        ri, rw = route.route(xi, k, "sigmoid", renorm=renorm, scale=2.0)
        assert np.array_equal(idx.cpu().numpy(), ri)
        best = xi.max(1, keepdims=True)
        D = np.where(renorm & (best < -20), best - np.where(np.isfinite(xi), xi, np.inf).min(1, keepdims=True), 0.0)
        assert np.all(np.abs(np64(w) - rw) <= (2 * D + 60) * U * np.abs(rw) + 2.0 ** -119 * 2.0)
        g = np64(fq.qf_moe_route_backward(t, idx, dw, scoring="sigmoid", renorm=renorm, scale=2.0))
        ref, mag = route.backward(xi, ri, np64(dw), "sigmoid", renorm, 2.0)
        tol = (4 * (2 * D + 60) + 64) * U * mag + 2.0 ** -116 * 2.0 * np64(dw.abs().sum(1, keepdim=True))
        if t.dtype == torch.bfloat16:
            tol = 2.0 ** -8 * (np.abs(ref) + tol) + tol
        assert np.all(np.abs(g - ref) <= tol)
        if renorm:
            assert np.allclose(np64(w).sum(1), 2.0, rtol=1e-6, atol=0)


def test_masked_rows_backward():
    x = logits(6, 32, 3, False)
    x[1] = -INF
    x[2, 5:] = -INF
    x[3, ::3] = -INF
    dw = torch.randn(6, 6, generator=torch.Generator().manual_seed(1)).cuda()
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, _ = fq.qf_moe_route(x, 6, scoring=scoring, renorm=renorm)
            g = check_backward(x, idx, dw, scoring, renorm, 1.0)
            assert not g[1].any()


def test_strides():
    big = torch.full((50, 75), float("nan"), device="cuda")
    x = big[:, 3:67]
    x.copy_(logits(50, 64, 8, False))
    idx, w = check(x, 6, "softmax")
    out = torch.full((50, 70), 7.0, device="cuda")
    check_backward(x, idx, torch.ones_like(w), "softmax", False, 1.0, d_logits=out[:, :64])
    assert bool((out[:, 64:] == 7.0).all())
    b16 = torch.full((50, 67), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 1:66]
    b16.copy_(logits(50, 65, 8, True))
    check(b16, 6, "sigmoid")


def test_graph_replays():
    x = logits(700, 128, 1, True)
    bias = torch.zeros(128, device="cuda")
    dw = torch.randn(700, 8, device="cuda")
    out = {}

    def step():
        out["i"], out["w"] = fq.qf_moe_route(x, 8, scoring="sigmoid", bias=bias, n_group=8, topk_group=4, group_rule="top2")
        out["g"] = fq.qf_moe_route_backward(x, out["i"], dw, scoring="sigmoid")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = dict(out)
    for seed in (2, 3, 4):
        x.copy_(logits(700, 128, seed, True))
        bias.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal(128) * 0.1))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in held.items()}
        step()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], out[k])


def test_empty_and_checks():
    e = torch.empty((0, 16), device="cuda")
    i, w = fq.qf_moe_route(e, 4)
    assert i.shape == (0, 4) and fq.qf_moe_route_backward(e, i, w).shape == (0, 16)
    x = logits(4, 16, 1, False)
    with pytest.raises(fq.QFError):
        fq.qf_moe_route(x, 17)
    with pytest.raises(fq.QFError):
        fq.qf_moe_route(x, 4, n_group=3)
    with pytest.raises(ValueError):
        fq.qf_moe_route(x, 4, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        fq.qf_moe_route_backward(x, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(4, 4, device="cuda"))
