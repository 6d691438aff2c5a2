"""qf_row_plan and qf_lora_apply on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import fp4_fake_quant_amd as fq
from oracle import primitives as prim
from oracle import rows
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu
INF = float("inf")


def ids_of(n, n_ids, seed, none=0.1, runs=False):
    rng = np.random.default_rng(seed)
    ids = np.sort(rng.integers(0, n_ids, n)) if runs else rng.integers(0, n_ids, n)
    ids = np.where(rng.random(n) < none, rng.choice([-1, -7, n_ids, 2 ** 31 - 1], n), ids)
    return ids.astype(np.int32)


def check_plan(ids, n_ids):
    p = fq.qf_row_plan(torch.from_numpy(ids).cuda(), n_ids)
    for got, want, name in zip((p.offsets, p.order, p.tiles), rows.plan(ids, n_ids), ("offsets", "order", "tiles")):
        assert np.array_equal(got.cpu().numpy(), want), f"{name}, n={ids.size}, n_ids={n_ids}"
    return p


@pytest.mark.parametrize("n", [0, 1, 31, 64, 65, 511, 513, 2048, 2049, 6000, 32768, 32769, 131072, 300001])
@pytest.mark.parametrize("n_ids", [1, 2, 5, 128, 1000, 1024])
def test_plan(n, n_ids):
    check_plan(ids_of(n, n_ids, n + n_ids, runs=n % 2 == 1), n_ids)


@pytest.mark.parametrize("n", [70, 9000])
def test_plan_one_group_and_none(n):
    check_plan(np.full(n, 3, np.int32), 5)
    check_plan(np.full(n, -1, np.int32), 5)
    a = np.full(n, -1, np.int32)
    a[-1] = 4
    check_plan(a, 5)


def bf(rng, shape, scale=1.0):
    return prim.f32_to_bf16((rng.standard_normal(shape) * scale).astype(np.float32))


def case(T, K, N, r, E, seed, none=0.1, per=1, ldx=None, ldy=None, runs=False):
    rng = np.random.default_rng(seed)
    c = dict(X=bf(rng, (-(-T // per), K)), A=bf(rng, (E, r, K), K ** -0.5), B=bf(rng, (E, N, r), 0.2), Y=bf(rng, (T, N)),
             scale=(rng.random(E) + 0.5).astype(np.float32), ids=ids_of(T, E, seed + 1, none, runs), per=per)
    ldx, ldy = ldx or K, ldy or N
    d = dict(A=dev(c["A"]), B=dev(c["B"]), scale=torch.from_numpy(c["scale"]).cuda(), ids=torch.from_numpy(c["ids"]).cuda())
    d["X"] = torch.full((c["X"].shape[0], ldx), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :K]
    d["X"].copy_(dev(c["X"]))
    d["Yfull"] = torch.full((T, ldy), 7.0, dtype=torch.bfloat16, device="cuda")
    d["Y"] = d["Yfull"][:, :N]
    d["Y"].copy_(dev(c["Y"]))
    return c, d


def check_apply(c, d, planned, scaled=True):
    K, N, r = c["X"].shape[1], c["Y"].shape[1], c["A"].shape[1]
    f = prim.bf16_to_f32
    scale = c["scale"] if scaled else None
    y, P, y0 = rows.apply(f(c["X"]), f(c["A"]), f(c["B"]), c["ids"], f(c["Y"]), scale, c["per"])
    d["Y"].copy_(dev(c["Y"]))
    kw = dict(scale=d["scale"] if scaled else None, rows_per_x=c["per"])
    if planned:
        plan = fq.qf_row_plan(d["ids"], c["A"].shape[0])
        fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], plan, d["Y"], **kw)
    else:
        fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"], d["Y"], **kw)
    got = host(d["Y"])
    err = np.abs(f(got).astype(np.float64) - y)
    bound = rows.apply_bound(y, P, y0, K, r)
    assert np.all(err <= bound), f"worst {np.max(err / np.maximum(bound, 1e-300))} of the bound"
    none = (c["ids"] < 0) | (c["ids"] >= c["A"].shape[0])
    assert np.array_equal(got[none], c["Y"][none])
    if d["Yfull"].shape[1] > N:
        assert bool((d["Yfull"][:, N:] == 7.0).all())
    return got


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("T,K,N,r,E", [
    (1, 8, 1, 1, 1), (1, 4096, 512, 16, 3), (3, 72, 17, 3, 2), (64, 2056, 300, 16, 9), (256, 2056, 300, 16, 9), (257, 2056, 300, 16, 9), (2, 8200, 2100, 17, 3), (5, 520, 70, 128, 2), (32, 264, 66, 40, 5), (33, 264, 66, 40, 5), (64, 520, 1100, 64, 5), (65, 520, 70, 64, 5), (128, 264, 130, 32, 7), (129, 264, 130, 32, 7), (1, 4096, 70, 65, 2), (9, 1000, 130, 72, 2),
    (33, 256, 64, 32, 1), (100, 520, 130, 33, 2), (97, 128, 257, 64, 5), (200, 200, 72, 128, 3), (430, 64, 40, 100, 40), (500, 640, 72, 128, 3), (444, 520, 130, 33, 2),
    (300, 96, 2000, 8, 1000), (1000, 1024, 96, 4, 7)])
def test_apply(T, K, N, r, E, planned):
    c, d = case(T, K, N, r, E, T + r)
    got = check_apply(c, d, planned)
    assert np.array_equal(check_apply(c, d, planned), got)                 # the same bits again


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("T", [40, 700])
def test_apply_strides_runs_no_scale(T, planned):
    c, d = case(T, 320, 136, 16, 6, 5, ldx=336, ldy=144, runs=True)
    check_apply(c, d, planned, scaled=False)
    c, d = case(T, 320, 133, 16, 6, 6, ldx=328, ldy=135)                   # Y rows of 2-byte alignment
    check_apply(c, d, planned)


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("T", [48, 1200])
def test_apply_token_expert_pairs(T, planned):
    """Rows t * k + j of Y share X's row t."""
    c, d = case(T, 256, 192, 16, 32, 8, per=8)
    check_apply(c, d, planned)
    c, d = case(T + 3, 256, 192, 16, 32, 9, per=8)                         # a last row of X with fewer
    check_apply(c, d, planned)


@pytest.mark.parametrize("T", [24, 500])
def test_one_row_of_x_for_all(T):
    c, d = case(T, 96, 72, 16, 3, 33, per=T)
    for planned in (False, True):
        got = check_apply(c, d, planned)
        for per in (T + 1, (1 << 24) + 1, 1 << 40):
            y = dev(c["Y"])
            if planned:
                fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], fq.qf_row_plan(d["ids"], 3), y, scale=d["scale"], rows_per_x=per)
            else:
                fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"], y, scale=d["scale"], rows_per_x=per)
            assert np.array_equal(host(y), got)


@pytest.mark.parametrize("planned", [False, True])
def test_apply_all_and_none(planned):
    for T in (20, 500):
        c, d = case(T, 128, 96, 16, 4, 10, none=1.1)
        check_apply(c, d, planned)
        c, d = case(T, 128, 96, 16, 4, 11, none=0.0)
        c["ids"][:] = 2
        d["ids"].fill_(2)
        check_apply(c, d, planned)


def test_apply_beyond_the_caches():
    """Y of more than 160 MiB takes another cache policy; sampled rows against the oracle."""
    T, K, N, r, E = 7100, 64, 12000, 16, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    X, Y = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, K), (T, N)))
    A, B = torch.randn((E, r, K), generator=g, device="cuda").bfloat16(), torch.randn((E, N, r), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, E, (T,), generator=g, device="cuda").int()
    before = Y.clone()
    fq.qf_lora_apply(X, A, B, ids, Y)
    pick = np.r_[0:40, 3000:3040, T - 40:T]
    f = prim.bf16_to_f32
    at = torch.from_numpy(pick).cuda()
    y, P, y0 = rows.apply(f(host(X[at])), f(host(A)), f(host(B)), ids[at].cpu().numpy(), f(host(before[at])))
    assert np.all(np.abs(f(host(Y[at])).astype(np.float64) - y) <= rows.apply_bound(y, P, y0, K, r))
    none = (ids < 0)
    assert torch.equal(Y[none], before[none])


def test_rows_without_adapter_are_not_read():
    """NaN in the X rows of requests without an adapter reaches nothing."""
    for T in (30, 500):
        c, d = case(T, 128, 96, 16, 4, 12, none=0.5)
        none = torch.from_numpy((c["ids"] < 0) | (c["ids"] >= 4)).cuda()
        d["X"][none] = float("nan")
        check_apply(c, d, False)
        check_apply(c, d, True)


@pytest.mark.parametrize("r", [1, 8, 16, 24, 64, 100])
@pytest.mark.parametrize("T", [24, 500])
def test_infinite_and_huge_inner_products(T, r):
    """A x that overflows, or holds an infinity, gives the infinities of the formula in its own row
    alone; A x between the largest bf16 and the largest fp32 stays finite."""
    K, N, E = 64, 72, 2
    X, A, B = torch.zeros(T, K), torch.zeros(E, r, K), torch.zeros(E, N, r)
    big = torch.finfo(torch.bfloat16).max
    X[:, 0] = 1.0
    X[3, 1], X[5, 1], X[9, 1] = INF, big, big
    X[9, 2] = 1.5 * 2.0 ** 119                           # above half a bf16 step past the largest
    A[:, :, 0], A[:, :, 1], A[:, :, 2] = 0.5, 1.0, 1.0
    A[1, :, 1] = 4.0                                     # overflows
    B[:] = torch.where(torch.arange(N) % 3 == 0, -1.0, 1.0)[None, :, None] * 2.0 ** -100
    Y = torch.arange(N).float().repeat(T, 1)
    ids = torch.arange(T) % 2
    ids[9], ids[5] = 0, 1
    s = (X * A[ids, 0]).sum(1, keepdim=True)             # the same for all adapter rows
    assert s[3, 0] == INF and s[5, 0] == INF and big + 2.0 ** 119 < s[9, 0] < INF
    want = Y + s * B[0, :, 0] * r
    X, A, B, Y, ids = (t.cuda() for t in (X.bfloat16(), A.bfloat16(), B.bfloat16(), Y.bfloat16(), ids.int()))
    plan = fq.qf_row_plan(ids, E)
    for planned in (False, True):
        y = Y.clone()
        if planned:
            fq.qf_lora_apply_planned(X, A, B, plan, y)
        else:
            fq.qf_lora_apply(X, A, B, ids, y)
        y = y.float().cpu()
        assert torch.equal(y.isinf(), want.isinf()) and not bool(y.isnan().any())
        assert torch.equal(y[want.isinf()], want[want.isinf()])
        fin = want.isfinite()                            # one bf16 rounding, the parts of A x 2^-17, fp32 sums
        assert bool(((y - want).abs()[fin] <= (2.0 ** -8 + 2.0 ** -14) * want.abs()[fin]).all())


@pytest.mark.parametrize("r", [4, 8, 16, 24, 72])
@pytest.mark.parametrize("T", [24, 500])
def test_bad_adapter_values_stay_in_their_outputs(T, r):
    """An infinity or NaN in B[e][n] reaches column n of e's rows alone, one in another adapter nothing."""
    c, d = case(T, 64, 70, r, 5, 31, none=0.1)
    d["ids"][d["ids"] == 4] = 0                          # adapter 4 has no rows
    own = (d["ids"] == 2).nonzero()[:, 0]
    for planned in (False, True):
        out = []
        for bad in (None, INF, float("nan")):
            A, B, Y = d["A"].clone(), d["B"].clone(), d["Y"].clone()
            if bad is not None:
                B[2, 69, r - 1], B[2, 5, 0] = bad, bad
                A[4], B[4] = bad, bad
            if planned:
                fq.qf_lora_apply_planned(d["X"], A, B, fq.qf_row_plan(d["ids"], 5), Y)
            else:
                fq.qf_lora_apply(d["X"], A, B, d["ids"], Y)
            out.append(Y)
        for Y in out[1:]:
            assert not bool(Y[own][:, [5, 69]].isfinite().any())
            Y[own[:, None], torch.tensor([[5, 69]], device="cuda")] = out[0][own[:, None], torch.tensor([[5, 69]], device="cuda")]
            assert torch.equal(Y, out[0])


def test_forms_agree_with_a_prefix():
    """A plan of fewer ids than adapters, and an empty batch."""
    c, d = case(500, 128, 96, 16, 6, 13, none=0.0)
    c["ids"] %= 4
    d["ids"] %= 4
    plan = fq.qf_row_plan(d["ids"], 4)
    fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], plan, d["Y"], scale=d["scale"])
    got = host(d["Y"])
    assert np.array_equal(got, check_apply(c, d, True))
    e = torch.empty((0, 96), dtype=torch.bfloat16, device="cuda")
    fq.qf_lora_apply(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), d["A"], d["B"],
                     torch.empty(0, dtype=torch.int32, device="cuda"), e)


@pytest.mark.parametrize("r", [8, 40, 128])
def test_foreign_plans_stay_inside_the_call(r):
    """Plan arrays that hold other numbers (another batch's, or never filled) reach no memory outside
    the workspace and Y's rows, whatever they are."""
    T, K, N, E = 77, 64, 70, 5
    _, d = case(T, K, N, r, E, 41)
    need = fq.qf_lora_apply_workspace(T, K, r, E, True)
    rng = np.random.default_rng(r)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    for values in ([lo], [lo, 0, 1, 2, 3, 4, 76], [hi, hi - 31, 0, 4], [-1, 0, 1, 40, 76, 77, 78], [lo, lo + 1, lo + 77, 1, 2, 76, hi]):
        plan = fq.RowPlan(T, E, "cuda")
        for t in (plan.offsets, plan.order, plan.tiles):
            t.copy_(torch.from_numpy(rng.choice(np.array(values, np.int32), t.shape)))
        plan.tiles[:len(plan.tiles) // 2, 0] = torch.from_numpy(rng.integers(0, E, len(plan.tiles) // 2).astype(np.int32))
        plan.tiles[:len(plan.tiles) // 2, 1] = torch.from_numpy(rng.integers(0, T, len(plan.tiles) // 2).astype(np.int32))
        ws = torch.full((need + 65536,), 77, dtype=torch.uint8, device="cuda")
        Y = torch.full((T + 64, N + 2), 7.0, dtype=torch.bfloat16, device="cuda")
        fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], plan, Y[32:32 + T, :N], ws=ws[32768:32768 + need])
        torch.cuda.synchronize()
        assert bool((ws[:32768] == 77).all()) and bool((ws[32768 + need:] == 77).all())
        assert bool((Y[:32] == 7.0).all()) and bool((Y[32 + T:] == 7.0).all()) and bool((Y[:, N:] == 7.0).all())


@pytest.mark.parametrize("T", [24, 5000])
def test_graph_replays(T):
    """Plan and adapters captured once; ids, X and Y change between replays."""
    E = 5
    _, d = case(T, 256, 160, 16, E, 14)
    ws = torch.empty(fq.qf_lora_apply_workspace(T, 256, 16, E), dtype=torch.uint8, device="cuda")

    def step():
        fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"], d["Y"], scale=d["scale"], ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (21, 22, 23):
        c, n = case(T, 256, 160, 16, E, seed, runs=seed == 22)
        for k in ("X", "ids", "Y", "A", "B", "scale"):
            d[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        got = host(d["Y"])
        assert np.array_equal(got, check_apply(c, n, False))


def test_binding_checks():
    _, d = case(10, 64, 40, 8, 4, 1)
    with pytest.raises(ValueError):
        fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"][:9], d["Y"])
    with pytest.raises(ValueError):
        fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"], d["Y"], rows_per_x=2)
    with pytest.raises(ValueError):
        fq.qf_lora_apply(d["X"], d["A"][:3], d["B"], d["ids"], d["Y"])
    with pytest.raises(ValueError):
        fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], fq.qf_row_plan(d["ids"], 5), d["Y"])
    with pytest.raises(TypeError):
        fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], d["ids"], d["Y"])
    with pytest.raises(ValueError):
        fq.qf_row_plan(d["ids"], 1025)
    with pytest.raises(fq.QFError):
        fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], fq.qf_row_plan(d["ids"], 4), d["Y"],
                                 ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_workspace_must_be_one_run_of_memory():
    _, d = case(1000, 64, 40, 8, 4, 1)
    plan = fq.qf_row_plan(d["ids"], 4)
    need = max(fq.qf_lora_apply_workspace(1000, 64, 8, 4, p) for p in (False, True))
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need),
               torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            fq.qf_lora_apply(d["X"], d["A"], d["B"], d["ids"], d["Y"], ws=ws)
        with pytest.raises(ValueError, match="contiguous"):
            fq.qf_lora_apply_planned(d["X"], d["A"], d["B"], plan, d["Y"], ws=ws)
        with pytest.raises(ValueError, match="contiguous"):
            fq.qf_row_plan(torch.zeros(20000, dtype=torch.int32, device="cuda"), 4, ws=ws)
