"""Cases of four operators around the quantized layer: the AdamW step of the latent weights and
adapters, the routing of tokens to experts, the grouping of rows by adapter or expert, and the
low-rank adapters of many requests beside one shared projection.

``run`` computes an operator in its plain form (elementary torch operations), or, where ``own``
is set, through the library's entry points.  Formulas, with every product and sum rounded to fp32
unless said otherwise:

adamw       m = b1 m + (1 - b1) g;  v = b2 v + ((1 - b2) g) g;
            p = p (1 - lr wd) - (lr / (1 - b1^t)) (m / (sqrt(v) / sqrt(1 - b2^t) + eps));
            a bf16 copy of p.  States in fp32, or in 8 bits: blocks of 256 elements of a tensor hold
            E4M3 codes of m and of sqrt(v) with an fp32 scale (largest magnitude / 448), rounded
            stochastically with 16 bits of a hash of (seed, step, element index) each.
route       scores s = softmax(x) or sigmoid(x) of a token's logits; selection by s + bias within
            the best groups of experts; weights s[chosen] (divided by their sum) * scale.
route_bwd   the gradient of those weights with respect to the logits.
plan        stable grouping of rows by id: offsets, order, and a table of 32-row tiles.
lora        y[row] += scale[e] * B[e] (A[e] x[row]) with e = ids[row] (none for a negative id).
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256          # elements of an 8-bit state block
TILE = 32            # rows of a plan's tile
LR, BETA1, BETA2, EPS = 2e-5, 0.9, 0.999, 1e-8

# The four fused matrices of the 8B layer (rows * cols), as the other benchmarks have them.
DENSE_LAYER = "25165824,117440512,58720256,16777216"


def listed():
    return [
        # rank-16 adapters of one 8B layer: A and B of each matrix, a few hundred thousand elements
        dict(name="adamw32_adapters", op="adamw", bits=32, grad="f32", copy=True,
             sizes="65536,98304,65536,458752,229376,65536,65536,65536"),
        # the latent weights of the 8B layer, fp32 states, the straight-through fp32 gradient
        dict(name="adamw32_dense_layer", op="adamw", bits=32, grad="f32", copy=True, sizes=DENSE_LAYER),
        # the same with 8-bit states and the bf16 gradient of the matrix product
        dict(name="adamw8_dense_layer", op="adamw", bits=8, grad="bf16", copy=True, sizes=DENSE_LAYER),
        # adapters of an experts' share: many tensors of odd sizes, 8-bit states
        dict(name="adamw8_many", op="adamw", bits=8, grad="f32", copy=True,
             sizes=",".join(str(s) for s in [16 * 1536, 1536 * 16, 1000003, 77, 4096, 16 * 4097] * 20)),
        # one decode step of a small batch
        dict(name="route_decode", op="route", T=7, E=128, k=8, dtype="f32", scoring="softmax", bias=False,
             groups=1, kept=1, rule="max", renorm=True, scale=1.0),
        # a long prefill, sigmoid scores with a balance bias, experts in groups
        dict(name="route_grouped", op="route", T=32768, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True,
             groups=8, kept=4, rule="top2", renorm=True, scale=2.5),
        # training batches: the gradient of renormalised and of plain softmax weights
        dict(name="route_bwd_renorm", op="route_bwd", T=32768, E=128, k=8, dtype="bf16", scoring="softmax", renorm=True,
             scale=1.0),
        dict(name="route_bwd_plain", op="route_bwd", T=4099, E=128, k=6, dtype="f32", scoring="softmax", renorm=False,
             scale=16.0),
        # requests of a decode step; token-expert pairs of a long prefill
        dict(name="plan_decode", op="plan", n=61, ids=40, none=0.1),
        dict(name="plan_pairs", op="plan", n=262144, ids=256, none=0.0),
        # a decode step over many adapters, and a ragged prefill of a few long requests
        dict(name="lora_decode", op="lora", T=64, K=4096, N=6144, r=16, E=40, spread="mixed", none=0.1),
        dict(name="lora_prefill", op="lora", T=16384, K=4096, N=6144, r=16, E=24, spread="runs", none=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "route", "route_bwd", "plan", "lora"])
    if op == "adamw":
        many = rng.random() < 0.5
        n = rng.randint(8, 150) if many else rng.randint(1, 6)
        sizes = [_log(rng, 1, 1 << 20 if many else 3 << 23) for _ in range(n)]
        return dict(op=op, bits=rng.choice([8, 32]), grad=rng.choice(["f32", "bf16"]), copy=rng.random() < 0.7,
                    sizes=",".join(map(str, sizes)))
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 5, 8]) if op == "route" else 1
        E = groups * max(1, _log(rng, 4, 256) // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, max(1, min(16, E // groups * kept)))
        T = _log(rng, 1, 32768)
        c = dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["f32", "bf16"]), scoring=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, kept=kept, rule=rng.choice(["max", "top2"]))
        return c
    if op == "plan":
        return dict(op=op, n=_log(rng, 1, 262144), ids=_log(rng, 1, 1024), none=rng.choice([0.0, 0.1, 0.9]))
    T = _log(rng, 1, 8192)
    return dict(op=op, T=T, K=32 * rng.randint(8, 160), N=rng.randint(200, 6144), r=rng.choice([4, 8, 16, 24, 32, 64]),
                E=_log(rng, 1, 64), spread=rng.choice(["mixed", "runs"]), none=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs ----
def _layout(sizes):
    """Tensors in one flat buffer, each in a slot of whole 256-element blocks."""
    n = np.array([int(s) for s in sizes.split(",")], dtype=np.int64)
    blocks = (n + BLOCK - 1) // BLOCK
    first = np.concatenate([[0], np.cumsum(blocks)])
    owner = np.repeat(np.arange(len(n)), blocks)
    at = (np.arange(first[-1]) - first[owner]) * BLOCK      # element index of each block in its tensor
    return n, first, owner, at


def _prepare_adamw(case, gen, dev):
    n, first, owner, at = _layout(case["sizes"])
    blocks = int(first[-1])
    ow, at = torch.from_numpy(owner).to(dev), torch.from_numpy(at).to(dev)
    left = torch.from_numpy(n).to(dev)[ow] - at              # elements of the block that the tensor has
    pad = torch.arange(BLOCK, device=dev)[None, :] >= left[:, None]

    def noise(scale):
        return torch.randn((blocks, BLOCK), generator=gen, device=dev).mul_(scale).masked_fill_(pad, 0)

    s = dict(case=case, op="adamw", step=20, seed=12345, owner=ow, at=at, n=n, first=first)
    # gradients of a weight differ by rows and outliers, so a block's magnitudes spread over decades
    size = torch.exp(1.5 * torch.randn((blocks, BLOCK), generator=gen, device=dev)).mul_(2e-4)
    s["p"] = noise(0.02)
    g = noise(1.0).mul_(size)
    s["g"] = g.bfloat16() if case["grad"] == "bf16" else g
    m = noise(0.3).mul_(size)
    r = (noise(0.3).abs_().add_(0.7).mul_(size * 0.14)).masked_fill_(pad, 0)
    del size, g
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", r)):
            sc = x.abs().amax(1) / 448.0
            y = (x / sc.clamp_min(1e-30)[:, None]).clamp_(-448, 448)
            if name == "v":
                y = torch.where(y > 0, y.clamp_min(2.0 ** -9), y)
            s[name] = y.to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = sc
    else:
        s["m"], s["v"] = m, r.mul_(r)
    del m, r, pad
    s["p16"] = s["p"].bfloat16() if case["copy"] else None
    # matrices decay, every third tensor (a vector's stand-in) does not
    s["decay"] = [0.0 if i % 3 == 2 else 0.1 for i in range(len(n))]
    s["keep"] = torch.tensor([1.0 - LR * d for d in s["decay"]], dtype=torch.float64).float().to(dev)
    return s


def _ids(T, E, spread, none, gen, dev):
    if spread == "runs":       # requests one after another, each with its own adapter
        cuts = torch.sort(torch.randint(0, T + 1, (max(1, E - 1),), generator=gen, device=dev)).values
        run = torch.searchsorted(cuts, torch.arange(T, device=dev), right=True)
        ids = torch.randperm(E, generator=gen, device=dev)[run.clamp_max(E - 1)]
    else:
        ids = torch.randint(0, E, (T,), generator=gen, device=dev)
    drop = torch.rand((T,), generator=gen, device=dev) < none
    return torch.where(drop, -1, ids).int()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    if op == "adamw":
        s = _prepare_adamw(case, gen, dev)
        if own:                # the descriptors of the tensors, which a training program keeps
            import fp4_fake_quant_amd as fq
            items = []
            for i, n in enumerate(s["n"].tolist()):
                b, e = int(s["first"][i]), int(s["first"][i + 1])
                flat = {k: s[k][b:e].reshape(-1)[:n] for k in ("p", "g", "m", "v")}
                flat["p16"] = s["p16"][b:e].reshape(-1)[:n] if case["copy"] else None
                if case["bits"] == 8:
                    flat.update(m_scale=s["m_scale"][b:e], v_scale=s["v_scale"][b:e])
                items.append(dict(flat, weight_decay=s["decay"][i]))
            s["batch"] = fq.AdamwBatch(items, state_bits=case["bits"])
        return s
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        x = torch.randn((T, E), generator=gen, device=dev) * 1.5
        x = x.bfloat16() if case["dtype"] == "bf16" else x
        s = dict(case=case, op=op, x=x)
        if op == "route":
            s["bias"] = torch.randn((E,), generator=gen, device=dev) * 0.05 if case["bias"] else None
        else:
            s["dw"] = torch.randn((T, k), generator=gen, device=dev)
            s["indices"] = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
        return s
    if op == "plan":
        return dict(case=case, op=op, ids=_ids(case["n"], case["ids"], "mixed", case["none"], gen, dev))
    T, K, N, r, E = (case[c] for c in ("T", "K", "N", "r", "E"))
    s = dict(case=case, op=op, ids=_ids(T, E, case["spread"], case["none"], gen, dev))
    s["X"] = torch.randn((T, K), generator=gen, device=dev).bfloat16()
    s["A"] = (torch.randn((E, r, K), generator=gen, device=dev) / math.sqrt(K)).bfloat16()
    s["B"] = (torch.randn((E, N, r), generator=gen, device=dev) * 0.1).bfloat16()
    s["scale"] = torch.rand((E,), generator=gen, device=dev) + 0.5
    s["Y"] = torch.randn((T, (N + 7) // 8 * 8), generator=gen, device=dev).bfloat16()[:, :N]
    return s


# -------------------------------------------------------------- plain forms ----
def _hash(x):
    """A 32-bit finaliser (xor-shifts and two odd multipliers) on int64 tensors or ints below 2^32."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _decode8(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[:, None]


def _encode8(x, rnd, lift):
    """Codes and scales of blocks x [blocks, 256]: stochastic rounding of |x| / scale onto E4M3 with
    rnd (16 bits); `lift`: a positive value is never rounded to zero."""
    top = x.abs().amax(1)
    live = top >= 2.0 ** -100
    scale = torch.where(live, top * (1.0 / 448.0), 0.0)
    inv = torch.where(live, torch.reciprocal(scale), 0.0)
    y = (x.abs() * inv[:, None]).clamp_max_(448.0)
    small = torch.floor(y * 512.0 + rnd.float() * 2.0 ** -16).int()
    large = ((y.view(torch.int32) + (rnd << 4).int()) >> 20) - 960
    code = torch.where(y < 2.0 ** -6, small, large)
    if lift:
        code = torch.where(y > 0, code.clamp_min(1), code)
    code = code + torch.where(x < 0, 128, 0)
    return code.to(torch.uint8), scale


def _plain_adamw(s, step):
    bits8 = s["case"]["bits"] == 8
    g = s["g"].float()
    m = _decode8(s["m"], s["m_scale"]) if bits8 else s["m"]
    if bits8:
        r = _decode8(s["v"], s["v_scale"])
        v = r * r
    else:
        v = s["v"]
    size = LR / (1.0 - BETA1 ** step)
    root = 1.0 / math.sqrt(1.0 - BETA2 ** step)
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    r = v.sqrt()
    p = s["p"] * s["keep"][s["owner"]][:, None] - (m / (r * root + EPS)) * size
    s["p"].copy_(p)
    if s["p16"] is not None:
        s["p16"].copy_(p)
    if bits8:
        key = _hash(s["seed"] ^ _hash(step))
        h = _hash((s["at"][:, None] + torch.arange(BLOCK, device=p.device)[None, :] + key) & 0xFFFFFFFF)
        for name, x, rnd in (("m", m, h & 0xFFFF), ("v", r, h >> 16)):
            code, scale = _encode8(x, rnd, name == "v")
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _scores(x, scoring):
    """Scores in 64 bits; a logit of minus infinity scores zero."""
    x = x.double()
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _best(v, k):
    """Indices of the k largest along the last axis, ties to the lowest index."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(s):
    c, x = s["case"], s["x"]
    T, E, G = c["T"], c["E"], c["groups"]
    sc = _scores(x, c["scoring"])
    key = sc + s["bias"].double() if c["bias"] else sc
    if G > 1:
        per = key.view(T, G, E // G)
        if c["rule"] == "top2" and E // G > 1:
            g = torch.gather(per, 2, _best(per, 2)).sum(2)
        else:
            g = per.amax(2)
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, _best(g, c["kept"]), True)
        key = torch.where(keep[:, :, None], per, -math.inf).reshape(T, E)
    idx = _best(key, c["k"])
    w = torch.gather(sc, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * c["scale"]).float()


def _plain_route_bwd(s):
    c, x, dw, idx = s["case"], s["x"].float(), s["dw"], s["indices"].long()
    if c["scoring"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        sc = e / e.sum(1, keepdim=True)
    u = torch.gather(sc, 1, idx)
    du = dw * c["scale"]
    if c["renorm"]:
        total = u.sum(1, keepdim=True)
        du = (du - (du * u).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(sc).scatter_(1, idx, du)
    if c["scoring"] == "sigmoid":
        dx = ds * sc * (1.0 - sc)
    else:
        dx = sc * (ds - (ds * sc).sum(1, keepdim=True))
    return dx.to(s["x"].dtype)


def _plain_plan(s):
    ids, n_ids = s["ids"].long(), s["case"]["ids"]
    n = ids.numel()
    ids = torch.where((ids >= 0) & (ids < n_ids), ids, n_ids)
    key, order = torch.sort(ids, stable=True)
    order = torch.where(key < n_ids, order, -1)
    offsets = torch.searchsorted(key, torch.arange(n_ids + 1, device=ids.device))
    tiles = (offsets[1:] - offsets[:-1] + TILE - 1) // TILE
    last = torch.cumsum(tiles, 0)
    t = torch.arange((n + TILE - 1) // TILE + min(n, n_ids), device=ids.device)
    e = torch.searchsorted(last, t, right=True)
    c = e.clamp_max(n_ids - 1)
    first = offsets[c] + TILE * (t - (last[c] - tiles[c]))
    used = e < n_ids
    table = torch.stack([torch.where(used, e, -1), torch.where(used, first, 0)], 1)
    return offsets.int(), order.int(), table.int()


def _plain_lora(s):
    X, A, B, ids = s["X"].float(), s["A"].float(), s["B"].float(), s["ids"].long()
    E, r, K = A.shape
    # every row against every adapter in one product; the rows' own adapters are kept
    S = (X @ A.reshape(E * r, K).t()).view(-1, E, r)
    S = S * (torch.arange(E, device=ids.device)[None, :] == ids[:, None])[:, :, None] * s["scale"][None, :, None]
    Y = s["Y"].float() + S.reshape(-1, E * r) @ B.permute(0, 2, 1).reshape(E * r, -1)
    s["Y"].copy_(Y)
    return s["Y"]


# ------------------------------------------------------------------- passes ----
def _adamw_outputs(s):
    out = [s["p"]] + ([s["p16"]] if s["p16"] is not None else [])
    if s["case"]["bits"] == 8:     # a code's value, and the scale of its block
        f8 = torch.float8_e4m3fn
        return out + [s["m"].view(f8), s["m_scale"], s["v"].view(f8), s["v_scale"]]
    return out + [s["m"], s["v"]]


def run(state):
    s = state
    c = s["case"]
    if s["op"] == "adamw":
        s["step"] += 1
        if own:
            import fp4_fake_quant_amd as fq
            fq.qf_adamw_step(s["batch"], LR, s["step"], BETA1, BETA2, EPS, seed=s["seed"])
        else:
            _plain_adamw(s, s["step"])
        return _adamw_outputs(s)
    if not own:
        return {"route": _plain_route, "route_bwd": _plain_route_bwd, "plan": _plain_plan, "lora": _plain_lora}[s["op"]](s)
    import fp4_fake_quant_amd as fq
    if s["op"] == "route":
        return fq.qf_moe_route(s["x"], c["k"], scoring=c["scoring"], bias=s["bias"], n_group=c["groups"],
                               topk_group=c["kept"], group_rule=c["rule"], renorm=c["renorm"], scale=c["scale"])
    if s["op"] == "route_bwd":
        return fq.qf_moe_route_backward(s["x"], s["indices"], s["dw"], scoring=c["scoring"], renorm=c["renorm"],
                                        scale=c["scale"])
    if s["op"] == "plan":
        plan = fq.qf_row_plan(s["ids"], c["ids"])
        return plan.offsets, plan.order, plan.tiles
    return fq.qf_lora_apply(s["X"], s["A"], s["B"], s["ids"], s["Y"], scale=s["scale"])


# --------------------------------------------------------------------- work ----
def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(int(v) for v in case["sizes"].split(","))
        per = (4 if case["grad"] == "f32" else 2) + 8 + (16 if case["bits"] == 32 else 4) + (2 if case["copy"] else 0)
        return dict(bytes=n * per + (16 * n // BLOCK if case["bits"] == 8 else 0), flops=16 * n)
    if op in ("route", "route_bwd"):
        T, E, k, sz = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return dict(bytes=T * E * sz + 8 * T * k + (4 * E if case["bias"] else 0), flops=8 * T * E)
        reads = k if case["renorm"] or case["scoring"] == "sigmoid" else E
        return dict(bytes=T * (E * sz + reads * sz + 8 * k), flops=6 * T * reads)
    if op == "plan":
        n, ids = case["n"], case["ids"]
        return dict(bytes=8 * n + 4 * (ids + 1) + 8 * ((n + TILE - 1) // TILE + min(n, ids)), flops=n)
    T, K, N, r, E = (case[c] for c in ("T", "K", "N", "r", "E"))
    rows = T * (1.0 - case["none"])
    return dict(bytes=rows * (2 * K + 4 * N) + 4 * T + min(E, T) * (2 * r * (K + N) + 4), flops=2 * rows * r * (K + N))


# -------------------------------------------------------------------- exact ----
def _exact_adamw(s):
    step, bits8 = s["step"] + 1, s["case"]["bits"] == 8
    p = s["p"].double()
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().to(p.device)
    g = s["g"].double()
    if bits8:
        m = table[s["m"].int()] * s["m_scale"].double()[:, None]
        v = (table[s["v"].int()] * s["v_scale"].double()[:, None]) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    wd = torch.tensor(s["decay"], dtype=torch.float64, device=p.device)[s["owner"]][:, None]
    p = p - LR * wd * p - LR * (m / (1 - BETA1 ** step)) / (torch.sqrt(v / (1 - BETA2 ** step)) + EPS)
    outs = [p] + ([p] if s["p16"] is not None else [])
    if not bits8:
        return outs + [m, v]
    for name, x in (("m", m), ("v", v.sqrt())):
        # a stochastically rounded code has no 64-bit value of its own: its scale has
        outs += [None, x.abs().amax(1) / 448.0]
    return outs


def _exact_route(s):
    c, x = s["case"], s["x"].double().cpu().numpy()
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    if c["scoring"] == "sigmoid":
        sc = 1.0 / (1.0 + np.exp(-x))
    else:
        sc = np.exp(x - x.max(1, keepdims=True))
        sc /= sc.sum(1, keepdims=True)
    key = sc + s["bias"].double().cpu().numpy() if c["bias"] else sc.copy()
    if G > 1:
        per = np.sort(key.reshape(T, G, E // G), axis=2)
        g = per[:, :, -2:].sum(2) if c["rule"] == "top2" else per[:, :, -1]
        lose = np.argsort(-g, axis=1, kind="stable")[:, c["kept"]:]
        np.put_along_axis(key.reshape(T, G, E // G), lose[:, :, None], -np.inf, axis=1)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(sc, idx, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return idx.astype(np.int32), w * c["scale"]


def _exact_route_bwd(s):
    c, x, dw, idx = s["case"], s["x"].double(), s["dw"].double(), s["indices"].long()
    sc = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
    u = sc.gather(1, idx)
    p = u / u.sum(1, keepdim=True)
    dx = torch.zeros_like(x)
    if c["renorm"]:
        rest = dw - (dw * p).sum(1, keepdim=True)
        part = p * rest if c["scoring"] == "softmax" else p * (1 - u) * rest
    elif c["scoring"] == "sigmoid":
        part = dw * u * (1 - u)
    else:
        part = u * dw
        dx = -sc * part.sum(1, keepdim=True)
    return dx.scatter_add(1, idx, part) * c["scale"]


def _exact_lora(s):
    Y, ids = s["Y"].double(), s["ids"]
    for e in range(s["case"]["E"]):
        rows = (ids == e).nonzero()[:, 0]
        t = (s["X"][rows].double() @ s["A"][e].double().t()) * s["scale"][e].double()
        Y[rows] += t @ s["B"][e].double().t()
    return Y


def exact(case, seed):
    if case["op"] == "plan":       # whole numbers alone
        return None
    s = prepare(case, seed)
    return {"adamw": _exact_adamw, "route": _exact_route, "route_bwd": _exact_route_bwd, "lora": _exact_lora}[case["op"]](s)
