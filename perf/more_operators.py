"""Cases of the operators that carry a mixture's experts, or a whole linear layer, through 8-bit
matrix products: rows moved into expert order and back, block quantization to E4M3, the gated
activation, and the products themselves.

``run`` computes an operator in its plain form (elementary torch operations in fp32), or, where
``own`` is set, through the library's entry points.  Row i = t k + j is token t's j-th expert;
position p of a row plan holds row order[p], pos[i] is its inverse (-1: no expert).  Formulas:

dispatch     out[p] = x[order[p] / k]
combine      y[t] = sum_j w[t, j] r[pos[t k + j]]
combine_bwd  dr[p] = w[i] dy[i / k], i = order[p];  dw[i] = <r[pos[i]], dy[i / k]>
quant        E4M3 codes of x / s with one fp32 scale s = max |x| / 448 per block: 128 consecutive
             elements of a row ("rows", gathered into expert order or not), 128 rows of one expert
             in a column ("cols", transposed panels for a reduction over rows), or a 128 x 128
             tile ("tiles", weights and their transpose)
swiglu       a = u g / (1 + exp(-g)) of h = [g, u], quantized in rows;  swiglu_bwd: dh from da
gemm         y = sum over blocks b of 128 of sx[m, b] sw[n / 128, b] sum_(k in b) x[m, k] w[n, k]
experts      the same with w of the expert that position p belongs to
wgrad        dw[e] = sum over the blocks of expert e's rows of sy[n, b] sx[k, b] sum dy[p, n] x[p, k],
             in bf16 as the optimizer and the straight-through accumulation read it
"""

import math

import numpy as np
import torch

own = False

B = 128              # elements of a block
TOP = 448.0          # largest E4M3 value
F8 = torch.float8_e4m3fn


def listed():
    return [
        # a decode step of a small batch: the experts' outputs back into token order
        dict(name="combine_decode", op="combine", T=7, k=8, H=2048, E=128, none=0.0),
        # a long prefill
        dict(name="combine_prefill", op="combine", T=8192, k=8, H=4096, E=64, none=0.02),
        # a training batch: gradients of the rows and of the routing weights
        dict(name="combine_bwd", op="combine_bwd", T=4099, k=6, H=4096, E=64, none=0.0),
        # tokens into expert order, quantized on the way
        dict(name="dispatch_quant", op="quant", kind="rows", gather=True, T=8192, k=8, H=4096, E=64, none=0.02),
        # a training batch's activations as panels for the weight gradient
        dict(name="quant_panels", op="quant", kind="cols", gather=False, T=4096, k=8, H=4096, E=64, none=0.0),
        # between the gate/up and the down product, forward and backward
        dict(name="swiglu_experts", op="swiglu", P=65536, I=2048),
        dict(name="swiglu_bwd_experts", op="swiglu_bwd", P=32771, I=2048),
        # the fused QKV projection of a few requests
        dict(name="gemm_decode", op="gemm", M=7, N=6144, K=4096),
        # the up projection of the 8B layer over a long batch
        dict(name="gemm_prefill", op="gemm", M=32768, N=14336, K=4096),
        # a decode step through 128 experts: some have no row, most a few
        dict(name="experts_decode", op="experts", T=61, k=8, E=128, N=1536, K=2048, none=0.0),
        # a prefill through 64 experts
        dict(name="experts_prefill", op="experts", T=4096, k=8, E=64, N=4096, K=4096, none=0.0),
        # the weight gradients of an experts' share
        dict(name="wgrad_experts", op="wgrad", T=4096, k=8, E=64, N=2048, K=2048, none=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_bwd", "quant", "quant", "swiglu", "swiglu_bwd", "gemm", "gemm", "experts",
                     "experts", "wgrad"])
    none = rng.choice([0.0, 0.0, 0.05, 0.5])
    if op in ("dispatch", "combine", "combine_bwd"):
        return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 8), H=8 * _log(rng, 2, 512), E=_log(rng, 1, 256), none=none)
    if op == "quant":
        kind = rng.choice(["rows", "cols", "tiles"])
        if kind == "tiles":
            return dict(op=op, kind=kind, E=_log(rng, 1, 8), N=16 * _log(rng, 1, 256), K=16 * _log(rng, 1, 256))
        return dict(op=op, kind=kind, gather=rng.random() < 0.5, T=_log(rng, 1, 4096), k=rng.randint(1, 8),
                    H=16 * _log(rng, 1, 256), E=_log(rng, 1, 256), none=none)
    if op in ("swiglu", "swiglu_bwd"):
        return dict(op=op, P=_log(rng, 1, 32768), I=16 * _log(rng, 1, 128))
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 8192), K=16 * _log(rng, 1, 512))
    E = _log(rng, 1, 64)
    return dict(op=op, T=_log(rng, 1, 2048), k=rng.randint(1, 8), E=E, N=8 * _log(rng, 8, 256), K=16 * _log(rng, 4, 128), none=none)


# ------------------------------------------------------------------ inputs ----
def _ids(rows, E, none, gen, dev):
    """Experts of rows, some experts better liked than others."""
    liking = torch.exp(0.4 * torch.randn((E,), generator=gen, device=dev))
    ids = torch.multinomial(liking, rows, replacement=True, generator=gen)
    drop = torch.rand((rows,), generator=gen, device=dev) < none
    return torch.where(drop, -1, ids).int()


def _sort(s, ids, E):
    """The rows in expert order, as a program keeps them beside the batch: order and its inverse,
    the experts' first positions, and on the host the rows of each."""
    n = ids.numel()
    key = torch.where(ids < 0, E, ids.long())
    key, order = torch.sort(key, stable=True)
    s["order"] = torch.where(key < E, order, -1)
    s["offsets"] = torch.searchsorted(key, torch.arange(E + 1, device=ids.device))
    at = torch.where(key < E, torch.arange(n, device=ids.device), -1)
    s["pos"] = torch.empty_like(at).scatter_(0, order, at)
    s["owner"] = torch.where(key < E, key, 0)
    counts = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    s["most"], s["used"] = max(counts + [1]), sum(counts)
    s["n_blocks"] = sum((c + B - 1) // B for c in counts)


def _span(rows, cols, gen, dev, jitter=0.5):
    """bf16 rows whose sizes differ, as activations' do."""
    x = torch.randn((rows, cols), generator=gen, device=dev)
    x *= torch.exp(jitter * torch.randn((rows, 1), generator=gen, device=dev))
    return x.bfloat16()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op, c = case["op"], case
    s = dict(case=case, op=op)
    if "T" in c:
        n, E = c["T"] * c["k"], c["E"]
        ids = _ids(n, E, c["none"], gen, dev)
        _sort(s, ids, E)
        if own:
            import fp4_fake_quant_amd as fq
            s["plan"] = fq.qf_row_plan(ids, E, positions=True)
    if op == "dispatch":
        s["x"], s["out"] = _span(c["T"], c["H"], gen, dev), torch.zeros((n, c["H"]), dtype=torch.bfloat16, device=dev)
    elif op in ("combine", "combine_bwd"):
        s["r"] = _span(n, c["H"], gen, dev)
        s["w"] = torch.softmax(torch.randn((c["T"], c["k"]), generator=gen, device=dev), 1)
        if op == "combine_bwd":
            s["dy"], s["out"] = _span(c["T"], c["H"], gen, dev), torch.zeros_like(s["r"])
    elif op == "quant" and c["kind"] == "tiles":
        s["x"] = (_span(c["E"] * c["N"], c["K"], gen, dev, 0.3) * 0.02).view(c["E"], c["N"], c["K"])
    elif op == "quant":
        H = c["H"]
        s["x"] = _span(c["T"] if c["gather"] else n, H, gen, dev)
        if c["kind"] == "rows":
            s["codes"] = torch.zeros((n, H), dtype=torch.uint8, device=dev)
            s["scales"] = torch.zeros(((H + B - 1) // B, n), dtype=torch.float32, device=dev)
        else:
            blocks = (n + B - 1) // B + min(n, E)
            s["codes"] = torch.zeros((blocks, H, B), dtype=torch.uint8, device=dev)
            s["scales"] = torch.zeros((blocks, H), dtype=torch.float32, device=dev)
    elif op in ("swiglu", "swiglu_bwd"):
        s["h"] = _span(c["P"], 2 * c["I"], gen, dev)
        if op == "swiglu_bwd":
            s["da"] = _span(c["P"], c["I"], gen, dev)
    elif op == "gemm":
        s["xc"], s["xs"] = _rows8(_span(c["M"], c["K"], gen, dev).float())
        w = _span(c["N"], c["K"], gen, dev, 0.3) * 0.02
        s["wc"], s["ws"] = _tiles8(w[None])
        s["wc"], s["ws"] = s["wc"][0], s["ws"][0]
    elif op == "experts":
        s["xc"], s["xs"] = _rows8(_span(n, c["K"], gen, dev).float())
        w = _span(E * c["N"], c["K"], gen, dev, 0.3) * 0.02
        s["wc"], s["ws"] = _tiles8(w.view(E, c["N"], c["K"]))
        s["y"] = torch.zeros((n, c["N"]), dtype=torch.bfloat16, device=dev)
    else:                                          # wgrad
        blocks = (n + B - 1) // B + min(n, E)
        for name, cols in (("y", c["N"]), ("x", c["K"])):
            codes = torch.zeros((blocks, cols, B), dtype=torch.uint8, device=dev)
            scales = torch.zeros((blocks, cols), dtype=torch.float32, device=dev)
            part = _panels8(s, _span(n, cols, gen, dev).float())
            codes[:part[0].shape[0]], scales[:part[0].shape[0]] = part
            s[name + "c"], s[name + "s"] = codes, scales
    return s


# -------------------------------------------------------------- plain forms ----
def _encode(x, top):
    """Codes and scales of x (fp32) whose blocks have the largest magnitudes `top` (kept dimensions)."""
    live = top >= 2.0 ** -100
    scale = torch.where(live, top / TOP, 0.0)
    inv = torch.where(live, TOP / top, 0.0)
    return (x * inv).clamp_(-TOP, TOP).to(F8).view(torch.uint8), scale


def _rows8(x):
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, -cols % B)).view(rows, -1, B)
    codes, scale = _encode(pad, pad.abs().amax(2, keepdim=True))
    return codes.view(rows, -1)[:, :cols].contiguous(), scale[:, :, 0].t().contiguous()


def _tiles8(x):
    x = x.float()
    e, n, k = x.shape
    pad = torch.nn.functional.pad(x, (0, -k % B, 0, -n % B))
    pad = pad.view(e, pad.shape[1] // B, B, -1, B)
    codes, scale = _encode(pad, pad.abs().amax((2, 4), keepdim=True))
    codes = codes.view(e, codes.shape[1] * B, -1)[:, :n, :k].contiguous()
    return codes, scale[:, :, 0, :, 0].contiguous()


def _block_rows(s):
    """Positions [blocks, 128] of the blocks of every expert's rows, and whether they are there."""
    off = s["offsets"]
    blocks = (off[1:] - off[:-1] + B - 1) // B
    last = torch.cumsum(blocks, 0)
    b = torch.arange(s["n_blocks"], device=off.device)
    e = torch.searchsorted(last, b, right=True)
    at = (off[e] + (b - (last[e] - blocks[e])) * B)[:, None] + torch.arange(B, device=off.device)
    there = at < off[e + 1][:, None]
    return torch.where(there, at, 0), there


def _panels8(s, x):
    """Blocks of 128 rows of one expert, transposed: codes [blocks, cols, 128], scales [blocks, cols]."""
    at, there = _block_rows(s)
    x = torch.where(there[:, :, None], x[at], 0.0).transpose(1, 2)
    codes, scale = _encode(x, x.abs().amax(2, keepdim=True))
    return codes.contiguous(), scale[:, :, 0]


def _f32(codes):
    return codes.view(F8).float()


def _sort_back(s, x):
    """x of rows in token order, 0 where a row has no expert."""
    return torch.where((s["pos"] >= 0)[:, None], x[s["pos"].clamp_min(0)], 0.0)


def _plain_rows(s):
    c = s["case"]
    k = c["k"]
    there = (s["order"] >= 0)[:, None]
    i = s["order"].clamp_min(0)
    if s["op"] == "dispatch":
        s["out"].copy_(torch.where(there, s["x"][i // k], s["out"]))
        return s["out"]
    r = _sort_back(s, s["r"].float())
    if s["op"] == "combine":
        return (r.view(c["T"], k, -1) * s["w"][:, :, None]).sum(1).bfloat16()
    dy = s["dy"].float()
    dw = (r.view(c["T"], k, -1) * dy[:, None, :]).sum(2)
    s["out"].copy_(torch.where(there, dy[i // k] * s["w"].view(-1)[i][:, None], s["out"].float()))
    return s["out"], dw


def _plain_quant(s):
    c = s["case"]
    if c["kind"] == "tiles":
        codes, scales = _tiles8(s["x"])
        return [v for a, b in ((codes, scales), (codes.transpose(1, 2), scales.transpose(1, 2)))
                for v in (a.contiguous().view(F8), b.contiguous())]
    there = s["order"] >= 0
    x = s["x"].float()
    if c["gather"]:
        x = x[s["order"].clamp_min(0) // c["k"]]
    if c["kind"] == "rows":
        codes, scales = _rows8(x)
        s["codes"].copy_(torch.where(there[:, None], codes, s["codes"]))
        s["scales"].copy_(torch.where(there[None, :], scales, s["scales"]))
    else:
        codes, scales = _panels8(s, x)
        s["codes"][:s["n_blocks"]] = codes
        s["scales"][:s["n_blocks"]] = scales
    return s["codes"].view(F8), s["scales"]


def _plain_swiglu(s):
    h, n = s["h"].float(), s["case"]["I"]
    g, u = h[:, :n], h[:, n:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    if s["op"] == "swiglu":
        codes, scales = _rows8(u * (g * sig))
        return codes.view(F8), scales
    da = s["da"].float()
    return torch.cat([da * u * (sig * (1.0 + g * (1.0 - sig))), da * (g * sig)], 1).bfloat16()


def _spread(scales, rows, cols):
    """Scales of 128 x 128 tiles, one for each element."""
    return scales.repeat_interleave(B, -2)[..., :rows, :].repeat_interleave(B, -1)[..., :cols]


def _dequant_rows(s):
    xc = s["xc"]
    return _f32(xc) * s["xs"].t().repeat_interleave(B, 1)[:, :xc.shape[1]]


def _pad_groups(s, x, width):
    """Rows in expert order -> [experts, most rows, width], 0 behind an expert's last."""
    E, most = s["case"]["E"], s["most"]
    at = s["owner"] * most + torch.arange(x.shape[0], device=x.device) - s["offsets"][s["owner"]]
    pad = torch.zeros((E * most, width), device=x.device)
    pad[at[:s["used"]]] = x[:s["used"]]
    return pad.view(E, most, width), at


def _plain_gemm(s):
    c = s["case"]
    w = _f32(s["wc"]) * _spread(s["ws"], c["N"], c["K"])
    if s["op"] == "gemm":
        return (_dequant_rows(s) @ w.t()).bfloat16()
    pad, at = _pad_groups(s, _dequant_rows(s), c["K"])
    y = torch.bmm(pad, w.transpose(1, 2)).view(-1, c["N"])
    s["y"][:s["used"]] = y[at[:s["used"]]].bfloat16()
    return s["y"]


def _plain_wgrad(s):
    c, n = s["case"], s["n_blocks"]
    off = s["offsets"]
    blocks = (off[1:] - off[:-1] + B - 1) // B
    last = torch.cumsum(blocks, 0)
    b = torch.arange(n, device=off.device)
    e = torch.searchsorted(last, b, right=True)
    most = (s["most"] + B - 1) // B
    at = e * most + b - (last - blocks)[e]

    def groups(codes, scales, cols):
        x = (_f32(codes[:n]) * scales[:n, :, None]).transpose(1, 2)
        pad = torch.zeros((c["E"] * most, B, cols), device=off.device)
        pad[at] = x
        return pad.view(c["E"], most * B, cols)

    dy, x = groups(s["yc"], s["ys"], c["N"]), groups(s["xc"], s["xs"], c["K"])
    return torch.bmm(dy.transpose(1, 2), x).bfloat16()


# ------------------------------------------------------------------- passes ----
def run(state):
    s, op = state, state["op"]
    c = s["case"]
    if not own:
        if op in ("dispatch", "combine", "combine_bwd"):
            return _plain_rows(s)
        return {"quant": _plain_quant, "swiglu": _plain_swiglu, "swiglu_bwd": _plain_swiglu, "gemm": _plain_gemm,
                "experts": _plain_gemm, "wgrad": _plain_wgrad}[op](s)
    import fp4_fake_quant_amd as fq
    if op == "dispatch":
        return fq.qf_moe_dispatch(s["x"], s["plan"], rows_per_x=c["k"], out=s["out"])
    if op == "combine":
        return fq.qf_moe_combine(s["r"], s["plan"], s["w"])
    if op == "combine_bwd":
        return fq.qf_moe_combine_backward(s["dy"], s["r"], s["plan"], s["w"], d_rows=s["out"])
    if op == "quant":
        if c["kind"] == "tiles":
            codes, scales, codes_t, scales_t = fq.qf_quant_fp8_tiles(s["x"], transpose=True)
            return [codes.view(F8), scales, codes_t.view(F8), scales_t]
        call = fq.qf_quant_fp8 if c["kind"] == "rows" else fq.qf_quant_fp8_panels
        codes, scales = call(s["x"], plan=s["plan"], rows_per_x=c["k"] if c["gather"] else None, codes=s["codes"],
                             scales=s["scales"])
        return codes.view(F8), scales
    if op == "swiglu":
        codes, scales = fq.qf_swiglu_quant_fp8(s["h"])
        return codes.view(F8), scales
    if op == "swiglu_bwd":
        return fq.qf_swiglu_backward(s["h"], s["da"])
    if op == "gemm":
        return fq.qf_gemm_fp8(s["xc"], s["xs"], s["wc"], s["ws"])
    if op == "experts":
        return fq.qf_gemm_fp8_grouped(s["xc"], s["xs"], s["wc"], s["ws"], s["plan"], Y=s["y"])
    return fq.qf_gemm_fp8_wgrad(s["yc"], s["ys"], s["xc"], s["xs"], s["plan"])


# --------------------------------------------------------------------- work ----
def work(case):
    c, op = case, case["op"]
    if "T" in c:
        T, k, E = c["T"], c["k"], c["E"]
        n = T * k
        rows = n * (1.0 - c["none"])
        met = E * (1.0 - (1.0 - 1.0 / E) ** rows)      # experts that have a row
    if op == "dispatch":
        return dict(bytes=2 * c["H"] * (T + rows) + 4 * n, flops=0)
    if op == "combine":
        return dict(bytes=2 * c["H"] * (T + rows) + 8 * n, flops=2 * rows * c["H"])
    if op == "combine_bwd":
        return dict(bytes=2 * c["H"] * (T + 2 * rows) + 12 * n, flops=3 * rows * c["H"])
    if op == "quant":
        if c["kind"] == "tiles":
            n = c["E"] * c["N"] * c["K"]
            return dict(bytes=4 * n + 8 * n // (B * B), flops=3 * n)
        x = c["H"] * ((T if c["gather"] else rows) * 2 + rows * (1 + 4 / B))
        return dict(bytes=x + 4 * n, flops=3 * rows * c["H"])
    if op == "swiglu":
        return dict(bytes=c["P"] * c["I"] * (5 + 4 / B), flops=8 * c["P"] * c["I"])
    if op == "swiglu_bwd":
        return dict(bytes=10 * c["P"] * c["I"], flops=12 * c["P"] * c["I"])
    N, K = c["N"], c["K"]
    if op == "gemm":
        M = c["M"]
        return dict(bytes=M * K * (1 + 4 / B) + N * K * (1 + 4 / B ** 2) + 2 * M * N, flops=2 * M * N * K)
    if op == "experts":
        return dict(bytes=rows * K * (1 + 4 / B) + met * N * K * (1 + 4 / B ** 2) + 2 * rows * N, flops=2 * rows * N * K)
    return dict(bytes=rows * (N + K) * (1 + 4 / B) + 2 * E * N * K, flops=2 * rows * N * K)


# -------------------------------------------------------------------- exact ----
def _round_e4m3(y):
    """Nearest E4M3 value (ties to even) of float64 y, at most 448."""
    _, e = torch.frexp(y.abs().clamp_min(2.0 ** -6))           # |y| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return (torch.round(y / step) * step).clamp_(-TOP, TOP)


def _exact_block(x, dims):
    """Values of the codes, and scales, of x (float64) with blocks along `dims`."""
    top = x.abs().amax(dims, keepdim=True)
    inv = torch.where(top > 0, TOP / top, 0.0)
    return _round_e4m3(x * inv), (top / TOP).squeeze(dims)


def _exact_rows8(x):
    n, cols = x.shape
    nb = (cols + B - 1) // B
    pad = x.new_zeros((n, nb * B))
    pad[:, :cols] = x
    v, sc = _exact_block(pad.view(n, nb, B), (2,))
    return v.reshape(n, nb * B)[:, :cols], sc.t()


def _exact_quant(s):
    c, x = s["case"], s["x"].double()
    if c["kind"] == "tiles":
        v = torch.empty_like(x)
        nb, kb = (c["N"] + B - 1) // B, (c["K"] + B - 1) // B
        sc = x.new_empty((c["E"], nb, kb))
        for i in range(nb):
            for j in range(kb):
                part = x[:, i * B:(i + 1) * B, j * B:(j + 1) * B]
                v[:, i * B:(i + 1) * B, j * B:(j + 1) * B], sc[:, i, j] = _exact_block(part, (1, 2))
        return [v, sc, v.transpose(1, 2).contiguous(), sc.transpose(1, 2).contiguous()]
    order, n = s["order"], s["used"]
    if c["gather"]:
        x = x[order[:n] // c["k"]]
    if c["kind"] == "rows":
        v, sc = (z.new_zeros(o.shape, dtype=torch.float64) for z, o in ((x, s["codes"]), (x, s["scales"])))
        v[:n], sc[:, :n] = _exact_rows8(x[:n])
        return v, sc
    v, sc = torch.zeros(s["codes"].shape, dtype=torch.float64, device=x.device), torch.zeros(s["scales"].shape, dtype=torch.float64, device=x.device)
    b, off = 0, s["offsets"].tolist()
    for lo, hi in zip(off, off[1:]):
        for at in range(lo, hi, B):
            part = x[at:min(at + B, hi)]
            v[b, :, :part.shape[0]], sc[b] = (z.t() if z.dim() == 2 else z for z in _exact_block(part, (0,)))
            b += 1
    return v, sc


def _exact_rows(s):
    c = s["case"]
    k, n, order = c["k"], s["used"], s["order"]
    i = order[:n]
    if s["op"] == "dispatch":
        out = s["out"].double()
        out[:n] = s["x"][i // k].double()
        return out
    r, w = s["r"].double(), s["w"].double().view(-1)
    if s["op"] == "combine":
        y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=r.device)
        return y.index_add_(0, i // k, r[:n] * w[i][:, None])
    dy = s["dy"].double()[i // k]
    out = s["out"].double()
    out[:n] = dy * w[i][:, None]
    dw = torch.zeros_like(w)
    dw[i] = (dy * r[:n]).sum(1)
    return out, dw.view(c["T"], k)


def _exact_swiglu(s):
    g, u = s["h"].double().chunk(2, 1)
    sig = torch.sigmoid(g)
    if s["op"] == "swiglu":
        return _exact_rows8(u * g * sig)
    da = s["da"].double()
    return torch.cat([da * u * sig * (1 + g - g * sig), da * g * sig], 1)


def _exact_product(xc, xs, wc, ws):
    """Row-scaled x against tile-scaled w, block by block."""
    y = torch.zeros((xc.shape[0], wc.shape[0]), dtype=torch.float64, device=xc.device)
    for b in range(xs.shape[0]):
        x = xc[:, b * B:(b + 1) * B].view(F8).double() * xs[b].double()[:, None]
        w = wc[:, b * B:(b + 1) * B].view(F8).double() * ws[:, b].double().repeat_interleave(B)[:wc.shape[0], None]
        y += x @ w.t()
    return y


def _exact_experts(s):
    y = s["y"].double()
    off = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            y[lo:hi] = _exact_product(s["xc"][lo:hi], s["xs"][:, lo:hi], s["wc"][e], s["ws"][e])
    return y


def _exact_wgrad(s):
    c = s["case"]
    dw = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device=s["xc"].device)
    b, off = 0, s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        for _ in range(lo, hi, B):
            dy = s["yc"][b].view(F8).double() * s["ys"][b].double()[:, None]
            x = s["xc"][b].view(F8).double() * s["xs"][b].double()[:, None]
            dw[e] += dy @ x.t()
            b += 1
    return dw


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        return _exact_product(s["xc"], s["xs"], s["wc"], s["ws"])
    return {"dispatch": _exact_rows, "combine": _exact_rows, "combine_bwd": _exact_rows, "quant": _exact_quant,
            "swiglu": _exact_swiglu, "swiglu_bwd": _exact_swiglu, "experts": _exact_experts, "wgrad": _exact_wgrad}[op](s)
