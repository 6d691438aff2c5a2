"""Python binding of libqf (include/qf.h): MI355X simulated quantization.

Argument marshalling only.  Each function has the name of the C entry point
it calls, takes torch tensors that live on the GPU (bf16 data as
torch.bfloat16, packed bytes as torch.uint8, scales as torch.float32),
passes their device pointers, sizes and strides plus torch's current HIP
stream, and raises QFError on a non-zero status.  Outputs that are not
given are allocated with torch (device memory is torch's job here); every
computation runs in the library's HIP kernels.
"""

import ctypes

import torch

from ._lib import AdamwHyper, AdamwPlan, AdamwTensor, GgufTensor, LoraDesc, LoraExpertsDesc, RouteDesc, StTensor, TensorDesc, lib

QF_OK = 0
QF_QDQ_A, QF_QDQ_W, QF_FP4_CORES, QF_MX_NOCLIP = 1, 2, 4, 8
QF_FMT_NVFP4, QF_FMT_MXFP4, QF_FMT_Q4K = 0, 1, 2
QF_OP_NVFP4_TENSOR_SCALE, QF_OP_LORA, QF_OP_LINEAR_BACKWARD = 0, 1, 2
MAX_GROUPED = 16
BLOCK = {QF_FMT_NVFP4: 16, QF_FMT_MXFP4: 32, QF_FMT_Q4K: 256}


class QFError(RuntimeError):
    def __init__(self, status, where):
        msg = lib().qf_status_str(status).decode()
        if status == 5:
            msg += f" (hipError {lib().qf_last_hip_error()})"
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def _check(status, where):
    if status != QF_OK:
        raise QFError(status, where)


def _stream():
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _mat(x, name):
    """rows, cols, row stride of a 2-D tensor with unit column stride."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    rows, cols = shape
    ld, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    return rows, cols, ld if rows > 1 else max(cols, ld)


def _bf16(x, name):
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16")
    return x


def _out_like(x, y):
    return torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if y is None else _bf16(y, "y")


def _packed(fmt, rows, cols, device, codes, scales):
    if codes is None:
        codes = torch.empty((rows, cols // 2) if fmt != QF_FMT_Q4K else (rows, cols // 256, 144),
                            dtype=torch.uint8, device=device)
    if scales is None and fmt != QF_FMT_Q4K:
        scales = torch.empty((rows, cols // BLOCK[fmt]), dtype=torch.uint8, device=device)
    return codes, scales


# ------------------------------------------------------------ helpers ----
def qf_version():
    v = lib().qf_version()
    return (v >> 16, (v >> 8) & 0xFF, v & 0xFF)


def qf_packed_bytes(fmt, rows, cols):
    return lib().qf_packed_bytes(fmt, rows, cols)


def _descs(items):
    n = len(items)
    arr = (TensorDesc * max(n, 1))()
    for i, it in enumerate(items):
        x = _bf16(it["x"], "x")
        rows, cols, ldx = _mat(x, "x")
        d = arr[i]
        d.x, d.rows, d.cols, d.ldx = x.data_ptr(), rows, cols, ldx
        y = it.get("y")
        if y is not None:
            _bf16(y, "y")
            d.y, d.ldy = y.data_ptr(), _mat(y, "y")[2]
        d.codes = it["codes"].data_ptr() if it.get("codes") is not None else None
        d.scales = it["scales"].data_ptr() if it.get("scales") is not None else None
        d.group = int(it.get("group", 0))
    return arr, n


# --------------------------------------------------- NVFP4 tensor scale ---
def qf_nvfp4_tensor_scale_workspace(items):
    arr, n = _descs(items)
    return lib().qf_nvfp4_tensor_scale_workspace(ctypes.byref(arr), n)


def qf_nvfp4_tensor_scale_grouped(items, n_groups, d_scales=None, d_nonfinite=None, ws=None):
    """items: list of dict(x=bf16 tensor, group=int).  Returns the device float32 scales."""
    dev = items[0]["x"].device if items else torch.device("cuda")
    arr, n = _descs(items)
    need = lib().qf_nvfp4_tensor_scale_workspace(ctypes.byref(arr), n)
    if ws is None:
        ws = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    if d_scales is None:
        d_scales = torch.empty(n_groups, dtype=torch.float32, device=dev)
    _check(lib().qf_nvfp4_tensor_scale_grouped(ctypes.byref(arr), n, n_groups, _p(d_scales), _p(d_nonfinite),
                                                _p(ws), ws.numel() * ws.element_size(), _stream()),
           "qf_nvfp4_tensor_scale_grouped")
    return d_scales


def qf_nvfp4_tensor_scale_tracked(items, n_groups, d_amax, d_scales=None, d_nonfinite=None, ws=None):
    """Tensor scales from the running maximum d_amax (device float32 [n_groups], updated in
    place: max(d_amax, this call's group maxima)); items as qf_nvfp4_tensor_scale_grouped."""
    if d_amax.dtype != torch.float32 or d_amax.device.type != "cuda" or d_amax.numel() < n_groups:
        raise TypeError("d_amax must be a float32 device tensor with a value per group")
    dev = items[0]["x"].device if items else d_amax.device
    arr, n = _descs(items)
    need = lib().qf_nvfp4_tensor_scale_workspace(ctypes.byref(arr), n)
    if ws is None:
        ws = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    if d_scales is None:
        d_scales = torch.empty(n_groups, dtype=torch.float32, device=dev)
    _check(lib().qf_nvfp4_tensor_scale_tracked(ctypes.byref(arr), n, n_groups, _p(d_amax), _p(d_scales),
                                                _p(d_nonfinite), _p(ws), ws.numel() * ws.element_size(), _stream()),
           "qf_nvfp4_tensor_scale_tracked")
    return d_scales


def qf_workspace_size(op, rows, cols, n):
    return lib().qf_workspace_size(int(op), int(rows), int(cols), int(n))


def qf_nvfp4_tensor_scale(x, d_scale=None, d_nonfinite=None, ws=None):
    """Tensor scale of one tied group: x is a bf16 tensor or a list of them (e.g. Q, K, V).
    Contiguous members go through the pointer-array call, strided ones through the grouped
    call (same arithmetic).  Returns the device float32 scale (shape [1])."""
    xs = list(x) if isinstance(x, (list, tuple)) else [x]
    if not all(t.is_contiguous() for t in xs):
        return qf_nvfp4_tensor_scale_grouped([dict(x=t, group=0) for t in xs], 1, d_scale, d_nonfinite, ws)
    dev = xs[0].device if xs else torch.device("cuda")
    ptrs = (ctypes.c_void_p * max(len(xs), 1))(*[_bf16(t, "x").data_ptr() for t in xs])
    numel = (ctypes.c_int64 * max(len(xs), 1))(*[t.numel() for t in xs])
    need = lib().qf_workspace_size(QF_OP_NVFP4_TENSOR_SCALE, 1, max([t.numel() for t in xs] + [0]), len(xs))
    if ws is None:
        ws = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    if d_scale is None:
        d_scale = torch.empty(1, dtype=torch.float32, device=dev)
    _check(lib().qf_nvfp4_tensor_scale(ptrs, numel, len(xs), _p(d_scale), _p(d_nonfinite), _p(ws),
                                       ws.numel() * ws.element_size(), _stream()), "qf_nvfp4_tensor_scale")
    return d_scale


# ------------------------------------------------------------ QDQ/pack ----
def qf_qdq_nvfp4(x, d_scale, y=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    _check(lib().qf_qdq_nvfp4(_p(x), rows, cols, ldx, _p(d_scale), _p(y), _mat(y, "y")[2], _stream()), "qf_qdq_nvfp4")
    return y


def qf_pack_nvfp4(x, d_scale, codes=None, scales=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    codes, scales = _packed(QF_FMT_NVFP4, rows, cols, x.device, codes, scales)
    _check(lib().qf_pack_nvfp4(_p(x), rows, cols, ldx, _p(d_scale), _p(codes), _p(scales), _stream()), "qf_pack_nvfp4")
    return codes, scales


def qf_qdq_pack_nvfp4(x, d_scale, y=None, codes=None, scales=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    codes, scales = _packed(QF_FMT_NVFP4, rows, cols, x.device, codes, scales)
    _check(lib().qf_qdq_pack_nvfp4(_p(x), rows, cols, ldx, _p(d_scale), _p(y), _mat(y, "y")[2], _p(codes), _p(scales),
                                   _stream()), "qf_qdq_pack_nvfp4")
    return y, codes, scales


def qf_qdq_pack_nvfp4_grouped(items, d_scales):
    """items: list of dict(x, y=None, codes=None, scales=None, group)."""
    arr, n = _descs(items)
    _check(lib().qf_qdq_pack_nvfp4_grouped(ctypes.byref(arr), n, _p(d_scales), _stream()), "qf_qdq_pack_nvfp4_grouped")


def qf_qdq_mxfp4(x, y=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    _check(lib().qf_qdq_mxfp4(_p(x), rows, cols, ldx, _p(y), _mat(y, "y")[2], _stream()), "qf_qdq_mxfp4")
    return y


def qf_pack_mxfp4(x, codes=None, scales=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    codes, scales = _packed(QF_FMT_MXFP4, rows, cols, x.device, codes, scales)
    _check(lib().qf_pack_mxfp4(_p(x), rows, cols, ldx, _p(codes), _p(scales), _stream()), "qf_pack_mxfp4")
    return codes, scales


def qf_qdq_pack_mxfp4(x, y=None, codes=None, scales=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    codes, scales = _packed(QF_FMT_MXFP4, rows, cols, x.device, codes, scales)
    _check(lib().qf_qdq_pack_mxfp4(_p(x), rows, cols, ldx, _p(y), _mat(y, "y")[2], _p(codes), _p(scales), _stream()),
           "qf_qdq_pack_mxfp4")
    return y, codes, scales


def qf_qdq_pack_mxfp4_grouped(items):
    arr, n = _descs(items)
    _check(lib().qf_qdq_pack_mxfp4_grouped(ctypes.byref(arr), n, _stream()), "qf_qdq_pack_mxfp4_grouped")


def qf_qdq_q4k(x, y=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    _check(lib().qf_qdq_q4k(_p(x), rows, cols, ldx, _p(y), _mat(y, "y")[2], _stream()), "qf_qdq_q4k")
    return y


def qf_pack_q4k(x, blocks=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    blocks, _ = _packed(QF_FMT_Q4K, rows, cols, x.device, blocks, None)
    _check(lib().qf_pack_q4k(_p(x), rows, cols, ldx, _p(blocks), _stream()), "qf_pack_q4k")
    return blocks


def qf_qdq_pack_q4k(x, y=None, blocks=None):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    y = _out_like(x, y)
    blocks, _ = _packed(QF_FMT_Q4K, rows, cols, x.device, blocks, None)
    _check(lib().qf_qdq_pack_q4k(_p(x), rows, cols, ldx, _p(y), _mat(y, "y")[2], _p(blocks), _stream()), "qf_qdq_pack_q4k")
    return y, blocks


QF_MX_RULE_FLOOR, QF_MX_RULE_NOCLIP = 0, 1


def qf_qdq_pack_mxfp4_rule(items, rule):
    """qf_qdq_pack_mxfp4_grouped under shared-exponent rule QF_MX_RULE_FLOOR or QF_MX_RULE_NOCLIP."""
    arr, n = _descs(items)
    _check(lib().qf_qdq_pack_mxfp4_rule(ctypes.byref(arr), n, int(rule), _stream()), "qf_qdq_pack_mxfp4_rule")


QF_Q4K_RULE_MINMAX, QF_Q4K_RULE_MSE = 0, 1


def qf_qdq_pack_q4k_rule(items, rule):
    """qf_qdq_pack_q4k_grouped under sub-block scale rule QF_Q4K_RULE_MINMAX or QF_Q4K_RULE_MSE."""
    arr, n = _descs(items)
    _check(lib().qf_qdq_pack_q4k_rule(ctypes.byref(arr), n, int(rule), _stream()), "qf_qdq_pack_q4k_rule")


def qf_qdq_pack_q4k_grouped(items):
    arr, n = _descs(items)
    _check(lib().qf_qdq_pack_q4k_grouped(ctypes.byref(arr), n, _stream()), "qf_qdq_pack_q4k_grouped")


# ----------------------------------------------------------------- STE ----
def qf_ste_backward(g_q, g_latent=None, accumulate=False):
    _bf16(g_q, "g_q")
    if not g_q.is_contiguous():
        raise ValueError("g_q must be contiguous")
    if g_latent is None:
        g_latent = torch.empty(g_q.shape, dtype=torch.float32, device=g_q.device)
    if g_latent.dtype != torch.float32 or not g_latent.is_contiguous() or g_latent.numel() != g_q.numel():
        raise ValueError("g_latent must be a contiguous float32 tensor with g_q's element count")
    _check(lib().qf_ste_backward(_p(g_q), _p(g_latent), g_q.numel(), int(bool(accumulate)), _stream()), "qf_ste_backward")
    return g_latent


def _ste_clip_args(g_q, x, g_latent):
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    _bf16(g_q, "g_q")
    if tuple(g_q.shape) != (rows, cols) or not g_q.is_contiguous():
        raise ValueError("g_q must be a contiguous tensor of x's shape")
    if g_latent is None:
        g_latent = torch.empty((rows, cols), dtype=torch.float32, device=x.device)
    if g_latent.dtype != torch.float32 or tuple(g_latent.shape) != (rows, cols) or not g_latent.is_contiguous():
        raise ValueError("g_latent must be a contiguous float32 tensor of x's shape")
    return rows, cols, ldx, g_latent


def qf_ste_backward_clipped_nvfp4(g_q, x, d_scale, g_latent=None, accumulate=False):
    """g_latent = f32(g_q), or +0.0 where the NVFP4 quantizer (tensor scale d_scale)
    saturated x; added to g_latent when accumulate."""
    rows, cols, ldx, g_latent = _ste_clip_args(g_q, x, g_latent)
    _check(lib().qf_ste_backward_clipped_nvfp4(_p(g_q), _p(x), rows, cols, ldx, _p(d_scale), _p(g_latent),
                                               int(bool(accumulate)), _stream()), "qf_ste_backward_clipped_nvfp4")
    return g_latent


def qf_ste_backward_clipped_mxfp4(g_q, x, g_latent=None, accumulate=False, rule=QF_MX_RULE_FLOOR):
    """g_latent = f32(g_q), or +0.0 where the MXFP4 quantizer (shared-exponent rule `rule`)
    saturated x; added to g_latent when accumulate."""
    rows, cols, ldx, g_latent = _ste_clip_args(g_q, x, g_latent)
    _check(lib().qf_ste_backward_clipped_mxfp4(_p(g_q), _p(x), rows, cols, ldx, int(rule), _p(g_latent),
                                               int(bool(accumulate)), _stream()), "qf_ste_backward_clipped_mxfp4")
    return g_latent


# ---------------------------------------------------------------- LoRA ----
class LoraBatch:
    """Descriptor array for the qf_lora_* calls, built once and reusable.

    items: list of dict(W, A, B, group, M=None, y=None, codes=None, scales=None,
    G=None, dA=None, dB=None) of device tensors; W [rows, cols] bf16 with contiguous
    rows, A [r, cols] and B [rows, r] contiguous bf16.  The tensors must stay alive
    (and keep their storage) while the batch is used.
    """

    def __init__(self, items):
        self.items = items
        self.arr = (LoraDesc * max(len(items), 1))()
        self.n = len(items)
        self.device = items[0]["W"].device if items else torch.device("cuda")
        for i, it in enumerate(items):
            W = _bf16(it["W"], "W")
            rows, cols, ldw = _mat(W, "W")
            A, B = _bf16(it["A"], "A"), _bf16(it["B"], "B")
            if A.dim() != 2 or B.dim() != 2 or not A.is_contiguous() or not B.is_contiguous():
                raise ValueError("A [r, cols] and B [rows, r] must be contiguous 2-D tensors")
            r = A.shape[0]
            if A.shape[1] != cols or tuple(B.shape) != (rows, r):
                raise ValueError(f"adapter shapes {tuple(A.shape)}, {tuple(B.shape)} do not fit W {rows}x{cols}")
            d = self.arr[i]
            d.W, d.rows, d.cols, d.ldw = W.data_ptr(), rows, cols, ldw
            d.A, d.B, d.r, d.group = A.data_ptr(), B.data_ptr(), r, int(it.get("group", 0))
            for name in ("M", "y", "codes", "scales", "G", "dA", "dB"):
                t = it.get(name)
                if t is not None and not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
                setattr(d, name, t.data_ptr() if t is not None else None)
        self.ref = ctypes.byref(self.arr)
        self.workspace_bytes = lib().qf_lora_workspace(self.ref, self.n)


def _batch(items):
    return items if isinstance(items, LoraBatch) else LoraBatch(items)


def _lora_ws(b, ws):
    if ws is None:
        ws = torch.empty(max(b.workspace_bytes, 4), dtype=torch.uint8, device=b.device)
    return ws


def qf_lora_workspace(items):
    return _batch(items).workspace_bytes


def qf_lora_layout(items):
    """(most pass-1 tiles per wave, pass-1 workgroups, rows per gradient workgroup, gradient
    workgroups, rows per pass-2 unit, pass-2 workgroups) the LoRA calls choose for these
    descriptors (a host query)."""
    b = _batch(items)
    out = (ctypes.c_int32 * 6)()
    _check(lib().qf_lora_layout(b.ref, b.n, out), "qf_lora_layout")
    return tuple(out)


def qf_lora_merge_tensor_scale_nvfp4_grouped(items, n_groups, d_scales=None, d_nonfinite=None, ws=None):
    b = _batch(items)
    ws = _lora_ws(b, ws)
    if d_scales is None:
        d_scales = torch.empty(n_groups, dtype=torch.float32, device=b.device)
    _check(lib().qf_lora_merge_tensor_scale_nvfp4_grouped(b.ref, b.n, n_groups, _p(d_scales), _p(d_nonfinite),
                                                           _p(ws), ws.numel() * ws.element_size(), _stream()),
           "qf_lora_merge_tensor_scale_nvfp4_grouped")
    return d_scales


def qf_lora_merge_qdq_pack_nvfp4_grouped(items, d_scales):
    b = _batch(items)
    _check(lib().qf_lora_merge_qdq_pack_nvfp4_grouped(b.ref, b.n, _p(d_scales), _stream()),
           "qf_lora_merge_qdq_pack_nvfp4_grouped")


def qf_lora_adapter_grads_grouped(items, accumulate=False, ws=None):
    b = _batch(items)
    ws = _lora_ws(b, ws)
    _check(lib().qf_lora_adapter_grads_grouped(b.ref, b.n, int(bool(accumulate)), _p(ws),
                                               ws.numel() * ws.element_size(), _stream()),
           "qf_lora_adapter_grads_grouped")


class LoraExperts:
    """Stacked-experts descriptors for the qf_lora_experts_* calls, built once and reusable.

    items: list of dict(W, A, B, group, group_stride=1, y=None, codes=None, scales=None,
    G=None, dA=None, dB=None) of contiguous device tensors with a leading expert axis:
    W [E, rows, cols] bf16, A [E, r, cols], B [E, rows, r], y [E, rows, cols],
    codes [E, rows, cols/2], scales [E, rows, cols/16], G [E, rows, cols],
    dA [E, r, cols] and dB [E, rows, r] float32.  Expert e's tied group is
    group + e * group_stride.  There is no merge scratch (M).
    """

    def __init__(self, items):
        self.items = items
        self.arr = (LoraExpertsDesc * max(len(items), 1))()
        self.n = len(items)
        self.device = items[0]["W"].device if items else torch.device("cuda")
        for i, it in enumerate(items):
            W, A, B = _bf16(it["W"], "W"), _bf16(it["A"], "A"), _bf16(it["B"], "B")
            for t, name in ((W, "W"), (A, "A"), (B, "B")):
                if t.dim() != 3 or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous 3-D tensor [experts, ...]")
            E, rows, cols = W.shape
            r = A.shape[1]
            if tuple(A.shape) != (E, r, cols) or tuple(B.shape) != (E, rows, r):
                raise ValueError(f"adapter shapes {tuple(A.shape)}, {tuple(B.shape)} do not fit W {tuple(W.shape)}")
            x = self.arr[i]
            d = x.d
            d.W, d.rows, d.cols, d.ldw = W.data_ptr(), rows, cols, cols
            d.A, d.B, d.r, d.group = A.data_ptr(), B.data_ptr(), r, int(it.get("group", 0))
            d.M = None
            for name in ("y", "codes", "scales", "G", "dA", "dB"):
                t = it.get(name)
                if t is not None and (not t.is_contiguous() or t.shape[0] != E):
                    raise ValueError(f"{name} must be contiguous with {E} experts")
                setattr(d, name, t.data_ptr() if t is not None else None)
            x.count = E
            x.group_stride = int(it.get("group_stride", 1))
        self.ref = ctypes.byref(self.arr)
        self.workspace_bytes = lib().qf_lora_experts_workspace(self.ref, self.n)


def qf_lora_experts_layout(ex):
    """The launch layout of the stacked-experts calls (as qf_lora_layout)."""
    out = (ctypes.c_int32 * 6)()
    _check(lib().qf_lora_experts_layout(ex.ref, ex.n, out), "qf_lora_experts_layout")
    return tuple(out)


def qf_lora_experts_merge_tensor_scale_nvfp4(ex, n_groups, d_scales=None, d_nonfinite=None, ws=None):
    ws = _lora_ws(ex, ws)
    if d_scales is None:
        d_scales = torch.empty(n_groups, dtype=torch.float32, device=ex.device)
    _check(lib().qf_lora_experts_merge_tensor_scale_nvfp4(ex.ref, ex.n, n_groups, _p(d_scales), _p(d_nonfinite),
                                                           _p(ws), ws.numel() * ws.element_size(), _stream()),
           "qf_lora_experts_merge_tensor_scale_nvfp4")
    return d_scales


def qf_lora_experts_merge_qdq_pack_nvfp4(ex, d_scales):
    _check(lib().qf_lora_experts_merge_qdq_pack_nvfp4(ex.ref, ex.n, _p(d_scales), _stream()),
           "qf_lora_experts_merge_qdq_pack_nvfp4")


def qf_lora_experts_adapter_grads(ex, accumulate=False, ws=None):
    ws = _lora_ws(ex, ws)
    _check(lib().qf_lora_experts_adapter_grads(ex.ref, ex.n, int(bool(accumulate)), _p(ws),
                                               ws.numel() * ws.element_size(), _stream()),
           "qf_lora_experts_adapter_grads")


def _lora_single(W, A, B):
    for t, name in ((W, "W"), (A, "A"), (B, "B")):
        if not _bf16(t, name).is_contiguous() or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D bf16 tensor")
    rows, cols = W.shape
    r = A.shape[0]
    if A.shape[1] != cols or tuple(B.shape) != (rows, r):
        raise ValueError(f"adapter shapes {tuple(A.shape)}, {tuple(B.shape)} do not fit W {rows}x{cols}")
    return rows, cols, r


def _lora_single_ws(rows, cols, device, ws):
    if ws is None:
        ws = torch.empty(max(lib().qf_workspace_size(QF_OP_LORA, rows, cols, 1), 4), dtype=torch.uint8,
                         device=device)
    return ws


def qf_lora_merge_tensor_scale_nvfp4(W, A, B, d_scale=None, ws=None):
    """NVFP4 tensor scale of M = W + B.A for one contiguous matrix, merged in registers."""
    rows, cols, r = _lora_single(W, A, B)
    ws = _lora_single_ws(rows, cols, W.device, ws)
    if d_scale is None:
        d_scale = torch.empty(1, dtype=torch.float32, device=W.device)
    _check(lib().qf_lora_merge_tensor_scale_nvfp4(_p(W), _p(A), _p(B), rows, cols, r, _p(d_scale), _p(ws),
                                                   ws.numel() * ws.element_size(), _stream()),
           "qf_lora_merge_tensor_scale_nvfp4")
    return d_scale


def qf_lora_merge_qdq_pack_nvfp4(W, A, B, d_scale, y=None, codes=None, scales=None):
    """(y, codes, scales): NVFP4 QDQ + pack of M = W + B.A (merged again in registers)."""
    rows, cols, r = _lora_single(W, A, B)
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=W.device) if y is None else y
    codes, scales = _packed(QF_FMT_NVFP4, rows, cols, W.device, codes, scales)
    _check(lib().qf_lora_merge_qdq_pack_nvfp4(_p(W), _p(A), _p(B), rows, cols, r, _p(d_scale), _p(y), _p(codes),
                                               _p(scales), _stream()), "qf_lora_merge_qdq_pack_nvfp4")
    return y, codes, scales


def qf_lora_adapter_grads(G, A, B, dA=None, dB=None, accumulate=False, ws=None):
    """(dA [r, cols], dB [rows, r]) fp32 = (B^T . G, G . A^T) for one contiguous matrix."""
    rows, cols, r = _lora_single(G, A, B)
    ws = _lora_single_ws(rows, cols, G.device, ws)
    dA = torch.empty((r, cols), dtype=torch.float32, device=G.device) if dA is None else dA
    dB = torch.empty((rows, r), dtype=torch.float32, device=G.device) if dB is None else dB
    _check(lib().qf_lora_adapter_grads(_p(G), _p(A), _p(B), rows, cols, r, _p(dA), _p(dB), int(bool(accumulate)),
                                       _p(ws), ws.numel() * ws.element_size(), _stream()), "qf_lora_adapter_grads")
    return dA, dB


# ------------------------------------------------------------- routing ----
QF_ROUTE_SOFTMAX, QF_ROUTE_SIGMOID = 0, 1
QF_ROUTE_GROUP_MAX, QF_ROUTE_GROUP_TOP2 = 0, 1
_SCORING = {"softmax": QF_ROUTE_SOFTMAX, "sigmoid": QF_ROUTE_SIGMOID, 0: 0, 1: 1}
_GROUP_RULE = {"max": QF_ROUTE_GROUP_MAX, "top2": QF_ROUTE_GROUP_TOP2, 0: 0, 1: 1}


def _same_gpu(*tensors):
    """The index of the one GPU that holds every given tensor (None entries are skipped)."""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0 or dev >= 0:
                    raise (TypeError("tensors must live on the GPU") if i < 0 else
                           ValueError(f"tensors live on GPUs {dev} and {i}"))
                dev = i
            elif i < 0:
                raise TypeError("tensors must live on the GPU")
    return dev


def _call(dev, name, *args):
    """Calls an entry point with GPU dev current and dev's current stream as its last argument."""
    f = getattr(lib(), name)
    if dev == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    elif dev < 0:
        st = f(*args, _stream())
    else:
        with torch.cuda.device(dev):
            st = f(*args, _stream())
    if st != QF_OK:
        raise QFError(st, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _route_desc(logits, k, scoring, renorm, scale):
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16")
    if scoring not in _SCORING:
        raise ValueError("scoring is 'softmax' or 'sigmoid'")
    T, E, ld = _mat(logits, "logits")      # the fields in qf_route_desc's order
    return RouteDesc(logits.data_ptr(), T, ld, None, scale, logits.dtype is torch.bfloat16, E, k, _SCORING[scoring],
                     bool(renorm), 1, 1, 0), T, E


def _dense(t, name, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    return t


def qf_moe_route(logits, k, scoring="softmax", bias=None, n_group=1, topk_group=1, group_rule="max", renorm=True,
                 scale=1.0, indices=None, weights=None):
    """(indices int32 [T, k], weights float32 [T, k]) of the k experts of every row of logits
    [T, E] (float32 or bfloat16): scoring "softmax" or "sigmoid", chosen by score + bias (float32
    [E]) within the topk_group best of n_group groups (ranked by "max" or "top2"), weights =
    scores (over their sum when renorm) * scale."""
    d, T, E = _route_desc(logits, k, scoring, renorm, scale)
    if group_rule not in _GROUP_RULE:
        raise ValueError("group_rule is 'max' or 'top2'")
    dev = _same_gpu(logits, bias, indices, weights)
    if bias is not None:
        d.bias = _dense(bias, "bias", torch.float32, (E,)).data_ptr()
    if n_group != 1:
        d.n_group, d.topk_group, d.group_rule = n_group, topk_group, _GROUP_RULE[group_rule]
    elif topk_group != 1:
        d.topk_group = topk_group
    shape = (T, max(k, 0))
    if indices is None:
        indices = torch.empty(shape, dtype=torch.int32, device=logits.device)
    else:
        _dense(indices, "indices", torch.int32, shape)
    if weights is None:
        weights = torch.empty(shape, dtype=torch.float32, device=logits.device)
    else:
        _dense(weights, "weights", torch.float32, shape)
    _call(dev, "qf_moe_route", ctypes.byref(d), indices.data_ptr(), weights.data_ptr())
    return indices, weights


def qf_moe_route_backward(logits, indices, d_weights, scoring="softmax", renorm=True, scale=1.0, d_logits=None):
    """d_logits [T, E] (logits' type) from d_weights float32 [T, k] for the forward's indices."""
    d, T, E = _route_desc(logits, indices.shape[1] if indices.dim() == 2 else 0, scoring, renorm, scale)
    dev = _same_gpu(logits, indices, d_weights, d_logits)
    _dense(indices, "indices", torch.int32, (T, d.k))
    _dense(d_weights, "d_weights", torch.float32, (T, d.k))
    if d_logits is None:
        d_logits, ldd = torch.empty((T, E), dtype=logits.dtype, device=logits.device), E
    else:
        if d_logits.dtype != logits.dtype or tuple(d_logits.shape) != (T, E):
            raise ValueError("d_logits must have the logits' shape and type")
        ldd = _mat(d_logits, "d_logits")[2]
    _call(dev, "qf_moe_route_backward", ctypes.byref(d), indices.data_ptr(), d_weights.data_ptr(), d_logits.data_ptr(), ldd)
    return d_logits


# ---------------------------------------------------------------- rows ----
ROW_TILE, ROW_MAX_IDS = 32, 1024


def _ids(t, name):
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor")
    return t


def _space(ws):
    """Bytes of a workspace, which must be one run of memory (an expanded view has less than it counts)."""
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.numel() * ws.element_size()


class RowPlan:
    """Rows grouped by id (qf_row_plan): offsets [n_ids + 1], order [n] and tiles [t, 2], int32
    on the device, for n rows with ids in [0, n_ids); positions [n], order's inverse, or None.
    One allocation, with the workspace that building it takes."""

    def __init__(self, n, n_ids, device, positions=False):
        self.n, self.n_ids = n, n_ids
        t, self.ws_bytes = lib().qf_row_plan_tiles(n, n_ids), lib().qf_row_plan_workspace(n, n_ids)
        sizes = (2 * t, self.ws_bytes // 4, n_ids + 1, n)        # what is 8-byte aligned first
        if positions:
            sizes += (n,)
            tiles, self.ws, self.offsets, self.order, self.positions = torch.empty(
                sum(sizes), dtype=torch.int32, device=device).split_with_sizes(sizes)
        else:
            self.positions = None
            tiles, self.ws, self.offsets, self.order = torch.empty(sum(sizes), dtype=torch.int32,
                                                                   device=device).split_with_sizes(sizes)
        self.tiles = tiles.view(t, 2)


def qf_row_plan(ids, n_ids, plan=None, ws=None, positions=False):
    """The RowPlan of ids (int32 device tensor, any shape; row i is element i in memory order):
    rows with an id outside [0, n_ids) are in no group.  positions: with order's inverse, which
    qf_moe_combine reads.  plan: one of the same n and n_ids to write into; ws: a workspace other
    than the plan's own."""
    dev, n, n_ids = _same_gpu(_ids(ids, "ids"), ws), ids.numel(), int(n_ids)
    if plan is None:
        if not 1 <= n_ids <= ROW_MAX_IDS:
            raise ValueError(f"n_ids is 1..{ROW_MAX_IDS}")
        plan = RowPlan(n, n_ids, ids.device, positions)
    elif plan.n != n or plan.n_ids != n_ids or plan.offsets.get_device() != dev:
        raise ValueError(f"the plan is for {plan.n} rows of {plan.n_ids} ids on {plan.offsets.device}")
    elif positions and plan.positions is None:
        raise ValueError("the plan was built without positions")
    if ws is None:
        ws, ws_bytes = plan.ws, plan.ws_bytes
    else:
        ws_bytes = _space(ws)
    if plan.positions is None:
        _call(dev, "qf_row_plan", ids.data_ptr(), n, n_ids, plan.offsets.data_ptr(), plan.order.data_ptr(),
              plan.tiles.data_ptr(), ws.data_ptr(), ws_bytes)
    else:
        _call(dev, "qf_row_plan_positions", ids.data_ptr(), n, n_ids, plan.offsets.data_ptr(), plan.order.data_ptr(),
              plan.tiles.data_ptr(), plan.positions.data_ptr(), ws.data_ptr(), ws_bytes)
    return plan


# ----------------------------------------- rows into expert order and back ----
def _plan(plan):
    if not isinstance(plan, RowPlan):
        raise TypeError("plan must be a RowPlan")
    return plan


def _out16(t, name, rows, cols, device):
    """A bf16 output [rows, cols] and its row stride."""
    if t is None:
        return torch.empty(rows, cols, dtype=torch.bfloat16, device=device), cols
    if tuple(_bf16(t, name).shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, want {(rows, cols)}")
    return t, _mat(t, name)[2]


def _positions(plan):
    if _plan(plan).positions is None:
        raise ValueError("the plan must be built with positions=True")
    return plan.positions.data_ptr()


def _x_rows(rows, n, rows_per_x):
    if not 1 <= rows_per_x < 1 << 62 or rows != (n + rows_per_x - 1) // rows_per_x:
        raise ValueError(f"x has {rows} rows for {n} rows of the plan and rows_per_x={rows_per_x}")


def qf_moe_dispatch(X, plan, rows_per_x=1, out=None):
    """out[plan.positions[i]] = X[i // rows_per_x], bf16 [plan.n, H]: rows into the order of the plan's
    groups.  Rows behind the last group are left as they were (unspecified where out is new)."""
    positions = _positions(plan)
    dev = _same_gpu(X, out, plan.order)
    rows, H, ldx = _mat(_bf16(X, "X"), "X")
    _x_rows(rows, plan.n, rows_per_x)
    out, ldo = _out16(out, "out", plan.n, H, X.device)
    _call(dev, "qf_moe_dispatch", X.data_ptr(), ldx, rows_per_x, positions, plan.n, H, out.data_ptr(), ldo)
    return out


def _combine(plan, weights, k):
    _positions(plan)
    if weights is not None:
        if weights.dim() != 2 or k not in (None, weights.shape[1]):
            raise ValueError("weights must have shape [tokens, k]")
        k = weights.shape[1]
        _dense(weights, "weights", torch.float32, (plan.n // k if k else 0, k))
    if not k or k < 1 or plan.n % k:
        raise ValueError(f"k={k} does not divide the plan's {plan.n} rows")
    return plan.n // k, k


def qf_moe_combine(R, plan, weights=None, k=None, Y=None):
    """Y[t] = sum_j weights[t, j] * R[plan.positions[t * k + j]], bf16 [tokens, H], from R [plan.n,
    H] in the order of the plan's groups: weights float32 [tokens, k], or None with k given (all 1:
    the gradient of qf_moe_dispatch with rows_per_x = k).  Rows in no group add nothing."""
    tokens, k = _combine(plan, weights, k)
    dev = _same_gpu(R, weights, Y, plan.order)
    rows, H, ldr = _mat(_bf16(R, "R"), "R")
    if rows != plan.n:
        raise ValueError(f"R has {rows} rows, the plan {plan.n}")
    Y, ldy = _out16(Y, "Y", tokens, H, R.device)
    _call(dev, "qf_moe_combine", R.data_ptr(), ldr, plan.positions.data_ptr(), _ptr(weights), tokens, k, H, Y.data_ptr(), ldy)
    return Y


def qf_moe_combine_backward(dY, R, plan, weights=None, k=None, d_rows=None, d_weights=None, want=(True, True)):
    """(d_rows bf16 [plan.n, H], d_weights float32 [tokens, k]) of qf_moe_combine: d_rows[p] =
    weights * dY[t], d_weights = <R[p], dY[t]>; None for what is not wanted.  Rows of d_rows behind
    the last group are left as they were (unspecified where d_rows is new)."""
    tokens, k = _combine(plan, weights, k)
    if not want[1]:
        R = None
    dev = _same_gpu(dY, R, weights, d_rows, d_weights, plan.order)
    rows, H, ldd = _mat(_bf16(dY, "dY"), "dY")
    if rows != tokens:
        raise ValueError(f"dY has {rows} rows for {tokens} tokens")
    ldr = ldo = H
    if want[1]:
        if tuple(_bf16(R, "R").shape) != (plan.n, H):
            raise ValueError(f"R has shape {tuple(R.shape)}, want {(plan.n, H)}")
        ldr = _mat(R, "R")[2]
        if d_weights is None:
            d_weights = torch.empty(tokens, k, dtype=torch.float32, device=dY.device)
        else:
            _dense(d_weights, "d_weights", torch.float32, (tokens, k))
    if want[0]:
        d_rows, ldo = _out16(d_rows, "d_rows", plan.n, H, dY.device)
    _call(dev, "qf_moe_combine_backward", dY.data_ptr(), ldd, _ptr(R), ldr, plan.positions.data_ptr(), _ptr(weights), tokens,
          k, H, d_rows.data_ptr() if want[0] else None, ldo, d_weights.data_ptr() if want[1] else None)
    return (d_rows if want[0] else None), (d_weights if want[1] else None)


# ------------------------------------------------- 8-bit blocks of 128 ----
FP8_BLOCK = 128


def _codes(t, name, shape=None):
    """A uint8 matrix of codes with contiguous rows: its row stride."""
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be torch.uint8")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, want {shape}")
    return _mat(t, name)[2]


def _row_codes(rows, cols, device, codes, scales):
    """Outputs of a row quantization, with their row strides."""
    blocks = (cols + FP8_BLOCK - 1) // FP8_BLOCK
    if codes is None:
        codes, ldc = torch.empty(rows, cols, dtype=torch.uint8, device=device), cols
    else:
        ldc = _codes(codes, "codes", (rows, cols))
    if scales is None:
        return codes, ldc, torch.empty(blocks, rows, dtype=torch.float32, device=device), rows
    return codes, ldc, scales, _scales(scales, "scales", blocks, rows)


def _scales(t, name, blocks, rows):
    """Block-major scales [blocks, rows]: their row stride."""
    if t.dtype != torch.float32 or tuple(t.shape) != (blocks, rows):
        raise ValueError(f"{name} must be a float32 tensor of shape {(blocks, rows)}")
    return _mat(t, name)[2]


def qf_quant_fp8(x, plan=None, rows_per_x=None, codes=None, scales=None):
    """(codes uint8 [rows, cols], scales float32 [ceil(cols / 128), rows]): E4M3 codes of x bf16 in
    blocks of 128 along its rows.  plan: with rows_per_x, row plan.positions[i] is x[i // rows_per_x]
    (rows into expert order on the way); without, x's rows are in that order already.  Rows behind
    the plan's last group are left as they were (unspecified in new outputs)."""
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    dev = _same_gpu(x, codes, scales, None if plan is None else _plan(plan).order)
    positions = used = None
    if plan is not None:
        _x_rows(rows, plan.n, 1 if rows_per_x is None else rows_per_x)
        rows = plan.n
        if rows_per_x is None:
            used = plan.offsets.data_ptr() + 4 * plan.n_ids
        else:
            positions = _positions(plan)
    elif rows_per_x is not None:
        raise ValueError("rows_per_x needs a plan")
    codes, ldc, scales, lds = _row_codes(rows, cols, x.device, codes, scales)
    _call(dev, "qf_quant_fp8", x.data_ptr(), ldx, rows, cols, positions, rows_per_x or 1, used, codes.data_ptr(), ldc,
          scales.data_ptr(), lds)
    return codes, scales


def qf_fp8_panels(rows, n_ids=1):
    """Panels of 128 rows that rows in n_ids groups fill at most."""
    return lib().qf_fp8_panels(int(rows), int(n_ids))


def _panels(t, name, dtype, shape):
    """Panels or their scales, with room for at least shape[0]."""
    return _dense(t, name, dtype, (max(t.shape[0], shape[0]) if t.dim() else 0,) + shape[1:])


def qf_quant_fp8_panels(x, plan=None, rows_per_x=None, codes=None, scales=None):
    """(codes uint8 [panels, cols, 128], scales float32 [panels, cols]): E4M3 codes of x bf16 in blocks
    of 128 rows of one group of the plan (None: all rows are one), transposed, the operands of
    qf_gemm_fp8_wgrad.  rows_per_x as qf_quant_fp8.  codes and scales may hold more panels than
    qf_fp8_panels says; panels behind the last are left as they were."""
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    dev = _same_gpu(x, codes, scales, None if plan is None else _plan(plan).order)
    order = offsets = None
    n_ids = 1
    if plan is not None:
        _x_rows(rows, plan.n, 1 if rows_per_x is None else rows_per_x)
        rows, n_ids, offsets = plan.n, plan.n_ids, plan.offsets.data_ptr()
        order = None if rows_per_x is None else plan.order.data_ptr()
    elif rows_per_x is not None:
        raise ValueError("rows_per_x needs a plan")
    panels = lib().qf_fp8_panels(rows, n_ids)
    if codes is None:
        codes = torch.empty(panels, cols, FP8_BLOCK, dtype=torch.uint8, device=x.device)
    else:
        _panels(codes, "codes", torch.uint8, (panels, cols, FP8_BLOCK))
    if scales is None:
        scales = torch.empty(panels, cols, dtype=torch.float32, device=x.device)
    else:
        _panels(scales, "scales", torch.float32, (panels, cols))
    _call(dev, "qf_quant_fp8_panels", x.data_ptr(), ldx, rows, cols, order, rows_per_x or 1, offsets, n_ids,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def qf_quant_fp8_tiles(x, transpose=False, codes=None, scales=None, codes_t=None, scales_t=None):
    """(codes, scales) of x bf16 [rows, cols] or [count, rows, cols] in tiles of 128 x 128: codes of
    x's shape, scales float32 [..., ceil(rows / 128), ceil(cols / 128)]; with transpose also
    (codes_t, scales_t), the same values as codes and scales of x's transpose."""
    if _bf16(x, "x").dim() not in (2, 3):
        raise ValueError("x must be a 2-D or 3-D tensor")
    dev = _same_gpu(x, codes, scales, codes_t, scales_t)
    count = x.shape[0] if x.dim() == 3 else 1
    lead, (rows, cols) = tuple(x.shape[:-2]), x.shape[-2:]
    ld = x.stride(-2) if rows > 1 else x.stride(0) if rows and count > 1 else cols       # (a single row's own stride says nothing)
    if (x.stride(-1) != 1 and cols > 1) or (rows and count > 1 and x.stride(0) != rows * ld):
        raise ValueError("x must have contiguous rows, and its matrices must follow one another")
    rt, ct = (rows + FP8_BLOCK - 1) // FP8_BLOCK, (cols + FP8_BLOCK - 1) // FP8_BLOCK
    outs = [(codes, "codes", torch.uint8, lead + (rows, cols)), (scales, "scales", torch.float32, lead + (rt, ct))]
    if transpose:
        outs += [(codes_t, "codes_t", torch.uint8, lead + (cols, rows)), (scales_t, "scales_t", torch.float32, lead + (ct, rt))]
    elif codes_t is not None or scales_t is not None:
        raise ValueError("codes_t and scales_t need transpose=True")
    outs = [torch.empty(shape, dtype=kind, device=x.device) if t is None else _dense(t, name, kind, shape)
            for t, name, kind, shape in outs]
    _call(dev, "qf_quant_fp8_tiles", x.data_ptr(), ld, count, rows, cols, outs[0].data_ptr(), outs[1].data_ptr(),
          outs[2].data_ptr() if transpose else None, outs[3].data_ptr() if transpose else None)
    return tuple(outs)


def qf_swiglu_quant_fp8(h, plan=None, y=None, codes=None, scales=None):
    """(codes uint8 [rows, cols], scales float32 [ceil(cols / 128), rows]) of u * g * sigmoid(g), h bf16
    [rows, 2 cols] = [g, u], as qf_quant_fp8 lays them out; y (bf16 [rows, cols]) gets the product as
    well.  plan: rows behind its last group are left as they were."""
    rows, wide, ldh = _mat(_bf16(h, "h"), "h")
    dev = _same_gpu(h, y, codes, scales, None if plan is None else _plan(plan).order)
    if wide % 2 or (plan is not None and plan.n != rows):
        raise ValueError(f"h has shape {tuple(h.shape)}" + ("" if plan is None else f" for {plan.n} rows of the plan"))
    cols = wide // 2
    codes, ldc, scales, lds = _row_codes(rows, cols, h.device, codes, scales)
    ldy = cols
    if y is not None:
        y, ldy = _out16(y, "y", rows, cols, h.device)
    _call(dev, "qf_swiglu_quant_fp8", h.data_ptr(), ldh, rows, cols,
          None if plan is None else plan.offsets.data_ptr() + 4 * plan.n_ids, codes.data_ptr(), ldc, scales.data_ptr(), lds,
          _ptr(y), ldy)
    return codes, scales


def qf_swiglu_backward(h, da, plan=None, dh=None):
    """dh bf16 [rows, 2 cols] of a = u * g * sigmoid(g), h = [g, u], from da bf16 [rows, cols].  plan: rows
    behind its last group are left as they were (unspecified where dh is new)."""
    rows, wide, ldh = _mat(_bf16(h, "h"), "h")
    dev = _same_gpu(h, da, dh, None if plan is None else _plan(plan).order)
    if wide % 2 or (plan is not None and plan.n != rows) or tuple(_bf16(da, "da").shape) != (rows, wide // 2):
        raise ValueError(f"shapes h {tuple(h.shape)}, da {tuple(da.shape)} do not fit")
    dh, ldo = _out16(dh, "dh", rows, wide, h.device)
    _call(dev, "qf_swiglu_backward", h.data_ptr(), ldh, da.data_ptr(), _mat(da, "da")[2], rows, wide // 2,
          None if plan is None else plan.offsets.data_ptr() + 4 * plan.n_ids, dh.data_ptr(), ldo)
    return dh


def qf_gemm_fp8(Xc, Xs, Wc, Ws, Y=None):
    """Y bf16 [M, N] = X W^T of E4M3 codes: Xc [M, K] and Xs [ceil(K / 128), M] as qf_quant_fp8 gives
    them, Wc [N, K] and Ws [ceil(N / 128), ceil(K / 128)] as qf_quant_fp8_tiles."""
    dev = _same_gpu(Xc, Xs, Wc, Ws, Y)
    ldx, ldw = _codes(Xc, "Xc"), _codes(Wc, "Wc")
    (M, K), (N, K2) = Xc.shape, Wc.shape
    if K != K2:
        raise ValueError(f"Xc has K={K} but Wc has K={K2}")
    blocks = (K + FP8_BLOCK - 1) // FP8_BLOCK
    ldxs = _scales(Xs, "Xs", blocks, M)
    _dense(Ws, "Ws", torch.float32, ((N + FP8_BLOCK - 1) // FP8_BLOCK, blocks))
    Y, ldy = _out16(Y, "Y", M, N, Xc.device)
    _call(dev, "qf_gemm_fp8", Xc.data_ptr(), ldx, Xs.data_ptr(), ldxs, Wc.data_ptr(), ldw, Ws.data_ptr(), Y.data_ptr(), ldy,
          M, N, K)
    return Y


def qf_gemm_fp8_grouped(Xc, Xs, Wc, Ws, plan, Y=None):
    """qf_gemm_fp8 for rows in a plan's order, each group with its own weights: Wc [n_ids, N, K], Ws
    [n_ids, ceil(N / 128), ceil(K / 128)].  Rows of Y behind the last group are left as they were
    (unspecified where Y is new)."""
    dev = _same_gpu(Xc, Xs, Wc, Ws, Y, _plan(plan).order)
    ldx = _codes(Xc, "Xc")
    if Wc.dtype != torch.uint8 or Wc.dim() != 3 or not Wc.is_contiguous():
        raise ValueError("Wc must be a contiguous 3-D uint8 tensor")
    (M, K), (E, N, K2) = Xc.shape, Wc.shape
    if K != K2 or M != plan.n or E != plan.n_ids:
        raise ValueError(f"shapes Xc {tuple(Xc.shape)}, Wc {tuple(Wc.shape)} do not fit a plan of {plan.n} rows, {plan.n_ids} ids")
    blocks = (K + FP8_BLOCK - 1) // FP8_BLOCK
    ldxs = _scales(Xs, "Xs", blocks, M)
    _dense(Ws, "Ws", torch.float32, (E, (N + FP8_BLOCK - 1) // FP8_BLOCK, blocks))
    Y, ldy = _out16(Y, "Y", M, N, Xc.device)
    _call(dev, "qf_gemm_fp8_grouped", Xc.data_ptr(), ldx, Xs.data_ptr(), ldxs, Wc.data_ptr(), K, Ws.data_ptr(),
          plan.offsets.data_ptr(), plan.tiles.data_ptr(), E, Y.data_ptr(), ldy, M, N, K)
    return Y


def qf_gemm_fp8_wgrad(Dc, Ds, Xc, Xs, plan=None, dW=None):
    """dW bf16 [n_ids, N, K] (plan None: [N, K]) from the panels of dY (Dc [panels, N, 128], Ds
    [panels, N]) and X (Xc [panels, K, 128], Xs) under the same plan (qf_quant_fp8_panels; panels behind
    its last are not read, without a plan all are summed): the gradient of qf_gemm_fp8_grouped's weights,
    zero for a group without rows."""
    dev = _same_gpu(Dc, Ds, Xc, Xs, dW, None if plan is None else _plan(plan).order)
    if Dc.dim() != 3 or Xc.dim() != 3:
        raise ValueError("Dc and Xc must be panels [panels, cols, 128]")
    panels, N, K = Dc.shape[0], Dc.shape[1], Xc.shape[1]
    rows = panels * FP8_BLOCK if plan is None else plan.n
    n_ids = 1 if plan is None else plan.n_ids
    check = _dense                                   # without a plan every panel is taken
    if plan is not None:
        panels, check = lib().qf_fp8_panels(rows, n_ids), _panels
    for c, s, cols, name in ((Dc, Ds, N, "D"), (Xc, Xs, K, "X")):
        check(c, name + "c", torch.uint8, (panels, cols, FP8_BLOCK))
        check(s, name + "s", torch.float32, (panels, cols))
    shape = (N, K) if plan is None else (n_ids, N, K)
    if dW is None:
        dW = torch.empty(shape, dtype=torch.bfloat16, device=Dc.device)
    else:
        _dense(dW, "dW", torch.bfloat16, shape)
    _call(dev, "qf_gemm_fp8_wgrad", Dc.data_ptr(), Ds.data_ptr(), Xc.data_ptr(), Xs.data_ptr(),
          None if plan is None else plan.offsets.data_ptr(), n_ids, rows, dW.data_ptr(), N, K)
    return dW


# ------------------------------------- adapters of many requests at once ----
def qf_lora_apply_workspace(rows, K, r, n_adapters, planned=False):
    return lib().qf_lora_apply_workspace(int(rows), int(K), int(r), int(n_adapters), int(bool(planned)))


def _lora_apply(name, X, A, B, where, Y, scale, rows_per_x, ws):
    plan = where if isinstance(where, RowPlan) else None
    dev = _same_gpu(X, A, B, Y, scale, ws, where if plan is None else plan.order)
    xrows, K, ldx = _mat(_bf16(X, "X"), "X")
    rows, N, ldy = _mat(_bf16(Y, "Y"), "Y")
    for t, what in ((A, "A"), (B, "B")):
        if _bf16(t, what).dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous 3-D tensor [adapters, ...]")
    E, r, AK = A.shape
    if AK != K or B.shape != (E, N, r):
        raise ValueError(f"adapter shapes {tuple(A.shape)}, {tuple(B.shape)} do not fit X {tuple(X.shape)}, Y {tuple(Y.shape)}")
    if rows_per_x < 1 or xrows != (rows + rows_per_x - 1) // rows_per_x:
        raise ValueError(f"X has {xrows} rows for {rows} rows of Y and rows_per_x={rows_per_x}")
    if scale is not None and (scale.dtype != torch.float32 or not scale.is_contiguous() or scale.numel() != E):
        raise ValueError("scale must be a contiguous float32 tensor with a value per adapter")
    if plan is not None and (plan.n != rows or plan.n_ids > E):
        raise ValueError(f"the plan is for {plan.n} rows of {plan.n_ids} adapters")
    if plan is None and _ids(where, "ids").numel() != rows:
        raise ValueError("ids must hold an id per row of Y")
    if ws is None:
        ws_bytes = lib().qf_lora_apply_workspace(rows, K, r, E, plan is not None)
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=X.device)
    else:
        ws_bytes = _space(ws)
    if plan is None:
        _call(dev, name, X.data_ptr(), ldx, rows_per_x, A.data_ptr(), B.data_ptr(), _ptr(scale), E, where.data_ptr(),
              Y.data_ptr(), ldy, rows, N, K, r, _ptr(ws), ws_bytes)
    else:
        _call(dev, name, X.data_ptr(), ldx, rows_per_x, A.data_ptr(), B.data_ptr(), _ptr(scale), E,
              plan.offsets.data_ptr(), plan.order.data_ptr(), plan.tiles.data_ptr(), plan.n_ids, Y.data_ptr(), ldy, rows, N,
              K, r, _ptr(ws), ws_bytes)
    return Y


def qf_lora_apply(X, A, B, ids, Y, scale=None, rows_per_x=1, ws=None):
    """Y[i] += scale[e] * B[e] (A[e] X[i // rows_per_x]), e = ids[i] (none outside [0, E)), in
    place: X [rows / rows_per_x, K], A [E, r, K], B [E, N, r], Y [rows, N] bf16, ids int32."""
    if isinstance(ids, RowPlan):
        raise TypeError("ids must be a tensor; qf_lora_apply_planned takes a RowPlan")
    return _lora_apply("qf_lora_apply", X, A, B, ids, Y, scale, rows_per_x, ws)


def qf_lora_apply_planned(X, A, B, plan, Y, scale=None, rows_per_x=1, ws=None):
    """qf_lora_apply with the RowPlan of the rows' ids, which serves every projection of a batch."""
    if not isinstance(plan, RowPlan):
        raise TypeError("plan must be a RowPlan")
    return _lora_apply("qf_lora_apply_planned", X, A, B, plan, Y, scale, rows_per_x, ws)


# --------------------------------------------------------------- AdamW ----
ADAMW_BLOCK = 256


def _flat(t, name, dtype, n):
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def adamw_state(n, state_bits=32, device="cuda"):
    """Zeroed moments of a tensor of n elements: dict(m, v) in fp32, or dict(m, v, m_scale,
    v_scale) for 8-bit states."""
    if state_bits not in (8, 32):
        raise ValueError("state_bits is 8 or 32")
    kind = torch.uint8 if state_bits == 8 else torch.float32
    s = {k: torch.zeros(n, dtype=kind, device=device) for k in ("m", "v")}
    if state_bits == 8:
        blocks = (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK
        s.update({k: torch.zeros(blocks, dtype=torch.float32, device=device) for k in ("m_scale", "v_scale")})
    return s


class AdamwBatch:
    """Descriptors of the tensors that qf_adamw_step updates, built once and reusable.

    items: list of dict(p, g, m, v, m_scale=None, v_scale=None, p16=None, weight_decay=0.0) of
    contiguous device tensors with the same element count: p float32, g float32 or bfloat16,
    m and v float32 (state_bits 32) or uint8 with float32 scales per 256 elements (8), p16
    bfloat16.  The batch holds the tensors; they must keep their storage while it is used (a
    gradient put elsewhere needs a new batch).  More than FEW
    tensors are described by a table in device memory (built here, outside a stream capture),
    so that a step is one launch per gradient type; a graph that captured the step reads the
    table on every replay, so the batch must outlive it.
    """

    FEW = 8

    def __init__(self, items, state_bits=32):
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        # own copies of the dicts: the step writes through the tensors' addresses, so they stay alive
        # here whatever becomes of the caller's
        items = [dict(it) for it in items]
        self.items, self.state_bits, self.n = items, state_bits, len(items)
        self.arr = (AdamwTensor * max(len(items), 1))()
        self.device = _same_gpu(*[t for it in items for t in it.values() if isinstance(t, torch.Tensor)])
        state = torch.uint8 if state_bits == 8 else torch.float32
        written = []                                     # (address, bytes) of what the step writes
        for i, it in enumerate(items):
            n = it["p"].numel()
            d = self.arr[i]
            d.p = _flat(it["p"], "p", torch.float32, n)
            if it["g"].dtype not in (torch.float32, torch.bfloat16):
                raise TypeError("g must be float32 or bfloat16")
            d.g = _flat(it["g"], "g", it["g"].dtype, n)
            d.g_bf16 = int(it["g"].dtype == torch.bfloat16)
            d.m, d.v = _flat(it["m"], "m", state, n), _flat(it["v"], "v", state, n)
            if state_bits == 8:
                blocks = (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK
                d.m_scale = _flat(it["m_scale"], "m_scale", torch.float32, blocks)
                d.v_scale = _flat(it["v_scale"], "v_scale", torch.float32, blocks)
            if it.get("p16") is not None:
                d.p16 = _flat(it["p16"], "p16", torch.bfloat16, n)
            d.n, d.weight_decay = n, float(it.get("weight_decay", 0.0))
            if n:
                size = n * state_bits // 8
                written += ((d.p, n * 4), (d.m, size), (d.v, size))
                if state_bits == 8:
                    written += ((d.m_scale, blocks * 4), (d.v_scale, blocks * 4))
                if d.p16:
                    written.append((d.p16, n * 2))
        # the tensors of a launch run at the same time
        written.sort()
        if any(a + size > b for (a, size), (b, _) in zip(written, written[1:])):
            raise ValueError("a tensor may appear once per batch, and what a step writes must not overlap")
        self.ref = ctypes.byref(self.arr)
        self.plan = self.table = None
        if self.n > self.FEW:
            host = torch.empty(lib().qf_adamw_table_bytes(self.n), dtype=torch.uint8)
            self.plan = AdamwPlan()
            _check(lib().qf_adamw_table(self.ref, self.n, state_bits, host.data_ptr(), host.numel(),
                                        ctypes.byref(self.plan)), "qf_adamw_table")
            self.table = host.to(torch.device("cuda", self.device))
            self.stream = torch._C._cuda_getCurrentRawStream(self.device)


def qf_adamw_step(batch, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, seed=0, d_lr=None, d_step=None,
                  d_grad_scale=None, d_skip=None):
    """One AdamW step of every tensor of an AdamwBatch, in place.  step counts from 1.  d_lr
    (float32 [1]) and d_step (int64 [1]) on the device replace lr and step (a captured step
    reads them on every replay); d_grad_scale (float32 [1]) multiplies the gradients; nothing
    is written where d_skip (int32 or uint32 [1]) is not 0.  seed: of the 8-bit states'
    stochastic rounding."""
    for t, name, kinds in ((d_lr, "d_lr", (torch.float32,)), (d_step, "d_step", (torch.int64,)),
                           (d_grad_scale, "d_grad_scale", (torch.float32,)),
                           (d_skip, "d_skip", (torch.int32, torch.uint32))):
        if t is not None and (t.dtype not in kinds or t.numel() != 1 or t.get_device() < 0 or
                              batch.device >= 0 and t.get_device() != batch.device):
            raise TypeError(f"{name} must be one {kinds[0]} on the tensors' device")
    h = AdamwHyper(lr, beta1, beta2, eps, step, _ptr(d_lr), _ptr(d_step), _ptr(d_grad_scale), _ptr(d_skip),
                   seed & 0xFFFFFFFF)
    if batch.table is None:
        _call(batch.device, "qf_adamw_step", batch.ref, batch.n, batch.state_bits, ctypes.byref(h))
    else:
        # a step on another stream than the table's: the allocator keeps the table until that step is done
        if torch._C._cuda_getCurrentRawStream(batch.device) != batch.stream and not torch.cuda.is_current_stream_capturing():
            batch.table.record_stream(torch.cuda.current_stream(batch.device))
        _call(batch.device, "qf_adamw_step_table", ctypes.byref(batch.plan), batch.table.data_ptr(), ctypes.byref(h))


# ------------------------------------------------------------- dequant ----
def _dequant_out(rows, cols, device, y):
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.bfloat16, device=device)
    _bf16(y, "y")
    if tuple(y.shape) != (rows, cols):
        raise ValueError(f"y has shape {tuple(y.shape)}, want {(rows, cols)}")
    return y


def _u8(t, name):
    if t.dtype != torch.uint8 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous uint8 tensor")
    return t


def qf_dequant_nvfp4(codes, scales, d_scale, y=None):
    """bf16 [rows, cols] from NVFP4 codes [rows, cols/2] and E4M3 scales [rows, cols/16]."""
    rows, cols = _u8(codes, "codes").shape[0], codes.shape[1] * 2
    y = _dequant_out(rows, cols, codes.device, y)
    _check(lib().qf_dequant_nvfp4(_p(codes), _p(_u8(scales, "scales")), rows, cols, _p(d_scale), _p(y),
                                  _mat(y, "y")[2], _stream()), "qf_dequant_nvfp4")
    return y


def qf_dequant_mxfp4(codes, scales, y=None):
    """bf16 [rows, cols] from MXFP4 codes [rows, cols/2] and E8M0 scales [rows, cols/32]."""
    rows, cols = _u8(codes, "codes").shape[0], codes.shape[1] * 2
    y = _dequant_out(rows, cols, codes.device, y)
    _check(lib().qf_dequant_mxfp4(_p(codes), _p(_u8(scales, "scales")), rows, cols, _p(y), _mat(y, "y")[2],
                                  _stream()), "qf_dequant_mxfp4")
    return y


def qf_dequant_q4k(blocks, rows, cols, y=None):
    """bf16 [rows, cols] from Q4_K blocks (rows * cols / 256 blocks of 144 bytes)."""
    _u8(blocks, "blocks")
    if blocks.numel() != rows * (cols // 256) * 144:
        raise ValueError("blocks do not match rows x cols")
    y = _dequant_out(rows, cols, blocks.device, y)
    _check(lib().qf_dequant_q4k(_p(blocks), rows, cols, _p(y), _mat(y, "y")[2], _stream()), "qf_dequant_q4k")
    return y


# ---------------------------------------------------------------- GEMM ----
def qf_gemm_mxfp4(X, W, Y=None, flags=QF_QDQ_A | QF_QDQ_W):
    """Y[M, N] = QDQ(X)[M, K] . QDQ(W)[N, K]^T (bf16 in, fp32 accumulate, bf16 out)."""
    M, K, ldx = _mat(_bf16(X, "X"), "X")
    N, K2, ldw = _mat(_bf16(W, "W"), "W")
    if K2 != K:
        raise ValueError(f"X has K={K} but W has K={K2}")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _bf16(Y, "Y")
    _check(lib().qf_gemm_mxfp4(_p(X), ldx, _p(W), ldw, _p(Y), _mat(Y, "Y")[2], M, N, K, int(flags), _stream()),
           "qf_gemm_mxfp4")
    return Y


def qf_gemm_nvfp4(X, W, d_scale_x, d_scale_w, Y=None, flags=QF_QDQ_A | QF_QDQ_W):
    """Y[M, N] = QDQ(X) . QDQ(W)^T on the NVFP4 grid with the device fp32 tensor scales
    d_scale_x, d_scale_w (one element each; None for an operand that is not quantized)."""
    M, K, ldx = _mat(_bf16(X, "X"), "X")
    N, K2, ldw = _mat(_bf16(W, "W"), "W")
    if K2 != K:
        raise ValueError(f"X has K={K} but W has K={K2}")
    for t, name in ((d_scale_x, "d_scale_x"), (d_scale_w, "d_scale_w")):
        if t is not None and (t.dtype != torch.float32 or t.device.type != "cuda"):
            raise TypeError(f"{name} must be a float32 device tensor")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _bf16(Y, "Y")
    _check(lib().qf_gemm_nvfp4(_p(X), ldx, _p(W), ldw, _p(Y), _mat(Y, "Y")[2], M, N, K, int(flags), _p(d_scale_x),
                               _p(d_scale_w), _stream()), "qf_gemm_nvfp4")
    return Y


def _linear_forward_args(X, W, Y, Xq, Wq, flags):
    M, K, ldx = _mat(_bf16(X, "X"), "X")
    N, K2, ldw = _mat(_bf16(W, "W"), "W")
    if K2 != K:
        raise ValueError(f"X has K={K} but W has K={K2}")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if Xq is None and flags & QF_QDQ_A:
        Xq = torch.empty((M, K), dtype=torch.bfloat16, device=X.device)
    if Wq is None and flags & QF_QDQ_W:
        Wq = torch.empty((N, K), dtype=torch.bfloat16, device=X.device)
    _bf16(Y, "Y")
    ldxq = _mat(_bf16(Xq, "Xq"), "Xq")[2] if Xq is not None else 0
    ldwq = _mat(_bf16(Wq, "Wq"), "Wq")[2] if Wq is not None else 0
    return M, N, K, ldx, ldw, Y, Xq, ldxq, Wq, ldwq


def qf_linear_forward_mxfp4(X, W, Y=None, flags=QF_QDQ_A | QF_QDQ_W, Xq=None, Wq=None):
    """(Y, Xq, Wq): Xq = QDQ(X), Wq = QDQ(W) (MXFP4, for the flagged operands), then
    Y = Xq . Wq^T on the BF16 matrix cores; Y equals qf_gemm_mxfp4(X, W, flags) bit for bit."""
    M, N, K, ldx, ldw, Y, Xq, ldxq, Wq, ldwq = _linear_forward_args(X, W, Y, Xq, Wq, flags)
    _check(lib().qf_linear_forward_mxfp4(_p(X), ldx, _p(W), ldw, _p(Y), _mat(Y, "Y")[2], M, N, K, int(flags),
                                         _p(Xq), ldxq, _p(Wq), ldwq, _stream()), "qf_linear_forward_mxfp4")
    return Y, Xq, Wq


def qf_linear_forward_nvfp4(X, W, d_scale_x, d_scale_w, Y=None, flags=QF_QDQ_A | QF_QDQ_W, Xq=None, Wq=None):
    """(Y, Xq, Wq) as qf_linear_forward_mxfp4 on the NVFP4 grid with the device fp32 tensor
    scales d_scale_x, d_scale_w; Y equals qf_gemm_nvfp4 with the same arguments bit for bit."""
    for t, name in ((d_scale_x, "d_scale_x"), (d_scale_w, "d_scale_w")):
        if t is not None and (t.dtype != torch.float32 or t.device.type != "cuda"):
            raise TypeError(f"{name} must be a float32 device tensor")
    M, N, K, ldx, ldw, Y, Xq, ldxq, Wq, ldwq = _linear_forward_args(X, W, Y, Xq, Wq, flags)
    _check(lib().qf_linear_forward_nvfp4(_p(X), ldx, _p(W), ldw, _p(Y), _mat(Y, "Y")[2], M, N, K, int(flags),
                                         _p(d_scale_x), _p(d_scale_w), _p(Xq), ldxq, _p(Wq), ldwq, _stream()),
           "qf_linear_forward_nvfp4")
    return Y, Xq, Wq


def qf_transpose_bf16(x, y=None, qdq_mxfp4=False, rule=QF_MX_RULE_FLOOR):
    """y [cols, rows] = x^T, MXFP4-QDQ'd along x's rows first (under `rule`) when qdq_mxfp4."""
    rows, cols, ldx = _mat(_bf16(x, "x"), "x")
    if y is None:
        y = torch.empty((cols, rows), dtype=torch.bfloat16, device=x.device)
    _bf16(y, "y")
    _check(lib().qf_transpose_bf16(_p(x), rows, cols, ldx, _p(y), _mat(y, "y")[2], (1 + int(rule == QF_MX_RULE_NOCLIP)) if qdq_mxfp4 else 0, _stream()),
           "qf_transpose_bf16")
    return y


def qf_linear_backward_workspace(M, N, K):
    return lib().qf_linear_backward_workspace(M, N, K)


def qf_linear_backward_mxfp4(X, W, dY, dX=None, dW=None, flags=QF_QDQ_A | QF_QDQ_W, ws=None, want=(True, True)):
    """(dX, dW) of Y = Xq . Wq^T: dX = dY . Wq [M, K], dW = dY^T . Xq [N, K] (bf16)."""
    M, K, ldx = _mat(_bf16(X, "X"), "X")
    N, K2, ldw = _mat(_bf16(W, "W"), "W")
    M2, N2, lddy = _mat(_bf16(dY, "dY"), "dY")
    if K2 != K or M2 != M or N2 != N:
        raise ValueError(f"shapes X {tuple(X.shape)}, W {tuple(W.shape)}, dY {tuple(dY.shape)} do not fit")
    if dX is None and want[0]:
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=X.device)
    if dW is None and want[1]:
        dW = torch.empty((N, K), dtype=torch.bfloat16, device=X.device)
    need = lib().qf_linear_backward_workspace(M, N, K)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=X.device)
    _check(lib().qf_linear_backward_mxfp4(_p(X), ldx, _p(W), ldw, _p(dY), lddy, _p(dX),
                                          _mat(dX, "dX")[2] if dX is not None else 0, _p(dW),
                                          _mat(dW, "dW")[2] if dW is not None else 0, M, N, K, int(flags), _p(ws),
                                          ws.numel(), _stream()), "qf_linear_backward_mxfp4")
    return dX, dW


def qf_gemm_mxfp4_packed_w(X, Wc, Ws, Y=None):
    """Y[M, N] = QDQ(X) . dequant(Wc, Ws)^T on the MXFP4 matrix cores; Wc [N, K/2] and
    Ws [N, K/32] uint8 as qf_pack_mxfp4 writes them (contiguous)."""
    M, K, ldx = _mat(_bf16(X, "X"), "X")
    if Wc.dtype != torch.uint8 or Ws.dtype != torch.uint8 or not Wc.is_contiguous() or not Ws.is_contiguous():
        raise ValueError("Wc and Ws must be contiguous uint8 tensors")
    N = Wc.shape[0]
    if tuple(Wc.shape) != (N, K // 2) or tuple(Ws.shape) != (N, K // 32):
        raise ValueError(f"packed W shapes {tuple(Wc.shape)}, {tuple(Ws.shape)} do not fit K={K}")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _bf16(Y, "Y")
    _check(lib().qf_gemm_mxfp4_packed_w(_p(X), ldx, _p(Wc), _p(Ws), _p(Y), _mat(Y, "Y")[2], M, N, K, _stream()),
           "qf_gemm_mxfp4_packed_w")
    return Y


def qf_gemm_mxfp4_packed(Xc, Xs, Wc, Ws, Y=None):
    """Y[M, N] = dequant(Xc, Xs) . dequant(Wc, Ws)^T on the MXFP4 matrix cores; all four
    arrays uint8 as qf_pack_mxfp4 writes them (contiguous), K a multiple of 128."""
    for name, t in (("Xc", Xc), ("Xs", Xs), ("Wc", Wc), ("Ws", Ws)):
        if t.dtype != torch.uint8 or not t.is_contiguous() or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D uint8 tensor")
    M, N, K = Xc.shape[0], Wc.shape[0], Xc.shape[1] * 2
    if Wc.shape[1] * 2 != K or tuple(Xs.shape) != (M, K // 32) or tuple(Ws.shape) != (N, K // 32):
        raise ValueError("packed operand shapes do not agree")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=Xc.device)
    _bf16(Y, "Y")
    _check(lib().qf_gemm_mxfp4_packed(_p(Xc), _p(Xs), _p(Wc), _p(Ws), _p(Y), _mat(Y, "Y")[2], M, N, K, _stream()),
           "qf_gemm_mxfp4_packed")
    return Y


def qf_selftest_conversions(device="cuda"):
    counts = torch.zeros(8, dtype=torch.int64, device=device)
    _check(lib().qf_selftest_conversions(_p(counts), _stream()), "qf_selftest_conversions")
    return counts


# ------------------------------------------------- checkpoint containers ----
_ST_DTYPE = {torch.uint8: "U8", torch.int8: "I8", torch.bool: "BOOL", torch.float8_e4m3fn: "F8_E4M3",
             torch.float8_e5m2: "F8_E5M2", torch.float8_e8m0fnu: "F8_E8M0", torch.int16: "I16",
             torch.float16: "F16", torch.bfloat16: "BF16", torch.int32: "I32", torch.float32: "F32",
             torch.int64: "I64", torch.float64: "F64"}
_ST_SIZE = {"U8": 1, "I8": 1, "BOOL": 1, "F8_E4M3": 1, "F8_E5M2": 1, "F8_E8M0": 1, "U16": 2, "I16": 2, "F16": 2,
            "BF16": 2, "U32": 4, "I32": 4, "F32": 4, "U64": 8, "I64": 8, "F64": 8}


def _host_bytes(t):
    return t.detach().contiguous().cpu()


def _cstrings(strs):
    arr = (ctypes.c_char_p * max(len(strs), 1))(*[x.encode() for x in strs])
    return arr


def qf_write_safetensors(path, tensors, metadata=None):
    """Write a safetensors file.  tensors: list of (name, tensor, dtype) with tensor on any
    device and dtype a safetensors dtype string or None (taken from the tensor); a uint8
    tensor of E4M3 / E8M0 scale bytes is written as "F8_E4M3" / "F8_E8M0" by naming that
    dtype.  metadata: dict of str -> str."""
    keep = []
    arr = (StTensor * max(len(tensors), 1))()
    for i, (name, t, dt) in enumerate(tensors):
        h = _host_bytes(t)
        dt = dt or _ST_DTYPE.get(h.dtype)
        if dt is None or _ST_SIZE.get(dt) != h.element_size():
            raise TypeError(f"{name}: cannot write a {h.dtype} tensor as {dt}")
        shape = (ctypes.c_int64 * max(h.dim(), 1))(*h.shape)
        keep += [h, shape, name.encode(), dt.encode()]
        arr[i].name, arr[i].dtype, arr[i].ndim = keep[-2], keep[-1], h.dim()
        arr[i].shape = ctypes.cast(shape, ctypes.POINTER(ctypes.c_int64))
        arr[i].data = h.data_ptr() if h.numel() else None
    meta = metadata or {}
    keys, vals = _cstrings(list(meta)), _cstrings([str(v) for v in meta.values()])
    _check(lib().qf_write_safetensors(str(path).encode(), ctypes.byref(arr), len(tensors), keys, vals, len(meta)),
           "qf_write_safetensors")


def qf_write_gguf(path, tensors, kv=None):
    """Write a GGUF-style file.  tensors: list of (name, tensor of raw bytes, dims innermost
    first, type code); kv: dict of str -> str."""
    keep = []
    arr = (GgufTensor * max(len(tensors), 1))()
    for i, (name, t, dims, typ) in enumerate(tensors):
        h = _host_bytes(t)
        d = (ctypes.c_int64 * len(dims))(*dims)
        keep += [h, d, name.encode()]
        arr[i].name, arr[i].ndim = keep[-1], len(dims)
        arr[i].dims = ctypes.cast(d, ctypes.POINTER(ctypes.c_int64))
        arr[i].type, arr[i].data = int(typ), (h.data_ptr() if h.numel() else None)
        arr[i].nbytes = h.numel() * h.element_size()
    kv = kv or {}
    keys, vals = _cstrings(list(kv)), _cstrings([str(v) for v in kv.values()])
    _check(lib().qf_write_gguf(str(path).encode(), ctypes.byref(arr), len(tensors), keys, vals, len(kv)),
           "qf_write_gguf")


GGUF_TYPE_Q4_K = 12
Q4K_BLOCK_LAYOUT = ("144-byte blocks per 256 weights along a row: d (fp16 LE), dmin (fp16 LE), a 96-bit "
                    "little-endian stream with the 6-bit sub-block scale j at bits 6j and min j at bits 48+6j, "
                    "128 code bytes with element 2i in the low nibble and 2i+1 in the high nibble; "
                    "w = d*sc_j*q - dmin*m_j")


def export_fp4_tensors(prefix, fmt, codes, scales, d_scale=None, d_input_scale=None):
    """The (name, tensor, dtype) list of one packed NVFP4 / MXFP4 layer in the names this
    library uses ("compressed-tensors-style"): weight_packed, weight_scale (E4M3 or E8M0
    bytes), and for NVFP4 weight_global_scale (the layer group's dequant multiplier s_t)
    and, when given, input_global_scale (the tracked activation s_t)."""
    out = [(f"{prefix}.weight_packed", codes, "U8"),
           (f"{prefix}.weight_scale", scales, "F8_E4M3" if fmt == QF_FMT_NVFP4 else "F8_E8M0")]
    if fmt == QF_FMT_NVFP4:
        if d_scale is None:
            raise ValueError("NVFP4 needs the tensor scale")
        out.append((f"{prefix}.weight_global_scale", d_scale.reshape(-1)[:1], "F32"))
        if d_input_scale is not None:
            out.append((f"{prefix}.input_global_scale", d_input_scale.reshape(-1)[:1], "F32"))
    return out


def export_q4k_tensor(name, blocks, rows, cols):
    """The (name, bytes, dims, type) entry of one Q4_K matrix for qf_write_gguf."""
    return (name, blocks, (cols, rows), GGUF_TYPE_Q4_K)
