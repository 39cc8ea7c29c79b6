"""The operators on either side of the gradient reduction (argument
marshalling only, as in the package's other calls): the products of a linear
layer, forward and backward (``dpred_linear*``), and the orthogonalised
optimizer step that an owner runs on its whole gradient matrices
(``dpred_newton_schulz``, ``dpred_muon_step``).  All device work runs in
libdpred's kernels; there is no fallback."""
from __future__ import annotations

import ctypes
import math

ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = 0, 1, 2, 3
_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "silu": ACT_SILU,
         ACT_NONE: ACT_NONE, ACT_RELU: ACT_RELU, ACT_GELU: ACT_GELU, ACT_SILU: ACT_SILU, None: ACT_NONE}
NS_COEFFS = (3.4445, -4.7750, 2.0315)


class _MuonMatrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("momentum", ctypes.c_void_p), ("ldm", ctypes.c_int64),
                ("grad", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of these entry points on the loaded library."""
    i32, i64, vp, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    L.dpred_linear_workspace_bytes.restype = sz
    L.dpred_linear_workspace_bytes.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64]
    L.dpred_linear.argtypes = [i64, i64, i64, vp, i64, vp, i64, i32, vp, i32, vp, i64, vp, i64, i32, vp, i64, vp, sz,
                               vp]
    L.dpred_linear_dgrad.argtypes = [i64, i64, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp, sz, vp]
    L.dpred_linear_wgrad.argtypes = [i64, i64, i64, vp, i64, vp, i64, i32, i32, vp, i64, vp, vp, sz, vp]
    L.dpred_newton_schulz_workspace_bytes.restype = sz
    L.dpred_newton_schulz_workspace_bytes.argtypes = [i32, i64, i64]
    L.dpred_newton_schulz.argtypes = [i32, i64, i64, i32, vp, i64, i64, i32, vp, i64, i64, i32, vp, f32, vp, sz, vp]
    L.dpred_muon_workspace_bytes.restype = sz
    L.dpred_muon_workspace_bytes.argtypes = [vp, i32]
    L.dpred_muon_step.argtypes = [vp, i32, i32, i32, f32, f32, i32, f32, i32, vp, f32, vp, sz, vp]


def _zc():
    import zero_collectives_gb300 as zc
    return zc


def _matrix(t, name: str, dtypes, shape=None):
    """(data pointer, row stride) of a 2-D CUDA tensor with unit column stride."""
    import torch
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 2 or not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} must be a 2-D tensor on the current CUDA device")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    rs, cs = t.stride()
    if cs != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (rs if t.shape[0] > 1 else t.shape[1])


def _empty(shape, dtype, stream):
    """Device memory that belongs to the stream of the call."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(need: int, given, stream):
    import torch
    if given is not None:
        return given, given.data_ptr(), given.numel() * given.element_size()
    if not need:
        return None, None, 0
    ws = _empty(need, torch.uint8, stream)
    return ws, ws.data_ptr(), need


def _act(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"unknown activation {act!r}: none, relu, gelu or silu")
    return _ACTS[act]


def _unaligned(*mats) -> bool:
    return any(p % 16 or (r > 1 and ld % 8) for p, r, ld in mats)


def linear(x, w, bias=None, act="none", residual=None, preact=None, out=None, out_dtype=None, workspace=None,
           stream=None):
    """y = act(x w^T + bias) + residual.  x: bf16 [m, k]; w: bf16 [n, k]; bias:
    bf16 or fp32 [n]; residual: bf16 [m, n]; preact: bf16 [m, n], receives
    x w^T + bias (what linear_dgrad of the next layer down needs).  out: bf16
    or fp32 [m, n] (allocated on the call's stream when None).  Rows may be
    strided; m may be 1 (a single token)."""
    import torch
    zc = _zc()
    bf, ok = (torch.bfloat16,), (torch.bfloat16, torch.float32)
    xp, ldx = _matrix(x, "x", bf)
    m, k = x.shape
    wp, ldw = _matrix(w, "w", bf, (w.shape[0], k))
    n = w.shape[0]
    if out is None:
        out = _empty((m, n), out_dtype or torch.bfloat16, stream)
    yp, ldy = _matrix(out, "out", ok, (m, n))
    rp, ldr = (None, 0) if residual is None else _matrix(residual, "residual", bf, (m, n))
    pp, ldp = (None, 0) if preact is None else _matrix(preact, "preact", bf, (m, n))
    bp, bdt = None, 0
    if bias is not None:
        if tuple(bias.shape) != (n,) or bias.dtype not in ok or not bias.is_cuda or (n > 1 and bias.stride(0) != 1):
            raise ValueError("bias must be a contiguous bf16 or fp32 CUDA tensor of n elements")
        bp, bdt = bias.data_ptr(), zc._dtype_code(bias)
    L = zc.lib()
    need = L.dpred_linear_workspace_bytes(xp, m, k, ldx, wp, n, k, ldw) \
        if workspace is None and _unaligned((xp, m, ldx), (wp, n, ldw)) else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_linear(m, n, k, xp, ldx, wp, ldw, bdt, bp, _act(act), rp, ldr, pp, ldp, zc._dtype_code(out), yp,
                             ldy, wsp, wsb, zc._stream(stream)))
    return out


def linear_dgrad(dy, w, preact=None, act="none", residual=None, out=None, out_dtype=None, workspace=None,
                 stream=None):
    """dx = (dy w + residual) * act'(preact).  dy: bf16 [m, n]; w: bf16 [n, k];
    preact: the stored pre-activation of the layer below, bf16 [m, k] (needed
    unless act is "none"); residual: bf16 [m, k], the gradient that joins from
    a residual branch.  out: bf16 or fp32 [m, k]."""
    import torch
    zc = _zc()
    bf, ok = (torch.bfloat16,), (torch.bfloat16, torch.float32)
    dp, ldd = _matrix(dy, "dy", bf)
    m, n = dy.shape
    wp, ldw = _matrix(w, "w", bf, (n, w.shape[1]))
    k = w.shape[1]
    if out is None:
        out = _empty((m, k), out_dtype or torch.bfloat16, stream)
    op, ldo = _matrix(out, "out", ok, (m, k))
    a = _act(act)
    if a != ACT_NONE and preact is None:
        raise ValueError("an activation's gradient needs preact")
    zp, ldz = (None, 0) if preact is None or a == ACT_NONE else _matrix(preact, "preact", bf, (m, k))
    rp, ldr = (None, 0) if residual is None else _matrix(residual, "residual", bf, (m, k))
    L = zc.lib()
    need = L.dpred_linear_workspace_bytes(dp, m, n, ldd, wp, n, k, ldw) \
        if workspace is None and _unaligned((dp, m, ldd), (wp, n, ldw)) else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_linear_dgrad(m, n, k, dp, ldd, wp, ldw, a, zp, ldz, rp, ldr, zc._dtype_code(out), op, ldo, wsp,
                                   wsb, zc._stream(stream)))
    return out


def linear_wgrad(dy, x, out, bias_grad=None, accumulate: bool = False, workspace=None, stream=None):
    """out = dy^T x and bias_grad = column sums of dy, or both added to what
    the outputs hold (accumulate=True).  dy: bf16 [m, n]; x: bf16 [m, k]; out:
    [n, k] bf16 (a view of the gradient row that a flush reads) or fp32 (a view
    of the accumulator of accumulate_microbatch); bias_grad: fp32 [n]."""
    import torch
    zc = _zc()
    bf, ok = (torch.bfloat16,), (torch.bfloat16, torch.float32)
    dp, ldd = _matrix(dy, "dy", bf)
    m, n = dy.shape
    xp, ldx = _matrix(x, "x", bf, (m, x.shape[1]))
    k = x.shape[1]
    op, ldo = _matrix(out, "out", ok, (n, k))
    bp = None
    if bias_grad is not None:
        if tuple(bias_grad.shape) != (n,) or bias_grad.dtype != torch.float32 or not bias_grad.is_cuda \
                or (n > 1 and bias_grad.stride(0) != 1):
            raise ValueError("bias_grad must be a contiguous fp32 CUDA tensor of n elements")
        bp = bias_grad.data_ptr()
    L = zc.lib()
    need = L.dpred_linear_workspace_bytes(dp, m, n, ldd, xp, m, k, ldx) \
        if workspace is None and _unaligned((dp, m, ldd), (xp, m, ldx)) else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_linear_wgrad(m, n, k, dp, ldd, xp, ldx, int(accumulate), zc._dtype_code(out), op, ldo, bp, wsp,
                                   wsb, zc._stream(stream)))
    return out


def _coeffs(coeffs):
    return None if coeffs is None else (ctypes.c_float * 3)(*coeffs)


def newton_schulz(g, out=None, steps: int = 5, eps: float = 1e-7, coeffs=None, workspace=None, stream=None):
    """The orthogonalised matrix of g ([m, n], or [batch, m, n] of one shape;
    bf16 or fp32): `steps` steps of X = a X + (b A + c A^2) X, A = X X^T, from
    g / (|g|_F + eps).  out: bf16 (the default) or fp32, same shape; it carries
    16-bit accuracy either way (see dpred_newton_schulz)."""
    import torch
    zc = _zc()
    ok = (torch.bfloat16, torch.float32)
    if g.dim() not in (2, 3):
        raise ValueError("g must be [m, n] or [batch, m, n]")
    if out is None:
        out = _empty(tuple(g.shape), torch.bfloat16, stream)
    if tuple(out.shape) != tuple(g.shape):
        raise ValueError("out must have the shape of g")
    batch = g.shape[0] if g.dim() == 3 else 1
    if batch == 0:
        return out
    gp, ldg = _matrix(g[0] if g.dim() == 3 else g, "g", ok)
    op, ldo = _matrix(out[0] if g.dim() == 3 else out, "out", ok)
    gb, ob = (g.stride(0), out.stride(0)) if g.dim() == 3 else (0, 0)
    m, n = g.shape[-2:]
    L = zc.lib()
    need = L.dpred_newton_schulz_workspace_bytes(batch, m, n) if workspace is None else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_newton_schulz(batch, m, n, zc._dtype_code(g), gp, ldg, gb, zc._dtype_code(out), op, ldo, ob,
                                    int(steps), _coeffs(coeffs), float(eps), wsp, wsb, zc._stream(stream)))
    return out


def update_scale(rows: int, cols: int, rule) -> float:
    """Factor of the orthogonalised update of a rows x cols weight: "spectral"
    sqrt(max(1, rows / cols)), "rms" 0.2 sqrt(max(rows, cols)) (an update whose
    root mean square is near 0.2, for learning rates as AdamW's), or a number."""
    if rule == "spectral":
        return math.sqrt(max(1.0, rows / cols)) if cols else 1.0
    if rule == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    return float(rule)


def _muon_table(weights, momenta, grads, scale):
    import torch
    if not (len(weights) == len(momenta) == len(grads)):
        raise ValueError("weights, momenta and grads must have one entry per matrix")
    ok = (torch.bfloat16, torch.float32)
    table = (_MuonMatrix * max(len(weights), 1))()
    for i, (w, m, g) in enumerate(zip(weights, momenta, grads)):
        if w.dtype != weights[0].dtype or g.dtype != grads[0].dtype:
            raise TypeError("all weights must have one dtype, and all grads one")
        shape = tuple(w.shape)
        t = table[i]
        t.weight, t.ldw = _matrix(w, "weight", ok)
        t.momentum, t.ldm = _matrix(m, "momentum", (torch.float32,), shape)
        t.grad, t.ldg = _matrix(g, "grad", ok, shape)
        t.rows, t.cols = shape
        t.scale = update_scale(*shape, scale)
    return table


def muon_step(weights, momenta, grads, lr: float, momentum: float = 0.95, nesterov: bool = True,
              weight_decay: float = 0.0, scale="spectral", steps: int = 5, eps: float = 1e-7, coeffs=None,
              workspace=None, stream=None) -> None:
    """One orthogonalised-momentum step of a list of matrices, in place:
    momentum = mu momentum + grad, then weight = (1 - lr weight_decay) weight -
    lr scale X with X the orthogonalised grad + mu momentum (or momentum when
    nesterov is False).  weights: bf16 or fp32; momenta: fp32; grads: bf16 or
    fp32, e.g. an owner's views in GradBuffers.  scale: see update_scale."""
    zc = _zc()
    n = len(weights)
    table = _muon_table(weights, momenta, grads, scale)
    if n == 0:
        return
    L = zc.lib()
    need = L.dpred_muon_workspace_bytes(table, n) if workspace is None else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_muon_step(table, n, zc._dtype_code(weights[0]), zc._dtype_code(grads[0]), float(lr),
                                float(momentum), int(nesterov), float(weight_decay), int(steps), _coeffs(coeffs),
                                float(eps), wsp, wsb, zc._stream(stream)))


class Muon:
    """The optimizer state of one owner's matrices: fp32 momenta and the
    workspace, allocated once.  ``step(grads, lr)`` updates the weights in
    place from the reduced gradients."""

    def __init__(self, weights, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                 scale="spectral", steps: int = 5, eps: float = 1e-7, coeffs=None):
        import torch
        self.weights = list(weights)
        self.momenta = [torch.zeros(tuple(w.shape), dtype=torch.float32, device=w.device) for w in self.weights]
        self.momentum, self.nesterov, self.weight_decay = momentum, nesterov, weight_decay
        self.scale, self.steps, self.eps, self.coeffs = scale, steps, eps, coeffs
        table = _muon_table(self.weights, self.momenta, self.momenta, scale)
        need = _zc().lib().dpred_muon_workspace_bytes(table, len(self.weights))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    def step(self, grads, lr: float, stream=None) -> None:
        """Steps of one object run one after another (they share its workspace):
        use one stream, or order the streams."""
        muon_step(self.weights, self.momenta, grads, lr, self.momentum, self.nesterov, self.weight_decay, self.scale,
                  self.steps, self.eps, self.coeffs, self.workspace, stream)
