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


torch = _zc = _BF = _OK = None  # bound by the first call (the package imports without torch)


def _bind() -> None:
    global torch, _zc, _BF, _OK
    import torch as t

    import zero_collectives_gb300 as zc
    torch, _zc = t, zc
    _BF, _OK = (t.bfloat16,), (t.bfloat16, t.float32)


def _device() -> int:
    if torch is None:
        _bind()
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _matrix(t, name: str, dtypes, device: int, rows=None, cols=None):
    """(data pointer, row stride, rows, columns) of a 2-D tensor on the current
    device with unit column stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or t.get_device() != device:
        raise ValueError(f"{name} must be a 2-D tensor on the current CUDA device")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must have shape ({'*' if rows is None else rows}, {'*' if cols is None else cols}), "
                         f"got {tuple(shape)}")
    rs, cs = t.stride()
    if cs != 1 and c > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (rs if r > 1 else c), r, c


def _vector(t, name: str, dtypes, device: int, n: int) -> int:
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or t.get_device() != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements on the current CUDA device")
    return t.data_ptr()


def _code(t) -> int:
    return 0 if t.dtype is _BF[0] else 1


def _empty(shape, dtype, stream):
    """Device memory that belongs to the stream of the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(need: int, given, stream):
    if given is not None:
        if given.get_device() != _device() or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if not need:
        return None, 0, 0
    ws = _empty(need, torch.uint8, stream)
    return ws, ws.data_ptr(), need


def _pack_space(a, ar, ac, lda, b, br, bc, ldb, given, stream):
    """Workspace of a product: only operands without 16-byte aligned rows need
    one (the sizes of dpred_linear_workspace_bytes)."""
    if given is not None:
        return _workspace(0, given, stream)
    need = 0
    if a % 16 or (ar > 1 and lda % 8):
        need = (ar * (ac + 7 & -8) * 2 + 255) & -256
    if b % 16 or (br > 1 and ldb % 8):
        need += (br * (bc + 7 & -8) * 2 + 255) & -256
    return _workspace(need, None, stream) if need else (None, 0, 0)


_fn: dict = {}


def _call(name: str, *args) -> None:
    """One entry point with integer arguments (0 = NULL): through the CPython
    module where it was built, else through ctypes."""
    fc = _zc._FC if _zc._FC is not None else _zc._fast_call_module()
    L = _zc.lib()
    if fc is not None:
        fn = _fn.get(name)
        if fn is None:
            fn = _fn[name] = (getattr(fc, name), ctypes.cast(getattr(L, "dpred_" + name), ctypes.c_void_p).value)
        rc = fn[0](fn[1], *args)
    else:
        rc = getattr(L, "dpred_" + name)(*args)
    if rc:
        _zc._check(rc)


def _act(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"unknown activation {act!r}: none, relu, gelu or silu")
    return _ACTS[act]


def linear(x, w, bias=None, act="none", residual=None, preact=None, out=None, out_dtype=None, workspace=None,
           stream=None):
    """y = act(x w^T + bias) + residual.  x: bf16 [m, k]; w: bf16 [n, k]; bias:
    bf16 or fp32 [n]; residual: bf16 [m, n]; preact: bf16 [m, n], receives
    x w^T + bias (what linear_dgrad of the next layer down needs).  out: bf16
    or fp32 [m, n] (allocated on the call's stream when None).  Rows may be
    strided; m may be 1 (a single token).  A NaN before the activation stays
    one after it, relu included."""
    dev = _device()
    xp, ldx, m, k = _matrix(x, "x", _BF, dev)
    wp, ldw, n, _ = _matrix(w, "w", _BF, dev, None, k)
    a = _act(act)
    if out is None:
        out = _empty((m, n), out_dtype or _BF[0], stream)
    yp, ldy, _, _ = _matrix(out, "out", _OK, dev, m, n)
    rp = ldr = pp = ldp = bp = bdt = 0
    if residual is not None:
        rp, ldr, _, _ = _matrix(residual, "residual", _BF, dev, m, n)
    if preact is not None:
        pp, ldp, _, _ = _matrix(preact, "preact", _BF, dev, m, n)
    if bias is not None:
        bp, bdt = _vector(bias, "bias", _OK, dev, n), _code(bias)
    ws, wsp, wsb = _pack_space(xp, m, k, ldx, wp, n, k, ldw, workspace, stream)
    _call("linear", m, n, k, xp, ldx, wp, ldw, bdt, bp, a, rp, ldr, pp, ldp, _code(out), yp, ldy, wsp, wsb,
          _zc._stream(stream))
    return out


def linear_dgrad(dy, w, preact=None, act="none", residual=None, out=None, out_dtype=None, workspace=None,
                 stream=None):
    """dx = (dy w + residual) * act'(preact).  dy: bf16 [m, n]; w: bf16 [n, k];
    preact: the stored pre-activation of the layer below, bf16 [m, k] (needed
    unless act is "none"); residual: bf16 [m, k], the gradient that joins from
    a residual branch.  out: bf16 or fp32 [m, k]."""
    dev = _device()
    dp, ldd, m, n = _matrix(dy, "dy", _BF, dev)
    wp, ldw, _, k = _matrix(w, "w", _BF, dev, n, None)
    a = _act(act)
    if a != ACT_NONE and preact is None:
        raise ValueError("an activation's gradient needs preact")
    if out is None:
        out = _empty((m, k), out_dtype or _BF[0], stream)
    op, ldo, _, _ = _matrix(out, "out", _OK, dev, m, k)
    zp = ldz = rp = ldr = 0
    if a != ACT_NONE:
        zp, ldz, _, _ = _matrix(preact, "preact", _BF, dev, m, k)
    if residual is not None:
        rp, ldr, _, _ = _matrix(residual, "residual", _BF, dev, m, k)
    ws, wsp, wsb = _pack_space(dp, m, n, ldd, wp, n, k, ldw, workspace, stream)
    _call("linear_dgrad", m, n, k, dp, ldd, wp, ldw, a, zp, ldz, rp, ldr, _code(out), op, ldo, wsp, wsb,
          _zc._stream(stream))
    return out


def linear_wgrad(dy, x, out, bias_grad=None, accumulate: bool = False, workspace=None, stream=None):
    """out = dy^T x and bias_grad = column sums of dy, or both added to what
    the outputs hold (accumulate=True).  dy: bf16 [m, n]; x: bf16 [m, k]; out:
    [n, k] bf16 (a view of the gradient row that a flush reads) or fp32 (a view
    of the accumulator of accumulate_microbatch); bias_grad: fp32 [n]."""
    dev = _device()
    dp, ldd, m, n = _matrix(dy, "dy", _BF, dev)
    xp, ldx, _, k = _matrix(x, "x", _BF, dev, m, None)
    op, ldo, _, _ = _matrix(out, "out", _OK, dev, n, k)
    bp = 0 if bias_grad is None else _vector(bias_grad, "bias_grad", _OK[1:], dev, n)
    ws, wsp, wsb = _pack_space(dp, m, n, ldd, xp, m, k, ldx, workspace, stream)
    _call("linear_wgrad", m, n, k, dp, ldd, xp, ldx, 1 if accumulate else 0, _code(out), op, ldo, bp, wsp, wsb,
          _zc._stream(stream))
    return out


def _coeffs(coeffs):
    if coeffs is None:
        return None
    c = [float(x) for x in coeffs]
    if len(c) != 3:
        raise ValueError("coeffs must be (a, b, c)")
    return (ctypes.c_float * 3)(*c)


def newton_schulz(g, out=None, steps: int = 5, eps: float = 1e-7, coeffs=None, workspace=None, stream=None):
    """The orthogonalised matrix of g ([m, n], or [batch, m, n] of one shape;
    bf16 or fp32): `steps` steps of X = a X + (b A + c A^2) X, A = X X^T, from
    g / (|g|_F + eps).  out: bf16 (the default) or fp32, same shape; it carries
    16-bit accuracy either way (see dpred_newton_schulz)."""
    dev = _device()
    zc = _zc
    if g.dim() not in (2, 3):
        raise ValueError("g must be [m, n] or [batch, m, n]")
    if out is None:
        out = _empty(tuple(g.shape), _BF[0], stream)
    if tuple(out.shape) != tuple(g.shape):
        raise ValueError("out must have the shape of g")
    batch = g.shape[0] if g.dim() == 3 else 1
    if batch == 0:
        return out
    gp, ldg, m, n = _matrix(g[0] if g.dim() == 3 else g, "g", _OK, dev)
    op, ldo, _, _ = _matrix(out[0] if g.dim() == 3 else out, "out", _OK, dev)
    gb, ob = (g.stride(0), out.stride(0)) if g.dim() == 3 else (0, 0)
    L = zc.lib()
    need = L.dpred_newton_schulz_workspace_bytes(batch, m, n) if workspace is None else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_newton_schulz(batch, m, n, _code(g), gp, ldg, gb, _code(out), op, ldo, ob, int(steps),
                                    _coeffs(coeffs), float(eps), wsp or None, wsb, zc._stream(stream)))
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
    dev = _device()
    if not (len(weights) == len(momenta) == len(grads)):
        raise ValueError("weights, momenta and grads must have one entry per matrix")
    table = (_MuonMatrix * max(len(weights), 1))()
    for i, (w, m, g) in enumerate(zip(weights, momenta, grads)):
        if w.dtype != weights[0].dtype or g.dtype != grads[0].dtype:
            raise TypeError("all weights must have one dtype, and all grads one")
        t = table[i]
        t.weight, t.ldw, r, c = _matrix(w, "weight", _OK, dev)
        t.momentum, t.ldm, _, _ = _matrix(m, "momentum", _OK[1:], dev, r, c)
        t.grad, t.ldg, _, _ = _matrix(g, "grad", _OK, dev, r, c)
        t.rows, t.cols, t.scale = r, c, update_scale(r, c, scale)
    return table


def muon_step(weights, momenta, grads, lr: float, momentum: float = 0.95, nesterov: bool = True,
              weight_decay: float = 0.0, scale="spectral", steps: int = 5, eps: float = 1e-7, coeffs=None,
              workspace=None, stream=None) -> None:
    """One orthogonalised-momentum step of a list of matrices, in place:
    momentum = mu momentum + grad, then weight = (1 - lr weight_decay) weight -
    lr scale X with X the orthogonalised grad + mu momentum (or momentum when
    nesterov is False).  weights: bf16 or fp32; momenta: fp32; grads: bf16 or
    fp32, e.g. an owner's views in GradBuffers.  scale: see update_scale."""
    n = len(weights)
    table = _muon_table(weights, momenta, grads, scale)
    if n == 0:
        return
    zc, L = _zc, _zc.lib()
    need = L.dpred_muon_workspace_bytes(table, n) if workspace is None else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    zc._check(L.dpred_muon_step(table, n, _code(weights[0]), _code(grads[0]), float(lr),
                                float(momentum), int(nesterov), float(weight_decay), int(steps), _coeffs(coeffs),
                                float(eps), wsp or None, wsb, zc._stream(stream)))


class Muon:
    """The optimizer state of one owner's matrices: fp32 momenta and the
    workspace, allocated once.  ``step(grads, lr)`` updates the weights in
    place from the reduced gradients."""

    def __init__(self, weights, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                 scale="spectral", steps: int = 5, eps: float = 1e-7, coeffs=None):
        _device()
        self.weights = list(weights)
        self.momenta = [torch.zeros(tuple(w.shape), dtype=torch.float32, device=w.device) for w in self.weights]
        self.momentum, self.nesterov, self.weight_decay = momentum, nesterov, weight_decay
        self.scale, self.steps, self.eps, self.coeffs = scale, steps, eps, coeffs
        table = _muon_table(self.weights, self.momenta, self.momenta, scale)
        need = _zc.lib().dpred_muon_workspace_bytes(table, len(self.weights))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    def step(self, grads, lr: float, stream=None) -> None:
        """Steps of one object run one after another (they share its workspace):
        use one stream, or order the streams."""
        muon_step(self.weights, self.momenta, grads, lr, self.momentum, self.nesterov, self.weight_decay, self.scale,
                  self.steps, self.eps, self.coeffs, self.workspace, stream)
