"""The rest of a training step around the products and the reduction (argument
marshalling only, as in the package's other calls): the token embedding and its
gradient (``dpred_embedding*``), the norms, gate and residual sum between two
blocks and their gradients (``dpred_block_norm*``), and the global gradient norm
with clipping (``dpred_grad_norm``, ``dpred_clip_grads``).  All device work runs
in libdpred's kernels; there is no fallback."""
from __future__ import annotations

import ctypes

from . import train as _t
from .train import _call, _code, _device, _empty, _matrix, _vector, _workspace


class _GradTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("counted", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of these entry points on the loaded library."""
    i32, i64, vp, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    L.dpred_embedding.argtypes = [i64, i64, i64, i32, vp, i32, vp, i64, f32, i32, vp, i64, vp]
    L.dpred_embedding_grad_workspace_bytes.restype = sz
    L.dpred_embedding_grad_workspace_bytes.argtypes = [i64, i64, i64]
    L.dpred_embedding_grad.argtypes = [i64, i64, i64, i32, vp, i64, i32, vp, i64, f32, i32, i32, vp, i64, vp, sz, vp]
    L.dpred_block_norm.argtypes = [i64, i64, i32, vp, i64, vp, i64, i32, vp, i32, vp, i64, f32, i32, vp, f32, vp, i64, vp, i64, vp]
    L.dpred_block_norm_grad_workspace_bytes.restype = sz
    L.dpred_block_norm_grad_workspace_bytes.argtypes = [i64, i64, i64]
    L.dpred_block_norm_grad.argtypes = [i64, i64, i32, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i32, vp, i64, f32, i32, vp, f32, vp,
                                        i64, vp, i64, i32, vp, vp, vp, i32, vp, sz, vp]
    L.dpred_clip_workspace_bytes.restype = sz
    L.dpred_clip_workspace_bytes.argtypes = [i32]
    L.dpred_grad_norm.argtypes = [vp, i32, vp, vp, sz, vp]
    L.dpred_clip_grads.argtypes = [vp, i32, f32, f32, vp, vp, sz, vp]


def _like(t, stream):
    """Contiguous device memory of t's shape and type that belongs to the stream of the call."""
    if stream is None and t.is_contiguous():
        return _t.torch.empty_like(t)
    return _empty(tuple(t.shape), t.dtype, stream)


def _ids(ids, device: int):
    """(data pointer, bytes of an id, tokens) of a contiguous integer tensor."""
    if ids.dtype is not _t.torch.int64 and ids.dtype is not _t.torch.int32:
        raise TypeError(f"ids: unsupported dtype {ids.dtype}, int32 or int64")
    if ids.get_device() != device or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous tensor on the current CUDA device")
    return ids.data_ptr(), (8 if ids.dtype is _t.torch.int64 else 4), ids.numel()


def _rows_of(t, name: str, dtypes, device: int, rows: int, cols: int):
    """(data pointer, row stride) of [rows, cols], or of [..., cols] with the
    leading dimensions back to back."""
    if t.dim() != 2:
        lead = t.shape[:-1]
        n = 1
        for x in lead:
            n *= x
        if t.dim() == 0 or n != rows or t.shape[-1] != cols or not t.is_contiguous():
            raise ValueError(f"{name} must have {rows} rows of {cols}: two-dimensional, or contiguous")
        t = t.view(rows, cols)
    p, ld, _, _ = _matrix(t, name, dtypes, device, rows, cols)
    return p, ld


def embedding(ids, w, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """y[t] = scale w[ids[t]].  ids: contiguous int32 or int64 of any shape; w:
    bf16 or fp32 [v, d], rows may be strided.  out: [*ids.shape, d] (or, strided,
    [number of ids, d]) bf16 or fp32; allocated on the call's stream in out_dtype
    (w's without one) when None.  An id outside the table gives a row of zeros
    and is reported by device_status()."""
    dev = _device()
    ip, ib, t = _ids(ids, dev)
    wp, ldw, v, d = _matrix(w, "w", _t._OK, dev)
    if out is None:
        out = _empty((*ids.shape, d), out_dtype or w.dtype, stream)
        if out.dtype not in _t._OK:
            raise TypeError(f"out_dtype: unsupported dtype {out.dtype}")
        yp, ldy = out.data_ptr(), d
    else:
        yp, ldy = _rows_of(out, "out", _t._OK, dev, t, d)
    _call("embedding", t, v, d, ib, ip, _code(w), wp, ldw, float(scale), _code(out), yp, ldy, _t._zc._stream(stream))
    return out


def embedding_grad(ids, dy, out, scale: float = 1.0, padding=None, accumulate: bool = False, workspace=None, stream=None):
    """out[k] = scale * (sum of dy[t] over the t with ids[t] = k), for every row of
    out, or added to the rows that have a token (accumulate=True).  dy: bf16 or
    fp32 [*ids.shape, d] (or, strided, [number of ids, d]); out: [v, d] bf16 (a
    view of the gradient row that a flush reads) or fp32 (a view of the
    accumulator of accumulate_microbatch); padding: an id whose tokens give no
    gradient."""
    dev = _device()
    ip, ib, t = _ids(ids, dev)
    op, ldo, v, d = _matrix(out, "out", _t._OK, dev)
    dp, ldd = _rows_of(dy, "dy", _t._OK, dev, t, d)
    if padding is not None and not 0 <= padding < v:
        raise ValueError(f"padding {padding} is no row of out ({v} rows)")
    need = 0 if workspace is not None else _t._zc.lib().dpred_embedding_grad_workspace_bytes(t, v, d)
    ws, wsp, wsb = _workspace(need, workspace, stream)
    _call("embedding_grad", t, v, d, ib, ip, -1 if padding is None else int(padding), _code(dy), dp, ldd, float(scale),
          1 if accumulate else 0, _code(out), op, ldo, wsp, wsb, _t._zc._stream(stream))
    return out


def _gate(gate, name: str, dtypes, device: int, m: int, d: int):
    """(data pointer, gate rows) of [d] or a contiguous [rows, d] with rows dividing m."""
    if gate.dim() == 1:
        return _vector(gate, name, dtypes, device, d), 1
    p, ld, rows, _ = _matrix(gate, name, dtypes, device, None, d)
    if rows > 1 and ld != d:
        raise ValueError(f"{name} must be contiguous")
    if m and (rows < 1 or m % rows):
        raise ValueError(f"{name}: {rows} rows do not divide the {m} rows of the stream")
    return p, rows


def block_norm(x, y=None, post=None, gate=None, residual_scale: float = 1.0, pre=None, eps: float = 1e-6, out=None, out_norm=None,
               stream=None):
    """What stands between two blocks, with N(a, w) = w a / sqrt(mean(a^2) + eps):
    r = residual_scale x + gate N(y, post) and h = N(r, pre); returns (r, h).
    x: bf16 or fp32 [m, d], the residual stream; y: bf16 [m, d], the block's
    output (None: r is x, and only h is formed); post, pre: [d], bf16 or fp32 (None: no
    such norm; h is then None); gate: [d], or contiguous [k, d] where m / k
    consecutive rows share a gate row, bf16 or fp32.  out, out_norm: r (type of x) and
    h (bf16), allocated on the call's stream when None; out may be x, out_norm y."""
    dev = _device()
    xp, ldx, m, d = _matrix(x, "x", _t._OK, dev)
    yp = ldy = pp = pdt = gp = gdt = rp = ldr = wp = wdt = hp = ldh = gr = 0
    if (out is not None and y is None) or (out_norm is not None and pre is None):
        raise ValueError("out needs y (r is x without it), out_norm needs pre")
    r, h = x, None
    if y is not None:
        yp, ldy, _, _ = _matrix(y, "y", _t._BF, dev, m, d)
        if out is None:
            r = _like(x, stream)
            rp, ldr = r.data_ptr(), d
        else:
            r = out
            rp, ldr, _, _ = _matrix(r, "out", (x.dtype,), dev, m, d)
    if post is not None:
        pp, pdt = _vector(post, "post", _t._OK, dev, d), _code(post)
    if gate is not None:
        (gp, gr), gdt = _gate(gate, "gate", _t._OK, dev, m, d), _code(gate)
    if pre is not None:
        wp, wdt = _vector(pre, "pre", _t._OK, dev, d), _code(pre)
        if out_norm is None:
            h = _like(y, stream) if y is not None else _empty((m, d), _t._BF[0], stream)
            hp, ldh = h.data_ptr(), d
        else:
            h = out_norm
            hp, ldh, _, _ = _matrix(h, "out_norm", _t._BF, dev, m, d)
    if m and d:
        _call("block_norm", m, d, _code(x), xp, ldx, yp, ldy, pdt, pp, gdt, gp, gr, float(residual_scale), wdt, wp, float(eps), rp, ldr,
              hp, ldh, _t._zc._stream(stream))
    return r, h


def block_norm_grad(r, dr=None, dh=None, y=None, post=None, gate=None, residual_scale: float = 1.0, pre=None, eps: float = 1e-6,
                    dx=None, dy=None, post_grad=None, gate_grad=None, pre_grad=None, accumulate: bool = False, workspace=None,
                    stream=None):
    """The gradient of block_norm at its stored r: from dr (the residual stream's,
    type of r; None: no such gradient) and dh (of h, bf16) to dx (type of r) and dy (bf16; None
    without y); returns (dx, dy).  r, y, post, gate, pre: as block_norm had and gave
    them.  post_grad, gate_grad, pre_grad: written where given (one type, bf16 or
    fp32, shaped as the weights), or added to (accumulate=True).  dx may be dr, dy may
    be dh or y."""
    dev = _device()
    rp, ldr, m, d = _matrix(r, "r", _t._OK, dev)
    drp = lddr = dhp = lddh = yp = ldy = pp = pdt = gp = gdt = gr = wp = wdt = dyp = lddy = pg = gg = wg = gt = 0
    if (dh is None) != (pre is None):
        raise ValueError("dh and pre belong together")
    if dr is not None:
        drp, lddr, _, _ = _matrix(dr, "dr", (r.dtype,), dev, m, d)
    if dx is None:
        dx = _like(r, stream)
        dxp, lddx = dx.data_ptr(), d
    else:
        dxp, lddx, _, _ = _matrix(dx, "dx", (r.dtype,), dev, m, d)
    if y is not None:
        yp, ldy, _, _ = _matrix(y, "y", _t._BF, dev, m, d)
        if dy is None:
            dy = _like(y, stream)
            dyp, lddy = dy.data_ptr(), d
        else:
            dyp, lddy, _, _ = _matrix(dy, "dy", _t._BF, dev, m, d)
    elif dy is not None:
        raise ValueError("dy needs y")
    kinds = {g.dtype for g in (post_grad, gate_grad, pre_grad) if g is not None}
    if len(kinds) > 1:
        raise TypeError("post_grad, gate_grad and pre_grad must have one dtype")
    gt = _code(next(g for g in (post_grad, gate_grad, pre_grad) if g is not None)) if kinds else 0
    if post is not None:
        pp, pdt = _vector(post, "post", _t._OK, dev, d), _code(post)
    if post_grad is not None:
        pg = _vector(post_grad, "post_grad", _t._OK, dev, d)
    if gate is not None:
        (gp, gr), gdt = _gate(gate, "gate", _t._OK, dev, m, d), _code(gate)
        if gate_grad is not None:
            if gate_grad.shape != gate.shape:
                raise ValueError("gate_grad must have the shape of gate")
            gg, _ = _gate(gate_grad, "gate_grad", _t._OK, dev, m, d)
    elif gate_grad is not None:
        raise ValueError("gate_grad needs gate")
    if pre is not None:
        wp, wdt = _vector(pre, "pre", _t._OK, dev, d), _code(pre)
        dhp, lddh, _, _ = _matrix(dh, "dh", _t._BF, dev, m, d)
    if pre_grad is not None:
        wg = _vector(pre_grad, "pre_grad", _t._OK, dev, d)
    need = _t._zc.lib().dpred_block_norm_grad_workspace_bytes(m, d, gr) if kinds and workspace is None else 0
    ws, wsp, wsb = _workspace(need, workspace, stream)
    _call("block_norm_grad", m, d, _code(r), rp, ldr, drp, lddr, dhp, lddh, yp, ldy, pdt, pp, gdt, gp, gr, float(residual_scale), wdt, wp,
          float(eps), dxp, lddx, dyp, lddy, gt, pg, gg, wg, 1 if accumulate else 0, wsp, wsb, _t._zc._stream(stream))
    return dx, dy


def _grad_table(grads, copies):
    """The gradients as the library reads them: [.., cols] with unit column
    stride, their leading dimensions back to back where there are several."""
    dev = _device()
    n = len(grads) + len(copies)
    table = (_GradTensor * max(n, 1))()
    for i, g in enumerate((*grads, *copies)):
        if g.dtype not in _t._OK:
            raise TypeError(f"a gradient of unsupported dtype {g.dtype}")
        if g.get_device() != dev:
            raise ValueError("gradients must be on the current CUDA device")
        t = table[i]
        t.data, t.dtype, t.counted = g.data_ptr(), _code(g), int(i < len(grads))
        if g.is_contiguous():
            t.rows, t.cols, t.ld = 1, g.numel(), g.numel()
        else:
            m = g if g.dim() == 2 else g.unsqueeze(1) if g.dim() == 1 else None
            if m is None:
                raise ValueError("a gradient must be contiguous, a vector, or a matrix")
            _, t.ld, t.rows, t.cols = _matrix(m, "a gradient", _t._OK, dev)
    return table, n


class GradClip:
    """The gradients of a step, to be clipped together again and again: the table
    of their addresses and the workspace, made once.  ``norm()`` is their global
    2-norm, ``clip(max_norm)`` scales them in place by
    min(1, max_norm / (norm + eps)).  grads: bf16 or fp32 tensors on the current
    device, contiguous or with strided rows; copies: further copies of some of
    them (such as those of a parameter that several ranks hold), which are scaled
    and not counted.  Calls of one object scale the same gradients and share its
    workspace: one at a time, on one stream or on streams that are ordered.  The
    workspace belongs to the stream that is current here; a call on another one, or
    one that is captured, has memory of its own, so the object (the gradients are
    another matter) may go as soon as a call has returned."""

    def __init__(self, grads, copies=(), eps: float = 1e-6):
        self.grads, self.copies, self.eps = list(grads), list(copies), float(eps)
        self._device = _device()
        self._table, self._n = _grad_table(self.grads, self.copies)
        self.workspace = _t.torch.empty(_t._zc.lib().dpred_clip_workspace_bytes(self._n), dtype=_t.torch.uint8, device="cuda")
        self._args = ctypes.addressof(self._table), self._n
        self._own = self.workspace, self.workspace.data_ptr(), self.workspace.numel()
        self._stream = _t._zc._stream(None)

    def _space(self, stream):
        """A workspace that belongs to the stream of the call, or to the graph that
        captures it: the memory of another stream may still be in use there, and is
        given to others there while this call runs."""
        if _t._zc._stream(stream) == self._stream and not _t.torch._C._cuda_isCurrentStreamCapturing():
            return self._own
        return _workspace(self.workspace.numel(), None, stream)

    def norm(self, out=None, stream=None):
        """The norm: fp32 [1], on the device."""
        self._check()
        ws, *space = self._space(stream)
        return _norm(self._args, space, out, stream)

    def _check(self) -> None:
        if _device() != self._device:
            raise ValueError(f"the gradients are on CUDA device {self._device}, not the current one")

    def clip(self, max_norm: float, out=None, stream=None):
        """Scales the gradients; returns fp32 [2] on the device: the norm before
        and the factor."""
        self._check()
        ws, *space = self._space(stream)
        return _clip(self._args, space, max_norm, self.eps, out, stream)


def _result(out, n: int, stream):
    dev = _device()
    if out is None:
        out = _empty(n, _t._OK[1], stream)
        return out, out.data_ptr()
    return out, _vector(out, "out", _t._OK[1:], dev, n)


def _norm(args, space, out, stream):
    out, p = _result(out, 1, stream)
    _call("grad_norm", *args, p, *space, _t._zc._stream(stream))
    return out


def _clip(args, space, max_norm, eps, out, stream):
    out, p = _result(out, 2, stream)
    _call("clip_grads", *args, float(max_norm), eps, p, *space, _t._zc._stream(stream))
    return out


def _clip_space(n: int, workspace, stream):
    return _workspace(_t._zc.lib().dpred_clip_workspace_bytes(n) if workspace is None else 0, workspace, stream)


def grad_norm(grads, out=None, workspace=None, stream=None):
    """The 2-norm of all gradients together (see GradClip): fp32 [1] on the device."""
    table, n = _grad_table(list(grads), ())
    ws, *space = _clip_space(n, workspace, stream)
    return _norm((ctypes.addressof(table), n), space, out, stream)


def clip_grads(grads, max_norm: float, copies=(), eps: float = 1e-6, out=None, workspace=None, stream=None):
    """Scales the gradients in place by min(1, max_norm / (norm + eps)), norm their
    2-norm together; returns fp32 [2] on the device: norm and factor (see GradClip,
    which keeps the table of a step's gradients).  max_norm is finite: grad_norm is
    the norm alone."""
    table, n = _grad_table(list(grads), list(copies))
    ws, *space = _clip_space(n, workspace, stream)
    return _clip((ctypes.addressof(table), n), space, max_norm, float(eps), out, stream)
