"""Operators on the block of rows that a rank owns between a reduce-scatter and an all-gather
(C ABI in include/dtt_ops.h): the residual's addition with a root-mean-square norm, that norm's
backward pass, and the orthogonalisation of a momentum update.  Argument checks, marshalling and
the workspaces only; tensors are torch CUDA tensors whose rows are contiguous (any row pitch).
An object lives as long as the graphs that hold its calls."""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence, Tuple, Union

import device_triggered_transfers_gb300 as D

_CODES = {"bf16": D.BF16, "f32": D.F32, "e4m3": D.E4M3}
_SIZES = {"bf16": 2, "f32": 4, "e4m3": 1}


def _torch_types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _code(who: str, name: str, dtype: str) -> int:
    if dtype not in _CODES:
        raise D.DttError(D.EINVAL, f"{who}: {name} is one of {sorted(_CODES)}, not {dtype!r}")
    return _CODES[dtype]


def _torch_stream(stream, device):
    """torch's object for a `stream` argument (None: the default stream; an address; or a torch stream)."""
    import torch
    if stream is None:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream


class _Workspace:
    """A device buffer from torch's allocator, handed to calls on any stream: the allocating
    stream is done with it before its first use, and it is not reused while a call may run."""

    _UNUSED = object()               # None is the default stream

    def __init__(self, nbytes: int, device):
        import torch
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        torch.cuda.current_stream(self.buffer.device).synchronize()
        self.address, self.nbytes = self.buffer.data_ptr(), nbytes
        self._last = self._UNUSED

    def use(self, stream) -> None:
        """A call on `stream` is about to be launched: the allocator must not give the buffer away before
        it has finished, whatever stream the buffer was allocated on."""
        if stream is self._last:
            return
        self.buffer.record_stream(_torch_stream(stream, self.buffer.device))
        self._last = stream

    def wait(self) -> None:
        """Until the last call's stream has run out of work."""
        if self._last is not self._UNUSED:
            _torch_stream(self._last, self.buffer.device).synchronize()

    @classmethod
    def on(cls, stream, nbytes: int, device) -> "_Workspace":
        """One whose first call is on `stream`: allocated in that stream's order, so that nothing waits and the
        stream may be capturing (the graph's own pool then has the buffer)."""
        import torch
        w = cls.__new__(cls)
        with torch.cuda.stream(_torch_stream(stream, device)):
            w.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        w.address, w.nbytes, w._last = w.buffer.data_ptr(), nbytes, stream
        return w


class RMSNorm:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, row by row, and its gradients
    (dtt_rmsnorm_forward / dtt_rmsnorm_backward: see there for the definitions).

    x, residual, weight, y: element types, "bf16" or "f32" (y also "e4m3", with `group` columns per
    scale: 0 for one scale per row, 32, 64 or 128).  Keeps the backward pass's workspace (allocated by
    the first call with a dweight, in the order of that call's stream), so one object serves one stream at a time (or
    the caller orders the streams)."""

    def __init__(self, cols: int, x: str = "bf16", residual: str = "bf16", weight: str = "bf16",
                 y: str = "bf16", group: int = 0, eps: float = 1e-6):
        who = "RMSNorm"
        self.desc = D.dtt_rmsnorm_desc(_code(who, "x", x), _code(who, "residual", residual),
                                       _code(who, "weight", weight), _code(who, "y", y), group, eps, cols)
        need = C.c_uint64()
        D._check(D.lib().dtt_rmsnorm_workspace(C.byref(self.desc), C.byref(need)))
        self.cols, self.group, self.workspace_bytes = cols, group, need.value
        types = _torch_types()
        self._x, self._res, self._w, self._y = types[x], types[residual], types[weight], types[y]
        self._f32 = types["f32"]
        self._xe, self._rese, self._ye = (_SIZES[k] for k in (x, residual, y))
        self.scale_cols = -(-cols // group) if group else 1
        self._workspace = None
        self._ref = C.byref(self.desc)
        self._forward, self._backward = D.lib().dtt_rmsnorm_forward, D.lib().dtt_rmsnorm_backward

    def _rows(self, name: str, t, shape, dtype, size: int) -> Tuple[int, int]:
        """(address, pitch in bytes) of a [rows, cols] argument of `size`-byte elements; (0, 0) for None."""
        if t is None:
            return 0, 0
        if t.dtype != dtype or t.shape != shape:
            raise D.DttError(D.EINVAL, f"RMSNorm: {name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
        row, col = t.stride()
        if not t.is_cuda or (col != 1 and self.cols > 1):
            raise D.DttError(D.EINVAL, f"RMSNorm: {name} must be on the GPU with contiguous rows")
        return t.data_ptr(), row * size

    def _flat(self, name: str, t, n: int, dtype) -> int:
        """Address of a contiguous argument of n elements; 0 for None."""
        if t is None:
            return 0
        if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
            raise D.DttError(D.EINVAL, f"RMSNorm: {name} must be {n} contiguous {dtype} on the GPU")
        return t.data_ptr()

    def forward(self, x, weight, y, residual=None, residual_out=None, scales=None, rstd=None, stream=None) -> None:
        """y, and where given residual_out (= h; may be residual itself), scales ([rows, scale_cols]
        f32, with an e4m3 y) and rstd ([rows] f32, which the backward pass needs)."""
        rows = x.shape[0]
        shape = (rows, self.cols)
        xp, xs = self._rows("x", x, shape, self._x, self._xe)
        rp, rs = self._rows("residual", residual, shape, self._res, self._rese)
        op, os_ = self._rows("residual_out", residual_out, shape, self._res, self._rese)
        yp, ys = self._rows("y", y, shape, self._y, self._ye)
        rc = self._forward(self._ref, rows, xp, xs, rp, rs, self._flat("weight", weight, self.cols, self._w),
                           op, os_, yp, ys, self._flat("scales", scales, rows * self.scale_cols, self._f32),
                           self._flat("rstd", rstd, rows, self._f32), D._stream(stream))
        if rc:
            D._check(rc)

    def backward(self, dy, h, weight, rstd, dx, dweight=None, dres=None, stream=None) -> None:
        """dx ([rows, cols] in the residual's type: the gradient of x and of residual; may be dres
        itself) and, where given, dweight ([cols] f32), from the forward's h and rstd and the
        gradients dy of y and dres of residual_out (None: zero)."""
        rows = dy.shape[0]
        shape = (rows, self.cols)
        gp, gs = self._rows("dy", dy, shape, self._x, self._xe)
        hp, hs = self._rows("h", h, shape, self._res, self._rese)
        sp, ss = self._rows("dres", dres, shape, self._res, self._rese)
        xp, xs = self._rows("dx", dx, shape, self._res, self._rese)
        ws, need = 0, 0
        if dweight is not None:
            if self._workspace is None or self._workspace.buffer.device != dy.device:
                self._workspace = _Workspace.on(stream, self.workspace_bytes, dy.device)
            self._workspace.use(stream)
            ws, need = self._workspace.address, self.workspace_bytes
        rc = self._backward(self._ref, rows, gp, gs, hp, hs, self._flat("weight", weight, self.cols, self._w),
                            self._flat("rstd", rstd, rows, self._f32), sp, ss, xp, xs,
                            self._flat("dweight", dweight, self.cols, self._f32), ws, need, D._stream(stream))
        if rc:
            D._check(rc)


class Orthogonalizer:
    """The Newton-Schulz orthogonalisation of a batch of rows x cols updates (owner of a dtt_ortho*
    and its workspace; dtt_ops.h has the definition).

    coeffs: one (a, b, c) for every step, or a list of `steps` of them.  mu: the momentum's factor
    (None: no momentum).  One object serves one stream at a time (or the caller orders the
    streams)."""

    def __init__(self, rows: int, cols: int, batch: int = 1, dtype: str = "bf16", steps: int = 5,
                 coeffs: Union[Sequence[float], Sequence[Sequence[float]]] = (3.4445, -4.7750, 2.0315),
                 eps: float = 1e-7, scale: float = 1.0, mu: Optional[float] = None, nesterov: bool = False,
                 device=None):
        import torch
        self._h = None
        d = D.dtt_ortho_desc()
        d.x_dtype = _code("Orthogonalizer", "dtype", dtype)
        d.batch, d.rows, d.cols, d.steps = batch, rows, cols, steps
        d.momentum, d.nesterov, d.mu = int(mu is not None), int(bool(nesterov) and mu is not None), mu or 0.0
        d.eps, d.scale = eps, scale
        per_step = [tuple(coeffs)] * steps if len(coeffs) == 3 and not hasattr(coeffs[0], "__len__") else list(coeffs)
        if len(per_step) != steps or any(len(c) != 3 for c in per_step):
            raise D.DttError(D.EINVAL, "Orthogonalizer: coeffs is one (a, b, c) or one per step")
        for k, c in enumerate(per_step[:D.ORTHO_MAX_STEPS]):
            d.coeffs[k][:] = c
        self.desc, self.batch, self.rows, self.cols = d, batch, rows, cols
        types = _torch_types()
        self._dtype, self._f32, self._bf16 = types[dtype], types["f32"], types["bf16"]
        need = C.c_uint64()
        D._check(D.lib().dtt_ortho_workspace(C.byref(d), C.byref(need)))
        self.workspace_bytes = need.value
        # the error word follows the workspace proper
        self._workspace = _Workspace(need.value + 4, device or "cuda")
        self._err = self._workspace.buffer[need.value:].view(torch.int32)
        self._err.zero_()
        torch.cuda.current_stream(self._err.device).synchronize()
        self._err_ptr = self._err.data_ptr()
        out = C.c_void_p()
        D._check(D.lib().dtt_ortho_create(C.byref(d), self._workspace.address, need.value, C.byref(out)))
        self._h = out
        self._run = D.lib().dtt_ortho_run

    def _matrices(self, name: str, t, dtype) -> Tuple[int, int, int]:
        """(address, pitch, stride in bytes) of a [batch, rows, cols] (batch 1: or [rows, cols]) argument."""
        if t is None:
            return 0, 0, 0
        if t.dim() == 2 and self.batch == 1:
            t = t[None]
        if t.dtype != dtype or tuple(t.shape) != (self.batch, self.rows, self.cols):
            raise D.DttError(D.EINVAL, f"Orthogonalizer: {name} must be {dtype} "
                                       f"[{self.batch}, {self.rows}, {self.cols}], not {t.dtype} {tuple(t.shape)}")
        stride, pitch, col = t.stride()
        if not t.is_cuda or (col != 1 and self.cols > 1):
            raise D.DttError(D.EINVAL, f"Orthogonalizer: {name} must be on the GPU with contiguous rows")
        e = t.element_size()
        return t.data_ptr(), pitch * e, stride * e

    def run(self, x, out, momentum=None, stream=None) -> None:
        """out (bf16) from x and, where mu was given, momentum (f32, updated in place)."""
        xp, xs, xb = self._matrices("x", x, self._dtype)
        mp, ms, mb = self._matrices("momentum", momentum, self._f32)
        op, os_, ob = self._matrices("out", out, self._bf16)
        self._workspace.use(stream)
        rc = self._run(self._h, xp, xs, xb, mp, ms, mb, op, os_, ob, self._err_ptr, D._stream(stream))
        if rc:
            D._check(rc)

    @property
    def errors(self) -> int:
        """Internal waits that gave up so far (0).  Waits for the last call's stream, and so for all of this
        object's calls, but not for replays of a graph that holds some."""
        self._workspace.wait()
        return int(self._err.item())

    def close(self) -> None:
        if self._h is not None and self._h.value:
            D.lib().dtt_ortho_destroy(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
        return False

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
