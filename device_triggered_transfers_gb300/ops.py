"""Operators on what a rank owns between a reduce-scatter and an all-gather (C ABI in
include/dtt_ops.h): the residual's addition with a root-mean-square norm or a layer norm and their
backward passes, tokens' rows sorted by expert and back, the orthogonalisation of a momentum update,
and AdamW over the tensors of the rank's share.  Argument checks, marshalling and the workspaces only;
tensors are torch CUDA tensors whose rows are contiguous (any row pitch).
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


def _workspace_on(op, device, stream) -> int:
    """Address of `op`'s workspace on a GPU, for a call on `stream`.  Once allocated a GPU's stays as long as `op`, whatever
    other GPUs it is used on: graphs hold its address."""
    w = op._workspace                                  # the last call's
    if w is None or w.buffer.device != device:
        w = op._workspaces.get(device)
        if w is None:
            w = op._workspaces[device] = _Workspace.on(stream, op.workspace_bytes, device)
        op._workspace = w
    w.use(stream)
    return w.address


class RMSNorm:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, row by row, and its gradients
    (dtt_rmsnorm_forward / dtt_rmsnorm_backward: see there for the definitions).

    x, residual, weight, y: element types, "bf16" or "f32" (y also "e4m3", with `group` columns per
    scale: 0 for one scale per row, 32, 64 or 128).  Keeps the backward pass's workspace (allocated by
    the first call with a dweight, in the order of that call's stream), so one object serves one stream at a time (or
    the caller orders the streams)."""

    _who, _calls = "RMSNorm", "dtt_rmsnorm_"

    def __init__(self, cols: int, x: str = "bf16", residual: str = "bf16", weight: str = "bf16",
                 y: str = "bf16", group: int = 0, eps: float = 1e-6):
        who = self._who
        self.desc = D.dtt_rmsnorm_desc(_code(who, "x", x), _code(who, "residual", residual),
                                       _code(who, "weight", weight), _code(who, "y", y), group, eps, cols)
        need = C.c_uint64()
        workspace, self._forward, self._backward = (getattr(D.lib(), self._calls + k) for k in ("workspace", "forward", "backward"))
        D._check(workspace(C.byref(self.desc), C.byref(need)))
        self.cols, self.group, self.workspace_bytes = cols, group, need.value
        types = _torch_types()
        self._x, self._res, self._w, self._y = types[x], types[residual], types[weight], types[y]
        self._f32 = types["f32"]
        self._xe, self._rese, self._ye = (_SIZES[k] for k in (x, residual, y))
        self.scale_cols = -(-cols // group) if group else 1
        self._workspace, self._workspaces = None, {}
        self._ref = C.byref(self.desc)

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
            ws, need = _workspace_on(self, dy.device, stream), self.workspace_bytes
        rc = self._backward(self._ref, rows, gp, gs, hp, hs, self._flat("weight", weight, self.cols, self._w),
                            self._flat("rstd", rstd, rows, self._f32), sp, ss, xp, xs,
                            self._flat("dweight", dweight, self.cols, self._f32), ws, need, D._stream(stream))
        if rc:
            D._check(rc)


def _current_device() -> int:
    """torch.cuda.current_device, in whose place the first call puts it: an import takes 0.1 us of each call."""
    global _current_device
    import torch
    _current_device = torch.cuda.current_device
    return _current_device()


def _here(who: str, name: str, t) -> int:
    """The number of t's GPU, which is the current one: the calls launch there."""
    device = t.get_device()
    if device < 0 or device != _current_device():
        raise D.DttError(D.EINVAL, f"{who}: {name} must be on the current GPU")
    return device


class LayerNorm(RMSNorm):
    """h = x + residual; y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias, row by row, and its gradients
    (dtt_layernorm_forward / dtt_layernorm_backward: see there for the definitions).

    Arguments as RMSNorm's; the bias has the weight's type.  Keeps the backward pass's workspace in the same way
    (allocated by the first call with a dweight or a dbias)."""

    _who, _calls = "LayerNorm", "dtt_layernorm_"

    def __init__(self, cols: int, x: str = "bf16", residual: str = "bf16", weight: str = "bf16",
                 y: str = "bf16", group: int = 0, eps: float = 1e-5):
        super().__init__(cols, x, residual, weight, y, group, eps)

    def _rows(self, name: str, t, shape, dtype, size: int) -> Tuple[int, int]:
        if t is None:
            return 0, 0
        if t.dtype != dtype or t.shape != shape:
            raise D.DttError(D.EINVAL, f"LayerNorm: {name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
        row, col = t.stride()
        if t.get_device() != self._device or (col != 1 and self.cols > 1):
            raise D.DttError(D.EINVAL, f"LayerNorm: {name} must be on the current GPU with contiguous rows")
        return t.data_ptr(), row * size

    def _flat(self, name: str, t, n: int, dtype) -> int:
        if t is None:
            return 0
        if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != self._device:
            raise D.DttError(D.EINVAL, f"LayerNorm: {name} must be {n} contiguous {dtype} on the current GPU")
        return t.data_ptr()

    def forward(self, x, weight, bias, y, residual=None, residual_out=None, scales=None, mean=None, rstd=None,
                stream=None) -> None:
        """y, and where given residual_out (= h; may be residual itself), scales ([rows, scale_cols] f32, with an
        e4m3 y), mean and rstd ([rows] f32, which the backward pass needs).  weight, bias: or None."""
        rows = x.shape[0]
        shape = (rows, self.cols)
        self._device = _here(self._who, "x", x)
        xp, xs = self._rows("x", x, shape, self._x, self._xe)
        rp, rs = self._rows("residual", residual, shape, self._res, self._rese)
        op, os_ = self._rows("residual_out", residual_out, shape, self._res, self._rese)
        yp, ys = self._rows("y", y, shape, self._y, self._ye)
        rc = self._forward(self._ref, rows, xp, xs, rp, rs, self._flat("weight", weight, self.cols, self._w),
                           self._flat("bias", bias, self.cols, self._w), op, os_, yp, ys,
                           self._flat("scales", scales, rows * self.scale_cols, self._f32),
                           self._flat("mean", mean, rows, self._f32), self._flat("rstd", rstd, rows, self._f32),
                           D._stream(stream))
        if rc:
            D._check(rc)

    def backward(self, dy, h, weight, mean, rstd, dx, dweight=None, dbias=None, dres=None, stream=None) -> None:
        """dx ([rows, cols] in the residual's type: the gradient of x and of residual; may be dres itself)
        and, where given, dweight and dbias ([cols] f32), from the forward's h, mean and rstd and the
        gradients dy of y and dres of residual_out (None: zero)."""
        rows = dy.shape[0]
        shape = (rows, self.cols)
        self._device = _here(self._who, "dy", dy)
        gp, gs = self._rows("dy", dy, shape, self._x, self._xe)
        hp, hs = self._rows("h", h, shape, self._res, self._rese)
        sp, ss = self._rows("dres", dres, shape, self._res, self._rese)
        xp, xs = self._rows("dx", dx, shape, self._res, self._rese)
        flat = self._flat
        args = (flat("weight", weight, self.cols, self._w), flat("mean", mean, rows, self._f32),
                flat("rstd", rstd, rows, self._f32), sp, ss, xp, xs,
                flat("dweight", dweight, self.cols, self._f32), flat("dbias", dbias, self.cols, self._f32))
        ws, need = 0, 0
        if dweight is not None or dbias is not None:
            ws, need = _workspace_on(self, dy.device, stream), self.workspace_bytes
        rc = self._backward(self._ref, rows, gp, gs, hp, hs, *args, ws, need, D._stream(stream))
        if rc:
            D._check(rc)


class ExpertRows:
    """Tokens' rows sorted by the experts first .. first + experts - 1 that a rank holds, and back with weights,
    and their gradients (dtt_experts_*: see there for the definitions).

    top_k: choices of a token.  align: an expert's rows are filled up to a multiple of it, with zeros.  Keeps the
    sort's workspace (allocated by the first `route`, in the order of that call's stream), so that one object
    routes on one stream at a time (or the caller orders the streams); the other calls need none."""

    _who = "ExpertRows"

    def __init__(self, experts: int, top_k: int, first: int = 0, align: int = 1):
        for name, v, most in (("experts", experts, 1024), ("top_k", top_k, 32), ("first", first, 2 ** 31 - 1), ("align", align, 65536)):
            if not 0 <= v <= most:
                raise D.DttError(D.EINVAL, f"ExpertRows: {name} must be at most {most} and not negative, not {v}")
        self.desc = D.dtt_experts_desc(experts, first, top_k, align)
        need = C.c_uint64()
        D._check(D.lib().dtt_experts_workspace(C.byref(self.desc), C.byref(need)))
        self.experts, self.top_k, self.first, self.align = experts, top_k, first, align
        self.workspace_bytes = need.value
        self._workspace, self._workspaces = None, {}
        self._ref = C.byref(self.desc)
        import torch
        self._i32, self._i64, self._f32 = torch.int32, torch.int64, torch.float32
        self._row_types = {torch.bfloat16: D.BF16, torch.float32: D.F32}
        L = D.lib()
        self._route, self._dispatch, self._combine, self._combine_backward = (
            L.dtt_experts_route, L.dtt_experts_dispatch, L.dtt_experts_combine, L.dtt_experts_combine_backward)

    def most_rows(self, tokens: int) -> int:
        """Rows that are always enough for so many tokens."""
        return tokens * self.top_k + self.experts * (self.align - 1)

    def _flat(self, name: str, t, shape, dtype) -> int:
        """Address of a contiguous argument; 0 for None."""
        if t is None:
            return 0
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._device:
            raise D.DttError(D.EINVAL, f"ExpertRows: {name} must be contiguous {dtype} {list(shape)} on the current GPU, "
                                       f"not {t.dtype} {list(t.shape)}")
        return t.data_ptr()

    def _rows(self, name: str, t, rows, cols, dtypes=None) -> Tuple[int, int]:
        """(address, pitch in bytes) of an argument of rows (None: any number) x cols; (0, 0) for None."""
        if t is None:
            return 0, 0
        shape = t.shape
        if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
            raise D.DttError(D.EINVAL, f"ExpertRows: {name} must be [{'any' if rows is None else rows}, {cols}], not {list(shape)}")
        if dtypes is not None and t.dtype not in dtypes:
            raise D.DttError(D.EINVAL, f"ExpertRows: {name} must be one of {list(dtypes)}, not {t.dtype}")
        row, col = t.stride()
        if t.get_device() != self._device or (col != 1 and cols > 1):
            raise D.DttError(D.EINVAL, f"ExpertRows: {name} must be on the current GPU with contiguous rows")
        return t.data_ptr(), row * t.element_size()

    def _sorted(self, tokens: int, position, offsets, counts) -> Tuple[int, int, int]:
        return (self._flat("position", position, (tokens, self.top_k), self._i32),
                self._flat("offsets", offsets, (self.experts + 1,), self._i32),
                self._flat("counts", counts, (self.experts,), self._i32))

    def route(self, ids, position, offsets, counts, max_rows: Optional[int] = None, stream=None) -> None:
        """ids: [tokens, top_k] int32 or int64, any values (those that are not this rank's experts have no row).
        position ([tokens, top_k] int32): each pair's row, or -1; offsets ([experts + 1] int32): where each expert's
        rows begin; counts ([experts] int32): how many pairs it has.  max_rows: rows that there are room for
        (None: most_rows(tokens)); pairs beyond get -1."""
        self._device = _here(self._who, "ids", ids)
        tokens = ids.shape[0]
        ip = self._flat("ids", ids, (tokens, self.top_k), self._i64 if ids.dtype == self._i64 else self._i32)
        pp = self._flat("position", position, (tokens, self.top_k), self._i32)
        op, cp = self._flat("offsets", offsets, (self.experts + 1,), self._i32), self._flat("counts", counts, (self.experts,), self._i32)
        ws = _workspace_on(self, ids.device, stream)
        rows = self.most_rows(tokens) if max_rows is None else max_rows
        if not 0 <= rows < 2 ** 31:
            raise D.DttError(D.EINVAL, f"ExpertRows: max_rows must be 0 .. 2^31 - 1, not {rows}")
        rc = self._route(self._ref, tokens, ip, ids.element_size(), rows, pp, op, cp, ws, self.workspace_bytes,
                         D._stream(stream))
        if rc:
            D._check(rc)

    def dispatch(self, x, position, offsets, counts, rows, scales=None, row_scales=None, stream=None) -> None:
        """rows[position[t, j]] = x[t] (both of one type, any), and row_scales[position[t, j]] = scales[t] (f32, both or
        neither); zeros in the rows that fill an expert's up; rows behind the last expert's are left as they were."""
        self._device = _here(self._who, "x", x)
        shape = x.shape
        tokens, cols = shape[0], shape[-1]
        xp, xs = self._rows("x", x, tokens, cols)
        rp, rs = self._rows("rows", rows, None, cols, (x.dtype,))
        pp, op, cp = self._sorted(tokens, position, offsets, counts)
        sp = ss = tp = ts = n = 0
        if scales is not None or row_scales is not None:
            if scales is None or row_scales is None:
                raise D.DttError(D.EINVAL, "ExpertRows: scales and row_scales go together")
            n = scales.shape[-1]
            sp, ss = self._rows("scales", scales, tokens, n, (self._f32,))
            tp, ts = self._rows("row_scales", row_scales, rows.shape[0], n, (self._f32,))
        rc = self._dispatch(self._ref, tokens, pp, op, cp, xp, xs, cols * x.element_size(), rp, rs, rows.shape[0],
                            sp, ss, n, tp, ts, D._stream(stream))
        if rc:
            D._check(rc)

    def combine(self, rows, position, out, weights=None, stream=None) -> None:
        """out[t] = sum of weights[t, j] rows[position[t, j]] over the pairs with a row (rows, out: bf16 or f32; weights:
        [tokens, top_k] f32).  weights None: 1, the gradient of `dispatch`, whose rows' gradient `rows` is then."""
        self._device = _here(self._who, "out", out)
        tokens, cols = out.shape[0], out.shape[-1]
        op, os_ = self._rows("out", out, tokens, cols, self._row_types)
        rp, rs = self._rows("rows", rows, None, cols, self._row_types)
        pairs = (tokens, self.top_k)
        rc = self._combine(self._ref, tokens, cols, self._flat("position", position, pairs, self._i32), rp,
                           self._row_types[rows.dtype], rs, rows.shape[0], self._flat("weights", weights, pairs, self._f32),
                           op, self._row_types[out.dtype], os_, D._stream(stream))
        if rc:
            D._check(rc)

    def combine_backward(self, dout, rows, position, weights, offsets, counts, drows, dweights=None, stream=None) -> None:
        """drows[position[t, j]] = weights[t, j] dout[t], zeros in the rows that fill an expert's up (those behind the last
        expert's are left as they were), and where given dweights[t, j] = dout[t] . rows[position[t, j]] ([tokens, top_k]
        f32, 0 for a pair without a row).  rows may be None without dweights; drows has its type."""
        self._device = _here(self._who, "dout", dout)
        tokens, cols = dout.shape[0], dout.shape[-1]
        gp, gs = self._rows("dout", dout, tokens, cols, self._row_types)
        dp, ds = self._rows("drows", drows, None, cols, self._row_types)
        rp, rs = self._rows("rows", rows, drows.shape[0], cols, (drows.dtype,))
        pp, op, cp = self._sorted(tokens, position, offsets, counts)
        pairs = (tokens, self.top_k)
        rc = self._combine_backward(self._ref, tokens, cols, pp, op, cp, gp, self._row_types[dout.dtype], gs, rp,
                                    self._row_types[drows.dtype], rs, drows.shape[0],
                                    self._flat("weights", weights, pairs, self._f32), dp, ds,
                                    self._flat("dweights", dweights, pairs, self._f32), D._stream(stream))
        if rc:
            D._check(rc)


class AdamW:
    """AdamW over a list of tensors in one pass (owner of a dtt_adamw*; dtt_ops.h has the definition).

    params, grads: lists of contiguous tensors, each list of one type, bf16 or f32.  m, v: the states, all f32, or all
    torch.float8_e4m3fn with m_scales and v_scales (f32, `blocks(n)` of a tensor of n elements); zeros, scales
    too, before the first step; v holds the root's codes then.  copies: bf16 tensors that get the new weights too
    (with f32 weights; None in a place: none).  weight_decay: one for all or one a tensor.  seed: None, rounding
    to nearest; 0 .. 2^32 - 1, rounding codes and bf16 weights at random.

    The object keeps the tensors alive, and their addresses: a tensor must stay where it is."""

    BLOCK = 128

    @classmethod
    def blocks(cls, n: int) -> int:
        """Scales of a tensor of n elements with 8-bit states."""
        return -(-n // cls.BLOCK)

    def __init__(self, params: Sequence, grads: Sequence, m: Sequence, v: Sequence, m_scales: Optional[Sequence] = None,
                 v_scales: Optional[Sequence] = None, copies: Optional[Sequence] = None, betas: Sequence[float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01, seed: Optional[int] = None):
        import torch
        self._h = None
        who, count = "AdamW", len(params)
        bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
        codes = {bf16: D.BF16, f32: D.F32, e4m3: D.E4M3}
        if not count:
            raise D.DttError(D.EINVAL, f"{who}: no tensors")
        decay = [weight_decay] * count if isinstance(weight_decay, (int, float)) else list(weight_decay)
        small = m[0].dtype == e4m3 if len(m) else False
        self._lists = {"params": list(params), "grads": list(grads), "m": list(m), "v": list(v)}
        for name, given in (("m_scales", m_scales), ("v_scales", v_scales), ("copies", copies)):
            self._lists[name] = [None] * count if given is None else list(given)
        for name, ts in (*self._lists.items(), ("weight_decay", decay)):
            if len(ts) != count:
                raise D.DttError(D.EINVAL, f"{who}: {len(ts)} {name} for {count} params")
        kinds = {"params": (params[0].dtype, (bf16, f32)), "grads": (grads[0].dtype, (bf16, f32)), "m": (m[0].dtype, (f32, e4m3)),
                 "v": (m[0].dtype, (f32, e4m3)), "m_scales": (f32, (f32,)), "v_scales": (f32, (f32,)), "copies": (bf16, (bf16,))}
        table = (D.dtt_adamw_tensor * count)()
        for name, ts in self._lists.items():
            dtype, allowed = kinds[name]
            if dtype not in allowed:
                raise D.DttError(D.EINVAL, f"{who}: {name} are {list(allowed)}, not {dtype}")
            for i, t in enumerate(ts):
                if t is None:
                    if name == "copies" or (name in ("m_scales", "v_scales") and not small):
                        continue
                    raise D.DttError(D.EINVAL, f"{who}: {name}[{i}] is missing")
                n = params[i].numel()
                if t.dtype != dtype or t.numel() != (self.blocks(n) if name in ("m_scales", "v_scales") else n) or not t.is_contiguous():
                    raise D.DttError(D.EINVAL, f"{who}: {name}[{i}] must be contiguous {dtype} of params[{i}]'s size, not "
                                               f"{t.dtype} of {t.numel()} elements")
                _here(who, f"{name}[{i}]", t)
        for i, e in enumerate(table):
            at = {name: ts[i].data_ptr() if ts[i] is not None and params[i].numel() else None for name, ts in self._lists.items()}
            e.param, e.grad, e.m, e.v = at["params"], at["grads"], at["m"], at["v"]
            e.m_scales, e.v_scales, e.copy = at["m_scales"], at["v_scales"], at["copies"]
            e.n, e.weight_decay = params[i].numel(), decay[i]
        if seed is not None and not 0 <= seed < 2 ** 32:
            raise D.DttError(D.EINVAL, f"{who}: seed must be 0 .. 2^32 - 1, not {seed}")
        self.desc = D.dtt_adamw_desc(codes[params[0].dtype], codes[grads[0].dtype], codes[m[0].dtype], seed is not None,
                                     betas[0], betas[1], eps, seed or 0)
        self.count, self._grad_type, self._device = count, grads[0].dtype, params[0].get_device()
        self._f32, self._i32, self._current = f32, torch.int32, torch.cuda.current_device
        out = C.c_void_p()
        D._check(D.lib().dtt_adamw_create(C.byref(self.desc), table, count, C.byref(out)))
        self._h = out
        self._run = D.lib().dtt_adamw_run

    def _scalar(self, name: str, t, dtype) -> int:
        if t.dtype != dtype or t.numel() != 1 or not t.is_cuda or t.get_device() != self._device:
            raise D.DttError(D.EINVAL, f"AdamW: {name} must be one {dtype} on the tensors' GPU")
        return t.data_ptr()

    def run(self, lr, step, grad_scale=None, grads: Optional[Sequence] = None, stream=None) -> None:
        """One step.  lr: a number, or one f32 on the GPU.  step: its number, from 1, or one int32 on the GPU, the
        steps made so far, which the call counts up (what a captured call needs).  grad_scale: one f32 on the GPU that
        the gradients are multiplied by.  grads: this step's gradients where they are not the constructor's
        (like these; the caller keeps them alive)."""
        if self._current() != self._device:
            raise D.DttError(D.EINVAL, "AdamW: the tensors' GPU must be the current one")
        lr_at = step_at = 0
        if not isinstance(lr, (int, float)):
            lr, lr_at = 0.0, self._scalar("lr", lr, self._f32)
        if not isinstance(step, int):
            step, step_at = 0, self._scalar("step", step, self._i32)
        elif not 1 <= step < 2 ** 32:
            raise D.DttError(D.EINVAL, f"AdamW: step must be 1 .. 2^32 - 1, not {step}")
        table = None
        if grads is not None:
            if len(grads) != self.count:
                raise D.DttError(D.EINVAL, f"AdamW: {len(grads)} grads for {self.count} params")
            for i, (g, p) in enumerate(zip(grads, self._lists["params"])):
                if g.dtype != self._grad_type or g.numel() != p.numel() or not g.is_contiguous() or g.get_device() != self._device:
                    raise D.DttError(D.EINVAL, f"AdamW: grads[{i}] must be like the constructor's")
            table = D._ptr_array(grads)
        rc = self._run(self._h, table, lr, step, lr_at, step_at,
                       0 if grad_scale is None else self._scalar("grad_scale", grad_scale, self._f32), D._stream(stream))
        if rc:
            D._check(rc)

    def close(self) -> None:
        if self._h is not None and self._h.value:
            D.lib().dtt_adamw_destroy(self._h)
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
