"""Training operators of a decoder layer: LayerNorm's forward with its row
statistics and its gradients, and the AdamW step that applies gradients to the
weights the forward kernels read.  Argument marshalling and buffers only: every
step of the computation runs in libtxl.so's CUDA kernels."""
from __future__ import annotations

import contextlib
import functools
from typing import Sequence

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import TXL_BF16, TXL_F32, AdamwTensor, GradTensor, TxlError, _dtype_code, _invoke, _need, _stream

_HERE = contextlib.nullcontext()
_LINEAR_GRADS = frozenset(("dx", "dw", "db"))
STATE_BLOCK = 256  # elements of one block of a flat optimizer state
_INT_MAX = 0x7FFFFFFF  # ctypes cuts a larger size to its low 32 bits without a word


def _on(stream, device):
    """Context in which buffers for a call on ``stream`` are allocated: torch
    hands freed memory out again in the order of the stream it was allocated
    on, so a call's buffers belong to the call's stream."""
    if stream is None:
        return _HERE
    if not hasattr(stream, "cuda_stream"):
        # (torch takes a null handle for none given, and makes a stream of its own for it)
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


@contextlib.contextmanager
def _between(stream, device):
    """Torch operations on the current stream, in order with a call's ``stream``:
    they see what it has done, and what it does next sees them."""
    if stream is None:
        yield
        return
    with _on(stream, device):
        own = torch.cuda.current_stream(device)
    here = torch.cuda.current_stream(device)
    here.wait_stream(own)
    yield
    own.wait_stream(here)


def _scratch(workspace, need: int, device) -> int:
    """Address of a caller's workspace (the C call checks its alignment)."""
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if workspace.numel() * workspace.element_size() < need:
        raise TxlError(-7, "workspace")
    return workspace.data_ptr()


@functools.lru_cache(maxsize=1024)
def _workspace_need(index: int, name: str, *sizes) -> int:
    """Workspace of a call of these sizes on device ``index``: a function of both alone."""
    if max(sizes) > _INT_MAX:
        raise TxlError(-2, name)
    return int(_invoke(index, name, *sizes))


def _row_args(x, y, gamma):
    """Checks the tensors that both LayerNorm calls share; returns (rows, d, shape, dtype, device)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor [..., d]")
    shape, dt, dev = x.shape, x.dtype, x.device
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"unsupported dtype {dt}: bf16 or fp32 only")
    d = shape[-1]
    if d == 0:
        raise ValueError("x must have a last axis of at least one element")
    if d > _INT_MAX:
        raise TxlError(-2, "last axis of x")
    _need(x, "x", shape, dt)
    if y is not None:
        _need(y, "y", shape, dt, dev)
    _need(gamma, "gamma", (d,), dt, dev)
    return x.numel() // d, d, shape, dt, dev


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def layer_norm_fwd(x, gamma, beta, y=None, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """txl_layer_norm_fwd: LayerNorm(x + y) * gamma + beta over the last axis
    (y optional), keeping the statistics that layer_norm_bwd takes.  x [..., d]
    bf16 or fp32 with 1 <= d <= 16384; mean, rstd fp32 [...].  Returns
    (out, mean, rstd); out overlaps no input."""
    rows, d, shape, dt, dev = _row_args(x, y, gamma)
    _need(beta, "beta", (d,), dt, dev)
    st, f32 = shape[:-1], torch.float32
    with _on(stream, dev):
        if out is None:
            out = torch.empty_like(x)
        else:
            _need(out, "out", shape, dt, dev)
        if mean is None:
            mean = torch.empty(st, dtype=f32, device=dev)
        else:
            _need(mean, "mean", st, f32, dev)
        if rstd is None:
            rstd = torch.empty(st, dtype=f32, device=dev)
        else:
            _need(rstd, "rstd", st, f32, dev)
    rc = _invoke(dev, "txl_layer_norm_fwd", x.data_ptr(), _ptr(y), gamma.data_ptr(), beta.data_ptr(), rows, d,
                 float(eps), out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _dtype_code(x), _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_layer_norm_fwd")
    return out, mean, rstd


def layer_norm_bwd_workspace_bytes(rows, d, dtype=torch.bfloat16, device=None) -> int:
    """txl_layer_norm_bwd_workspace_bytes for a call on ``device`` (default: the
    current one)."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"unsupported dtype {dtype}: bf16 or fp32 only")
    if max(rows, d) > _INT_MAX:
        return 0  # as for every size that the call refuses
    code = TXL_BF16 if dtype is torch.bfloat16 else TXL_F32
    dev = device if device is not None else torch.cuda.current_device()
    return int(_invoke(dev, "txl_layer_norm_bwd_workspace_bytes", rows, d, code))


def layer_norm_bwd(dout, x, gamma, mean, rstd, y=None, dres=None, stream=None, workspace=None, grads=None):
    """txl_layer_norm_bwd: gradients of layer_norm_fwd's output.  dout, x, y as
    its out, x, y; mean, rstd as it returned them; dres [..., d] (optional) is
    added to dx: the gradient that reaches x + y along a residual path.
    Returns a dict dx (x's type; the gradient of x and of y), dgamma, dbeta
    (fp32 [d], summed in a fixed order).  grads: a dict of preallocated tensors
    to fill; workspace: a uint8 tensor of at least
    layer_norm_bwd_workspace_bytes(...) bytes (allocated here when None)."""
    rows, d, shape, dt, dev = _row_args(x, y, gamma)
    st, f32, code = shape[:-1], torch.float32, TXL_BF16 if dt is torch.bfloat16 else TXL_F32
    _need(dout, "dout", shape, dt, dev)
    if dres is not None:
        _need(dres, "dres", shape, dt, dev)
    _need(mean, "mean", st, f32, dev)
    _need(rstd, "rstd", st, f32, dev)
    need = _workspace_need(dev.index, "txl_layer_norm_bwd_workspace_bytes", rows, d, code)
    with _on(stream, dev):
        if grads is None:
            dx = torch.empty_like(x)
            dgamma = torch.empty(d, dtype=f32, device=dev)
            dbeta = torch.empty(d, dtype=f32, device=dev)
            grads = {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        else:
            dx, dgamma, dbeta = grads["dx"], grads["dgamma"], grads["dbeta"]
            _need(dx, "dx", shape, dt, dev)
            _need(dgamma, "dgamma", (d,), f32, dev)
            _need(dbeta, "dbeta", (d,), f32, dev)
        if workspace is not None:
            at = _scratch(workspace, need, dev)
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            at = workspace.data_ptr()
        else:
            at = 0
    rc = _invoke(dev, "txl_layer_norm_bwd", dout.data_ptr(), x.data_ptr(), _ptr(y), gamma.data_ptr(),
                 mean.data_ptr(), rstd.data_ptr(), _ptr(dres), rows, d, dx.data_ptr(), dgamma.data_ptr(),
                 dbeta.data_ptr(), code, at, need, _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_layer_norm_bwd")
    return grads


def _linear_shape(x):
    """(layout, B, T, K) of a Linear input: [B, T, K] rows or [B, K/64, T, 64] heads."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() == 3:
        return (0, *x.shape)
    if x.dim() == 4 and x.shape[3] == 64:
        B, H, T, _ = x.shape
        return 1, B, T, H * 64
    raise ValueError("x must be [B, T, K] or [B, K/64, T, 64]")


def linear_bwd_workspace_bytes(x_shape, N, want=("dx", "dw", "db"), device=None) -> int:
    """txl_linear_bwd_workspace_bytes for x of shape [B, T, K] or
    [B, K/64, T, 64] and N output columns, on ``device`` (default: the current
    one; the split depends on its SM count)."""
    layout, B, T, K = _linear_shape(torch.empty(x_shape, device="meta"))
    if max(B, T, K, N) > _INT_MAX:
        return 0  # as for every size that the call refuses
    dev = device if device is not None else torch.cuda.current_device()
    return int(_invoke(dev, "txl_linear_bwd_workspace_bytes", layout, B, T, K, N, *("dx" in want, "dw" in want, "db" in want)))


def linear_bwd(dy, x, w, relu_in=False, want=("dx", "dw", "db"), stream=None, workspace=None, grads=None):
    """txl_linear_bwd: gradients of linear's out = x w^T + bias from dy
    [B, T, N], the gradient of out.  x [B, T, K] or heads [B, K/64, T, 64], w
    [N, K], all bf16.  Returns a dict of what ``want`` names: dx (bf16, x's
    layout), dw (fp32 [N, K]), db (fp32 [N], only along with dw).  relu_in: x is
    the output of a ReLU, and dx becomes the gradient of the ReLU's input.
    grads: a dict of preallocated tensors to fill; workspace: a uint8 tensor of
    at least linear_bwd_workspace_bytes(...) bytes (allocated here when None)."""
    layout, B, T, K = _linear_shape(x)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [N, K]")
    if not want or not _LINEAR_GRADS.issuperset(want):
        raise ValueError(f"want names gradients out of dx, dw, db: got {want}")
    N, dev, bf, f32 = w.shape[0], x.device, torch.bfloat16, torch.float32
    _need(x, "x", x.shape, bf)
    _need(w, "w", (N, K), bf, dev)
    _need(dy, "dy", (B, T, N), bf, dev)
    wx, ww, wb = "dx" in want, "dw" in want, "db" in want
    need = _workspace_need(dev.index, "txl_linear_bwd_workspace_bytes", layout, B, T, K, N, wx, ww, wb)
    dx = dw = db = None
    with _on(stream, dev):
        if grads is None:
            grads = {}
            if wx:
                grads["dx"] = dx = torch.empty_like(x)
            if ww:
                grads["dw"] = dw = torch.empty((N, K), dtype=f32, device=dev)
            if wb:
                grads["db"] = db = torch.empty(N, dtype=f32, device=dev)
        else:
            if wx:
                dx = grads["dx"]
                _need(dx, "dx", x.shape, bf, dev)
            if ww:
                dw = grads["dw"]
                _need(dw, "dw", (N, K), f32, dev)
            if wb:
                db = grads["db"]
                _need(db, "db", (N,), f32, dev)
        if workspace is not None:
            at = _scratch(workspace, need, dev)
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            at = workspace.data_ptr()
        else:
            at = 0
    rc = _invoke(dev, "txl_linear_bwd", dy.data_ptr(), x.data_ptr(), layout, B, T, K, w.data_ptr(), N,
                 int(bool(relu_in)), _ptr(dx), _ptr(dw), _ptr(db), at, need, _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_linear_bwd")
    return grads


class _Bound:
    """What is bound to tensors once and then called on streams: ``device``, ``_storages``
    (the bound memory) and _own() (tensors of its own, made on the stream that _made
    records)."""

    def _made(self) -> None:
        made_on = torch.cuda.current_stream(self.device)
        # (made in a capture, the fills run with its replay: no event outside stands for them)
        self._ready = None if torch.cuda.is_current_stream_capturing() else made_on.record_event()
        self._joined = {made_on.cuda_stream}  # streams whose calls come after the fills

    def _join(self, handle: int) -> None:
        """Puts the calls on a further stream behind the constructor's fills, and the
        release of all memory that they use behind them."""
        with _on(handle, self.device):
            if torch.cuda.is_current_stream_capturing():
                return  # a graph cannot wait for what is outside of it
            st = torch.cuda.current_stream(self.device)
        if self._ready is not None:
            st.wait_event(self._ready)
        bound = [torch.empty(0, dtype=torch.uint8, device=self.device).set_(x) for x in self._storages]
        for t in self._own() + bound:
            if t is not None:
                t.record_stream(st)
        self._joined.add(handle)


class AdamW(_Bound):
    """AdamW over a list of parameters in one launch sequence (txl_adamw_step),
    with the moments in fp32 or in 8 bits.

    ``params``: contiguous CUDA tensors of one type, fp32 or bf16 (bf16
    parameters get an fp32 master copy, which the steps update and round into
    them: the forward kernels keep reading the same tensors); ``grads``: one
    gradient per parameter, fp32 or bf16, the buffers that the backward calls
    fill.  Both are bound here, as a captured graph binds them: step() reads the
    gradients from this memory and updates the parameters in this memory, which
    the optimizer keeps alive (a tensor that is given other storage later, as by
    ``p.data = ...``, is no longer the one that is stepped).  A step moves the
    parameters' version counters, so that autograd refuses a backward pass through what
    was computed from the old values (a graph's replay moves none).  ``weight_decay``: one
    number, or one per parameter.  ``max_norm``: gradients are scaled by
    min(1, max_norm / norm), norm the 2-norm of all of them, kept in ``grad_norm``
    [1]; a norm that is not finite makes the step change nothing.  ``eps``: 0, or at
    least 2^-126.  ``state_bits`` 8:
    the moments as e4m3 codes with one scale per 256 elements, rounded at random
    from ``seed``.  ``stream``: the stream of the steps (default: the current one
    of each call); what is enqueued on the current stream when the optimizer is made
    is waited for.  A first step on a further stream waits for what the constructor
    enqueued, and the memory of the optimizer is not handed out again before that
    stream has done with it; gradients, parameters and steps on several streams are the
    caller's to order.  A captured step waits for nothing outside its graph, and its
    graph is replayed only while the optimizer lives.

    Device values: ``lr`` [1] fp32 (set_lr), ``steps`` [1] int64 (steps done), the
    flat ``master`` (None for fp32 parameters) and states(); parameter i's part of
    the flat buffers starts at ``starts[i]``.  A step reads all of them when it
    runs: captured in a graph it can be replayed."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr: float,
                 betas: tuple = (0.9, 0.999), eps: float = 1e-8, weight_decay: float | Sequence[float] = 0.0,
                 state_bits: int = 32, max_norm: float | None = None, seed: int = 0,
                 stream: torch.cuda.Stream | None = None):
        self.params, self.grads = list(params), list(grads)
        n = len(self.params)
        if n == 0 or len(self.grads) != n:
            raise ValueError("need one gradient per parameter, and at least one parameter")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive, or None")
        decay = [float(weight_decay)] * n if not isinstance(weight_decay, (list, tuple)) else list(map(float, weight_decay))
        if len(decay) != n:
            raise ValueError("need one weight_decay, or one per parameter")
        p0, g0 = self.params[0], self.grads[0]
        for t in (p0, g0):
            if not isinstance(t, torch.Tensor):
                raise TypeError("params and grads must be torch.Tensors")
        self.device = dev = p0.device
        self._param_dtype, self._grad_dtype = _dtype_code(p0), _dtype_code(g0)
        self._table = (AdamwTensor * n)()
        self.starts, total = [], 0
        for i, (p, g) in enumerate(zip(self.params, self.grads)):
            _need(p, f"params[{i}]", p.shape, p0.dtype, dev)
            _need(g, f"grads[{i}]", p.shape, g0.dtype, dev)
            self._table[i] = AdamwTensor(p.data_ptr(), g.data_ptr(), p.numel(), decay[i], 0)
            self.starts.append(total)
            total += -(-p.numel() // STATE_BLOCK) * STATE_BLOCK
        self._storages = [t.untyped_storage() for t in self.params + self.grads]
        self.betas, self.eps, self.weight_decay = tuple(map(float, betas)), float(eps), decay
        self.state_bits, self.max_norm, self.seed = state_bits, max_norm, int(seed) & 0xFFFFFFFF
        self._fixed_stream = stream
        if _invoke(dev, "txl_adamw_state_elements", self._table, n) != total:
            raise TxlError(-1, "txl_adamw_state_elements")
        need = int(_invoke(dev, "txl_adamw_workspace_bytes", self._table, n))
        f32 = dict(dtype=torch.float32, device=dev)
        here = torch.cuda.current_stream(dev)
        with _on(stream, dev):
            if stream is not None:
                torch.cuda.current_stream(dev).wait_stream(here)  # what is still writing the parameters
            self.lr = torch.full((1,), float(lr), **f32)
            self.steps = torch.zeros(1, dtype=torch.int64, device=dev)
            self.grad_norm = torch.zeros(1, **f32) if max_norm is not None else None
            self.master = None
            if p0.dtype == torch.bfloat16:
                self.master = torch.zeros(total, **f32)
                self._copy_masters()
            code = torch.float8_e4m3fn if state_bits == 8 else torch.float32
            self.exp_avg = torch.zeros(total, **f32).to(code)
            self.exp_avg_sq = torch.zeros(total, **f32).to(code)
            blocks = total // STATE_BLOCK
            self.exp_avg_scale = torch.zeros(blocks, **f32) if state_bits == 8 else None
            self.exp_avg_sq_scale = torch.zeros(blocks, **f32) if state_bits == 8 else None
            self._workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            self._made()
        args = (self._table, n, self._param_dtype, self._grad_dtype, state_bits, _ptr(self.master),
                self.exp_avg.data_ptr(), _ptr(self.exp_avg_scale), self.exp_avg_sq.data_ptr(),
                _ptr(self.exp_avg_sq_scale), self.steps.data_ptr(), self.lr.data_ptr(), *self.betas, self.eps,
                float(max_norm or 0.0), self.seed, _ptr(self.grad_norm), self._workspace.data_ptr(), need)
        # converted once for all steps (0.5 us of each)
        types = _lib.load().txl_adamw_step.argtypes[1:]
        self._args = (self._table, *(of(a) for of, a in zip(types, args[1:])))

    def _copy_masters(self) -> None:
        with torch.no_grad():
            for p, a in zip(self.params, self.starts):
                self.master[a:a + p.numel()].copy_(p.reshape(-1))

    def _own(self) -> list:
        return [self.lr, self.steps, self.grad_norm, self.master, self._workspace, *self.states()]

    def step(self, stream=None) -> None:
        """One step from the gradients as they stand, on ``stream`` (default:
        the constructor's, else the current one)."""
        handle = _stream(stream if stream is not None else self._fixed_stream, self.device)
        if handle not in self._joined:
            self._join(handle)
        rc = _invoke(self.device, "txl_adamw_step", *self._args, handle)
        if rc != 0:
            raise TxlError(rc, "txl_adamw_step")
        increment_version(self.params)

    def set_lr(self, lr: float) -> None:
        """Learning rate of the steps that follow (in the order of the current
        stream, and of the constructor's if it was given one)."""
        with _between(self._fixed_stream, self.device):
            self.lr.fill_(float(lr))

    def states(self) -> list:
        """The flat moments: [exp_avg, exp_avg_sq] in fp32, or with 8 bits
        [codes of exp_avg, scales, codes of sqrt(exp_avg_sq), scales]."""
        if self.state_bits == 32:
            return [self.exp_avg, self.exp_avg_sq]
        return [self.exp_avg, self.exp_avg_scale, self.exp_avg_sq, self.exp_avg_sq_scale]

    def state_dict(self) -> dict:
        """Step count, moments and master copy (checkpoint/resume; the
        parameters are the caller's)."""
        with _between(self._fixed_stream, self.device):
            return {"steps": self.steps.clone(), "lr": self.lr.clone(), "states": [s.clone() for s in self.states()],
                    "master": None if self.master is None else self.master.clone()}

    def load_state_dict(self, sd: dict) -> None:
        """Restores state_dict's values.  bf16 parameters are set to the
        rounding of the restored master copy."""
        if len(sd["states"]) != len(self.states()) or (sd["master"] is None) != (self.master is None):
            raise ValueError("state of another state_bits or parameter type")
        pairs = list(zip(self.states() + [self.steps, self.lr], list(sd["states"]) + [sd["steps"], sd["lr"]]))
        if self.master is not None:
            pairs.append((self.master, sd["master"]))
        for mine, given in pairs:
            if mine.shape != given.shape or mine.dtype != given.dtype:
                raise ValueError(f"state is {given.dtype} {tuple(given.shape)}, expected {mine.dtype} {tuple(mine.shape)}")
        with torch.no_grad(), _between(self._fixed_stream, self.device):
            for mine, given in pairs:
                mine.copy_(given)
            if self.master is not None:
                for p, a in zip(self.params, self.starts):
                    p.copy_(self.master[a:a + p.numel()].view(p.shape))


class GradNorm(_Bound):
    """The norms of many gradients, and their clipping, in two launches (txl_grad_norm).

    ``grads``: contiguous CUDA tensors, fp32 or bf16, of both types if need be; their memory
    is bound here, as AdamW binds it (which clips by itself where it is given a max_norm:
    this is for gradients that something else reads, or that are to be watched).  Device
    values: ``norm`` [1], the 2-norm of all, and ``norms`` [n], that of each, fp32; both
    written by measure() and, before the scaling, by clip().  Calls on several streams are
    the caller's to order; the first on a further stream waits for the constructor."""

    def __init__(self, grads: Sequence[torch.Tensor]):
        self.grads = list(grads)
        n = len(self.grads)
        if n == 0:
            raise ValueError("need at least one gradient")
        self._table, dev = (GradTensor * n)(), None
        for i, g in enumerate(self.grads):
            if not isinstance(g, torch.Tensor):
                raise TypeError("grads must be torch.Tensors")
            code = _dtype_code(g)
            _need(g, f"grads[{i}]", g.shape, g.dtype, dev)
            dev = g.device
            self._table[i] = GradTensor(g.data_ptr(), g.numel(), code, 0)
        self.device = dev
        self._storages = [t.untyped_storage() for t in self.grads]
        need = int(_invoke(dev, "txl_grad_norm_workspace_bytes", self._table, n))
        self.norm = torch.empty(1, dtype=torch.float32, device=dev)
        self.norms = torch.empty(n, dtype=torch.float32, device=dev)
        self._workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):
            self._made()
        # (views of one tensor share its version counter)
        self._versions = list({id(t if t._base is None else t._base): t for t in self.grads}.values())
        types = _lib.load().txl_grad_norm.argtypes
        args = (self.norm.data_ptr(), self.norms.data_ptr(), self._workspace.data_ptr(), need)
        self._args = tuple(of(a) for of, a in zip(types[3:], args))

    def _own(self) -> list:
        return [self.norm, self.norms, self._workspace]

    def _call(self, max_norm: float, stream) -> None:
        handle = _stream(stream, self.device)
        if handle not in self._joined:
            self._join(handle)
        rc = _invoke(self.device, "txl_grad_norm", self._table, len(self._table), max_norm, *self._args, handle)
        if rc != 0:
            raise TxlError(rc, "txl_grad_norm")

    def measure(self, stream=None) -> None:
        """Norms of the gradients as they stand, on ``stream`` (default: the current one)."""
        self._call(0.0, stream)

    def clip(self, max_norm: float, stream=None) -> None:
        """measure(), and gradients scaled in place by max_norm / norm where norm is above
        max_norm and finite.  Moves the gradients' version counters, as AdamW's step the
        parameters'."""
        if not max_norm > 0:
            raise ValueError("max_norm must be positive")
        self._call(float(max_norm), stream)
        increment_version(self._versions)
