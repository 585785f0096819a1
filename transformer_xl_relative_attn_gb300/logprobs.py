"""Log probabilities of given tokens, behind a decoder's last layer: from logits,
with each row's log-sum-exp, entropy and best alternatives, and their gradient; or
straight from hidden states and the output weights, without the logits.
Argument marshalling and buffers only: every step of the computation runs in
libtxl.so's CUDA kernels."""
from __future__ import annotations

import operator

import torch
from torch.autograd.graph import increment_version

from ._lib import TXL_BF16, TXL_F32, TxlError, _invoke, _need, _stream
from .train import _INT_MAX, _on, _ptr, _scratch, _workspace_need

_F32, _I64, _BF16 = torch.float32, torch.int64, torch.bfloat16
_TOP_MOST = 32
_CODES = {_BF16: TXL_BF16, _F32: TXL_F32}


def _rows(t, name: str):
    """(rows, V, distance of the rows in elements) of logits [..., V]: each row
    contiguous, all rows at one distance (a slice of a wider, padded buffer is fine)."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise ValueError(f"{name} must be a tensor [..., V]")
    V = t.shape[-1]
    if V == 0:
        raise ValueError(f"{name} must have a last axis of at least one element")
    rows = t.numel() // V
    if t.is_contiguous():
        return rows, V, V
    ld, size = None, 1  # elements between rows, rows of the axes seen so far
    if V > 1 and t.stride(-1) != 1:
        raise ValueError(f"each row of {name} must be contiguous")
    for n, step in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = step
        if step != ld * size or ld < V:
            raise ValueError(f"the rows of {name} must lie at one distance of at least their length")
        size *= n
    return rows, V, V if ld is None else ld


def _type_of(t, name: str) -> int:
    """The type of logits, which must be on a GPU."""
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}: bf16 or fp32 only")
    _on_gpu(t, name)
    return code


def _on_gpu(t, name: str, device=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")


def _new(shape, top: int, dev):
    """New outputs: logprob, lse, entropy, and with top its two (an allocation each; parts of one
    buffer take twice the time)."""
    logprob = torch.empty(shape, dtype=_F32, device=dev)
    lse = torch.empty(shape, dtype=_F32, device=dev)
    entropy = torch.empty(shape, dtype=_F32, device=dev)
    if not top:
        return logprob, lse, entropy, None, None
    shape = (*shape, top)
    return logprob, lse, entropy, torch.empty(shape, dtype=_I64, device=dev), torch.empty(shape, dtype=_F32, device=dev)


def _outputs(shape, top: int, dev, stream, outs):
    """logprob, lse, entropy, top_index, top_logprob: the caller's, or new ones."""
    if outs is None:
        if stream is None:
            return _new(shape, top, dev)
        with _on(stream, dev):
            return _new(shape, top, dev)
    for n in ("logprob", "lse", "entropy"):
        _need(outs[n], n, shape, _F32, dev)
    if not top:
        return outs["logprob"], outs["lse"], outs["entropy"], None, None
    _need(outs["top_index"], "top_index", (*shape, top), _I64, dev)
    _need(outs["top_logprob"], "top_logprob", (*shape, top), _F32, dev)
    return outs["logprob"], outs["lse"], outs["entropy"], outs["top_index"], outs["top_logprob"]


def token_logprobs(logits, tokens, top=0, stream=None, outs=None):
    """txl_token_logprobs: of each row of logits [..., V] (bf16 or fp32; rows
    contiguous, at one distance) and its token (int64 [...], negative: none) a dict of
    logprob, lse, entropy (fp32 [...]): ln p of the token (0 without one, NaN for a
    token of V or more), ln sum e^x, -sum p ln p; with top > 0 (at most 32) also
    top_index (int64) and top_logprob (fp32) [..., top]: the largest logits, of equal
    ones the lower index first, and their ln p.  outs: a dict of preallocated tensors
    to fill.  A row of nothing but -inf: lse, ln p -inf, entropy 0; a row with NaN or
    +inf: NaN."""
    rows, V, ld = _rows(logits, "logits")
    code, dev, shape = _type_of(logits, "logits"), logits.device, logits.shape[:-1]
    _need(tokens, "tokens", shape, _I64, dev)
    if type(top) is not int:  # an integer of another type, as NumPy's are
        try:
            top = int(operator.index(top))
        except TypeError:
            raise ValueError("top must be a count") from None
    if top < 0:
        raise ValueError("top must be a count")
    if V > _INT_MAX or rows > _INT_MAX or top > _TOP_MOST:  # (ahead of buffers for so many)
        raise TxlError(-1 if top > V else -2, "txl_token_logprobs")
    logprob, lse, entropy, index, value = _outputs(shape, top, dev, stream, outs)
    rc = _invoke(dev, "txl_token_logprobs", logits.data_ptr(), ld, tokens.data_ptr(), rows, V, top, logprob.data_ptr(),
                 lse.data_ptr(), entropy.data_ptr(), _ptr(index), _ptr(value), code, _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_token_logprobs")
    if outs is not None:
        return outs
    outs = {"logprob": logprob, "lse": lse, "entropy": entropy}
    if top:
        outs["top_index"], outs["top_logprob"] = index, value
    return outs


def token_logprobs_bwd(logits, tokens, lse, dlogprob=None, dlse=None, dentropy=None, entropy=None, out=None, stream=None):
    """txl_token_logprobs_bwd: the gradient of logits (their type) from those of
    token_logprobs' logprob, lse and entropy (fp32 [...], None: zeros; one at least).
    lse, and with dentropy also entropy, as it returned them.  out: like logits, may be
    logits itself, whose place the gradient then takes.  A row without a token takes
    nothing from dlogprob; a row whose gradients are all 0 gets zeros whatever its
    logits hold."""
    rows, V, ld = _rows(logits, "logits")
    code, dev, shape = _type_of(logits, "logits"), logits.device, logits.shape[:-1]
    _need(tokens, "tokens", shape, _I64, dev)
    _need(lse, "lse", shape, _F32, dev)
    if dlogprob is None and dlse is None and dentropy is None:
        raise ValueError("need at least one of dlogprob, dlse, dentropy")
    if dlogprob is not None:
        _need(dlogprob, "dlogprob", shape, _F32, dev)
    if dlse is not None:
        _need(dlse, "dlse", shape, _F32, dev)
    if dentropy is not None:
        _need(dentropy, "dentropy", shape, _F32, dev)
        _need(entropy, "entropy", shape, _F32, dev)
    if V > _INT_MAX or rows > _INT_MAX:
        raise TxlError(-2, "txl_token_logprobs_bwd")
    if out is None:
        if stream is None:
            out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        else:
            with _on(stream, dev):
                out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        ldd = V
    else:
        if not isinstance(out, torch.Tensor) or out.shape != logits.shape or out.dtype is not logits.dtype:
            raise ValueError(f"out must be a tensor {tuple(logits.shape)} of {logits.dtype}")
        _on_gpu(out, "out", dev)
        _, _, ldd = _rows(out, "out")
    rc = _invoke(dev, "txl_token_logprobs_bwd", logits.data_ptr(), ld, tokens.data_ptr(), lse.data_ptr(),
                 entropy.data_ptr() if dentropy is not None else 0, _ptr(dlogprob), _ptr(dlse), _ptr(dentropy), rows, V,
                 out.data_ptr(), ldd, code, _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_token_logprobs_bwd")
    if out.data_ptr() == logits.data_ptr() and not out.is_inference():
        increment_version([out])  # what was computed from the logits is not differentiated any more
    return out


def linear_logprobs_workspace_bytes(rows, K, V, device=None) -> int:
    """txl_linear_logprobs_workspace_bytes for a call on ``device`` (default: the current
    one; the split depends on its SM count)."""
    if max(rows, K, V) > _INT_MAX:
        return 0  # as for every size that the call refuses
    dev = device if device is not None else torch.cuda.current_device()
    return int(_invoke(dev, "txl_linear_logprobs_workspace_bytes", rows, K, V))


def linear_logprobs(x, w, tokens, bias=None, stream=None, workspace=None, outs=None):
    """txl_linear_logprobs: token_logprobs' logprob, lse and entropy (a dict, fp32 [...])
    of the logits x w^T + bias, which are never written: x [..., K], w [V, K], bias [V]
    (or None) bf16, K a multiple of 8; tokens int64 [...] as there.  outs: a dict of
    preallocated tensors to fill; workspace: a uint8 tensor of at least
    linear_logprobs_workspace_bytes(...) bytes (allocated here when None)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor [..., K]")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [V, K]")
    K, V, dev, shape = x.shape[-1], w.shape[0], x.device, x.shape[:-1]
    if K == 0:
        raise ValueError("x must have a last axis of at least one element")
    _need(x, "x", x.shape, _BF16)
    _need(w, "w", (V, K), _BF16, dev)
    if bias is not None:
        _need(bias, "bias", (V,), _BF16, dev)
    _need(tokens, "tokens", shape, _I64, dev)
    rows = x.numel() // K
    need = _workspace_need(dev.index, "txl_linear_logprobs_workspace_bytes", rows, K, V)
    logprob, lse, entropy, _, _ = _outputs(shape, 0, dev, stream, outs)
    if workspace is not None:
        at = _scratch(workspace, need, dev)
    elif stream is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        at = workspace.data_ptr()
    else:
        with _on(stream, dev):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        at = workspace.data_ptr()
    rc = _invoke(dev, "txl_linear_logprobs", x.data_ptr(), w.data_ptr(), _ptr(bias), tokens.data_ptr(), rows, K, V,
                 logprob.data_ptr(), lse.data_ptr(), entropy.data_ptr(), at, need, _stream(stream, dev))
    if rc != 0:
        raise TxlError(rc, "txl_linear_logprobs")
    return {"logprob": logprob, "lse": lse, "entropy": entropy} if outs is None else outs
