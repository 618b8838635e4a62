"""Python binding of the loss over a vocabulary, its gradients and the orthogonalised
adapter updates (argument marshalling only; the C ABI is include/gptq_train.h).

Tensors must live on the current HIP device; work is enqueued on torch's current
stream.
"""
from __future__ import annotations

import torch

from . import _lib
from .adapter import _check_out, _device, _ld, _ptr, _rows, _rows16, _stream
from .gptq import _DT, Workspace, _need, _ws

__all__ = ["linear_cross_entropy", "linear_cross_entropy_backward", "adapter_orthogonalize"]


def _vector(t, name, dtype, n):
    _need(t, name, dtype, 1, on_gpu=False)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of length {n}")


def _head(X, W, target):
    """(n, d, vocab) of checked hidden states, output head and targets."""
    _rows16(X, "X")
    n, d = X.shape
    _rows16(W, "W", None, d, X.dtype)
    _vector(target, "target", torch.int64, n)
    return n, d, W.shape[0]


def _outputs(out, names):
    o = dict(out or {})
    unknown = set(o) - set(names)
    if unknown:
        raise ValueError(f"unknown output names {sorted(unknown)}")
    return o


def linear_cross_entropy(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor,
                         out: tuple[torch.Tensor, torch.Tensor] | None = None,
                         ws: Workspace | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse), fp32 [n] each, of hidden states X [n, d] under the output head W
    [vocab, d] (both bf16 or both fp16; d a multiple of 8): loss = lse - z[target]
    with z = X W^T, which is never kept.  target int64 [n]; a value outside 0 .. vocab-1
    (torch's -100) is no target: loss and lse are 0, whatever the token's X holds.

    The mean over a corpus, exponentiated, is a quantized model's perplexity; W may
    be a quantized head's w_hat rounded by round16."""
    n, d, vocab = _head(X, W, target)
    if out is not None:
        for t, name in zip(out, ("out[0]", "out[1]"), strict=True):
            _vector(t, name, torch.float32, n)
    dev = _device(X, W, target, *(out or ()))
    buf, nb = _ws(ws, _lib.query("gptq_linear_cross_entropy_workspace_size", n, d, vocab), dev)
    loss, lse = out if out is not None else (torch.empty(n, dtype=torch.float32, device=dev) for _ in range(2))
    _lib.call("gptq_linear_cross_entropy", _ptr(X), _DT[X.dtype], n, d, _ld(X), _ptr(W), vocab, _ld(W), _ptr(target), _ptr(loss),
              _ptr(lse), _ptr(buf), nb, _stream(dev))
    return loss, lse


def linear_cross_entropy_backward(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                                  dloss: torch.Tensor | None = None, want_dX: bool = True, want_dW: bool = False,
                                  out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Gradients of linear_cross_entropy, whose lse is given, from dloss fp32 [n], the
    gradient that arrives at each token's loss (None: 1).

    Returns {X [n, d] or None, W [vocab, d] or None}, of X's type: D W and D^T X with D
    = dloss (softmax - onehot).  Tokens without a target have zero rows of dX and
    enter dW with nothing.  `out` may supply preallocated tensors with those keys."""
    n, d, vocab = _head(X, W, target)
    _vector(lse, "lse", torch.float32, n)
    if dloss is not None:
        _vector(dloss, "dloss", torch.float32, n)
    o = _outputs(out, ("X", "W"))
    dX, dW = o.get("X"), o.get("W")
    _check_out(dX, "out['X']", n, d, X.dtype)
    _check_out(dW, "out['W']", vocab, d, X.dtype)
    want_dX, want_dW = want_dX or dX is not None, want_dW or dW is not None
    if not want_dX and not want_dW:
        raise ValueError("neither dX nor dW is wanted")
    dev = _device(X, W, target, lse, dloss, dX, dW)
    buf, nb = _ws(ws, _lib.query("gptq_linear_cross_entropy_backward_workspace_size", n, d, vocab, int(want_dX), int(want_dW)), dev)
    if want_dX and dX is None:
        dX = torch.empty((n, d), dtype=X.dtype, device=dev)
    if want_dW and dW is None:
        dW = torch.empty((vocab, d), dtype=X.dtype, device=dev)
    _lib.call("gptq_linear_cross_entropy_backward", _ptr(X), _DT[X.dtype], n, d, _ld(X), _ptr(W), vocab, _ld(W), _ptr(target),
              _ptr(lse), _ptr(dloss), _ptr(dX), _ld(dX) if want_dX else 0, _ptr(dW), _ld(dW) if want_dW else 0, _ptr(buf), nb,
              _stream(dev))
    return {"X": dX, "W": dW}


def adapter_orthogonalize(A: torch.Tensor | None = None, B: torch.Tensor | None = None, steps: int = 5,
                          coefficients: tuple[float, float, float] = (3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                          out_dtype: torch.dtype | None = None, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Orthogonalised updates from the gradients (or momenta of them) of adapters'
    factors, A [m, rank, c] and B [m, r, rank] as adapter_backward gives them, either
    or both: each matrix is divided by its Frobenius norm + eps and its singular
    values s go through a s + b s^3 + c s^5 `steps` times (Newton-Schulz; 1 to 16), in
    64 bits throughout.

    Returns {A, B} (None where not given) of the inputs' type (float32, bfloat16 or
    float16) or out_dtype.  The shorter side of a matrix is at most 128."""
    if A is None and B is None:
        raise ValueError("neither A nor B is given")
    a, b, c3 = (float(v) for v in coefficients)
    for t, name in ((A, "A"), (B, "B")):
        if t is not None:
            _need(t, name, None, 3, on_gpu=False)
            if t.dtype not in _DT:
                raise TypeError(f"{name} must be float32, bfloat16 or float16")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    if A is not None and B is not None and (A.dtype != B.dtype or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2]):
        raise ValueError(f"A must be [m, rank, c] and B [m, r, rank] of one type, got {tuple(A.shape)} and {tuple(B.shape)}")
    first = A if A is not None else B
    m, rank = first.shape[0], first.shape[1] if A is not None else first.shape[2]
    c, r = A.shape[2] if A is not None else 0, B.shape[1] if B is not None else 0
    o = _outputs(out, ("A", "B"))
    ot = out_dtype or next((t.dtype for t in o.values() if t is not None), first.dtype)
    if ot not in _DT:
        raise TypeError("the result must be float32, bfloat16 or float16")
    for k, t in (("A", A), ("B", B)):
        if o.get(k) is not None:
            if t is None:
                raise ValueError(f"out[{k!r}] without {k}")
            _need(o[k], f"out[{k!r}]", ot, 3, on_gpu=False)
            if o[k].shape != t.shape or not o[k].is_contiguous():
                raise ValueError(f"out[{k!r}] must be a contiguous tensor of shape {tuple(t.shape)}")
    dev = _device(first, A, B, *o.values())
    buf, nb = _ws(ws, _lib.query("gptq_adapter_orthogonalize_workspace_size", m, rank, c, r, int(steps)), dev)
    got = {k: o.get(k) if o.get(k) is not None or t is None else torch.empty(t.shape, dtype=ot, device=dev)
           for k, t in (("A", A), ("B", B))}
    _lib.call("gptq_adapter_orthogonalize", _ptr(A), _ptr(B), _DT[first.dtype], m, rank, c, r, int(steps), a, b, c3, float(eps),
              _ptr(got["A"]), _ptr(got["B"]), _DT[ot], _ptr(buf), nb, _stream(dev))
    return got
