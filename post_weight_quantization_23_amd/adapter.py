"""Python binding of the packed products for many tokens and of the low-rank
adapters beside them (argument marshalling only; the C ABI is
include/gptq_adapter.h).

Tensors must live on the current HIP device; work is enqueued on torch's
current stream.  Adapters of several requests are stacked: A [m, rank, c] and
B [m, r, rank] of the activations' 16-bit type, alpha fp32 [m] (None: 1) and
index int32 [tokens] (any value outside 0 .. m-1: no adapter; None: adapter 0
for every token).
"""
from __future__ import annotations

import torch

from . import _lib
from .gptq import _DT, Workspace, _need, _ws

__all__ = ["packed_linear", "packed_linear_backward", "adapter_add", "adapter_backward"]

_16 = (torch.bfloat16, torch.float16)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _rows16(t, name, n=None, d=None, dtype=None):
    """A bf16 / fp16 matrix with unit column stride (and the given sizes and type)."""
    _need(t, name, dtype, 2, on_gpu=False)
    if t.dtype not in _16:
        raise TypeError(f"{name} must be bfloat16 or float16")
    _rows(t, name, n, d)


def _rows(t, name, n, d):
    if (n is not None and t.shape[0] != n) or (d is not None and t.shape[1] != d):
        raise ValueError(f"{name} must be {'tokens' if n is None else n} x {'columns' if d is None else d}, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must not have overlapping rows")


def _ld(t):
    """Row stride; of a single row (whose stride says nothing) its length, rounded up to whole vectors."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _adapters(A, B, index, alpha, dtype, n, r, c):
    """(m, rank) of checked adapters, (0, 0) without."""
    if A is None and B is None:
        if index is not None or alpha is not None:
            raise ValueError("index / alpha without A and B")
        return 0, 0
    _need(A, "A", dtype, 3, on_gpu=False)
    _need(B, "B", dtype, 3, on_gpu=False)
    m, rank = A.shape[0], A.shape[1]
    if A.shape[2] != c or B.shape != (m, r, rank):
        raise ValueError(f"A must be [m, rank, {c}] and B [m, {r}, rank], got {tuple(A.shape)} and {tuple(B.shape)}")
    if not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A and B must be contiguous")
    for t, name, dt, k in ((index, "index", torch.int32, n), (alpha, "alpha", torch.float32, m)):
        if t is not None:
            _need(t, name, dt, 1, on_gpu=False)
            if t.numel() != k or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous vector of length {k}")
    return m, rank


def _layer(packed, scales, zeros, bits, c, perm):
    """Checks of a packed layer with c columns; its row count."""
    _need(packed, "packed", torch.uint32, 2, on_gpu=False)
    _need(scales, "scales", torch.float32, 2, on_gpu=False)
    _need(zeros, "zeros", torch.int32, 2, on_gpu=False)
    r = packed.shape[0]
    if packed.shape[1] * 32 < c * bits:
        raise ValueError(f"packed holds fewer than {c} columns of {bits} bits")
    if scales.shape != zeros.shape or scales.stride() != zeros.stride() or scales.shape[0] != r:
        raise ValueError("scales and zeros must have one row per packed row and the same shape and strides")
    for t, name in ((packed, "packed"), (scales, "scales")):
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"the rows of {name} must be contiguous")
    if perm is not None:
        _need(perm, "perm", torch.int32, 1, on_gpu=False)
        if perm.numel() != c or not perm.is_contiguous():
            raise ValueError("perm must be a contiguous int32 vector of length c")
    return r


def _groups(scales, groupsize, c):
    n = (c + groupsize - 1) // groupsize if 0 < groupsize < c else 1
    if scales.shape[1] < n:
        raise ValueError(f"scales / zeros need {n} groups per row")


def _device(first, *rest):
    """Every tensor on the current HIP device."""
    if not first.is_cuda:
        raise ValueError("tensors must be on the GPU")
    dev = first.device
    for t in rest:
        if t is not None and t.device != dev:
            raise ValueError(f"a tensor is on {t.device}, expected {dev}")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _check_out(out, name, n, d, dtype):
    if out is not None:
        _need(out, name, dtype, 2, on_gpu=False)
        _rows(out, name, n, d)


def _out_type(out, out_dtype, dtype):
    got = out_dtype or (out.dtype if out is not None else dtype)
    if got not in (dtype, torch.float32):
        raise TypeError(f"the result must be float32 or {dtype}")
    return got


def packed_linear(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, bits: int,
                  groupsize: int, perm: torch.Tensor | None = None, A: torch.Tensor | None = None,
                  B: torch.Tensor | None = None, index: torch.Tensor | None = None, alpha: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  ws: Workspace | None = None) -> torch.Tensor:
    """Y = X W_hat^T for a packed layer and any number of tokens, plus
    alpha_a B_a (A_a x) for each token's adapter a when A and B are given.

    X [n, c] bf16 / fp16; packed, scales, zeros, perm as for dequant_gemv; the
    result [n, r] is of X's type or float32 (out_dtype).  Weights are not rounded,
    except for 16-bit results of 1024 tokens or more, which take them rounded to X's
    type as linear_forward does; float32 results never do."""
    _rows16(X, "X")
    n, c = X.shape
    r = _layer(packed, scales, zeros, bits, c, perm)
    _groups(scales, groupsize, c)
    m, rank = _adapters(A, B, index, alpha, X.dtype, n, r, c)
    yt = _out_type(out, out_dtype, X.dtype)
    _check_out(out, "out", n, r, yt)
    dev = _device(X, packed, scales, zeros, perm, A, B, index, alpha, out)
    buf, nb = _ws(ws, _lib.query("gptq_packed_linear_workspace_size", n, r, c, _DT[yt], rank, int(perm is not None)), dev)
    out = torch.empty((n, r), dtype=yt, device=dev) if out is None else out
    _lib.call("gptq_packed_linear", _ptr(X), _DT[X.dtype], n, _ld(X), _ptr(packed), r, c, int(bits), _ld(packed),
              _ptr(scales), _ptr(zeros), _ld(scales), int(groupsize), _ptr(perm), _ptr(A), _ptr(B), m, rank, _ptr(index),
              _ptr(alpha), _ptr(out), _DT[yt], _ld(out), _ptr(buf), nb, _stream(dev))
    return out


def packed_linear_backward(dY: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, bits: int,
                           groupsize: int, perm: torch.Tensor | None = None, A: torch.Tensor | None = None,
                           B: torch.Tensor | None = None, index: torch.Tensor | None = None,
                           alpha: torch.Tensor | None = None, cols: int | None = None, out: torch.Tensor | None = None,
                           out_dtype: torch.dtype | None = None, ws: Workspace | None = None) -> torch.Tensor:
    """dX = dY W_hat, plus alpha_a (dY B_a) A_a for each token's adapter: the
    gradient of packed_linear for its input.

    dY [n, r] bf16 / fp16; the result [n, c] is of dY's type, with weights rounded to
    it, or float32 (out_dtype), with weights held in as many 16-bit terms as float32
    has bits.  c is `cols`, or what the packed words hold.  perm must be a
    permutation."""
    _rows16(dY, "dY")
    _need(packed, "packed", torch.uint32, 2, on_gpu=False)
    n = dY.shape[0]
    if bits not in (3, 4):
        raise ValueError("bits must be 3 or 4")
    c = int(cols) if cols is not None else packed.shape[1] * 32 // int(bits)
    r = _layer(packed, scales, zeros, bits, c, perm)
    if dY.shape[1] != r:
        raise ValueError(f"dY must be tokens x {r}, got {tuple(dY.shape)}")
    _groups(scales, groupsize, c)
    m, rank = _adapters(A, B, index, alpha, dY.dtype, n, r, c)
    ot = _out_type(out, out_dtype, dY.dtype)
    _check_out(out, "out", n, c, ot)
    dev = _device(dY, packed, scales, zeros, perm, A, B, index, alpha, out)
    buf, nb = _ws(ws, _lib.query("gptq_packed_linear_backward_workspace_size", n, r, c, _DT[dY.dtype], _DT[ot], m, rank), dev)
    out = torch.empty((n, c), dtype=ot, device=dev) if out is None else out
    _lib.call("gptq_packed_linear_backward", _ptr(dY), _DT[dY.dtype], n, _ld(dY), _ptr(packed), r, c, int(bits), _ld(packed),
              _ptr(scales), _ptr(zeros), _ld(scales), int(groupsize), _ptr(perm), _ptr(A), _ptr(B), m, rank, _ptr(index),
              _ptr(alpha), _ptr(out), _DT[ot], _ld(out), _ptr(buf), nb, _stream(dev))
    return out


def adapter_add(Y: torch.Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, index: torch.Tensor | None = None,
                alpha: torch.Tensor | None = None, out: torch.Tensor | None = None,
                ws: Workspace | None = None) -> torch.Tensor:
    """Y + alpha_a B_a (A_a x) for each token's adapter a: the adapters beside a
    projection computed elsewhere (linear_forward).  Y [n, r] is of X's type or
    float32; out may be Y."""
    _rows16(X, "X")
    _need(Y, "Y", None, 2, on_gpu=False)
    n, c = X.shape
    r = Y.shape[1]
    if Y.dtype not in (X.dtype, torch.float32):
        raise TypeError(f"Y must be float32 or {X.dtype}")
    _rows(Y, "Y", n, r)
    if A is None or B is None:
        raise TypeError("A and B must be torch.Tensor")
    m, rank = _adapters(A, B, index, alpha, X.dtype, n, r, c)
    _check_out(out, "out", n, r, Y.dtype)
    dev = _device(X, Y, A, B, index, alpha, out)
    buf, nb = _ws(ws, _lib.query("gptq_adapter_add_workspace_size", n, c, rank), dev)
    out = torch.empty((n, r), dtype=Y.dtype, device=dev) if out is None else out
    _lib.call("gptq_adapter_add", _ptr(X), _DT[X.dtype], n, c, _ld(X), _ptr(A), _ptr(B), m, rank, r, _ptr(index),
              _ptr(alpha), _ptr(Y), _DT[Y.dtype], _ld(Y), _ptr(out), _ld(out), _ptr(buf), nb, _stream(dev))
    return out


def adapter_backward(dY: torch.Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                     index: torch.Tensor | None = None, alpha: torch.Tensor | None = None, want_dX: bool = False,
                     base: torch.Tensor | None = None, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Gradients of the adapters from dY [n, r] and X [n, c].

    Returns {A fp32 [m, rank, c], B fp32 [m, r, rank], dX [n, c] or None}: sums
    over each adapter's own tokens, zero for one without tokens; with want_dX
    also the gradient for X through the adapters alone, added to `base` (X's
    type or float32, which is then dX's type) when that is given.  `out` may
    supply preallocated tensors with those keys; out["dX"] may be base."""
    _rows16(X, "X")
    _rows16(dY, "dY", X.shape[0], None, X.dtype)
    n, c = X.shape
    r = dY.shape[1]
    if A is None or B is None:
        raise TypeError("A and B must be torch.Tensor")
    m, rank = _adapters(A, B, index, alpha, X.dtype, n, r, c)
    o = dict(out or {})
    unknown = set(o) - {"A", "B", "dX"}
    if unknown:
        raise ValueError(f"unknown output names {sorted(unknown)}")
    for k, shape in (("A", (m, rank, c)), ("B", (m, r, rank))):
        if o.get(k) is not None:
            _need(o[k], f"out[{k!r}]", torch.float32, 3, on_gpu=False)
            if tuple(o[k].shape) != shape or not o[k].is_contiguous():
                raise ValueError(f"out[{k!r}] must be a contiguous float32 tensor of shape {shape}")
    dX = o.get("dX")
    want_dX = want_dX or dX is not None
    if base is not None and not want_dX:
        raise ValueError("base without want_dX")
    ot = base.dtype if base is not None else (dX.dtype if dX is not None else X.dtype)
    if ot not in (X.dtype, torch.float32):
        raise TypeError(f"base and dX must be float32 or {X.dtype}")
    for t, name in ((base, "base"), (dX, "out['dX']")):
        _check_out(t, name, n, c, ot)
    dev = _device(X, dY, A, B, index, alpha, base, *o.values())
    buf, nb = _ws(ws, _lib.query("gptq_adapter_backward_workspace_size", n, r, c, m, rank), dev)
    gA = o["A"] if o.get("A") is not None else torch.empty((m, rank, c), dtype=torch.float32, device=dev)
    gB = o["B"] if o.get("B") is not None else torch.empty((m, r, rank), dtype=torch.float32, device=dev)
    ldd = c
    if want_dX:
        if dX is None:
            dX = torch.empty_strided((n, c), (_ld(base) if base is not None else c, 1), dtype=ot, device=dev)
        ldd = _ld(dX)
        if base is not None and n > 1 and _ld(base) != ldd:
            raise ValueError("base and out['dX'] must have the same row stride")
    _lib.call("gptq_adapter_backward", _ptr(dY), _ld(dY), _ptr(X), _ld(X), _DT[X.dtype], n, r, c, _ptr(A), _ptr(B), m, rank,
              _ptr(index), _ptr(alpha), _ptr(gA), _ptr(gB), _ptr(base), _ptr(dX), _DT[ot], ldd, _ptr(buf), nb, _stream(dev))
    return {"A": gA, "B": gB, "dX": dX}
