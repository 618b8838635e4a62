"""Products whose contraction is split into parts, and 16-bit results from the
dequantized copy, against float64 with the weights rounded as the copy holds
them, so that a lost step, row or column of the contraction cannot hide in the
weights' own rounding.

Bounds (elementwise, eps = 2^-24; an addition on the matrix cores is counted as
off by a whole step, 2 eps of the sum of magnitudes):
  main product   a chain of K terms: K 2 eps sum |x W|; each weight is exact in
                 16 bits (fp32 results: held to 2^-25 in three bf16 terms; to
                 2^-22 and 2^-25 absolute in two fp16 ones)
  adapters       rank values (d + 32) 2 eps sum |A x|; at most six products per rank
                 go onto the sums, 6 rank 2 eps.  Split into two bf16 terms (16-bit
                 results) the values lose 2^-17, and beside fp16 factors, two terms
                 of 8 and 3 bits, the product of both second terms, 2^-16, is left
                 out; three terms (fp32 results) lose 2^-26 and 2^-25
and u |y| for the output's own rounding, u half a step of its type.
"""
import pytest
import torch

from test_gpu_adapter import DT, EPS, Layer, U, check, gq, make_adapters, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.empty_cache()


def product64(x, W, w_err, ad, down, up, out_dtype):
    """(value, bound) of x W^T + alpha (x down_a^T) up_a; W float64 [o, K], w_err its elementwise error or None."""
    x64, K = x.double(), x.shape[1]
    want, mag = x64 @ W.T, x64.abs() @ W.abs().T
    bound = torch.zeros_like(want) if w_err is None else x64.abs() @ w_err.T
    rank = 0
    if ad:
        m, rank = down.shape[0], down.shape[1]
        idx = ad["index"] if ad["index"] is not None else torch.zeros(len(x), dtype=torch.int32, device=x.device)
        split = 2.0 ** -24 if out_dtype == torch.float32 else 2.0 ** -17 + (2.0 ** -16 if x.dtype == torch.float16 else 0.0)
        for a in range(m):
            t = torch.nonzero(idx == a).flatten()
            f, d64, u64 = ad["alpha"][a].double(), down[a].double(), up[a].double()
            want[t] += f * ((x64[t] @ d64.T) @ u64)
            low = f * ((x64[t].abs() @ d64.abs().T) @ u64.abs())
            mag[t] += low
            bound[t] += ((K + 32) * 2 * EPS + split) * low
    return want, bound + (K + 6 * rank + 32) * 2 * EPS * mag


def copy_error(W, dt, out_dtype):
    """What is left of fp32 weights in the terms of the copy."""
    if out_dtype != torch.float32:
        return None
    return EPS * W.abs() + (2.0 ** -25 * W.abs() if dt == torch.bfloat16 else 2.0 ** -22 * W.abs() + 2.0 ** -25)


def backward_case(n, r, c, bits, gs, act, dt, out, low):
    print(f"\n[backward] n={n} {r}x{c} {bits}-bit g{gs} act={act} {dt}->{out} low={low}", flush=True)
    L = Layer(r, c, bits, gs, 60 + n + r, act)
    dY = normal((n, r), n + r, 0.1).to(DT[dt])
    ad = make_adapters(low[0], low[1], r, c, n, DT[dt], n + c, low[2]) if low else {}
    dX = gq().packed_linear_backward(dY, *L.args(), perm=L.perm, out_dtype=DT[out], **ad)
    torch.cuda.synchronize()
    W = L.W if out == "fp32" else L.W.float().to(DT[dt]).double()
    W = W.T.contiguous()
    check("dX", dX, *product64(dY, W, copy_error(W, DT[dt], DT[out]), ad, ad["B"].transpose(1, 2) if ad else None,
                               ad["A"] if ad else None, DT[out]))


def forward_case(n, r, c, bits, gs, act, dt, low):
    print(f"\n[forward] n={n} {r}x{c} {bits}-bit g{gs} act={act} {dt} low={low}", flush=True)
    L = Layer(r, c, bits, gs, 40 + n + r, act)
    X = normal((n, c), n + c).to(DT[dt])
    ad = make_adapters(low[0], low[1], r, c, n, DT[dt], n + r, low[2]) if low else {}
    Y = gq().packed_linear(X, *L.args(), perm=L.perm, **ad)
    torch.cuda.synchronize()
    check("Y", Y, *product64(X, L.W.float().to(DT[dt]).double(), None, ad, ad["A"] if ad else None,
                             ad["B"].transpose(1, 2) if ad else None, DT[dt]))


# n, r, c, bits, group, act-order, type, output, adapters.  Contractions that once left the last parts empty: 108 and 135
# steps (fp32, three terms), 90 (two terms), 131 and 129 steps (16-bit), one token in the last tile; and an even split.
BACKWARD = [
    (64, 2304, 2304, 4, 128, False, "bf16", "fp32", None),
    (64, 2880, 2880, 3, 96, True, "bf16", "fp32", None),
    (129, 2880, 256, 4, 32, False, "fp16", "fp32", (3, 24, "mixed")),
    (1, 8384, 1024, 4, 128, False, "fp16", "fp16", None),
    (65, 8256, 1024, 3, 64, True, "bf16", "bf16", (2, 16, "runs")),
    (129, 8570, 160, 4, 32, False, "bf16", "bf16", (5, 72, "mixed")),
    (40, 4096, 640, 4, 128, False, "fp16", "fp16", (40, 8, "runs")),
    # one part, the largest tiles over many steps
    (4000, 1030, 4096, 4, 128, False, "bf16", "bf16", (2, 64, "mixed")),
    (2085, 640, 4096, 3, 64, True, "fp16", "fp32", (4, 24, "runs")),
    (4096, 832, 4096, 4, 32, False, "bf16", "fp32", None),
]


@pytest.mark.parametrize("n,r,c,bits,gs,act,dt,out,low", BACKWARD)
def test_input_gradient_in_parts(n, r, c, bits, gs, act, dt, out, low):
    backward_case(n, r, c, bits, gs, act, dt, out, low)


# forward through the copy: 129 steps in 15 parts of 9, one row in the last tile of 128; 81 steps, adapters in order
FORWARD = [
    (1025, 129, 8256, 4, 128, False, "bf16", None),
    (1153, 1, 8320, 3, 64, True, "fp16", None),
    (1030, 200, 5184, 4, 96, False, "bf16", (3, 40, "mixed")),
    (1100, 257, 5120, 4, 128, True, "fp16", (2, 16, "runs")),
    # one part, the largest tiles over many steps
    (2085, 4096, 2048, 4, 128, False, "bf16", (5, 64, "runs")),
    (4096, 4096, 1056, 3, 32, True, "fp16", (3, 72, "mixed")),
    (4000, 4090, 1024, 4, -1, False, "bf16", (1, 128, "all")),
]


@pytest.mark.parametrize("n,r,c,bits,gs,act,dt,low", FORWARD)
def test_forward_in_parts(n, r, c, bits, gs, act, dt, low):
    forward_case(n, r, c, bits, gs, act, dt, low)
