"""Batches whose outputs pass 2^31 elements, on some of their rows against float64
(bounds as in test_gpu_adapter_parts.py), the adapters' gradients over all of them."""
import pytest
import torch

from test_gpu_adapter import EPS, Layer, check, gq, low64, make_adapters, normal
from test_gpu_adapter_parts import copy_error, product64

pytestmark = pytest.mark.gpu

N, R, C = 262144, 11008, 32


@pytest.fixture(scope="module")
def batch():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    L = Layer(R, C, 4, -1, 3, False)
    ad = make_adapters(4, 8, R, C, N, torch.bfloat16, 7)
    rows = torch.cat([torch.arange(40), torch.randint(0, N, (300,), generator=torch.Generator().manual_seed(1)),
                      torch.arange(N - 40, N)]).cuda()
    yield L, ad, {**ad, "index": ad["index"][rows].contiguous()}, rows
    torch.cuda.empty_cache()


def test_forward_and_adapters_of_a_large_batch(batch):
    L, ad, some, rows = batch
    X = normal((N, C), 1).bfloat16()
    up = ad["B"].transpose(1, 2)
    for out in (torch.bfloat16, torch.float32):
        print(f"\n[forward] {N} tokens {R}x{C} -> {out}", flush=True)
        Y = gq().packed_linear(X, *L.args(), **ad, out_dtype=out)
        torch.cuda.synchronize()
        W = L.W.float().bfloat16().double() if out == torch.bfloat16 else L.W
        want, bound = product64(X[rows], W, None, some, ad["A"], up, out)
        # fp32 results of unrounded weights: the codes' whole numbers carry larger sums
        check("Y", Y[rows], want, bound + (128 + 32) * 2 * EPS * (X[rows].double().abs() @ L.mag.T))
    print("[adapter_add] in place", flush=True)
    before = Y[rows].clone()
    gq().adapter_add(Y, X, **ad, out=Y)
    v, b = low64(some, X[rows], ad["A"], up)
    check("add", Y[rows], before.double() + v, b + EPS * (before.double().abs() + v.abs()))


def test_gradients_of_a_large_batch(batch):
    L, ad, some, rows = batch
    X, dY = normal((N, C), 2).bfloat16(), torch.empty((N, R), dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, N // 8):
        dY[i:i + N // 8] = normal((N // 8, R), 10 + i, 0.1)
    print(f"\n[backward] {N} tokens {R}x{C}", flush=True)
    dX = gq().packed_linear_backward(dY, *L.args(), **ad)
    torch.cuda.synchronize()
    W = L.W.float().bfloat16().double().T.contiguous()
    check("dX", dX[rows], *product64(dY[rows], W, None, some, ad["B"].transpose(1, 2), ad["A"], torch.bfloat16))
    print("[adapter_backward]", flush=True)
    g = gq().adapter_backward(dY, X, **ad)
    torch.cuda.synchronize()
    for a in range(4):
        t = torch.nonzero(ad["index"] == a).flatten()
        A, B, f = ad["A"][a].double(), ad["B"][a].double(), ad["alpha"][a].double()
        want = [torch.zeros((8, C), dtype=torch.float64, device="cuda"), torch.zeros((R, 8), dtype=torch.float64, device="cuda")]
        mag = [torch.zeros_like(w) for w in want]
        for part in t.split(16384):
            y, x = dY[part].double(), X[part].double()
            want[0] += f * (y @ B).T @ x
            mag[0] += f * (y.abs() @ B.abs()).T @ x.abs()
            want[1] += f * y.T @ (x @ A.T)
            mag[1] += f * y.abs().T @ (x.abs() @ A.abs().T)
        chain = (3 * len(t) + 64) * 2 * EPS + 2.0 ** -24
        check(f"gA[{a}]", g["A"][a], want[0], (chain + (R + 32) * 2 * EPS) * mag[0])
        check(f"gB[{a}]", g["B"][a], want[1], (chain + (C + 32) * 2 * EPS) * mag[1])
