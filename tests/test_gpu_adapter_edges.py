"""Ends of the ranges of the packed products and adapters, through the Python calls."""
import pytest
import torch

from test_gpu_adapter import Layer, gq, make_adapters, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [0, 5, 1100])
def test_a_layer_without_rows(n):
    c = 64
    X = normal((n, c), 1).bfloat16()
    ad = make_adapters(2, 8, 0, c, n, torch.bfloat16, 3)
    layer = (torch.empty((0, c // 8), dtype=torch.uint32, device="cuda"), torch.empty((0, 1), device="cuda"),
             torch.empty((0, 1), dtype=torch.int32, device="cuda"), 4, -1)
    for low in ({}, ad):
        assert gq().packed_linear(X, *layer, **low).shape == (n, 0)
    assert gq().adapter_add(torch.empty((n, 0), dtype=torch.bfloat16, device="cuda"), X, **ad).shape == (n, 0)


def wide(x, left, right, fill=7.0):
    """x inside a matrix of longer rows at an odd place, and that matrix."""
    w = torch.full((x.shape[0] + 2, x.shape[1] + left + right), fill, dtype=x.dtype, device="cuda")
    view = w[1:-1, left:left + x.shape[1]]
    view.copy_(x)
    return view, w


def beside(view, w, fill=7.0):
    """What lies beside a view of wide() is as it was."""
    view.fill_(fill)
    return bool((w == fill).all())


# few tokens, tiles, the copy, parts; odd row lengths
SIZES = [(3, 45, 96, 2, 8), (64, 33, 416, 64, 24), (130, 301, 160, 3, 72), (600, 515, 544, 4, 16), (1030, 131, 1056, 2, 40),
         (1100, 1033, 96, 5, 16), (1025, 77, 5216, 3, 8)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,r,c,m,rank", SIZES)
def test_rows_anywhere_give_the_same_bits(n, r, c, m, rank, dt):
    """Strided, odd-aligned matrices against dense ones, and nothing written beside the results."""
    L = Layer(r, c, 3, 32, n + r, True)
    ad = make_adapters(m, rank, r, c, n, dt, 3)
    ad["index"][::7] = torch.tensor([2 ** 31 - 1, -2 ** 31] * n, dtype=torch.int32, device="cuda")[:len(ad["index"][::7])]
    X, dY, Y = normal((n, c), 1).to(dt), normal((n, r), 2, 0.1).to(dt), normal((n, r), 3).to(dt)
    Xo, dYo = wide(X, 3, 6)[0], wide(dY, 5, 2)[0]
    for out in (dt, torch.float32):
        to, tw = wide(torch.zeros((n, r), dtype=out, device="cuda"), 1, 4)
        gq().packed_linear(Xo, *L.args(), perm=L.perm, **ad, out=to)
        assert torch.equal(to, gq().packed_linear(X, *L.args(), perm=L.perm, **ad, out_dtype=out)) and beside(to, tw)
        do, dw = wide(torch.zeros((n, c), dtype=out, device="cuda"), 3, 2)
        gq().packed_linear_backward(dYo, *L.args(), perm=L.perm, **ad, out=do)
        assert torch.equal(do, gq().packed_linear_backward(dY, *L.args(), perm=L.perm, **ad, out_dtype=out)) and beside(do, dw)
        bo, bw = wide(normal((n, c), 4).to(out), 3, 2)
        want = gq().adapter_backward(dY, X, **ad, base=bo.clone().contiguous(), want_dX=True)
        got = gq().adapter_backward(dYo, Xo, **ad, base=bo, out={"dX": bo})
        assert all(torch.equal(got[k], want[k]) for k in ("A", "B", "dX")) and beside(bo, bw)
        yo, yw = wide(Y.to(out), 1, 2)
        gq().adapter_add(yo, Xo, **ad, out=yo)
        assert torch.equal(yo, gq().adapter_add(Y.to(out), X, **ad)) and beside(yo, yw)


def test_aligned_strided_rows_without_a_permutation():
    for n, r, c in ((40, 200, 512), (500, 300, 512), (1200, 300, 512), (1200, 300, 544)):
        L = Layer(r, c, 4, 64, n, False)
        X = normal((n, c), 1).half()
        Xo = torch.zeros((n, c + 24), dtype=torch.float16, device="cuda")[:, 8:8 + c]
        Xo.copy_(X)
        for out in (torch.float16, torch.float32):
            assert torch.equal(gq().packed_linear(Xo, *L.args(), out_dtype=out), gq().packed_linear(X, *L.args(), out_dtype=out))


@pytest.mark.parametrize("n", [40, 700, 1100])
def test_what_is_not_finite_stays_so(n):
    """An infinity or NaN among a request's own tokens or factors: infinities or NaN where it enters, and nothing beyond."""
    r, c, m, rank = 72, 160, 3, 16
    L = Layer(r, c, 4, 32, 9, False)
    ad = make_adapters(m, rank, r, c, n, torch.bfloat16, 3, "runs")
    X, dY, Y = normal((n, c), 1).bfloat16(), normal((n, r), 2).bfloat16(), normal((n, r), 4).bfloat16()
    t = n // 2                               # a token of adapter 1
    for bad in (float("inf"), float("nan")):
        X2, dY2, A2 = X.clone(), dY.clone(), ad["A"].clone()
        X2[t, 5], dY2[t, 7], A2[1, 2, 9] = bad, bad, bad
        others = torch.arange(n, device="cuda") != t
        for out in (torch.bfloat16, torch.float32):
            for f, x, x2 in ((lambda v, **k: gq().packed_linear(v, *L.args(), **k, out_dtype=out), X, X2),
                             (lambda v, **k: gq().packed_linear_backward(v, *L.args(), **k, out_dtype=out), dY, dY2),
                             (lambda v, **k: gq().adapter_add(Y.to(out), v, **k), X, X2)):
                got, want = f(x2, **ad), f(x, **ad)
                assert not torch.isfinite(got[t]).any() and torch.equal(got[others], want[others])
            got = gq().packed_linear(X, *L.args(), **{**ad, "A": A2}, out_dtype=out)
            assert bool((torch.isfinite(got).any(1) == (ad["index"] != 1)).all())
        g, w = gq().adapter_backward(dY, X2, **ad), gq().adapter_backward(dY, X, **ad)
        assert not torch.isfinite(g["A"][1, :, 5]).any() and not torch.isfinite(g["B"][1]).any()
        keep = torch.arange(c, device="cuda") != 5
        assert torch.equal(g["A"][1][:, keep], w["A"][1][:, keep])
        assert all(torch.equal(g[k][a], w[k][a]) for k in "AB" for a in (0, 2))
