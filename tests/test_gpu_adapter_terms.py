"""Every weight, factor and term by itself: tokens with a single entry, so that a
result is one product (or one per 16-bit term) and no sum hides what a kernel
loses.

What is exact: the product of two 16-bit values (at most 22 bits) and of a code
less its zero with one (at most 18) in fp32, and adding zeros.  So
  forward, unrounded weights   one rounding, of scale (q - z) x
  through the 16-bit copy      the copied weight times the entry, exact
and the result's own rounding: equal bit for bit.  Where a value of 24 bits goes
into the matrix cores in terms:
  weights of fp32 gradients    rounded once, EPS; three bf16 terms hold it to 2^-26,
                               two of fp16 to 2^-22 and 2^-25 absolute; two or
                               three additions, each off by a step, 2 EPS
  rank values                  two roundings (times alpha), 2 EPS; three terms lose
                               2^-26 and beside fp16's two 2^-25, two terms 2^-17 and
                               2^-16; at most six products, 2 EPS each
"""
import math

import pytest
import torch

from test_gpu_adapter import DT, EPS, U, Layer, gq, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.empty_cache()


def single(n, d, dt, seed, distinct=False):
    """[n, d] with one entry per row, and its columns."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    at = torch.randperm(d, generator=g, device="cuda")
    at = at[:n] if distinct else at.repeat(-(-n // d))[:n]          # every column in turn
    x = torch.zeros((n, d), dtype=dt, device="cuda")
    v = normal((n,), seed + 1)
    x[torch.arange(n, device="cuda"), at] = torch.where(v.abs() < 0.1, torch.full_like(v, 0.75), v).to(dt)
    return x, at


def entry(x, at):
    return x[torch.arange(len(x), device="cuda"), at].double().unsqueeze(1)


def same(name, got, want):
    bad = int((got != want).sum())
    print(f"  {name}: {bad} of {got.numel()} differ", flush=True)
    assert got.dtype == want.dtype and bad == 0, name


def near(name, got, want, bound):
    err, lim = (got.double() - want).abs(), bound + U[got.dtype] * want.abs()
    if got.dtype == torch.float16:
        lim += 2.0 ** -25       # fp16 has no exponent below 2^-14: its steps there are 2^-24, half of one is 2^-25
    ratio = err / lim.clamp_min(1e-300)
    worst = float(ratio.max())
    print(f"  {name}: max err / bound {worst:.3g} at {float(want.flatten()[ratio.argmax()]):.3g}", flush=True)
    assert bool((err <= lim).all()), (name, worst)


# n, r, c, bits, group, act-order, type, output
FORWARD = [
    (1, 333, 1056, 4, 128, False, "bf16", "fp32"), (16, 200, 416, 3, 96, False, "fp16", "fp16"),
    (40, 8003, 256, 4, 64, True, "bf16", "bf16"), (61, 12007, 160, 3, 32, False, "fp16", "fp32"),
    (33, 4100, 4128, 4, -1, False, "bf16", "fp32"), (64, 4096, 2048, 3, 128, True, "bf16", "bf16"),
    (300, 96, 768, 4, 32, True, "fp16", "fp32"),
    (520, 4100, 4128, 4, 128, False, "bf16", "bf16"), (517, 4096, 2048, 3, 64, True, "bf16", "fp32"),
    (700, 6001, 2048, 4, 32, False, "fp16", "fp16"), (1023, 2048, 1024, 3, -1, False, "bf16", "bf16"),
    (1100, 130, 1024, 3, 64, True, "bf16", "fp32"), (4100, 700, 4096, 4, 128, False, "fp16", "fp32"),
    # through the copy: its tile shapes over many steps, parts, and 1024 tokens
    (2085, 4096, 4096, 4, 128, False, "bf16", "bf16"), (4096, 4096, 2048, 3, 64, True, "fp16", "fp16"),
    (1024, 4096, 1056, 4, 32, False, "bf16", "bf16"), (1050, 2900, 1024, 3, -1, False, "fp16", "fp16"),
    (1100, 1500, 2080, 4, 96, True, "bf16", "bf16"), (8300, 129, 8256, 4, 128, False, "bf16", "bf16"),
    (1025, 65, 5216, 3, 128, False, "fp16", "fp16"), (6000, 5504, 640, 4, 128, False, "bf16", "bf16"),
]


@pytest.mark.parametrize("n,r,c,bits,gs,act,dt,out", FORWARD)
def test_forward_holds_every_weight(n, r, c, bits, gs, act, dt, out):
    print(f"\n[forward] n={n} {r}x{c} {bits}-bit g{gs} act={act} {dt}->{out}", flush=True)
    L = Layer(r, c, bits, gs, 40 + n + r, act)
    X, at = single(n, c, DT[dt], n + c)
    Y = gq().packed_linear(X, *L.args(), perm=L.perm, out_dtype=DT[out])
    torch.cuda.synchronize()
    W = L.W.float().to(DT[dt]).double() if out != "fp32" and n >= 1024 else L.W
    same("Y", Y, (W.T[at] * entry(X, at)).float().to(DT[out]))


BACKWARD = [
    (3, 17, 96, 3, 32, True, "fp16", "fp16"), (70, 333, 416, 4, 96, False, "bf16", "bf16"),
    (2085, 1024, 4096, 4, 128, False, "bf16", "bf16"), (4096, 640, 4096, 3, 64, True, "fp16", "fp16"),
    (512, 4096, 2752, 3, 128, True, "bf16", "bf16"), (64, 8640, 320, 4, 32, False, "fp16", "fp16"),
    (3, 17, 96, 3, 32, True, "fp16", "fp32"), (70, 333, 416, 4, 96, False, "bf16", "fp32"),
    (2900, 2880, 256, 4, 128, False, "bf16", "fp32"), (2304, 2304, 1024, 3, 64, True, "bf16", "fp32"),
    (2085, 1024, 4096, 4, 32, False, "fp16", "fp32"), (129, 2880, 160, 4, -1, False, "fp16", "fp32"),
]


@pytest.mark.parametrize("n,r,c,bits,gs,act,dt,out", BACKWARD)
def test_input_gradient_holds_every_weight(n, r, c, bits, gs, act, dt, out):
    print(f"\n[backward] n={n} {r}x{c} {bits}-bit g{gs} act={act} {dt}->{out}", flush=True)
    L = Layer(r, c, bits, gs, 60 + n + r, act)
    dY, at = single(n, r, DT[dt], n + r)
    dX = gq().packed_linear_backward(dY, *L.args(), perm=L.perm, out_dtype=DT[out])
    torch.cuda.synchronize()
    d = entry(dY, at)
    if out != "fp32":
        same("dX", dX, (L.W.float().to(DT[dt]).double()[at] * d).float().to(DT[out]))
    elif dt == "bf16":
        near("dX", dX, L.W[at] * d, (EPS + 2.0 ** -26 + 6 * EPS) * (L.W[at] * d).abs())
    else:
        near("dX", dX, L.W[at] * d, (EPS + 2.0 ** -22 + 4 * EPS) * (L.W[at] * d).abs() + 2.0 ** -25 * d.abs())


def sparse_rows(m, o, rank, dt, seed):
    """[m, o, rank] with one entry in every row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    p = torch.randint(0, rank, (m, o, 1), generator=g, device="cuda")
    return torch.zeros((m, o, rank), dtype=dt, device="cuda").scatter_(2, p, normal((m, o, 1), seed + 1, 0.5).to(dt))


def low_terms(x, at, index, alpha, down, up, out_dtype):
    """(value, bound) of alpha (x down^T) up^T, up [m, o, rank] with single entries."""
    a = index.clamp(0, len(alpha) - 1).long()
    s = alpha[a].double().unsqueeze(1) * down.double()[a, :, at] * entry(x, at)              # [n, rank]
    v = torch.empty((len(x), up.shape[1]), dtype=torch.float64, device="cuda")
    for k in range(len(alpha)):
        t = torch.nonzero(a == k).flatten()
        v[t] = s[t] @ up[k].double().T
    v = torch.where(((index >= 0) & (index < len(alpha))).unsqueeze(1), v, torch.zeros_like(v))
    f16 = x.dtype == torch.float16
    lost = 2.0 ** -26 + (2.0 ** -25 if f16 else 0) if out_dtype == torch.float32 else 2.0 ** -17 + (2.0 ** -16 if f16 else 0)
    return v, (2 * EPS + lost + 12 * EPS) * v.abs()


def adapters(m, rank, n, kind, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if kind == "mixed":
        index = torch.randint(-1, m + 1, (n,), generator=g, device="cuda").to(torch.int32)
    else:
        index = (torch.arange(n, device="cuda") * m // n).to(torch.int32)
    return index, 0.5 + normal((m,), seed + 2).abs()


# n, r, c, type, m, rank, kind: the few-token kernels, tiles shared and by order, ranks past 64, parts
LOW = [
    (5, 300, 96, "bf16", 3, 16, "mixed"), (40, 257, 160, "fp16", 40, 64, "runs"), (60, 90, 96, "bf16", 4, 128, "mixed"),
    (130, 333, 256, "fp16", 3, 8, "mixed"), (150, 200, 64, "bf16", 50, 40, "runs"),
    (700, 300, 352, "bf16", 5, 72, "runs"), (1100, 530, 96, "fp16", 4, 24, "mixed"), (1500, 264, 416, "bf16", 6, 128, "runs"),
    (2085, 4096, 64, "bf16", 5, 64, "runs"), (1100, 200, 2080, "fp16", 1, 32, "runs"),
]


@pytest.mark.parametrize("n,r,c,dt,m,rank,kind", LOW)
def test_adapters_hold_every_term(n, r, c, dt, m, rank, kind):
    print(f"\n[adapters] n={n} {c}->{r} {dt} m={m} rank={rank} {kind}", flush=True)
    dt = DT[dt]
    index, alpha = adapters(m, rank, n, kind, n + r)
    X, at = single(n, c, dt, n)
    dY, aty = single(n, r, dt, n + 1)
    A, B = normal((m, rank, c), 5).to(dt), sparse_rows(m, r, rank, dt, 6)
    low = dict(index=index, alpha=alpha)
    for out in (dt, torch.float32):
        Y = normal((n, r), 7, 0.1).to(out)
        v, b = low_terms(X, at, index, alpha, A, B, out)
        near(f"add {out}", gq().adapter_add(Y, X, A, B, **low), Y.double() + v, b + 2 * EPS * (Y.double().abs() + v.abs()))
        L = Layer(r, c, 4, 32, n + c, True)
        W = L.W.float().to(dt).double() if out == dt and n >= 1024 else L.W
        main = W.T[at] * entry(X, at)
        near(f"forward {out}", gq().packed_linear(X, *L.args(), perm=L.perm, A=A, B=B, **low, out_dtype=out), main + v,
             b + 16 * EPS * (main.abs() + v.abs()))
    # the gradient's factors the other way round: rank values through B, one entry in every column of A
    B2, A2 = normal((m, r, rank), 8).to(dt), sparse_rows(m, c, rank, dt, 9).transpose(1, 2).contiguous()
    for out in (dt, torch.float32):
        base = normal((n, c), 11, 0.1).to(out)
        v, b = low_terms(dY, aty, index, alpha, B2.transpose(1, 2), A2.transpose(1, 2), out)
        got = gq().adapter_backward(dY, X, A2, B2, **low, base=base, want_dX=True)
        near(f"dX {out}", got["dX"], base.double() + v, b + 2 * EPS * (base.double().abs() + v.abs()))
        W = L.W.float().to(dt).double() if out == dt else L.W
        main, d = W[aty] * entry(dY, aty), entry(dY, aty).abs()
        lost = 0 if out == dt else (7 * EPS + 2.0 ** -22) * main.abs() + 2.0 ** -25 * d
        near(f"input gradient {out}", gq().packed_linear_backward(dY, *L.args(), perm=L.perm, A=A2, B=B2, **low, out_dtype=out),
             main + v, b + lost + 18 * EPS * (main.abs() + v.abs()))


# tokens of distinct rows and columns: every value of a gradient has one product or none
GRAD = [(1, 9, 16, "bf16", 1, 8, "runs"), (60, 130, 96, "fp16", 7, 24, "mixed"), (90, 200, 104, "bf16", 1, 128, "runs"),
        (700, 777, 800, "bf16", 3, 16, "mixed"), (1500, 1601, 1504, "fp16", 4, 72, "runs"), (1500, 1504, 1600, "bf16", 9, 40, "mixed"),
        (4000, 4096, 4104, "bf16", 1, 8, "runs"), (300, 320, 304, "fp16", 150, 8, "mixed")]


@pytest.mark.parametrize("n,r,c,dt,m,rank,kind", GRAD)
def test_gradients_hold_every_term(n, r, c, dt, m, rank, kind):
    print(f"\n[gradients] n={n} {c}->{r} {dt} m={m} rank={rank} {kind}", flush=True)
    dt = DT[dt]
    index, alpha = adapters(m, rank, n, kind, n + r)
    X, at = single(n, c, dt, n, distinct=True)
    dY, aty = single(n, r, dt, n + 1, distinct=True)
    A, B = normal((m, rank, c), 5).to(dt), normal((m, r, rank), 6).to(dt)
    got = gq().adapter_backward(dY, X, A, B, index=index, alpha=alpha)
    torch.cuda.synchronize()
    gA, gB = torch.zeros((m, rank, c), dtype=torch.float64, device="cuda"), torch.zeros((m, r, rank), dtype=torch.float64, device="cuda")
    t = torch.nonzero((index >= 0) & (index < m)).flatten()
    a, x, y = index[t].long(), entry(X, at)[t], entry(dY, aty)[t]
    f = alpha[a].double().unsqueeze(1)
    gA[a, :, at[t]] = f * y * B.double()[a, aty[t]] * x
    gB[a, aty[t]] = f * y * (A.double()[a, :, at[t]] * x)
    lost = 2 * EPS + 2.0 ** -26 + (2.0 ** -25 if dt == torch.float16 else 0) + 12 * EPS
    near("gA", got["A"], gA, lost * gA.abs())
    near("gB", got["B"], gB, lost * gB.abs())


@pytest.mark.parametrize("n,r,c,bits,gs,dt", [(1, 40, 416, 4, 32, "bf16"), (40, 70, 416, 3, 96, "fp16"), (300, 130, 1024, 4, 64, "bf16"),
                                              (1100, 130, 1024, 3, 128, "fp16"), (1100, 130, 1024, 4, 32, "bf16")])
def test_zeros_far_from_the_codes(n, r, c, bits, gs, dt):
    """Zeros of -1000 .. 1000: code less zero has 10 bits, its product with an entry 21, still exact."""
    L = Layer(r, c, bits, gs, n + r, False)
    g = torch.Generator().manual_seed(n)
    zeros = torch.randint(-1000, 1001, L.zeros.shape, generator=g, dtype=torch.int32).cuda()
    zeros[:2], zeros[2:4] = -1000, 1000
    of = torch.arange(c, device="cuda") // gs
    L.W = L.W + L.scales.double()[:, of] * (L.zeros - zeros).double()[:, of]       # s (q - z): 35 bits, exact in float64
    L.zeros = zeros
    X, at = single(n, c, DT[dt], n + c)
    dY, aty = single(n, r, DT[dt], n + r)
    for out in (DT[dt], torch.float32):
        W = L.W.float().to(DT[dt]).double() if out != torch.float32 and n >= 1024 else L.W
        same(f"Y {out}", gq().packed_linear(X, *L.args(), out_dtype=out), (W.T[at] * entry(X, at)).float().to(out))
    W = L.W.float().to(DT[dt]).double()
    same("dX", gq().packed_linear_backward(dY, *L.args()), (W[aty] * entry(dY, aty)).float().to(DT[dt]))


def test_the_longest_contractions():
    """Columns past the tiles' 2^22 - 128 (the few-token kernel takes any number of tokens then), and 2^22 - 64 rows."""
    L = Layer(17, 1 << 22, 4, 128, 5, False)
    X, at = single(65, 1 << 22, torch.bfloat16, 3)
    at[::3] = (1 << 22) - 1 - torch.arange(22, device="cuda")
    X = torch.zeros_like(X).scatter_(1, at.unsqueeze(1), normal((65, 1), 4).bfloat16())
    for out in (torch.bfloat16, torch.float32):
        same(f"Y {out}", gq().packed_linear(X, *L.args(), out_dtype=out), (L.W.T[at] * entry(X, at)).float().to(out))
    dY, aty = single(65, 17, torch.bfloat16, 6)
    W = L.W.float().bfloat16().double()
    same("dX", gq().packed_linear_backward(dY, *L.args()), (W[aty] * entry(dY, aty)).float().bfloat16())
    del L, X, W
    r = (1 << 22) - 64
    L = Layer(r, 32, 4, -1, 7, False)
    dY, aty = single(130, r, torch.bfloat16, 8)
    aty[::2] = r - 1 - torch.arange(65, device="cuda")
    dY = torch.zeros_like(dY).scatter_(1, aty.unsqueeze(1), normal((130, 1), 9).bfloat16())
    W, d = L.W.float().bfloat16().double(), entry(dY, aty)
    same("dX", gq().packed_linear_backward(dY, *L.args()), (W[aty] * d).float().bfloat16())
    near("dX fp32", gq().packed_linear_backward(dY, *L.args(), out_dtype=torch.float32), L.W[aty] * d,
         (EPS + 2.0 ** -26 + 6 * EPS) * (L.W[aty] * d).abs())
    X, at = single(40, 32, torch.bfloat16, 10)
    same("Y", gq().packed_linear(X, *L.args()), (L.W.T[at] * entry(X, at)).float().bfloat16())
