"""The loss, its gradients and the adapters' update where they can go wrong: workspaces
that hold anything, tiles of 256 x 256 over many steps of the contraction, many pieces of the
vocabulary, heads past 2^31 elements, gradients of less than full rank and many steps.  Bounds as in
test_gpu_train.py unless said."""
import math

import pytest
import torch

from test_gpu_train import COEF, DT, EPS, U, Head, check, gq, matrices, normal, targets, update64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import post_weight_quantization_23_amd as q  # noqa: F401  (loads the library, raises if missing)
    yield
    torch.cuda.empty_cache()


def filled(byte, nbytes=1 << 22):
    """A workspace every byte of which is `byte` (0xFF: NaN in every type, -1)."""
    ws = gq().Workspace()
    ws.get(nbytes, torch.device("cuda", torch.cuda.current_device()))[0].fill_(byte)
    return ws


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_no_tokens_write_zeros_whatever_the_workspace_holds(dt):
    W = normal((300, 64), 1).to(DT[dt])
    X, y, v = W[:0], torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    for dloss in (None, v):
        got = gq().linear_cross_entropy_backward(X, W, y, v, dloss, want_dX=False, want_dW=True, ws=filled(0xFF))
        assert bool((got["W"] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [40, 200, 1300])
def test_results_do_not_depend_on_what_the_workspace_holds(n, dt):
    h = Head(n, 700, 200, DT[dt], 5, "prompt")
    A, B = matrices(2, 24, 100, 1, torch.float32), matrices(2, 24, 90, 2, torch.float32).transpose(1, 2).contiguous()

    def step(byte):
        ws = [filled(byte) for _ in range(3)]
        loss, lse = gq().linear_cross_entropy(h.X, h.W, h.y, ws=ws[0])
        g = gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, h.dloss, want_dW=True, ws=ws[1])
        u = gq().adapter_orthogonalize(A, B, ws=ws[2])
        return loss, lse, g["X"], g["W"], u["A"], u["B"]

    for a, b in zip(step(0xFF), step(0)):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


# ---------------------------------------------------------------- tiles of 256 x 256
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("mask", ["none", "prompt"])
@pytest.mark.parametrize("n,vocab,d", [(1025, 257, 136), (1100, 1031, 520), (2300, 700, 328), (1537, 513, 1160), (4097, 300, 192)])
def test_many_tokens_over_many_steps(n, vocab, d, mask, dt):
    """More than 1024 tokens, of which several tiles of 256 remain, over 3 to 19 steps of 64 values
    with and without a tail."""
    h = Head(n, vocab, d, DT[dt], 500 + n, mask).exact()
    loss, lse = gq().linear_cross_entropy(h.X, h.W, h.y)
    check("lse", lse, h.keep_lse, h.dlse)
    check("loss", loss, h.loss, h.dloss_bound)
    dloss = h.dloss * (4096 if dt == "fp16" else 1)   # results that are normal numbers
    (dX, bX), (dW, bW) = h.gradients(dloss)
    got = gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, dloss, want_dW=True)
    check("dX", got["X"], dX, bX)
    check("dW", got["W"], dW, bW)
    assert bool((got["X"][~h.there] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [5, 70])
def test_vocabulary_in_pieces_of_few_tokens(n, dt):
    """Pieces hold at most 2^21 entries, however few the tokens; targets on both sides of the border."""
    vocab = (1 << 21) + 300
    h = Head(n, vocab, 16, DT[dt], 600 + n)
    h.y[: n // 2] = (1 << 21) - n // 4 + torch.arange(n // 2, device="cuda")
    h.at = h.y
    h.exact()
    loss, lse = gq().linear_cross_entropy(h.X, h.W, h.y)
    check("lse", lse, h.keep_lse, h.dlse)
    check("loss", loss, h.loss, h.dloss_bound)
    dloss = h.dloss * (4096 if dt == "fp16" else 1)   # results that are normal numbers
    (dX, bX), (dW, bW) = h.gradients(dloss)
    got = gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, dloss, want_dW=True)
    check("dX", got["X"], dX, bX)
    check("dW", got["W"], dW, bW)


# ---------------------------------------------------------------- the target's entry
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("mask", ["none", "prompt"])
@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("n,vocab,d", [(1, 300, 8), (50, 4000, 72), (60, 9000, 136), (130, 700, 264), (700, 5003, 320), (1500, 20000, 72)])
def test_gradients_with_the_targets_entry_unrounded(n, vocab, d, same, mask, dt):
    """Of D the targets' entries enter dX in fp32 and dW in two 16-bit terms: u^2 |D| and the step of the second
    term instead of u |D|, 4 EPS |D| for the fp32 value itself.  same: a few entries are the targets of all tokens."""
    h = Head(n, vocab, d, DT[dt], 700 + n, mask)
    if same:
        h.y = torch.where(h.there, vocab // 2 + 37 * (torch.arange(n, device="cuda") % 5) % (vocab // 2), h.y)
        h.at = torch.where(h.there, h.y, 0)
    h.exact()
    dloss = h.dloss * (4096 if dt == "fp16" else 1)
    (dX, bX), (dW, bW) = h.gradients(dloss)
    g = torch.where(h.there, dloss.double(), 0)
    D = g * (torch.exp(h.z.gather(1, h.at.unsqueeze(1)).squeeze(1) - h.lse) - 1)
    less = (U[h.dt] - U[h.dt] ** 2 - 4 * EPS) * D.abs()
    bX -= less.unsqueeze(1) * h.W[h.at].double().abs()
    bW.index_add_(0, h.at, -less.unsqueeze(1) * h.X.double().nan_to_num().abs())
    lse = h.keep_lse.float()
    got = gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, dloss, want_dW=True)
    check("dX", got["X"], dX, bX)
    check("dW", got["W"], dW, bW)
    only = gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, dloss, want_dX=False, want_dW=True)
    assert torch.equal(only["W"], got["W"])


# ---------------------------------------------------------------- past 2^31 elements
@pytest.mark.parametrize("n", [3, 300])
def test_head_past_32_bits_entry_by_entry(n):
    """A head, and its gradient, of more than 2^31 elements.  Targets are dealt over the whole
    vocabulary, a third of them past 2^31 elements, and each token's hidden state leans to its
    target, so that another row of W in its place is a loss off by a unit or more.  Every bound is
    entry by entry, and far below the result itself."""
    vocab, d, dt = 270001, 8192, torch.bfloat16
    W = torch.empty((vocab, d), dtype=dt, device="cuda")
    parts = range(0, vocab, 30000)
    for a in parts:
        W[a:a + 30000] = normal((min(30000, vocab - a), d), 170 + a, 1 / math.sqrt(d)).to(dt)
    y = (torch.arange(n, device="cuda") * 7919 + vocab - 1 - 7919 * (n // 3)) % vocab
    X = (normal((n, d), 172) + 4 * W[y].float()).to(dt)
    dloss = 1 + normal((n,), 173).abs()
    loss, lse = gq().linear_cross_entropy(X, W, y)
    x, zy = X.double(), torch.arange(n, device="cuda")
    z = torch.cat([x @ W[a:a + 30000].double().T for a in parts], 1)
    dz = (d + 32) * 2 * EPS * torch.cat([x.abs() @ W[a:a + 30000].double().abs().T for a in parts], 1)
    want = torch.logsumexp(z, 1)
    arg = (z.max(1).values - z.min(1).values).clamp_max(90) + 2
    dlse = dz.max(1).values + arg * 4 * EPS + (64 + 3 * (16 + vocab / 4096)) * 2 * EPS + 4 * EPS * want.abs()
    check("lse", lse, want, dlse)
    bound = dlse + dz[zy, y] + 4 * EPS * (want.abs() + z[zy, y].abs())
    check("loss", loss, want - z[zy, y], bound)
    assert float(bound.max()) < 0.25       # another row's logit is about N(0, 1) where the target's is 4 higher
    got = gq().linear_cross_entropy_backward(X, W, y, want.float(), dloss, want_dW=True)
    p = torch.exp(z - want.unsqueeze(1))
    D = p.clone()
    D[zy, y] -= 1
    D *= dloss.double().unsqueeze(1)
    off = dloss.double().unsqueeze(1) * p * (dz + EPS * want.abs().unsqueeze(1) + ((z - want.unsqueeze(1)).abs() + 2) * 4 * EPS) + U[dt] * D.abs()
    dX, bX = torch.zeros_like(x), torch.zeros_like(x)
    for a in parts:
        w = W[a:a + 30000].double()
        dX += D[:, a:a + 30000] @ w
        bX += (off[:, a:a + 30000] + (vocab / 16 + 64) * 2 * EPS * D[:, a:a + 30000].abs()) @ w.abs()
    check("dX", got["X"], dX, bX)
    assert float(bX.norm()) < 0.3 * float(dX.norm())
    rows = torch.cat([y, (y + 1) % vocab, torch.arange(vocab - 300, vocab, device="cuda"), torch.arange(0, vocab, 997, device="cuda")])
    dW, bW = D[:, rows].T @ x, (off[:, rows] + (n + 64) * 2 * EPS * D[:, rows].abs()).T @ x.abs()
    check("dW", got["W"][rows], dW, bW)
    assert float(bW[:n].norm()) < 0.3 * float(dW[:n].norm())


# ---------------------------------------------------------------- updates of less than full rank, many steps
def deficient(kind, m, p, q, seed):
    if kind == "one row repeated":
        return normal((m, 1, q), seed).expand(m, p, q).contiguous()
    k = {"rank 1": 1, "rank 10": min(10, p - 1), "half rank": p // 2}[kind]
    return normal((m, p, k), seed) @ normal((m, k, q), seed + 1)


def single(values):
    """Coefficients as the C call takes them, in fp32 (2.0315 is then off by 5e-8 of it, a step of the result)."""
    return tuple(float(torch.tensor(v, dtype=torch.float32)) for v in values)


def steps_bound(p, n):
    """Spectral norm of what the update of a p x q matrix (q up to 1024) may be off after n of Muon's
    steps, in first order, and so of any of its entries, with e = 2^-53.
    S is off by at most 64 e (chains of at most 48 sums of products, the norm of |M| |M|^T being at most 1) and
    by (p + 8) e a step from its own products, of norms below 1.5.  An error of S grows by at most a^2 a
    step (the slope of s q(s)^2, largest at 0); q(S) is off by (|b| + 2 |c| 1.5) = 11 times it, which
    meets M of norm below 1.25, and grows by at most 4 a step from there, the largest slope
    of p(s) = a s + b s^3 + c s^5 up to p's largest value 1.2025.  S is formed again from M after at most 5
    steps: 2 * 11 * 1.25 * (64 + p + 8) e a^8 at the last of them, twice that for all of them.  The products
    of R and M are off by (p + 8) e a step, and grow likewise."""
    e, a = 2.0 ** -53, COEF[0]
    block = min(n, 5)
    once = 2 * 2 * 11 * 1.25 * (72 + p) * e * a ** (2 * (block - 1)) + block * (p + 8) * math.sqrt(p) * e * a ** block
    return sum(once * 4.0 ** max(0, n - block - k) for k in range(0, n, 5))


@pytest.mark.parametrize("kind", ["one row repeated", "rank 1", "rank 10", "half rank"])
@pytest.mark.parametrize("p,q", [(8, 512), (24, 100), (48, 200), (64, 1024), (80, 200), (112, 300), (128, 1000)])
def test_update_of_less_than_full_rank(p, q, kind):
    """Gradients of fewer tokens than ranks: S has eigenvalues of zero, whose rounding must not grow."""
    A = deficient(kind, 2, p, q, 11)
    B = deficient(kind, 2, p, q - 40, 12).transpose(1, 2).contiguous()
    for steps in (1, 2, 5, 6, 8, 10, 12, 16):
        got = gq().adapter_orthogonalize(A, B, steps=steps)
        tau = steps_bound(p, steps)
        for k, G in (("A", A), ("B", B.transpose(1, 2))):
            mine = got[k] if k == "A" else got[k].transpose(1, 2)
            want, _ = update64(G, steps, single(COEF), *single((1e-7,)))
            norm = float(torch.linalg.matrix_norm(mine.double(), 2).max())
            print(f"  {kind}, {steps} steps: norm {norm:.4f}, off {float((mine.double() - want).norm() / want.norm()):.2g}", flush=True)
            check(f"{k}, {steps} steps", mine, want, torch.full_like(want, tau))
            assert norm < 1.2025 + math.sqrt(p * q) * EPS + tau


@pytest.mark.parametrize("p,q", [(16, 300), (72, 300)])
@pytest.mark.parametrize("coef,steps", [((1.5, -0.5, 0.0), 16), ((2.0, -1.5, 0.5), 16), ((5.0, -20.0, 16.0), 3),
                                        ((-1.5, 0.5, 0.0), 7), ((1.0, 0.0, 0.0), 1), ((0.0, 0.0, 0.0), 2)])
def test_update_with_other_coefficients(p, q, coef, steps):
    """Any coefficients on matrices of full and of half rank.  In first order: every product is off by (p + 72) 2^-53 of
    its factors' norms, S's errors reach q(S) by |b| + 2 |c| and M by one more factor 2, and each later step multiplies an error by at
    most L, the largest slope of p, or of p's values over s, up to the largest value reached, found on a grid; S, formed from
    M again where L^(2 k) would pass 2^16, adds at most that."""
    a, b, c = coef
    top, L = 1.0, 1.0
    for _ in range(steps):
        s = torch.linspace(1e-3, top, 4000, dtype=torch.float64)
        L = max(L, float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max()), float((a + b * s ** 2 + c * s ** 4).abs().max()), abs(a))
        top = max(top, float((a * s + b * s ** 3 + c * s ** 5).abs().max()))
    tau = steps * (p + 72) * 2.0 ** -53 * max(top, 1.0) ** 3 * 4 * (1 + abs(b) + 2 * abs(c)) * min(L ** (2 * steps), 2.0 ** 16) * L ** steps
    for G in (matrices(2, p, q, 3, torch.float32), deficient("half rank", 2, p, q, 5)):
        got = gq().adapter_orthogonalize(A=G, steps=steps, coefficients=coef)["A"]
        want, _ = update64(G, steps, single(coef), *single((1e-7,)))
        assert tau < 0.1 * float(want.abs().max()) or float(want.abs().max()) == 0
        check("update", got, want, torch.full_like(want, tau))


@pytest.mark.parametrize("p", [16, 72])
@pytest.mark.parametrize("a,steps", [(300.0, 3), (1e4, 2), (1e-3, 4)])
def test_update_of_a_line(p, a, steps):
    """b = c = 0: M_0 times a^steps, each product off by (p + 72) 2^-53 of its factors' norms."""
    G = matrices(2, p, 300, 3, torch.float32)
    got = gq().adapter_orthogonalize(A=G, steps=steps, coefficients=(a, 0.0, 0.0))["A"]
    a, eps = single((a, 1e-7))
    M = G.double() / (G.double().square().sum((1, 2), keepdim=True).sqrt() + eps)
    check("update", got, a ** steps * M, torch.full_like(M, steps * (p + 72) * 2.0 ** -53 * 4 * a ** steps))


@pytest.mark.parametrize("gt,ot", [("fp32", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("rank,c,r", [(72, 40, 500), (72, 200, 80), (16, 8, 300), (40, 64, 33)])
def test_update_of_many_steps_of_both_factors(rank, c, r, gt, ot):
    """Matrices of other numbers of tile rows beside each other, lying and standing, in all types."""
    A, B = normal((3, rank, c), 31).to(DT[gt]), normal((3, r, 2), 32) @ normal((3, 2, rank), 33)
    B = B.to(DT[gt])
    got = gq().adapter_orthogonalize(A, B, steps=12, out_dtype=DT[ot])
    for k, G in (("A", A), ("B", B)):
        flip = G.shape[1] > G.shape[2]
        want, _ = update64(G.transpose(1, 2) if flip else G, 12, single(COEF), *single((1e-7,)))
        check(k, got[k].transpose(1, 2) if flip else got[k], want, torch.full_like(want, steps_bound(min(G.shape[1:]), 12)))


@pytest.mark.parametrize("p", [24, 96])
def test_many_steps_in_a_graph(p):
    """S formed again within a captured call, replayed on other matrices with eager calls between."""
    G = deficient("rank 1", 3, p, 400, 41)
    ws, out = gq().Workspace(), {"A": torch.empty_like(G)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gq().adapter_orthogonalize(A=G, steps=16, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq().adapter_orthogonalize(A=G, steps=16, out=out, ws=ws)
    for seed, kind in enumerate(("half rank", "one row repeated", "rank 1")):
        G.copy_(deficient(kind, 3, p, 400, 50 + seed))
        want = gq().adapter_orthogonalize(A=G, steps=16)["A"]
        out["A"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["A"], want), kind


@pytest.mark.parametrize("p", [16, 72])
def test_many_steps_of_far_sizes_zeros_and_what_is_not_finite(p):
    G = matrices(5, p, 200, 5, torch.float32)
    far = G * torch.tensor([1e-30, 1e30, 1.0, 1.0, 1.0], device="cuda").view(5, 1, 1)
    far[2], far[3, 4, 5] = 0.0, float("inf")
    got = gq().adapter_orthogonalize(B=far.transpose(1, 2).contiguous(), eps=0.0, steps=12)["B"].transpose(1, 2)
    tau = torch.full((1, p, 200), steps_bound(p, 12), dtype=torch.float64, device="cuda")
    for i in (0, 1, 4):
        check(f"matrix {i}", got[i:i + 1], update64(far[i:i + 1], 12, single(COEF), 0.0)[0], tau)
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[3]).all())
    assert bool((gq().adapter_orthogonalize(A=far[2:3], steps=12)["A"] == 0).all())
