"""The loss, its gradients and the adapters' update as a program uses them: a training
step through a packed layer, HIP graphs, streams of their own, and matrices past 2^31
elements.  Bounds as in test_gpu_train.py."""
import math

import pytest
import torch

from synth import inputs as S
from test_gpu_train import COEF, DT, EPS, U, Head, check, gq, matrices, normal, targets, update64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import post_weight_quantization_23_amd as q  # noqa: F401  (loads the library, raises if missing)
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_training_step(dt):
    """Packed layer with adapters -> loss -> its gradient -> adapters' gradients -> their update,
    each stage against float64 on what the program had before it; errors of the loss's gradient
    carried through to the adapters' by magnitudes.  adapter_backward's own: chains over the tokens
    ((n + 64) 2 EPS) and rank values of (r + 32) or (c + 32) terms and two 2^-15."""
    dt, n, c, r, vocab, m, rank = DT[dt], 300, 256, 384, 1500, 3, 16
    codes, scales, zeros, _ = S.packed_layer_host(r, c, 4, 128, 5, False)
    dev = "cuda"
    words = gq().pack(torch.from_numpy(codes).to(dev), 4)
    scales, zeros = torch.from_numpy(scales).to(dev), torch.from_numpy(zeros).to(dev)
    A, B = normal((m, rank, c), 1, 1 / math.sqrt(c)).to(dt), normal((m, r, rank), 2, 0.3).to(dt)
    index = (torch.arange(n, device=dev) * (m + 1) // n).to(torch.int32)        # the last requests have no adapter
    alpha = 0.5 + normal((m,), 3).abs()
    X = normal((n, c), 4).to(dt)
    low = dict(A=A, B=B, index=index, alpha=alpha)
    H = gq().packed_linear(X, words, scales, zeros, 4, 128, **low)
    h = Head(n, vocab, r, dt, 6, "prompt")
    h.X, h.dloss = H, normal((n,), 7).abs() * (64 if dt == torch.float16 else 1 / n)
    h.exact()
    loss, lse = gq().linear_cross_entropy(H, h.W, h.y)
    check("loss", loss, h.loss, h.dloss_bound)
    dH = gq().linear_cross_entropy_backward(H, h.W, h.y, lse, h.dloss)["X"]
    (dX64, bX), _ = h.gradients(h.dloss)
    check("dH", dH, dX64, bX)
    dX = gq().packed_linear_backward(dH, words, scales, zeros, 4, 128, **low)
    assert dX.shape == X.shape and bool(torch.isfinite(dX.double()).all())
    g = gq().adapter_backward(dH, X, **low)
    off = bX + U[dt] * dX64.abs() + 2.0 ** -25
    for a in range(m):
        t = torch.nonzero(index == a).flatten()
        x, d, o, al = X[t].double(), dX64[t], off[t], float(alpha[a])
        Aa, Ba = A[a].double(), B[a].double()
        chain = (n + 64) * 2 * EPS + 2.0 ** -14 + (max(r, c) + 32) * 2 * EPS
        check(f"gA[{a}]", g["A"][a], al * (d @ Ba).T @ x, al * ((o + chain * d.abs()) @ Ba.abs()).T @ x.abs())
        check(f"gB[{a}]", g["B"][a], al * d.T @ (x @ Aa.T), al * (o + chain * d.abs()).T @ (x.abs() @ Aa.abs().T))
    up = gq().adapter_orthogonalize(g["A"], g["B"], out_dtype=dt)
    for k, G in (("A", g["A"]), ("B", g["B"].transpose(1, 2))):
        want, mag = update64(G, 5, COEF, 1e-7)
        check("update " + k, up[k] if k == "A" else up[k].transpose(1, 2), want, (rank + 33) * 2 * EPS * mag)
    A.add_(up["A"], alpha=-0.02)
    B.add_(up["B"], alpha=-0.02)
    assert bool(torch.isfinite(gq().linear_cross_entropy(gq().packed_linear(X, words, scales, zeros, 4, 128, **low), h.W, h.y)[0]).all())


@pytest.mark.parametrize("n", [40, 700])
def test_graph_replays(n):
    """A step in one HIP graph, replayed with other inputs, targets and masks, with eager work between."""
    vocab, d, dt = 900, 192, torch.bfloat16
    W = normal((vocab, d), 1, 1 / math.sqrt(d)).to(dt)
    X, y, dloss = normal((n, d), 2).to(dt), targets(n, vocab, 3, "none"), normal((n,), 4)
    A = matrices(2, 80, 300, 5, torch.float32)
    B = matrices(2, 80, 500, 6, torch.float32).transpose(1, 2).contiguous()
    ws = [gq().Workspace() for _ in range(3)]
    out = (torch.empty(n, device="cuda"), torch.empty(n, device="cuda"))
    grads = {"X": torch.empty_like(X), "W": torch.empty_like(W)}
    ups = {"A": torch.empty_like(A), "B": torch.empty_like(B)}

    def step(ws=(None, None, None), out=None, grads=None, ups=None):
        loss, lse = gq().linear_cross_entropy(X, W, y, out=out, ws=ws[0])
        g = gq().linear_cross_entropy_backward(X, W, y, lse, dloss, want_dW=True, out=grads, ws=ws[1])
        u = gq().adapter_orthogonalize(A, B, out=ups, ws=ws[2])
        return loss, lse, g["X"], g["W"], u["A"], u["B"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws, out, grads, ups)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ws, out, grads, ups)
    for k, mask in enumerate(("none", "some", "all", "prompt")):
        X.copy_(normal((n, d), 20 + k).to(dt))
        y.copy_(targets(n, vocab, 30 + k, mask))
        dloss.copy_(normal((n,), 40 + k))
        A.copy_(matrices(2, 80, 300, 50 + k, torch.float32))
        want = [t.clone() for t in step()]
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), (k, mask)


def test_streams_of_their_own():
    """Two calls at once on two streams, each with its own workspace, give what they give alone."""
    heads = [Head(600, 2000, 256, torch.bfloat16, 60 + k, "some") for k in range(2)]
    want = []
    for h in heads:
        loss, lse = gq().linear_cross_entropy(h.X, h.W, h.y)
        want.append((loss, gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, h.dloss)["X"]))
    torch.cuda.synchronize()
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [gq().Workspace() for _ in range(4)]
    got = [None, None]
    for _ in range(3):
        for k, h in enumerate(heads):
            with torch.cuda.stream(streams[k]):
                loss, lse = gq().linear_cross_entropy(h.X, h.W, h.y, ws=ws[2 * k])
                got[k] = (loss, gq().linear_cross_entropy_backward(h.X, h.W, h.y, lse, h.dloss, ws=ws[2 * k + 1])["X"])
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][1], want[k][1])


@pytest.mark.parametrize("n", [3, 300])
def test_head_past_32_bits(n):
    """A head, and its gradient, of more than 2^31 elements: the last entries of the vocabulary
    lie past them."""
    vocab, d, dt = 270001, 8192, torch.bfloat16
    W = torch.empty((vocab, d), dtype=dt, device="cuda")
    for a in range(0, vocab, 30000):
        W[a:a + 30000] = normal((min(30000, vocab - a), d), 70 + a, 1 / math.sqrt(d)).to(dt)
    y = targets(n, vocab, 71, "none")
    y[: n // 2] = vocab - 1 - torch.arange(n // 2, device="cuda")
    X = (normal((n, d), 72) + 2 * W[y].float()).to(dt)
    dloss = normal((n,), 73)
    loss, lse = gq().linear_cross_entropy(X, W, y)
    x = X.double()
    z = torch.cat([x @ W[a:a + 30000].double().T for a in range(0, vocab, 30000)], 1)
    dz = (d + 32) * 2 * EPS * 8 * float(x.norm(dim=1).max()) / math.sqrt(d) * math.sqrt(d)   # |w| is below 8 / sqrt(d), |x|_1 below |x|_2 sqrt(d)
    want = torch.logsumexp(z, 1) - z.gather(1, y.unsqueeze(1)).squeeze(1)
    slack = 2 * dz + (float(z.abs().max()) * 2 + 2) * 4 * EPS + (64 + 3 * (16 + vocab / 2048)) * 2 * EPS
    check("loss", loss, want, torch.full_like(want, slack))
    got = gq().linear_cross_entropy_backward(X, W, y, lse, dloss, want_dW=True)
    D = torch.softmax(z, 1)
    D[torch.arange(n), y] -= 1
    D *= dloss.double().unsqueeze(1)
    off = D.abs() * (2 * slack + U[dt])
    dX, bX = torch.zeros_like(x), torch.zeros_like(x)
    for a in range(0, vocab, 30000):
        w = W[a:a + 30000].double()
        dX += D[:, a:a + 30000] @ w
        bX += (off[:, a:a + 30000] + (vocab + 64) * 2 * EPS * D[:, a:a + 30000].abs()) @ w.abs()
    check("dX", got["X"], dX, bX)
    rows = torch.cat([y, torch.arange(vocab - 300, vocab, device="cuda"), torch.arange(0, vocab, 997, device="cuda")])
    check("dW", got["W"][rows], D[:, rows].T @ x, (off[:, rows] + (n + 64) * 2 * EPS * D[:, rows].abs()).T @ x.abs())
