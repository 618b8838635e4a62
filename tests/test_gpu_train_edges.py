"""The loss, its gradients and the adapters' update where they can go wrong.  Bounds as in
test_gpu_train.py unless said."""
import pytest
import torch

from test_gpu_train import DT, Head, gq, matrices, normal

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
