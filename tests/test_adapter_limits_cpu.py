"""Sizes at the launches' limits (fewer than 2^32 threads each): a call is
refused for a launch that it makes, and for no other.  Nothing here reaches the
device: a size that passes goes on to ask for its workspace (status 6)."""
import ctypes as C
import os
import random

import pytest

from post_weight_quantization_23_amd import _lib

F32, BF16, F16 = 0, 1, 2


def P(k):
    """A made-up address, 2^48 apart per k; never dereferenced."""
    return C.c_void_p((k + 1) << 48)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from post_weight_quantization_23_amd import build
        build.build()
    return _lib.load()


def forward(lib, n, r, c, yt=BF16, m=0, rank=0):
    low = (P(4), P(5)) if m else (None, None)
    return lib.gptq_packed_linear(P(0), BF16, n, c, P(1), r, c, 4, c // 8, P(2), P(3), 1, -1, None, *low, m, rank, None, None, P(6),
                                  yt, r, None, 0, None)


def backward(lib, n, r, c, ot=BF16, m=0, rank=0):
    low = (P(4), P(5)) if m else (None, None)
    return lib.gptq_packed_linear_backward(P(0), BF16, n, r, P(1), r, c, 4, c // 8, P(2), P(3), 1, -1, None, *low, m, rank, None,
                                           None, P(6), ot, c, None, 0, None)


def add(lib, n, r, c, m, rank):
    return lib.gptq_adapter_add(P(0), BF16, n, c, c, P(1), P(2), m, rank, r, None, None, P(3), BF16, r, P(4), r, None, 0, None)


def grads(lib, n, r, c, m, rank):
    return lib.gptq_adapter_backward(P(0), r, P(1), c, BF16, n, r, c, P(2), P(3), m, rank, None, None, P(4), P(5), None, P(6), BF16,
                                     c, None, 0, None)


# prompts against an output layer, long batches, a large bank of adapters
@pytest.mark.parametrize("n,r,c", [(16384, 152064, 4096), (262144, 11008, 4096), (131072, 65536, 1024), (1 << 20, 4096, 64)])
def test_large_products_are_taken(lib, n, r, c):
    out = C.c_size_t()
    for yt in (BF16, F32):
        assert lib.gptq_packed_linear_workspace_size(n, r, c, yt, 16, 0, C.byref(out)) == 0, yt
        assert forward(lib, n, r, c, yt) == 6 and forward(lib, n, r, c, yt, 8, 16) == 6
    assert lib.gptq_packed_linear_backward_workspace_size(n, r, c, BF16, BF16, 8, 16, C.byref(out)) == 0
    assert backward(lib, n, r, c) == 6 and backward(lib, n, r, c, F32, 8, 16) == 6
    assert add(lib, n, r, c, 8, 16) == 6
    assert lib.gptq_adapter_backward_workspace_size(n, r, c, 8, 16, C.byref(out)) == 0
    assert grads(lib, n, r, c, 8, 16) == 6


def test_a_large_bank_of_adapters_is_taken(lib):
    for n in (16, 4096, 300000):
        assert add(lib, n, 4096, 4096, 32768, 8) == 6 and grads(lib, n, 4096, 4096, 32768, 8) == 6
        assert backward(lib, n, 4096, 4096, m=32768, rank=8) == 6


def test_launches_past_the_limit_are_refused(lib):
    # a workgroup per token of what fp32 results prepare; not so for 16-bit ones
    assert forward(lib, (1 << 24) - 1, 8, 32, F32) == 6 and forward(lib, 1 << 24, 8, 32, F32) == 5
    assert forward(lib, 1 << 24, 8, 32) == 6
    # rows of 2080 columns are padded to 2112: it is the copy that has to fit
    n = ((1 << 32) - 1) // 2112 * 8
    assert forward(lib, n - 4096, 8, 2080) == 6 and forward(lib, n + 4096, 8, 2080) == 5
    # rows taken as they are in 512 threads for 48 x 48 outputs at most
    assert forward(lib, 16, 1 << 29, 32) == 5 and forward(lib, 16, 1 << 26, 32, m=1, rank=8) == 6
    # a wave per rank value where tokens are taken one by one, 256 outputs a workgroup
    assert add(lib, 1 << 20, 8, 8, 1 << 20, 128) == 5 and add(lib, 1 << 18, 8, 8, 1 << 18, 128) == 6
    assert grads(lib, 1 << 18, 8, 8, 1 << 18, 128) == 5 and grads(lib, 1 << 17, 8, 8, 1 << 17, 128) == 6
    assert add(lib, 1 << 19, 1 << 14, 8, 1 << 17, 8) == 5 and add(lib, 1 << 19, 1 << 14, 8, 1 << 10, 8) == 6
    assert add(lib, 1 << 29, 1 << 22, 8, 1, 8) == 5
    # gradients: 128 columns of an adapter a wave; 64 x 64 values of two adapters' factors a workgroup of 1024
    assert grads(lib, 16, 1 << 14, 8, 1 << 20, 8) == 5 and grads(lib, 16, 4096, 4096, 65536, 8) == 5
    # the dequantized copy, 64 x 256 weights a workgroup, and tiles of the product
    assert backward(lib, 1 << 12, 1 << 21, 1 << 21) == 5 and backward(lib, 1 << 12, 1 << 20, 1 << 16) == 6
    assert backward(lib, 1 << 29, 1 << 20, 1 << 14) == 5


def test_a_layer_without_rows_beside_adapters(lib):
    """Nothing to do: B has no values then, so its address may be NULL (an empty tensor's is); sizes are still checked."""
    for n in (0, 4, 2000):
        for m, rank, want in ((2, 8, 0), (0, 8, 1), (2, 12, 5)):
            assert lib.gptq_packed_linear(P(0), BF16, n, 64, None, 0, 64, 4, 8, None, None, 2, 32, None, P(4), None, m, rank, None,
                                          None, None, BF16, 0, None, 0, None) == want
            assert lib.gptq_adapter_add(P(0), BF16, n, 64, 64, P(1), None, m, rank, 0, None, None, None, BF16, 0, None, 0, None, 0,
                                        None) == want


def test_what_the_header_says_always_fits(lib):
    rng, seen = random.Random(3), 0

    def log2(bits):
        return min(int(2 ** rng.uniform(0, bits)), 2 ** bits - 1)

    while seen < 5000:
        n, r, c, m, rank = log2(24), log2(24), max(32, log2(24) // 32 * 32), max(1, log2(20)), 8 * rng.randint(1, 16)
        if n * max(r, c) > 2 ** 31 or r * c > 2 ** 37 or m * rank * max(r, c) > 2 ** 29 or (n <= 4 * m and n * rank >= 2 ** 25):
            continue
        seen += 1
        for yt in (F32, BF16):
            assert forward(lib, n, r, c, yt, m, rank) == 6, (n, r, c, m, rank)
            assert r > 2 ** 22 - 64 or backward(lib, n, r, c, yt, m, rank) == 6, (n, r, c, m, rank)
        assert add(lib, n, r, c, m, rank) == 6 and grads(lib, n, r, c, m, rank) == 6, (n, r, c, m, rank)
