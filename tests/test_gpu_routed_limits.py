"""Routed calls at the ends of their size ranges: sizes next to 2^31, and
launches of 2^32 threads and more. Every case has a 288 GB card in mind and
keeps its operands below 100 GB; outputs are checked on the device, exactly
where the arithmetic is exact."""
import pytest
import torch

import precision_dense_gemm_03_amd as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32, I32 = torch.float16, torch.float32, torch.int32


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(DEV)
    g.lib()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def all_equal(t, want, step=1 << 28):
    """Every element of the flat t equals want (a value, or a function of the indices), in pieces."""
    for lo in range(0, t.numel(), step):
        piece = t[lo:lo + step]
        ref = want if not callable(want) else want(torch.arange(lo, lo + piece.numel(), device=t.device))
        if not bool((piece == ref).all()):
            return False
    return True


def test_route_of_the_most_tokens():
    """tokens * topk of 2^31 - 1: one expert, which every token chooses."""
    T = (1 << 31) - 1
    say(f"route of {T} tokens, one expert")
    logits = torch.zeros((T, 1), device=DEV)
    expert, weight, offsets, row, token = g.moe_route_f32(logits, 1)
    assert offsets.tolist() == [0, T]
    assert all_equal(expert.view(-1), 0) and all_equal(weight.view(-1), 1.0)
    assert all_equal(row.view(-1), lambda i: i) and all_equal(token, lambda i: i)
