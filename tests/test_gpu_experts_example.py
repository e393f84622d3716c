"""The example that runs routing, grouped products, their gradients and the
adapters together (examples/experts.py): training, its gradients against 64-bit
autograd and against differences, and serving from a captured graph; and the
routing calls on another stream than the current one."""
import os
import sys

import pytest
import torch

import precision_dense_gemm_03_amd as g

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import experts as ex  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


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


def layer64(x, router, w1, w2, chosen):
    """The layer in 64 bits on the CPU, the experts of each token given (-1: none)."""
    logits = x @ router.t()
    y = torch.zeros_like(x)
    picked = torch.where(chosen >= 0, torch.gather(logits, 1, chosen.clamp(min=0)), torch.tensor(-torch.inf).double())
    weight = torch.softmax(picked, dim=1)
    for j in range(chosen.shape[1]):
        for e in range(router.shape[0]):
            t = (chosen[:, j] == e).nonzero().flatten()
            if len(t):
                out = torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()
                y = y.index_add(0, t, weight[t, j:j + 1] * out)
    return y


@pytest.mark.parametrize("tokens,width,hidden,experts,topk", [(70, 48, 64, 5, 2), (300, 136, 200, 12, 3), (1, 64, 40, 4, 1)])
def test_layer_gradients(tokens, width, hidden, experts, topk):
    """Every path from a parameter to the gradient passes at most 8 roundings to FP16, each off by at most 2^-11 of
    the value, and sums of them err no more than the terms do: 8 * 2^-11 of the sum of the terms' sizes. Norms over
    whole gradients, whose terms add with random signs, stay within 4 times that of the gradient's own norm."""
    say(f"layer {tokens} x {width}, hidden {hidden}, {experts} experts, {topk} each")
    layer = ex.Experts(width, hidden, experts, topk, 11)
    gen = torch.Generator(device=DEV).manual_seed(12)
    x = torch.randn((tokens, width), generator=gen, device=DEV).half()
    dy = torch.randn((tokens, width), generator=gen, device=DEV).half()
    y, kept = layer.forward(x)
    got = layer.backward(dy, kept)
    torch.cuda.synchronize()
    chosen = kept["route"]["expert"].cpu().long()
    leaves = [t.cpu().double().requires_grad_() for t in (x, layer.router, layer.w1, layer.w2)]
    ref = layer64(*leaves, chosen)
    tol = 4 * 8 * 2.0 ** -11
    assert (y.cpu().double() - ref.detach()).norm() <= tol * ref.detach().norm()
    d64 = dy.cpu().double()
    want = torch.autograd.grad((ref * d64).sum(), leaves)
    for name, a, b in zip(("x", "router", "w1", "w2"), got, want):
        a, size = a.cpu().double(), b.norm()
        if topk == 1 and name == "router":
            assert a.abs().max() == 0    # one expert's weight is always 1
            continue
        assert (a - b).norm() <= tol * size, (name, ((a - b).norm() / size).item())
    # along a direction, against central differences of the 64-bit layer (error of order h^2)
    rnd = torch.Generator().manual_seed(13)
    step = 1e-4
    for i, (leaf, a) in enumerate(zip(leaves, got)):
        if topk == 1 and i == 1:
            continue
        # half along the gradient, half at random, so that the slope is not lost in its own rounding
        v = torch.randn(leaf.shape, generator=rnd, dtype=torch.float64)
        v = v / v.norm() + want[i] / want[i].norm()
        ends = []
        for sign in (1.0, -1.0):
            moved = [p.detach() + (sign * step * v if k == i else 0.0) for k, p in enumerate(leaves)]
            ends.append((layer64(*moved, chosen) * d64).sum())
        slope = (ends[0] - ends[1]) / (2 * step)
        assert abs(slope - (a.cpu().double() * v).sum()) <= (tol + 1e-4) * 2 * want[i].norm(), i


def test_training_lowers_the_loss():
    losses = ex.train(steps=30, tokens=256, say=say)
    assert losses[-1] < 0.8 * losses[0], losses


def test_training_repeats_bit_for_bit():
    a = ex.train(steps=4, tokens=200, width=72, hidden=88, experts=5, say=say)
    assert a == ex.train(steps=4, tokens=200, width=72, hidden=88, experts=5, say=say)


@pytest.mark.parametrize("requests", [1, 16, 90])
def test_serving_from_a_graph(requests):
    assert ex.serve(steps=4, requests=requests, say=say)


def test_another_stream():
    """Calls on a stream of their own, outputs left to the binding: nothing of them waits for, or is undone by, what
    the current stream still has to do."""
    gen = torch.Generator(device=DEV).manual_seed(21)
    lg = torch.randn((200, 16), generator=gen, device=DEV)
    x = torch.randn((200, 72), generator=gen, device=DEV).half()
    dy = torch.randn((200, 72), generator=gen, device=DEV).half()
    expert, weight, offsets, row, token = g.moe_route_f32(lg, 2)
    z = g.moe_gather(x, token)
    dz, dw = g.moe_combine_backward(dy, z, row, weight)
    la, lb = torch.randn((3, 8, 72), device=DEV).half(), torch.randn((3, 40, 8), device=DEV).half()
    bt, ad, sc = torch.randn((40, 72), device=DEV).half(), (expert[:, 0] % 4 - 1).contiguous(), torch.ones(3, device=DEV)
    c = torch.empty((200, 40), dtype=torch.float16, device=DEV)
    want_c = g.gemm_f16_lora_bt(x, bt, la, lb, ad, sc, torch.empty_like(c))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.empty(1 << 28, device=DEV)
    for how in (side, side.cuda_stream):
        for _ in range(4):
            big.fill_(1.0)    # the current stream is busy for some hundred microseconds
        got = g.moe_route_f32(lg, 2, stream=how)
        gz = g.moe_gather(x, got[4], stream=how)
        gdz, gdw = g.moe_combine_backward(dy, gz, got[3], got[1], stream=how)
        g.gemm_f16_lora_bt(x, bt, la, lb, ad, sc, c, stream=how)
        side.synchronize()
        with torch.cuda.stream(side):
            same = [torch.equal(p, q) for p, q in zip(list(got) + [gz, gdz, gdw, c],
                                                      [expert, weight, offsets, row, token, z, dz, dw, want_c])]
        torch.cuda.synchronize()
        assert all(same), same
        assert torch.equal(gdz, dz)
