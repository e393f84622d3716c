"""Routed calls whose operands pass 2^32 bytes: weights, weight gradients, and
rows of experts, each checked where its offsets are largest. Tolerances are
those of routed_ref.py."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from routed_ref import REL, check, half_step_f16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32 = torch.float16, torch.float32


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
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("per", [1, 40, 200])
def test_grouped_weights(per, bt):
    """70 weights of 64 MiB; rows in the first and the last group only, the rest of the weights NaN."""
    groups, n, k = 70, 8192, 4096
    gn = gen(1)
    b = torch.full((groups, n, k) if bt else (groups, k, n), float("nan"), dtype=F16, device=DEV)
    for e in (0, groups - 1):
        b[e] = (torch.randn(tuple(b.shape[1:]), generator=gn, device=DEV) * 0.05).half()
    a = torch.randn((2 * per, k), generator=gn, device=DEV).half()
    offsets = torch.tensor([0] + [per] * (groups - 1) + [2 * per], dtype=torch.int32, device=DEV)
    c = torch.empty((2 * per, n), dtype=F32, device=DEV)
    say(f"grouped, weights of {b.numel() * 2 >> 20} MiB, {per} rows a group, bt {bt}")
    (g.gemm_f16_grouped_bt if bt else g.gemm_f16_grouped)(a, b, offsets, c)
    for e, lo in ((0, 0), (groups - 1, per)):
        w = (b[e].t().contiguous() if bt else b[e]).double()
        x = a[lo:lo + per].double()
        check(c[lo:lo + per], x @ w, REL * (x.abs() @ w.abs()), f"group {e}")


def test_weight_gradients():
    """40 gradients of 128 MiB."""
    groups, m, n = 40, 4096, 8192
    gn = gen(2)
    rows = 3 * groups
    a = torch.randn((rows, m), generator=gn, device=DEV).half()
    b = torch.randn((rows, n), generator=gn, device=DEV).half()
    offsets = torch.arange(0, rows + 1, 3, dtype=torch.int32, device=DEV)
    c = torch.full((groups, m, n), float("nan"), dtype=F32, device=DEV)
    say(f"wgrad, {c.numel() * 4 >> 20} MiB")
    g.gemm_f16_grouped_wgrad(a, b, offsets, c)
    for e in (0, 33, groups - 1):
        x, y = a[3 * e:3 * e + 3].double().t().contiguous(), b[3 * e:3 * e + 3].double()
        check(c[e], x @ y, REL * (x.abs() @ y.abs()), f"group {e}")


def test_rows_of_experts():
    """300000 rows of 8192 halves: gather to them, combine from them, and the gradient."""
    tokens, width, rows = 64, 8192, 300000
    gn = gen(3)
    x = torch.randn((tokens, width), generator=gn, device=DEV).half()
    row = (rows - 1 - torch.randperm(tokens * 2, generator=gn, device=DEV) * 7).to(torch.int32).reshape(tokens, 2)
    token = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    token[row.long().reshape(-1)] = torch.arange(tokens * 2, device=DEV, dtype=torch.int32) // 2
    weight = torch.rand((tokens, 2), generator=gn, device=DEV)
    say("gather, combine and its gradient over 4.6 GiB of rows")
    z = g.moe_gather(x, token)
    assert torch.equal(z[row.long()[:, 1]], x) and bool((z[:1000] == 0).all())
    y = g.moe_combine(z, row, weight, torch.empty((tokens, width), dtype=F32, device=DEV))
    ref = x.double() * weight.double().sum(1, keepdim=True)
    check(y, ref, 4 * 2.0 ** -24 * ref.abs(), "combine")
    dz, dw = g.moe_combine_backward(x, z, row, weight)
    want = x.double() * weight.double()[:, :1]
    check(dz[row.long()[:, 0]], want, 2.0 ** -24 * want.abs() + half_step_f16(want), "dz")
    dot = (x.double() ** 2).sum(1, keepdim=True).expand(-1, 2)
    check(dw, dot, REL * dot, "dw")
