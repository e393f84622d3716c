"""Routed calls at the ends of their size ranges: sizes next to 2^31, and
launches of 2^32 threads and more. Every case has a 288 GB card in mind and
takes at most 130 GB of it; outputs are checked on the device, exactly
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


# more rows than 2^32 threads hold at a workgroup of 256 each (rows of over 128 16-byte units)
MANY = (1 << 24) + 5


def test_gather_of_many_wide_rows():
    width = 2053
    say(f"gather to {MANY} rows of {width} bytes")
    x = torch.randint(0, 256, (7, width), device=DEV, dtype=torch.uint8)
    token = (torch.arange(MANY, device=DEV) % 8).to(I32)     # 7: no such token
    y = g.moe_gather(x, token)
    zero = torch.cat([x, torch.zeros_like(x[:1])])
    for lo in range(0, MANY, 1 << 21):
        hi = min(MANY, lo + (1 << 21))
        want = zero[torch.arange(lo, hi, device=DEV) % 8]
        assert torch.equal(y[lo:hi], want), lo


def test_combine_of_many_wide_rows():
    """y[t] = z[row[t]]; then its gradient, with rows of z for the last tokens only."""
    width, rows = 1032, 4096
    say(f"combine of {MANY} tokens of {width} halves")
    gn = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn((rows, width), generator=gn, device=DEV).half()
    row = (torch.arange(MANY, device=DEV) % (rows + 1)).to(I32).view(-1, 1)     # `rows`: none
    y = g.moe_combine(z, row, None)
    padded = torch.cat([z, torch.zeros_like(z[:1])])
    step = 1 << 21
    for lo in range(0, MANY, step):
        hi = min(MANY, lo + step)
        assert torch.equal(y[lo:hi], padded[row[lo:hi, 0].long()]), lo
    # the gradient with dy = y: <z, z> and z in the named rows
    row.fill_(-1)
    row[MANY - rows:, 0] = torch.arange(rows, device=DEV).to(I32)
    weight = torch.ones((MANY, 1), device=DEV)
    say("and its gradient")
    dz, dw = g.moe_combine_backward(y, z, row, weight)
    last = y[MANY - rows:]
    assert torch.equal(dz, last)
    assert bool((dw[:MANY - rows] == 0).all())
    dot = (z.double() * last.double()).sum(1, keepdim=True)
    size = (z.double() * last.double()).abs().sum(1, keepdim=True)
    assert bool(((dw[MANY - rows:].double() - dot).abs() <= 1e-5 * size).all())


def test_route_backward_of_many_tokens():
    """Four tokens to a workgroup of 256: 2^32 threads from 2^26 tokens on. Two experts of weight 1/2 and dweight
    (t % 4, 0): dlogits (t % 4) / 4 and its negative, exactly."""
    T = (1 << 26) + 21
    say(f"route backward of {T} tokens")
    t = torch.arange(T, device=DEV) % 4
    logits = torch.zeros((T, 2), device=DEV)
    expert = torch.tensor([[0, 1]], dtype=I32, device=DEV).repeat(T, 1)
    weight = torch.full((T, 2), 0.5, device=DEV)
    dweight = torch.stack([t.float(), torch.zeros_like(t, dtype=F32)], 1)
    for renorm in (True, False):
        d = g.moe_route_backward_f32(logits, expert, weight, dweight, renorm=renorm)
        assert torch.equal(d[:, 0], t.float() / 4) and torch.equal(d[:, 1], -t.float() / 4), renorm


def grouped_rows(rows, n, k, out, name, monkeypatch):
    """C[r] = A[r] B[g] in small whole numbers, two groups, rows of no group at both ends."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    lead, cut, tail = 1001, rows // 2 + 3, 70
    gn = torch.Generator(device=DEV).manual_seed(2)
    a = torch.randint(-3, 4, (rows, k), generator=gn, device=DEV, dtype=torch.int8).half()
    b = torch.randint(-3, 4, (2, n, k), generator=gn, device=DEV).half()
    offsets = torch.tensor([lead, cut, rows - tail], dtype=I32, device=DEV)
    c = torch.full((rows, n), 9.0, dtype=out, device=DEV)
    say(f"{name} over {rows} rows")
    g.gemm_f16_grouped_bt(a, b, offsets, c)
    step = 1 << 24
    for e, (lo, hi) in enumerate(((lead, cut), (cut, rows - tail))):
        w = b[e].float().t().contiguous()
        for at in range(lo, hi, step):
            end = min(hi, at + step)
            assert torch.equal(c[at:end].float(), a[at:end].float() @ w), (e, at)
    assert bool((c[:lead] == 0).all()) and bool((c[rows - tail:] == 0).all())


@pytest.mark.parametrize("name,rows", [("grouped_ring", (1 << 26) + 4001), ("grouped_pp_128", (1 << 26) + 4001),
                                       ("grouped_pp_256", (1 << 27) + 4001), ("grouped_tile_64", (1 << 26) + 4001)])
def test_grouped_of_many_rows(name, rows, monkeypatch):
    """Workgroups of 256 or 512 threads that reach 2^32 threads."""
    grouped_rows(rows, 8, 8, F16, name, monkeypatch)


@pytest.mark.parametrize("name,m,n", [("wgrad_pp", 8, (1 << 19) + 256), ("wgrad_tile_128", 1, (1 << 19) + 128),
                                      ("wgrad_tile_64", 1, (1 << 18) + 64)])
def test_weight_gradients_of_many_tiles(name, m, n, monkeypatch):
    """4096 groups whose tiles reach 2^32 threads; rows in every 1365th, the last group among them."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    groups, every, per = 4096, 1365, 2
    gn = torch.Generator(device=DEV).manual_seed(3)
    full = range(0, groups, every)
    sizes = torch.zeros(groups, dtype=torch.int64)
    sizes[::every] = per
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(I32).to(DEV)
    rows = int(offsets[-1])
    a = torch.randint(-3, 4, (rows, m), generator=gn, device=DEV).half()
    b = torch.randint(-3, 4, (rows, n), generator=gn, device=DEV).half()
    c = torch.full((groups, m, n), 9.0, dtype=F16, device=DEV)
    say(f"{name}: {groups} gradients of {m} x {n}")
    g.gemm_f16_grouped_wgrad(a, b, offsets, c)
    assert full[-1] == groups - 1
    for i, e in enumerate(full):
        x, y = a[per * i:per * i + per].float().t().contiguous(), b[per * i:per * i + per].float()
        assert torch.equal(c[e].float(), x @ y), e
    for lo, hi in zip(full, full[1:]):
        assert bool((c[lo + 1:hi] == 0).all()), lo


def lora_rows(rows, n, k, rank, name, monkeypatch, count=3):
    """Small whole numbers; adapters in turn, every fourth row without one."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    gn = torch.Generator(device=DEV).manual_seed(4)
    unit = torch.randint(-3, 4, (4001, k), generator=gn, device=DEV).half()      # 4001 rows over and over
    a = torch.empty((rows, k), dtype=F16, device=DEV)
    whole = rows // 4001 * 4001
    a[:whole].view(-1, 4001, k).copy_(unit)
    a[whole:] = unit[:rows - whole]
    b = torch.randint(-3, 4, (n, k), generator=gn, device=DEV).half()
    la = torch.randint(-2, 3, (count, rank, k), generator=gn, device=DEV).half()
    lb = torch.randint(-2, 3, (count, n, rank), generator=gn, device=DEV).half()
    scale = torch.tensor([1.0, 2.0, 0.5][:count], device=DEV)
    adapter = torch.arange(rows, dtype=I32, device=DEV)
    adapter.remainder_(count + 1).sub_(1)
    c = torch.full((rows, n), 9.0, dtype=F16, device=DEV)
    say(f"{name} over {rows} rows, rank {rank}")
    g.gemm_f16_lora_bt(a, b, la, lb, adapter, scale, c)
    step = 1 << 24
    for at in range(0, rows, step):
        x, who = a[at:at + step].float(), adapter[at:at + step]
        ref = x @ b.float().t()
        for e in range(count):
            y = (x @ la[e].float().t()) @ lb[e].float().t() * scale[e]
            ref += torch.where((who == e)[:, None], y, torch.zeros_like(y))
        assert torch.equal(c[at:at + step].float(), ref), at


@pytest.mark.parametrize("name,rows,k", [("lora_tile_64", (1 << 27) + 19, 1), ("lora_ring", (1 << 28) + 4001, 8),
                                         ("lora_tile_64", (1 << 30) + 77, 1), ("lora_ring", (1 << 30) + 77, 8),
                                         ("lora_pp_192", 192 * (1 << 23) + 77, 8)])
def test_adapters_of_many_rows(name, rows, k, monkeypatch):
    """Low-rank values of 2^27 and 2^28 rows, and products of 2^30 and more, reach 2^32 threads."""
    lora_rows(rows, 8 if k == 8 else 1, k, 2, name, monkeypatch)


@pytest.mark.parametrize("rows,name", [(64, "lora_ring"), (65, "lora_tile_64"), (65, "lora_ring")])
def test_adapters_of_a_large_rank(rows, name, monkeypatch):
    """rows * rank waves of 64 threads reach 2^32; more than 2^16 blocks of 64 low-rank values."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    n, k, rank = 8, 8, (1 << 22) + 88
    gn = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(-3, 4, (rows, k), generator=gn, device=DEV).half()
    b = torch.randint(-3, 4, (n, k), generator=gn, device=DEV).half()
    at = torch.tensor([0, 5, 63, 64, 1 << 20, (1 << 20) + 1, (1 << 22) - 1, 1 << 22, rank - 1], device=DEV)
    la = torch.zeros((2, rank, k), dtype=F16, device=DEV)
    lb = torch.randint(-2, 3, (2, n, rank), generator=gn, device=DEV, dtype=torch.int8).half()
    la[:, at] = torch.randint(-2, 3, (2, len(at), k), generator=gn, device=DEV).half()
    adapter = (torch.arange(rows, device=DEV) % 3 - 1).to(I32)
    scale = torch.tensor([1.0, 2.0], device=DEV)
    c = torch.full((rows, n), 9.0, dtype=F32, device=DEV)
    say(f"{name}: {rows} rows, rank {rank}")
    g.gemm_f16_lora_bt(a, b, la, lb, adapter, scale, c)
    ref = a.float() @ b.float().t()
    for e in range(2):
        y = (a.float() @ la[e, at].float().t()) @ lb[e][:, at].float().t() * scale[e]
        ref += torch.where((adapter == e)[:, None], y, torch.zeros_like(y))
    assert torch.equal(c, ref)
