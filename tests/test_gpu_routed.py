"""GPU parity of the products whose weight depends on the row: grouped by
expert (gemm_*_grouped*, gemm_f16_grouped_wgrad) and with per-row adapters
(gemm_*_lora_bt), against 64-bit references (routed_ref.py). Each test prints
the case it is about to launch."""
import random

import numpy as np
import pytest
import torch

import oracle as orc
import precision_dense_gemm_03_amd as g
from parity import fp8_dot_allowance
from routed_ref import REL, check, cut, group_of, grouped, half_step_f16, lora

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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(gn, shape, std=1.0):
    return torch.randn(shape, generator=gn, device=DEV) * std


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bound_of(v, s, out, extra=0.0):
    b = REL * s + extra
    return b + half_step_f16(v) if out == F16 else b


def run_f16(seed, sizes, n, k, bt, out, lead=0, tail=0):
    offsets = cut(sizes, lead)
    rows = offsets[-1] + tail
    gn = gen(seed)
    a = normal(gn, (rows, k)).half()
    b = normal(gn, (len(sizes), n, k) if bt else (len(sizes), k, n), 0.1).half()
    c = torch.full((rows, n), float("nan"), dtype=out, device=DEV)
    (g.gemm_f16_grouped_bt if bt else g.gemm_f16_grouped)(a, b, i32(offsets), c)
    v, s = grouped(a, b, offsets, bt)
    check(c, v, bound_of(v, s, out), f"grouped f16 sizes {sizes} n {n} k {k} bt {bt}")
    assert bool((c[group_of(offsets, rows) < 0] == 0).all()), "rows of no group are zeros"


SIZES = [
    [1], [0, 0, 5], [16, 0, 1, 33], [64, 64], [3] * 40, [130, 0, 7, 251, 1], [513, 300], [0, 0],
]


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:6])))
def test_grouped_f16(sizes, out, bt):
    for n, k in ((128, 64), (200, 176), (129, 65), (64, 1), (7, 8), (1, 130), (272, 1000)):
        say(f"grouped f16 {sizes[:6]} n {n} k {k} bt {bt} {out}")
        run_f16(n + k, sizes, n, k, bt, out)


@pytest.mark.parametrize("bt", [True, False])
def test_grouped_f16_rows_of_no_group(bt):
    for sizes, lead, tail in (([5, 0, 70], 3, 0), ([5, 0, 70], 0, 200), ([0, 0], 4, 1), ([300], 129, 513)):
        say(f"grouped f16 lead {lead} sizes {sizes} tail {tail} bt {bt}")
        run_f16(3, sizes, 136, 96, bt, F16, lead, tail)


# rows per group from a few to hundreds and wide weights: every kernel the rules choose
LARGE = [([8] * 6 + [0] * 6, 2048, 1024), ([40, 17, 90, 3], 1024, 512), ([200, 60, 90, 130], 1040, 528),
         ([700, 1500, 0, 900], 1536, 256), ([1030, 770, 513, 1], 1288, 520), ([1100, 2000, 900, 130], 2080, 416),
         ([2100], 2056, 72), ([300] * 9, 768, 2048)]


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("sizes,n,k", LARGE, ids=lambda v: str(v if isinstance(v, int) else sum(v)))
def test_grouped_f16_large(sizes, n, k, bt):
    for out in (F16, F32):
        say(f"grouped f16 {sizes} n {n} k {k} bt {bt} {out}")
        run_f16(n * 7 + k, sizes, n, k, bt, out, tail=3)


@pytest.mark.parametrize("bt", [True, False])
def test_grouped_f16_many_groups(bt):
    rnd = random.Random(5)
    for count in (61, 62, 63, 64, 65, 130, 300):
        sizes = [rnd.choice((0, 0, 1, 2, 17)) for _ in range(count)]
        say(f"grouped f16 {count} groups of {sum(sizes)} rows bt {bt}")
        run_f16(count, sizes, 48, 40, bt, F32, lead=2, tail=5)


@pytest.mark.parametrize("bt", [True, False])
def test_grouped_other_groups_do_not_reach_a_row(bt):
    """NaN and infinities in the other groups' rows and weights stay there."""
    for sizes, n, k in (([20, 33, 9], 72, 100), ([700, 900, 600], 768, 520), ([200, 130, 70], 256, 264)):
        say(f"grouped NaN neighbours {sizes} bt {bt}")
        offsets = cut(sizes)
        gn = gen(1)
        a = normal(gn, (offsets[-1], k)).half()
        b = normal(gn, (3, n, k) if bt else (3, k, n), 0.1).half()
        v, s = grouped(a, b, offsets, bt)
        lo, hi = offsets[1], offsets[2]
        a[:lo] = float("nan")
        a[hi:] = float("inf")
        b[0] = float("inf")
        b[2] = float("nan")
        c = torch.zeros((offsets[-1], n), dtype=F32, device=DEV)
        (g.gemm_f16_grouped_bt if bt else g.gemm_f16_grouped)(a, b, i32(offsets), c)
        check(c[lo:hi], v[lo:hi], REL * s[lo:hi], "the middle group")
        assert bool(c[:lo].isnan().all()) and bool(c[hi:].isnan().all())


def test_grouped_offsets_out_of_range_stay_inside():
    """Offsets out of order or out of [0, rows]: no access outside the operands, rows below stay as they were."""
    n, k, rows = 96, 64, 150
    gn = gen(9)
    a = normal(gn, (rows, k)).half()
    b = normal(gn, (3, n, k)).half()
    for off in ([0, 90, 40, 150], [-5, 50, 100, 900], [10, 10, 10, 10], [150, 100, 50, 0]):
        say(f"grouped offsets {off}")
        room = torch.full((rows + 64, n), 7.0, dtype=F32, device=DEV)
        g.gemm_f16_grouped_bt(a, b, i32(off), room[:rows])
        assert bool((room[rows:] == 7.0).all())
        assert bool(room[:rows].isfinite().all())


def test_grouped_unaligned_pointers():
    """Operands that start at any element."""
    n, k, sizes = 80, 72, [30, 0, 41]
    offsets = cut(sizes)
    rows = offsets[-1]
    gn = gen(4)
    a = normal(gn, (rows * k + 1,)).half()[1:].view(rows, k)
    for bt in (True, False):
        b = normal(gn, (3 * n * k + 3,), 0.1).half()[3:].view((3, n, k) if bt else (3, k, n))
        c = torch.zeros(rows * n + 1, dtype=F16, device=DEV)[1:].view(rows, n)
        say(f"grouped unaligned bt {bt}")
        (g.gemm_f16_grouped_bt if bt else g.gemm_f16_grouped)(a, b, i32(offsets), c)
        v, s = grouped(a, b, offsets, bt)
        check(c, v, bound_of(v, s, F16), "unaligned")


def fp8(x, fmt):
    t = torch.float8_e5m2 if fmt == g.FMT_E5M2 else torch.float8_e4m3fn
    return x.to(t)


def run_fp8(seed, sizes, n, k, bt, channel, out, fa=0, fb=0, lead=0, tail=0):
    offsets = cut(sizes, lead)
    rows = offsets[-1] + tail
    gn = gen(seed)
    qa = fp8(normal(gn, (rows, k), 8.0), fa)
    qb = fp8(normal(gn, (len(sizes), n, k) if bt else (len(sizes), k, n), 8.0), fb)
    G = len(sizes)
    sa = torch.rand(rows if channel else 1, generator=gn, device=DEV) + 0.5
    sb = torch.rand((G, n) if channel else (G,), generator=gn, device=DEV) + 0.5
    name = "gemm_fp8_grouped" + ("_channel" if channel else "") + ("_bt" if bt else "")
    s_out = None
    if out in (F16, F32):
        c = torch.full((rows, n), float("nan"), dtype=out, device=DEV)
    else:
        c = torch.full((rows, n), 0x55, dtype=torch.uint8, device=DEV).view(out)
        s_out = torch.tensor([64.0 * k ** 0.5], device=DEV)
    getattr(g, name)(qa, fa, qb, fb, i32(offsets), sa, sb, c, sOut=s_out)
    v, s = grouped(qa.float(), qb.float(), offsets, bt)
    t = torch.zeros_like(s)
    for e in range(G):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            w = qb[e].view(torch.uint8)
            w = w.t().contiguous() if bt else w
            t[lo:hi] = torch.from_numpy(fp8_dot_allowance(qa[lo:hi].view(torch.uint8).cpu().numpy(), w.cpu().numpy(),
                                                          fmt_a=orc.FMT_E5M2 if fa else orc.FMT_E4M3,
                                                          fmt_b=orc.FMT_E5M2 if fb else orc.FMT_E4M3)).to(DEV)
    group = group_of(offsets, rows)
    gi = torch.from_numpy(np.maximum(group, 0)).to(DEV)
    sc = (sa.double()[:, None] * sb.double()[gi]) if channel else (sa.double() * sb.double()[gi])[:, None]
    if s_out is not None:
        sc = sc / s_out.double()
        v, b = v * sc, (REL * s + t) * sc
        m, tiny, top = (2, 2.0 ** -17, 57344.0) if out == torch.float8_e5m2 else (3, 2.0 ** -10, 448.0)
        b = b + torch.clamp((v.abs() + b) * 2.0 ** -(m + 1), min=tiny)    # half a step
        check(c.float(), v.clamp(-top, top), b, f"{name} {sizes} n {n} k {k} {out}")
    else:
        # three FP32 products after the sum: 3 * 2^-24 of the value
        v, b = v * sc, (REL * s + t) * sc
        b = b + 3 * 2.0 ** -24 * v.abs()
        check(c, v, b + half_step_f16(v) if out == F16 else b, f"{name} {sizes} n {n} k {k} {out}")
    assert bool((c.float()[torch.from_numpy(group < 0).to(DEV)] == 0).all())


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("channel", [True, False])
def test_grouped_fp8(channel, bt):
    for i, (sizes, n, k) in enumerate((([1, 0, 20], 64, 128), ([70, 3], 144, 272), ([5, 5, 0, 5], 33, 65),
                                       ([17, 140], 257, 130), ([2], 16, 16), ([9, 1], 5, 3))):
        for out in (F16, F32, torch.float8_e4m3fn, torch.float8_e5m2):
            say(f"grouped fp8 {sizes} n {n} k {k} bt {bt} channel {channel} {out}")
            run_fp8(i, sizes, n, k, bt, channel, out, lead=i % 2, tail=2 * (i % 3))


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 0), (1, 1)])
def test_grouped_fp8_formats(fa, fb, bt):
    for sizes, n, k in (([6, 0, 21], 80, 144), ([130, 70], 65, 129), ([300, 290], 512, 64)):
        say(f"grouped fp8 formats {fa} {fb} {sizes} n {n} k {k} bt {bt}")
        run_fp8(2, sizes, n, k, bt, False, F32, fa, fb)


@pytest.mark.parametrize("bt", [True, False])
def test_grouped_fp8_large(bt):
    for sizes, n, k, channel, out in (([4] * 20, 1024, 256, True, F16), ([50, 20, 64], 512, 256, False, F32),
                                      ([800, 500, 300], 768, 192, True, F16), ([1000, 700, 77], 784, 80, False, F16),
                                      ([600, 555], 520, 144, True, torch.float8_e4m3fn)):
        say(f"grouped fp8 {sizes} n {n} k {k} bt {bt} channel {channel} {out}")
        run_fp8(6, sizes, n, k, bt, channel, out, tail=1)


def run_wgrad(seed, sizes, m, n, out, lead=0, tail=0):
    offsets = cut(sizes, lead)
    rows = offsets[-1] + tail
    gn = gen(seed)
    a, b = normal(gn, (rows, m)).half(), normal(gn, (rows, n)).half()
    v = torch.zeros((len(sizes), m, n), dtype=torch.float64, device=DEV)
    s = torch.zeros_like(v)
    for e in range(len(sizes)):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            x, y = a[lo:hi].double().t().contiguous(), b[lo:hi].double()
            v[e], s[e] = x @ y, x.abs() @ y.abs()
    a[:lead], b[:lead] = float("nan"), float("nan")      # rows of no group take no part
    a[offsets[-1]:], b[offsets[-1]:] = float("inf"), float("nan")
    c = torch.full((len(sizes), m, n), float("nan"), dtype=out, device=DEV)
    g.gemm_f16_grouped_wgrad(a, b, i32(offsets), c)
    check(c, v, bound_of(v, s, out), f"wgrad {sizes} m {m} n {n} {out}")


@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("sizes", SIZES + [[31, 32, 33, 63, 65]], ids=lambda s: "-".join(map(str, s[:6])))
def test_wgrad(sizes, out):
    for m, n in ((128, 128), (64, 200), (129, 65), (1, 7), (272, 16), (264, 520)):
        say(f"wgrad {sizes[:6]} m {m} n {n} {out}")
        run_wgrad(m + n, sizes, m, n, out, lead=2, tail=3)


@pytest.mark.parametrize("out", [F16, F32])
def test_wgrad_large(out):
    for sizes, m, n in (([700, 0, 1111], 768, 512), ([2000], 1032, 1288), ([100] * 12, 512, 776)):
        say(f"wgrad {sizes} m {m} n {n} {out}")
        run_wgrad(8, sizes, m, n, out)


def test_wgrad_other_groups_do_not_reach_a_group():
    offsets = [0, 45, 90, 200]
    gn = gen(2)
    a, b = normal(gn, (200, 256)).half(), normal(gn, (200, 264)).half()
    x, y = a[45:90].double().t().contiguous(), b[45:90].double()
    v, s = x @ y, x.abs() @ y.abs()
    a[:45], a[90:], b[:45], b[90:] = float("nan"), float("inf"), float("inf"), float("nan")
    c = torch.zeros((3, 256, 264), dtype=F32, device=DEV)
    say("wgrad NaN neighbours")
    g.gemm_f16_grouped_wgrad(a, b, i32(offsets), c)
    check(c[1], v, REL * s, "the middle group")


def test_wgrad_is_the_gradient():
    """<dC, A W> differentiated by W: wgrad against differences of the forward call, in exact small integers."""
    sizes, n, k = [3, 0, 4], 8, 8
    offsets = i32(cut(sizes))
    gn = gen(3)
    a = torch.randint(-3, 4, (7, k), generator=gn, device=DEV).half()
    w = torch.randint(-3, 4, (3, k, n), generator=gn, device=DEV).half()
    dc = torch.randint(-3, 4, (7, n), generator=gn, device=DEV).half()

    def loss(w):
        c = torch.empty((7, n), dtype=F32, device=DEV)
        g.gemm_f16_grouped(a, w, offsets, c)
        return (c.double() * dc.double()).sum()

    dw = torch.empty((3, k, n), dtype=F32, device=DEV)
    say("wgrad against differences")
    g.gemm_f16_grouped_wgrad(a, dc, offsets, dw)
    for e, i, j in ((0, 0, 0), (0, 7, 3), (1, 2, 2), (2, 5, 7), (2, 0, 1)):
        step = torch.zeros_like(w)
        step[e, i, j] = 1.0
        assert (loss(w + step) - loss(w - step)).item() / 2 == dw[e, i, j].item()


# ------------------------------------------------------------------- adapters

def adapters_of(rnd, rows, count, runs):
    out = []
    while len(out) < rows:
        a = rnd.choice([-1] + list(range(count)) * 2)
        out += [a] * (rnd.randint(1, runs) if runs > 1 else 1)
    return out[:rows]


def run_lora(seed, rows, n, k, rank, count, runs, out, kind="f16", workspace=True):
    gn, rnd = gen(seed), random.Random(seed)
    x = normal(gn, (rows, k))
    x16 = x.half()
    la = normal(gn, (count, rank, k), k ** -0.5).half()
    lb = normal(gn, (count, n, rank), 0.2).half()
    scale = torch.rand(count, generator=gn, device=DEV) * 2 + 0.25
    ad = i32(adapters_of(rnd, rows, count, runs))
    c = torch.full((rows, n), float("nan"), dtype=out, device=DEV)
    ws = None
    if workspace:
        ws = torch.full((g.lora_workspace_size(rows, rank) + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    if kind == "f16":
        b = normal(gn, (n, k), 0.05).half()
        g.gemm_f16_lora_bt(x16, b, la, lb, ad, scale, c, workspace=ws)
        w = b.double().t().contiguous()
        v, s = x16.double() @ w, x16.double().abs() @ w.abs()
        base = REL * s
    else:
        fa, fb = kind
        qa, qb = fp8(x * 16, fa), fp8(normal(gn, (n, k), 8.0), fb)
        sa = torch.rand(rows, generator=gn, device=DEV) * 0.05 + 0.01
        sb = torch.rand(n, generator=gn, device=DEV) * 0.05 + 0.01
        g.gemm_fp8_lora_bt(qa, fa, qb, fb, sa, sb, x16, la, lb, ad, scale, c, workspace=ws)
        w = qb.double().t().contiguous()
        sc = sa.double()[:, None] * sb.double()
        v, s = (qa.double() @ w) * sc, (qa.double().abs() @ w.abs()) * sc
        t = torch.from_numpy(fp8_dot_allowance(qa.view(torch.uint8).cpu().numpy(),
                                               qb.view(torch.uint8).t().contiguous().cpu().numpy(),
                                               fmt_a=orc.FMT_E5M2 if fa else orc.FMT_E4M3,
                                               fmt_b=orc.FMT_E5M2 if fb else orc.FMT_E4M3)).to(DEV)
        base = REL * s + t * sc + 3 * 2.0 ** -24 * v.abs()
    lv, lbound = lora(x16, la, lb, ad, scale, n)
    y = v + lv
    bound = base + lbound + 2.0 ** -23 * (v.abs() + lv.abs())   # the last FP32 addition
    check(c, y, bound + half_step_f16(y) if out == F16 else bound, f"lora {kind} rows {rows} n {n} k {k} rank {rank}")


@pytest.mark.parametrize("rank", [1, 4, 8, 16, 24, 64, 100, 128, 160])
@pytest.mark.parametrize("rows", [1, 7, 16, 33, 65, 200, 300])
def test_lora_f16(rows, rank):
    for n, k, count, runs, out in ((64, 128, 3, 1, F16), (200, 176, 20, 5, F32), (65, 33, 2, 40, F16), (8, 5, 1, 1, F32)):
        say(f"lora f16 rows {rows} n {n} k {k} rank {rank} adapters {count} runs {runs} {out}")
        run_lora(rows * rank + n, rows, n, k, rank, count, runs, out)


@pytest.mark.parametrize("rows,n,k,rank,count,runs", [(700, 1536, 512, 16, 5, 200), (4096, 1040, 264, 64, 8, 900),
                                                     (2100, 4096, 96, 24, 6, 64), (1500, 1281, 257, 32, 9, 300),
                                                     (2048, 2048, 128, 128, 3, 5), (16, 4096, 4096, 16, 16, 1)])
def test_lora_f16_large(rows, n, k, rank, count, runs):
    for out in (F16, F32):
        say(f"lora f16 rows {rows} n {n} k {k} rank {rank} adapters {count} {out}")
        run_lora(5, rows, n, k, rank, count, runs, out, workspace=False)


@pytest.mark.parametrize("kind", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_lora_fp8(kind):
    for rows, n, k, rank, count, runs, out in ((5, 64, 128, 8, 4, 1, F16), (40, 80, 144, 16, 9, 2, F32),
                                               (130, 65, 65, 4, 3, 30, F16), (300, 272, 272, 64, 4, 90, F16),
                                               (900, 768, 160, 20, 4, 200, F16)):
        say(f"lora fp8 {kind} rows {rows} n {n} k {k} rank {rank} {out}")
        run_lora(rows, rows, n, k, rank, count, runs, out, kind)


@pytest.mark.parametrize("rows", [12, 80, 400, 3000])
def test_lora_other_adapters_do_not_reach_a_row(rows):
    n, k, rank = 1024, 64, 16
    gn = gen(7)
    x, b = normal(gn, (rows, k)).half(), normal(gn, (n, k), 0.1).half()
    la, lb = normal(gn, (3, rank, k)).half(), normal(gn, (3, n, rank)).half()
    scale = torch.ones(3, device=DEV)
    ad = i32([(-1, 1, 0, 5, 1, 2)[i % 6] for i in range(rows)])
    w = b.double().t().contiguous()
    v, s = x.double() @ w, x.double().abs() @ w.abs()
    only = torch.where(ad == 1, ad, torch.full_like(ad, -1))
    lv, lbound = lora(x, la, lb, only, scale, n)
    la[0], lb[2], scale[0] = float("nan"), float("inf"), float("nan")
    c = torch.zeros((rows, n), dtype=F32, device=DEV)
    say(f"lora NaN adapters rows {rows}")
    g.gemm_f16_lora_bt(x, b, la, lb, ad, scale, c)
    clean = (ad == -1) | (ad == 1) | (ad == 5)           # 5: no such adapter
    y = v + lv
    check(c[clean], y[clean], (REL * s + lbound + 2.0 ** -23 * (v.abs() + lv.abs()))[clean], "rows of adapter 1 or none")
    assert not bool(c[ad == 0].isfinite().any())


@pytest.mark.parametrize("rows", [10, 500])
@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 600.0])
def test_lora_range(rows, size):
    """Low-rank values far below and above FP16's range, FP32 out."""
    n, k, rank = 160, 512, 40
    gn = gen(11)
    x = normal(gn, (rows, k), size).half()
    b = torch.zeros((n, k), dtype=F16, device=DEV)
    la, lb = normal(gn, (2, rank, k), min(size, 60.0)).half(), normal(gn, (2, n, rank)).half()
    scale = torch.tensor([1.0, 30.0], device=DEV)
    ad = i32([i % 2 for i in range(rows)])
    c = torch.zeros((rows, n), dtype=F32, device=DEV)
    say(f"lora range {size} rows {rows}")
    g.gemm_f16_lora_bt(x, b, la, lb, ad, scale, c)
    lv, lbound = lora(x, la, lb, ad, scale, n)
    check(c, lv, lbound + 2.0 ** -23 * lv.abs(), "lora range")


def test_lora_without_adapters_is_the_plain_product():
    gn = gen(12)
    x, b = normal(gn, (40, 96)).half(), normal(gn, (72, 96)).half()
    c, d = torch.empty((40, 72), dtype=F16, device=DEV), torch.empty((40, 72), dtype=F16, device=DEV)
    say("lora rank 0")
    g.gemm_f16_lora_bt(x, b, torch.empty((2, 0, 96), dtype=F16, device=DEV),
                       torch.empty((2, 72, 0), dtype=F16, device=DEV), i32([0] * 40), torch.ones(2, device=DEV), c)
    g.gemm_f16_bt(x, b, d)
    assert torch.equal(c, d)


# ------------------------------------------------------------ streams, repeats

def test_repeats_are_bitwise_equal_and_captured():
    """Calls repeat bit for bit, eagerly and as a captured graph replayed between other work."""
    gn = gen(13)
    offsets = i32(cut([33, 0, 300, 128]))
    a, b = normal(gn, (461, 264)).half(), normal(gn, (4, 520, 264)).half()
    dc = normal(gn, (461, 520)).half()
    la, lb = normal(gn, (3, 16, 264)).half(), normal(gn, (3, 520, 16)).half()
    ad, sc = i32([i // 60 % 3 for i in range(461)]), torch.ones(3, device=DEV)
    ws = torch.empty(g.lora_workspace_size(461, 16), dtype=torch.uint8, device=DEV)

    def outs():
        return [torch.zeros((461, 520), dtype=F16, device=DEV), torch.zeros((4, 264, 520), dtype=F32, device=DEV),
                torch.zeros((461, 520), dtype=F16, device=DEV)]

    def calls(o):
        g.gemm_f16_grouped_bt(a, b, offsets, o[0])
        g.gemm_f16_grouped_wgrad(a, dc, offsets, o[1])
        g.gemm_f16_lora_bt(a, b[0], la, lb, ad, sc, o[2], workspace=ws)

    first = outs()
    calls(first)
    torch.cuda.synchronize()
    held = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        calls(held)
    for i in range(4):
        for t in held:
            t.fill_(float(i))
        torch.cuda.synchronize()
        graph.replay()
        (first[0].float() @ dc.float().t()).sum()
        torch.cuda.synchronize()
        for t, f in zip(held, first):
            assert torch.equal(t, f), i
