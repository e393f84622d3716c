"""Operand formats, FP8 outputs and column counts of the products whose weight
depends on the row, on every kernel: pairs with E5M2, E5M2 outputs, and
K-major weights whose columns are no multiple of a 16-byte piece. Each test
asserts that the named kernel is the one the call launches. References and
tolerances are those of test_gpu_routed.py; the last test's sums are exact."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from test_gpu_routed import F16, F32, cut, fp8, i32, run_f16, run_fp8, run_lora, say

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
CODE = {F32: g.OUT_F32, F16: g.OUT_F16, E4M3: g.OUT_E4M3, E5M2: g.OUT_E5M2}

GROUPED = ["grouped_pp_256", "grouped_pp_192", "grouped_pp_128", "grouped_ring", "grouped_tile_128", "grouped_tile_64"]
MIXED = ["grouped_pp_192", "grouped_ring", "grouped_tile_128", "grouped_tile_64"]   # pairs with E5M2: one tall kernel
LORA = ["lora_pp_192", "lora_ring", "lora_tile_128", "lora_tile_64"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(DEV)
    g.lib()
    yield
    torch.cuda.synchronize()


def f16(name, sizes, n, k, bt, out, lead, tail):
    rows = lead + sum(sizes) + tail
    assert g.select_config_grouped(g.KIND_F16, CODE[out], rows, n, k, len(sizes), b_kmajor=bt) == name
    say(f"{name} f16 {sizes} n {n} k {k} bt {bt} {out}")
    run_f16(n + k, sizes, n, k, bt, out, lead=lead, tail=tail)


def f8(name, sizes, n, k, bt, channel, out, fa, fb, lead, tail):
    rows = lead + sum(sizes) + tail
    assert g.select_config_grouped(g.KIND_FP8, CODE[out], rows, n, k, len(sizes), fa, fb, bt) == name
    say(f"{name} fp8 {(fa, fb)} {sizes} n {n} k {k} bt {bt} channel {channel} {out}")
    run_fp8(n + k, sizes, n, k, bt, channel, out, fa, fb, lead=lead, tail=tail)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("pair", [(0, 1), (1, 0), (1, 1)], ids=str)
@pytest.mark.parametrize("name", MIXED)
def test_pairs_with_e5m2(name, pair, bt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    f8(name, [1, 0, 63, 130], 272, 208, bt, True, F16, *pair, 1, 3)
    f8(name, [200, 66], 336, 80, bt, False, F32, *pair, 0, 0)
    f8(name, [17, 194], 144, 400, bt, pair == (0, 1), E5M2, *pair, 2, 1)
    f8(name, [40, 3], 80, 64, bt, pair == (1, 0), E4M3, *pair, 0, 5)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("name", GROUPED)
def test_e5m2_outputs(name, bt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    f8(name, [193, 0, 66], 512, 64, bt, False, E5M2, 0, 0, 3, 1)
    f8(name, [300, 5], 144, 272, bt, True, E5M2, 0, 0, 0, 2)


@pytest.mark.parametrize("name", GROUPED)
def test_kmajor_columns_that_cut_a_piece(name, monkeypatch):
    """N of no whole 16 bytes of C (element stores), and of whole ones for one output type only."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for n, k in ((1001, 72), (1004, 64), (255, 136), (3, 64)):
        for out in (F16, F32):
            f16(name, [193, 257, 0, 65], n, k, True, out, 1, 70)
    for n, k, channel, out in ((1001, 80, True, F16), (1004, 64, False, E5M2), (257, 144, True, E4M3),
                               (1004, 64, True, F32), (3, 64, False, F32), (3, 64, True, F16)):
        f8(name, [193, 66], n, k, True, channel, out, 0, 0, 1, 2)


@pytest.mark.parametrize("pair", [(0, 1), (1, 0), (1, 1)], ids=str)
@pytest.mark.parametrize("name", LORA)
def test_adapters_beside_pairs_with_e5m2(name, pair, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for rows, n, k, rank, count, runs, out in ((200, 101, 528, 70, 4, 9, F32), (17, 80, 144, 9, 3, 1, F16),
                                               (300, 272, 80, 16, 2, 100, F16)):
        assert g.select_config_lora(g.KIND_FP8, CODE[out], rows, n, k, rank, count, *pair) == name
        say(f"{name} {pair} {rows} x {n} x {k} rank {rank} {out}")
        run_lora(rows, rows, n, k, rank, count, runs, out, pair)


@pytest.mark.parametrize("name,sizes,n,k,pair,bt", [
    ("grouped_pp_192", [700, 0, 1500, 333, 64, 1000, 471, 28], 4096, 1024, (1, 0), True),
    ("grouped_pp_192", [700, 0, 1500, 333, 64, 1000, 471, 28], 4096, 1024, (1, 0), False),
    ("grouped_pp_192", [700, 0, 1500, 333, 64, 1000, 471, 28], 2048, 2048, (0, 1), False),
    ("grouped_ring", [16] * 60 + [0, 50, 14, 0], 2048, 4096, (1, 0), True),
    ("grouped_pp_256", [4100, 3900, 4000, 4192], 4096, 1024, (0, 0), True)])
def test_chosen_by_the_rules(name, sizes, n, k, pair, bt):
    """Sizes of training and serving, where the rules pick the kernel. Codes of small whole numbers: every product and
    sum is exact."""
    assert g.select_config_grouped(g.KIND_FP8, g.OUT_F32, sum(sizes), n, k, len(sizes), *pair, bt) == name
    gn = torch.Generator(device=DEV).manual_seed(n)
    a = torch.randint(-2, 3, (sum(sizes), k), generator=gn, device=DEV).float()
    b = torch.randint(-2, 3, (len(sizes), n, k) if bt else (len(sizes), k, n), generator=gn, device=DEV).float()
    sa, sb = torch.tensor([0.5], device=DEV), 2.0 ** torch.arange(len(sizes), device=DEV).remainder(3).float()
    c = torch.full((sum(sizes), n), 7.0, dtype=F32, device=DEV)
    offsets = cut(sizes)
    say(f"{name} {pair} {sum(sizes)} rows n {n} k {k} bt {bt}")
    call = g.gemm_fp8_grouped_bt if bt else g.gemm_fp8_grouped
    call(fp8(a, pair[0]), pair[0], fp8(b, pair[1]), pair[1], i32(offsets), sa, sb, c)
    for e in range(len(sizes)):
        lo, hi = offsets[e], offsets[e + 1]
        w = b[e].t().contiguous() if bt else b[e]
        assert torch.equal(c[lo:hi], (a[lo:hi] @ w) * (sa * sb[e])), e
