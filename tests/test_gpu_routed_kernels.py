"""Every kernel behind the products whose weight depends on the row, named
through LIBGEMM_CONFIG (it replaces the choice where that kernel takes the
operands), on ragged sizes: partial tiles of rows, columns and K, operands
narrower than a 16-byte piece, groups of a row or none, K long enough for the
adapters' slices. References and tolerances are those of test_gpu_routed.py."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from test_gpu_routed import F16, F32, run_f16, run_fp8, run_lora, run_wgrad, say

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")

GROUPED = ["grouped_pp_256", "grouped_pp_192", "grouped_pp_128", "grouped_ring", "grouped_tile_128", "grouped_tile_64"]
LORA = ["lora_pp_256", "lora_pp_192", "lora_ring", "lora_tile_128", "lora_tile_64"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(DEV)
    g.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("name", GROUPED)
def test_grouped_f16(name, bt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for sizes in ([1, 0, 63, 130], [193, 257, 0, 65], [449]):
        for n, k in ((256, 64), (264, 200), (520, 72), (64, 8)):
            say(f"{name} f16 {sizes} n {n} k {k} bt {bt}")
            run_f16(n + k, sizes, n, k, bt, F16, lead=1, tail=70)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("name", ["grouped_tile_128", "grouped_tile_64"])
def test_grouped_any_alignment(name, bt, monkeypatch):
    """K and N that cut 16-byte pieces at every place, and narrower ones."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for n, k in ((129, 193), (130, 67), (135, 391), (71, 9), (8, 129), (7, 129), (65, 7), (9, 8), (263, 1)):
        say(f"{name} f16 n {n} k {k} bt {bt}")
        run_f16(n * k, [1, 70, 0, 66], n, k, bt, F32, tail=3)
    for n, k in ((129, 193), (145, 391), (71, 17), (16, 129), (15, 129), (65, 15), (17, 16)):
        say(f"{name} fp8 n {n} k {k} bt {bt}")
        run_fp8(n + k, [1, 70, 0, 66], n, k, bt, False, F32)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("name", GROUPED)
def test_grouped_fp8(name, bt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for sizes, n, k, channel, out in (([1, 0, 63, 130], 272, 208, True, F16), ([193, 66], 512, 64, False, F32),
                                      ([257, 5], 80, 400, True, torch.float8_e4m3fn)):
        say(f"{name} fp8 {sizes} n {n} k {k} bt {bt} {out}")
        run_fp8(n + k, sizes, n, k, bt, channel, out, tail=1)


@pytest.mark.parametrize("kind", ["f16", (0, 0), (0, 1)])
@pytest.mark.parametrize("name", LORA)
def test_lora(name, kind, monkeypatch):
    """rows, N, K, rank: K of 1024 and more cuts the low-rank values into slices, 2056 unevenly."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    cases = ((65, 264, 1104, 5, 3, 30), (200, 100, 2064, 70, 4, 9), (900, 272, 1040, 16, 2, 300), (17, 80, 144, 9, 3, 1),
             (1, 520, 4112, 8, 2, 1))
    for i, (rows, n, k, rank, count, runs) in enumerate(cases if kind == "f16" else cases[1:4]):
        say(f"{name} {kind} {rows} x {n} x {k} rank {rank}")
        run_lora(i, rows, n, k, rank, count, runs, F16 if i % 2 else F32, kind)


@pytest.mark.parametrize("rows,k,rank", [(65, 8, 1), (66, 1023, 4), (300, 4096, 130), (4100, 1024, 33), (2050, 520, 64)])
def test_lora_slices(rows, k, rank):
    for out in (F16, F32):
        say(f"lora {rows} rows, K {k}, rank {rank}")
        run_lora(rows + k, rows, 72, k, rank, 5, max(1, rows // 7), out)


@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("name", ["wgrad_pp", "wgrad_tile_128", "wgrad_tile_64"])
def test_wgrad(name, out, monkeypatch):
    """Rows of every remainder of a step, operands cut at every place of a 16-byte piece or narrower than one, and
    C in whole 128-byte lines."""
    monkeypatch.setenv("LIBGEMM_CONFIG", name)
    for sizes in ([1, 0, 63, 64, 65], [31, 32, 33, 200], [257, 0, 321]):
        for m, n in ((64, 64), (72, 256), (264, 136), (129, 67), (65, 390), (8, 130), (7, 70), (300, 5), (1, 1)):
            say(f"{name} {sizes} m {m} n {n} {out}")
            run_wgrad(m + n, sizes, m, n, out, lead=2, tail=3)
