"""Plain calls whose launch would take 2^32 threads or more, of which HIP runs
only the number modulo 2^32 without a word: they are refused."""
import pytest
import torch

import precision_dense_gemm_03_amd as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(DEV)
    g.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def ones(*shape, dtype=F16):
    return torch.ones(shape, dtype=dtype, device=DEV)


def zeros(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def one():
    return torch.ones(1, device=DEV)


CALLS = {
    "decode, K-major weight": lambda: g.gemm_f16_bt(ones(1, 1), ones((1 << 25) + 8, 1), zeros(1, (1 << 25) + 8)),
    "decode, row-major weight": lambda: g.gemm_f16(ones(1, 1), ones(1, 1 << 30), zeros(1, 1 << 30)),
    "narrow product": lambda: g.gemm_f16(ones((1 << 30) + 70, 1), ones(1, 1), zeros((1 << 30) + 70, 1)),
    "FP8 narrow product": lambda: g.gemm_fp8_scaled(torch.full(((1 << 30) + 70, 1), 0x38, dtype=torch.uint8, device=DEV),
                                                    torch.full((1, 1), 0x38, dtype=torch.uint8, device=DEV), one(), one(),
                                                    zeros((1 << 30) + 70, 1)),
    "weight re-layout": lambda: g.pack_b_kmajor(ones(1, 1 << 30), zeros(1 << 30, 1)),
    "transposed quantize": lambda: g.quantize_fp8_transposed(ones(1, (1 << 31) - 1, dtype=F32), one(),
                                                               zeros((1 << 31) - 1, 1, dtype=torch.uint8)),
}


@pytest.mark.parametrize("what", CALLS)
def test_launches_past_2_to_32_threads(what):
    """Refused, or right: every input is 1, every output 1 (code 0x38 in E4M3)."""
    print(what, flush=True)
    try:
        y = CALLS[what]()
    except g.GemmError as e:
        assert e.status == -5     # GEMM_ERR_LAUNCH
        return
    torch.cuda.synchronize()
    y = y.view(-1)
    for lo in range(0, y.numel(), 1 << 28):
        right = bool((y[lo:lo + (1 << 28)] == (1 if y.dtype != torch.uint8 else 0x38)).all())
        assert right, lo
