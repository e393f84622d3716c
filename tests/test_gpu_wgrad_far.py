"""The gradient to the weights from 8-bit values on every kernel, operands of 4.36e9
elements: their end rows make the sum, the rows between are zero."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import REL, values
from routed_ref import check
from test_gpu_dense_far import _gpu, ends, long  # noqa: F401
from test_gpu_norm import DEV, gen, say

pytestmark = pytest.mark.gpu

ROWS, WIDE, NARROW = 1060003, 4112, 64


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("wide", ["codes", "halves"])
@pytest.mark.parametrize("config", ["wgrad_pp", "wgrad_tile_128", "wgrad_tile_64", "wgrad_tile_64_split"])
def test_far(config, wide, second, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    gn = gen(9)
    m, n = (WIDE, NARROW) if wide == "codes" else (NARROW, WIDE)
    q, s = g.quantize_mx_fp8(long(ROWS, m, gn))
    b = long(ROWS, n, gn)
    c = torch.full((n, m) if second else (m, n), float("nan"), device=DEV)
    say(f"{config}, {q.numel() >> 20} MiB of codes, {b.numel() * 2 >> 20} MiB of halves, second {second}")
    assert g.select_config_mx_wgrad(g.OUT_F32, ROWS, m, n, 1, second) == config
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, b, c, q_second=second)
    xv, bv = values(ends(q), ends(s), "e4m3"), ends(b).double()
    v, mag = xv.t().contiguous() @ bv, xv.abs().t().contiguous() @ bv.abs()
    check(c.t() if second else c, v, REL * mag, "C")
    del q, s, b
    torch.cuda.empty_cache()
