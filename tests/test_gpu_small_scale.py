"""FP8 results of the products with bias and activation whose output scale is
so small that its reciprocal is no FP32 number (below 2^-128): FP8(y / sOut) all
the same, zeros among them. z is the bias here (A is zero), so the quotients are
exact and the codes are compared bit for bit."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import CODE, FP8_MAX, as_bytes, codes_of
from test_gpu_norm import DEV, _gpu, say  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = ["bias_act_pp_256", "bias_act_pp_192", "bias_act_ring", "bias_act_tile_128", "bias_act_tile_64"]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("config", KERNELS)
def test_codes(config, fmt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    m, n, k = 70, 112, 64
    e = torch.randint(0, 20, (n,), generator=torch.Generator().manual_seed(3))
    part = torch.randint(-15, 16, (n,), generator=torch.Generator().manual_seed(4)).double()
    part[::9] = 0.0
    a = torch.zeros((m, k), dtype=torch.float8_e4m3fn, device=DEV)
    b = torch.ones((n, k), dtype=torch.float8_e4m3fn, device=DEV)
    one = torch.ones(1, device=DEV)
    for power in (-149, -140, -129, -128, -127, -126, -20):
        # multiples of FP32's least number that are small numbers of sOut, and one far past the format's range
        v = torch.ldexp(part, (e - 6 + power).clamp(min=-149))
        v[5] = 1.0
        bias, sout = v.float().to(DEV), torch.tensor([2.0 ** power], device=DEV)
        assert torch.equal(bias.double().cpu(), v) and sout.item() > 0
        for act in (g.ACT_NONE, g.ACT_RELU):
            for bt in (True, False):
                say(f"{config} {fmt} sOut 2^{power} activation {act} bt {bt}")
                c = torch.empty((m, n), dtype=CODE[fmt], device=DEV)
                f = g.gemm_fp8_bias_act_bt if bt else g.gemm_fp8_bias_act
                f(a, g.FMT_E4M3, b if bt else b.t().contiguous(), g.FMT_E4M3, one, one, c, bias=bias, act=act, sOut=sout)
                y = torch.where(v < 0, torch.zeros_like(v), v) if act else v
                w = (y / 2.0 ** power).clamp(-FP8_MAX[fmt], FP8_MAX[fmt])
                ref = as_bytes(codes_of(w, fmt)).to(DEV)
                got = as_bytes(c)
                got = torch.where(got == 0x80, torch.zeros_like(got), got)   # (-0: a zero of either sign)
                ref = torch.where(ref == 0x80, torch.zeros_like(ref), ref)
                assert torch.equal(got, ref.expand(m, n)), f"codes at sOut 2^{power}"
