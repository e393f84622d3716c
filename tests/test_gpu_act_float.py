"""Activations whose result is FP32, through every kernel's epilogue (A is zero:
z is the bias exactly): relative errors over the whole range, small tails among
them; and the derivative's tail.

Bounds, in units u = 2^-24 of the value, fixed before the first run. The hardware's
2^x and 1/x are off by 1 ulp, 2 u. SILU and the tanh form: exponential 2 u, what its
argument's remainder brings 1 u and the product with that 1 u, sum 1 u, reciprocal
2 u, product with z 1 u: 8 u, 2^-21. GELU: the fitted polynomial 1.2 u, its evaluation
3 u (the partial sums' sizes over the result's), t = 1 / (1 + 0.35 a) 3 u, which count
2.3 times (the slope of the logarithm of t times the polynomial), exponential 4 u as
above, three products and the difference from 1 at 1 u each: 20 u. Below 2^-120 results may be flushed."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import act
from routed_ref import check
from test_gpu_norm import DEV, F16, F32, _gpu, gen, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu

ACT = {"gelu": g.ACT_GELU, "gelu_tanh": g.ACT_GELU_TANH, "silu": g.ACT_SILU}
LEAST = {"gelu": -12.5, "gelu_tanh": -9.5, "silu": -80.0}   # (results of 2^-110 and more)
BOUND = {"gelu": 20 * 2.0 ** -24, "gelu_tanh": 2.0 ** -21, "silu": 2.0 ** -21}
KERNELS = ["bias_act_pp_256", "bias_act_pp_192", "bias_act_ring", "bias_act_tile_128", "bias_act_tile_64"]


def exact(z, name):
    """act in forms that keep a tail's bits in 64 bits."""
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / 2.0 ** 0.5)
    if name == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * (2.0 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z / (1.0 + torch.exp(-z))


def range_of(name):
    z = torch.cat([torch.linspace(LEAST[name], 40.0, 60001), torch.linspace(LEAST[name], 0.0, 60001),
                   torch.linspace(-1.0, 1.0, 20001), torch.linspace(-1e-3, 1e-3, 1001),
                   torch.tensor([0.0, -0.0, 1e3, -1e3, 1e19, -1e19, 3e38, -3e38])])
    return z.to(DEV)


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("kind", ["f16", "fp8"])
@pytest.mark.parametrize("config", KERNELS)
def test_results(config, kind, name, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    z = range_of(name)
    n, k = z.numel(), 64
    dt = F16 if kind == "f16" else torch.float8_e4m3fn
    a, b = torch.zeros((2, k), dtype=dt, device=DEV), torch.zeros((n, k), dtype=dt, device=DEV)
    c = torch.empty((2, n), device=DEV)
    say(f"{config} {kind} {name}: {n} values")
    if kind == "f16":
        g.gemm_f16_bias_act_bt(a, b, c, bias=z, act=ACT[name])
    else:
        one = torch.ones(1, device=DEV)
        g.gemm_fp8_bias_act_bt(a, g.FMT_E4M3, b, g.FMT_E4M3, one, one, c, bias=z, act=ACT[name])
    zd = z.double()
    far = zd.abs() > 500
    y = torch.where(far, zd.clamp(min=0), exact(zd.clamp(-500, 500), name))
    check(c, y.expand(2, -1), (y.abs() * BOUND[name] + 2.0 ** -120).expand(2, -1), name)


@pytest.mark.parametrize("name", list(ACT))
def test_one_row(name):
    """The decode kernel, and NaN and infinities."""
    z = range_of(name)
    z = torch.cat([z, torch.tensor([float("inf"), float("nan")], device=DEV)])
    n = z.numel()
    a, b = torch.zeros((1, 64), dtype=F16, device=DEV), torch.zeros((n, 64), dtype=F16, device=DEV)
    assert g.select_config_bias_act(g.KIND_F16, g.OUT_F32, 1, n, 64, b_kmajor=1) == "bias_act_gemv"
    c = torch.empty((1, n), device=DEV)
    say(f"decode {name}")
    g.gemm_f16_bias_act_bt(a, b, c, bias=z, act=ACT[name])
    assert c[0, -2].item() == float("inf") and bool(c[0, -1].isnan())
    zd = z[:-2].double()
    far = zd.abs() > 500
    y = torch.where(far, zd.clamp(min=0), exact(zd.clamp(-500, 500), name))
    check(c[0, :-2], y, y.abs() * BOUND[name] + 2.0 ** -120, name)


@pytest.mark.parametrize("name", list(ACT))
def test_definitions_agree(name):
    """The form of `exact` is the definition."""
    z = torch.linspace(-6.0, 6.0, 1001, dtype=torch.float64)
    assert float((exact(z, name) - act(z, name)).abs().max()) < 1e-14


def test_derivative_tail():
    """GELU's derivative P(z) + z p(z) keeps its relative precision down to -7: P by a polynomial of 2.7e-7, both terms by
    an exponential whose argument z^2 / 2 takes three roundings (the square, the factor, their product)."""
    z = torch.linspace(-7.0, 0.0, 70001, device=DEV).reshape(1, -1)
    say("slope tail")
    dz, _ = g.bias_act_backward(torch.ones_like(z), z, g.ACT_GELU)
    zd = z.double()
    p, q = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5, 0.5 * torch.special.erfc(-zd / 2.0 ** 0.5)
    check(dz, q + zd * p, (q + zd.abs() * p) * (2.0 ** -20 + 1.5 * zd * zd * 2.0 ** -24), "slope")
