"""8-bit z of the products' epilogues where z is exactly zero (by zero operands,
by sums that cancel, by an empty sum): scale 1, zero codes, for every kernel; and
FP8 products of small integers, which are exact in any order, so that every K tile
and the cut last one show."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import CODE, as_bytes, codes_of, mx_pack, powers, spread
from test_gpu_norm import DEV, F16, F32, _gpu, gen, say  # noqa: F401

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
KERNELS = ["bias_act_pp_256", "bias_act_pp_192", "bias_act_ring", "bias_act_tile_128", "bias_act_tile_64"]


def product(kind, bt, a, b, c, fa=E4, fb=E4, scale=1.0, **kw):
    """b[n, k]."""
    b = b if bt else b.t().contiguous()
    if kind == "f16":
        return (g.gemm_f16_bias_act_bt if bt else g.gemm_f16_bias_act)(a, b, c, **kw)
    fmt = {E4: g.FMT_E4M3, E5: g.FMT_E5M2}
    sa, sb = torch.full((1,), scale, device=DEV), torch.ones(1, device=DEV)
    return (g.gemm_fp8_bias_act_bt if bt else g.gemm_fp8_bias_act)(a, fmt[fa], b, fmt[fb], sa, sb, c, **kw)


def kept(m, n, zt):
    return (torch.full((m, n), 0xA5, dtype=torch.uint8, device=DEV).view(zt),
            torch.full((m, (n + 31) // 32), 0xA5, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("zt", [E4, E5], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["f16", "fp8"])
@pytest.mark.parametrize("config", KERNELS)
def test_zero(config, kind, zt, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    dt = F16 if kind == "f16" else E4
    gn = gen(1)
    for m, n, k, bt in ((1, 48, 64, True), (70, 112, 96, True), (70, 112, 96, False), (67, 61, 96, True), (300, 301, 64, True)):
        # zero rows beside others; in the others the halves of K cancel
        a = torch.randint(-8, 9, (m, k // 2), generator=gn, device=DEV).float()
        a[::3] = 0
        a = torch.cat([a, a], dim=1).to(dt)
        b = torch.randint(-8, 9, (n, k // 2), generator=gn, device=DEV).float()
        b = torch.cat([b, -b], dim=1).to(dt)
        c = torch.full((m, n), float("nan"), dtype=F16, device=DEV)
        z, zs = kept(m, n, zt)
        say(f"zero z {config} {kind} {m}x{n}x{k} bt {bt} {zt}")
        product(kind, bt, a, b, c, act=g.ACT_GELU, Z=z, Zscale=zs)
        assert bool((zs == 127).all()), "scales"
        assert bool(((as_bytes(z) & 0x7F) == 0).all()), "codes"
        assert bool((c == 0).all())


@pytest.mark.parametrize("zt", [E4, E5], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["f16", "fp8"])
def test_empty_sum(kind, zt):
    dt = F16 if kind == "f16" else E4
    for m, n in ((1, 40), (70, 131)):
        a, b = torch.empty((m, 0), dtype=dt, device=DEV), torch.empty((n, 0), dtype=dt, device=DEV)
        c = torch.full((m, n), float("nan"), device=DEV)
        z, zs = kept(m, n, zt)
        say(f"empty sum {kind} {m}x{n} {zt}")
        product(kind, True, a, b, c, act=g.ACT_SILU, Z=z, Zscale=zs)
        assert bool((zs == 127).all()) and bool((as_bytes(z) == 0).all()) and bool((c == 0).all())


def integers(gn, shape, most, dt):
    return torch.randint(-most, most + 1, shape, generator=gn, device=DEV).float().to(dt)


@pytest.mark.parametrize("fa,fb", [(E4, E4), (E4, E5), (E5, E4), (E5, E5)], ids=str)
@pytest.mark.parametrize("config", KERNELS)
def test_fp8_integers(config, fa, fb, monkeypatch):
    """Operands of -2 to 2: products and sums are whole numbers below 2^24, z is 2^-10 times one plus a multiple of 2^-10.
    Z and C come back exactly, and 8-bit Z bit for bit."""
    if config == "bias_act_pp_256" and (fa is E5 or fb is E5):
        config = "bias_act_pp_192"
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    gn = gen(7)
    for m, n, k, bt in ((3, 64, 4112, True), (200, 272, 1040, True), (130, 144, 528, False), (33, 80, 16, True)):
        a, b = integers(gn, (m, k), 2, fa), integers(gn, (n, k), 2, fb)
        bias = torch.randint(-4096, 4097, (n,), generator=gn, device=DEV).float() / 1024
        zr = (a.double() @ b.double().t().contiguous()) / 1024 + bias.double()
        for zt in (F32, E4):
            c = torch.empty((m, n), device=DEV)
            z, zs = (torch.empty((m, n), device=DEV), None) if zt is F32 else kept(m, n, zt)
            say(f"integers {config} {fa} x {fb} {m}x{n}x{k} bt {bt} Z {zt}")
            product("fp8", bt, a, b, c, fa, fb, 2.0 ** -10, bias=bias, Z=z, Zscale=zs)
            assert torch.equal(c.double(), zr), "C"
            if zt is F32:
                assert torch.equal(z.double(), zr), "Z"
            else:
                u, s = mx_pack(zr, "e4m3")
                assert torch.equal(powers(zs), s), "Z's scales"
                got, ref = as_bytes(z), as_bytes(codes_of(u, "e4m3"))
                assert torch.equal(got & 0x7F, ref & 0x7F) and torch.equal(z.float(), codes_of(u, "e4m3").float()), "Z's codes"
                assert float(spread(s, n).max()) < 2.0 ** 20 and z.dtype is CODE["e4m3"]


@pytest.mark.parametrize("m", [1, 3, 40, 520])
def test_fp8_weight_past_2_32(m):
    """A K-major FP8 weight of 4.4e9 codes, K = 512 * 128 + 16: whole numbers, exact in any order."""
    n, k, ends = 67000, 65552, 5
    gn = gen(m)
    a, w = integers(gn, (m, k), 1, E4), integers(gn, (2 * ends, k), 1, E4)
    # the cut last tile weighs most: leaving it out, or any whole tile, changes every sum
    w[:, -16:] = torch.ones((2 * ends, 16), device=DEV).to(E4)
    a[:, -16:] = torch.ones((m, 16), device=DEV).to(E4)
    b = torch.zeros((n, k), dtype=E4, device=DEV)
    b[:ends], b[-ends:] = w[:ends], w[-ends:]
    bias = torch.randint(-512, 513, (n,), generator=gn, device=DEV).float() / 256
    c, z = torch.empty((m, n), device=DEV), torch.empty((m, n), dtype=F16, device=DEV)
    say(f"{m} rows on a weight of {b.numel() >> 20} MiB")
    product("fp8", True, a, b, c, scale=2.0 ** -8, bias=bias, Z=z)
    cols = torch.cat([torch.arange(ends), torch.arange(n - ends, n)]).to(DEV)
    zr = a.double() @ w.double().t().contiguous() / 256 + bias[cols].double()
    assert torch.equal(c[:, cols].double(), zr), "C"
    assert torch.equal(z[:, cols], zr.float().half()), "Z"
    assert torch.equal(c[:, n // 2], bias[n // 2].expand(m)), "a weight of zeros: the bias alone"
    del b
    torch.cuda.empty_cache()
