"""GPU parity of the products with bias, activation and residual
(gemm_*_bias_act*) and of the epilogue's gradient (bias_act_backward), against
64-bit references (dense_ref.py). Each test prints the case it is about to
launch."""
import numpy as np
import pytest
import torch

import oracle as orc
import precision_dense_gemm_03_amd as g
from dense_ref import (ACTS, CODE, FP8_MAX, REL, STEEPEST, act, act_error, code_step, mx_scale, powers, slope, slope_error,
                       spread, stored, values)
from parity import fp8_dot_allowance
from routed_ref import check
from test_gpu_norm import _gpu, gen, guarded, input_of, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32 = torch.float16, torch.float32
OUT = {F32: g.OUT_F32, F16: g.OUT_F16, torch.float8_e4m3fn: g.OUT_E4M3, torch.float8_e5m2: g.OUT_E5M2}
NAME = {torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}
ACT = {"none": g.ACT_NONE, "relu": g.ACT_RELU, "gelu": g.ACT_GELU, "gelu_tanh": g.ACT_GELU_TANH, "silu": g.ACT_SILU}


def check_held(z, zscale, zref, zerr, zt):
    """A stored pre-activation within zerr and its own rounding."""
    if zt in (F16, F32):
        check(z, zref, zerr + stored(zref, zt), "Z")
        return
    fmt = NAME[zt]
    cols = zref.shape[1]
    blocks = torch.nn.functional.pad(zref.abs(), (0, -cols % 32)).reshape(zref.shape[0], -1, 32)
    errs = torch.nn.functional.pad(zerr.expand_as(zref), (0, -cols % 32)).reshape(zref.shape[0], -1, 32)
    got = powers(zscale)
    lo = mx_scale((blocks - errs).clamp(min=0).amax(dim=2), fmt)
    hi = mx_scale((blocks + errs).amax(dim=2), fmt)
    fine = (got >= lo) & (got <= hi) | ((blocks - errs).amax(dim=2) <= 0)
    assert bool(fine.all()), "Z's scales"
    check(values(z, zscale, fmt), zref, zerr + code_step(zref.abs() + zerr, spread(got, cols), fmt), "Z's values")


_allowances = {}


def allowance(key, a, codes_b, bt, fa, fb, rows):
    """fp8_dot_allowance of operands that the key determines."""
    if key not in _allowances:
        _allowances[key] = fp8_dot_allowance(a.view(torch.uint8).cpu().numpy()[rows], codes_b.T if bt else codes_b,
                                             fmt_a=orc.FMT_E4M3 if fa == "e4m3" else orc.FMT_E5M2,
                                             fmt_b=orc.FMT_E4M3 if fb == "e4m3" else orc.FMT_E5M2)
    return _allowances[key]


def run(kind, m, n, k, bt, out, name, bias=True, res=None, zt=None, channel=True, fa="e4m3", fb="e4m3", offset=0,
        config=None, zero=None, rows=None):
    """One product against the reference; FP8 products allow for the matrix cores' alignment (parity.py)."""
    gn = gen(m + 3 * n + 7 * k)
    if kind == "f16":
        a = input_of(normal(gn, (m, k)).half(), offset)
        b = input_of((normal(gn, (n, k) if bt else (k, n)) / max(k, 1) ** 0.5).half(), offset)
        av, bv = a.double(), b.double().t().contiguous() if bt else b.double()
        v, s = av @ bv, av.abs() @ bv.abs()
        sa = sb = None
    else:
        a = input_of((normal(gn, (m, k)) * FP8_MAX[fa] / 8).clamp(-FP8_MAX[fa], FP8_MAX[fa]).to(CODE[fa]), offset)
        b = input_of((normal(gn, (n, k) if bt else (k, n)) * FP8_MAX[fb] / 8).clamp(-FP8_MAX[fb], FP8_MAX[fb]).to(CODE[fb]),
                     offset)
        sa = (torch.rand((m if channel else 1,), generator=gn, device=DEV) + 0.5) * (8 / FP8_MAX[fa])
        sb = (torch.rand((n if channel else 1,), generator=gn, device=DEV) + 0.5) * (8 / FP8_MAX[fb] / max(k, 1) ** 0.5)
        av, bv = a.double(), b.double().t().contiguous() if bt else b.double()
        f = (sa.double()[:, None] * sb.double()[None, :]) if channel else sa.double() * sb.double()
        codes_b = b.view(torch.uint8).cpu().numpy()
        t = np.zeros((m, n))
        if k:
            at = slice(None) if rows is None else rows
            t[at] = allowance((m, n, k, bt, fa, fb, str(rows)), a, codes_b, bt, fa, fb, at)
        v, s = (av @ bv) * f, (av.abs() @ bv.abs() + torch.from_numpy(t).to(DEV) / REL) * f
    bi = normal(gn, (n,)) if bias else None
    r = input_of(normal(gn, (m, n)).to(res), offset) if res else None
    zref = v if bi is None else v + bi.double()
    zerr = REL * s + (zref.abs() + v.abs()) * 2.0 ** -22
    c, guard_c = guarded((m, n), out, offset)
    z, zscale, guards = None, None, [guard_c]
    if zt is not None:
        z, gz = guarded((m, n), zt, offset)
        guards.append(gz)
        if zt in NAME:
            zscale, gs = guarded((m, (n + 31) // 32), torch.uint8, offset)
            guards.append(gs)
    sout = torch.full((1,), 4.0 / FP8_MAX[NAME[out]], device=DEV) if out in NAME else None
    if config:
        kd = g.KIND_F16 if kind == "f16" else g.KIND_FP8
        assert g.select_config_bias_act(kd, OUT[out], m, n, k, g.FMT_E5M2 if fa == "e5m2" else 0,
                                        g.FMT_E5M2 if fb == "e5m2" else 0, 1 if bt else 0,
                                        -1 if zt is None else OUT[zt]) == config
    kw = dict(bias=bi, act=ACT[name], residual=r, Z=z, Zscale=zscale)
    if kind == "f16":
        (g.gemm_f16_bias_act_bt if bt else g.gemm_f16_bias_act)(a, b, c, **kw)
    else:
        (g.gemm_fp8_bias_act_bt if bt else g.gemm_fp8_bias_act)(
            a, g.FMT_E5M2 if fa == "e5m2" else g.FMT_E4M3, b, g.FMT_E5M2 if fb == "e5m2" else g.FMT_E4M3, sa, sb, c,
            channel=channel, sOut=sout, **kw)
    y = act(zref, name)
    err = STEEPEST * zerr + act_error(zref, name)
    if r is not None:
        y = y + r.double()
        err = err + y.abs() * 2.0 ** -23
    keep = slice(None) if rows is None else torch.as_tensor(rows, device=DEV)
    if out in NAME:
        w = y / sout.double()
        e = err / sout.double() + w.abs() * 2.0 ** -22
        w = w.clamp(-FP8_MAX[NAME[out]], FP8_MAX[NAME[out]])
        check(c[keep].double() if rows is None else c.view(torch.uint8)[keep].view(out).double(), w[keep],
              (e + code_step(w.abs() + e, torch.ones_like(w), NAME[out]))[keep], "C")
    else:
        check(c[keep], y[keep], (err + stored(y.abs() + err, out))[keep], "C")
    if zt is not None and rows is None:
        check_held(z, zscale, zref, zerr, zt)
    for f in guards:
        f()


E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
SHAPES = [(1, 1, 1), (1, 4096, 512), (1, 33, 64), (3, 7, 5), (4, 1000, 256), (5, 64, 64), (16, 200, 130), (33, 256, 96),
          (64, 65, 520), (100, 129, 65), (130, 272, 72), (257, 96, 33), (300, 520, 136)]


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_f16(m, n, k, bt):
    for i, (out, name, res, zt) in enumerate(((F16, "gelu", None, None), (F32, "silu", F16, F16), (F16, "relu", F32, E4),
                                              (F32, "gelu_tanh", None, E5), (F16, "none", F16, F32))):
        say(f"f16 {m}x{n}x{k} bt {bt} {out} {name} residual {res} Z {zt}")
        run("f16", m, n, k, bt, out, name, bias=i != 1, res=res, zt=zt)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_fp8(m, n, k, bt):
    for i, (out, name, res, zt, channel) in enumerate(((F16, "silu", F16, None, True), (E4, "gelu", None, E4, False),
                                                       (E5, "relu", F32, F16, True), (F32, "gelu_tanh", None, E5, True))):
        say(f"fp8 {m}x{n}x{k} bt {bt} {out} {name} residual {res} Z {zt} channel {channel}")
        run("fp8", m, n, k, bt, out, name, bias=i != 2, res=res, zt=zt, channel=channel)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("bt", [True, False])
def test_fp8_formats(fa, fb, bt):
    for m, n, k in ((1, 64, 128), (4, 96, 64), (70, 130, 96), (40, 64, 256)):
        say(f"fp8 {fa} x {fb} {m}x{n}x{k} bt {bt}")
        run("fp8", m, n, k, bt, F16, "gelu", res=F16, zt=E4 if m > 4 else None, fa=fa, fb=fb)


KERNELS = ["bias_act_pp_256", "bias_act_pp_192", "bias_act_ring", "bias_act_tile_128", "bias_act_tile_64"]


@pytest.mark.parametrize("kind", ["f16", "fp8"])
@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("config", KERNELS)
def test_kernels(config, bt, kind, monkeypatch):
    """Every kernel by name: tiles cut in rows and columns, partial and single K tiles, every output and kept type."""
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    shapes = ((5, 48, 32), (200, 272, 80), (257, 336, 1040), (70, 64, 16)) if kind == "f16" else \
        ((5, 48, 32), (200, 272, 80), (193, 336, 1040))
    outs = ((F16, "gelu", None, E4), (F32, "silu", F32, None), (F16, "none", F16, F16), (F32, "relu", F16, E5),
            (F16, "gelu_tanh", F32, F32))
    if kind == "fp8":
        outs += ((E4, "gelu", F16, None), (E5, "silu", F32, E4))
    for m, n, k in shapes:
        for i, (out, name, res, zt) in enumerate(outs):
            say(f"{config} {kind} {m}x{n}x{k} bt {bt} {out} {name} residual {res} Z {zt}")
            run(kind, m, n, k, bt, out, name, bias=i != 2, res=res, zt=zt, channel=i % 2 == 0, config=config)


@pytest.mark.parametrize("config", KERNELS)
def test_kernels_odd_columns(config, monkeypatch):
    """K-major weights of an odd number of rows: rows of C that start anywhere."""
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    for kind in ("f16", "fp8"):
        for n in (3, 61, 255, 301):
            for out, res, zt in ((F16, F16, E4), (F32, F32, F16), (F16, None, E5)):
                say(f"{config} {kind} 67x{n}x96 {out} residual {res} Z {zt}")
                run(kind, 67, n, 96, True, out, "silu", res=res, zt=zt, config=config)
        if kind == "fp8":
            say(f"{config} fp8 67x301x96 e4m3")
            run("fp8", 67, 301, 96, True, E4, "gelu", res=F16, config=config)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("config", ["bias_act_pp_192", "bias_act_ring", "bias_act_tile_128", "bias_act_tile_64"])
def test_kernels_formats(config, fa, fb, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    for bt in (True, False):
        say(f"{config} {fa} x {fb} bt {bt}")
        run("fp8", 90, 144, 208, bt, F16, "gelu", res=F16, zt=E4, fa=fa, fb=fb, config=config)


def test_decode_kernels():
    """One FP16 row on the decode kernel, and the few rows beside it, with every output."""
    for kind, m, n, k in (("f16", 1, 1003, 520), ("f16", 1, 8, 4096), ("f16", 1, 77, 65), ("f16", 2, 64, 520),
                          ("fp8", 1, 130, 528), ("fp8", 3, 77, 256), ("fp8", 4, 64, 65)):
        one = "bias_act_gemv" if kind == "f16" and m == 1 else None
        for out, name, res, zt in ((F16, "gelu", F16, F16), (F32, "silu", F32, F32), (F16, "none", None, None)):
            say(f"decode {kind} {m}x{n}x{k} {out}")
            run(kind, m, n, k, True, out, name, res=res, zt=zt, config=one)
        if kind == "fp8":
            run(kind, m, n, k, True, E4, "relu", res=F16, channel=False)


@pytest.mark.parametrize("kind", ["f16", "fp8"])
def test_unaligned(kind):
    for bt in (True, False):
        for m, n, k in ((1, 40, 48), (65, 96, 64), (130, 50, 33)):
            say(f"{kind} unaligned {m}x{n}x{k} bt {bt}")
            run(kind, m, n, k, bt, F16, "gelu", res=F16, zt=E4, offset=1)
            run(kind, m, n, k, bt, F32, "silu", res=F32, zt=F16, offset=3)


@pytest.mark.parametrize("name", ACTS)
def test_empty_sum(name):
    """K = 0: z is the bias."""
    for kind in ("f16", "fp8"):
        for m, n in ((1, 40), (70, 131)):
            say(f"{kind} {m}x{n}x0 {name}")
            run(kind, m, n, 0, True, F16, name, res=F16, zt=E4, channel=True)
            run(kind, m, n, 0, False, F32, name, bias=False, zt=F16)


@pytest.mark.parametrize("m,n,k", [(512, 1024, 768), (3000, 1040, 200), (700, 2048, 4096), (2100, 2304, 64)])
def test_large(m, n, k):
    """Sizes at which the rules choose the large tiles; every element in FP16, sampled rows in FP8."""
    for bt in (True, False):
        say(f"f16 {m}x{n}x{k} bt {bt}")
        run("f16", m, n, k, bt, F16, "gelu", res=F16, zt=E4)
    say(f"fp8 {m}x{n}x{k}")
    run("fp8", m, n, k, True, F16, "gelu_tanh", res=F16, rows=[0, 1, m // 2, m - 2, m - 1])


def test_special_values():
    """NaN and infinities in an input row, the bias and the residual reach their own elements only."""
    gn = gen(2)
    m, n, k = 70, 96, 64
    a, b = normal(gn, (m, k)).half(), normal(gn, (n, k), 0.1).half()
    a[3] = float("nan")
    bias = normal(gn, (n,))
    bias[7], bias[40], bias[41] = float("nan"), float("inf"), -float("inf")
    res = normal(gn, (m, n)).half()
    res[9, 50] = float("inf")
    for name in ACTS:
        for config in KERNELS:
            say(f"special values {config} {name}")
            import os
            os.environ["LIBGEMM_CONFIG"] = config
            try:
                c = torch.empty((m, n), device=DEV)
                z = torch.empty((m, n), dtype=torch.float8_e4m3fn, device=DEV)
                zs = torch.empty((m, 3), dtype=torch.uint8, device=DEV)
                g.gemm_f16_bias_act_bt(a, b, c, bias=bias, act=ACT[name], residual=res, Z=z, Zscale=zs)
            finally:
                del os.environ["LIBGEMM_CONFIG"]
            assert bool(c[3].isnan().all()) and bool(c[:, 7].isnan().all())
            rows = [i for i in range(m) if i != 3]
            assert bool((c[rows, 40] == float("inf")).all())
            if name == "none":
                assert bool((c[rows, 41] == -float("inf")).all())
            cols = [i for i in range(n) if i not in (7, 40, 41)]
            rest = c[rows][:, cols]
            assert int((~rest.isfinite()).sum()) == 1 and c[9, 50].item() == float("inf")
            zv = values(z, zs, "e4m3")
            assert bool(zv[3].isnan().all()) and bool(zv[:, [7, 40, 41]].isnan().all())
            ok = zv[rows][:, cols]
            v = (a[rows].double() @ b.double().t().contiguous() + bias.double())[:, cols]
            assert bool(((ok - v).abs() <= v.abs() * 2.0 ** -4 + 0.02).all())   # (a scale of at most 8 / 448 * 2: step 2^-10 of it)


def test_activation_range():
    """Every activation from -40 to 40 and at large values, through the epilogue (K = 0: z is the bias)."""
    z = torch.cat([torch.linspace(-40, 40, 8001), torch.linspace(-1, 1, 2001), torch.tensor([1e4, -1e4, 3e38, -3e38, 0.0, -0.0])])
    bias = z.to(DEV)
    n = bias.numel()
    a, b = torch.empty((3, 0), dtype=F16, device=DEV), torch.empty((n, 0), dtype=F16, device=DEV)
    zd = bias.double()
    for name in ACTS:
        say(f"activation {name}")
        c = torch.empty((3, n), device=DEV)
        g.gemm_f16_bias_act_bt(a, b, c, bias=bias, act=ACT[name])
        big = zd.abs() > 1e3
        y = torch.where(big, torch.where(zd > 0, zd, zd if name == "none" else torch.zeros_like(zd)), act(zd, name))
        e = torch.where(big, zd.abs() * 2.0 ** -22, act_error(zd, name) + y.abs() * 2.0 ** -23)
        check(c, y.expand(3, -1), (e + 2.0 ** -126 * 64).expand(3, -1), name)


# ------------------------------------------------------------------- gradient

def run_backward(rows, cols, dtype, zt, name, dbias=True, dz=True, offset=0):
    gn = gen(rows + 5 * cols)
    zx = normal(gn, (rows, cols), 2.0)
    zs = None
    if zt in NAME:
        z = torch.empty((rows, cols), dtype=zt, device=DEV)
        _, zs = g.quantize_mx_fp8(zx.half(), g.FMT_E4M3 if zt == E4 else g.FMT_E5M2, q=z)
        zv = values(z, zs, NAME[zt])
        zs = input_of(zs, offset)
    else:
        z = zx.to(zt)
        zv = z.double()
    z = input_of(z, offset)
    dy = input_of(normal(gn, (rows, cols)).to(dtype), offset)
    out, guard = guarded((rows, cols), dtype, offset)
    db, guard_b = guarded((cols,), F32, offset)
    n = max(16, g.bias_act_backward_workspace_size(rows, cols))
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    g.bias_act_backward(dy, z, ACT[name], dZ=out, dbias=db if dbias else None, Zscale=zs, workspace=ws[:n])
    assert bool((ws[n:] == 0xA5).all()), "past the workspace"
    d = dy.double()
    ref, err = d * slope(zv, name), d.abs() * slope_error(zv, name)
    check(out, ref, err + ref.abs() * 2.0 ** -23 + stored(ref.abs() + err, dtype), "dZ")
    if dbias:
        check(db, ref.sum(dim=0), REL * ref.abs().sum(dim=0) + err.sum(dim=0) + 2.0 ** -120, "dbias")
    else:
        assert bool((db.view(torch.uint8) == 0xA5).all())
    guard(), guard_b()


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("zt", [F16, F32, E4, E5], ids=str)
def test_backward(zt, name):
    for rows, cols in ((1, 1), (3, 7), (2, 64), (65, 100), (300, 33), (1000, 520), (9, 4100), (4099, 24)):
        for dtype in (F16, F32):
            say(f"act backward {rows}x{cols} {dtype} Z {zt} {name}")
            run_backward(rows, cols, dtype, zt, name)


def test_backward_forms():
    for cols in (40, 1000):
        say(f"act backward without dbias, unaligned, cols {cols}")
        run_backward(50, cols, F16, E4, "gelu", dbias=False)
        run_backward(50, cols, F16, E4, "gelu", offset=1)
        run_backward(50, cols, F32, F16, "silu", offset=3)
    say("act backward: column sums alone")
    dy = normal(gen(1), (777, 130)).half()
    db, ws = torch.empty(130, device=DEV), torch.empty(g.bias_act_backward_workspace_size(777, 130), dtype=torch.uint8, device=DEV)
    st = g.lib().bias_act_backward(dy.data_ptr(), g.OUT_F16, None, None, 0, g.ACT_NONE, None, db.data_ptr(), 777, 130,
                                   ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    check(db, dy.double().sum(dim=0), REL * dy.double().abs().sum(dim=0), "dbias")
    say("act backward, no rows")
    db = torch.full((9,), 4.0, device=DEV)
    e = torch.empty((0, 9), device=DEV)
    g.bias_act_backward(e, e, g.ACT_GELU, dbias=db)
    assert bool((db == 0).all())


def test_backward_large_rows():
    for rows, cols in ((20000, 64), (3000, 4096)):
        say(f"act backward {rows}x{cols}")
        run_backward(rows, cols, F16, E4, "gelu")


@pytest.mark.parametrize("name", ACTS)
def test_gradient_against_differences(name):
    """dZ against central differences of the activation in 64 bits (relu away from its corner)."""
    gn = gen(6)
    z = normal(gn, (40, 200), 2.0)
    if name == "relu":
        z = torch.where(z.abs() < 0.01, torch.full_like(z, 0.5), z)
    dy, e = normal(gn, (40, 200)), 1e-5
    say(f"act gradient against differences {name}")
    dz, _ = g.bias_act_backward(dy, z, ACT[name])
    d = (act(z.double() + e, name) - act(z.double() - e, name)) / (2 * e) * dy.double()
    # e^2 / 6 times the third derivative (at most 2), the difference's rounding |z| 2^-52 / e, and the kernel's own
    tol = dy.double().abs() * (slope_error(z.double(), name) + 1e-9 + z.double().abs() * 2.0 ** -51 / e) + d.abs() * 2.0 ** -22
    check(dz, d, tol, name)


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slope_range(name):
    """Derivatives from -40 to 40, at the largest numbers and at infinities (1 and 0); NaN gives NaN (relu: 0)."""
    large = torch.tensor([1e3, 1e4, 65504.0, 1e8, 1e10, 1e13, 1e19, 1e30, 3e38, float("inf")])
    z = torch.cat([torch.linspace(-40, 40, 8000), large, -large, torch.tensor([float("nan"), 0.0])]).to(DEV)
    for zt in (F32, F16):
        for cols in (z.numel(), 7):
            say(f"slope {name} {zt} {cols}")
            zz = (z if cols != 7 else z[-7 * 3:].reshape(3, 7)).reshape(-1, cols).to(zt)
            dy = torch.ones(zz.shape, device=DEV)
            dz, _ = g.bias_act_backward(dy, zz, ACT[name])
            nan = zz.isnan()
            assert torch.equal(dz[nan], torch.zeros_like(dz[nan])) if name == "relu" else bool(dz[nan].isnan().all())
            zd = torch.where(nan, torch.zeros_like(zz), zz).double()
            far = zd.abs() > 500
            ref = torch.where(far, (zd > 0).double(), slope(zd.clamp(-500, 500), name))
            err = torch.where(far, torch.zeros_like(zd), slope_error(zd.clamp(-500, 500), name)) + 2.0 ** -23
            ok = ~nan
            check(dz[ok], ref[ok], err[ok], "slope")
