"""A dense layer's calls whose operands pass 2^32 bytes and 2^31 and 2^32
elements, checked where their offsets are largest: what lies between is zero or
NaN that no checked element takes in. Bounds are those of dense_ref.py."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import (REL, STEEPEST, act, act_error, code_step, mx_pack, norm, norm_backward, powers, slope,
                       slope_error, spread, stored, values)
from routed_ref import check
from test_gpu_norm import DEV, F16, F32, gen, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5
ENDS = 5     # rows that are looked at, at either end


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(DEV)
    g.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def ends(t):
    return torch.cat([t[:ENDS], t[-ENDS:]])


def long(rows, cols, gn, dtype=F16):
    """[rows, cols] of zeros but for rows at both ends."""
    t = torch.zeros((rows, cols), dtype=dtype, device=DEV)
    t[:ENDS] = normal(gn, (ENDS, cols)).to(dtype)
    t[-ENDS:] = normal(gn, (ENDS, cols)).to(dtype)
    return t


ROWS, WIDTH = 1060000, 4104   # 4.35e9 elements


def test_norm_and_its_gradient():
    gn = gen(1)
    x, res = long(ROWS, WIDTH, gn), long(ROWS, WIDTH, gn)
    w = 1.0 + normal(gn, (WIDTH,), 0.2)
    h, q = torch.empty_like(x), torch.empty((ROWS, WIDTH), dtype=torch.float8_e4m3fn, device=DEV)
    scale, rstd = torch.empty(ROWS, device=DEV), torch.empty(ROWS, device=DEV)
    say(f"norm, {x.numel() * 2 >> 20} MiB")
    g.rms_norm(x, w, q, eps=EPS, residual=res, h=h, scale=scale, rstd=rstd)
    hr = (ends(x).float() + ends(res).float()).half()
    assert torch.equal(ends(h), hr)
    v, r = norm(hr.double(), w.double(), EPS)
    check(ends(rstd), r, r * REL, "rstd")
    got = ends(scale).double()[:, None]
    check(ends(q).double() * got, v, code_step(v, got, "e4m3") * (1 + 2 * REL) + v.abs() * 2 * REL, "codes")
    assert float(scale[ROWS // 2]) == 1.0 and float(h[ROWS // 2].abs().max()) == 0.0
    del q, x, res
    dy, dx, dw = long(ROWS, WIDTH, gn), torch.empty_like(h), torch.empty(WIDTH, device=DEV)
    say("its gradient")
    g.rms_norm_backward(dy, h, w, rstd, dx=dx, dweight=dw)
    re = ends(rstd).double()
    vx, vw, mx, mw = norm_backward(ends(dy).double(), hr.double(), w.double(), re, None)
    check(ends(dx), vx, mx * REL * 4 + stored(vx, F16), "dx")
    check(dw, vw, mw * REL * 2, "dweight")
    assert float(dx[ROWS // 2].abs().max()) == 0.0


def test_epilogue_gradient_and_8_bit_values():
    gn = gen(2)
    z = long(ROWS, WIDTH, gn)
    say(f"8-bit values of {z.numel() * 2 >> 20} MiB")
    q, s = g.quantize_mx_fp8(z)
    u, sc = mx_pack(ends(z), "e4m3", half=True)
    assert torch.equal(powers(ends(s)), sc)
    check(values(ends(q), ends(s), "e4m3"), ends(z).double(), code_step(ends(z).double(), spread(sc, WIDTH), "e4m3"), "codes")
    back = torch.empty_like(z)
    g.dequantize_mx_fp8(q, s, g.FMT_E4M3, back)
    zv = values(ends(q), ends(s), "e4m3")
    assert torch.equal(ends(back).double(), zv)   # what the codes of FP16 values stand for are FP16 values
    del back, z
    dy, dz, db = long(ROWS, WIDTH, gn), torch.empty((ROWS, WIDTH), dtype=F16, device=DEV), torch.empty(WIDTH, device=DEV)
    say("the epilogue's gradient")
    g.bias_act_backward(dy, q, g.ACT_GELU, dZ=dz, dbias=db, Zscale=s, z_fmt=g.FMT_E4M3)
    d = ends(dy).double()
    v = d * slope(zv, "gelu")
    e = d.abs() * slope_error(zv, "gelu") + v.abs() * 2.0 ** -22
    check(ends(dz), v, e + stored(v.abs() + e, F16), "dZ")
    check(db, v.sum(dim=0), (e + REL * v.abs()).sum(dim=0), "dbias")


@pytest.mark.parametrize("rows,cols", [(2, 1 << 30), (3, (1 << 30) + 8)])
def test_few_long_rows(rows, cols):
    """Rows past 2^31 and 2^32 bytes: ones, and a run of values at a row's end."""
    x = torch.ones((rows, cols), dtype=F16, device=DEV)
    x[-1, -64:] = 3.0
    w = torch.ones(cols, device=DEV)
    w[-1] = 2.0
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    say(f"norm of {rows} rows of {cols}")
    g.rms_norm(x, w, y, eps=0.0, rstd=rstd)
    ms = torch.tensor([1.0] * (rows - 1) + [(cols - 64 + 64 * 9.0) / cols], dtype=torch.float64, device=DEV)
    check(rstd, ms ** -0.5, ms ** -0.5 * REL, "rstd")
    v = (x[:, -80:].double() * (ms ** -0.5)[:, None]) * w[-80:].double()
    check(y[:, -80:], v, v * REL + stored(v, F16), "y")
    assert bool((y[0, :80] == 1.0).all())
    del y
    q, s = g.quantize_mx_fp8(x)
    end = 64 + (cols % 32 or 32)   # the last three blocks
    assert torch.equal(values(q[:, -end:], s[:, -3:], "e4m3"), x[:, -end:].double())
    back = torch.empty_like(x)
    g.dequantize_mx_fp8(q, s, g.FMT_E4M3, back)
    assert torch.equal(back, x)


@pytest.mark.parametrize("m", [1, 3, 40, 520])
@pytest.mark.parametrize("kind", ["f16", "fp8"])
def test_weights(m, kind):
    """A K-major weight of 4.4e9 elements; columns at the end and the beginning."""
    n, k = 67000, 65552
    gn = gen(3)
    f16 = kind == "f16"
    b = torch.zeros((n, k), dtype=F16 if f16 else torch.float8_e4m3fn, device=DEV)
    a = normal(gn, (m, k))
    ends_w = normal(gn, (2 * ENDS, k))
    c, z = torch.empty((m, n), dtype=F16, device=DEV), torch.empty((m, n), dtype=F16, device=DEV)
    bias, res = normal(gn, (n,)), normal(gn, (m, n)).half()
    say(f"{kind}, {m} rows on a weight of {b.numel() * b.element_size() >> 20} MiB")
    if f16:
        ends_w = (ends_w / k ** 0.5).half()
        a = a.half()
        f = 1.0
    else:
        ends_w, a = (ends_w * 64).to(b.dtype), (a * 64).to(b.dtype)
        f = 1.0 / (64 * 64 * k ** 0.5)
    b[:ENDS], b[-ENDS:] = ends_w[:ENDS], ends_w[ENDS:]
    if f16:
        g.gemm_f16_bias_act_bt(a, b, c, bias=bias, act=g.ACT_SILU, residual=res, Z=z)
    else:
        sa, sb = torch.full((1,), f, device=DEV), torch.ones(1, device=DEV)
        g.gemm_fp8_bias_act_bt(a, g.FMT_E4M3, b, g.FMT_E4M3, sa, sb, c, bias=bias, act=g.ACT_SILU, residual=res, Z=z)
    cols = torch.cat([torch.arange(ENDS), torch.arange(n - ENDS, n)]).to(DEV)
    av, bv = a.double(), ends_w.double()
    zr = av @ bv.t() * f + bias[cols].double()
    mag = av.abs() @ bv.abs().t() * f
    # (the matrix cores' FP8 sums: eight products, each within 2^-13 of the largest)
    e = (REL if f16 else 2.0 ** -9) * mag + zr.abs() * 2.0 ** -20
    check(z[:, cols], zr, e + stored(zr.abs() + e, F16), "Z")
    y = act(zr, "silu") + res[:, cols].double()
    e = STEEPEST * e + act_error(zr, "silu") + y.abs() * 2.0 ** -22
    check(c[:, cols], y, e + stored(y.abs() + e, F16), "C")
    mid = bias[n // 2].double().expand(m)   # a weight of zeros: the bias alone
    check(z[:, n // 2], mid, mid.abs() * 2.0 ** -22 + stored(mid, F16), "Z of the bias")


@pytest.mark.parametrize("zt", ["f16", "e4m3"])
def test_outputs(zt):
    """C, residual and Z of 4.35e9 elements."""
    k = 40
    gn = gen(4)
    a = long(ROWS, k, gn)
    b = (normal(gn, (WIDTH, k)) / k ** 0.5).half()
    res = long(ROWS, WIDTH, gn)
    c = torch.empty((ROWS, WIDTH), dtype=F16, device=DEV)
    mx = zt == "e4m3"
    z = torch.empty((ROWS, WIDTH), dtype=torch.float8_e4m3fn if mx else F16, device=DEV)
    zs = torch.empty((ROWS, (WIDTH + 31) // 32), dtype=torch.uint8, device=DEV) if mx else None
    say(f"C of {c.numel() * 2 >> 20} MiB, Z {zt}")
    g.gemm_f16_bias_act_bt(a, b, c, act=g.ACT_GELU_TANH, residual=res, Z=z, Zscale=zs)
    av, bv = ends(a).double(), b.double()
    zr = av @ bv.t()
    e = REL * (av.abs() @ bv.abs().t())
    if mx:
        check(values(ends(z), ends(zs), "e4m3"), zr,
              e + code_step(zr.abs() + e, spread(powers(ends(zs)), WIDTH), "e4m3"), "Z")
    else:
        check(ends(z), zr, e + stored(zr.abs() + e, F16), "Z")
    y = act(zr, "gelu_tanh") + ends(res).double()
    e = STEEPEST * e + act_error(zr, "gelu_tanh") + y.abs() * 2.0 ** -22
    check(ends(c), y, e + stored(y.abs() + e, F16), "C")
    assert float(c[ROWS // 2].abs().max()) == 0.0


@pytest.mark.parametrize("second", [False, True])
def test_weight_gradient(second):
    """8-bit values of 4.35e9 elements, and FP16 rows of as many: the ends' rows make the sum."""
    gn = gen(5)
    n = 72
    q, s = g.quantize_mx_fp8(long(ROWS, WIDTH, gn))
    b = long(ROWS, n, gn)
    c = torch.empty((n, WIDTH) if second else (WIDTH, n), device=DEV)
    say(f"gradient to the weights over {ROWS} rows, second {second}")
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, b, c, q_second=second)
    xv, bv = values(ends(q), ends(s), "e4m3"), ends(b).double()
    v, mag = xv.t() @ bv, xv.abs().t() @ bv.abs()
    check(c.t() if second else c, v, REL * mag, "C")
    del q, s, b
    q, s = g.quantize_mx_fp8(long(ROWS, n, gn))
    b = long(ROWS, WIDTH, gn)
    c = torch.empty((WIDTH, n) if second else (n, WIDTH), device=DEV)
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, b, c, q_second=second)
    xv, bv = values(ends(q), ends(s), "e4m3"), ends(b).double()
    v, mag = xv.t() @ bv, xv.abs().t() @ bv.abs()
    check(c.t() if second else c, v, REL * mag, "C")


def test_weight_gradients_of_groups():
    """40 gradients of 128 MiB."""
    groups, m, n = 40, 4096, 8192
    gn = gen(6)
    rows = 3 * groups
    q, s = g.quantize_mx_fp8(normal(gn, (rows, m)).half())
    b = normal(gn, (rows, n)).half()
    offsets = torch.arange(0, rows + 1, 3, dtype=torch.int32, device=DEV)
    c = torch.full((groups, m, n), float("nan"), device=DEV)
    say(f"gradients of {c.numel() * 4 >> 20} MiB")
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, b, c, offsets=offsets)
    xv = values(q, s, "e4m3")
    for e in (0, 33, groups - 1):
        x, y = xv[3 * e:3 * e + 3].t().contiguous(), b[3 * e:3 * e + 3].double()
        check(c[e], x @ y, REL * (x.abs() @ y.abs()), f"group {e}")
