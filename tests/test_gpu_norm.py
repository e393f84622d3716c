"""GPU parity of rms_norm and its gradient against 64-bit references
(dense_ref.py). Each test prints the case it is about to launch."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import HALF_CODE, REL, code_step, norm, norm_backward, stored, values
from routed_ref import check

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32 = torch.float16, torch.float32
EPS = 1e-5


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


def guarded(shape, dtype, offset=0):
    """A tensor inside a larger buffer (offset elements off alignment) and the function that checks the rest of it."""
    n = 1
    for s in shape:
        n *= s
    es = torch.empty((), dtype=dtype).element_size()
    buf = torch.full(((n + offset + 64) * es,), 0xA5, dtype=torch.uint8, device=DEV)
    t = buf[offset * es:(offset + n) * es].view(dtype).reshape(shape)

    def untouched():
        assert bool((buf[:offset * es] == 0xA5).all()) and bool((buf[(offset + n) * es:] == 0xA5).all())
    return t, untouched


def input_of(x, offset):
    """x at an address off 16-byte alignment."""
    t, _ = guarded(tuple(x.shape), x.dtype, offset)
    t.copy_(x)
    return t


def run_norm(rows, width, dtype, out, residual, pow2=False, offset=0, seed=0):
    gn = gen(seed + rows + width)
    x = input_of((normal(gn, (rows, width)) * torch.exp(normal(gn, (rows, 1)))).to(dtype), offset)
    res = input_of(normal(gn, (rows, width)).to(dtype), offset) if residual else None
    w = 1.0 + normal(gn, (width,), 0.2)
    fmt = {torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}.get(out)
    y, guard_y = guarded((rows, width), out, offset)
    h, guard_h = guarded((rows, width), dtype, offset)
    rstd, guard_r = guarded((rows,), F32, 1)
    scale, guard_s = guarded((rows,), F32, 1)
    g.rms_norm(x, w, y, eps=EPS, residual=res, h=h, scale=scale if fmt else None, rstd=rstd, pow2=pow2)
    href = x if res is None else (x.float() + res.float()).to(dtype)
    assert torch.equal(h, href), "h is the rounded sum"
    v, r = norm(href.double(), w.double(), EPS)
    check(rstd, r, r * REL, "rstd")
    if fmt is None:
        check(y, v, v.abs() * REL + stored(v, out), "y")
    else:
        s = v.abs().amax(dim=1) / {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
        s = torch.where(s > 0, s, torch.ones_like(s))
        got = scale.double()
        if pow2:
            assert bool((torch.log2(got) == torch.log2(got).round()).all())
            assert bool((got >= s * (1 - REL)).all()) and bool((got <= 2 * s * (1 + REL)).all())
        else:
            check(scale, s, s * REL, "scale")
        check(y.double() * got[:, None], v, code_step(v, got[:, None], fmt) * (1 + 2 * REL) + v.abs() * 2 * REL, "codes")
    for f in (guard_y, guard_h, guard_r, guard_s):
        f()


WIDTHS = [1, 7, 8, 64, 100, 511, 512, 1000, 1024, 1025, 2048, 2056, 4096, 4099, 8192, 9000, 16384, 16385, 40000]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, F32])
def test_norm_widths(width, dtype):
    for out, rows, residual in ((F16, 3, True), (torch.float8_e4m3fn, 5, True), (F32, 2, False),
                                (torch.float8_e5m2, 4, False)):
        say(f"norm rows {rows} width {width} {dtype} -> {out} residual {residual}")
        run_norm(rows, width, dtype, out, residual)


@pytest.mark.parametrize("rows,width", [(1, 4096), (9, 40), (4097, 96), (20000, 24), (5000, 1032), (4099, 16400)])
def test_norm_rows(rows, width):
    for out in (F16, torch.float8_e4m3fn):
        say(f"norm rows {rows} width {width} -> {out}")
        run_norm(rows, width, F16, out, True)


@pytest.mark.parametrize("offset", [1, 3])
@pytest.mark.parametrize("width", [96, 515, 4096, 17001])
def test_norm_unaligned(width, offset):
    for dtype, out in ((F16, F16), (F16, torch.float8_e4m3fn), (F32, torch.float8_e5m2), (F32, F32)):
        say(f"norm width {width} {dtype} -> {out} offset {offset}")
        run_norm(6, width, dtype, out, True, offset=offset)


def test_norm_pow2_and_no_optional_outputs():
    for out in (torch.float8_e4m3fn, torch.float8_e5m2):
        say(f"norm pow2 {out}")
        run_norm(17, 1000, F16, out, True, pow2=True)
    x, w = normal(gen(1), (5, 300)).half(), torch.ones(300, device=DEV)
    y = torch.empty_like(x)
    say("norm without h, rstd")
    g.rms_norm(x, w, y)
    v, _ = norm(x.double(), w.double(), 1e-5)
    check(y, v, v.abs() * REL + stored(v, F16), "y")


@pytest.mark.parametrize("width", [200, 5000, 20000])
def test_norm_special_rows(width):
    """A row of zeros, a NaN, an infinity and the largest FP16 numbers: only their own rows feel them."""
    gn = gen(3)
    x = normal(gn, (6, width)).half()
    x[1] = 0
    x[2, width // 2] = float("nan")
    x[3, width - 1] = float("inf")
    x[4] = 65504.0
    w = 1.0 + normal(gn, (width,), 0.2)
    for out in (F16, F32, torch.float8_e4m3fn):
        say(f"norm special rows width {width} -> {out}")
        y = torch.empty((6, width), dtype=out, device=DEV)
        scale = torch.empty(6, device=DEV) if out == torch.float8_e4m3fn else None
        g.rms_norm(x, w, y, eps=EPS, scale=scale)
        assert bool((y[1].float() == 0).all()) and (scale is None or scale[1].item() == 1.0)
        assert bool(y[2].float().isnan().all())
        assert bool(y[3, -1].float().isnan())
        for r in (0, 4, 5):
            v, _ = norm(x[r:r + 1].double(), w.double(), EPS)
            if scale is None:
                check(y[r:r + 1], v, v.abs() * REL + stored(v, out), f"row {r}")
            else:
                s = scale[r].double()
                check(y[r:r + 1].double() * s, v, code_step(v, s, "e4m3") * (1 + 2 * REL) + v.abs() * 2 * REL, f"row {r}")


def held(x, kind):
    """(h, hscale, the numbers it stands for)."""
    if kind in (F16, F32):
        t = x.to(kind)
        return t, None, t.double()
    q, s = g.quantize_mx_fp8(x.half(), g.FMT_E4M3 if kind == "e4m3" else g.FMT_E5M2,
                             q=torch.empty(x.shape, dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.float8_e5m2,
                                           device=DEV))
    return q, s, values(q, s, kind)


def run_backward(rows, width, dtype, kind, joins, want_dw=True, offset=0):
    gn = gen(rows * 3 + width)
    h, hs, hv = held(normal(gn, (rows, width)) * torch.exp(normal(gn, (rows, 1))), kind)
    if offset:
        h = input_of(h, offset)
        hs = None if hs is None else input_of(hs, offset)
    w = 1.0 + normal(gn, (width,), 0.2)
    rstd = (1.0 / torch.sqrt((hv * hv).mean(dim=1) + EPS)).float()
    dy = input_of(normal(gn, (rows, width)).to(dtype), offset)
    dh = input_of(normal(gn, (rows, width)).to(dtype), offset) if joins else None
    dx, guard_x = guarded((rows, width), dtype, offset)
    dw, guard_w = guarded((width,), F32, offset)
    n = g.rms_norm_backward_workspace_size(rows, width)
    ws = torch.full((max(n, 16) + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    out = g.rms_norm_backward(dy, h, w, rstd, dx=dx, dweight=dw if want_dw else None, dh=dh, hscale=hs, workspace=ws[:max(n, 16)])
    assert bool((ws[max(n, 16):] == 0xA5).all()), "past the workspace"
    rx, rw, mx, mw = norm_backward(dy.double(), hv, w.double(), rstd.double(), None if dh is None else dh.double())
    check(dx, rx, REL * mx + stored(rx, dtype), "dx")
    if want_dw:
        check(dw, rw, REL * mw + stored(rw, F32), "dweight")
    else:
        assert out[1] is None
        assert bool((dw.view(torch.uint8) == 0xA5).all())
    guard_x(), guard_w()


@pytest.mark.parametrize("kind", [F16, F32, "e4m3", "e5m2"], ids=str)
@pytest.mark.parametrize("width", [1, 8, 33, 100, 512, 1000, 1025, 2048, 4096, 4100, 8192, 12000, 16384, 16385, 33000])
def test_backward_widths(width, kind):
    for dtype, rows, joins in ((F16, 3, True), (F32, 7, False)):
        say(f"norm backward rows {rows} width {width} {dtype} held {kind} joins {joins}")
        run_backward(rows, width, dtype, kind, joins)


@pytest.mark.parametrize("rows,width", [(1, 300), (1023, 40), (1025, 520), (4099, 2048), (9000, 64), (1030, 17000)])
def test_backward_rows(rows, width):
    for kind in (F16, "e4m3"):
        say(f"norm backward rows {rows} width {width} held {kind}")
        run_backward(rows, width, F16, kind, True)


def test_backward_without_weight_gradient_and_unaligned():
    for width in (520, 4096, 17003):
        say(f"norm backward without dweight, width {width}")
        run_backward(11, width, F16, F16, True, want_dw=False)
        for kind in (F16, "e4m3"):
            say(f"norm backward unaligned width {width} held {kind}")
            run_backward(5, width, F32, kind, True, offset=3)


def test_backward_no_rows():
    say("norm backward, no rows")
    dw = torch.full((77,), 5.0, device=DEV)
    z = torch.empty((0, 77), device=DEV)
    g.rms_norm_backward(z, z, torch.ones(77, device=DEV), torch.empty(0, device=DEV), dweight=dw)
    assert bool((dw == 0).all())


def test_backward_repeats():
    """The same bits twice, beside other work."""
    gn = gen(9)
    dy, h = normal(gn, (3000, 1000)).half(), normal(gn, (3000, 1000)).half()
    w, rstd = torch.ones(1000, device=DEV), torch.ones(3000, device=DEV)
    got = []
    for _ in range(3):
        say("norm backward repeat")
        dw = torch.empty(1000, device=DEV)
        dx, _ = g.rms_norm_backward(dy, h, w, rstd, dweight=dw)
        got.append((dx, dw))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


@pytest.mark.parametrize("width", [65, 1000])
def test_gradient_against_differences(width):
    """The gradients against central differences of the norm in 64 bits, along a random direction."""
    gn = gen(width)
    rows, e = 9, 1e-6
    x, res, dy = (normal(gn, (rows, width)) for _ in range(3))
    w = 1.0 + normal(gn, (width,), 0.2)
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV)
    say(f"norm gradient against differences, width {width}")
    g.rms_norm(x, w, y, eps=EPS, residual=res, h=h, rstd=rstd)
    dw = torch.empty(width, device=DEV)
    dx, _ = g.rms_norm_backward(dy, h, w, rstd, dweight=dw)
    vx, vw = normal(gn, (rows, width)).double(), normal(gn, (width,)).double()

    def loss(t):
        return (norm(h.double() + t * vx, w.double() + t * vw, EPS)[0] * dy.double()).sum()
    slope = ((loss(e) - loss(-e)) / (2 * e)).item()
    along = (dx.double() * vx).sum().item() + (dw.double() * vw).sum().item()
    size = (dx.double() * vx).abs().sum().item() + (dw.double() * vw).abs().sum().item()
    # REL of the terms' magnitudes for the kernels, 1e-6 of them for the difference (e^2 and rounding 2^-52 / e)
    assert abs(slope - along) <= 2 * REL * size


@pytest.mark.parametrize("width", [67, 100, 1001, 4099, 12003])
def test_infinity_at_a_cut_row_end(width):
    """An infinity in one of the last eight columns, which two lanes read: the row is zeros beside it (its norm is
    infinite) and NaN at it, as the formula says; in the gradient the other columns are infinite, of either sign."""
    x = normal(gen(width), (9, width))
    w = torch.ones(width, device=DEV)
    for i in range(8):
        x[i, width - 1 - i] = float("inf")
    say(f"infinity at a row's end, width {width}")
    y, rstd = torch.empty_like(x), torch.empty(9, device=DEV)
    g.rms_norm(x, w, y, eps=EPS, rstd=rstd)
    at = x.isinf()
    assert bool(y[at].isnan().all()) and bool((y[:8][~at[:8]] == 0).all()) and bool((rstd[:8] == 0).all())
    assert bool(y[8].isfinite().all()) and bool((y[8] != 0).any())
    h = normal(gen(width + 1), (9, width))
    h[h == 0] = 1.0
    dx, _ = g.rms_norm_backward(x, h, w, torch.ones(9, device=DEV))
    for i in range(8):
        j = width - 1 - i
        other = torch.arange(width, device=DEV) != j
        want = -h[i].sign() * h[i, j].sign() * float("inf")
        assert torch.equal(dx[i][other], want[other]), i
        assert bool(dx[i, j].isnan())
    assert bool(dx[8].isfinite().all())


@pytest.mark.parametrize("width", [64, 1000, 4099, 20000])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows_near_the_least_numbers(width, pow2):
    """FP32 rows, and weights, so small that 1 / scale is beyond FP32: codes as of any other row."""
    gn = gen(width)
    x = normal(gn, (6, width))
    x[0:2] *= 1e-37
    x[4:] = 0.0
    w = 1.0 + normal(gn, (width,), 0.2)
    for out, fmt, top in ((torch.float8_e4m3fn, "e4m3", 448.0), (torch.float8_e5m2, "e5m2", 57344.0)):
        for weight in (w, w * (1e-35 if fmt == "e4m3" else 1e-33)):
            say(f"norm of least numbers, width {width} {fmt} pow2 {pow2}")
            y, scale = torch.empty((6, width), dtype=out, device=DEV), torch.empty(6, device=DEV)
            rows = slice(0, 4) if weight is w else slice(2, 4)
            if weight is w and fmt == "e5m2":
                rows = slice(2, 4)   # (the small rows' scale is no normal number)
            g.rms_norm(x, weight, y, eps=EPS, scale=scale, pow2=pow2)
            v, _ = norm(x.double(), weight.double(), EPS)
            s = scale.double()[:, None]
            if not pow2:
                check(s[rows, 0], v[rows].abs().amax(dim=1) / top, v[rows].abs().amax(dim=1) / top * REL, "scale")
            check((y.double() * s)[rows], v[rows], (code_step(v, s, fmt) * (1 + 2 * REL) + v.abs() * 2 * REL)[rows], "codes")
            assert bool((y[4:].float() == 0).all()) and bool((scale[4:] == 1.0).all())
