"""GPU parity of 8-bit values with a power-of-two scale per 32 of a row:
quantize_mx_fp8 and dequantize_mx_fp8 bit for bit against a 64-bit reference,
and the gradient to the weights that reads them (gemm_mx_wgrad)."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import CODE, FP8_MAX, as_bytes, codes_of, mx_pack, powers, scale_bytes, spread, stored, values
from routed_ref import REL, check, cut
from test_gpu_norm import _gpu, gen, guarded, input_of, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, F32 = torch.float16, torch.float32
FMT = {"e4m3": g.FMT_E4M3, "e5m2": g.FMT_E5M2}


def awkward(gn, rows, cols, dtype):
    """Values over the whole range, ties between codes, borders of the scale, zeros."""
    x = normal(gn, (rows, cols)) * torch.exp2(torch.randint(-30, 16, (rows, cols), generator=gn, device=DEV).float() *
                                              (torch.rand((rows, 1), generator=gn, device=DEV) < 0.5))
    x[::5] = torch.round(x[::5] * 16) / 16                                     # ties
    x[1::5] = torch.exp2(torch.round(torch.log2(x[1::5].abs() + 1e-30)).clamp(-20, 14)) * 1.75   # 0.875 of a power of two
    x[2::7] = 0
    x[3::11, ::3] = -0.0
    if dtype == F16:
        x = x.clamp(-65504, 65504)
    return x.to(dtype)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("cols", [1, 8, 31, 32, 33, 64, 100, 512, 1000, 4096, 4099])
def test_pack(cols, dtype, fmt):
    for rows, offset in ((1, 0), (37, 0), (260, 1)):
        say(f"pack rows {rows} cols {cols} {dtype} {fmt} offset {offset}")
        x = input_of(awkward(gen(rows + cols), rows, cols, dtype), offset)
        q, guard_q = guarded((rows, cols), torch.uint8, offset)
        s, guard_s = guarded((rows, (cols + 31) // 32), torch.uint8, offset)
        g.quantize_mx_fp8(x, FMT[fmt], q=q, scale=s)
        u, sr = mx_pack(x, fmt, half=dtype == F16)
        assert torch.equal(s, scale_bytes(sr)), "scales"
        assert torch.equal(q, as_bytes(codes_of(u, fmt))), "codes"
        guard_q(), guard_s()
        v = values(q, s, fmt)
        for t in (F32, F16):
            say(f"unpack rows {rows} cols {cols} {t} {fmt}")
            y, guard_y = guarded((rows, cols), t, offset)
            g.dequantize_mx_fp8(q, s, FMT[fmt], y)
            assert torch.equal(y, v.to(torch.float32).to(t) if t == F32 else v.float().to(F16)), "values"
            guard_y()
            if dtype == F16 and t == F16:
                assert bool(y.isfinite().all()), "FP16 values stay FP16 values"


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_pack_special(dtype, fmt):
    """NaN and infinities do not take part in the scale and stay what they are (E4M3 has no infinity); tiny and huge
    blocks, and the largest FP16 numbers."""
    gn = gen(5)
    x = normal(gn, (64, 96)).to(dtype)
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    x[3] = float("nan")
    x[4, :32] = 65504.0
    x[5, 32:64] = 2.0 ** -24
    if dtype == F32:
        x[6, :32] = 3e38
        x[7, 32:64] = 2.0 ** -149
        x[8, :64] = torch.tensor([2.0 ** -140, 2.0 ** -130] * 32, device=DEV)
    say(f"pack special {dtype} {fmt}")
    q, s = g.quantize_mx_fp8(x, FMT[fmt])
    u, sr = mx_pack(x, fmt, half=dtype == F16)
    assert torch.equal(s, scale_bytes(sr))
    c, ref = q.view(CODE[fmt]).float(), codes_of(torch.where(u.isfinite(), u, torch.zeros_like(u)), fmt).float()
    fin = x.isfinite()
    assert torch.equal(c[fin], ref[fin])
    assert bool(c[x.isnan()].isnan().all())
    if fmt == "e5m2":
        assert torch.equal(c[x.isinf()], x[x.isinf()].float())
    else:
        assert bool(c[x.isinf()].isnan().all())
    y = torch.empty_like(x)
    g.dequantize_mx_fp8(q, s, FMT[fmt], y)
    assert torch.equal(y.isfinite(), fin)


def test_pack_shapes_without_work():
    say("pack of nothing")
    for shape in ((0, 40), (3, 0)):
        q, s = g.quantize_mx_fp8(torch.empty(shape, device=DEV))
        assert q.shape == shape and s.shape == (shape[0], (shape[1] + 31) // 32)


def test_unpack_scales():
    """Every scale byte, 0 (2^-127) and 255 (NaN) among them."""
    q = torch.full((256, 32), 0x38, dtype=torch.uint8, device=DEV)   # E4M3: 1.0
    s = torch.arange(256, dtype=torch.uint8, device=DEV).reshape(256, 1)
    y = torch.empty((256, 32), device=DEV)
    say("unpack every scale")
    g.dequantize_mx_fp8(q, s, g.FMT_E4M3, y)
    ref = torch.tensor([2.0 ** (e - 127) for e in range(255)], device=DEV)
    assert torch.equal(y[:255, 0], ref) and bool(y[255].isnan().all())


# ------------------------------------------------------- gradient to the weights

def run_wgrad(sizes, m, n, fmt, second, out, lead=0, tail=0, offset=0, grouped=True, config=None, monkeypatch=None):
    offsets = cut(sizes, lead)
    rows = offsets[-1] + tail
    gn = gen(rows + m + n)
    x = normal(gn, (rows, m)) * torch.exp(normal(gn, (rows, 1)))
    q, s = g.quantize_mx_fp8(x.half(), FMT[fmt])
    if tail or lead:   # rows of no group may hold anything
        for t in (q, s):
            t[:lead] = 0xFF
            t[offsets[-1]:] = 0xFF
    q, s = input_of(q, offset), input_of(s, offset)
    b = normal(gn, (rows, n)).half()
    if tail or lead:
        b[:lead] = float("nan")
        b[offsets[-1]:] = float("nan")
    b = input_of(b, offset)
    shape = (n, m) if second else (m, n)
    c, guard = guarded(((len(sizes),) if grouped else ()) + shape, out, offset)
    if config:
        assert g.select_config_mx_wgrad(g.OUT_F32 if out == F32 else g.OUT_F16, rows, m, n, len(sizes), second) == config
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV) if grouped else None
    g.gemm_mx_wgrad(q, s, FMT[fmt], b, c, offsets=off, q_second=second)
    xv, bv = values(q, s, fmt), b.double()
    c3 = c if grouped else c.reshape(1, *shape)
    for e in range(len(sizes)):
        lo, hi = offsets[e], offsets[e + 1]
        l, r = (bv, xv) if second else (xv, bv)
        v = l[lo:hi].t().contiguous() @ r[lo:hi]
        a = l[lo:hi].abs().t().contiguous() @ r[lo:hi].abs()
        check(c3[e], v, REL * a + stored(v, out), f"group {e}")
    guard()


SHAPES = [(1, 1), (7, 40), (32, 8), (33, 129), (100, 64), (130, 257), (256, 256), (272, 520), (1000, 136)]


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m,n", SHAPES)
def test_wgrad(m, n, fmt, second):
    for sizes, out in (([1], F32), ([31, 0, 70], F16), ([129], F32), ([513, 32, 5, 64], F16)):
        say(f"wgrad sizes {sizes} m {m} n {n} {fmt} second {second} {out}")
        run_wgrad(sizes, m, n, fmt, second, out)


@pytest.mark.parametrize("config", ["wgrad_pp", "wgrad_tile_128", "wgrad_tile_64", "wgrad_tile_64_split"])
@pytest.mark.parametrize("second", [False, True])
def test_wgrad_kernels(config, second, monkeypatch):
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    for sizes, m, n, fmt in (([1], 16, 16, "e4m3"), ([32], 272, 272, "e4m3"), ([33, 0, 64, 95], 528, 304, "e5m2"),
                             ([224, 256, 259], 256, 512, "e4m3"), ([1029], 304, 1040, "e4m3")):
        for out in (F16, F32):
            say(f"wgrad {config} sizes {sizes} m {m} n {n} {fmt} second {second} {out}")
            run_wgrad(sizes, m, n, fmt, second, out, config=config)
    say(f"wgrad {config} rows of no group")
    run_wgrad([40, 0, 100], 64, 96, "e4m3", second, F32, lead=3, tail=9, config=config)


@pytest.mark.parametrize("second", [False, True])
def test_wgrad_one_group_without_offsets(second):
    for rows, m, n in ((1, 40, 24), (700, 512, 768), (2051, 96, 136)):
        say(f"wgrad whole rows {rows} m {m} n {n} second {second}")
        run_wgrad([rows], m, n, "e4m3", second, F32, grouped=False)


@pytest.mark.parametrize("second", [False, True])
def test_wgrad_unaligned(second):
    for m, n in ((96, 64), (101, 77), (3, 5)):
        say(f"wgrad unaligned m {m} n {n} second {second}")
        run_wgrad([70, 9], m, n, "e4m3", second, F16, offset=1)


@pytest.mark.parametrize("config", ["wgrad_pp", "wgrad_tile_128", "wgrad_tile_64", "wgrad_tile_64_split"])
def test_wgrad_special(config, monkeypatch):
    """A NaN and a scale that is NaN reach their own weights only; values past FP16's range are infinities."""
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    gn = gen(4)
    rows, m, n = 80, 96, 64
    q, s = g.quantize_mx_fp8(normal(gn, (rows, m)).half())
    b = normal(gn, (rows, n)).half()
    q[5, 40] = 0x7F
    s[7, 2] = 255
    s[9, 0] = 127 + 30          # codes times 2^30: beyond FP16
    q[9, :32] = 0x38
    b[9] = 1.0
    c = torch.empty((m, n), device=DEV)
    say(f"wgrad special {config}")
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, b, c)
    assert bool(c[40].isnan().all()) and bool(c[64:].isnan().all()) and bool((c[:32] == float("inf")).all())
    rest = [i for i in range(32, 64) if i != 40]
    x = values(q, s, "e4m3")[:, rest]
    v, a = x.t().contiguous() @ b.double(), x.abs().t().contiguous() @ b.double().abs()
    check(c[rest], v, REL * a + stored(v, F32), "others")


def test_wgrad_no_rows():
    say("wgrad, no rows")
    c = torch.full((2, 40, 24), 3.0, device=DEV)
    q, s = torch.empty((0, 40), dtype=torch.uint8, device=DEV), torch.empty((0, 2), dtype=torch.uint8, device=DEV)
    g.gemm_mx_wgrad(q, s, g.FMT_E4M3, torch.empty((0, 24), dtype=F16, device=DEV), c,
                    offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert bool((c == 0).all())


def test_pack_keeps_what_fits():
    """Numbers of four significant bits within the block's range come back as they were."""
    gn = gen(8)
    x = torch.randint(8, 16, (50, 320), generator=gn, device=DEV).float() * torch.exp2(
        torch.randint(-6, 6, (50, 320), generator=gn, device=DEV).float())
    say("pack of what fits")
    q, s = g.quantize_mx_fp8(x.half())
    y = torch.empty((50, 320), dtype=F16, device=DEV)
    g.dequantize_mx_fp8(q, s, g.FMT_E4M3, y)
    assert torch.equal(y.float(), x) and float(spread(s.float(), 320).max()) < 255 and FP8_MAX["e4m3"] == 448.0


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_pack_least_and_largest_numbers(fmt):
    """FP32 blocks from the least subnormal numbers to the largest: codes and scales as for any others."""
    gn = gen(12)
    x = normal(gn, (256, 96)) * torch.ldexp(torch.ones(256, 1, device=DEV), torch.arange(-150, 106, device=DEV)[:, None])
    x[0, 0], x[255, 40] = 2.0 ** -149, 3.4e38
    say(f"pack from the least to the largest numbers {fmt}")
    q, s = g.quantize_mx_fp8(x, FMT[fmt])
    u, sc = mx_pack(x, fmt)
    assert torch.equal(powers(s), sc), "scales"
    assert torch.equal(q, as_bytes(codes_of(u, fmt))), "codes"
