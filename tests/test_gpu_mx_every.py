"""8-bit values, exhaustively: every code with every scale byte as it is read
(alone, in the gradients, by the gradient to the weights), and every FP16 number
at every scale that holds it as it is written."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import CODE, FP8_MAX, as_bytes, codes_of, mx_pack, powers, scale_bytes, values
from test_gpu_norm import DEV, F16, F32, _gpu, say  # noqa: F401

pytestmark = pytest.mark.gpu

FMT = {"e4m3": g.FMT_E4M3, "e5m2": g.FMT_E5M2}


def same(a, b):
    """Equal, with NaN for NaN."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def every(cols):
    """Row e: all codes (and again from the first to fill `cols`), every scale byte e."""
    q = (torch.arange(cols, device=DEV) % 256).to(torch.uint8).expand(256, cols).contiguous()
    s = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].expand(256, (cols + 31) // 32).contiguous()
    return q, s


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_read_alone(fmt):
    """Whole pieces of eight, and rows cut in every way (the last piece element by element)."""
    for cols in (256, 257, 263, 509):
        q, s = every(cols)
        v = values(q, s, fmt)
        for t in (F32, F16):
            say(f"every code and scale {fmt}, {cols} columns into {t}")
            y = torch.empty((256, cols), dtype=t, device=DEV)
            g.dequantize_mx_fp8(q, s, FMT[fmt], y)
            assert same(y, v.float() if t == F32 else v.float().half())
    for first in range(0, 256, 7):   # rows of fewer than eight
        q = ((torch.arange(7, device=DEV) + first) % 256).to(torch.uint8).expand(256, 7).contiguous()
        s = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].contiguous()
        y = torch.empty((256, 7), device=DEV)
        g.dequantize_mx_fp8(q, s, FMT[fmt], y)
        assert same(y, values(q, s, fmt).float())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_read_by_a_gradient(fmt):
    """One row with dy = rstd = 1: the gradient to the norm's weights is what the row's codes stand for."""
    for cols in (256, 261):   # whole pieces, and a last one that overlaps the one before
        q, s = every(cols)
        v = values(q, s, fmt).float()
        one, dy = torch.ones(1, device=DEV), torch.ones((1, cols), device=DEV)
        w, dx, dw = torch.ones(cols, device=DEV), torch.empty((1, cols), device=DEV), torch.empty((256, cols), device=DEV)
        ws = torch.empty(g.rms_norm_backward_workspace_size(1, cols), dtype=torch.uint8, device=DEV)
        say(f"every code and scale {fmt} in the norm's gradient, {cols} columns")
        for e in range(256):
            g.rms_norm_backward(dy, q[e:e + 1], w, one, dx=dx, dweight=dw[e], hscale=s[e:e + 1], h_fmt=FMT[fmt],
                                workspace=ws)
        assert same(dw, v)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("config", ["wgrad_pp", "wgrad_tile_128", "wgrad_tile_64", "wgrad_tile_64_split"])
def test_read_by_the_gradient_to_the_weights(config, second, fmt, monkeypatch):
    """A group for each scale byte, of one row: its product with ones is the row in FP16."""
    monkeypatch.setenv("LIBGEMM_CONFIG", config)
    for cols in (256,) if config == "wgrad_pp" else (256, 259):
        q, s = every(cols)
        n = 16
        shape = (256, n, cols) if second else (256, cols, n)
        c = torch.full(shape, -1.0, device=DEV)
        off = torch.arange(257, dtype=torch.int32, device=DEV)
        say(f"every code and scale {fmt}, {config}, second {second}, {cols} columns")
        assert g.select_config_mx_wgrad(g.OUT_F32, 256, cols, n, 256, second) == config
        g.gemm_mx_wgrad(q, s, FMT[fmt], torch.ones((256, n), dtype=F16, device=DEV), c, offsets=off, q_second=second)
        v = values(q, s, fmt).float().half().float()
        assert same(c, (v[:, None, :] if second else v[:, :, None]).expand(shape))


def blocks_of(values_, anchor):
    """[.., 32]: 31 of the values and the anchor in each block (the last padded with zeros)."""
    v = torch.nn.functional.pad(values_, (0, -values_.numel() % 31)).reshape(-1, 31)
    return torch.cat([v, torch.full((v.shape[0], 1), anchor, dtype=v.dtype, device=v.device)], dim=1).reshape(1, -1)


def finite_f16():
    h = torch.arange(0, 0x7C00, dtype=torch.int16, device=DEV).view(F16)
    return torch.cat([h, -h])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_write_f16(fmt):
    """For every scale an FP16 block can have, every FP16 number that such a block can hold."""
    top, most = {"e4m3": 61440.0, "e5m2": 57344.0}[fmt], FP8_MAX[fmt]
    h = finite_f16()
    seen = set()
    for e in range(-41, 9):
        limit = min(most * 2.0 ** e, top)
        fits = h[h.double().abs() <= limit]
        anchor = float(fits.double().max())
        if anchor <= most * 2.0 ** (e - 1) or anchor == 0.0:
            continue                      # (no FP16 number has this scale)
        seen.add(e)
        x = blocks_of(fits, anchor)
        say(f"every FP16 number at scale 2^{e} {fmt}: {x.numel()}")
        u, sr = mx_pack(x, fmt, half=True)
        assert bool((scale_bytes(sr) == e + 127).all())
        for shape in ((1, -1), (x.numel() // 32, 32)):
            for cut in (0, 3):            # whole blocks in a run, and rows cut by three columns
                xx = x.reshape(shape)[:, :-cut].contiguous() if cut else x.reshape(shape)
                if cut and shape[0] != 1:
                    continue              # (the anchor stands in the columns that were cut)
                q, s = g.quantize_mx_fp8(xx, FMT[fmt])
                n = s.shape[1] - (1 if cut else 0)
                assert bool((s[:, :n] == e + 127).all()), "scales"
                ref = as_bytes(codes_of(u, fmt)).reshape(shape)
                assert torch.equal(q[:, :32 * n], ref[:, :32 * n]), "codes"
    assert max(seen) == (8 if fmt == "e4m3" else 0) and len(seen) >= 40


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_write_f32(fmt):
    """Every scale byte of FP32 blocks, with every sign, exponent and eleven leading bits that lie within 2^17 of the
    block's largest (and an odd last bit below them, which breaks ties)."""
    most = FP8_MAX[fmt]
    m = torch.arange(1024, 2048, device=DEV).double()
    base = torch.cat([m * 2.0 ** (p - 10) for p in range(-12, 9 if fmt == "e4m3" else 16)])
    base = torch.cat([base, base * (1 + 2.0 ** -23), base * (1 - 2.0 ** -23)])
    base = torch.cat([base, -base])
    base = base[base.abs() <= most]
    for e in range(-127, 128 - (8 if fmt == "e4m3" else 15)):
        x = blocks_of((base * 2.0 ** e).float(), most * 2.0 ** e)
        if e % 32 == 1:
            say(f"FP32 blocks at scale 2^{e} {fmt}: {x.numel()}")
        q, s = g.quantize_mx_fp8(x, FMT[fmt])
        u, sr = mx_pack(x, fmt)
        assert bool((s == e + 127).all()) and torch.equal(powers(s), sr), f"scales at 2^{e}"
        assert torch.equal(q, as_bytes(codes_of(u, fmt))), f"codes at 2^{e}"
        assert q.view(CODE[fmt]).isnan().sum().item() == 0
