"""Refusals of what a dense layer does around its products: invalid arguments
return before anything touches a GPU (no GPU needed), and the binding checks
types and shapes. Also the host-only queries."""
import pytest
import torch

import precision_dense_gemm_03_amd as g

P = [i << 40 for i in range(1, 20)]     # never dereferenced: every call below fails validation first
NULL, DIM, DTYPE, SCALE, ALIAS, WORKSPACE = -1, -2, -3, -4, -8, -9
BIG = 1 << 31


def norm(**kw):
    a = dict(x=P[0], res=P[1], dt=1, w=P[2], h=P[3], y=P[4], yt=1, s=P[5], rstd=P[6], rows=8, width=64)
    a.update(kw)
    return g.lib().rms_norm(a["x"], a["res"], a["dt"], a["w"], 1e-5, a["h"], a["y"], a["yt"], a["s"], 0, a["rstd"],
                            a["rows"], a["width"], None)


def test_norm_refusals():
    assert norm(dt=2) == DTYPE and norm(yt=4) == DTYPE and norm(yt=-1) == DTYPE
    assert norm(rows=-1) == DIM and norm(width=BIG) == DIM
    for bad in (dict(x=None), dict(w=None), dict(y=None)):
        assert norm(**bad) == NULL, bad
    assert norm(yt=2, s=None) == SCALE and norm(yt=3, s=None) == SCALE
    for bad in (dict(h=P[0] + 2 * 8 * 64 - 2), dict(y=P[1]), dict(h=P[1] + 4), dict(y=P[3] + 8), dict(rstd=P[2] + 8),
                dict(yt=2, s=P[6]), dict(yt=2, s=P[4] + 8 * 64 - 1), dict(rstd=P[4] - 4)):
        assert norm(**bad) == ALIAS, bad
    assert norm(rows=0) == 0 and norm(width=0, x=None) == 0


def norm_back(**kw):
    a = dict(dy=P[0], dh=P[1], dt=1, h=P[2], hs=P[3], ht=1, w=P[4], rstd=P[5], dx=P[6], dw=P[7], rows=8, width=64,
             ws=P[8], n=1 << 30)
    a.update(kw)
    return g.lib().rms_norm_backward(a["dy"], a["dh"], a["dt"], a["h"], a["hs"], a["ht"], a["w"], a["rstd"], a["dx"],
                                     a["dw"], a["rows"], a["width"], a["ws"], a["n"], None)


def test_norm_backward_refusals():
    assert norm_back(dt=3) == DTYPE and norm_back(ht=5) == DTYPE
    assert norm_back(rows=BIG) == DIM and norm_back(width=-2) == DIM
    for bad in (dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(ws=None)):
        assert norm_back(**bad) == NULL, bad
    assert norm_back(ht=2, hs=None) == SCALE
    need = g.rms_norm_backward_workspace_size(8, 64)
    assert norm_back(n=need - 1) == WORKSPACE and norm_back(ws=P[8] + 8) == WORKSPACE
    for bad in (dict(dx=P[0]), dict(dx=P[1] + 2), dict(dw=P[4]), dict(ws=P[2] + 16), dict(dw=P[6] + 4),
                dict(ht=2, ws=P[3])):
        assert norm_back(**bad) == ALIAS, bad
    assert norm_back(width=0) == 0 and norm_back(rows=0, dw=None) == 0
    assert g.rms_norm_backward_workspace_size(0, 64) == 0
    with pytest.raises(g.GemmError):
        g.rms_norm_backward_workspace_size(-1, 4)


def product(kind, bt=True, **kw):
    a = dict(A=P[0], fa=0, B=P[1], fb=0, sA=P[2], sB=P[3], ch=1, so=P[4], bias=P[5], res=P[6], rt=1, C=P[7], out=1,
             act=1, Z=P[8], zs=P[9], zt=2, M=16, N=64, K=32)
    a.update(kw)
    tail = (a["bias"], a["res"], a["rt"], a["C"], a["out"], a["act"], a["Z"], a["zs"], a["zt"], a["M"], a["N"], a["K"],
            None)
    name = f"gemm_{kind}_bias_act" + ("_bt" if bt else "")
    if kind == "f16":
        return getattr(g.lib(), name)(a["A"], a["B"], *tail)
    return getattr(g.lib(), name)(a["A"], a["fa"], a["B"], a["fb"], a["sA"], a["sB"], a["ch"], a["so"], *tail)


@pytest.mark.parametrize("bt", [True, False])
@pytest.mark.parametrize("kind", ["f16", "fp8"])
def test_product_refusals(kind, bt):
    def call(**kw):
        return product(kind, bt, **kw)
    assert call(out=-1) == DTYPE and call(out=2 if kind == "f16" else 4) == DTYPE
    assert call(act=5) == DTYPE and call(act=-1) == DTYPE and call(rt=2) == DTYPE and call(zt=4) == DTYPE
    assert call(res=None, rt=9, C=P[0]) == ALIAS        # (a type without its matrix does not matter)
    for bad in (dict(M=-1), dict(N=BIG - 1), dict(K=BIG), dict(M=BIG - 65535)):
        assert call(**bad) == DIM, bad
    for bad in (dict(A=None), dict(B=None), dict(C=None)):
        assert call(**bad) == NULL, bad
    assert call(zs=None) == SCALE
    for bad in (dict(C=P[0]), dict(C=P[1] + 8), dict(C=P[5] + 4), dict(C=P[6]), dict(C=P[8] + 16), dict(Z=P[6] + 2),
                dict(zs=P[8] + 16 * 64 - 1), dict(zs=P[5] + 4 * 64 - 1), dict(zt=1, Z=P[7] - 2)):
        assert call(**bad) == ALIAS, bad
    if kind == "fp8":
        assert call(fa=2) == DTYPE and call(fb=-1) == DTYPE
        assert call(sA=None) == NULL and call(sB=None) == NULL
        assert call(out=2, so=None) == SCALE and call(out=3, so=None) == SCALE
        assert call(out=2, so=P[7]) == ALIAS
        assert call(sB=P[7] - 4 * 64 + 4) == ALIAS and call(sA=P[7] - 4 * 16 + 4) == ALIAS
    assert call(M=0) == 0 and call(N=0, C=None) == 0


def act_back(**kw):
    a = dict(dy=P[0], dt=1, z=P[1], zs=P[2], zt=2, act=2, dz=P[3], db=P[4], rows=8, cols=64, ws=P[5], n=1 << 30)
    a.update(kw)
    return g.lib().bias_act_backward(a["dy"], a["dt"], a["z"], a["zs"], a["zt"], a["act"], a["dz"], a["db"], a["rows"],
                                     a["cols"], a["ws"], a["n"], None)


def test_act_backward_refusals():
    assert act_back(dt=2) == DTYPE and act_back(zt=4) == DTYPE and act_back(act=7) == DTYPE
    assert act_back(rows=-1) == DIM and act_back(cols=BIG) == DIM
    for bad in (dict(dy=None), dict(z=None), dict(dz=None, db=None), dict(ws=None)):
        assert act_back(**bad) == NULL, bad
    assert act_back(zs=None) == SCALE
    need = g.bias_act_backward_workspace_size(8, 64)
    assert act_back(n=need - 1) == WORKSPACE and act_back(ws=P[5] + 4) == WORKSPACE
    for bad in (dict(dz=P[0]), dict(dz=P[1] + 8), dict(db=P[3] + 8), dict(ws=P[1]), dict(db=P[2]), dict(dz=P[4] - 2)):
        assert act_back(**bad) == ALIAS, bad
    assert act_back(cols=0) == 0 and act_back(rows=0, db=None) == 0


def test_mx_refusals():
    def pack(x=P[0], dt=1, rows=8, cols=40, fmt=0, q=P[1], s=P[2]):
        return g.lib().quantize_mx_fp8(x, dt, rows, cols, fmt, q, s, None)

    def unpack(q=P[0], s=P[1], fmt=0, rows=8, cols=40, y=P[2], dt=1):
        return g.lib().dequantize_mx_fp8(q, s, fmt, rows, cols, y, dt, None)
    for f in (pack, unpack):
        assert f(dt=2) == DTYPE and f(fmt=2) == DTYPE and f(rows=-1) == DIM and f(cols=BIG) == DIM
        assert f(q=None) == NULL and f(s=None) == NULL and f(rows=0) == 0 and f(cols=0) == 0
    assert pack(x=None) == NULL and unpack(y=None) == NULL
    assert pack(q=P[0] + 1) == ALIAS and pack(s=P[1] + 8 * 40 - 1) == ALIAS and pack(s=P[0] + 639) == ALIAS
    assert unpack(y=P[0] + 2) == ALIAS and unpack(y=P[1] + 14) == ALIAS


def test_wgrad_refusals():
    def call(q=P[0], s=P[1], fmt=0, b=P[2], off=P[3], c=P[4], out=0, rows=8, m=40, n=24, groups=2, second=0):
        return g.lib().gemm_mx_wgrad(q, s, fmt, b, off, c, out, rows, m, n, groups, second, None)
    assert call(out=2) == DTYPE and call(fmt=2) == DTYPE
    for bad in (dict(rows=-1), dict(m=BIG), dict(groups=-1), dict(groups=4097), dict(n=BIG - 65535)):
        assert call(**bad) == DIM, bad
    for bad in (dict(q=None), dict(b=None), dict(c=None), dict(off=None)):
        assert call(**bad) == NULL, bad
    assert call(s=None) == SCALE
    for bad in (dict(c=P[0] - 4), dict(c=P[1]), dict(c=P[2]), dict(c=P[3] + 8), dict(off=None, groups=1, c=P[0])):
        assert call(**bad) == ALIAS, bad
    assert call(groups=0, c=None) == 0 and call(m=0) == 0 and call(n=0, second=1) == 0


def test_binding_refusals():
    f16, f32 = torch.float16, torch.float32
    x, w = torch.zeros((4, 64), dtype=f16), torch.ones(64)
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    bad = [
        lambda: g.rms_norm(x.double(), w, x),
        lambda: g.rms_norm(x, w, x[:, :3]),
        lambda: g.rms_norm(x, w, codes),                                    # no scale
        lambda: g.rms_norm(x, w, x),                                        # host tensors
        lambda: g.rms_norm_backward(x, x.double(), w, w),
        lambda: g.rms_norm_backward(x, codes, w, w),                        # no hscale
        lambda: g.gemm_f16_bias_act(x, x, x),
        lambda: g.gemm_f16_bias_act_bt(x.float(), x, x),
        lambda: g.gemm_f16_bias_act_bt(x, x, torch.zeros((4, 4)), bias=torch.zeros(5)),
        lambda: g.gemm_f16_bias_act_bt(x, x, torch.zeros((4, 4)), residual=torch.zeros((4, 5))),
        lambda: g.gemm_f16_bias_act_bt(x, x, torch.zeros((4, 4)), Z=torch.zeros((4, 4), dtype=torch.uint8)),
        lambda: g.gemm_fp8_bias_act_bt(codes, 0, codes, 0, w, w, torch.zeros((4, 4))),          # one scale each
        lambda: g.gemm_fp8_bias_act_bt(codes, 0, codes, 0, w, w, torch.zeros((4, 4)), channel=True),
        lambda: g.gemm_fp8_bias_act_bt(codes.view(torch.float8_e5m2), 0, codes, 0, w, w, torch.zeros((4, 4))),
        lambda: g.bias_act_backward(x, x[:2], g.ACT_RELU),
        lambda: g.bias_act_backward(x, codes, g.ACT_RELU),
        lambda: g.quantize_mx_fp8(x.double()),
        lambda: g.quantize_mx_fp8(x, q=codes[:2], scale=scales),
        lambda: g.quantize_mx_fp8(x, q=codes, scale=scales[:, :1]),
        lambda: g.quantize_mx_fp8(x, g.FMT_E5M2, q=codes.view(torch.float8_e4m3fn), scale=scales),
        lambda: g.dequantize_mx_fp8(codes, scales.float(), g.FMT_E4M3, x),
        lambda: g.dequantize_mx_fp8(codes, scales, g.FMT_E4M3, x[:2]),
        lambda: g.gemm_mx_wgrad(codes, scales, g.FMT_E4M3, x[:2], torch.zeros((64, 64))),
        lambda: g.gemm_mx_wgrad(codes, scales, g.FMT_E4M3, x.float(), torch.zeros((64, 64))),
        lambda: g.gemm_mx_wgrad(codes, scales, g.FMT_E4M3, x, torch.zeros((64, 63))),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(f"call {i} went through")
    assert f32 is torch.float32


def test_queries():
    q = g.select_config_bias_act
    assert q(g.KIND_F16, g.OUT_F16, 1, 4096, 4096, b_kmajor=1) == "bias_act_gemv"
    assert q(g.KIND_FP8, g.OUT_F16, 1, 4096, 4096, b_kmajor=1) == "bias_act_ring"
    assert q(g.KIND_F16, g.OUT_F16, 1, 4096, 4096, b_kmajor=1, z_dtype=g.OUT_E4M3) != "bias_act_gemv"
    assert q(g.KIND_F16, g.OUT_F16, 1, 4096, 4096) == "bias_act_ring"
    assert q(g.KIND_F16, g.OUT_F16, 16, 4096, 4096, b_kmajor=1) == "bias_act_ring"
    assert q(g.KIND_FP8, g.OUT_F16, 16384, 12288, 4096, b_kmajor=1) == "bias_act_pp_256"
    assert q(g.KIND_FP8, g.OUT_F16, 16384, 12288, 4096, fmt_a=1, b_kmajor=1) == "bias_act_pp_192"
    assert q(g.KIND_F16, g.OUT_F32, 300, 77, 33).startswith("bias_act_tile")
    assert q(g.KIND_F16, g.OUT_F32, 300, 77, 0) == "bias_act_tile_64"
    assert g.select_config_mx_wgrad(g.OUT_F32, 8192, 4096, 4096) == "wgrad_pp"
    assert g.select_config_mx_wgrad(g.OUT_F32, 8192, 4100, 4096) != "wgrad_pp"
    for f in (lambda: q(2, 1, 1, 1, 1), lambda: q(0, 2, 1, 1, 1), lambda: q(1, 1, 1, 1, 1, fmt_a=3),
              lambda: q(1, 1, -1, 1, 1), lambda: q(1, 1, 1, 1, 1, z_dtype=4),
              lambda: g.select_config_mx_wgrad(2, 1, 1, 1), lambda: g.select_config_mx_wgrad(0, 1, 1, 1, 5000)):
        with pytest.raises(g.GemmError):
            f()


def test_split_stays_small(monkeypatch):
    """Sixteen waves per workgroup only where a launch of them stays far below 2^32 threads, and not for fewer than
    eight columns of either operand."""
    q = g.select_config_mx_wgrad
    monkeypatch.setenv("LIBGEMM_CONFIG", "wgrad_tile_64_split")
    assert q(g.OUT_F32, 5000, 400, 72) == "wgrad_tile_64_split"
    assert q(g.OUT_F32, 4, 1 << 17, 1 << 16) != "wgrad_tile_64_split"
    assert q(g.OUT_F32, 4, 1 << 12, 1 << 12, 4096) != "wgrad_tile_64_split"
    assert q(g.OUT_F32, 5000, 7, 72) != "wgrad_tile_64_split" and q(g.OUT_F32, 5000, 72, 7) != "wgrad_tile_64_split"
    monkeypatch.delenv("LIBGEMM_CONFIG")
    assert q(g.OUT_F32, 8155, 464, 72) == "wgrad_tile_64_split"
    assert q(g.OUT_F32, 8192, 4096, 4096) == "wgrad_pp"
