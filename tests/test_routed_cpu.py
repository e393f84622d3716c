"""Refusals of the products whose weight depends on the row and of expert
routing: invalid arguments return before anything touches a GPU (no GPU
needed), and the binding checks types and shapes."""
import pytest
import torch

import precision_dense_gemm_03_amd as g

P = [i << 40 for i in range(1, 20)]     # never dereferenced: every call below fails validation first
NULL, DIM, DTYPE, SCALE, ALIAS, WORKSPACE = -1, -2, -3, -4, -8, -9


def f16_grouped(**kw):
    a = dict(A=P[0], B=P[1], off=P[2], C=P[3], out=1, rows=8, N=16, K=16, groups=2)
    a.update(kw)
    return [f(a["A"], a["B"], a["off"], a["C"], a["out"], a["rows"], a["N"], a["K"], a["groups"], None)
            for f in (g.lib().gemm_f16_grouped, g.lib().gemm_f16_grouped_bt)]


def test_grouped_f16_refusals():
    assert f16_grouped(out=2) == [DTYPE] * 2 and f16_grouped(out=-1) == [DTYPE] * 2
    for bad in (dict(rows=-1), dict(N=1 << 31), dict(K=-5), dict(groups=-1), dict(groups=4097),
                dict(N=(1 << 31) - 1, K=(1 << 31) - 1, groups=4096)):
        assert f16_grouped(**bad) == [DIM] * 2, bad
    for bad in (dict(A=None), dict(B=None), dict(off=None), dict(C=None)):
        assert f16_grouped(**bad) == [NULL] * 2, bad
    for bad in (dict(C=P[0] + 8), dict(C=P[1] + 2 * 16 * 16 * 2 - 2), dict(C=P[2] + 8)):
        assert f16_grouped(**bad) == [ALIAS] * 2, bad
    assert f16_grouped(rows=0) == [0] * 2 and f16_grouped(N=0, C=None) == [0] * 2


def fp8_grouped(channel, **kw):
    a = dict(A=P[0], fa=0, B=P[1], fb=0, off=P[2], sA=P[3], sB=P[4], sOut=P[5], C=P[6], out=1, rows=8, N=16, K=16,
             groups=2)
    a.update(kw)
    name = "gemm_fp8_grouped" + ("_channel" if channel else "")
    return [getattr(g.lib(), name + s)(a["A"], a["fa"], a["B"], a["fb"], a["off"], a["sA"], a["sB"], a["sOut"], a["C"],
                                       a["out"], a["rows"], a["N"], a["K"], a["groups"], None) for s in ("", "_bt")]


@pytest.mark.parametrize("channel", [False, True])
def test_grouped_fp8_refusals(channel):
    assert fp8_grouped(channel, out=4) == [DTYPE] * 2 and fp8_grouped(channel, fa=2) == [DTYPE] * 2
    assert fp8_grouped(channel, fb=-1) == [DTYPE] * 2
    assert fp8_grouped(channel, groups=5000) == [DIM] * 2
    for bad in (dict(sA=None), dict(sB=None), dict(A=None), dict(off=None)):
        assert fp8_grouped(channel, **bad) == [NULL] * 2, bad
    assert fp8_grouped(channel, out=2, sOut=None) == [SCALE] * 2
    assert fp8_grouped(channel, out=3, sOut=P[6]) == [ALIAS] * 2
    # the scales' extents follow the call
    last = P[6] - 4 * (2 * 16 if channel else 2)
    assert fp8_grouped(channel, sB=last + 4) == [ALIAS] * 2
    assert fp8_grouped(channel, sA=P[6] - (4 * 8 if channel else 4) + 4) == [ALIAS] * 2


def test_wgrad_refusals():
    def call(A=P[0], B=P[1], off=P[2], C=P[3], out=0, rows=8, M=16, N=16, groups=2):
        return g.lib().gemm_f16_grouped_wgrad(A, B, off, C, out, rows, M, N, groups, None)
    assert call(out=2) == DTYPE and call(groups=-1) == DIM and call(M=-1) == DIM
    assert call(A=None) == NULL and call(C=None) == NULL and call(off=None) == NULL
    assert call(C=P[1] + 4) == ALIAS and call(groups=0, C=None) == 0 and call(N=0) == 0


def lora(kind, **kw):
    a = dict(A=P[0], fa=0, B=P[1], fb=0, sA=P[2], sB=P[3], X=P[4], LA=P[5], LB=P[6], ad=P[7], ls=P[8], C=P[9], out=1,
             rows=8, N=16, K=16, rank=4, adapters=3, ws=P[10], wsb=8 * 8 * 4)
    a.update(kw)
    tail = (a["LA"], a["LB"], a["ad"], a["ls"], a["C"], a["out"], a["rows"], a["N"], a["K"], a["rank"], a["adapters"],
            a["ws"], a["wsb"], None)
    if kind == "f16":
        return g.lib().gemm_f16_lora_bt(a["A"], a["B"], *tail)
    return g.lib().gemm_fp8_lora_bt(a["A"], a["fa"], a["B"], a["fb"], a["sA"], a["sB"], a["X"], *tail)


@pytest.mark.parametrize("kind", ["f16", "fp8"])
def test_lora_refusals(kind):
    assert lora(kind, out=2) == DTYPE
    for bad in (dict(rows=-1), dict(rank=-1), dict(adapters=1 << 31), dict(rank=(1 << 31) - 1)):
        assert lora(kind, **bad) == DIM, bad
    for bad in (dict(A=None), dict(B=None), dict(C=None), dict(LA=None), dict(LB=None), dict(ad=None), dict(ls=None),
                dict(ws=None)):
        assert lora(kind, **bad) == NULL, bad
    if kind == "fp8":
        assert lora(kind, X=None) == NULL and lora(kind, sA=None) == NULL and lora(kind, fa=3) == DTYPE
    assert lora(kind, wsb=8 * 8 * 4 - 1) == WORKSPACE and lora(kind, ws=P[10] + 4) == WORKSPACE
    for bad in (dict(C=P[10] + 16), dict(C=P[5]), dict(ws=P[7]), dict(ws=P[0] + 16)):
        assert lora(kind, **bad) == ALIAS, bad
    assert lora(kind, rows=0, ws=None) == 0
    assert g.lib().gemm_lora_workspace_size(5, 9) == 5 * 16 * 4
    assert g.lib().gemm_lora_workspace_size(-1, 9) == DIM


def test_route_refusals():
    L = g.lib()

    def call(lg=P[0], T=100, E=16, K=2, ex=P[1], w=P[2], off=P[3], row=P[4], tok=P[5], ws=P[6], wsb=1 << 20):
        return L.moe_route_f32(lg, T, E, K, 1, ex, w, off, row, tok, ws, wsb, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(K=33, E=64),
                dict(T=(1 << 31) - 1, K=2)):
        assert call(**bad) == DIM, bad
    for bad in ("lg", "ex", "w", "off", "row", "tok", "ws"):
        assert call(**{bad: None}) == NULL, bad
    assert call(wsb=2 * 16 * 4 - 1) == WORKSPACE and call(ws=P[6] + 8) == WORKSPACE
    assert call(row=P[1] + 4) == ALIAS and call(tok=P[0]) == ALIAS and call(off=P[6]) == ALIAS
    assert L.moe_route_workspace_size(64, 16) == 0 and L.moe_route_workspace_size(65, 16) == 2 * 16 * 4
    assert L.moe_route_workspace_size(1 << 20, 1024) == 256 * 1024 * 4
    assert L.moe_route_workspace_size(1, 2000) == DIM
    assert L.moe_route_backward_f32(P[0], P[1], P[2], P[3], 4, 8, 9, 1, P[4], None) == DIM
    assert L.moe_route_backward_f32(P[0], P[1], P[2], None, 4, 8, 2, 1, P[4], None) == NULL
    assert L.moe_route_backward_f32(P[0], P[1], P[2], P[3], 4, 8, 2, 1, P[0], None) == ALIAS


def test_rows_refusals():
    L = g.lib()
    assert L.moe_gather(P[0], P[1], P[2], 4, 8, 16, 3, None) == DTYPE
    assert L.moe_gather(P[0], P[1], P[2], 4, -8, 16, 2, None) == DIM
    assert L.moe_gather(P[0], None, P[2], 4, 8, 16, 2, None) == NULL
    assert L.moe_gather(P[0], P[1], P[0] + 100, 4, 8, 16, 2, None) == ALIAS
    assert L.moe_gather(None, None, None, 4, 0, 16, 2, None) == 0
    assert L.moe_combine(P[0], 2, P[1], P[2], P[3], 1, 4, 2, 8, 16, None) == DTYPE
    assert L.moe_combine(P[0], 1, P[1], P[2], P[3], 3, 4, 2, 8, 16, None) == DTYPE
    assert L.moe_combine(P[0], 1, P[1], P[2], P[3], 1, 4, 33, 8, 16, None) == DIM
    assert L.moe_combine(P[0], 1, None, P[2], P[3], 1, 4, 2, 8, 16, None) == NULL
    assert L.moe_combine(P[0], 1, P[1], P[2], P[2] + 4, 1, 4, 2, 8, 16, None) == ALIAS
    assert L.moe_combine_backward(P[0], P[1], 2, P[2], P[3], P[4], P[5], 4, 2, 8, 16, None) == DTYPE
    assert L.moe_combine_backward(P[0], P[1], 1, P[2], None, P[4], P[5], 4, 2, 8, 16, None) == NULL
    assert L.moe_combine_backward(P[0], P[1], 1, P[2], P[3], P[1], P[5], 4, 2, 8, 16, None) == ALIAS
    assert L.moe_combine_backward(P[0], P[1], 1, P[2], P[3], P[4], P[4] + 4, 4, 2, 8, 16, None) == ALIAS


def test_binding_refusals():
    h, f, i = torch.float16, torch.float32, torch.int32
    a, b, c = torch.empty((4, 8), dtype=h), torch.empty((2, 8, 6), dtype=h), torch.empty((4, 6), dtype=h)
    off = torch.zeros(3, dtype=i)
    for bad in ((a.float(), b, off, c), (a, b[0], off, c), (a, b, off[:2], c), (a, b, off.long(), c),
                (a, b, off, c[:, :5]), (a, b.transpose(1, 2), off, c), (a, b, off, c.bfloat16())):
        with pytest.raises(ValueError):
            g.gemm_f16_grouped(*bad)
    with pytest.raises(ValueError, match="device tensors"):
        g.gemm_f16_grouped(a, b, off, c)
    qa, qb = torch.empty((4, 8), dtype=torch.uint8), torch.empty((2, 6, 8), dtype=torch.uint8)
    with pytest.raises(ValueError, match="sB"):
        g.gemm_fp8_grouped_bt(qa, 0, qb, 0, off, torch.ones(1), torch.ones(3), c)
    with pytest.raises(ValueError, match="sA"):
        g.gemm_fp8_grouped_channel_bt(qa, 0, qb, 0, off, torch.ones(1), torch.ones((2, 6)), c)
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_wgrad(a, a[:3], off, torch.empty((2, 8, 8)))
    la, lb, ad, ls = torch.empty((3, 2, 8), dtype=h), torch.empty((3, 6, 2), dtype=h), off[:1].repeat(4), torch.ones(3)
    bt = torch.empty((6, 8), dtype=h)
    for bad in ((a, bt, la[:, :, :7], lb, ad, ls, c), (a, bt, la, lb[:2], ad, ls, c), (a, bt, la, lb, ad[:3], ls, c),
                (a, bt, la, lb, ad, ls.half(), c), (a, bt, la.float(), lb, ad, ls, c)):
        with pytest.raises(ValueError):
            g.gemm_f16_lora_bt(*bad)
    lg = torch.empty((4, 8))
    for bad in (dict(topk=9), dict(topk=0), dict(topk=2, expert=torch.empty((4, 3), dtype=i)),
                dict(topk=2, offsets=torch.empty(8, dtype=i)), dict(topk=2, weight=torch.empty((4, 2), dtype=h))):
        with pytest.raises(ValueError):
            g.moe_route_f32(lg, **bad)
    with pytest.raises(ValueError):
        g.moe_route_f32(lg.half(), 2)
    with pytest.raises(ValueError):
        g.moe_gather(a, off, torch.empty((3, 8)))
    with pytest.raises(ValueError):
        g.moe_combine(a, ad.reshape(2, 2), torch.ones((2, 1)))
    with pytest.raises(ValueError):
        g.moe_combine_backward(a, a, ad.reshape(2, 2), torch.ones((2, 2)))


LARGEST = (1 << 31) - 65536


@pytest.mark.parametrize("size", [LARGEST + 1, (1 << 31) - 200, (1 << 31) - 1])
def test_sizes_whose_last_tile_passes_2_to_31(size):
    """Row, column and K indices run past the size, to the end of a tile or a step, in 32 bits: refused before any
    launch."""
    small = dict(rows=1, N=1, K=1, groups=1, A=1 << 50, B=2 << 50, off=3 << 50, C=4 << 50)
    for which in ("rows", "N", "K"):
        assert f16_grouped(**{**small, which: size}) == [DIM] * 2, which
        fp8 = {**small, which: size, "sA": 5 << 50, "sB": 6 << 50}
        assert fp8_grouped(False, **fp8) == [DIM] * 2 and fp8_grouped(True, **fp8) == [DIM] * 2, which
    L = g.lib()
    for dims in ((size, 1, 1), (1, size, 1), (1, 1, size)):
        assert L.gemm_f16_grouped_wgrad(1 << 50, 2 << 50, 3 << 50, 4 << 50, 0, *dims, 1, None) == DIM, dims
    far = dict(rows=1, N=1, K=1, rank=1, adapters=1, wsb=1 << 45, **{n: (i + 1) << 50 for i, n in enumerate(
        ("A", "B", "sA", "sB", "X", "LA", "LB", "ad", "ls", "C", "ws"))})
    for which in ("rows", "N", "K", "rank"):
        for kind in ("f16", "fp8"):
            assert lora(kind, **{**far, which: size}) == DIM, which
    assert L.gemm_lora_workspace_size(size, 1) == DIM and L.gemm_lora_workspace_size(1, size) == DIM


def test_largest_sizes_are_taken():
    assert g.lib().gemm_lora_workspace_size(LARGEST, 1) == LARGEST * 8 * 4
    for which in ("N", "K"):
        assert f16_grouped(**{**dict(rows=0, N=1, K=1), which: LARGEST}) == [0, 0]
    assert f16_grouped(rows=LARGEST, N=0) == [0, 0]


def test_select_config_of_the_routed_calls(monkeypatch):
    monkeypatch.delenv("LIBGEMM_CONFIG", raising=False)
    h, f8 = g.KIND_F16, g.KIND_FP8
    sel, lo, wg = g.select_config_grouped, g.select_config_lora, g.select_config_wgrad
    assert sel(h, g.OUT_F16, 16, 4096, 4096, 16, b_kmajor=1) == "grouped_ring"
    assert sel(h, g.OUT_F16, 5003, 1416, 2048, 32) == "grouped_pp_128"
    assert sel(f8, g.OUT_F16, 16384, 12288, 4096, 16, b_kmajor=1) == "grouped_pp_256"
    assert sel(f8, g.OUT_F16, 16384, 4096, 4096, 16, 1, 0, 1) == "grouped_pp_192"       # E5M2 pairs: one height
    assert sel(h, g.OUT_F16, 5000, 4096, 1001, 4, b_kmajor=1).startswith("grouped_tile")   # rows of no whole 16 bytes
    assert wg(g.OUT_F32, 8192, 2048, 4096, 8) == "wgrad_pp" and wg(g.OUT_F32, 8192, 2047, 4096, 8) != "wgrad_pp"
    assert lo(h, g.OUT_F16, 16, 4096, 4096, 16, 16) == "lora_ring" and lo(h, g.OUT_F16, 4096, 4096, 4096, 64, 8) == "lora_pp_256"
    monkeypatch.setenv("LIBGEMM_CONFIG", "grouped_pp_256")
    assert sel(h, g.OUT_F16, 16, 4096, 4096, 16) == "grouped_pp_256"
    assert sel(f8, g.OUT_F16, 16, 4096, 4096, 16, 0, 1) == "grouped_pp_192"
    assert sel(h, g.OUT_F16, 16, 4096, 4095, 16, b_kmajor=1) != "grouped_pp_256"            # not its operands
    monkeypatch.setenv("LIBGEMM_CONFIG", "wgrad_tile_64")
    assert wg(g.OUT_F32, 8192, 2048, 4096, 8) == "wgrad_tile_64"
    monkeypatch.setenv("LIBGEMM_CONFIG", "lora_pp_256")
    assert lo(f8, g.OUT_F16, 4, 64, 64, 8, 2, 1, 1) == "lora_pp_192" and lo(f8, g.OUT_F16, 4, 64, 64, 8, 2) == "lora_pp_256"


def test_select_config_of_the_routed_calls_refusals():
    import ctypes
    L, buf = g.lib(), ctypes.create_string_buffer(64)
    assert L.gemm_select_config_grouped(2, 0, 1, 1, 1, 1, 0, 0, 0, buf, 64) == DTYPE
    assert L.gemm_select_config_grouped(0, 2, 1, 1, 1, 1, 0, 0, 0, buf, 64) == DTYPE
    assert L.gemm_select_config_grouped(1, 3, 1, 1, 1, 1, 2, 0, 0, buf, 64) == DTYPE
    assert L.gemm_select_config_grouped(1, 3, 1, 1, 1, 4097, 0, 0, 0, buf, 64) == DIM
    assert L.gemm_select_config_grouped(1, 3, 1, 1, 1, 1, 0, 0, 0, None, 64) == NULL
    assert L.gemm_select_config_grouped(1, 3, 0, 0, 0, 0, 0, 0, 0, buf, 64) == 0
    assert L.gemm_select_config_wgrad(2, 1, 1, 1, 1, buf, 64) == DTYPE
    assert L.gemm_select_config_wgrad(0, -1, 1, 1, 1, buf, 64) == DIM
    assert L.gemm_select_config_wgrad(0, 0, 0, 0, 0, buf, 0) == NULL and L.gemm_select_config_wgrad(0, 0, 0, 0, 0, buf, 8) == 0
    assert L.gemm_select_config_lora(1, 2, 1, 1, 1, 1, 1, 0, 0, buf, 64) == DTYPE
    assert L.gemm_select_config_lora(1, 1, 1, 1, 1, 1 << 31, 1, 0, 0, buf, 64) == DIM
    assert L.gemm_select_config_lora(1, 1, 0, 0, 0, 0, 0, 0, 0, buf, 64) == 0
