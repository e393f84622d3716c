"""A dense layer's calls together: one training step of norm, two products with
their epilogues and every gradient, one decoding step in FP8, each alone, on
other streams, two at once, and captured as a graph and replayed.

Bounds follow the calls: every value carries how far it may be from the 64-bit
one, each call adds its own error (dense_ref.py) and passes on its inputs' by
its derivatives' bounds. The second derivative of the activations is at most 1
(GELU: 2 / sqrt(2 pi) = 0.80, its tanh form the same to 0.02, SiLU 0.5)."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from dense_ref import (REL, STEEPEST, act, act_error, code_step, norm, norm_backward, powers, slope, slope_error, spread,
                       stored, values)
from routed_ref import check
from test_gpu_norm import DEV, F16, F32, _gpu, gen, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5
CURVE = 1.0
NAMES = {"gelu": g.ACT_GELU, "gelu_tanh": g.ACT_GELU_TANH, "silu": g.ACT_SILU}


class Layer:
    """out = h + W2 act(W1 norm(h) + b1) + b2 with h = x + residual; W1 [hidden, width] and W2 [width, hidden] as the
    _bt calls take them. The normalised rows, the activation and z are kept in 8 bits."""

    def __init__(self, rows, width, hidden, name, seed=0):
        gn = gen(seed + rows + 3 * width + 5 * hidden)
        self.name, self.act = name, NAMES[name]
        self.x = normal(gn, (rows, width)).half()
        self.res = normal(gn, (rows, width)).half()
        self.w = 1.0 + normal(gn, (width,), 0.2)
        self.w1 = (normal(gn, (hidden, width)) / width ** 0.5).half()
        self.b1 = normal(gn, (hidden,), 0.3)
        self.w2 = (normal(gn, (width, hidden)) / hidden ** 0.5).half()
        self.b2 = normal(gn, (width,), 0.3)
        self.dout = normal(gn, (rows, width)).half()

        def new(shape, dtype):
            return torch.full(shape, 7, dtype=dtype, device=DEV)

        def mx(cols):
            return new((rows, cols), torch.uint8), new((rows, (cols + 31) // 32), torch.uint8)

        self.h, self.y, self.out, self.dx, self.dy = (new((rows, width), F16) for _ in range(5))
        self.rstd = new((rows,), F32)
        self.a, self.da, self.dz = (new((rows, hidden), F16) for _ in range(3))
        self.qy, self.qa, self.qz = mx(width), mx(hidden), mx(hidden)
        self.dw, self.db2 = new((width,), F32), new((width,), F32)
        self.db1 = new((hidden,), F32)
        self.dw1, self.dw2 = new((hidden, width), F32), new((width, hidden), F32)
        self.work = torch.empty(max(g.rms_norm_backward_workspace_size(rows, width),
                                    g.bias_act_backward_workspace_size(rows, hidden),
                                    g.bias_act_backward_workspace_size(rows, width), 16), dtype=torch.uint8, device=DEV)

    def step(self):
        g.rms_norm(self.x, self.w, self.y, eps=EPS, residual=self.res, h=self.h, rstd=self.rstd)
        g.quantize_mx_fp8(self.y, q=self.qy[0], scale=self.qy[1])
        g.gemm_f16_bias_act_bt(self.y, self.w1, self.a, bias=self.b1, act=self.act, Z=self.qz[0], Zscale=self.qz[1],
                               z_fmt=g.FMT_E4M3)
        g.quantize_mx_fp8(self.a, q=self.qa[0], scale=self.qa[1])
        g.gemm_f16_bias_act_bt(self.a, self.w2, self.out, bias=self.b2, residual=self.h)

        g.bias_act_backward(self.dout, None, g.ACT_NONE, dZ=self.dy, dbias=self.db2, workspace=self.work)
        g.gemm_mx_wgrad(*self.qa, g.FMT_E4M3, self.dout, self.dw2, q_second=True)
        g.gemm_f16(self.dout, self.w2, self.da)
        g.bias_act_backward(self.da, self.qz[0], self.act, dZ=self.dz, dbias=self.db1, Zscale=self.qz[1], z_fmt=g.FMT_E4M3,
                            workspace=self.work)
        g.gemm_mx_wgrad(*self.qy, g.FMT_E4M3, self.dz, self.dw1, q_second=True)
        g.gemm_f16(self.dz, self.w1, self.dy)
        g.rms_norm_backward(self.dy, self.h, self.w, self.rstd, dx=self.dx, dweight=self.dw, dh=self.dout,
                            workspace=self.work)

    def results(self):
        return {"h": self.h, "out": self.out, "qy": self.qy[0], "sy": self.qy[1], "qz": self.qz[0], "sz": self.qz[1],
                "dx": self.dx, "dw": self.dw, "dw1": self.dw1, "db1": self.db1, "dw2": self.dw2, "db2": self.db2}

    def inputs(self):
        return [t.double() for t in (self.x, self.res, self.w, self.w1, self.b1, self.w2, self.b2)]


def forward(x, res, w, w1, b1, w2, b2, name):
    """The layer in 64 bits, with what the gradients need."""
    h = x + res
    y, rstd = norm(h, w, EPS)
    z = y @ w1.t() + b1
    return h + act(z, name) @ w2.t() + b2, h, y, rstd, z


def backward(p, h, y, rstd, z, dout, name):
    """Gradients of x, w, w1, b1, w2 and b2 by the formulas, 64 bits."""
    _, _, w, w1, _, w2, _ = p
    dz = (dout @ w2) * slope(z, name)
    dx, dw, _, _ = norm_backward(dz @ w1, h, w, rstd, dout)
    return dx, dw, dz.t() @ y, dz.sum(dim=0), dout.t() @ act(z, name), dout.sum(dim=0)


def product(a, ea, b, eb=None):
    """(a @ b, its error) of values a off by ea and b off by eb."""
    A, B = a.abs() + ea, b.abs()
    e = ea @ B + REL * (A @ B)
    if eb is not None:
        e = e + A @ eb * (1 + REL)
    return a @ b, e


def half(v, e):
    return e + stored(v.abs() + e, F16)


def kept(v, e, scale):
    return e + code_step(v.abs() + e, spread(powers(scale), v.shape[1]), "e4m3")


def within(layer):
    """Every result of a step against 64 bits."""
    name, p = layer.name, layer.inputs()
    x, res, w, w1, b1, w2, b2 = p
    dout = layer.dout.double()
    out, h, y, r, z = forward(*p, name)
    eh = half(h, h.abs() * 2.0 ** -23)
    off = (2 * h.abs() * eh + eh * eh).mean(dim=1)
    er = (0.5 * off * ((h * h).mean(dim=1) + EPS - off) ** -1.5 + REL * r)[:, None]
    rc = r[:, None]
    en = eh * (rc + er) + h.abs() * er
    ey = half(y, w.abs() * en + REL * y.abs())
    v, ez = product(y, ey, w1.t())
    ez = ez + (v.abs() + z.abs()) * 2.0 ** -22
    a = act(z, name)
    ea = half(a, STEEPEST * ez + act_error(z, name))
    v, eo = product(a, ea, w2.t())
    eo = half(out, eo + eh + (v.abs() + out.abs()) * 2.0 ** -21)
    check(layer.h, h, eh, "h")
    check(layer.out, out, eo, "out")
    check(values(*layer.qz, "e4m3"), z, kept(z, ez, layer.qz[1]), "z")

    eyk, eak, ezk = kept(y, ey, layer.qy[1]), kept(a, ea, layer.qa[1]), kept(z, ez, layer.qz[1])
    dx, dw, dw1, db1, dw2, db2 = backward(p, h, y, r, z, dout, name)
    zero = torch.zeros_like(dout)
    check(layer.db2, db2, REL * dout.abs().sum(dim=0), "db2")
    _, e = product(dout.t(), zero.t(), a, eak)
    check(layer.dw2, dw2, e + stored(dw2, F32), "dw2")
    da, eda = product(dout, zero, w2)
    eda = half(da, eda)
    s = slope(z, name)
    es = CURVE * ezk + slope_error(z, name)
    dz = da * s
    edz = eda * (s.abs() + es) + da.abs() * es + REL * dz.abs()
    check(layer.db1, db1, edz.sum(dim=0) + REL * (dz.abs() + edz).sum(dim=0), "db1")
    edz = half(dz, edz)
    _, e = product(dz.t(), edz.t(), y, eyk)
    check(layer.dw1, dw1, e + stored(dw1, F32), "dw1")
    dy, edy = product(dz, edz, w1)
    edy = half(dy, edy)
    n, gr = h * rc, dy * w
    eg = w.abs() * edy
    c = (gr * n).mean(dim=1, keepdim=True)
    ec = (eg * (n.abs() + en) + gr.abs() * en).mean(dim=1, keepdim=True) + REL * (gr * n).abs().mean(dim=1, keepdim=True)
    mag = rc * (gr.abs() + n.abs() * (gr * n).abs().mean(dim=1, keepdim=True)) + dout.abs()
    e = er * (gr - n * c).abs() + (rc + er) * (eg + en * c.abs() + (n.abs() + en) * ec) + REL * mag
    check(layer.dx, dx, half(dx, e), "dx")
    e = (edy * (n.abs() + en) + dy.abs() * en).sum(dim=0) + REL * ((dy.abs() + edy) * (n.abs() + en)).sum(dim=0)
    check(layer.dw, dw, e, "dw")


SIZES = [(1, 64, 96), (7, 129, 77), (65, 200, 136), (200, 256, 520), (300, 1000, 264), (1030, 512, 1288)]


@pytest.mark.parametrize("name", list(NAMES))
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_training_step(rows, width, hidden, name):
    say(f"step of {rows} rows, {width} -> {hidden}, {name}")
    layer = Layer(rows, width, hidden, name)
    layer.step()
    within(layer)


@pytest.mark.parametrize("name", list(NAMES))
def test_formula_against_differences(name):
    """The formulas' gradients against central differences of the layer in 64 bits along random directions: off by the
    third derivative's share of h^2 (1e-10 of values of some hundreds) and 2^-53 / h of the loss."""
    layer = Layer(19, 64, 96, name)
    p, dout = layer.inputs(), layer.dout.double()
    out, h, y, r, z = forward(*p, name)
    grads = backward(p, h, y, r, z, dout, name)
    gn = gen(5)
    for at, grad in zip((0, 2, 3, 4, 5, 6), grads):
        d = torch.randn(p[at].shape, generator=gn, device=DEV, dtype=torch.float64)
        step = 1e-5
        loss = [(forward(*[q + (t * step * d if i == at else 0.0) for i, q in enumerate(p)], name)[0] * dout).sum()
                for t in (1, -1)]
        got, want = (loss[0] - loss[1]) / (2 * step), (grad * d).sum()
        assert abs(float(got - want)) <= 1e-5 * float((grad * d).abs().sum()), (at, float(got), float(want))


def snapshot(layer):
    return {k: t.clone() for k, t in layer.results().items()}


def same(layer, first, what):
    for k, t in layer.results().items():
        assert torch.equal(t, first[k]), f"{what}: {k}"


def test_two_layers_on_two_streams():
    """Two steps at once on streams of their own, buffers apart: each as alone."""
    layers = [Layer(300, 512, 1288, "gelu"), Layer(301, 520, 1032, "silu", seed=1)]
    for x in layers:
        x.step()
    first = [snapshot(x) for x in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    say("two layers at once")
    for turn in range(3):
        for x in layers:
            for t in x.results().values():
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for x, s in zip(layers, streams):
                with torch.cuda.stream(s):
                    x.step()
        torch.cuda.synchronize()
        for x, f in zip(layers, first):
            same(x, f, f"turn {turn}")


@pytest.mark.parametrize("rows,width,hidden", [(7, 129, 77), (300, 512, 1288)])
def test_captured_step(rows, width, hidden):
    """The step as a graph, replayed for other inputs, with eager work between."""
    layer = Layer(rows, width, hidden, "gelu")
    layer.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.current_stream().wait_stream(side)
    say("capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    gn = gen(11)
    for turn in range(4):
        layer.x.copy_(normal(gn, (rows, width)).half())
        layer.dout.copy_(normal(gn, (rows, width)).half())
        layer.step()
        first = snapshot(layer)
        for t in layer.results().values():
            t.zero_()
        layer.work.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        (layer.w1.float() @ layer.y.float().t()).sum()
        torch.cuda.synchronize()
        same(layer, first, f"replay {turn}")
    within(layer)


class Decode:
    """A decoding step of two layers on FP8 weights with a scale per column: norm into codes, product with bias and SiLU
    into codes, product onto the residual, and the next layer's norm joins what came before."""

    def __init__(self, rows, width, hidden, layers=2):
        gn = gen(rows + width)
        e4 = torch.float8_e4m3fn

        def new(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=DEV)

        def weight(n, k):
            w = normal(gn, (n, k)) / k ** 0.5
            s = w.abs().amax(dim=1) / 448.0
            return (w / s[:, None]).to(e4), s

        self.rows, self.width = rows, width
        self.x = normal(gn, (rows, width)).half()
        self.res = normal(gn, (rows, width)).half()
        self.layers = [{"w": 1.0 + normal(gn, (width,), 0.2), "w1": weight(hidden, width), "b1": normal(gn, (hidden,), 0.3),
                        "w2": weight(width, hidden), "b2": normal(gn, (width,), 0.3), "h": new((rows, width), F16),
                        "q": new((rows, width), e4), "s": new((rows,), F32), "a": new((rows, hidden), e4),
                        "out": new((rows, width), F16)} for _ in range(layers)]
        self.sout = torch.full((1,), 6.0 / 448.0, device=DEV)
        self.sa = self.sout.expand(rows).contiguous()

    def step(self):
        x, res = self.x, self.res
        for t in self.layers:
            g.rms_norm(x, t["w"], t["q"], eps=EPS, residual=res, h=t["h"], scale=t["s"])
            g.gemm_fp8_bias_act_bt(t["q"], g.FMT_E4M3, t["w1"][0], g.FMT_E4M3, t["s"], t["w1"][1], t["a"], bias=t["b1"],
                                   act=g.ACT_SILU, channel=True, sOut=self.sout)
            g.gemm_fp8_bias_act_bt(t["a"], g.FMT_E4M3, t["w2"][0], g.FMT_E4M3, self.sa, t["w2"][1], t["out"], bias=t["b2"],
                                   channel=True)
            x, res = t["out"], t["h"]
        return x

    def check_step(self):
        """Each call against 64 bits on what it was given (the matrix cores' FP8 sums within 2^-9 of the magnitudes)."""
        x, res = self.x, self.res
        for i, t in enumerate(self.layers):
            h = (x.float() + res.float()).half()
            assert torch.equal(t["h"], h), i
            v, _ = norm(h.double(), t["w"].double(), EPS)
            s = v.abs().amax(dim=1) / 448.0
            check(t["s"], s, s * REL, "scale")
            got = t["s"].double()[:, None]
            check(t["q"].double() * got, v, code_step(v, got, "e4m3") * (1 + 2 * REL) + v.abs() * 2 * REL, "codes")
            for a, sa, w, b, y in ((t["q"], t["s"], t["w1"], t["b1"], t["a"]), (t["a"], self.sa, t["w2"], t["b2"], t["out"])):
                av, bv = a.double() * sa.double()[:, None], w[0].double() * w[1].double()[:, None]
                z = av @ bv.t() + b.double()
                e = 2.0 ** -9 * (av.abs() @ bv.abs().t()) + z.abs() * 2.0 ** -20
                if y.dtype == F16:
                    check(y, z, half(z, e), "out")
                else:
                    u = act(z, "silu") / self.sout.double()
                    e = (STEEPEST * e + act_error(z, "silu")) / self.sout.double() + u.abs() * 2.0 ** -22
                    u = u.clamp(-448.0, 448.0)
                    check(y.double(), u, e + code_step(u.abs() + e, torch.ones_like(u), "e4m3"), "a")
            x, res = t["out"], t["h"]


@pytest.mark.parametrize("rows", [1, 2, 5, 16, 33])
def test_decoding_step(rows):
    """Against 64 bits, then captured and replayed for other tokens."""
    d = Decode(rows, 512, 1040)
    say(f"decoding, {rows} rows")
    d.step()
    d.check_step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        y = d.step()
    gn = gen(3)
    for turn in range(4):
        d.x.copy_(normal(gn, (rows, 512)).half())
        first = d.step().clone()
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        (d.x.float() @ d.x.float().t()).sum()
        torch.cuda.synchronize()
        assert torch.equal(y, first), turn
    d.check_step()


def test_step_on_another_stream():
    """All calls on a stream given by argument or current, with work of the default stream beside it."""
    layer = Layer(130, 264, 520, "gelu_tanh")
    layer.step()
    first = snapshot(layer)
    side = torch.cuda.Stream()
    for t in layer.results().values():
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer.step()
    side.synchronize()
    same(layer, first, "side stream")
    y, a, z = torch.zeros_like(layer.y), torch.zeros_like(layer.a), [torch.zeros_like(t) for t in layer.qz]
    torch.cuda.synchronize()
    g.rms_norm(layer.x, layer.w, y, eps=EPS, residual=layer.res, stream=side)
    g.gemm_f16_bias_act_bt(y, layer.w1, a, bias=layer.b1, act=layer.act, Z=z[0], Zscale=z[1], z_fmt=g.FMT_E4M3, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.y) and torch.equal(a, layer.a)
