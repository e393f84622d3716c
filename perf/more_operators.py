"""Cases of a dense layer's operators around its matrix products: the
root-mean-square norm with the residual's addition (into FP16, or into FP8
codes with a scale per row) and its gradient; products with bias, activation
and residual in the epilogue, and the gradient of that epilogue; activations
kept in 8 bits (FP8 codes with a power-of-two scale per 32 values of a row),
and the gradients that read them.

`listed()` gives the named cases, `draw(rng)` one more of the same ranges,
`prepare(case, seed)` the inputs on the GPU, `run(state)` one pass (the plain
form in elementary torch operations, or with `own` the library's calls),
`exact(case, seed)` the same outputs from the definitions in 64 bits and
`work(case)` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
BLOCK = 32               # values that share a scale
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F16_TOP = {"e4m3": 61440.0, "e5m2": 57344.0}   # the largest FP16 number with as few mantissa bits
TORCH = {"f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SIZE = {"f16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of sixteen requests, in front of an FP8 product: latency
        {"name": "norm_decode_fp8", "op": "norm", "rows": 16, "width": 4096, "dtype": "f16", "out": "e4m3",
         "residual": True, "keep": False},
        # prompts, in front of an FP8 product
        {"name": "norm_prefill_fp8", "op": "norm", "rows": 16384, "width": 4096, "dtype": "f16", "out": "e4m3",
         "residual": True, "keep": False},
        # training, gradient of the norm that joins the residual's
        {"name": "norm_backward_f16", "op": "norm_backward", "rows": 8192, "width": 4096, "dtype": "f16", "held": "f16",
         "joins": True},
        # the same with an FP32 stream whose activation was kept in 8 bits, odd sizes
        {"name": "norm_backward_odd", "op": "norm_backward", "rows": 1003, "width": 1000, "dtype": "f32", "held": "e4m3",
         "joins": False},
        # one decoding step: the layer's first product, weights streamed once
        {"name": "linear_decode_f16", "op": "linear", "kind": "f16", "layout": "bt", "rows": 4, "n": 12288, "k": 4096,
         "bias": True, "act": "silu", "residual": "none", "out": "f16", "save": "none"},
        # training, forward: the pre-activation stays behind in 8 bits
        {"name": "linear_train_f16", "op": "linear", "kind": "f16", "layout": "bt", "rows": 4096, "n": 4096, "k": 4096,
         "bias": True, "act": "gelu", "residual": "none", "out": "f16", "save": "e4m3"},
        # a long batch of prompts on FP8 weights, added to the residual: the largest product
        {"name": "linear_prefill_fp8", "op": "linear", "kind": "fp8", "layout": "bt", "rows": 16384, "n": 12288,
         "k": 4096, "bias": True, "act": "gelu_tanh", "residual": "f16", "out": "f16", "save": "none"},
        # training, gradient of the epilogue from the kept 8-bit values
        {"name": "act_backward_mx", "op": "act_backward", "rows": 8192, "n": 12288, "dtype": "f16", "held": "e4m3",
         "act": "gelu"},
        # the same of a short batch, FP16 values, odd sizes
        {"name": "act_backward_odd", "op": "act_backward", "rows": 1001, "n": 1416, "dtype": "f16", "held": "f16",
         "act": "silu"},
        # training, forward: activations put away
        {"name": "checkpoint_pack", "op": "pack", "rows": 8192, "width": 4096, "dtype": "f16", "fmt": "e4m3"},
        # training, gradient to the weights from them
        {"name": "checkpoint_wgrad", "op": "wgrad", "rows": 8192, "m": 4096, "n": 4096, "fmt": "e4m3", "second": True,
         "out": "f32"},
        # the same of a short batch, odd sizes, the weight held row-major
        {"name": "checkpoint_wgrad_odd", "op": "wgrad", "rows": 1003, "m": 1000, "n": 520, "fmt": "e4m3",
         "second": False, "out": "f16"},
    ]


MOST_FLOPS = 2.0 * 16384 * 12288 * 4096   # the largest listed product
MOST_BYTES = 0.9e9                        # ... and the most bytes of a drawn case


def _size(rng, lo, hi, multiple=1, odd=0.0):
    """A size spread over the logarithm of [lo, hi]: a multiple, or with chance `odd` any whole number."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    m = 1 if rng.random() < odd else multiple
    return int(max(lo, min(hi, round(v / m) * m)))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "norm_backward", "linear", "linear", "linear", "act_backward", "pack", "wgrad",
                         "wgrad"])
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        if op == "norm":
            case = {"op": op, "rows": _size(rng, 1, 32768), "width": _size(rng, 64, 16384, 8, 0.15),
                    "dtype": rng.choice(["f16", "f16", "f32"]), "out": rng.choice(["e4m3", "e4m3", "f16"]),
                    "residual": rng.random() < 0.7, "keep": rng.random() < 0.5}
        elif op == "norm_backward":
            case = {"op": op, "rows": _size(rng, 1, 16384), "width": _size(rng, 64, 16384, 8, 0.15),
                    "dtype": rng.choice(["f16", "f32"]), "held": rng.choice(["f16", "e4m3", "e5m2"]),
                    "joins": rng.random() < 0.5}
        elif op == "linear":
            kind = rng.choice(["f16", "fp8"])
            save = rng.choice(["none", "none", "f16", "e4m3"])
            case = {"op": op, "kind": kind, "layout": rng.choice(["bt", "bt", "rm"]), "rows": _size(rng, 1, 16384),
                    "n": _size(rng, 128, 12288, 16, 0.1), "k": _size(rng, 128, 8192, 16, 0.1),
                    "bias": rng.random() < 0.7, "act": act, "residual": rng.choice(["none", "f16", "f32"]),
                    "out": rng.choice(["f16", "f16", "e4m3"] if kind == "fp8" else ["f16", "f16", "f32"]), "save": save}
        elif op == "act_backward":
            case = {"op": op, "rows": _size(rng, 1, 16384), "n": _size(rng, 64, 16384, 8, 0.15),
                    "dtype": rng.choice(["f16", "f16", "f32"]), "held": rng.choice(["f16", "e4m3", "e4m3", "e5m2"]),
                    "act": act}
        elif op == "pack":
            case = {"op": op, "rows": _size(rng, 1, 32768), "width": _size(rng, 64, 16384, 8, 0.15),
                    "dtype": rng.choice(["f16", "f32"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
        else:
            case = {"op": op, "rows": _size(rng, 1, 16384), "m": _size(rng, 128, 8192, 8, 0.1),
                    "n": _size(rng, 128, 8192, 8, 0.1), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                    "second": rng.random() < 0.5, "out": rng.choice(["f16", "f32"])}
        w = work(case)
        if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES:
            return case


def _held_bytes(case, rows, width, key="held"):
    t = case[key]
    return rows * width * SIZE[t] + (0 if t in ("f16", "f32") else rows * -(-width // BLOCK))


def work(case):
    op, r = case["op"], case["rows"]
    if op == "norm":
        w, es = case["width"], SIZE[case["dtype"]]
        b = r * w * (es * (3 if case["residual"] else 1) + SIZE[case["out"]]) + 4 * w
        return {"bytes": b + (4 * r if case["out"] == "e4m3" else 0) + (4 * r if case["keep"] else 0), "flops": 6 * r * w}
    if op == "norm_backward":
        w, es = case["width"], SIZE[case["dtype"]]
        return {"bytes": r * w * es * (3 if case["joins"] else 2) + _held_bytes(case, r, w) + 8 * w + 4 * r,
                "flops": 10 * r * w}
    if op == "linear":
        n, k, es = case["n"], case["k"], 2 if case["kind"] == "f16" else 1
        b = r * k * es + n * k * es + r * n * SIZE[case["out"]] + (4 * n if case["bias"] else 0)
        if case["kind"] == "fp8":
            b += 4 * (r + n)
        if case["residual"] != "none":
            b += r * n * SIZE[case["residual"]]
        if case["save"] != "none":
            b += _held_bytes(case, r, n, "save")
        return {"bytes": b, "flops": 2 * r * n * k}
    if op == "act_backward":
        n = case["n"]
        held = 0 if case["act"] == "none" else _held_bytes(case, r, n)
        return {"bytes": 2 * r * n * SIZE[case["dtype"]] + held + 4 * n, "flops": 12 * r * n}
    if op == "pack":
        w = case["width"]
        return {"bytes": r * w * SIZE[case["dtype"]] + _held_bytes(case, r, w, "fmt"), "flops": 2 * r * w}
    m, n = case["m"], case["n"]
    return {"bytes": _held_bytes(case, r, m, "fmt") + r * n * 2 + m * n * SIZE[case["out"]], "flops": 2 * r * m * n}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _stream(g, rows, width, dtype):
    """A residual stream: rows of different sizes, and a few columns that stand out."""
    x = _normal(g, (rows, width)) * torch.exp(0.5 * _normal(g, (rows, 1)))
    return (x * (1.0 + 20.0 * (torch.rand((width,), generator=g, device=DEV) < 0.004))).to(TORCH[dtype])


def _blocks(t, rows, cols):
    """Room for 8-bit values: codes and their scales."""
    return (torch.empty((rows, cols), dtype=TORCH[t], device=DEV),
            torch.empty((rows, -(-cols // BLOCK)), dtype=torch.float8_e8m0fnu, device=DEV))


def _held(st, x, t):
    """What the forward pass left of x: itself, or 8-bit values."""
    if t in ("f16", "f32"):
        st["held"], st["held_scale"] = x.to(TORCH[t]), None
    else:
        st["held"], st["held_scale"] = _pack(x, t)


def prepare(case, seed):
    g = _gen(seed)
    op, r = case["op"], case["rows"]
    st = {"case": case}
    if op in ("norm", "norm_backward"):
        w, dt = case["width"], case["dtype"]
        st["weight"] = 1.0 + _normal(g, (w,), 0.1)
    if op == "norm":
        st["x"] = _stream(g, r, w, dt)
        st["residual"] = _stream(g, r, w, dt) if case["residual"] else None
        st["h"] = torch.empty((r, w), dtype=TORCH[dt], device=DEV) if case["residual"] else None
        st["y"] = torch.empty((r, w), dtype=TORCH[case["out"]], device=DEV)
        st["scale"] = torch.empty((r,), device=DEV) if case["out"] == "e4m3" else None
        st["rstd"] = torch.empty((r,), device=DEV) if case["keep"] else None
    elif op == "norm_backward":
        h = _stream(g, r, w, "f16")
        st["rstd"] = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
        _held(st, h, case["held"])
        st["dy"] = _normal(g, (r, w), 0.1).to(TORCH[dt])
        st["dh"] = _normal(g, (r, w), 0.1).to(TORCH[dt]) if case["joins"] else None
        st["dx"], st["dweight"] = torch.empty((r, w), dtype=TORCH[dt], device=DEV), torch.empty((w,), device=DEV)
        st["ws"] = torch.empty(4 * w * 1024, dtype=torch.uint8, device=DEV)
    elif op == "linear":
        n, k, bt = case["n"], case["k"], case["layout"] == "bt"
        x, b = _normal(g, (r, k)), _normal(g, (n, k) if bt else (k, n), 1.2 / math.sqrt(k))
        if case["kind"] == "f16":
            st["a"], st["b"] = x.half(), b.half()
        else:
            st["sa"], over = x.abs().amax(dim=1) / 448.0, 1 if bt else 0
            st["sb"] = b.abs().amax(dim=over) / 448.0
            st["a"] = (x / st["sa"].unsqueeze(1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            st["b"] = (b / st["sb"].unsqueeze(over)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        del x, b
        st["bias"] = _normal(g, (n,), 0.5) if case["bias"] else None
        st["residual"] = None if case["residual"] == "none" else _normal(g, (r, n)).to(TORCH[case["residual"]])
        st["c"] = torch.empty((r, n), dtype=TORCH[case["out"]], device=DEV)
        st["sout"] = torch.full((1,), 1.0 / 32.0, device=DEV) if case["out"] == "e4m3" else None
        st["z"], st["zscale"] = None, None
        if case["save"] == "f16":
            st["z"] = torch.empty((r, n), dtype=torch.float16, device=DEV)
        elif case["save"] != "none":
            st["z"], st["zscale"] = _blocks(case["save"], r, n)
    elif op == "act_backward":
        n, dt = case["n"], case["dtype"]
        _held(st, _normal(g, (r, n), 1.3).half(), case["held"])
        st["dy"] = _normal(g, (r, n), 0.1).to(TORCH[dt])
        st["dz"], st["dbias"] = torch.empty((r, n), dtype=TORCH[dt], device=DEV), torch.empty((n,), device=DEV)
        st["ws"] = torch.empty(4 * n * 1024, dtype=torch.uint8, device=DEV)
    elif op == "pack":
        st["x"] = _stream(g, r, case["width"], case["dtype"])
        st["q"], st["scale"] = _blocks(case["fmt"], r, case["width"])
    else:
        m, n = case["m"], case["n"]
        st["q"], st["scale"] = _pack(_stream(g, r, m, "f16"), case["fmt"])
        st["b"] = _normal(g, (r, n), 0.1).half()
        st["c"] = torch.empty((n, m) if case["second"] else (m, n), dtype=TORCH[case["out"]], device=DEV)
    return st


# ---------------------------------------------------------------- plain forms
def _pack(x, fmt):
    """FP8 codes of x's rows and the power-of-two scale of each 32 values: the least with |x| / scale <= the format's
    largest. FP16 values stay within FP16's range."""
    rows, cols = x.shape
    v = x.float()
    if x.dtype == torch.float16:
        v = v.clamp(-F16_TOP[fmt], F16_TOP[fmt])
    v = torch.nn.functional.pad(v, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
    part, power = torch.frexp(v.abs().amax(dim=2))
    top, top_power = math.frexp(FP8_MAX[fmt])
    e = torch.where(part > 0, power - top_power + (part > top), torch.zeros_like(power)).clamp(-127, 127)
    code = torch.ldexp(v, -e.unsqueeze(2)).reshape(rows, -1)[:, :cols].to(TORCH[fmt])
    return code.contiguous(), torch.ldexp(torch.ones_like(part), e).to(torch.float8_e8m0fnu)


def _value(st):
    """What the forward pass left, as numbers."""
    if st["held_scale"] is None:
        return st["held"].float()
    return _unpack(st["held"], st["held_scale"])


def _unpack(q, scale):
    rows, cols = q.shape
    s = scale.float().unsqueeze(2).expand(-1, -1, BLOCK).reshape(rows, -1)[:, :cols]
    return q.float() * s


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _slope(z, act):
    """The derivative of _act."""
    if act == "relu":
        return (z > 0.0).float()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z * z * z))
        return s + z * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1.0 - s)
    return torch.ones_like(z)


def _plain_norm(st):
    case = st["case"]
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    h = h.to(st["x"].dtype)
    v = h.float()
    rstd = torch.rsqrt(v.square().mean(dim=1) + EPS)
    y = v * st["weight"] * rstd.unsqueeze(1)
    out = [] if st["h"] is None else [h]
    if case["keep"]:
        out.append(rstd)
    if case["out"] != "e4m3":
        return out + [y.to(TORCH[case["out"]])]
    scale = y.abs().amax(dim=1) / 448.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return out + [(y / scale.unsqueeze(1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale]


def _plain_norm_backward(st):
    dy, n = st["dy"].float(), _value(st) * st["rstd"].unsqueeze(1)
    g = dy * st["weight"]
    dx = st["rstd"].unsqueeze(1) * (g - n * (g * n).mean(dim=1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return [dx.to(st["dy"].dtype), (dy * n).sum(dim=0)]


def _plain_linear(st):
    case = st["case"]
    b = st["b"].float()
    z = st["a"].float() @ (b.t() if case["layout"] == "bt" else b)
    if case["kind"] == "fp8":
        z = z * st["sa"].unsqueeze(1) * st["sb"]
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    if case["out"] == "e4m3":
        y = (y / st["sout"]).clamp(-448.0, 448.0)
    out = [y.to(TORCH[case["out"]])]
    if case["save"] == "f16":
        out.append(z.half())
    elif case["save"] != "none":
        out += _pack(z, case["save"])
    return out


def _plain_act_backward(st):
    dz = st["dy"].float() * _slope(_value(st), st["case"]["act"])
    return [dz.to(st["dy"].dtype), dz.sum(dim=0)]


def _plain_pack(st):
    return list(_pack(st["x"], st["case"]["fmt"]))


def _plain_wgrad(st):
    x, b = _unpack(st["q"], st["scale"]), st["b"].float()
    return (b.t() @ x if st["case"]["second"] else x.t() @ b).to(st["c"].dtype)


# ---------------------------------------------------------- the library's calls
def _own(st):
    import precision_dense_gemm_03_amd as g

    case = st["case"]
    op = case["op"]
    fmt = {"e4m3": g.FMT_E4M3, "e5m2": g.FMT_E5M2}
    act = {"none": g.ACT_NONE, "relu": g.ACT_RELU, "gelu": g.ACT_GELU, "gelu_tanh": g.ACT_GELU_TANH, "silu": g.ACT_SILU}
    if op == "norm":
        g.rms_norm(st["x"], st["weight"], st["y"], eps=EPS, residual=st["residual"], h=st["h"], scale=st["scale"],
                   rstd=st["rstd"])
        return [st[s] for s in ("h", "rstd", "y", "scale") if st[s] is not None]
    if op == "norm_backward":
        return list(g.rms_norm_backward(st["dy"], st["held"], st["weight"], st["rstd"], dx=st["dx"],
                                        dweight=st["dweight"], dh=st["dh"], hscale=st["held_scale"],
                                        workspace=st["ws"]))
    if op == "linear":
        more = {"bias": st["bias"], "act": act[case["act"]], "residual": st["residual"], "Z": st["z"],
                "Zscale": st["zscale"]}
        bt = case["layout"] == "bt"
        if case["kind"] == "f16":
            f = g.gemm_f16_bias_act_bt if bt else g.gemm_f16_bias_act
            f(st["a"], st["b"], st["c"], **more)
        else:
            f = g.gemm_fp8_bias_act_bt if bt else g.gemm_fp8_bias_act
            f(st["a"], g.FMT_E4M3, st["b"], g.FMT_E4M3, st["sa"], st["sb"], st["c"], channel=True, sOut=st["sout"],
              **more)
        return [st[s] for s in ("c", "z", "zscale") if st[s] is not None]
    if op == "act_backward":
        return list(g.bias_act_backward(st["dy"], st["held"], act[case["act"]], dZ=st["dz"], dbias=st["dbias"],
                                        Zscale=st["held_scale"], workspace=st["ws"]))
    if op == "pack":
        return list(g.quantize_mx_fp8(st["x"], fmt[case["fmt"]], q=st["q"], scale=st["scale"]))
    return g.gemm_mx_wgrad(st["q"], st["scale"], fmt[case["fmt"]], st["b"], st["c"], q_second=case["second"])


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "linear": _plain_linear,
         "act_backward": _plain_act_backward, "pack": _plain_pack, "wgrad": _plain_wgrad}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------- 64-bit outputs
def _numbers(values, scale):
    """The numbers that 8-bit values stand for, in 64 bits, block by block."""
    out = values.to(torch.float64)
    for c in range(scale.shape[1]):
        out[:, c * BLOCK:(c + 1) * BLOCK] *= scale[:, c:c + 1].double()
    return out


def _coded(x, fmt, half):
    """Codes and scales of 64-bit x (half: of FP16 values) as 64-bit numbers, from the formats' steps."""
    rows, cols = x.shape
    top, bits, least = (448.0, 4, -6) if fmt == "e4m3" else (57344.0, 3, -14)
    if half:
        x = torch.minimum(torch.maximum(x, torch.full_like(x, -F16_TOP[fmt])), torch.full_like(x, F16_TOP[fmt]))
    code = torch.empty_like(x)
    scale = torch.empty((rows, (cols + BLOCK - 1) // BLOCK), dtype=torch.float64, device=x.device)
    for c in range(scale.shape[1]):
        v = x[:, c * BLOCK:(c + 1) * BLOCK]
        most = v.abs().amax(dim=1)
        s = torch.exp2(torch.ceil(torch.log2(torch.where(most > 0, most, torch.full_like(most, top)) / top)))
        s = torch.where(most / s > top, s * 2, s)          # (the logarithm's rounding)
        s = torch.where(most / (s / 2) <= top, s / 2, s)
        s = torch.where(most > 0, s, torch.ones_like(s)).clamp(2.0 ** -127, 2.0 ** 127)
        u = v / s[:, None]
        power = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** least)))
        step = torch.exp2(power - (bits - 1))
        code[:, c * BLOCK:(c + 1) * BLOCK] = torch.round(u / step) * step
        scale[:, c] = s
    return code, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = (h + st["residual"].double()).to(st["x"].dtype).double()
        root = torch.sqrt((h * h).sum(dim=1) / case["width"] + EPS)
        y = h / root[:, None] * st["weight"].double()[None, :]
        out = ([] if st["h"] is None else [h]) + ([1.0 / root] if case["keep"] else [])
        if case["out"] != "e4m3":
            return out + [y]
        s = y.abs().max(dim=1).values / 448.0
        s[s == 0] = 1.0
        return out + [y / s[:, None], s]
    if op == "norm_backward":
        h = st["held"].double() if st["held_scale"] is None else _numbers(st["held"], st["held_scale"])
        r, w, dy = st["rstd"].double()[:, None], st["weight"].double()[None, :], st["dy"].double()
        along = (dy * w * h).sum(dim=1, keepdim=True)
        dx = w * dy * r - h * r ** 3 * along / case["width"]
        if st["dh"] is not None:
            dx += st["dh"].double()
        return [dx, (dy * (h * r)).sum(dim=0)]
    if op == "act_backward":
        z = st["held"].double() if st["held_scale"] is None else _numbers(st["held"], st["held_scale"])
        dz = st["dy"].double() * _exact_act(z, case["act"])[1]
        return [dz, dz.sum(dim=0)]
    if op == "pack":
        return list(_coded(st["x"].double(), case["fmt"], case["dtype"] == "f16"))
    if op == "wgrad":
        x, b = _numbers(st["q"], st["scale"]), st["b"].double()
        return torch.matmul(b.t().contiguous(), x) if case["second"] else torch.matmul(x.t().contiguous(), b)
    b = st["b"].double()
    z = torch.matmul(st["a"].double(), b.t().contiguous() if case["layout"] == "bt" else b)
    if case["kind"] == "fp8":
        z *= st["sa"].double()[:, None]
        z *= st["sb"].double()[None, :]
    if st["bias"] is not None:
        z += st["bias"].double()[None, :]
    y = _exact_act(z, case["act"], False)[0]
    if st["residual"] is not None:
        y = y + st["residual"].double()
    out = [y / st["sout"].double() if case["out"] == "e4m3" else y]
    if case["save"] == "f16":
        out.append(z)
    elif case["save"] != "none":
        out += list(_coded(z, case["save"], False))
    return out


def _exact_act(z, act, slope=True):
    """The activation and its derivative from their definitions, by the normal distribution and by tanh."""
    if act == "none":
        return z, torch.ones_like(z) if slope else None
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double() if slope else None
    if act == "silu":
        e = 1.0 + torch.exp(-z)
        return z / e, 1.0 / e + z * (e - 1.0) / (e * e) if slope else None
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi) if slope else None
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 0.134145 * z * z) if slope else None
