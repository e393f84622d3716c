"""A layer of experts behind a projection with per-request adapters, on the library's calls.

    python examples/experts.py          # trains the layer for some steps, then serves single tokens (needs the GPU)

Training: the layer's forward and backward pass (routing, gather, grouped
products, combine, and all their gradients) fitted to another layer's outputs.
Serving: one token per request through a projection to which each request adds
its own low-rank adapter, then through the layer, captured once as a graph and
replayed. PyTorch supplies memory, streams, the activation and the optimizer's
arithmetic; every product and every routing step is the library's.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import precision_dense_gemm_03_amd as g

DEV = "cuda:0"
F16, F32, I32 = torch.float16, torch.float32, torch.int32


def silu(h):
    return (h.float() * torch.sigmoid(h.float())).half()


def silu_backward(da, h):
    x = h.float()
    s = torch.sigmoid(x)
    return (da.float() * s * (1.0 + x * (1.0 - s))).half()


class Experts:
    """y[t] = sum over the token's topk experts e of weight * W2[e] silu(W1[e] x[t]); the weights are the softmax
    over the chosen logits R x[t]. W1 [experts, hidden, width], W2 [experts, width, hidden], R [experts, width]."""

    def __init__(self, width, hidden, experts, topk, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=gen, device=DEV) / shape[-1] ** 0.5).half()

        self.router, self.w1, self.w2 = normal(experts, width), normal(experts, hidden, width), normal(experts, width,
                                                                                                      hidden)
        self.topk = topk

    def buffers(self, tokens):
        """What a pass over `tokens` rows writes, kept from call to call."""
        experts, hidden, width = self.w1.shape
        rows = tokens * self.topk
        route = {"expert": torch.empty((tokens, self.topk), dtype=I32, device=DEV),
                 "weight": torch.empty((tokens, self.topk), dtype=F32, device=DEV),
                 "offsets": torch.empty(experts + 1, dtype=I32, device=DEV),
                 "row": torch.empty((tokens, self.topk), dtype=I32, device=DEV),
                 "token": torch.empty(rows, dtype=I32, device=DEV),
                 "workspace": torch.empty(max(16, g.moe_route_workspace_size(tokens, experts)), dtype=torch.uint8,
                                          device=DEV)}
        return {"route": route, "logits": torch.empty((tokens, experts), dtype=F32, device=DEV),
                "xs": torch.empty((rows, width), dtype=F16, device=DEV),
                "h": torch.empty((rows, hidden), dtype=F16, device=DEV),
                "z": torch.empty((rows, width), dtype=F16, device=DEV),
                "y": torch.empty((tokens, width), dtype=F16, device=DEV)}

    def forward(self, x, kept=None):
        b = kept or self.buffers(x.shape[0])
        g.gemm_f16_bt(x, self.router, b["logits"])
        _, weight, offsets, row, token = g.moe_route_f32(b["logits"], self.topk, **b["route"])
        g.moe_gather(x, token, b["xs"])
        g.gemm_f16_grouped_bt(b["xs"], self.w1, offsets, b["h"])
        b["a"] = silu(b["h"])
        g.gemm_f16_grouped_bt(b["a"], self.w2, offsets, b["z"])
        g.moe_combine(b["z"], row, weight, b["y"])
        b["x"] = x
        return b["y"], b

    def backward(self, dy, b):
        """Gradients of (x, router, w1, w2), those of the parameters in float32."""
        r, x = b["route"], b["x"]
        offsets, tokens = r["offsets"], x.shape[0]
        dz, dweight = g.moe_combine_backward(dy, b["z"], r["row"], r["weight"])
        da, dxs = torch.empty_like(b["h"]), torch.empty_like(b["xs"])
        dw1, dw2 = (torch.empty(w.shape, dtype=F32, device=DEV) for w in (self.w1, self.w2))
        g.gemm_f16_grouped(dz, self.w2, offsets, da)
        g.gemm_f16_grouped_wgrad(dz, b["a"], offsets, dw2)
        dh = silu_backward(da, b["h"])
        g.gemm_f16_grouped(dh, self.w1, offsets, dxs)
        g.gemm_f16_grouped_wgrad(dh, b["xs"], offsets, dw1)
        dx = g.moe_combine(dxs, r["row"], None, torch.empty(x.shape, dtype=F32, device=DEV))
        dlogits = g.moe_route_backward_f32(b["logits"], r["expert"], r["weight"], dweight).half()
        by_router = torch.empty(x.shape, dtype=F32, device=DEV)
        g.gemm_f16(dlogits, self.router, by_router)
        drouter = torch.empty((1,) + tuple(self.router.shape), dtype=F32, device=DEV)
        g.gemm_f16_grouped_wgrad(dlogits, x, torch.tensor([0, tokens], dtype=I32, device=DEV), drouter)
        return dx + by_router, drouter[0], dw1, dw2


def train(steps=30, tokens=512, width=128, hidden=256, experts=8, topk=2, rate=2e-2, say=print):
    """Fits a layer to another one's outputs; the losses of the steps."""
    target, layer = Experts(width, hidden, experts, topk, 1), Experts(width, hidden, experts, topk, 2)
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((tokens, width), generator=gen, device=DEV).half()
    goal = target.forward(x)[0].float()
    params = ("router", "w1", "w2")
    whole = {p: getattr(layer, p).float() for p in params}
    first, second = ({p: torch.zeros_like(w) for p, w in whole.items()} for _ in range(2))
    kept, losses = layer.buffers(tokens), []
    scale = 1024.0    # the gradients' FP16 steps stay in range
    for step in range(1, steps + 1):
        y, b = layer.forward(x, kept)
        diff = y.float() - goal
        losses.append(diff.square().mean())
        grads = dict(zip(params, layer.backward((diff * (2.0 * scale / diff.shape[0])).half(), b)[1:]))
        for p, d in grads.items():
            d = d / scale
            first[p].mul_(0.9).add_(d, alpha=0.1)
            second[p].mul_(0.99).add_(d * d, alpha=0.01)
            whole[p] -= rate * (first[p] / (1 - 0.9 ** step)) / ((second[p] / (1 - 0.99 ** step)).sqrt() + 1e-8) * 0.1
            setattr(layer, p, whole[p].half())
        if step == 1 or step % 10 == 0:
            say(f"step {step:3d}  loss {losses[-1].item():.5f}")
    return torch.stack(losses).tolist()


class Server:
    """One token per request: p = proj x + scale[a] LB[a] (LA[a] x), a the request's adapter, then the experts.
    The step is a graph over kept buffers."""

    def __init__(self, layer, requests, adapters, rank, seed):
        width = layer.router.shape[1]
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=gen, device=DEV) / shape[-1] ** 0.5).half()

        self.layer, self.kept = layer, layer.buffers(requests)
        self.proj, self.la, self.lb = normal(width, width), normal(adapters, rank, width), normal(adapters, width, rank)
        self.scale = torch.full((adapters,), 0.5, device=DEV)
        self.adapter = torch.full((requests,), -1, dtype=I32, device=DEV)
        self.x, self.p = (torch.empty((requests, width), dtype=F16, device=DEV) for _ in range(2))
        self.x.zero_()
        self.ws = torch.empty(g.lora_workspace_size(requests, rank), dtype=torch.uint8, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.calls()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.calls()

    def calls(self):
        g.gemm_f16_lora_bt(self.x, self.proj, self.la, self.lb, self.adapter, self.scale, self.p, workspace=self.ws)
        return self.layer.forward(self.p, self.kept)[0]

    def step(self, x, adapter):
        self.x.copy_(x)
        self.adapter.copy_(adapter)
        self.graph.replay()
        return self.y


def serve(steps=4, requests=16, width=128, hidden=256, experts=8, topk=2, adapters=5, rank=8, say=print):
    """Graph replays beside eager calls on the same inputs; True if all agree bit for bit."""
    server = Server(Experts(width, hidden, experts, topk, 4), requests, adapters, rank, 5)
    gen = torch.Generator(device=DEV).manual_seed(6)
    same = True
    for i in range(steps):
        x = torch.randn((requests, width), generator=gen, device=DEV).half()
        adapter = torch.randint(-1, adapters, (requests,), generator=gen, device=DEV).to(I32)
        y = server.step(x, adapter).clone()
        p = torch.empty_like(x)
        g.gemm_f16_lora_bt(x, server.proj, server.la, server.lb, adapter, server.scale, p)
        same = same and torch.equal(server.layer.forward(p)[0], y)
        say(f"token {i}: |y| = {y.float().norm().item():.4f}, graph and eager {'agree' if same else 'differ'}")
    return same


if __name__ == "__main__":
    torch.cuda.set_device(DEV)
    train()
    sys.exit(0 if serve() else 1)
