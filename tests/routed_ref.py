"""64-bit references and bounds for the products whose weight depends on the
row (test_gpu_routed.py) and for expert routing (test_gpu_moe.py).

Bounds, fixed before the first run. A product's FP32 sum over K terms of exact
products is off by at most 1e-5 * S, S = sum |a b| (the accumulation allowance
of parity.py); storing FP16 adds half a step, 2^-11 relative to the value or
2^-25 below the smallest normal. FP8 products add the matrix cores' alignment
allowance T (parity.py). An adapter's term is a sum over the rank of FP32
low-rank values (each off by 1e-5 of its own absolute sum) that meet LB as an
FP16 pair of 22 bits: 2^-21 of the row's largest low-rank value per term.
"""
import numpy as np
import torch

REL = 1e-5


def half_step_f16(v):
    return torch.clamp(v.abs() * 2.0 ** -11, min=2.0 ** -25)


def check(got, ref, bound, what):
    """|got - ref| <= bound per element, on the device; everything finite where ref is."""
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound; first at {i}: got "
                             f"{got[i].item()!r} ref {ref[i].item()!r} bound {bound[i].item()!r}")


def cut(sizes, lead=0):
    """offsets of consecutive groups of these sizes after `lead` rows of no group."""
    return [lead] + [lead + int(c) for c in np.cumsum(sizes)]


def group_of(offsets, rows):
    g = np.full(rows, -1, np.int64)
    for e in range(len(offsets) - 1):
        g[offsets[e]:offsets[e + 1]] = e
    return g


def grouped(a, b, offsets, bt):
    """(value, absolute sum) in 64 bits; a [rows, K] and b [G, ...] hold decoded values."""
    rows, n = a.shape[0], b.shape[1] if bt else b.shape[2]
    v = torch.zeros((rows, n), dtype=torch.float64, device=a.device)
    s = torch.zeros_like(v)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            w = b[e].double().t().contiguous() if bt else b[e].double()
            x = a[lo:hi].double()
            v[lo:hi] = x @ w
            s[lo:hi] = x.abs() @ w.abs()
    return v, s


def lora(x, la, lb, adapter, lscale, n):
    """(value, bound) of the adapters' term in 64 bits."""
    rows = x.shape[0]
    v = torch.zeros((rows, n), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(v)
    ad = adapter.cpu().numpy()
    for a in sorted(set(int(i) for i in ad) & set(range(la.shape[0]))):
        idx = torch.from_numpy(np.nonzero(ad == a)[0]).to(x.device)
        xr, l, m = x[idx].double(), la[a].double(), lb[a].double()
        sc = lscale[a].double()
        low = sc * (xr @ l.t().contiguous())
        low_abs = sc.abs() * (xr.abs() @ l.abs().t().contiguous())
        mt = m.t().contiguous()
        v[idx] = low @ mt
        top = low.abs().amax(dim=1, keepdim=True) if low.shape[1] else low.new_zeros((low.shape[0], 1))
        per = REL * low_abs + 2.0 ** -21 * top
        bound[idx] = per @ mt.abs() + REL * (low.abs() @ mt.abs())
    return v, bound
