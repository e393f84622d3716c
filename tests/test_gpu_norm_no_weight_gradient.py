"""rms_norm_backward without the gradient to the weights: in no workspace for rows
of up to 16384 values, in one FP32 word a row beyond; dx as with it, bit for bit."""
import pytest
import torch

import precision_dense_gemm_03_amd as g
from test_gpu_norm import DEV, F16, F32, _gpu, gen, normal, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("rows,width", [(1, 5), (7, 64), (300, 1000), (33, 4099), (5, 16384), (3, 16385), (700, 20000)])
def test_same_dx(rows, width, dtype):
    gn = gen(rows + width)
    h, dy, dh = (normal(gn, (rows, width)).to(dtype) for _ in range(3))
    w, rstd = 1.0 + normal(gn, (width,), 0.2), torch.rand(rows, generator=gn, device=DEV) + 0.5
    dw = torch.empty(width, device=DEV)
    ref, _ = g.rms_norm_backward(dy, h, w, rstd, dweight=dw, dh=dh)
    say(f"norm backward without dweight, {rows}x{width} {dtype}")
    long = width > 16384
    ws = torch.full((4 * rows + 256,), 0xA5, dtype=torch.uint8, device=DEV) if long else None
    out = torch.empty_like(dy)
    st = g.lib().rms_norm_backward(dy.data_ptr(), dh.data_ptr(), g.OUT_F16 if dtype == F16 else g.OUT_F32, h.data_ptr(),
                                   None, g.OUT_F16 if dtype == F16 else g.OUT_F32, w.data_ptr(), rstd.data_ptr(),
                                   out.data_ptr(), None, rows, width, ws.data_ptr() if long else None,
                                   4 * rows if long else 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(out, ref)
    if long:
        assert bool((ws[4 * rows:] == 0xA5).all()), "past the workspace"
    # the binding allocates what is needed, and nothing where nothing is
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    dx, none = g.rms_norm_backward(dy, h, w, rstd, dx=out, dh=dh)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] - before == (1 if long else 0)
    assert none is None and torch.equal(dx, ref)
