"""Calls beside other calls: after one that failed, from two threads at once."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def test_a_failed_launch_is_not_reported_again():
    """The legacy stream takes no launch while a blocking stream is being captured: the
    plan's launch is refused. The next call, on a stream of its own, is not concerned."""
    desc = api.make_desc(1, 1, 2, 8, 8, 64, 0.0)
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 1, 128, 64, generator=gen, device="cuda").bfloat16() for _ in range(3))
    mask = torch.ones(2, 2, dtype=torch.bool, device="cuda")
    ws, out, side = api.alloc_workspace(desc), torch.empty_like(q), torch.cuda.Stream()
    api.plan_mask(desc, mask, ws)
    want = api.fwd(desc, q, k, v, ws, torch.empty_like(q))
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert cu.cuStreamBeginCapture_v2(stream, 0) == 0
    try:
        with pytest.raises(api.SparseAttnError):
            api.plan_mask(desc, mask, ws, stream=0)
        api.fwd(desc, q, k, v, ws, out, stream=side)
    finally:
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))  # an error: the capture is invalid
        cu.cuStreamDestroy_v2(stream)
    side.synchronize()
    assert torch.equal(out, want)
