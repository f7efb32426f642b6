"""Calls beside other calls: after one that failed, from two threads at once."""
import ctypes
import threading

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


def test_two_threads_with_grids_of_different_size():
    """The kernels' shared memory grows with the grid's offset tables: calls of a large and
    a small grid from two threads at once, each on a stream of its own."""
    jobs = []
    for i, grid in enumerate(((400, 8, 8), (2, 8, 8))):
        for d in (64, 128):
            desc = api.make_desc(1, 1, *grid, d, 0.0)
            S = grid[0] * 64
            gen = torch.Generator("cuda").manual_seed(i)
            x = [torch.randn(1, 1, S, d, generator=gen, device="cuda").bfloat16() for _ in range(4)]
            ws = api.alloc_workspace(desc)
            api.plan_mask(desc, torch.eye(grid[0], dtype=torch.bool, device="cuda"), ws)
            bucket, n = api.relative_buckets(*grid)
            table = torch.randn(1, n, generator=gen, device="cuda").bfloat16()
            jobs.append((desc, x, ws, table, bucket))

    def step(job, stream):
        desc, (q, k, v, g), ws, table, bucket = job
        lse = torch.empty(q.shape[:3], device="cuda")
        out = api.fwd_bias(desc, q, k, v, table, bucket, ws, lse=lse, stream=stream)
        return (out, lse) + api.bwd_bias(desc, q, k, v, table, bucket, out, g, lse, ws, stream=stream)

    want = [step(job, None) for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(mine):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(200):
                for i in mine:
                    try:
                        got = step(jobs[i], stream)
                    except api.SparseAttnError as e:
                        wrong.append(str(e))
                        return
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[mine[-1]])):
                wrong.append(f"outputs of job {mine[-1]}")

    threads = [threading.Thread(target=work, args=(m,)) for m in ((0, 1), (2, 3), (1, 0), (3, 2))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert all(api.check(desc, ws) == api.SA_OK for desc, _, ws, _, _ in jobs)


@pytest.mark.parametrize("tile,d", [(None, 128), (None, 64), ((1, 2, 32), 64)])
def test_a_list_entry_out_of_range_is_reported_and_read_as_block_0(tile, d):
    """A plan's list with a block id that the grid does not have: the status says so, and
    the bias of that entry is block 0's, as its keys and values are."""
    desc = api.make_desc(1, 2, 2, 8, 64, d, 0.0, tile=tile)
    gen = torch.Generator("cuda").manual_seed(3)
    q, k, v, g = (torch.randn(1, 2, 1024, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    bucket, n = api.relative_buckets(2, 8, 64)
    table = torch.randn(2, n, generator=gen, device="cuda").bfloat16()
    res = []
    for first in (0, 3):
        mask = torch.zeros(16, 16, dtype=torch.bool, device="cuda")
        mask[:, [first, 6]] = True
        ws = api.alloc_workspace(desc)
        api.plan_mask(desc, mask, ws)
        if first:
            entries = api.get_mask(desc, ws)["tile_idx"][:, :, 0]
            assert bool((entries & 0xFFFF == first).all())
            entries |= 0xFFFF
        lse = torch.empty(q.shape[:3], device="cuda")
        out = api.fwd_bias(desc, q, k, v, table, bucket, ws, lse=lse)
        dq = api.bwd_bias(desc, q, k, v, table, bucket, out, g, lse, ws)[0]
        res.append((out, lse, dq))
        assert api.check(desc, ws) == (api.SA_ERR_DEVICE_TIMEOUT if first else api.SA_OK)
    assert all(torch.equal(a, b) for a, b in zip(*res))
