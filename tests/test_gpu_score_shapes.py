"""Every block shape, and lists of unequal length. The table's gradient: shapes of
one frame against the oracle and bit for bit the same at every run, the others
against the oracle (bounds and problems of test_gpu_score)."""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api
from tests.test_gpu_score import Problem, check_bias, check_diff, run_bias

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

SHAPES = [(1 << t, 1 << h, 1 << (6 - t - h)) for t in range(7) for h in range(7 - t)]


def problem(tile, d, **kw):
    """At least three blocks along rows or columns, two to four along time, lone tiles too."""
    pt, ph, pw = tile
    grid = (3 * pt if pt <= 4 else 2 * pt, ph * (3 if ph <= 8 else 1), pw * (3 if pw <= 8 else 2))
    return Problem((1, 2, *grid, d, tile, True), **kw)


@pytest.mark.parametrize("tile", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_table_gradient_of_every_shape(tile):
    p = problem(tile, 64 if tile[0] % 4 == 2 else 128, seed=21, density=0.6)
    q, k, v, g = p.dev()
    out, lse, grads = run_bias(p, q, k, v, g, p.table.cuda(), torch.from_numpy(p.bucket).cuda())
    p.check_ok()
    check_bias(p, out, lse, grads)


@pytest.mark.parametrize("tile", [s for s in SHAPES if s[0] == 1],
                         ids=["x".join(map(str, s)) for s in SHAPES if s[0] == 1])
def test_same_bits_of_every_shape_of_one_frame(tile):
    _, ph, pw = tile
    p = Problem((2, 4, 5, ph * max(1, 32 // ph), pw * max(1, 32 // pw), 128, tile, True), seed=22)
    q, k, v, g = p.dev()
    table, bucket = p.table.cuda(), torch.from_numpy(p.bucket).cuda()
    first = run_bias(p, q, k, v, g, table, bucket)
    for _ in range(20):
        again = run_bias(p, q, k, v, g, table, bucket)
        assert all(torch.equal(a, b) for a, b in zip(first[:2] + first[2], again[:2] + again[2]))


@pytest.mark.parametrize("d", [64, 128])
def test_chains_of_unequal_length(d):
    """More than four tiles per SM, two tiles a head: CTAs whose two tiles have 0 to 12
    steps, in every pairing of a short and a long list."""
    H = 100
    p = Problem((1, H, 2, 8, 48, d, None, False), seed=23)  # 12 blocks, 6 tiles
    sizes = [0, 1, 2, 3, 4, 12]
    for h in range(H):
        p.mask[h] = False
        for tile in range(6):
            a, b = tile, tile + 6  # a frame's block and the next one's
            n = sizes[(h + tile * (1 + h // 6 % 5)) % 6]
            keep = np.random.default_rng(100 * h + tile).permutation(12)[:n]
            p.mask[h, a, keep] = True
            p.mask[h, b, keep[: n // 2 + 1]] = True
    q, k, v, g = p.dev()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    out = api.fwd_bias(p.desc, q, k, v, p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.ws, lse=lse)
    out_d = api.fwd_diff(p.desc, q, k, v, p.lam.cuda(), p.ws)
    p.check_ok()
    check_bias(p, out, lse)
    check_diff(p, out_d, None, None)


@pytest.mark.parametrize("d", [64, 128])
def test_same_bits_of_long_lists(d):
    """Steps whose scores overwrite what the products of two steps before read: lists of
    about 100 steps, more tiles than SMs, 10 runs of everything."""
    desc = api.make_desc(1, 6, 8, 32, 32, d, 0.0)
    gen = torch.Generator("cuda").manual_seed(d)
    q, k, v, g = (torch.randn(1, 6, 8192, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    ws = api.alloc_workspace(desc)
    api.plan_mask(desc, torch.rand(6, 128, 128, generator=gen, device="cuda") < 0.6, ws)
    bucket, n = api.relative_buckets(8, 32, 32)
    table = torch.randn(6, n, generator=gen, device="cuda").bfloat16()
    lam = torch.rand(6, generator=gen, device="cuda").bfloat16()
    lse, lse2, out2 = torch.empty(1, 6, 8192, device="cuda"), torch.empty(2, 1, 6, 8192, device="cuda"), \
        torch.empty_like(q)

    def run():
        a = api.fwd_bias(desc, q, k, v, table, bucket, ws, lse=lse)
        b = api.fwd_diff(desc, q, k, v, lam, ws, out2=out2, lse=lse2)
        return (a, b, out2.clone()) + api.bwd_bias(desc, q, k, v, table, bucket, a, g, lse, ws) + \
            api.bwd_diff(desc, q, k, v, lam, b, out2, g, lse2, ws)
    first = run()
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, run()))
    assert api.check(desc, ws) == api.SA_OK
