"""The table's gradient of every block shape: the shapes of one frame against the
oracle and bit for bit the same at every run, the others against the oracle (bounds
and problems of test_gpu_score)."""
import pytest
import torch

from tests.test_gpu_score import Problem, check_bias, run_bias

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
