"""Heads of extreme shape. One frame of blocks in one column has a tile per
block, so 4,097 to 6,144 tiles a head have to be put in order; one block per
frame and up to 6,144 frames is the longest list of temporal pairs. Every q-block keeps itself and up to two others; the outputs and the
gradients of all blocks against fp64, with the bounds of test_gpu_score."""
import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api
from tests.test_gpu_score import E, U

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

D = 64
GRIDS = [((1, 8 * 4097, 8), None), ((1, 8 * 6144, 8), None), ((64, 4500, 1), (64, 1, 1)),
         ((5957, 8, 8), None), ((6144, 8, 8), None)]


class Band:
    """q-block i keeps i, (i + 1) if i is odd, and (i + 5) if 3 divides i (cyclic)."""

    def __init__(self, grid, tile, seed):
        self.desc = api.make_desc(1, 1, *grid, D, 0.0, tile=tile, out_fp32=True)
        T, Hh, Ww = grid
        pt, ph, pw = tile or (1, 8, 8)
        self.S, self.nb = T * Hh * Ww, T * Hh * Ww // 64
        gen = torch.Generator("cuda").manual_seed(seed)
        self.x = [torch.randn(1, 1, self.S, D, generator=gen, device="cuda").bfloat16()
                  for _ in range(4)]
        p = torch.arange(self.S, device="cuda")
        t, h, w = p // (Hh * Ww), p // Ww % Hh, p % Ww
        block = ((t // pt) * (Hh // ph) + h // ph) * (Ww // pw) + w // pw
        self.order = torch.argsort(block, stable=True)  # position in fractal order -> token
        i = torch.arange(self.nb, device="cuda")
        self.cols = torch.stack([i, (i + 1) % self.nb, (i + 5) % self.nb], 1)
        self.kept = torch.stack([i >= 0, i % 2 == 1, i % 3 == 0], 1)
        self.mask = torch.zeros(self.nb, self.nb, dtype=torch.bool, device="cuda")
        self.mask[i[:, None].expand(-1, 3)[self.kept], self.cols[self.kept]] = True
        self.ws = api.alloc_workspace(self.desc)
        api.plan_mask(self.desc, self.mask, self.ws)

    def blocks(self, t):
        return t[0, 0, self.order].double().view(self.nb, 64, D)

    def keys(self, b):  # [nb, 192, channels]: the keys of every q-block's candidates
        return b[self.cols].reshape(self.nb, 192, b.shape[2])

    def maps(self, q, k):
        z = q @ self.keys(k).transpose(1, 2) / q.shape[2] ** 0.5
        drop = ~self.kept.repeat_interleave(64, 1)[:, None]
        return torch.softmax(z.masked_fill(drop, -float("inf")), 2)

    def back(self, w, x):  # sum over q-blocks of w^T x, at the keys
        out = torch.zeros(self.nb, 64, x.shape[2], dtype=torch.float64, device="cuda")
        part = (w.transpose(1, 2) @ x).view(self.nb, 3, 64, x.shape[2])
        return out.index_add_(0, self.cols.reshape(-1), part.reshape(-1, 64, x.shape[2]))

    def near(self, name, got, want, tol):
        bad = ~((self.blocks(got) - want).abs() <= tol + 1e-6)  # (NaN is bad)
        assert not bad.any(), f"{name}: {int(bad.sum())} outside"


@pytest.mark.parametrize("grid,tile", GRIDS, ids=["4097", "6144", "4500_deep", "5957_frames",
                                                  "6144_frames"])
def test_long_heads(grid, tile):
    p = Band(grid, tile, 3)
    tiles = p.nb if grid[0] in (1, 64) else (p.nb + 1) // 2
    assert api.get_mask(p.desc, p.ws)["tile_cnt"].shape[-1] == tiles
    q, k, v, g = p.x
    Q, K, V, G = (p.blocks(t) for t in p.x)
    # plain attention
    out = api.fwd(p.desc, q, k, v, p.ws, torch.full(q.shape, float("nan"), device="cuda"))
    assert api.check(p.desc, p.ws) == api.SA_OK
    P = p.maps(Q, K)
    p.near("out", out, P @ p.keys(V), (U + E) * (P @ p.keys(V.abs())))
    # differential attention and its gradients
    lam, e, s = 0.5, D // 2, (D // 2) ** -0.5
    out2 = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.empty(2, 1, 1, p.S, device="cuda")
    lam_t = torch.tensor([lam], device="cuda").bfloat16()
    out = api.fwd_diff(p.desc, q, k, v, lam_t, p.ws, out2=out2, lse=lse)
    dq, dk, dv, dl = (torch.full(sh, float("nan"), device="cuda")
                      for sh in (q.shape, q.shape, q.shape, (1,)))
    api.bwd_diff(p.desc, q, k, v, lam_t, out, out2, g, lse, p.ws, dq, dk, dv, dl)
    assert api.check(p.desc, p.ws) == api.SA_OK
    half = (slice(0, e), slice(e, D))
    A = [p.maps(Q[..., c], K[..., c]) for c in half]
    t2 = (U + E) * (A[1] @ p.keys(V.abs()))
    t1 = (U + E) * (A[0] @ p.keys(V.abs())) + lam * t2
    p.near("diff out", out, (A[0] - lam * A[1]) @ p.keys(V), t1)
    p.near("out2", out2, A[1] @ p.keys(V), t2)
    dP = G @ p.keys(V).transpose(1, 2)
    Pc = A[0] - lam * A[1]
    p.near("dv", dv, p.back(Pc, G), p.back(U * Pc.abs() + E * (A[0] + lam * A[1]), G.abs()))
    d2 = (G.abs() * t2).sum(2, keepdim=True)
    d1 = (G.abs() * t1).sum(2, keepdim=True) + lam * d2
    for m, (c, w, off) in enumerate(((half[0], 1.0, d1), (half[1], lam, d2))):
        Dm = (A[m] * dP).sum(2, keepdim=True)
        dS = (1.0 if m == 0 else -lam) * A[m] * (dP - Dm)
        term = U * dS.abs() + E * w * A[m] * (dP.abs() + Dm.abs())
        near = term + 2 * U * w * off * A[m]
        got = torch.zeros_like(dq), torch.zeros_like(dk)
        got[0][..., c], got[1][..., c] = dq[..., c], dk[..., c]
        want, tol = torch.zeros_like(Q), torch.zeros_like(Q)
        want[..., c], tol[..., c] = s * dS @ p.keys(K)[..., c], s * near @ p.keys(K.abs())[..., c]
        p.near(f"dq{m}", got[0], want, tol)
        want[..., c], tol[..., c] = s * p.back(dS, Q)[..., c], s * p.back(term, Q.abs())[..., c]
        p.near(f"dk{m}", got[1], want, tol)
    want = -(A[1] * dP).sum()
    assert abs(float(dl) - float(want)) <= 2 * E * float((A[1] * dP.abs()).sum()) + 1e-6


@pytest.mark.parametrize("T,nh", [(1, 4097), (1, 6144), (5958, 1), (6144, 1)])
def test_the_plan_of_q_and_k_reaches_every_tile(T, nh):
    """Values of 1 give 1 in every row (P is rounded once to bf16 and its sum is not), so a
    tile that no CTA works on shows."""
    desc = api.make_desc(1, 1, T, 8 * nh, 8, D, 0.9, out_fp32=True)
    gen = torch.Generator("cuda").manual_seed(nh)
    q, k = (torch.randn(1, 1, 64 * T * nh, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    ws = api.alloc_workspace(desc)
    api.plan(desc, q, k, ws)
    out = torch.full(q.shape, float("nan"), device="cuda")
    api.fwd(desc, q, k, torch.ones_like(q), ws, out)
    assert api.check(desc, ws) == api.SA_OK
    assert bool(((out - 1).abs() <= U + E).all())
