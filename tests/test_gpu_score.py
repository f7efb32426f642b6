"""Attention with a relative position bias and differential attention over a
block mask, on the GPU against the fp64 oracle (oracle/score.py), element by
element.

Tolerances, derived from the roundings (u = 2^-8, half a bf16 step relative to
the value; e = 2^-11 for the fp32 arithmetic: scores of |z| <= 64 are sums of at
most 128 products with 2^-24 each and 2^-22 from the exponential, so P is within
64 * 128 * 2^-24 = 2^-11 of itself at worst, and sums of such terms add no more
in relative terms):
  out      P is rounded once to bf16 for the product: (u + e) sum P |v|; a bf16
           output once more: u |out|
  dv       the same with dout; differential: the rounded factor is P1 - lam P2,
           whose fp32 error is e (P1 + lam P2)
  dk       dS rounded once: (u + e) sum |dS|' |q| scale, |dS|' = P (|dP| + |D|)
           standing for the fp32 error's size and |dS| for the rounding's
  dq       the same, and the provisional D~ = rowsum(dout * stored out), off by
           dD <= sum |dout| tol(out): dS~ is |dS| + P dD at most, and its
           correction dD * P K carries P's rounding: 2 u dD sum P |k| scale
  dtable   fp32 sums of dS: 2 e sum |dS|' (2: the sum's own roundings), bf16: u
  dlam     fp32 sums of P2 dP: 2 e sum P2 |dP|, bf16: u
  lse      e in absolute terms (ln of a sum of terms with relative error e)
Every bound gets 1e-6 for values near zero.
"""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api
from oracle import score

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

U, E = 2.0 ** -8, 2.0 ** -11
N_T, N_H, N_W = 6, 8, 10  # buckets of each axis in the tests' maps

# (B, H, T, Hh, Ww, d, tile, fp32): every block shape's column count, both head
# sizes, odd frame counts (lone tiles), one block per head, a batch
CASES = [
    (1, 2, 4, 8, 8, 64, None, True),
    (1, 1, 1, 8, 8, 128, None, True),           # one block per head
    (1, 2, 3, 8, 24, 128, None, True),          # odd frames: pairs along columns, a lone block
    (2, 2, 5, 16, 16, 128, None, False),
    (1, 2, 4, 8, 16, 128, (2, 4, 8), True),
    (1, 2, 6, 16, 16, 64, (2, 4, 8), False),
    (1, 1, 8, 8, 8, 128, (4, 4, 4), True),
    (1, 2, 2, 8, 32, 128, (1, 4, 16), True),
    (1, 1, 3, 4, 64, 64, (1, 2, 32), True),
    (1, 1, 3, 2, 128, 128, (1, 1, 64), True),
    (1, 1, 2, 64, 6, 128, (1, 32, 2), True),
    (1, 1, 64, 3, 5, 128, (64, 1, 1), True),
    (1, 1, 16, 8, 8, 64, (8, 8, 1), False),
]
IDS = ["x".join(map(str, c[:6])) + ("" if c[6] is None else "t" + "".join("_%d" % x for x in c[6])) +
       ("f" if c[7] else "b") for c in CASES]


class Problem:
    def __init__(self, case, seed=0, density=0.5, empty=True):
        self.B, self.H, self.T, self.Hh, self.Ww, self.d, tile, self.fp32 = case
        self.tile = tile or (1, 8, 8)
        self.S = self.T * self.Hh * self.Ww
        self.nb = self.S // 64
        rng = np.random.default_rng(seed + 7 * self.S + self.d)
        self.desc = api.make_desc(self.B, self.H, self.T, self.Hh, self.Ww, self.d, 0.0, tile=tile,
                                  out_fp32=self.fp32)
        shape = (self.B, self.H, self.S, self.d)
        base = rng.standard_normal(shape)  # q and k share a part: scores of some size
        self.q = self.bf16(rng.standard_normal(shape) + base)
        self.k = self.bf16(rng.standard_normal(shape) + base)
        self.v, self.g = self.bf16(rng.standard_normal(shape)), self.bf16(rng.standard_normal(shape))
        self.mask = rng.random((self.B * self.H, self.nb, self.nb)) < density
        if empty and self.nb > 2:
            self.mask[:, 1] = False          # a q-block that keeps nothing
            self.mask[0, :, 2] = False       # a k-block that nobody keeps
        if empty and self.nb > 5:            # a whole query tile that keeps nothing
            a, b = api.tile_blocks(self.desc, 1)
            self.mask[-1, [x for x in (a, b) if x >= 0]] = False
        if self.nb <= 2:
            self.mask[:] = True
        n = 2 * (self.T + self.Hh + self.Ww) - 3
        self.bucket = np.concatenate([
            rng.integers(0, N_T, 2 * self.T - 1), N_T + rng.integers(0, N_H, 2 * self.Hh - 1),
            N_T + N_H + rng.integers(0, N_W, 2 * self.Ww - 1)]).astype(np.int32)
        assert len(self.bucket) == n
        self.table = self.bf16(rng.standard_normal((self.H, N_T + N_H + N_W)))
        self.lam = self.bf16(rng.uniform(0.1, 0.9, self.H))

    @staticmethod
    def bf16(x):
        return torch.from_numpy(np.asarray(x, np.float32)).bfloat16()

    def dev(self):
        self.ws = api.alloc_workspace(self.desc)
        api.plan_mask(self.desc, torch.from_numpy(self.mask).cuda(), self.ws)
        return [x.cuda() for x in (self.q, self.k, self.v, self.g)]

    def head(self, bh):
        b, h = divmod(bh, self.H)
        return [x[b, h].double().numpy() for x in (self.q, self.k, self.v, self.g)]

    def keep(self, bh):
        return score.token_mask(self.mask[bh], self.T, self.Hh, self.Ww, self.tile)

    def out_tol(self, out, size, e):
        return (U + e) * size + (0 if self.fp32 else U) * np.abs(out) + 1e-6

    def check_ok(self):
        assert api.check(self.desc, self.ws) == api.SA_OK


def near(name, got, want, tol):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - want) > tol
    worst = np.max(np.abs(got - want) / tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, worst {worst:.2f} of the bound"


def check_bias(p, out, lse, grads=None, e=E):
    dq, dk, dv, dt = grads if grads is not None else (None,) * 4
    table = p.table.double().numpy()
    s, sums, sizes = 1 / np.sqrt(p.d), np.zeros(table.shape), np.zeros(table.shape)
    rnd = 0 if p.fp32 else U
    for bh in range(p.B * p.H):
        b, h = divmod(bh, p.H)
        q, k, v, g = p.head(bh)
        bias = score.bias_matrix(table[h], p.bucket, p.T, p.Hh, p.Ww)
        O, P, L = score.bias_head(q, k, v, p.keep(bh), bias)
        tol = p.out_tol(O, P @ np.abs(v), e)
        near("out", out[b, h], O, tol)
        if lse is not None:
            l = lse[b, h].double().cpu().numpy()
            assert np.array_equal(np.isinf(l), np.isinf(L))
            assert np.all(np.abs(l[np.isfinite(L)] - L[np.isfinite(L)]) <= e)
        if grads is None:
            continue
        rq, rk, rv, dS = score.bias_head_backward(q, k, v, g, P, O)
        dP = g @ v.T
        D = np.abs((g * O).sum(1, keepdims=True))
        big = P * (np.abs(dP) + D)
        dD = (np.abs(g) * tol).sum(1, keepdims=True)
        near("dv", dv[b, h], rv, (U + e) * (P.T @ np.abs(g)) + rnd * np.abs(rv) + 1e-6)
        near("dk", dk[b, h], rk, s * (U * np.abs(dS) + e * big).T @ np.abs(q) + rnd * np.abs(rk) + 1e-6)
        near("dq", dq[b, h], rq, s * (U * np.abs(dS) + e * big + 2 * U * dD * P) @ np.abs(k) +
             rnd * np.abs(rq) + 1e-6)
        sums[h] += score.bucket_sums(dS, p.bucket, table.shape[1], p.T, p.Hh, p.Ww)
        sizes[h] += score.bucket_sums(big, p.bucket, table.shape[1], p.T, p.Hh, p.Ww)
    if grads is not None:
        near("dtable", dt, sums, 2 * e * sizes + rnd * np.abs(sums) + 1e-6)


def check_diff(p, out, out2, lse, grads=None):
    dq, dk, dv, dl = grads if grads is not None else (None,) * 4
    lam = p.lam.double().numpy()
    e, rnd = p.d // 2, 0 if p.fp32 else U
    s = 1 / np.sqrt(e)
    sums, sizes = np.zeros(p.H), np.zeros(p.H)
    for bh in range(p.B * p.H):
        b, h = divmod(bh, p.H)
        q, k, v, g = p.head(bh)
        O, O2, P, L = score.diff_head(q, k, v, p.keep(bh), lam[h])
        t2 = (U + E) * (P[1] @ np.abs(v))
        t1 = (U + E) * (P[0] @ np.abs(v)) + lam[h] * t2
        near("out", out[b, h], O, t1 + rnd * np.abs(O) + 1e-6)
        if out2 is not None:
            near("out2", out2[b, h], O2, t2 + rnd * np.abs(O2) + 1e-6)
        if lse is not None:
            for m in range(2):
                l = lse[m, b, h].double().cpu().numpy()
                assert np.array_equal(np.isinf(l), np.isinf(L[m]))
                assert np.all(np.abs(l[np.isfinite(L[m])] - L[m][np.isfinite(L[m])]) <= E)
        if grads is None:
            continue
        rq, rk, rv, rl, dS = score.diff_head_backward(q, k, v, g, P, lam[h])
        dP = g @ v.T
        Pc, both = np.abs(P[0] - lam[h] * P[1]), P[0] + lam[h] * P[1]
        near("dv", dv[b, h], rv, (U * Pc + E * both).T @ np.abs(g) + rnd * np.abs(rv) + 1e-6)
        # D~ of map 2 from the stored out2, of map 1 from out + lam out2
        d2 = (np.abs(g) * (t2 + rnd * np.abs(O2))).sum(1, keepdims=True)
        d1 = (np.abs(g) * (t1 + rnd * np.abs(O))).sum(1, keepdims=True) + lam[h] * d2
        tq, tk = np.zeros_like(rq), np.zeros_like(rk)
        for m, (c, w, dD) in enumerate(((slice(0, e), 1.0, d1), (slice(e, p.d), lam[h], d2))):
            D = np.abs((P[m] * dP).sum(1, keepdims=True))
            term = U * np.abs(dS[m]) + E * w * P[m] * (np.abs(dP) + D)
            tk[:, c] = s * term.T @ np.abs(q[:, c])
            tq[:, c] = s * (term + 2 * U * w * dD * P[m]) @ np.abs(k[:, c])
        near("dk", dk[b, h], rk, tk + rnd * np.abs(rk) + 1e-6)
        near("dq", dq[b, h], rq, tq + rnd * np.abs(rq) + 1e-6)
        sums[h] += rl
        sizes[h] += (P[1] * np.abs(dP)).sum()
    if grads is not None:
        near("dlam", dl, sums, 2 * E * sizes + rnd * np.abs(sums) + 1e-6)


def run_bias(p, q, k, v, g, table, bucket, **kw):
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    out = api.fwd_bias(p.desc, q, k, v, table, bucket, p.ws, lse=lse, **kw)
    return out, lse, api.bwd_bias(p.desc, q, k, v, table, bucket, out, g, lse, p.ws, **kw)


def run_diff(p, q, k, v, g, lam, **kw):
    lse = torch.empty((2,) + tuple(q.shape[:3]), dtype=torch.float32, device="cuda")
    out2 = torch.empty(q.shape, dtype=torch.float32 if p.fp32 else torch.bfloat16, device="cuda")
    out = api.fwd_diff(p.desc, q, k, v, lam, p.ws, out2=out2, lse=lse, **kw)
    return out, out2, lse, api.bwd_diff(p.desc, q, k, v, lam, out, out2, g, lse, p.ws, **kw)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_bias_matches_oracle(case):
    p = Problem(case)
    q, k, v, g = p.dev()
    out, lse, grads = run_bias(p, q, k, v, g, p.table.cuda(), torch.from_numpy(p.bucket).cuda())
    p.check_ok()
    check_bias(p, out, lse, grads)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_diff_matches_oracle(case):
    p = Problem(case, seed=1)
    q, k, v, g = p.dev()
    out, out2, lse, grads = run_diff(p, q, k, v, g, p.lam.cuda())
    p.check_ok()
    check_diff(p, out, out2, lse, grads)


@pytest.mark.parametrize("density", [0.0, 0.05, 1.0])
def test_densities(density):
    """Nothing kept at all, sparse lists, everything kept."""
    p = Problem((1, 2, 3, 16, 16, 128, None, True), seed=2, density=density, empty=density < 1)
    q, k, v, g = p.dev()
    bucket = torch.from_numpy(p.bucket).cuda()
    check_bias(p, *run_bias(p, q, k, v, g, p.table.cuda(), bucket))
    check_diff(p, *run_diff(p, q, k, v, g, p.lam.cuda()))
    p.check_ok()


@pytest.mark.parametrize("d", [64, 128])
def test_more_tiles_than_one_wave(d):
    """600 query tiles, 5 a head: two tiles per CTA in the biased forward (a lone one in
    each head's last), key tiles sorted, heads dealt out in groups."""
    p = Problem((10, 12, 3, 8, 24, d, None, False), seed=13, density=0.4)
    q, k, v, g = p.dev()
    check_bias(p, *run_bias(p, q, k, v, g, p.table.cuda(), torch.from_numpy(p.bucket).cuda()))
    check_diff(p, *run_diff(p, q, k, v, g, p.lam.cuda()))
    p.check_ok()


def test_masked_offsets():
    """Entries of -inf and of the lowest value mask; a row with all offsets masked is
    one that keeps nothing."""
    p = Problem((1, 2, 4, 8, 8, 128, None, True), seed=3, empty=False)
    p.table[0, N_T + 2] = -float("inf")
    p.table[0, N_T + N_H + 1] = torch.finfo(torch.bfloat16).min
    p.table[1, 1] = -1e30  # bf16: -1.0003e30, below the limit
    p.bucket[:7] = [0, 1, 1, 1, 1, 1, 0]  # offsets of -3 .. 3 frames
    p.mask[1] = np.eye(p.nb, dtype=bool)  # head 1: only offsets of frame 0, which are masked
    q, k, v, g = p.dev()
    out, lse, grads = run_bias(p, q, k, v, g, p.table.cuda(), torch.from_numpy(p.bucket).cuda())
    p.check_ok()
    assert torch.all(out[0, 1] == 0) and torch.all(lse[0, 1] == -float("inf"))
    assert all(torch.all(x[0, 1] == 0) for x in grads[:3]) and torch.all(grads[3][1] == 0)
    check_bias(p, out, lse, grads)


def test_large_scores():
    """Scores whose exponentials overflow without the running maximum."""
    p = Problem((1, 1, 2, 8, 8, 64, None, True), seed=4, empty=False)
    p.table = p.bf16(80.0 * p.table.float().numpy())
    q, k, v, g = p.dev()
    out, lse, grads = run_bias(p, q, k, v, g, p.table.cuda(), torch.from_numpy(p.bucket).cuda())
    p.check_ok()
    assert all(torch.isfinite(x.float()).all() for x in (out,) + grads)
    # |z| <= 400 instead of 64: the fp32 score error is that much larger
    check_bias(p, out, lse, grads, e=E * 400 / 64)


def test_forward_alone_and_optional_outputs():
    p = Problem((1, 2, 3, 8, 24, 128, None, False), seed=5)
    q, k, v, g = p.dev()
    bucket = torch.from_numpy(p.bucket).cuda()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    a = api.fwd_bias(p.desc, q, k, v, p.table.cuda(), bucket, p.ws)
    b = api.fwd_bias(p.desc, q, k, v, p.table.cuda(), bucket, p.ws, lse=lse)
    assert torch.equal(a, b)
    check_bias(p, a, None)
    a = api.fwd_diff(p.desc, q, k, v, p.lam.cuda(), p.ws)
    check_diff(p, a, None, None)
    assert torch.equal(a, run_diff(p, q, k, v, g, p.lam.cuda())[0])


def test_same_bits_every_run():
    p = Problem((1, 4, 6, 24, 24, 128, None, True), seed=6)
    q, k, v, g = p.dev()
    table, bucket, lam = p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.lam.cuda()
    first = run_bias(p, q, k, v, g, table, bucket), run_diff(p, q, k, v, g, lam)
    for _ in range(3):
        again = run_bias(p, q, k, v, g, table, bucket), run_diff(p, q, k, v, g, lam)
        for x, y in zip(first, again):
            assert all(torch.equal(a, b) for a, b in zip(x[:-1], y[:-1]))
            assert all(torch.equal(a, b) for a, b in zip(x[-1], y[-1]))


def lists(p, ws):
    m = api.get_mask(p.desc, ws)
    out = [m["cnt"].clone(), m["tile_cnt"].clone()]
    for cnt, idx in ((m["cnt"], m["idx"]), (m["tile_cnt"], m["tile_idx"])):
        col = torch.arange(idx.shape[2], device="cuda")
        out.append(torch.where(col < cnt[..., None], idx, -1))
    return out


@pytest.mark.parametrize("case", [CASES[2], CASES[3], CASES[4], (1, 3, 9, 24, 40, 64, None, True)])
def test_plan_mask_equals_plan_of_the_same_mask(case):
    """The mask that sparse_attn_plan chose, given back as bytes, makes the same lists;
    a shared mask is that mask for every head."""
    p = Problem(case, seed=7)
    q, k, v, g = p.dev()
    d = api.make_desc(p.B, p.H, p.T, p.Hh, p.Ww, p.d, 0.3, tile=case[6], out_fp32=p.fp32)
    ws, ws2 = api.alloc_workspace(d), api.alloc_workspace(d)
    api.plan(d, q, k, ws)
    cnt, _, idx, _ = lists(p, ws)
    mask = torch.zeros(p.B * p.H, p.nb, p.nb + 1, dtype=torch.uint8, device="cuda")
    mask.scatter_(2, torch.where(idx < 0, p.nb, idx).long(), 200)  # any non-zero byte keeps
    mask = mask[:, :, :p.nb].contiguous()
    api.plan_mask(d, mask, ws2)
    assert all(torch.equal(a, b) for a, b in zip(lists(p, ws), lists(p, ws2)))
    api.plan_mask(d, mask.view(p.B, p.H, p.nb, p.nb), ws2)
    assert all(torch.equal(a, b) for a, b in zip(lists(p, ws), lists(p, ws2)))
    a, b = torch.empty_like(q, dtype=torch.float32 if p.fp32 else torch.bfloat16), None
    api.fwd(d, q, k, v, ws, a)
    b = api.fwd(d, q, k, v, ws2, torch.empty_like(a))
    assert torch.equal(a, b)
    api.plan_mask(d, mask[0].contiguous().bool(), ws)
    api.plan_mask(d, mask[:1].expand(p.B * p.H, -1, -1).contiguous(), ws2)
    assert all(torch.equal(a, b) for a, b in zip(lists(p, ws), lists(p, ws2)))


def test_plain_attention_on_rows_that_keep_nothing():
    """sparse_attn_fwd, fwd_lse and bwd over a caller's mask: empty rows are written."""
    p = Problem((1, 2, 6, 16, 16, 128, None, True), seed=8)
    q, k, v, g = p.dev()
    out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float32, device="cuda")
    api.fwd_lse(p.desc, q, k, v, p.ws, out, lse)
    grads = api.bwd(p.desc, q, k, v, out, g, lse, p.ws)
    p.check_ok()
    p.table[:] = 0
    check_bias(p, out, lse)
    for bh in range(2):
        keep = torch.from_numpy(p.keep(bh))
        rows, cols = ~keep.any(1), ~keep.any(0)
        assert rows.any() and torch.all(out[0, bh].cpu()[rows] == 0)
        assert torch.all(grads[0][0, bh].cpu()[rows] == 0)
        assert torch.all(grads[1][0, bh].cpu()[cols] == 0) and torch.all(grads[2][0, bh].cpu()[cols] == 0)
    empty = Problem((1, 1, 2, 8, 8, 64, None, False), seed=8)
    q, k, v, g = empty.dev()
    api.plan_mask(empty.desc, torch.zeros(2, 2, dtype=torch.bool, device="cuda"), empty.ws)
    out = api.fwd(empty.desc, q, k, v, empty.ws, torch.full_like(q, 3.0))
    empty.check_ok()
    assert torch.all(out == 0)


def test_a_layer_of_all_of_them():
    """One plan of the layer's own q and k, read by biased and by differential heads;
    their outputs add up and so do the gradients."""
    p = Problem((1, 2, 4, 16, 24, 128, None, True), seed=9)
    p.desc = api.make_desc(1, 2, 4, 16, 24, 128, 0.2, out_fp32=True)
    attn = api.NablaAttention(1, 2, 4, 16, 24, 128, 0.2, out_fp32=True)
    q, k, v, g = p.dev()
    attn.plan(q, k)
    _, _, idx, _ = lists(p, attn.workspace)
    mask = torch.zeros(2, p.nb, p.nb + 1, dtype=torch.bool, device="cuda")
    mask.scatter_(2, torch.where(idx < 0, p.nb, idx).long(), True)
    p.mask = mask[:, :, :p.nb].cpu().numpy()
    table, bucket, lam = p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.lam.cuda()
    a, la = attn.forward_bias(q, k, v, table, bucket)
    b, b2, lb = attn.forward_diff(q, k, v, lam)
    ga = attn.backward_bias(q, k, v, table, bucket, a, g, la)
    gb = attn.backward_diff(q, k, v, lam, b, b2, g, lb)
    assert attn.check() == api.SA_OK
    check_bias(p, a, la, ga)
    check_diff(p, b, b2, lb, gb)
    total = [x + y for x, y in zip(ga[:3], gb[:3])]
    for bh in range(2):
        q_, k_, v_, g_ = p.head(bh)
        O, P, _ = score.bias_head(q_, k_, v_, p.keep(bh), score.bias_matrix(
            p.table[bh].double().numpy(), p.bucket, 4, 16, 24))
        r1 = score.bias_head_backward(q_, k_, v_, g_, P, O)
        _, _, P2, _ = score.diff_head(q_, k_, v_, p.keep(bh), float(p.lam[bh]))
        r2 = score.diff_head_backward(q_, k_, v_, g_, P2, float(p.lam[bh]))
        for x, y, z in zip(total, r1, r2):
            want = y + z
            assert np.linalg.norm(x[0, bh].cpu().numpy() - want) <= 4 * U * np.linalg.norm(want)


def test_other_stream_and_graphs():
    """On a stream of its own, and captured into two CUDA graphs on buffers of their own:
    replays follow new inputs and equal direct calls bit for bit."""
    p = Problem((1, 2, 5, 16, 16, 128, None, True), seed=10)
    q, k, v, g = p.dev()
    table, bucket, lam = p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.lam.cuda()
    want = run_bias(p, q, k, v, g, table, bucket), run_diff(p, q, k, v, g, lam)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run_bias(p, q, k, v, g, table, bucket, stream=side), run_diff(p, q, k, v, g, lam, stream=side)
    side.synchronize()
    for x, y in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(x[:-1] + x[-1], y[:-1] + y[-1]))
    graphs = []
    for fn, more in ((run_bias, (table, bucket)), (run_diff, (lam,))):
        bufs = [x.clone() for x in (q, k, v, g)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fn(p, *bufs, *more)
        graphs.append((graph, bufs, out, fn, more))
    fresh = [torch.roll(x, 1, dims=2).contiguous() for x in (q, k, v, g)]
    for graph, bufs, *_ in graphs:
        for b, x in zip(bufs, fresh):
            b.copy_(x)
    for graph, *_ in graphs:
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    for _, _, out, fn, more in graphs:
        direct = fn(p, *fresh, *more)
        assert all(torch.equal(a, b) for a, b in zip(out[:-1] + out[-1], direct[:-1] + direct[-1]))
    p.check_ok()


def test_binding_refuses_wrong_tensors():
    p = Problem((1, 2, 4, 8, 8, 64, None, False), seed=14, empty=False)
    q, k, v, g = p.dev()
    table, bucket, lam = p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.lam.cuda()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    for mask in (torch.ones(3, 4, 4, dtype=torch.bool), torch.ones(2, 4, 4),
                 torch.ones(4, 2, 4, dtype=torch.bool).transpose(0, 1)):
        with pytest.raises(ValueError):
            api.plan_mask(p.desc, mask.cuda(), p.ws)
    for t, b, kw in ((table.float(), bucket, {}), (table[:1], bucket, {}), (table, bucket[1:], {}),
                     (table, bucket.long(), {}), (table, bucket, {"lse": lse[..., 1:]}),
                     (table, bucket, {"out": q.float()})):
        with pytest.raises(ValueError):
            api.fwd_bias(p.desc, q, k, v, t, b, p.ws, **kw)
    with pytest.raises(ValueError):
        api.fwd_bias(p.desc, q.transpose(2, 3).contiguous().transpose(2, 3), k, v, table, bucket, p.ws)
    for kw in ({"lse": lse}, {"out2": q.float()}):
        with pytest.raises(ValueError):
            api.fwd_diff(p.desc, q, k, v, lam, p.ws, **kw)
    with pytest.raises(ValueError):
        api.fwd_diff(p.desc, q, k, v, lam[:1], p.ws)
    with pytest.raises(ValueError):
        api.bwd_bias(p.desc, q, k, v, table, bucket, q, g, lse, p.ws, dtable=table.float())
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(api.SparseAttnError):
        api.bwd_bias(p.desc, q, k, v, table, bucket, q, g, lse, p.ws, scratch=small)
    with pytest.raises(api.SparseAttnError):
        api.plan_mask(p.desc, torch.ones(4, 4, dtype=torch.bool, device="cuda"), small)
    p.check_ok()


def test_bad_bucket_is_reported():
    p = Problem((1, 1, 2, 8, 8, 64, None, True), seed=11, empty=False)
    q, k, v, g = p.dev()
    bucket = torch.from_numpy(p.bucket).cuda()
    bucket[0], bucket[5] = -1, N_T + N_H + N_W  # both read entry 0
    out, lse, grads = run_bias(p, q, k, v, g, p.table.cuda(), bucket)
    assert api.check(p.desc, p.ws) == api.SA_ERR_DEVICE_TIMEOUT
    p.bucket[0] = p.bucket[5] = 0
    check_bias(p, out, lse, grads)


@pytest.mark.parametrize("op", ["bias", "diff"])
def test_a_wait_that_runs_out_is_reported(op):
    """The test hook's load that never comes: the calls end, the status says so, and the
    next calls are right."""
    p = Problem((1, 1, 3, 8, 24, 128, None, True), seed=12)
    q, k, v, g = p.dev()
    table, bucket, lam = p.table.cuda(), torch.from_numpy(p.bucket).cuda(), p.lam.cuda()
    good, stall = p.desc, api.make_desc(1, 1, 3, 8, 24, 128, 0.0, out_fp32=True,
                                        debug_flags=api.SA_DEBUG_STALL_LOADER)
    run = (lambda: run_bias(p, q, k, v, g, table, bucket)) if op == "bias" else \
        (lambda: run_diff(p, q, k, v, g, lam))
    p.desc = stall
    run()
    assert api.check(stall, p.ws) == api.SA_ERR_DEVICE_TIMEOUT
    p.desc = good
    p.dev()  # plans again
    res = run()
    p.check_ok()
    check_bias(p, *res) if op == "bias" else check_diff(p, *res)


def test_lists_longer_than_the_staged_ones():
    """2,944 blocks: a query tile whose union list and a key tile whose list run past
    the 2,880 entries staged in shared memory. Every q-block keeps itself and block c;
    q-block r keeps all."""
    T, Hh, Ww, d = 46, 64, 64, 128
    nb, S, r, c = 2944, 46 * 64 * 64, 1500, 700
    gen = torch.Generator("cuda").manual_seed(5)
    q, k, v, g = (torch.randn(1, 1, S, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    mask = torch.eye(nb, dtype=torch.bool, device="cuda")
    mask[r] = True
    mask[:, c] = True
    desc = api.make_desc(1, 1, T, Hh, Ww, d, 0.0, out_fp32=True)
    ws = api.alloc_workspace(desc)
    api.plan_mask(desc, mask, ws)
    bucket, n = api.relative_buckets(T, Hh, Ww)
    table = torch.randn(1, n, generator=gen, device="cuda").bfloat16()
    lam = torch.tensor([0.5], device="cuda").bfloat16()

    class P:
        pass
    p = P()
    p.desc, p.ws, p.fp32 = desc, ws, True
    out, lse, (dq, dk, dv, dt) = run_bias(p, q, k, v, g, table, bucket)
    o_d, o2, l_d, (dq_d, dk_d, dv_d, dl) = run_diff(p, q, k, v, g, lam)
    assert api.check(desc, ws) == api.SA_OK
    # fp64 over blocks in fractal order
    pos = torch.arange(S, device="cuda")
    t, h, w = pos // (Hh * Ww), pos // Ww % Hh, pos % Ww
    order = torch.argsort((t * 8 + h // 8) * 8 + w // 8, stable=True)
    x = [y[0, 0, order].double() for y in (q, k, v, g)]
    tab = torch.where(table[0].double() <= score.MASKED, -float("inf"), table[0].double())
    base = (0, 2 * T - 1, 2 * T - 1 + 2 * Hh - 1)
    co = [y[order] for y in (t, h, w)]

    def block_rows(i, keys):
        rows = slice(64 * i, 64 * i + 64)
        Q, K, V, G = x[0][rows], x[1][keys], x[2][keys], x[3][rows]
        bias = sum(tab[bucket[base[a] + (co[a][keys][None] - co[a][rows][:, None]) + m - 1].long()]
                   for a, m in enumerate((T, Hh, Ww)))
        P = torch.softmax(Q @ K.T / d ** 0.5 + bias, 1)
        dP = G @ V.T
        dS = P * (dP - (P * dP).sum(1, keepdim=True))
        e = d // 2
        A = [torch.softmax(Q[:, s] @ K[:, s].T / e ** 0.5, 1) for s in (slice(0, e), slice(e, d))]
        Z = [a * (dP - (a * dP).sum(1, keepdim=True)) for a in A]
        Pd = A[0] - 0.5 * A[1]
        return (P @ V, dS @ K / d ** 0.5, dS.T @ Q / d ** 0.5, P.T @ G, Pd @ V,
                torch.cat([Z[0] @ K[:, :e], -0.5 * Z[1] @ K[:, e:]], 1) / e ** 0.5,
                torch.cat([Z[0].T @ Q[:, :e], -0.5 * Z[1].T @ Q[:, e:]], 1) / e ** 0.5, Pd.T @ G)

    full = torch.arange(S, device="cuda")
    row = block_rows(r, full)
    at = order[64 * r:64 * r + 64]
    kc = torch.arange(64 * c, 64 * c + 64, device="cuda")
    col = [torch.zeros(64, d, dtype=torch.float64, device="cuda") for _ in range(4)]
    for i in range(nb):
        if i == r:
            part = [z[kc] for z in (row[2], row[3], row[6], row[7])]
        else:
            keys = kc if i == c else torch.cat([torch.arange(64 * i, 64 * i + 64, device="cuda"), kc])
            b = block_rows(i, keys)
            part = [z[-64:] for z in (b[2], b[3], b[6], b[7])]
        for s, z in zip(col, part):
            s += z
    ck = order[kc]
    # whole blocks in the 2-norm: independent roundings of u each, 1.5 u in all
    for name, got, want in (("out", out[0, 0, at], row[0]), ("dq", dq[0, 0, at], row[1]),
                            ("diff out", o_d[0, 0, at], row[4]), ("diff dq", dq_d[0, 0, at], row[5]),
                            ("dk", dk[0, 0, ck], col[0]), ("dv", dv[0, 0, ck], col[1]),
                            ("diff dk", dk_d[0, 0, ck], col[2]), ("diff dv", dv_d[0, 0, ck], col[3])):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 1.5 * U, (name, off)
