"""Everything that lists past the staged 2,880 entries give, and the plain gradients
beside rows that keep nothing: element by element against fp64 (bounds of
test_gpu_score; the plain backward's D is rowsum(dout * stored out), off by dD =
sum |dout| tol(out), which goes into its dS as P dD)."""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api
from oracle import score
from tests.test_gpu_score import E, U, Problem, near

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

LN = -float("inf")


def test_every_value_of_lists_longer_than_the_staged_ones():
    """2,944 blocks, each keeping itself and block c; block r keeps all: dtable, dlambda
    and the log-sum-exps with the rest, on offset tables of 300 entries."""
    T, Hh, Ww, d, nb, r, c = 46, 64, 64, 128, 2944, 1500, 700
    S, e = 64 * nb, d // 2
    gen = torch.Generator("cuda").manual_seed(6)
    q, k, v, g = (torch.randn(1, 1, S, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    mask = torch.eye(nb, dtype=torch.bool, device="cuda")
    mask[r] = True
    mask[:, c] = True
    desc = api.make_desc(1, 1, T, Hh, Ww, d, 0.0, out_fp32=True)
    ws = api.alloc_workspace(desc)
    api.plan_mask(desc, mask, ws)
    bucket, n = api.relative_buckets(T, Hh, Ww)
    table = torch.randn(1, n, generator=gen, device="cuda").bfloat16()
    lam_t, lam = torch.tensor([0.5], device="cuda").bfloat16(), 0.5
    lse, lse2 = torch.empty(1, 1, S, device="cuda"), torch.empty(2, 1, 1, S, device="cuda")
    out = api.fwd_bias(desc, q, k, v, table, bucket, ws, lse=lse)
    got = dict(zip(("dq", "dk", "dv", "dt"),
                   api.bwd_bias(desc, q, k, v, table, bucket, out, g, lse, ws)), out=out, lse=lse)
    out2 = torch.empty_like(out)
    out_d = api.fwd_diff(desc, q, k, v, lam_t, ws, out2=out2, lse=lse2)
    got_d = dict(zip(("dq", "dk", "dv", "dl"),
                     api.bwd_diff(desc, q, k, v, lam_t, out_d, out2, g, lse2, ws)),
                 out=out_d, out2=out2, lse=lse2)
    assert api.check(desc, ws) == api.SA_OK

    pos = torch.arange(S, device="cuda")
    co = [pos // (Hh * Ww), pos // Ww % Hh, pos % Ww]
    order = torch.argsort((co[0] * 8 + co[1] // 8) * 8 + co[2] // 8, stable=True)
    co = [x[order].view(nb, 64) for x in co]
    Q, K, V, G = (x[0, 0, order].double().view(nb, 64, d) for x in (q, k, v, g))
    names = ("out", "dq", "dk", "dv", "out_d", "out2", "dq_d", "dk_d", "dv_d")
    want, tol = ({s: torch.zeros(nb, 64, d, dtype=torch.float64, device="cuda") for s in names}
                 for _ in range(2))
    stats = torch.zeros(3, nb, 64, dtype=torch.float64, device="cuda")
    sums, sizes = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    dl, dl_size = 0.0, 0.0
    tab, first = table[0].double(), (0, 2 * T - 1, 2 * T - 1 + 2 * Hh - 1)

    def rows(blocks, keys, keep):
        """q-blocks [b], their k-blocks [b, m], kept [b, m]."""
        nonlocal dl, dl_size
        b, m = keys.shape
        x, gy = Q[blocks], G[blocks]
        kk, vv = (t[keys].reshape(b, 64 * m, d) for t in (K, V))
        drop = ~keep.repeat_interleave(64, 1)[:, None]
        idx = [bucket[first[a] + (co[a][keys].reshape(b, 1, -1) - co[a][blocks][:, :, None]) + size - 1].long()
               for a, size in enumerate((T, Hh, Ww))]

        def put(where, name, w, t):
            where[name].view(nb, 64, d).index_add_(0, keys.reshape(-1), (w.transpose(1, 2) @ t).view(
                b * m, 64, d))
        dP = gy @ vv.transpose(1, 2)
        ga, va = gy.abs(), vv.abs()
        # the bias
        z = (x @ kk.transpose(1, 2) / d ** 0.5 + sum(tab[i] for i in idx)).masked_fill(drop, LN)
        stats[0, blocks] = z.logsumexp(2)
        P = torch.softmax(z, 2)
        O, to = P @ vv, (U + E) * (P @ va)
        want["out"][blocks], tol["out"][blocks] = O, to
        D = (P * dP).sum(2, keepdim=True)
        dS, big = P * (dP - D), P * (dP.abs() + D.abs())
        off = (ga * to).sum(2, keepdim=True)
        s = d ** -0.5
        want["dq"][blocks] = s * dS @ kk
        tol["dq"][blocks] = s * (U * dS.abs() + E * big + 2 * U * off * P) @ kk.abs()
        put(want, "dk", s * dS, x), put(tol, "dk", s * (U * dS.abs() + E * big), x.abs())
        put(want, "dv", P, gy), put(tol, "dv", (U + E) * P, ga)
        for i in idx:
            sums.index_add_(0, i.reshape(-1), dS.reshape(-1))
            sizes.index_add_(0, i.reshape(-1), big.reshape(-1))
        # the two maps
        s, half = e ** -0.5, (slice(0, e), slice(e, d))
        Z = [(x[..., h] @ kk[..., h].transpose(1, 2) * s).masked_fill(drop, LN) for h in half]
        A = [torch.softmax(t, 2) for t in Z]
        for i in range(2):
            stats[1 + i, blocks] = Z[i].logsumexp(2)
        t2 = (U + E) * (A[1] @ va)
        t1 = (U + E) * (A[0] @ va) + lam * t2
        Pc = A[0] - lam * A[1]
        want["out_d"][blocks], tol["out_d"][blocks] = Pc @ vv, t1
        want["out2"][blocks], tol["out2"][blocks] = A[1] @ vv, t2
        put(want, "dv_d", Pc, gy), put(tol, "dv_d", U * Pc.abs() + E * (A[0] + lam * A[1]), ga)
        d2 = (ga * t2).sum(2, keepdim=True)
        d1 = (ga * t1).sum(2, keepdim=True) + lam * d2
        for i, (h, w, off) in enumerate(((half[0], 1.0, d1), (half[1], lam, d2))):
            D = (A[i] * dP).sum(2, keepdim=True)
            dS = (1.0 if i == 0 else -lam) * A[i] * (dP - D)
            term = U * dS.abs() + E * w * A[i] * (dP.abs() + D.abs())
            want["dq_d"][blocks, :, h] = s * dS @ kk[..., h]
            tol["dq_d"][blocks, :, h] = s * (term + 2 * U * w * off * A[i]) @ kk[..., h].abs()
            part = torch.zeros_like(x)
            part[..., h] = x[..., h]
            put(want, "dk_d", s * dS, part), put(tol, "dk_d", s * term, part.abs())
        dl -= float((A[1] * dP).sum())
        dl_size += float((A[1] * dP.abs()).sum())

    others = torch.tensor([i for i in range(nb) if i != r], device="cuda")
    for part in others.split(368):
        keys = torch.stack([part, torch.full_like(part, c)], 1)
        keep = torch.stack([torch.ones_like(part, dtype=torch.bool), part != c], 1)
        rows(part, keys, keep)
    rows(torch.tensor([r], device="cuda"), torch.arange(nb, device="cuda")[None],
         torch.ones(1, nb, dtype=torch.bool, device="cuda"))

    def close(name, x, ref, bound):
        bad = ~((x[0, 0, order].double().view(nb, 64, d) - ref).abs() <= bound + 1e-6)
        assert not bad.any(), f"{name}: {int(bad.sum())} outside"
    for name in ("out", "dq", "dk", "dv"):
        close(name, got[name], want[name], tol[name])
        close("diff " + name, got_d[name], want[name + "_d"], tol[name + "_d"])
    close("out2", got_d["out2"], want["out2"], tol["out2"])
    for x, ref in zip((got["lse"][0, 0], lse2[0, 0, 0], lse2[1, 0, 0]), stats):
        assert bool(((x[order].double().view(nb, 64) - ref).abs() <= E).all())
    assert bool(((got["dt"][0].double() - sums).abs() <= 2 * E * sizes + 1e-6).all())
    assert abs(float(got_d["dl"]) - dl) <= 2 * E * dl_size + 1e-6


@pytest.mark.parametrize("d", [64, 128])
def test_plain_gradients_beside_rows_that_keep_nothing(d):
    p = Problem((1, 2, 6, 16, 16, d, None, True), seed=24)
    q, k, v, g = p.dev()
    out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float32, device="cuda")
    api.fwd_lse(p.desc, q, k, v, p.ws, out, lse)
    grads = api.bwd(p.desc, q, k, v, out, g, lse, p.ws)
    p.check_ok()
    s = d ** -0.5
    for bh in range(2):
        Q, K, V, G = p.head(bh)
        keep = p.keep(bh)
        assert (~keep.any(1)).any()
        O, P, L = score.bias_head(Q, K, V, keep, 0.0)
        tol = (U + E) * (P @ np.abs(V))
        near("out", out[0, bh], O, tol + 1e-6)
        rq, rk, rv, dS = score.bias_head_backward(Q, K, V, G, P, O)
        dP = G @ V.T
        big = P * (np.abs(dP) + np.abs((G * O).sum(1, keepdims=True)))
        term = U * np.abs(dS) + E * big + P * (np.abs(G) * tol).sum(1, keepdims=True)
        near("dq", grads[0][0, bh], rq, s * term @ np.abs(K) + 1e-6)
        near("dk", grads[1][0, bh], rk, s * term.T @ np.abs(Q) + 1e-6)
        near("dv", grads[2][0, bh], rv, (U + E) * (P.T @ np.abs(G)) + 1e-6)
