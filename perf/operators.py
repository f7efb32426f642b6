"""Attention operators over a caller's block mask, as cases to measure: attention with a learned relative position
bias by buckets, and differential attention, each as a forward pass and as a training step (forward and gradients).

The tokens of a head are a video grid (T, Hh, Ww) in natural order, t outermost. A block is N = 64 tokens: an 8 x 8
patch of one frame, or a tile (pt, ph, pw). A block mask says which k-blocks each q-block attends to; it is what a
program has in hand from its own scorer, here the best blocks of the pooled map of each row, with some rows left empty.
"""
import math

import torch

own = False
N = 64
_CHUNK = 1 << 28  # scores of one chunk of the plain form: 1 GB in 32 bits

# op: bias or diff; train: forward and gradients, otherwise the forward alone; keep: the share of the k-blocks that a
# row keeps; empty: rows of each head that keep none (padding); pt, ph, pw = 0: 8 x 8 patches.


def _case(name, op, train, B, H, grid, d, keep, empty=0, tile=(0, 0, 0)):
    return {"name": name, "op": op, "train": train, "B": B, "H": H, "T": grid[0], "Hh": grid[1], "Ww": grid[2],
            "d": d, "keep": keep, "empty": empty, "pt": tile[0], "ph": tile[1], "pw": tile[2]}


def listed():
    return [
        # the smallest clip: a preview of four frames, where the launches' latency counts
        _case("bias_fwd_256", "bias", False, 1, 2, (4, 8, 8), 64, 0.5),
        # a short clip at low resolution, batch of two, blocks that reach over frames, padded rows
        _case("bias_fwd_2x5760_tile", "bias", False, 2, 6, (6, 24, 40), 64, 0.3, 3, (2, 4, 8)),
        # one layer's heads on a short clip
        _case("bias_fwd_8192", "bias", False, 1, 12, (8, 32, 32), 128, 0.25),
        # a whole clip of the middle size
        _case("bias_fwd_37632", "bias", False, 1, 12, (21, 32, 56), 128, 0.12),
        # a training step on a crop: odd frame count, few blocks, an empty row
        _case("bias_train_1920", "bias", True, 1, 4, (5, 16, 24), 64, 0.4, 1),
        # a training step on a short clip
        _case("bias_train_8192", "bias", True, 1, 12, (8, 32, 32), 128, 0.25),
        # the same range for differential attention
        _case("diff_fwd_256", "diff", False, 1, 2, (4, 8, 8), 64, 0.5),
        _case("diff_fwd_8192", "diff", False, 1, 12, (8, 32, 32), 128, 0.25),
        # the longest clip, a few heads of it (a shard of the layer)
        _case("diff_fwd_61440", "diff", False, 1, 4, (16, 48, 80), 128, 0.1),
        # a crop of a single frame with every block kept (dense)
        _case("diff_train_2x960_dense", "diff", True, 2, 3, (1, 24, 40), 64, 1.0, 0),
        _case("diff_train_8192", "diff", True, 1, 12, (8, 32, 32), 128, 0.25, 2),
        # a training step on the clip of the middle size, half the heads
        _case("diff_train_37632", "diff", True, 1, 6, (21, 32, 56), 128, 0.12),
    ]


def draw(rng):
    while True:
        tile = rng.choice([(0, 0, 0)] * 5 + [(2, 4, 8), (4, 4, 4), (1, 4, 16)])
        pt, ph, pw = tile if tile[0] else (1, 8, 8)
        T = pt * max(1, round(math.exp(rng.uniform(0, math.log(24.5))) / pt))
        Hh, Ww = ph * rng.randint(1, 48 // ph), pw * rng.randint(1, 80 // pw)
        B, H = rng.choice([1, 1, 1, 2, 3]), rng.randint(1, 12)
        S = T * Hh * Ww
        train = rng.random() < 0.5
        keep = round(math.exp(rng.uniform(math.log(0.05), 0)), 2)
        nb = S // N
        cost = B * H * S * S
        if 1 <= nb and cost <= 6 * 37632 ** 2 and rng.random() < min(1.0, nb / 8):
            c = _case("", rng.choice(["bias", "diff"]), train, B, H, (T, Hh, Ww), rng.choice([64, 128, 128]),
                      keep, rng.choice([0, 0, min(2, nb - 1)]), tile)
            del c["name"]
            return c


# ---------------------------------------------------------------------------- inputs

def _tile(c):
    return (c["pt"], c["ph"], c["pw"]) if c["pt"] else (1, 8, 8)


def _sizes(c):
    S = c["T"] * c["Hh"] * c["Ww"]
    return S, S // N, max(1, round(c["keep"] * (S // N)))


def _positions(c, device):
    p = torch.arange(c["T"] * c["Hh"] * c["Ww"], device=device)
    return p // (c["Hh"] * c["Ww"]), p // c["Ww"] % c["Hh"], p % c["Ww"]


def _block_of(c, device):
    """The block that each token lies in."""
    pt, ph, pw = _tile(c)
    t, h, w = _positions(c, device)
    return ((t // pt) * (c["Hh"] // ph) + h // ph) * (c["Ww"] // pw) + w // pw


def _bucket_map(n, half, far):
    """Bucket of each offset -(n-1) .. n-1 along an axis: one a step up to half / 2, then spaced by the logarithm up
    to `far`, the two signs apart (2 * half buckets)."""
    exact, m = max(1, half // 2), []
    for off in range(-(n - 1), n):
        a = abs(off)
        b = a if a < exact else min(half - 1, exact + int(math.log(a / exact) / math.log(far / exact) * (half - exact)))
        m.append(b + (half if off > 0 else 0))
    return m


_HALF, _FAR = (8, 12, 12), (32, 64, 64)  # buckets of one sign and the farthest distance told apart, per axis
_BUCKETS = 2 * sum(_HALF)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 17)
    S, nb, keep = _sizes(c)
    B, H, d = c["B"], c["H"], c["d"]

    def noise(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # activations: noise and a smooth field of the position that q and k share, so that attention is local in space
    t, h, w = _positions(c, dev)
    x = torch.stack([t / c["T"], h / c["Hh"], w / c["Ww"]], 1)
    basis = torch.cos(2 * math.pi * (x @ (1.5 * noise(3, 16))) + 6.2831853 * torch.rand(16, generator=gen, device=dev))
    field = 2.0 * math.sqrt(2 * 0.265 / 16) * torch.einsum("sf,bhfd->bhsd", basis, noise(B, H, 16, d))
    q = (noise(B, H, S, d) + field).bfloat16()
    k = (noise(B, H, S, d) + field).bfloat16()
    del field
    v = noise(B, H, S, d).bfloat16()
    s = {"case": dict(c), "q": q, "k": k, "v": v}
    if c["train"]:
        s["dout"] = noise(B, H, S, d).bfloat16()

    # the block mask: the best `keep` k-blocks of each row of the pooled map, some rows emptied
    at = torch.argsort(_block_of(c, dev), stable=True)
    qb, kb = (z.float()[:, :, at].view(B * H, nb, N, d).mean(2) for z in (q, k))
    best = (qb @ kb.transpose(1, 2)).topk(keep, dim=2).indices
    mask = torch.zeros(B * H, nb, nb, dtype=torch.bool, device=dev).scatter_(2, best, True)
    if c["empty"]:
        mask[:, torch.randperm(nb, generator=gen, device=dev)[: c["empty"]]] = False
    s["mask"] = mask

    if c["op"] == "bias":
        s["table"] = noise(H, _BUCKETS).bfloat16()
        buckets, base = [], 0
        for n, half, far in zip((c["T"], c["Hh"], c["Ww"]), _HALF, _FAR):
            buckets += [base + b for b in _bucket_map(n, half, far)]
            base += 2 * half
        s["buckets"] = torch.tensor(buckets, dtype=torch.int32, device=dev)
    else:
        s["lam"] = (0.2 + 0.6 * torch.rand(H, generator=gen, device=dev)).bfloat16()
    return s


# ---------------------------------------------------------------------------- the plain form, in 32 bits

def _chunks(BH, S, budget):
    """(heads, rows) of one chunk each: whole heads where they fit, else rows of one head."""
    if S * S <= budget:
        n = budget // (S * S)
        return [(slice(i, min(BH, i + n)), slice(0, S)) for i in range(0, BH, n)]
    n = max(1, budget // S)
    return [(slice(i, i + 1), slice(r, min(S, r + n))) for i in range(BH) for r in range(0, S, n)]


def _dropped(s, hs, rs, blk):
    """Where the block mask drops the key, for a chunk's rows."""
    return ~s["mask"][hs][:, blk[rs]][:, :, blk]


def _softmax(z, dropped):
    """Softmax over the kept keys; a row that keeps none is 0."""
    z = z.masked_fill_(dropped, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_(min=-3e38)
    z = z.sub_(top).exp_()
    return z.div_(z.sum(-1, keepdim=True).clamp_(min=1e-38))


def _axis_index(s, axis, rs):
    """Table index of each (row's coordinate, key's coordinate) along an axis: [rows, n]."""
    c = s["case"]
    n = (c["T"], c["Hh"], c["Ww"])
    base = sum(2 * m - 1 for m in n[:axis])
    coord = _positions(c, s["q"].device)[axis][rs]
    off = torch.arange(n[axis], device=coord.device)[None] - coord[:, None] + (n[axis] - 1)
    return s["buckets"][base + off].long()


def _plain_bias(s):
    c = s["case"]
    S, d, BH = _sizes(c)[0], c["d"], c["B"] * c["H"]
    dev, grid, scale = s["q"].device, (c["T"], c["Hh"], c["Ww"]), 1.0 / math.sqrt(c["d"])
    q, k, v = (s[n].float().view(BH, S, d) for n in ("q", "k", "v"))
    g = s["dout"].float().view(BH, S, d) if c["train"] else None
    table = s["table"].float().repeat(c["B"], 1)
    blk = _block_of(c, dev)
    out = torch.empty_like(q)
    if g is not None:
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dt = torch.zeros(BH, _BUCKETS, dtype=torch.float64, device=dev)  # long sums
    for hs, rs in _chunks(BH, S, _CHUNK):
        idx = [_axis_index(s, a, rs) for a in range(3)]
        z = (q[hs, rs] @ k[hs].transpose(1, 2)).mul_(scale)
        z5 = z.view(z.shape[0], z.shape[1], *grid)
        z5 += table[hs][:, idx[0]][:, :, :, None, None]
        z5 += table[hs][:, idx[1]][:, :, None, :, None]
        z5 += table[hs][:, idx[2]][:, :, None, None, :]
        p = _softmax(z, _dropped(s, hs, rs, blk))
        out[hs, rs] = p @ v[hs]
        if g is None:
            continue
        gr = g[hs, rs]
        dv[hs] += p.transpose(1, 2) @ gr
        ds = (gr @ v[hs].transpose(1, 2)).sub_((gr * out[hs, rs]).sum(-1, keepdim=True)).mul_(p)
        dq[hs, rs] = (ds @ k[hs]).mul_(scale)
        dk[hs] += (ds.transpose(1, 2) @ q[hs, rs]).mul_(scale)
        d5 = ds.view(ds.shape[0], ds.shape[1], *grid)
        for a, others in enumerate(((3, 4), (2, 4), (2, 3))):
            part = d5.sum(others).double().flatten(1)
            dt[hs] = dt[hs].index_add(1, idx[a].flatten(), part)
    shape = s["q"].shape
    if g is None:
        return {"out": out.bfloat16().view(shape)}
    return {"out": out.bfloat16().view(shape), "dq": dq.bfloat16().view(shape), "dk": dk.bfloat16().view(shape),
            "dv": dv.bfloat16().view(shape), "dtable": dt.view(c["B"], c["H"], _BUCKETS).sum(0).bfloat16()}


def _plain_diff(s):
    c = s["case"]
    S, d, BH = _sizes(c)[0], c["d"], c["B"] * c["H"]
    dev, e, scale = s["q"].device, c["d"] // 2, 1.0 / math.sqrt(c["d"] // 2)
    q, k, v = (s[n].float().view(BH, S, d) for n in ("q", "k", "v"))
    g = s["dout"].float().view(BH, S, d) if c["train"] else None
    lam = s["lam"].float().repeat(c["B"])[:, None, None]
    blk = _block_of(c, dev)
    out = torch.empty_like(q)
    if g is not None:
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dl = torch.zeros(BH, dtype=torch.float64, device=dev)  # long sums
    for hs, rs in _chunks(BH, S, _CHUNK):
        dropped = _dropped(s, hs, rs, blk)
        p1 = _softmax((q[hs, rs, :e] @ k[hs, :, :e].transpose(1, 2)).mul_(scale), dropped)
        p2 = _softmax((q[hs, rs, e:] @ k[hs, :, e:].transpose(1, 2)).mul_(scale), dropped)
        pd = p1 - lam[hs] * p2
        out[hs, rs] = pd @ v[hs]
        if g is None:
            continue
        gr = g[hs, rs]
        dv[hs] += pd.transpose(1, 2) @ gr
        dp = gr @ v[hs].transpose(1, 2)
        d1, d2 = (dp * p1).sum(-1, keepdim=True), (dp * p2).sum(-1, keepdim=True)
        dl[hs] -= d2.double().sum((1, 2))
        ds = p1.mul_(dp - d1)
        dq[hs, rs, :e] = (ds @ k[hs, :, :e]).mul_(scale)
        dk[hs, :, :e] += (ds.transpose(1, 2) @ q[hs, rs, :e]).mul_(scale)
        ds = p2.mul_(dp.sub_(d2)).mul_(-lam[hs])
        dq[hs, rs, e:] = (ds @ k[hs, :, e:]).mul_(scale)
        dk[hs, :, e:] += (ds.transpose(1, 2) @ q[hs, rs, e:]).mul_(scale)
    shape = s["q"].shape
    if g is None:
        return {"out": out.bfloat16().view(shape)}
    return {"out": out.bfloat16().view(shape), "dq": dq.bfloat16().view(shape), "dk": dk.bfloat16().view(shape),
            "dv": dv.bfloat16().view(shape), "dlam": dl.view(c["B"], c["H"]).sum(0).bfloat16()}


# ---------------------------------------------------------------------------- the framework's calls

def _own(s):
    from dynamic_block_sparse_fractal_b200 import api

    c = s["case"]
    desc = api.make_desc(c["B"], c["H"], c["T"], c["Hh"], c["Ww"], c["d"], 0.0,
                         tile=(c["pt"], c["ph"], c["pw"]) if c["pt"] else None)
    q, k, v = s["q"], s["k"], s["v"]
    ws = api.alloc_workspace(desc)
    api.plan_mask(desc, s["mask"], ws)
    if c["op"] == "bias":
        if not c["train"]:
            return {"out": api.fwd_bias(desc, q, k, v, s["table"], s["buckets"], ws)}
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        out = api.fwd_bias(desc, q, k, v, s["table"], s["buckets"], ws, lse=lse)
        dq, dk, dv, dt = api.bwd_bias(desc, q, k, v, s["table"], s["buckets"], out, s["dout"], lse, ws)
        return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dtable": dt}
    if not c["train"]:
        return {"out": api.fwd_diff(desc, q, k, v, s["lam"], ws)}
    lse = torch.empty((2,) + tuple(q.shape[:3]), dtype=torch.float32, device=q.device)
    out2 = torch.empty_like(q)
    out = api.fwd_diff(desc, q, k, v, s["lam"], ws, out2=out2, lse=lse)
    dq, dk, dv, dl = api.bwd_diff(desc, q, k, v, s["lam"], out, out2, s["dout"], lse, ws)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dlam": dl}


def run(state):
    if own:
        return _own(state)
    return _plain_bias(state) if state["case"]["op"] == "bias" else _plain_diff(state)


# ---------------------------------------------------------------------------- what a pass needs

def work(case):
    """Each input and output once; products of the kept blocks alone: 2 of the forward (a differential forward has one
    of scores and two with the values), 5 of the gradients."""
    c = case
    S, nb, keep = _sizes(c)
    rows = c["B"] * c["H"] * (nb - c["empty"])
    unit = 2.0 * N * N * c["d"] * rows * keep
    tensor = 2.0 * c["B"] * c["H"] * S * c["d"]
    return {"bytes": tensor * (8 if c["train"] else 4) + c["B"] * c["H"] * nb * nb,
            "flops": unit * ((2 if c["op"] == "bias" else 3) + (5 if c["train"] else 0))}


# ---------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    """Differentiated by torch, a few rows of queries at a time, over tokens in the order of their blocks."""
    s, c = prepare(case, seed), case
    S, nb, _ = _sizes(c)
    B, H, d, e = c["B"], c["H"], c["d"], c["d"] // 2
    dev = s["q"].device
    blk = _block_of(c, dev)
    order = torch.argsort(blk, stable=True)
    back = torch.argsort(order)
    pos = [p[order] for p in _positions(c, dev)]
    n = (c["T"], c["Hh"], c["Ww"])
    bucket, axes = s["buckets"].long() if c["op"] == "bias" else None, []
    if bucket is not None:
        axes = list(bucket.split([2 * m - 1 for m in n]))
    leaf = s["table"] if c["op"] == "bias" else s["lam"]
    names = ("q", "k", "v")
    res = {"out": torch.zeros(B, H, S, d, dtype=torch.float64, device=dev)}
    if c["train"]:
        res |= {"d" + m: torch.zeros_like(res["out"]) for m in names}
        dleaf = torch.zeros(leaf.shape, dtype=torch.float64, device=dev)
    rows = max(1, min(nb, (1 << 27) // (S * N))) * N
    for b in range(B):
        for h in range(H):
            x = [s[m][b, h, order].double().requires_grad_(c["train"]) for m in names]
            y = leaf[h].double().requires_grad_(c["train"])
            kept = s["mask"][b * H + h]
            for r in range(0, S, rows):
                at = slice(r, min(S, r + rows))
                ok = kept[r // N: (at.stop - 1) // N + 1].repeat_interleave(N, 0).repeat_interleave(N, 1)
                some = ok.any(1, keepdim=True)
                fill = torch.zeros(ok.shape, dtype=torch.float64, device=dev).masked_fill_(~ok & some, -math.inf)

                def weights(qq, kk, more=None):
                    z = qq @ kk.T / math.sqrt(qq.shape[1]) + fill
                    return torch.softmax(z if more is None else z + more, 1) * some

                q, k, v = x
                if c["op"] == "bias":
                    more = 0.0
                    for a in range(3):
                        near = y[axes[a][torch.arange(n[a], device=dev)[None] - pos[a][at][:, None] + n[a] - 1]]
                        more = more + near[:, pos[a]] if a else near[:, pos[a]]
                    w = weights(q[at], k, more)
                else:
                    w = weights(q[at, :e], k[:, :e]) - y * weights(q[at, e:], k[:, e:])
                o = w @ v
                res["out"][b, h, order[at]] = o.detach()
                if c["train"]:
                    grads = torch.autograd.grad((o * s["dout"][b, h, order[at]].double()).sum(), x + [y])
                    for m, gx in zip(names, grads):
                        res["d" + m][b, h] += gx[back]
                    dleaf[h] += grads[3]
    if c["train"]:
        res["dtable" if c["op"] == "bias" else "dlam"] = dleaf
    return res
