"""What the biased and the differential attention and the plan from a mask refuse
before anything is launched (CPU)."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_fractal_b200 import api

FAKE = ctypes.c_void_p(0x10000000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10000001)
BIG = ctypes.c_size_t(1 << 40)


def desc(**kw):
    return api.make_desc(**dict(dict(B=1, H=2, T=4, Hh=8, Ww=8, d=64, thr=0.0), **kw))


def rel(table=FAKE, bucket=FAKE, n=8):
    return api.SaRelBias(table, bucket, n)


def fwd_bias(d, r, q=FAKE, out=FAKE, lse=FAKE, ws=FAKE, size=BIG):
    return api.lib().sparse_attn_fwd_bias(ctypes.byref(d), r and ctypes.byref(r), q, FAKE, FAKE, ws,
                                          size, out, lse, None)


def bwd_bias(d, r, dt=FAKE, out=FAKE, scratch=FAKE, ssize=BIG, size=BIG):
    return api.lib().sparse_attn_bwd_bias(ctypes.byref(d), ctypes.byref(r), FAKE, FAKE, FAKE, out,
                                          FAKE, FAKE, FAKE, size, FAKE, FAKE, FAKE, dt, scratch,
                                          ssize, None)


def fwd_diff(d, lam=FAKE, out2=FAKE, lse=FAKE, size=BIG):
    return api.lib().sparse_attn_fwd_diff(ctypes.byref(d), lam, FAKE, FAKE, FAKE, FAKE, size, FAKE,
                                          out2, lse, None)


def bwd_diff(d, lam=FAKE, out2=FAKE, dl=FAKE, scratch=FAKE, ssize=BIG, size=BIG):
    return api.lib().sparse_attn_bwd_diff(ctypes.byref(d), lam, FAKE, FAKE, FAKE, FAKE, out2, FAKE,
                                          FAKE, FAKE, size, FAKE, FAKE, FAKE, dl, scratch, ssize,
                                          None)


def plan_mask(d, mask=FAKE, heads=2, ws=FAKE, size=BIG):
    return api.lib().sparse_attn_plan_mask(ctypes.byref(d), mask, heads, ws, size, None)


def test_plan_mask_refusals():
    assert plan_mask(desc(), mask=None) == api.SA_ERR_INVALID_ARG
    for heads in (0, -1, 3):
        assert plan_mask(desc(), heads=heads) == api.SA_ERR_INVALID_ARG
    assert plan_mask(desc(), ws=ODD) == api.SA_ERR_INVALID_ARG
    need = api.workspace_size(desc())
    assert plan_mask(desc(), size=need - 1) == api.SA_ERR_WORKSPACE
    assert plan_mask(desc(Hh=12)) == api.SA_ERR_UNSUPPORTED


def test_bias_refusals():
    d = desc()
    for r in (rel(table=None), rel(bucket=None), rel(table=ODD), rel(bucket=ctypes.c_void_p(0x10000002)),
              rel(n=0), rel(n=4097)):
        assert fwd_bias(d, r) == api.SA_ERR_INVALID_ARG
        assert bwd_bias(d, r) == api.SA_ERR_INVALID_ARG
    assert fwd_bias(d, None) == api.SA_ERR_INVALID_ARG
    assert fwd_bias(d, rel(), q=ODD) == api.SA_ERR_INVALID_ARG
    assert fwd_bias(d, rel(), out=None) == api.SA_ERR_INVALID_ARG
    assert fwd_bias(d, rel(), lse=ODD) == api.SA_ERR_INVALID_ARG
    assert fwd_bias(d, rel(), size=api.workspace_size(d) - 1) == api.SA_ERR_WORKSPACE
    assert bwd_bias(d, rel(), dt=None) == api.SA_ERR_INVALID_ARG
    assert bwd_bias(d, rel(), dt=ctypes.c_void_p(0x10000002)) == api.SA_ERR_INVALID_ARG
    assert bwd_bias(d, rel(), out=None) == api.SA_ERR_INVALID_ARG
    assert bwd_bias(d, rel(), scratch=ctypes.c_void_p(0x10000010)) == api.SA_ERR_INVALID_ARG
    n = ctypes.c_size_t(0)
    assert api.lib().sparse_attn_bwd_bias_scratch_size(ctypes.byref(d), ctypes.byref(n)) == api.SA_OK
    assert bwd_bias(d, rel(), ssize=n.value - 1) == api.SA_ERR_WORKSPACE
    # the offset tables' limit: T + Hh + Ww <= 512
    long = desc(T=500)
    assert fwd_bias(long, rel()) == api.SA_ERR_UNSUPPORTED
    assert bwd_bias(long, rel()) == api.SA_ERR_UNSUPPORTED


def test_diff_refusals():
    d = desc()
    assert fwd_diff(d, lam=None) == api.SA_ERR_INVALID_ARG
    assert fwd_diff(d, lam=ODD) == api.SA_ERR_INVALID_ARG
    assert fwd_diff(d, out2=ODD) == api.SA_ERR_INVALID_ARG
    assert fwd_diff(d, lse=ODD) == api.SA_ERR_INVALID_ARG
    assert fwd_diff(d, size=16) == api.SA_ERR_WORKSPACE
    assert bwd_diff(d, lam=None) == api.SA_ERR_INVALID_ARG
    assert bwd_diff(d, out2=None) == api.SA_ERR_INVALID_ARG
    assert bwd_diff(d, dl=None) == api.SA_ERR_INVALID_ARG
    n = ctypes.c_size_t(0)
    assert api.lib().sparse_attn_bwd_diff_scratch_size(ctypes.byref(d), ctypes.byref(n)) == api.SA_OK
    assert bwd_diff(d, ssize=n.value - 1) == api.SA_ERR_WORKSPACE
    assert fwd_diff(desc(d=32)) == api.SA_ERR_UNSUPPORTED


def test_binding_refuses_other_tensors():
    d = desc()
    cpu = torch.zeros(1, 2, 256, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.plan_mask(d, torch.ones(2, 4, 4, dtype=torch.bool), cpu)
    with pytest.raises(ValueError):
        api.fwd_bias(d, cpu, cpu, cpu, torch.zeros(2, 8, dtype=torch.bfloat16),
                     torch.zeros(37, dtype=torch.int32), cpu)
    with pytest.raises(ValueError):
        api.fwd_diff(d, cpu, cpu, cpu, torch.zeros(2, dtype=torch.bfloat16), cpu)
