"""Host-side argument checks of the adapter and 8-bit activation entry points
(no GPU needed, no kernel launched), and the oracle's own consistency."""
import ctypes
import os

import numpy as np
import pytest

from oracle import lora_oracle as LO
from post_weight_quantization_25_b200 import _lib

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
OK, INVAL, UNSUP, WSMALL = 0, 1, 2, 3
BF, F = _lib.GPTQ_BF16, _lib.GPTQ_F32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from post_weight_quantization_25_b200 import build
        build.build()
    return _lib.load()


def lora(**kw):
    d = dict(A=0x10000, B=0x10000, wt=BF, n_slots=2, max_rank=16, n=64, rows=48, lda=64,
             stride_a=1024, ldb=16, stride_b=768, ranks=None, scales=None)
    d.update(kw)
    return _lib.GptqLora(*[d[f[0]] for f in _lib.GptqLora._fields_])


BAD_SETS = [(dict(wt=2), INVAL), (dict(n_slots=-1), INVAL), (dict(n_slots=65537), INVAL),
            (dict(max_rank=0), INVAL), (dict(max_rank=257, ldb=257), UNSUP), (dict(n=0), INVAL),
            (dict(n=57345), INVAL), (dict(rows=0), INVAL), (dict(lda=63), INVAL),
            (dict(ldb=15), INVAL), (dict(stride_a=-1), INVAL), (dict(A=None), INVAL),
            (dict(B=None), INVAL), (dict(A=0x10001), INVAL), (dict(B=0x10002, wt=F), INVAL),
            (dict(ranks=0x10002), INVAL), (dict(scales=0x10001), INVAL)]


def apply_args(ad, **kw):
    d = dict(order=P, start=P, ntok=8, x=P, xt=BF, ldx=64, y=P, yt=F, ldy=48, u=None, ldu=0,
             ws=P, wsb=1 << 20)
    d.update(kw)
    return (ctypes.byref(ad), d["order"], d["start"], d["ntok"], d["x"], d["xt"], d["ldx"],
            d["y"], d["yt"], d["ldy"], d["u"], d["ldu"], d["ws"], d["wsb"], None)


def backward_args(ad, **kw):
    d = dict(order=P, start=P, ntok=8, dy=P, dyt=BF, lddy=48, x=P, xt=BF, ldx=64, codes=None,
             cs=None, cg=128, u=P, ldu=16, dx=P, dxt=F, lddx=64, dA=P, dB=P, ws=P, wsb=1 << 24)
    d.update(kw)
    return (ctypes.byref(ad), d["order"], d["start"], d["ntok"], d["dy"], d["dyt"], d["lddy"],
            d["x"], d["xt"], d["ldx"], d["codes"], d["cs"], d["cg"], d["u"], d["ldu"], d["dx"],
            d["dxt"], d["lddx"], d["dA"], d["dB"], d["ws"], d["wsb"], None)


@pytest.mark.parametrize("kw,status", BAD_SETS)
def test_bad_adapter_sets_are_refused(lib, kw, status):
    assert lib.gptq_lora_apply(*apply_args(lora(**kw))) == status
    assert lib.gptq_lora_backward(*backward_args(lora(**kw))) == status


@pytest.mark.parametrize("kw,status", [
    (dict(order=None), INVAL), (dict(start=None), INVAL), (dict(order=ODD), INVAL),
    (dict(ntok=-1), INVAL), (dict(ntok=(1 << 24) + 1), INVAL), (dict(x=None), INVAL),
    (dict(y=None), INVAL), (dict(x=ODD), INVAL), (dict(y=ctypes.c_void_p(0x10002)), INVAL),
    (dict(xt=2), INVAL), (dict(yt=-1), INVAL), (dict(ldx=63), INVAL), (dict(ldy=47), INVAL),
    (dict(u=P, ldu=15), INVAL), (dict(u=ODD, ldu=16), INVAL), (dict(ntok=1 << 24, ws=None), WSMALL),
    (dict(ntok=1 << 24, wsb=8), WSMALL), (dict(ntok=1 << 24, ws=ctypes.c_void_p(0x10010), wsb=1 << 32), INVAL)])
def test_apply_refusals(lib, kw, status):
    assert lib.gptq_lora_apply(*apply_args(lora(), **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(order=None), INVAL), (dict(start=None), INVAL), (dict(ntok=-1), INVAL),
    (dict(dy=None), INVAL), (dict(dyt=3), INVAL), (dict(lddy=47), INVAL), (dict(dy=ODD), INVAL),
    (dict(x=None), INVAL), (dict(codes=P, cs=P), INVAL), (dict(xt=5), INVAL),
    (dict(ldx=60), INVAL), (dict(x=ODD), INVAL), (dict(x=None, codes=P), INVAL),
    (dict(x=None, codes=P, cs=ODD), INVAL), (dict(x=None, codes=P, cs=P, cg=0), INVAL),
    (dict(x=None, codes=P, cs=P, cg=48), UNSUP), (dict(u=None), INVAL), (dict(ldu=15), INVAL),
    (dict(u=ODD), INVAL), (dict(dxt=7), INVAL), (dict(lddx=63), INVAL), (dict(dx=ODD), INVAL),
    (dict(dA=ODD), INVAL), (dict(dB=ODD), INVAL), (dict(ws=None), WSMALL), (dict(wsb=8), WSMALL),
    (dict(ws=ctypes.c_void_p(0x10080)), INVAL)])
def test_backward_refusals(lib, kw, status):
    assert lib.gptq_lora_backward(*backward_args(lora(), **kw)) == status


def test_calls_with_nothing_to_do(lib):
    none = dict(order=None, start=None, ws=None, wsb=0)
    assert lib.gptq_lora_apply(*apply_args(lora(), ntok=0, x=None, y=None, **none)) == OK
    empty = lora(n_slots=0, A=None, B=None)
    assert lib.gptq_lora_apply(*apply_args(empty, **none)) == OK
    assert lib.gptq_lora_backward(*backward_args(empty, dA=None, dB=None, **none)) == OK
    assert lib.gptq_lora_backward(*backward_args(lora(), dx=None, dA=None, dB=None, **none)) == OK


def test_plan_refusals(lib):
    f = lib.gptq_lora_plan
    assert f(P, -1, 2, P, P, None, None) == INVAL
    assert f(P, 4, -1, P, P, None, None) == INVAL
    assert f(P, 4, 65537, P, P, None, None) == INVAL
    assert f(P, (1 << 24) + 1, 2, P, P, None, None) == INVAL
    assert f(None, 4, 2, P, P, None, None) == INVAL
    assert f(P, 4, 2, None, P, None, None) == INVAL
    assert f(P, 4, 2, P, None, None, None) == INVAL
    assert f(ODD, 4, 2, P, P, None, None) == INVAL
    assert f(P, 4, 2, P, P, ODD, None) == INVAL


def test_workspace_sizes(lib):
    out = ctypes.c_size_t(7)
    f = lib.gptq_lora_workspace_size
    ad = lora()
    assert f(ctypes.byref(ad), 1 << 24, 0, ctypes.byref(out)) == OK
    assert out.value >= (1 << 24) * 16 * 4
    # few tokens keep u to themselves
    assert f(ctypes.byref(ad), 100, 0, ctypes.byref(out)) == OK and out.value == 0
    assert f(ctypes.byref(ad), 100, 1, ctypes.byref(out)) == OK
    assert out.value >= 100 * 16 * 4
    assert f(ctypes.byref(ad), 0, 1, ctypes.byref(out)) == OK
    assert f(ctypes.byref(ad), -1, 0, ctypes.byref(out)) == INVAL
    assert f(ctypes.byref(ad), 100, 0, None) == INVAL
    assert f(None, 100, 0, ctypes.byref(out)) == INVAL
    bad = lora(max_rank=300)
    assert f(ctypes.byref(bad), 100, 0, ctypes.byref(out)) == UNSUP


def test_act8_refusals(lib):
    q, d = lib.gptq_quantize_act8, lib.gptq_dequant_act8
    assert q(None, BF, 0, 64, 64, 32, None, 64, None, None) == OK
    assert d(None, 0, 64, 64, None, 32, None, BF, 64, None) == OK
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=ODD), dict(scales=ODD),
               dict(xt=2), dict(rows=-1), dict(n=0), dict(n=57345), dict(ldx=63), dict(ldc=63),
               dict(group=0), dict(group=-2)):
        k = {**dict(x=P, xt=BF, rows=4, n=64, ldx=64, group=32, codes=P, ldc=64, scales=P), **kw}
        assert q(k["x"], k["xt"], k["rows"], k["n"], k["ldx"], k["group"], k["codes"], k["ldc"],
                 k["scales"], None) == INVAL, kw
        assert d(k["codes"], k["rows"], k["n"], k["ldc"], k["scales"], k["group"], k["x"],
                 k["xt"], k["ldx"], None) == INVAL, kw
    assert q(P, BF, 4, 64, 64, 48, P, 64, P, None) == UNSUP
    assert d(P, 4, 64, 64, P, 192, P, BF, 64, None) == UNSUP


# ------------------------------------------------------------------ the oracle itself
def _problem():
    rng = np.random.default_rng(0)
    x, A, B = rng.normal(size=(9, 12)), rng.normal(size=(3, 4, 12)), rng.normal(size=(3, 7, 4))
    ids = np.array([0, 2, -1, 2, 0, 1, 5, 2, 0])
    return x, A, B, ids, np.array([4, 2, 3]), np.array([0.5, 2.0, 1.5]), rng


def test_oracle_apply_token_by_token():
    x, A, B, ids, ranks, scales, rng = _problem()
    y = rng.normal(size=(9, 7))
    out, u, _, _ = LO.apply(x, A, B, ids, ranks, scales, y)
    for t, a in enumerate(ids):
        if a < 0 or a >= 3:
            assert np.array_equal(out[t], y[t]) and np.isnan(u[t]).all()
            continue
        want = y[t] + scales[a] * (B[a][:, :ranks[a]] @ (A[a][:ranks[a]] @ x[t]))
        np.testing.assert_allclose(out[t], want, rtol=1e-12)


def test_oracle_gradients_against_differences():
    x, A, B, ids, ranks, scales, rng = _problem()
    dy, zero = rng.normal(size=(9, 7)), np.zeros((9, 7))
    loss = lambda x, A, B: float((LO.apply(x, A, B, ids, ranks, scales, zero)[0] * dy).sum())  # noqa: E731
    u = np.nan_to_num(LO.project(x, A, ids, ranks))
    o = LO.backward(dy, u, x, A, B, ids, ranks, scales, np.zeros_like(x))
    for k, name in enumerate(("dx", "dA", "dB")):
        p = [x, A, B]
        e = rng.normal(size=p[k].shape)
        hi, lo = list(p), list(p)
        hi[k], lo[k] = p[k] + 0.5 * e, p[k] - 0.5 * e
        np.testing.assert_allclose(loss(*hi) - loss(*lo), (o[name] * e).sum(), rtol=1e-10)


def test_oracle_act8_rounds_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 100)).astype(np.float32).astype(np.float64)
    for g in (-1, 32, 128):
        q, s = LO.quantize_act8(x, g)
        gs = 100 if g < 0 else g
        step = np.repeat(s, gs, axis=1)[:, :100].astype(np.float64)
        assert np.all(np.abs(q * step - x) <= 0.5 * step * (1 + 1e-7))
        assert np.abs(q).max() == 127
    # a mistake of one code is seen: the check above fails for it
    q2 = q.copy()
    q2[0, 0] += 1 if q2[0, 0] < 0 else -1
    assert not np.all(np.abs(q2 * step - x) <= 0.5 * step)


# ------------------------------------------------------------------ the binding's checks
def test_workspaces_of_another_device_or_without_memory_of_their_own_are_refused():
    import torch

    import post_weight_quantization_25_b200 as G
    cpu, gpu = torch.device("cpu"), torch.device("cuda", 0)
    ws = torch.zeros(1000, dtype=torch.uint8)
    assert G._workspace(1000, cpu, ws) is ws
    assert G._workspace(0, gpu, None) is None
    with pytest.raises(G.GptqError, match="workspace"):
        G._workspace(1000, gpu, ws)
    with pytest.raises(G.GptqError, match="workspace"):
        G._workspace(1000, cpu, ws[:1].expand(1000))
    with pytest.raises(G.GptqError, match="workspace"):
        G._workspace(500, cpu, ws[::2])


@pytest.mark.parametrize("kw", [dict(stride_a=0), dict(stride_a=1023), dict(stride_b=0),
                                dict(stride_b=767), dict(lda=65), dict(ldb=17),
                                dict(stride_a=64, lda=128), dict(stride_b=16, ldb=32)])
def test_slots_that_overlap_or_interleave_are_refused(lib, kw):
    big = dict(ntok=1 << 20, ws=None, wsb=0)     # (what passes ends at the missing workspace)
    assert lib.gptq_lora_apply(*apply_args(lora(**kw), **big)) == INVAL
    assert lib.gptq_lora_backward(*backward_args(lora(**kw), **big)) == INVAL
    one = {**kw, "n_slots": 1}
    assert lib.gptq_lora_apply(*apply_args(lora(**one), **big)) == WSMALL
    assert lib.gptq_lora_backward(*backward_args(lora(**one), **big)) == WSMALL
    apart = {**kw, "stride_a": 1 << 14, "stride_b": 1 << 14}
    assert lib.gptq_lora_apply(*apply_args(lora(**apart), **big)) == WSMALL
    assert lib.gptq_lora_backward(*backward_args(lora(**apart), **big)) == WSMALL


def test_plans_that_would_hold_the_gpu_are_refused(lib):
    """Every slot reads all ids: 2^36 reads are the most."""
    f = lib.gptq_lora_plan
    assert f(P, 1 << 24, 65536, P, P, None, None) == UNSUP
    assert f(P, 1 << 24, 4097, P, P, None, None) == UNSUP
    assert f(P, (1 << 20) + 1, 65536, P, P, None, None) == UNSUP
    assert f(None, 1 << 24, 4096, P, P, None, None) == INVAL      # (not by the reads)
    assert f(None, 1 << 20, 65536, P, P, None, None) == INVAL
