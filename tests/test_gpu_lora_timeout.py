"""The time limits inside the adapter kernels: a wait that runs out makes the
outputs concerned NaN, everything else stays as it was, and the context stays
usable.  gptq_set_wait_gate makes a copying thread first wait for a flag that
nothing sets, with a short limit and nothing in flight."""
import contextlib

import pytest
import torch

import post_weight_quantization_25_b200 as G

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LIMIT_NS = 2_000_000      # 2 ms


@contextlib.contextmanager
def gate(opened):
    flag = torch.full((1,), int(opened), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    G.gptq_set_wait_gate(flag, LIMIT_NS)
    try:
        yield
    finally:
        G.gptq_set_wait_gate(None)
        torch.cuda.synchronize()


def layer(T, n, m, S, r, runs=True, yt=F32, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, S, (T,), generator=g, dtype=torch.int32)
    ids = ids.sort().values if runs else ids
    ids[T // 2] = -1
    return dict(
        ids=ids.cuda(), plan=G.gptq_lora_plan(ids.cuda(), S),
        ad=G.LowRankAdapters(torch.randn(S, r, n, generator=g).to(BF).cuda(),
                             torch.randn(S, m, r, generator=g).to(BF).cuda()),
        x=torch.randn(T, n, generator=g).to(BF).cuda(), u=torch.randn(T, r, generator=g).cuda(),
        dy=torch.randn(T, m, generator=g).to(BF).cuda(),
        y=torch.randn(T, m, generator=g).to(yt).cuda(),
        dx=torch.randn(T, n, generator=g).to(yt).cuda())


def gradients(c, group):
    saved = dict(x=c["x"])
    if group is not None:
        q, s = G.gptq_quantize_act8(c["x"], group)
        saved = dict(codes=q, code_scales=s, group_size=group)
    _, dA, dB = G.gptq_lora_backward(c["ad"], c["plan"], c["dy"], c["u"], **saved)
    return dA, dB


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("runs", [True, False])
@pytest.mark.parametrize("T,group", [(300, None), (300, 128), (1300, 256)])
def test_gradients_from_codes_and_of_few_tokens(T, group, runs, r):
    """(the products of few bf16 tokens and of 8-bit codes share a kernel)"""
    c = layer(T, 384, 264, 2, r, runs)
    want = gradients(c, group)
    with gate(True):                     # open: nothing changes
        got = gradients(c, group)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with gate(False):
        got = gradients(c, group)
    assert all(torch.isnan(t).all() for t in got)
    got = gradients(c, group)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("runs,r", [(True, 16), (False, 16), (True, 64), (False, 32)])
def test_the_projection_down_to_the_rank(runs, r):
    """One CTA of each cluster meets the limit: all ranks of all the cluster's
    tokens are NaN, not what the others' sums alone come to."""
    T, n, m = 2400, 4096, 4096
    c = layer(T, n, m, 1, r, runs)
    assert c["ad"].workspace_size(T) > 0          # a kernel for each projection
    live = c["ids"] >= 0

    def both():
        u = torch.full((T, r), 5.0, device="cuda")
        y = c["y"].clone()
        G.gptq_lora_apply(c["ad"], c["plan"], c["x"], y, u=u)
        return u, y

    want = both()
    with gate(True):
        got = both()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with gate(False):
        u, y = both()
    assert torch.isnan(u[live]).all() and torch.isnan(y[live]).all()
    assert torch.equal(u[~live], want[0][~live]) and torch.equal(y[~live], c["y"][~live])
    assert all(torch.equal(a, b) for a, b in zip(both(), want))


@pytest.mark.parametrize("runs,r,yt", [(True, 16, F32), (False, 16, BF), (True, 64, BF),
                                       (False, 32, F32)])
def test_the_projection_back_from_the_rank(runs, r, yt):
    """(fp32 x with bf16 adapters: only this kernel of the call has a gate)"""
    T, n, m = 5000, 1024, 4096
    c = layer(T, n, m, 1, r, runs, yt)
    assert c["ad"].workspace_size(T) > 0
    x, live = c["x"].float(), c["ids"] >= 0

    def both():
        u = torch.full((T, r), 5.0, device="cuda")
        y = c["y"].clone()
        G.gptq_lora_apply(c["ad"], c["plan"], x, y, u=u)
        return u, y

    want = both()
    with gate(True):
        got = both()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with gate(False):
        u, y = both()
    assert torch.equal(u, want[0])
    assert torch.isnan(y[live]).all() and torch.equal(y[~live], c["y"][~live])
    assert all(torch.equal(a, b) for a, b in zip(both(), want))


@pytest.mark.parametrize("T", [1400, 5000])
@pytest.mark.parametrize("runs,r", [(True, 16), (False, 16), (True, 64), (False, 32)])
def test_gradients_of_many_tokens(runs, r, T):
    c = layer(T, 1040, 520, 2, r, runs)
    want = gradients(c, None)
    with gate(True):
        got = gradients(c, None)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with gate(False):
        got = gradients(c, None)
    assert all(torch.isnan(t).all() for t in got)
    # dx: v of the projection down to the rank where that has a gate, then its own
    with gate(False):
        dx = G.gptq_lora_backward(c["ad"], c["plan"], c["dy"], dx=c["dx"].clone(), want_dA=False,
                                  want_dB=False)[0]
    live = c["ids"] >= 0
    assert torch.equal(dx[~live], c["dx"][~live])
    if c["ad"].workspace_size(T) > 0:
        assert torch.isnan(dx[live]).all()
    got = gradients(c, None)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
