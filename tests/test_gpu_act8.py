"""Activations in 8 bits on the GPU against the fp64 oracle.  Scales and codes
have to be equal: the scale is one correctly rounded division, and a code is
decided on the exact quotient, ties to even."""
import numpy as np
import pytest
import torch

import post_weight_quantization_25_b200 as G
from oracle import lora_oracle as LO

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(x, group, codes=None, scales=None):
    q, s = G.gptq_quantize_act8(x, group, codes=codes, scales=scales)
    wq, ws = LO.quantize_act8(x.cpu().double().numpy(), group)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), wq), np.argwhere(q.cpu().numpy() != wq)[:4]
    for dt in (F32, BF):
        xh = G.gptq_dequant_act8(q, s, group, out_dtype=dt)
        want = torch.from_numpy(LO.dequant_act8(wq, ws, group)).to(dt)
        assert torch.equal(xh.cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))
    return q, s


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group", [-1, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 31), (17, 32), (5, 100), (40, 128), (9, 1000),
                                    (33, 4096), (2, 28672), (130, 515), (4, 4097), (7, 2056)])
def test_codes_and_scales_equal_the_oracle(rows, n, group, dt):
    g = torch.Generator().manual_seed(rows * n)
    x = torch.randn(rows, n, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1),
                                                                     generator=g).float())
    check(x.to(dt).cuda(), group)


@pytest.mark.parametrize("group", [-1, 32, 128])
def test_ties_go_to_even(group):
    """The largest value 127 makes the scale 1: every half is a tie."""
    x = torch.arange(-254, 255, dtype=F32) / 2
    x = torch.cat([x, x.flip(0)])[None, :].repeat(3, 1)
    pad = (-x.shape[1]) % 32
    x = torch.nn.functional.pad(x, (0, pad))
    x[:, ::32] = 127.0
    check(x.cuda(), group)
    check((x * 2.0 ** -40).cuda(), group)


def test_quotients_next_to_a_tie():
    """fp32 values whose quotient lies next to k + 1/2, where an fp32 division
    would round onto the tie."""
    g = torch.Generator().manual_seed(4)
    amax = (torch.rand(200, 1, generator=g) + 1).double()
    sc = (amax.float().double() / 127).float().double()
    k = torch.randint(0, 126, (200, 255), generator=g).double() + 0.5
    x = (k * sc).float()
    step = torch.randint(-2, 3, x.shape, generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + step).view(F32)
    x = torch.cat([amax.float(), torch.where(torch.rand(x.shape, generator=g) < 0.5, -x, x)], 1)
    check(x.cuda(), -1)
    check(x.cuda(), 32)


@pytest.mark.parametrize("dt", [BF, F32])
def test_zeros_subnormals_and_the_largest_values(dt):
    rows = [torch.zeros(256), torch.full((256,), 1e-45), torch.full((256,), -2.0 ** -126),
            torch.arange(256) * 2.0 ** -140, torch.full((256,), torch.finfo(dt).max),
            -torch.arange(256).float() * 1e36, torch.arange(256).float() * 2.0 ** -126]
    check(torch.stack([r.float() for r in rows]).to(dt).cuda(), 128)
    check(torch.stack([r.float() for r in rows]).to(dt).cuda(), -1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group", [-1, 32, 64, 128])
def test_groups_with_nan_or_infinity_are_nan(dt, group):
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(1))
    x[1, 5], x[2, 299], x[3, 64], x[4, 0], x[4, 1] = (float("nan"), float("inf"), float("-inf"),
                                                      float("inf"), float("-inf"))
    q, s = check(x.to(dt).cuda(), group)
    assert int(torch.isnan(s).any(dim=1).sum()) == 4


@pytest.mark.parametrize("pad,off", [(16, 0), (16, 16), (5, 0), (1, 3)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_wider_buffers(pad, off, dt):
    rows, n = 21, 384
    x = torch.randn(rows, n, generator=torch.Generator().manual_seed(2)).to(dt)
    xb = torch.full((rows, n + pad + off), float("nan"), dtype=dt, device="cuda")
    cb = torch.full((rows, n + pad + off), 77, dtype=torch.int8, device="cuda")
    xv, cv = xb[:, off:off + n], cb[:, off:off + n]
    xv.copy_(x)
    for group in (-1, 64, 128):
        check(xv, group, codes=cv)
        out = torch.full((rows, n + pad + off), 9.0, dtype=dt, device="cuda")
        s = G.gptq_quantize_act8(xv, group)[1]
        G.gptq_dequant_act8(cv, s, group, out=out[:, off:off + n])
        edge = torch.ones(n + pad + off, dtype=torch.bool)
        edge[off:off + n] = False
        assert torch.all(cb[:, edge.cuda()] == 77) and torch.all(out[:, edge.cuda()] == 9.0)


def test_no_rows_streams_and_graphs():
    q, s = G.gptq_quantize_act8(torch.empty(0, 64, device="cuda"), 32)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    assert G.gptq_dequant_act8(q, s, 32).shape == (0, 64)
    x = torch.randn(64, 512, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    q1, s1 = G.gptq_quantize_act8(x, 128, stream=st)
    xh = G.gptq_dequant_act8(q1, s1, 128, stream=st)
    st.synchronize()
    q0, s0 = G.gptq_quantize_act8(x, 128)
    assert torch.equal(q0, q1) and torch.equal(s0, s1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q2, s2 = G.gptq_quantize_act8(x, 128)
        xh2 = G.gptq_dequant_act8(q2, s2, 128)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(xh, xh2)
    x.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, G.gptq_quantize_act8(x, 128)[0])


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    E = G.GptqError
    for bad in [dict(x=x.half()), dict(x=x[0]), dict(x=x.cpu()), dict(x=x.t()),
                dict(group=0), dict(group=-2), dict(group=16), dict(group=96),
                dict(codes=torch.zeros(4, 64, dtype=torch.uint8, device="cuda")),
                dict(codes=torch.zeros(4, 63, dtype=torch.int8, device="cuda")),
                dict(scales=torch.zeros(4, 3, device="cuda"))]:
        k = {**dict(x=x, group=32, codes=None, scales=None), **bad}
        with pytest.raises(E):
            G.gptq_quantize_act8(k["x"], k["group"], codes=k["codes"], scales=k["scales"])
    q, s = G.gptq_quantize_act8(x, 32)
    for bad in [dict(q=q.float()), dict(s=s.double()), dict(s=s[:3]), dict(group=64),
                dict(out=torch.zeros(4, 64, dtype=torch.float16, device="cuda")),
                dict(out=torch.zeros(4, 60, device="cuda"))]:
        k = {**dict(q=q, s=s, group=32, out=None), **bad}
        with pytest.raises(E):
            G.gptq_dequant_act8(k["q"], k["s"], k["group"], out=k["out"])


@pytest.mark.parametrize("group", [32, 128, 384, -1])
def test_quotients_next_to_a_tie_of_the_smallest_scales(group):
    """Scales S 2^-149 with an odd S in [2^23, 2^24): half of one is no fp32
    value, so what lies next to k + 1/2 scales must not be taken for a tie."""
    g = torch.Generator().manual_seed(6)
    S = torch.randint(2 ** 22, 2 ** 23, (400, 1), generator=g).double() * 2 + 1
    k = torch.randint(0, 4, (400, 383), generator=g).double()
    off = torch.randint(-1, 3, k.shape, generator=g).double()
    x = k * S + torch.floor(S / 2) + off
    x = torch.where(torch.rand(x.shape, generator=g) < 0.5, -x, x)
    x[:, 31::32] = 127 * S                      # the largest of every group
    x = (torch.cat([127 * S, x], 1) * 2.0 ** -149).float()
    q, s = check(x.cuda(), group)
    assert torch.equal(s[:, 0].cpu().double() * 2.0 ** 149, S[:, 0])
