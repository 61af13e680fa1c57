"""AdaptedLinear on streams of its own, on stored codes of either width, and
its refusals."""
import types

import numpy as np
import pytest
import torch

import post_weight_quantization_25_b200 as G
from oracle import lora_oracle as LO

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def linear(rows, n, T, S=3, r=8, bits=4, group=64, seed=0, **kw):
    """(layer, x, plan, ids, adapters' tensors on the CPU) of random stored codes."""
    g = gen(seed)
    codes = torch.randint(0, 2 ** bits, (rows, n), generator=g, dtype=torch.uint8).cuda()
    packed = (G.gptq_pack_int4 if bits == 4 else G.gptq_pack_int3)(codes)
    G_ = (n + group - 1) // group
    scales = (torch.rand(rows, G_, generator=g) * 0.02 + 0.01).cuda()
    zeros = torch.randint(0, 2 ** bits, (rows, G_), generator=g, dtype=torch.uint8).cuda()
    A = (torch.randn(S, r, n, generator=g) * n ** -0.5).to(BF)
    B = (torch.randn(S, rows, r, generator=g) * 0.3).to(BF)
    ad = G.LowRankAdapters(A.cuda(), B.cuda())
    x = torch.randn(T, n, generator=g).to(BF).cuda()
    ids = torch.randint(-1, S, (T,), generator=g, dtype=torch.int32)
    lin = G.AdaptedLinear(packed, bits, n, scales, zeros, group, ad, **kw)
    return lin, x, G.gptq_lora_plan(ids.cuda(), S), ids, A, B


def test_matvec_on_another_stream_uses_memory_of_that_stream():
    """Memory that the current stream has freed but still writes must not become
    the result or the scratch of a call on another stream."""
    T, rows, n = 64, 8192, 512
    lin, x, plan, *_ = linear(rows, n, T)
    want = lin.matvec(x, plan)
    s = torch.cuda.Stream()
    lin.matvec(x, plan, stream=s)                # the modules are loaded
    torch.cuda.synchronize()
    need = G.gptq_workspace_size(G.GPTQ_OP_DEQUANT_MATVEC, T, n)
    torch.cuda.empty_cache()
    y_sized = torch.empty(T, rows, device="cuda")
    ws_sized = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(1000)
    y_sized.fill_(float("nan"))                  # (these kernels are loaded, too)
    ws_sized.fill_(0xFF)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)               # about 0.1 s of the current stream
    y_sized.fill_(float("nan"))
    ws_sized.fill_(0xFF)
    del y_sized, ws_sized
    y = lin.matvec(x, plan, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_matvec_refuses_before_it_enqueues():
    lin, x, plan, *_ = linear(192, 256, 5)
    torch.cuda.synchronize()
    other = types.SimpleNamespace(device=torch.device("cuda", torch.cuda.device_count()),
                                  cuda_stream=0)
    before = G.gptq_launch_count()
    for xx, pl, kw in ((x, plan, dict(stream=other)), (x[0], plan, {}), (x.cpu(), plan, {}),
                       (x[:4], plan, {}), (x, (plan[0][:3], plan[1]), {})):
        with pytest.raises(G.GptqError):
            lin.matvec(xx, pl, **kw)
    assert G.gptq_launch_count() == before


def test_training_leaves_no_graph_of_the_base_product_alone():
    """y's own graph would not know of the adapters: a backward pass through it
    would give dx without their part."""
    lin, x, plan, *_ = linear(192, 256, 40)
    y, saved = lin.forward(x.clone().requires_grad_(), plan)
    assert not y.requires_grad
    dx, *_ = lin.backward(y.clone().requires_grad_(), plan, saved)
    assert not dx.requires_grad


@pytest.mark.parametrize("bits,perm", [(3, False), (4, False), (3, True), (4, True)])
@pytest.mark.parametrize("act_group", [None, -1, 64, 128])
def test_both_widths_serve_and_train(bits, perm, act_group):
    """Random stored codes of 3 and 4 bits, in their own and in sweep order."""
    rows, n, T, r = 136, 320, 37, 8
    kw = {}
    if perm:
        kw["perm"] = torch.randperm(n, generator=gen(5)).to(torch.int32).cuda()
    lin, x, plan, ids, A, B = linear(rows, n, T, r=r, bits=bits, seed=bits, act_group=act_group,
                                     **kw)
    # column k of the codes multiplies x[perm[k]]
    W = f64(G.gptq_dequant(lin.packed, bits, n, lin.scales, lin.zeros, 64))
    if perm:
        Wo = np.empty_like(W)
        Wo[:, kw["perm"].cpu().numpy()] = W
        W = Wo
    assert np.array_equal(f64(lin.weight(F32)), W)
    xs, ids, A, B = f64(x), ids.numpy(), f64(A), f64(B)
    base, bmag = xs @ W.T, np.abs(xs) @ np.abs(W).T
    want, u, _, dmag = LO.apply(xs, A, B, ids, None, None, base)
    # products exact in fp32, sums of n (and n, then r) terms: at most n + r + 8
    # roundings or truncations of 2^-23 of the magnitude
    c = lambda k: (k + 8) * 2.0 ** -23  # noqa: E731
    assert np.all(np.abs(f64(lin.matvec(x, plan)) - want) <= c(n) * bmag + c(n + r) * dmag)
    y, saved = lin.forward(x, plan)
    # bf16 weights, base product and sum: half a step of 2^-8 each
    room = 1.01 * 2.0 ** -8 * (bmag + 2 * np.abs(base) + np.abs(want)) \
        + c(n) * bmag + (2.0 ** -17 + c(n + r)) * dmag
    assert np.all(np.abs(f64(y) - want) <= room)
    g = gen(9)
    dyc = torch.randn(T, rows, generator=g).to(BF)
    dy, dx_base = f64(dyc), f64(dyc) @ W
    dx, dA, dB = lin.backward(dyc.cuda(), plan, saved)
    xo = xs if act_group is None else LO.dequant_act8(
        *LO.quantize_act8(xs, act_group), act_group).astype(np.float64)
    us = np.where((ids >= 0)[:, None], f64(saved["u"]), 0.0)
    o = LO.backward(dy, us, xo, A, B, ids, None, None, dx_base)
    room = 1.01 * 2.0 ** -8 * (np.abs(dy) @ np.abs(W) + 2 * np.abs(dx_base) + np.abs(o["dx"])) \
        + c(rows) * (np.abs(dy) @ np.abs(W)) + (2.0 ** -17 + c(rows + r)) * o["mdx"]
    assert np.all(np.abs(f64(dx) - o["dx"]) <= room)
    assert np.all(np.abs(f64(dA) - o["dA"]) <= (c(rows + T) + 2.0 ** -24) * o["mdA"])
    assert np.all(np.abs(f64(dB) - o["dB"]) <= c(T) * o["mdB"])


def test_what_cannot_serve_is_refused_when_it_is_made():
    lin, *_ = linear(64, 256, 5)
    good = dict(packed=lin.packed, bits=4, n=256, scales=lin.scales, zeros=lin.zeros,
                group_size=64, adapters=lin.adapters)
    G.AdaptedLinear(**good)
    g_idx = torch.zeros(256, dtype=torch.int32, device="cuda")
    G.AdaptedLinear(**good, g_idx=g_idx)
    for bad in (dict(act_group=48), dict(act_group=0), dict(act_group=-2), dict(bits=3),
                dict(packed=lin.packed.cpu()), dict(packed=lin.packed[:, :8]),
                dict(packed=lin.packed.to(torch.int64)), dict(scales=lin.scales[:63]),
                dict(scales=lin.scales[:, :3].contiguous()), dict(scales=None),
                dict(scales=lin.scales.double()), dict(zeros=lin.zeros[:, :2]),
                dict(zeros=None), dict(zeros=lin.zeros.int()), dict(group_size=32),
                dict(g_idx=g_idx[:128]), dict(g_idx=g_idx.long()), dict(perm=g_idx.cpu()),
                dict(perm=g_idx, g_idx=g_idx)):
        with pytest.raises(G.GptqError):
            G.AdaptedLinear(**{**good, **bad})


@pytest.mark.parametrize("perm", [False, True])
def test_captured_calls_follow_their_inputs(perm):
    """Serving and a training step in one graph, replayed with other inputs and
    adapters, give what the eager calls give."""
    kw = {}
    if perm:
        kw["perm"] = torch.randperm(256, generator=gen(5)).to(torch.int32).cuda()
    lin, x, _, ids, A, B = linear(192, 256, 40, seed=3, **kw)
    ids, dy = ids.cuda(), torch.randn(40, 192, generator=gen(8)).to(BF).cuda()

    def step():
        plan = G.gptq_lora_plan(ids, 3)
        served = lin.matvec(x, plan)
        y, saved = lin.forward(x, plan)
        return (served, y, *lin.backward(dy, plan, saved))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for k in range(3):
        ids.copy_(torch.randint(-1, 3, (40,), generator=gen(k), dtype=torch.int32))
        x.copy_(torch.randn(40, 256, generator=gen(20 + k)))
        lin.adapters.A.copy_(torch.randn(lin.adapters.A.shape, generator=gen(40 + k)) / 16)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_no_tokens():
    lin, x, *_ = linear(192, 256, 4)
    plan = G.gptq_lora_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert lin.matvec(x[:0], plan).shape == (0, 192)
    y, saved = lin.forward(x[:0], plan)
    dx, dA, dB = lin.backward(y, plan, saved)
    assert y.shape == (0, 192) and dx.shape == (0, 256) and not dA.any() and not dB.any()
