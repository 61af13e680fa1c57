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
