"""How accurate the adapter products are, in two kinds of inputs that show what
general ones hide.

All of one sign.  Nothing cancels, so whatever is lost with a sign of its own
adds up: the matrix instructions cut their fp32 sums off, always towards zero,
and products of two fp32 values leave out what is below 2^-21 of them.  The
library's promise (include/gptq.h) is that such sums are off by less than 5e-7
of themselves on average over the outputs.  A single output is also off by the
roundings of its partial sums, at most 64 of them, each by at most 2^-24 of it
and evenly spread: a standard deviation of 8 2^-24 / sqrt(3), taken six times.

One product each.  A sum of one product and zeros is off by what is left out of
the product and by one cut: every fp32 value here has bits down to 2^-23, with
2^-16 among them, so a factor held in two bf16 parts instead of three would be
off by 2^-17.
"""
import pytest
import torch

import post_weight_quantization_25_b200 as G

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
BIAS = 5e-7
ONE = BIAS + 6 * 8 * 2.0 ** -24 / 3 ** 0.5
CUT = 2.0 ** -23


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def positive(g, shape, dt):
    return (torch.rand(shape, generator=g, device="cuda") + 0.5).to(dt)


def plan_of(T, S=1):
    return G.gptq_lora_plan((torch.arange(T, device="cuda") * S // T).to(torch.int32), S)


SAME_SIGN = [(T, n, m, r, xt, wt, None)
             for T, n, m, r in ((16, 4096, 4096, 16), (700, 4096, 2048, 40), (5000, 1024, 1024, 64),
                                (3000, 2048, 512, 128))
             for xt, wt in ((BF, BF), (F32, F32), (F32, BF), (BF, F32))]
SAME_SIGN += [(5000, 1001, 515, 16, BF, BF, None),        # rows that are not 16-byte aligned
              (19000, 16384, 64, 16, BF, BF, None),       # a CTA sums all of a long axis
              (19000, 64, 16384, 32, BF, BF, None),
              (2048, 28672, 9216, 16, BF, BF, None),      # a piece of 2048 tokens a CTA
              (2048, 28672, 9216, 16, BF, BF, 128),
              (5000, 1024, 512, 16, BF, BF, 32), (5000, 1024, 512, 40, BF, BF, 64),
              (5000, 1024, 512, 64, BF, BF, 128), (5000, 1024, 512, 16, F32, F32, -1),
              (300, 1024, 512, 16, BF, BF, 128)]


@pytest.mark.parametrize("T,n,m,r,xt,wt,group", SAME_SIGN)
def test_sums_of_one_sign(T, n, m, r, xt, wt, group):
    g = gen(T + n + r)
    x, dy = positive(g, (T, n), xt), positive(g, (T, m), xt)
    A, B = positive(g, (1, r, n), wt), positive(g, (1, m, r), wt)
    ad, plan = G.LowRankAdapters(A, B), plan_of(T)
    y, dx = torch.zeros(T, m, device="cuda"), torch.zeros(T, n, device="cuda")
    u = torch.empty(T, r, device="cuda")
    G.gptq_lora_apply(ad, plan, x, y, u=u)
    saved = dict(x=x)
    if group is not None:
        q, s = G.gptq_quantize_act8(x, group)
        saved = dict(codes=q, code_scales=s, group_size=group)
    _, dA, dB = G.gptq_lora_backward(ad, plan, dy, u, dx=dx, **saved)
    A, B = A[0].double(), B[0].double()

    def check(name, got, want):
        e = (got.double() - want) / want
        assert abs(float(e.mean())) < BIAS, (name, float(e.mean()))
        assert float(e.abs().max()) <= ONE, (name, float(e.abs().max()))

    t = torch.arange(0, T, max(1, T // 200), device="cuda")      # some tokens and columns
    cn = torch.arange(0, n, max(1, n // 500), device="cuda")
    cm = torch.arange(0, m, max(1, m // 500), device="cuda")
    check("u", u[t], x[t].double() @ A.t())
    check("y", y[t][:, cm], u[t].double() @ B[cm].t())
    check("dx", dx[t][:, cn], dy[t].double() @ B @ A[:, cn])
    v = torch.cat([p.double() @ B for p in dy.split(4096)])
    if group is None:
        xs = x[:, cn].double()
    else:
        gs = n if group < 0 else group
        xs = q[:, cn].double() * s[:, torch.div(cn, gs, rounding_mode="floor")].double()
    check("dA", dA[0][:, cn], v.t() @ xs)
    check("dB", dB[0][cm], dy[:, cm].double().t() @ u.double())


def long_values(g, shape, dt):
    """1 .. 2 and of either sign, with the bit of 2^-16 among 24 (bf16: 8)."""
    k = torch.randint(0, 2 ** 23, shape, generator=g, device="cuda") | 1 << 7
    v = 1 + k.double() * 2.0 ** -23
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, -v, v).to(dt)


ONE_PRODUCT = [(T, n, m, r, xt, wt, None)
               for T, n, m, r in ((30, 64, 48, 16), (1100, 1104, 1160, 40), (4700, 4704, 4704, 64),
                                  (1500, 1504, 1504, 128))
               for xt, wt in ((BF, BF), (F32, F32), (F32, BF), (BF, F32))]
ONE_PRODUCT += [(700, 701, 703, 16, BF, BF, None), (1100, 1104, 1160, 40, BF, BF, 32),
                (1100, 1104, 1160, 40, BF, BF, 128), (4700, 4704, 4704, 64, BF, BF, -1)]


@pytest.mark.parametrize("T,n,m,r,xt,wt,group", ONE_PRODUCT)
def test_sums_of_one_product(T, n, m, r, xt, wt, group):
    """Token t's x is zero but in a column of its own, and so is its dy: u, v, dA
    and dB are single products, y and dx sums over the ranks."""
    g = gen(T + n)
    cx = torch.randperm(n, generator=g, device="cuda")[:T]
    cy = torch.randperm(m, generator=g, device="cuda")[:T]
    t = torch.arange(T, device="cuda")
    x, dy = torch.zeros(T, n, dtype=xt, device="cuda"), torch.zeros(T, m, dtype=xt, device="cuda")
    x[t, cx], dy[t, cy] = long_values(g, (T,), xt), long_values(g, (T,), xt)
    A, B = long_values(g, (1, r, n), wt), long_values(g, (1, m, r), wt)
    sc = long_values(g, (1,), F32).abs()
    ad, plan = G.LowRankAdapters(A, B, None, sc), plan_of(T)
    y, dx = torch.zeros(T, m, device="cuda"), torch.zeros(T, n, device="cuda")
    u = torch.empty(T, r, device="cuda")
    G.gptq_lora_apply(ad, plan, x, y, u=u)
    saved, xv = dict(x=x), x[t, cx].double()
    if group is not None:
        q, s = G.gptq_quantize_act8(x, group)
        saved = dict(codes=q, code_scales=s, group_size=group)
        gs = n if group < 0 else group
        xv = q[t, cx].double() * s[t, torch.div(cx, gs, rounding_mode="floor")].double()
    _, dA, dB = G.gptq_lora_backward(ad, plan, dy, u, dx=dx, **saved)
    A, B, sc = A[0].double(), B[0].double(), float(sc)
    left_out = lambda a, b: 2.0 ** -21 if a == b == F32 else 0.0  # noqa: E731
    half = 2.0 ** -24
    # one cut of the whole, and smaller ones of the parts' sums below 2^-6 of it
    cut = (1 + 2.0 ** -5) * CUT
    bu = cut + left_out(xt, wt)
    bv = bu + half                                       # times the scale, rounded
    # (each bound a little more for the product of two errors)
    ok = lambda got, want, b: bool(  # noqa: E731
        (((got.double() - want).abs()) <= 1.001 * b * want.abs()).all())
    us = x[t, cx].double()[:, None] * A[:, cx].t()
    assert ok(u, us, bu)
    vs = sc * dy[t, cy].double()[:, None] * B[cy]
    want = torch.zeros(r, n, dtype=torch.float64, device="cuda")
    want[:, cx] = vs.t() * xv
    # (codes: v times the code's scale is rounded as well)
    bA = bv + cut + left_out(F32, xt) + (half if group is not None else 0)
    assert ok(dA[0], want, bA)
    want = torch.zeros(m, r, dtype=torch.float64, device="cuda")
    want[cy] = sc * dy[t, cy].double()[:, None] * u.double()
    assert ok(dB[0], want, half + cut + left_out(F32, xt))
    # sums over the ranks, cut or rounded once for every 16 of each part
    steps = (r + 15) // 16
    br = half + (steps + 1) * cut + left_out(F32, wt)
    k = t[:: max(1, T // 300)]
    for got, f, W, b in ((y, sc * u[k].double(), B.t(), br),
                         (dx, vs[k], A, br + bv)):
        mag = f.abs() @ W.abs()
        assert bool(((got[k].double() - f @ W).abs() <= 1.001 * (b + half) * mag).all())
