"""Random cases of the adapter products over their whole range: types, ranks,
slots, order of the tokens, groups of codes, NaN in everything that does not
count.  Each is run three times, twice with u kept and once without, and must
repeat bit for bit; values are held to the bounds of test_gpu_lora.py,

  c(K) = (K / 16 + 40) 2^-23 of the magnitude of a sum of K products,

with half a step of the result's type, and 2^-17 of u or v towards bf16.  All
in 64 bits on the GPU.
"""
import random

import pytest
import torch

import post_weight_quantization_25_b200 as G

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def c_of(K):
    return (K / 16 + 40) * 2.0 ** -23


def draw(r, g):
    T = int(round(2 ** r.uniform(0, 13)))
    n = r.choice([8, 16, 64, 77, 128, 256, 384, 520, 1000, 1001, 1376, 2048])
    m = r.choice([8, 24, 64, 128, 264, 512, 515, 1032, 2056])
    S = r.choice([1, 1, 1, 2, 3, 5, 8, 20])
    rk = r.choice([1, 4, 8, 8, 12, 16, 16, 20, 24, 32, 40, 64, 64, 72, 128, 200, 256])
    mode = r.choice(["sorted", "random", "runs"])
    if mode == "runs":
        L = r.randint(1, 200)
        ids = torch.randint(0, S, ((T + L - 1) // L,), generator=g, device="cuda")
        ids = ids.repeat_interleave(L)[:T]
    else:
        ids = torch.randint(0, S, (T,), generator=g, device="cuda")
        ids = ids.sort().values if mode == "sorted" else ids
    if r.random() < 0.4:
        gone = torch.rand(T, generator=g, device="cuda") < r.choice([0.05, 0.5])
        ids = torch.where(gone, -1, ids)
    ranks = torch.full((S,), rk, device="cuda", dtype=torch.int32)
    if r.random() < 0.5:
        ranks = torch.randint(0, rk + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    types = [r.choice([BF, BF, BF, F32]) for _ in range(3)] + [r.choice([BF, F32])]
    return T, n, m, S, rk, types, ids.int(), ranks, r.choice([None, None, -1, 32, 64, 128, 256])


def one_case(r, g):
    T, n, m, S, rk, (xt, dyt, wt, yt), ids, ranks, group = draw(r, g)
    what = (T, n, m, S, rk, xt, dyt, wt, yt, group)
    N = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, dy = N(T, n).to(xt), N(T, m).to(dyt)
    A, B = (N(S, rk, n) * n ** -0.5).to(wt), (N(S, m, rk) * 0.3).to(wt)
    sc = torch.rand(S, generator=g, device="cuda") + 0.5
    y0, dx0 = N(T, m).to(yt), N(T, n).to(yt)
    An, Bn, xn, dyn, idle = A.clone(), B.clone(), x.clone(), dy.clone(), ids < 0
    for a in range(S):
        An[a, int(ranks[a]):] = float("nan")
        Bn[a, :, int(ranks[a]):] = float("nan")
    xn[idle], dyn[idle] = float("nan"), float("nan")
    saved, xs = dict(x=xn), x.double()
    if group is not None:
        q, qs = G.gptq_quantize_act8(x, group)
        xs = q.double() * qs.double().repeat_interleave(n if group < 0 else group, 1)[:, :n]
        qs[idle] = float("nan")
        saved = dict(codes=q, code_scales=qs, group_size=group)
    ad, plan = G.LowRankAdapters(An, Bn, ranks, sc), G.gptq_lora_plan(ids, S)
    runs = []
    for k in range(3):
        y, dx, u = y0.clone(), dx0.clone(), torch.full((T, rk), 3.0, device="cuda")
        G.gptq_lora_apply(ad, plan, xn, y, u=u if k != 1 else None)
        u = runs[0][1].clone() if k == 1 else u
        _, dA, dB = G.gptq_lora_backward(ad, plan, dyn, u, dx=dx, **saved)
        runs.append((y, u, dx, dA, dB))
    for o in runs[1:]:
        assert all(torch.equal(p, q_) for p, q_ in zip(o, runs[0])), what
    y, u, dx, dA, dB = runs[0]
    assert torch.equal(y[idle], y0[idle]) and torch.equal(dx[idle], dx0[idle]), what
    assert bool((u[idle] == 3.0).all()), what
    half = 2.0 ** -8 if yt == BF else 2.0 ** -24
    parts = 2.0 ** -17 if yt == BF else 0.0

    def check(name, got, want, room):
        err = (got.double() - want).abs()
        assert bool((err <= room).all()), (name, float((err - room).max()), what)

    for a in range(S):
        k, t = int(ranks[a]), (ids == a).nonzero().flatten()
        assert not dA[a, k:].any() and not dB[a, :, k:].any(), what
        assert not u[t, k:].any(), what
        Ad, Bd, s = A[a, :k].double(), B[a, :, :k].double(), float(sc[a])
        xd, dyd, ud = x[t].double(), dy[t].double(), u[t, :k].double()
        check("u", u[t, :k], xd @ Ad.t(), c_of(n) * (xd.abs() @ Ad.abs().t()))
        join = (rk + 8) * 2.0 ** -23
        for name, got, old, f, fm, W, K in (
                ("y", y, y0, s * xd @ Ad.t(), s * xd.abs() @ Ad.abs().t(), Bd.t(), n),
                ("dx", dx, dx0, s * dyd @ Bd, s * dyd.abs() @ Bd.abs(), Ad, m)):
            want, room = old[t].double() + f @ W, (c_of(K) + join + parts) * (fm @ W.abs())
            check(name, got[t], want, room + half * (want.abs() + room))
        v, vm = s * dyd @ Bd, s * dyd.abs() @ Bd.abs()
        check("dA", dA[a, :k], v.t() @ xs[t],
              (c_of(m) + c_of(T) + 2.0 ** -24) * (vm.t() @ xs[t].abs()))
        check("dB", dB[a, :, :k], s * dyd.t() @ ud, c_of(T) * s * (dyd.abs().t() @ ud.abs()))


@pytest.mark.parametrize("seed", range(8))
def test_random_cases(seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for _ in range(60):
        one_case(r, g)
