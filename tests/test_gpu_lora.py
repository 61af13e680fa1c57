"""Low-rank adapters on the GPU against the fp64 oracle: the token plan, the
forward product, its gradients, and the training step of an adapted linear.

Error bounds.  Every product and sum is kept to fp32 accuracy, so with K terms
summed at least 16 at a time (one rounding or truncation of at most 2^-23 of
the running magnitude each) plus at most 40 levels of joining and splitting:

  u      <= c(K) |x||A|^T                     c(K) = (K / 16 + 40) 2^-23
  delta  <= (c(n) + (rank + 8) 2^-23) |s| |x||A|^T|B|^T
  dx     <= (c(rows) + (rank + 8) 2^-23) |s| |dy||B||A|
  dA     <= (c(rows) + c(ntok)) sum |v||x|,   dB <= c(ntok) sum |s dy||u|

and the result is rounded once to its type: half a step, 2^-24 of an fp32
value, 2^-8 of a bf16 value; towards a bf16 result the factors u and v may be
held in two bf16 parts, 2^-17 of the magnitude.
"""
import types

import numpy as np
import pytest
import torch

import post_weight_quantization_25_b200 as G
from oracle import gptq_oracle as O
from oracle import lora_oracle as LO

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


def c_of(K):
    return (K / 16 + 40) * 2.0 ** -23


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad, offset=0):
    """The same values on the GPU as rows of a wider buffer."""
    if pad == 0 and offset == 0:
        return t.cuda()
    rows, n = t.shape
    buf = torch.full((rows, n + pad + offset), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[:, offset:offset + n]
    view.copy_(t)
    return view


def ranks_of(S, rmax, mixed):
    if not mixed:
        return None
    kinds = [rmax, max(1, rmax // 2), 0, max(1, rmax - 1), 1]
    return np.array([kinds[a % 5] for a in range(S)], np.int32)


class Case:
    """Seeded inputs of one layer and its adapters, on the CPU and the GPU."""

    def __init__(self, T, n, m, S, rmax, xt=BF, wt=BF, yt=F32, mixed=False, idle=0.1, seed=0,
                 runs=False, pad=0, offset=0, scaled=True):
        g = gen(1000 + seed)
        self.T, self.n, self.m, self.S, self.rmax = T, n, m, S, rmax
        self.x = torch.randn(T, n, generator=g).to(xt)
        self.A = (torch.randn(S, rmax, n, generator=g) * n ** -0.5).to(wt)
        self.B = (torch.randn(S, m, rmax, generator=g) * 0.3).to(wt)
        self.y = torch.randn(T, m, generator=g).to(yt)
        self.dy = torch.randn(T, m, generator=g).to(xt)
        self.dx = torch.randn(T, n, generator=g).to(yt)
        self.ranks = ranks_of(S, rmax, mixed)
        self.scales = (torch.rand(S, generator=g) + 0.5) if scaled else None
        if runs:
            ids = torch.sort(torch.randint(0, S, (T,), generator=g)).values
            ids = ids.flip(0)
        else:
            ids = torch.randint(0, S, (T,), generator=g)
        ids[torch.rand(T, generator=g) < idle] = -1
        self.ids = ids.to(torch.int32)
        # entries that do not count hold NaN
        Ad, Bd = self.A.clone(), self.B.clone()
        if mixed:
            for a, r in enumerate(self.ranks):
                Ad[a, r:] = float("nan")
                Bd[a, :, r:] = float("nan")
        xd = self.x.clone()
        xd[self.ids < 0] = float("nan")
        self.gx = strided(xd, pad, offset)
        self.gy = strided(self.y, pad, offset)
        self.gdy = strided(self.dy, pad, offset)
        self.gdx = strided(self.dx, pad, offset)
        self.ad = G.LowRankAdapters(
            Ad.cuda(), Bd.cuda(),
            None if self.ranks is None else torch.from_numpy(self.ranks).cuda(),
            None if self.scales is None else self.scales.cuda())
        self.plan = G.gptq_lora_plan(self.ids.cuda(), S)

    def oracle_scales(self):
        return None if self.scales is None else f64(self.scales)

    def want_apply(self):
        return LO.apply(f64(self.x), f64(self.A), f64(self.B), self.ids.numpy(), self.ranks,
                        self.oracle_scales(), f64(self.y))

    def out_bound(self, exact, mag, K):
        b = (c_of(K) + (self.rmax + 8) * 2.0 ** -23) * mag
        if self.gy.dtype == BF:
            return b + 2.0 ** -17 * mag + 2.0 ** -8 * (np.abs(exact) + b)
        return b + 2.0 ** -24 * (np.abs(exact) + b)

    def check_apply(self, u_given=True):
        u = torch.full((self.T, self.rmax), 7.0, device="cuda") if u_given else None
        y0 = self.gy.clone()
        out = G.gptq_lora_apply(self.ad, self.plan, self.gx, self.gy, u=u)
        torch.cuda.synchronize()
        assert out is self.gy
        want, wu, umag, dmag = self.want_apply()
        got = f64(self.gy)
        err, bound = np.abs(got - want), self.out_bound(want, dmag, self.n)
        assert np.all(err <= bound), (float((err - bound).max()), np.argwhere(err > bound)[:4])
        idle = self.ids.numpy() < 0
        assert torch.equal(self.gy[torch.from_numpy(idle).cuda()], y0[torch.from_numpy(idle).cuda()])
        if u_given:
            gu = f64(u)
            assert np.all(gu[idle] == 7.0)
            live = ~idle
            assert np.all(np.abs(gu - wu)[live] <= (c_of(self.n) * umag)[live])
            return u
        return None

    def check_backward(self, group=None, want=("dx", "dA", "dB")):
        u = torch.from_numpy(np.nan_to_num(LO.project(
            f64(self.x), f64(self.A), self.ids.numpy(), self.ranks), nan=0.0)).float().cuda()
        uo = f64(u)
        u[self.ids.cuda() < 0] = float("nan")
        idle = (self.ids < 0).cuda()
        gdy = self.gdy.clone() if self.gdy.is_contiguous() else self.gdy
        gdy[idle] = float("nan")
        dx0 = self.gdx.clone()
        if group is None:
            xo, saved = f64(self.x), dict(x=self.gx)
        else:
            q, sc = LO.quantize_act8(f64(self.x), group)
            xo = LO.dequant_act8(q, sc, group).astype(np.float64)
            gq, gs = torch.from_numpy(q).cuda(), torch.from_numpy(sc).cuda()
            gq[idle], gs[idle] = 99, float("nan")
            saved = dict(codes=gq, code_scales=gs, group_size=group)
        if "dA" not in want:
            saved = {}
        dx, dA, dB = G.gptq_lora_backward(
            self.ad, self.plan, gdy, u if "dB" in want else None,
            dx=self.gdx if "dx" in want else None, want_dA="dA" in want, want_dB="dB" in want,
            **saved)
        torch.cuda.synchronize()
        o = LO.backward(f64(self.dy), uo, xo, f64(self.A), f64(self.B), self.ids.numpy(),
                        self.ranks, self.oracle_scales(), f64(self.dx))
        if "dx" in want:
            err, bound = np.abs(f64(dx) - o["dx"]), self.out_bound(o["dx"], o["mdx"], self.m)
            assert np.all(err <= bound), ("dx", float((err - bound).max()))
            assert torch.equal(dx[idle], dx0[idle])
        else:
            assert dx is None
        # (a code restored to fp32 was rounded once: 2^-24 of x)
        ca = c_of(self.m) + c_of(self.T) + 2.0 ** -24
        if "dA" in want:
            err = np.abs(f64(dA) - o["dA"])
            assert np.all(err <= ca * o["mdA"]), ("dA", float((err - ca * o["mdA"]).max()))
        else:
            assert dA is None
        if "dB" in want:
            err = np.abs(f64(dB) - o["dB"])
            assert np.all(err <= c_of(self.T) * o["mdB"]), ("dB", float(err.max()))
        else:
            assert dB is None


# ------------------------------------------------------------------ the plan
@pytest.mark.parametrize("T,S", [(1, 1), (5, 3), (31, 40), (1024, 7), (1025, 1), (5000, 64),
                                 (70001, 13), (2, 2000)])
def test_plan_sorts_tokens_by_slot(T, S):
    ids = torch.randint(-2, S, (T,), generator=gen(T + S), dtype=torch.int32)
    info = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    order, start = G.gptq_lora_plan(ids.cuda(), S, info=info)
    wo, ws = LO.plan(ids.numpy(), S)
    assert np.array_equal(order.cpu().numpy(), wo) and np.array_equal(start.cpu().numpy(), ws)
    assert int(info.item()) == 0


def test_plan_reports_ids_past_the_slots_and_takes_them_as_none():
    ids = torch.tensor([0, 3, 1, 2 ** 31 - 1, -2 ** 31, 2], dtype=torch.int32)
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    order, start = G.gptq_lora_plan(ids.cuda(), 3, info=info)
    wo, ws = LO.plan(ids.numpy(), 3)
    assert np.array_equal(order.cpu().numpy(), wo) and np.array_equal(start.cpu().numpy(), ws)
    assert int(info.item()) == 1


def test_plan_of_no_tokens_and_of_no_slots():
    order, start = G.gptq_lora_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 4)
    assert order.numel() == 0 and start.tolist() == [0] * 5
    ids = torch.tensor([-1, -1, 0], dtype=torch.int32, device="cuda")
    order, start = G.gptq_lora_plan(ids, 0)
    assert start.tolist() == [0] and order.tolist() == [0, 1, 2]


# ------------------------------------------------------------------ forward
APPLY = [
    # T, n, m, slots, max_rank, xt, wt, yt, mixed
    (1, 512, 512, 1, 16, BF, BF, F32, False),
    (1, 40, 24, 1, 1, BF, BF, F32, False),
    (7, 4096, 1100, 3, 8, BF, BF, F32, False),
    (64, 1024, 768, 20, 64, BF, BF, F32, True),
    (33, 768, 4104, 33, 16, BF, BF, BF, True),
    (200, 1376, 512, 5, 24, BF, BF, F32, True),
    (300, 256, 320, 1, 128, BF, BF, BF, False),
    (130, 264, 136, 2, 256, BF, BF, F32, True),
    (95, 1001, 515, 4, 20, F32, F32, F32, True),
    (65, 333, 77, 3, 5, BF, BF, F32, True),
    (17, 130, 66, 2, 3, BF, F32, BF, True),
    (257, 640, 256, 2, 32, F32, BF, F32, False),
    (40, 512, 258, 2, 48, F32, F32, BF, True),
    (700, 300, 260, 2, 12, BF, F32, F32, True),
]


@pytest.mark.parametrize("T,n,m,S,rmax,xt,wt,yt,mixed", APPLY)
def test_apply_matches_the_oracle(T, n, m, S, rmax, xt, wt, yt, mixed):
    Case(T, n, m, S, rmax, xt, wt, yt, mixed, seed=T).check_apply()


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (0, 1), (2, 2)])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (BF, F32)])
def test_apply_on_rows_of_wider_buffers(pad, offset, xt, yt):
    Case(50, 384, 200, 3, 16, xt, BF, yt, True, seed=5, pad=pad, offset=offset).check_apply(
        u_given=False)


@pytest.mark.parametrize("T", [15, 16, 17, 63, 64, 65, 129, 600])
def test_apply_at_tile_edges_of_the_token_count(T):
    Case(T, 256, 264, 2, 16, idle=0.0, runs=True, seed=T).check_apply(u_given=False)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 255, 256, 257, 1023, 2050])
def test_apply_at_edges_of_the_inner_size(n):
    Case(20, n, 48, 2, 16, seed=n).check_apply()


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 63, 64, 65, 255, 257, 1030])
def test_apply_at_edges_of_the_outer_size(m):
    Case(90, 128, m, 2, 16, yt=BF if m % 2 else F32, seed=m).check_apply()


@pytest.mark.parametrize("rmax", [1, 4, 15, 16, 17, 31, 32, 33, 63, 65, 127, 129, 255])
def test_apply_and_backward_at_edges_of_the_rank(rmax):
    Case(70, 160, 144, 2, rmax, seed=rmax).check_apply()
    Case(70, 160, 144, 2, rmax, seed=rmax).check_backward()


@pytest.mark.parametrize("rmax", [96, 112, 128, 160, 176, 192, 208, 240, 256])
@pytest.mark.parametrize("T", [20, 520])
def test_large_ranks_of_every_tile_count(T, rmax):
    for yt in (BF, F32):
        Case(T, 64, 72, 1, rmax, BF, BF, yt, idle=0.0, seed=rmax).check_apply()
        Case(T, 64, 72, 1, rmax, BF, BF, yt, idle=0.0, seed=rmax).check_backward()


def test_apply_without_scales_and_ranks_and_with_all_tokens_idle():
    Case(30, 128, 64, 2, 8, scaled=False).check_apply()
    c = Case(30, 128, 64, 2, 8, idle=1.1)
    y0 = c.gy.clone()
    G.gptq_lora_apply(c.ad, c.plan, c.gx, c.gy)
    assert torch.equal(c.gy, y0)


def test_ranks_out_of_range_are_taken_as_the_nearer_end():
    c = Case(40, 128, 64, 2, 8)
    c.ad.ranks = torch.tensor([100, -3], dtype=torch.int32, device="cuda")
    ad = G.LowRankAdapters(c.ad.A, c.ad.B, c.ad.ranks, c.ad.scales)
    c.ranks = np.array([8, 0], np.int32)
    c.ad = ad
    c.check_apply()


def test_plan_arrays_out_of_range_are_clamped_and_skipped():
    """order entries outside the tokens are skipped; slot_start is clamped:
    the other tokens' results are as ever."""
    c = Case(40, 128, 64, 1, 8, idle=0.0)
    order, start = c.plan
    bad = order.clone()
    bad[3], bad[20] = -5, 4000
    gone = [int(order[3]), int(order[20])]
    s2 = torch.tensor([-7, 10 ** 6], dtype=torch.int32, device="cuda")
    y0 = c.gy.clone()
    G.gptq_lora_apply(c.ad, (bad, s2), c.gx, c.gy)
    want = c.want_apply()[0]
    for t in range(40):
        if t in gone:
            assert torch.equal(c.gy[t], y0[t])
        else:
            np.testing.assert_allclose(f64(c.gy[t]), want[t], rtol=1e-4, atol=1e-4)
    dx, dA, dB = G.gptq_lora_backward(c.ad, (bad, s2), c.gdy, torch.ones(40, 8, device="cuda"),
                                      x=c.gx)
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()


def test_infinities_and_nan_stay_in_their_own_rows():
    c = Case(50, 256, 96, 2, 16, idle=0.0, seed=3)
    bad = [4, 17, 30]
    x = c.gx.clone()
    x[4, 7], x[17, 100], x[30, 255] = float("nan"), float("inf"), float("-inf")
    clean = c.gy.clone()
    G.gptq_lora_apply(c.ad, c.plan, c.gx, clean)
    y = c.gy.clone()
    G.gptq_lora_apply(c.ad, c.plan, x, y)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[bad]).any()


@pytest.mark.parametrize("xt", [BF, F32])
def test_infinities_and_nan_of_one_token_leave_the_ranks_that_do_not_exist_zero(xt):
    c = Case(50, 256, 96, 2, 16, xt, mixed=True, idle=0.0, seed=4)
    x, dy = c.gx.clone(), c.gdy.clone()
    x[7], dy[9] = float("nan"), float("inf")
    u = torch.zeros(50, 16, device="cuda")
    G.gptq_lora_apply(c.ad, c.plan, x, c.gy, u=u)
    _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, dy, u, x=x)
    for a, r in enumerate(c.ranks[:2]):
        assert not u[c.ids.cuda() == a][:, r:].any()
        assert not dA[a, r:].any() and not dB[a, :, r:].any()


def test_unused_slots_may_hold_anything():
    """Slots that no token uses are not read: their NaN reach nothing."""
    c = Case(30, 128, 64, 3, 8, idle=0.0)
    c.ids[c.ids == 1] = 0
    c.plan = G.gptq_lora_plan(c.ids.cuda(), 3)
    c.ad.A[1], c.ad.B[1] = float("nan"), float("inf")
    c.check_apply()
    c.check_backward()


# ------------------------------------------------------------------ backward
BACKWARD = [
    (1, 512, 512, 1, 16, BF, BF, BF, False, None),
    (1, 64, 64, 1, 4, F32, F32, F32, False, None),
    (96, 1024, 512, 1, 8, BF, BF, BF, False, None),
    (300, 512, 768, 1, 64, BF, BF, BF, False, None),
    (150, 520, 264, 6, 16, BF, BF, F32, True, None),
    (333, 301, 203, 4, 12, F32, F32, F32, True, None),
    (65, 96, 330, 3, 5, F32, BF, F32, True, None),
    (200, 256, 256, 2, 128, BF, F32, BF, True, None),
    (40, 264, 136, 2, 256, BF, BF, F32, True, None),
    (257, 512, 128, 1, 16, BF, BF, BF, False, 128),
    (100, 500, 64, 3, 16, BF, BF, F32, True, 32),
    (100, 500, 64, 3, 24, F32, F32, F32, True, 64),
    (130, 1000, 72, 2, 32, BF, BF, BF, False, 256),
    (75, 333, 40, 2, 8, BF, F32, F32, True, -1),
    (600, 256, 128, 2, 16, BF, BF, F32, True, 128),
]


@pytest.mark.parametrize("T,n,m,S,rmax,xt,wt,yt,mixed,group", BACKWARD)
def test_backward_matches_the_oracle(T, n, m, S, rmax, xt, wt, yt, mixed, group):
    Case(T, n, m, S, rmax, xt, wt, yt, mixed, seed=T + n).check_backward(group)


@pytest.mark.parametrize("want", [("dx",), ("dA",), ("dB",), ("dx", "dA"), ("dx", "dB"),
                                  ("dA", "dB")])
@pytest.mark.parametrize("T,rmax,xt,group", [(50, 16, BF, None), (50, 16, BF, 128),
                                             (50, 24, F32, None), (1100, 64, BF, None),
                                             (1100, 16, BF, 128), (600, 8, F32, None)])
def test_backward_gives_what_is_asked_for(want, T, rmax, xt, group):
    c = Case(T, 256, 128, 3, rmax, xt, mixed=True, runs=T > 500)
    c.check_backward(want=want, group=group if "dA" in want else None)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (0, 1)])
@pytest.mark.parametrize("xt", [BF, F32])
def test_backward_on_rows_of_wider_buffers(pad, offset, xt):
    Case(50, 200, 136, 3, 16, xt, BF, F32, True, seed=6, pad=pad, offset=offset).check_backward()


@pytest.mark.parametrize("pad,offset", [(8, 8), (16, 0), (3, 0), (0, 1)])
@pytest.mark.parametrize("T,yt", [(700, BF), (1200, F32)])
def test_many_tokens_on_rows_of_wider_buffers(pad, offset, T, yt):
    Case(T, 200, 136, 3, 16, BF, BF, yt, True, seed=6, runs=True, pad=pad, offset=offset).check_apply()
    Case(T, 200, 136, 3, 16, BF, BF, yt, True, seed=7, runs=True, pad=pad,
         offset=offset).check_backward()


@pytest.mark.parametrize("n,group", [(1, -1), (7, 32), (33, 32), (127, 64), (129, 128), (513, 128)])
def test_backward_from_codes_at_edges_of_the_groups(n, group):
    Case(50, n, 40, 2, 8, seed=n).check_backward(group)


@pytest.mark.parametrize("runs", [False, True])
def test_backward_many_tokens_in_few_and_in_many_slots(runs):
    Case(3000, 64, 72, 1, 16, idle=0.0, runs=runs, seed=1).check_backward()
    Case(2500, 64, 72, 40, 8, mixed=True, runs=runs, seed=2).check_backward(128)


MANY = [
    # T, n, m, slots, max_rank, yt, mixed, runs, idle, group
    (1500, 320, 200, 1, 64, BF, False, True, 0.0, None),
    (1500, 328, 520, 1, 32, F32, False, False, 0.1, None),
    (2100, 136, 264, 3, 24, BF, True, True, 0.05, None),
    (2100, 264, 136, 5, 64, F32, True, False, 0.05, None),
    (1300, 128, 1032, 2, 128, BF, True, True, 0.0, None),
    (1300, 200, 72, 2, 40, F32, False, False, 0.0, None),
    (4500, 64, 96, 1, 16, BF, False, True, 0.0, None),
    (1100, 520, 256, 7, 16, BF, True, True, 0.1, 128),
    (1100, 384, 264, 4, 64, F32, True, False, 0.1, 256),
    (2300, 272, 128, 2, 32, BF, False, True, 0.0, -1),
    (1025, 640, 640, 30, 8, F32, True, False, 0.3, None),
]


@pytest.mark.parametrize("T,n,m,S,rmax,yt,mixed,runs,idle,group", MANY)
def test_many_bf16_tokens(T, n, m, S, rmax, yt, mixed, runs, idle, group):
    """The kernels for many tokens: whole and short pieces of consecutive rows,
    scattered rows, ranks that fill their tile and ranks that do not."""
    Case(T, n, m, S, rmax, BF, BF, yt, mixed, idle=idle, seed=T + n, runs=runs).check_apply()
    Case(T, n, m, S, rmax, BF, BF, yt, mixed, idle=idle, seed=T + m, runs=runs).check_backward(
        group)


WHOLE = [
    # the kernels of a launch each: tokens x rank x columns past the one-launch form
    # T, n, m, slots, max_rank, xt, wt, yt, mixed, runs, idle
    (4700, 512, 520, 1, 64, BF, BF, BF, False, True, 0.0),
    (4700, 520, 512, 1, 64, BF, BF, F32, False, False, 0.1),
    (9000, 2056, 2048, 3, 16, BF, BF, F32, True, True, 0.05),
    (9000, 1032, 1096, 3, 24, BF, BF, BF, True, False, 0.05),
    (8300, 1024, 1024, 1, 16, BF, BF, F32, False, True, 0.02),
    (6000, 512, 648, 7, 64, BF, BF, F32, True, True, 0.0),
    (5000, 392, 456, 2, 128, BF, BF, BF, False, True, 0.0),
    (5000, 401, 455, 2, 100, BF, BF, F32, True, True, 0.1),
    (4800, 512, 512, 1, 40, BF, F32, BF, False, True, 0.0),
    (4800, 512, 512, 2, 64, F32, F32, F32, True, False, 0.0),
    (4800, 512, 512, 1, 64, F32, BF, BF, False, True, 0.0),
]


@pytest.mark.parametrize("T,n,m,S,rmax,xt,wt,yt,mixed,runs,idle", WHOLE)
def test_a_launch_for_each_projection(T, n, m, S, rmax, xt, wt, yt, mixed, runs, idle):
    c = Case(T, n, m, S, rmax, xt, wt, yt, mixed, idle=idle, seed=T + n, runs=runs)
    assert c.ad.workspace_size(T) > 0        # u goes through memory
    c.check_apply()
    Case(T, n, m, S, rmax, xt, wt, yt, mixed, idle=idle, seed=T + m, runs=runs).check_backward()


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (0, 1)])
def test_a_launch_for_each_projection_on_rows_of_wider_buffers(pad, offset):
    c = Case(4700, 512, 520, 2, 64, BF, BF, BF, True, seed=6, runs=True, pad=pad, offset=offset)
    c.check_apply(u_given=False)
    Case(4700, 512, 520, 2, 64, BF, BF, F32, True, seed=7, runs=True, pad=pad,
         offset=offset).check_backward()


def test_a_launch_for_each_projection_repeats_and_keeps_nonfinite_tokens_apart():
    """Tiles reach into the next slot's tokens; what those hold stays there."""
    c = Case(5000, 512, 520, 2, 64, BF, BF, F32, idle=0.0, runs=True, seed=8)
    bad = (c.ids == 0).cuda()
    x = c.gx.clone()
    x[bad] = float("nan")
    dy = c.gdy.clone()
    dy[bad] = float("inf")
    outs = []
    for a, b in ((x, dy), (c.gx, c.gdy), (c.gx, c.gdy)):
        u, y, dx = torch.zeros(5000, 64, device="cuda"), c.gy.clone(), c.gdx.clone()
        G.gptq_lora_apply(c.ad, c.plan, a, y, u=u)
        _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, b, u, x=a, dx=dx)
        outs.append((y[~bad], u[~bad], dx[~bad], dA[1], dB[1], y, u, dx, dA, dB))
    assert all(torch.equal(p, q) for p, q in zip(outs[0][:5], outs[1][:5]))
    assert all(torch.equal(p, q) for p, q in zip(outs[1], outs[2]))


@pytest.mark.parametrize("n,m", [(8, 8), (24, 40), (72, 1096), (1096, 72), (2048, 16)])
def test_many_bf16_tokens_at_edges_of_the_sizes(n, m):
    Case(1200, n, m, 2, 16, BF, BF, BF, idle=0.0, runs=True, seed=n).check_apply()
    Case(1200, n, m, 2, 16, BF, BF, F32, idle=0.0, runs=True, seed=m).check_backward()


def test_a_short_piece_beside_nonfinite_tokens_of_the_next_slot():
    """Tiles reach into the next slot's tokens; what those hold stays there."""
    c = Case(1400, 192, 136, 2, 16, BF, BF, F32, idle=0.0, runs=True, seed=8)
    x, dy = c.gx.clone(), c.gdy.clone()
    # runs=True sorts the slots in descending order: slot 0's tokens are the last rows
    bad = (c.ids == 0).cuda()
    x[bad], dy[bad] = float("nan"), float("inf")
    u, u0 = torch.zeros(1400, 16, device="cuda"), torch.zeros(1400, 16, device="cuda")
    y, y0 = c.gy.clone(), c.gy.clone()
    G.gptq_lora_apply(c.ad, c.plan, x, y, u=u)
    G.gptq_lora_apply(c.ad, c.plan, c.gx, y0, u=u0)
    assert torch.equal(y[~bad], y0[~bad]) and torch.equal(u[~bad], u0[~bad])
    dx, dx0 = c.gdx.clone(), c.gdx.clone()
    _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, dy, u, x=x, dx=dx)
    _, wA, wB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u0, x=c.gx, dx=dx0)
    assert torch.equal(dx[~bad], dx0[~bad])
    assert torch.equal(dA[1], wA[1]) and torch.equal(dB[1], wB[1])
    assert not torch.isfinite(dA[0]).any()


def test_no_tokens_give_zero_gradients_and_leave_the_rest():
    c = Case(3, 64, 48, 2, 4)
    e = torch.empty(0, 64, device="cuda", dtype=BF)
    ey = torch.empty(0, 48, device="cuda", dtype=BF)
    plan = G.gptq_lora_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    assert G.gptq_lora_apply(c.ad, plan, e, ey.float()).shape == (0, 48)
    _, dA, dB = G.gptq_lora_backward(c.ad, plan, ey, torch.empty(0, 4, device="cuda"), x=e)
    assert not dA.any() and not dB.any()
    # and so do tokens that are all idle
    c = Case(30, 64, 48, 2, 4, idle=1.1)
    _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, torch.ones(30, 4, device="cuda"), x=c.gx)
    assert not dA.any() and not dB.any()


def test_gradients_against_differences():
    """The product is linear in x, in A and in B, so a central difference of
    sum(dy * y) along a direction has no error but its own rounding."""
    c = Case(60, 96, 80, 2, 8, F32, F32, F32, idle=0.0)
    zero = torch.zeros(60, 80, device="cuda")

    def loss(x, A, B):
        ad = G.LowRankAdapters(A, B, None, c.ad.scales)
        y = G.gptq_lora_apply(ad, c.plan, x, zero.clone())
        return float((y.double() * c.gdy.double()).sum())

    def room(x, A, B):
        # how far loss() may be off: its products and their rounding to fp32
        y, _, _, mag = LO.apply(f64(x), f64(A), f64(B), c.ids.numpy(), None, c.oracle_scales(),
                                np.zeros((60, 80)))
        return float((np.abs(f64(c.dy)) * ((c_of(96) + 16 * 2.0 ** -23) * mag
                                           + 2.0 ** -24 * np.abs(y))).sum())

    A, B, x = c.ad.A, c.ad.B, c.gx
    u = torch.empty(60, 8, device="cuda")
    G.gptq_lora_apply(c.ad, c.plan, x, zero.clone(), u=u)
    dx, dA, dB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u, x=x, dx=torch.zeros_like(x))
    o = LO.backward(f64(c.dy), f64(u), f64(x), f64(A), f64(B), c.ids.numpy(), None,
                    c.oracle_scales(), np.zeros((60, 96)))
    # u itself is good to c_of(96) of its magnitude, which reaches dB
    _, _, umag, _ = LO.apply(f64(x), f64(A), f64(B), c.ids.numpy(), None, None, np.zeros((60, 80)))
    mu = LO.backward(f64(c.dy), umag, f64(x), f64(A), f64(B), c.ids.numpy(), None,
                     c.oracle_scales(), np.zeros((60, 96)))["mdB"]
    grads = ((x, dx, (c_of(80) + 16 * 2.0 ** -23) * o["mdx"]),
             (A, dA, (c_of(80) + c_of(60)) * o["mdA"]),
             (B, dB, c_of(60) * o["mdB"] + c_of(96) * mu))
    for k, (t, d, slack) in enumerate(grads):
        e = torch.randint(-2, 3, t.shape, generator=gen(k)).float().cuda()
        args = [[x, A, B], [x, A, B]]
        args[0][k], args[1][k] = t + 4.0 * e, t - 4.0 * e
        # t +- 4 e is rounded to fp32: the direction is what the two differ by
        step = f64(args[0][k]) - f64(args[1][k])
        diff = loss(*args[0]) - loss(*args[1])
        want = float((f64(d) * step).sum())
        tol = room(*args[0]) + room(*args[1]) + float((np.abs(step) * slack).sum())
        assert abs(diff - want) <= tol, (k, diff, want, tol)
        assert tol < 0.01 * float(np.abs(f64(d) * step).sum())   # the check can tell


# ------------------------------------------------------------------ streams, graphs, repeats
def test_results_repeat_bit_for_bit():
    c = Case(500, 512, 384, 4, 16, mixed=True, yt=BF)
    outs = []
    for _ in range(3):
        y, dx = c.gy.clone(), c.gdx.clone()
        u = torch.zeros(500, 16, device="cuda")
        G.gptq_lora_apply(c.ad, c.plan, c.gx, y, u=u)
        _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u, x=c.gx, dx=dx)
        outs.append((y, u, dx, dA, dB))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_own_stream_own_workspace_and_two_calls_at_once():
    c = Case(400, 512, 384, 4, 16, mixed=True)
    d = Case(300, 256, 640, 2, 32, seed=9)
    want = [f64(G.gptq_lora_apply(k.ad, k.plan, k.gx, k.gy.clone())) for k in (c, d)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    ys = []
    for rep in range(4):
        for k, st in zip((c, d), s):
            with torch.cuda.stream(st):
                y = k.gy.clone()
            ws = torch.full((k.ad.workspace_size(k.T) + 256,), 0xFF, dtype=torch.uint8,
                            device="cuda") if rep % 2 else None
            torch.cuda.synchronize()
            ys.append(G.gptq_lora_apply(k.ad, k.plan, k.gx, y, ws=ws, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert np.array_equal(f64(y), want[i % 2])


def test_captured_step_follows_its_inputs():
    """Plan, apply, codes and backward in one graph: replayed with other ids,
    inputs and adapters it gives what the eager calls give."""
    c = Case(200, 256, 192, 3, 16, mixed=False)
    ids, x, dy = c.ids.cuda(), c.gx.clone(), c.gdy.clone()
    x.nan_to_num_()
    y, dx = torch.zeros(200, 192, device="cuda"), torch.zeros(200, 256, device="cuda")

    def step():
        y.zero_(), dx.zero_()
        plan = G.gptq_lora_plan(ids, 3)
        u = torch.empty(200, 16, device="cuda")
        G.gptq_lora_apply(c.ad, plan, x, y, u=u)
        q, s = G.gptq_quantize_act8(x, 128)
        return G.gptq_lora_backward(c.ad, plan, dy, u, codes=q, code_scales=s, group_size=128,
                                    dx=dx)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, dA, dB = step()
    with torch.cuda.graph(g2):
        _, dA2, dB2 = step()
    for k in range(3):
        ids.copy_(torch.randint(-1, 3, (200,), generator=gen(k), dtype=torch.int32))
        x.copy_(torch.randn(200, 256, generator=gen(50 + k)))
        c.ad.B.copy_(torch.randn(c.ad.B.shape, generator=gen(90 + k)))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dA, dB)]
        assert torch.equal(dA, dA2) and torch.equal(dB, dB2)
        _, wA, wB = step()
        for a, b in zip(got, (y, dx, wA, wB)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows that start beyond 2^31 elements of x and y."""
    T, n, m = 6, 256, 128
    step = 2 ** 29 + 64
    xb = torch.empty(step * (T - 1) + n, dtype=BF, device="cuda")
    yb = torch.empty(step * (T - 1) + n, dtype=BF, device="cuda")
    c = Case(T, n, m, 2, 8, yt=BF, idle=0.0)
    x, y = xb.as_strided((T, n), (step, 1)), yb.as_strided((T, m), (step, 1))
    x.copy_(c.gx), y.copy_(c.gy)
    c.gx, c.gy = x, y
    u = c.check_apply()
    dy = y
    dy.copy_(c.dy)
    _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, dy, u, x=x)
    _, wA, wB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u, x=c.x.cuda())
    assert torch.equal(dA, wA) and torch.equal(dB, wB)


def test_many_tokens_repeat_bit_for_bit_and_in_a_graph():
    """Three calls and a replay of the kernels for many tokens, on another
    stream than the default one."""
    c = Case(1500, 384, 264, 3, 32, BF, BF, BF, mixed=True, runs=True, idle=0.05)
    x, dy = c.gx.nan_to_num(), c.gdy.clone()
    y, dx = c.gy.clone(), c.gdx.clone()
    outs = []

    def step():
        y.copy_(c.gy), dx.copy_(c.gdx)
        u = torch.zeros(1500, 32, device="cuda")
        G.gptq_lora_apply(c.ad, c.plan, x, y, u=u)
        _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, dy, u, x=x, dx=dx)
        return u, dA, dB

    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(3):
            outs.append([t.clone() for t in (*step(), y, dx)])
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (*kept, y, dx)])
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


# ------------------------------------------------------------------ with the quantized layer
def _layer(rows, n, actorder, seed):
    g = gen(seed)
    W = (torch.randn(rows, n, generator=g) * 0.05).to(BF).cuda()
    X = torch.randn(n, 512, generator=g).to(BF).cuda()
    return G.quantize_linear(W, X, bits=4, group_size=64, actorder=actorder)


@pytest.mark.parametrize("actorder,sweep_order", [(False, False), (True, False), (True, True)])
def test_adapted_linear_serves_and_trains(actorder, sweep_order):
    """Quantize a layer, then serve and train adapters beside its codes."""
    rows, n, T, S, r = 192, 256, 48, 3, 8
    q = _layer(rows, n, actorder, 11)
    c = Case(T, n, rows, S, r, seed=12)
    x = c.x.cuda()
    if sweep_order:
        packed = G.gptq_pack_int4(G.gptq_gather_columns_u8(q.codes, q.perm))
        lin = G.AdaptedLinear(packed, 4, n, q.scales, q.zeros, 64, c.ad, perm=q.perm)
    else:
        lin = G.AdaptedLinear.from_quantized(q, c.ad)
    W = f64(G.gptq_dequant(q.packed, 4, n, q.scales, q.zeros, 64, q.g_idx))
    assert np.array_equal(f64(lin.weight(F32)), W)
    base = f64(c.x) @ W.T
    bmag = np.abs(f64(c.x)) @ np.abs(W).T
    want, _, _, dmag = LO.apply(f64(c.x), f64(c.A), f64(c.B), c.ids.numpy(), None,
                                c.oracle_scales(), base)
    y = f64(lin.matvec(x, c.plan))
    bound = 2 * (n / 32 + 24) * 2.0 ** -24 * bmag + (c_of(n) + (r + 8) * 2.0 ** -23) * dmag \
        + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(y - want) <= bound)
    # training: weights and the base product are rounded to bf16, then the sum
    yt, saved = lin.forward(x, c.plan)
    assert set(saved) == {"u", "codes", "code_scales", "group_size"}
    slack = 2.0 ** -8 * (bmag + 2 * np.abs(base) + np.abs(want)) + 2.0 ** -17 * dmag + bound
    assert np.all(np.abs(f64(yt) - want) <= 1.01 * slack)
    dx, dA, dB = lin.backward(c.gdy, c.plan, saved)
    qc, qs = LO.quantize_act8(f64(c.x), 128)
    xo = LO.dequant_act8(qc, qs, 128).astype(np.float64)
    u = np.nan_to_num(f64(saved["u"]))
    u[c.ids.numpy() < 0] = 0
    dbase = f64(c.dy) @ W
    o = LO.backward(f64(c.dy), u, xo, f64(c.A), f64(c.B), c.ids.numpy(), None, c.oracle_scales(),
                    dbase)
    dmagW = np.abs(f64(c.dy)) @ np.abs(W)
    slack = 2.0 ** -8 * (dmagW + 2 * np.abs(dbase) + np.abs(o["dx"])) \
        + (2.0 ** -17 + c_of(rows) + (r + 8) * 2.0 ** -23) * o["mdx"]
    assert np.all(np.abs(f64(dx) - o["dx"]) <= 1.01 * slack)
    assert np.all(np.abs(f64(dA) - o["dA"]) <= (c_of(rows) + c_of(T) + 2.0 ** -24) * o["mdA"])
    assert np.all(np.abs(f64(dB) - o["dB"]) <= c_of(T) * o["mdB"])
    keep = G.AdaptedLinear.from_quantized(q, c.ad, act_group=None).forward(x, c.plan)[1]
    assert keep["x"] is x


def test_moved_adapters_and_foreign_streams_are_refused():
    c = Case(10, 64, 48, 2, 4)
    y = c.gy.clone()
    other = types.SimpleNamespace(device=torch.device("cuda", torch.cuda.device_count()),
                                  cuda_stream=0)
    with pytest.raises(G.GptqError, match="stream"):
        G.gptq_lora_apply(c.ad, c.plan, c.gx, y, stream=other)
    with pytest.raises(G.GptqError, match="stream"):
        G.gptq_quantize_act8(c.gx, stream=other)
    with pytest.raises(G.GptqError, match="stream"):
        G.gptq_lora_plan(c.plan[0], 2, stream=other)
    old = c.ad.A.data
    c.ad.A.data = old.clone()
    with pytest.raises(G.GptqError, match="moved"):
        G.gptq_lora_apply(c.ad, c.plan, c.gx, y)
    with pytest.raises(G.GptqError, match="moved"):
        G.gptq_lora_backward(c.ad, c.plan, c.gy, x=c.gx, want_dB=False)
    c.ad.A.data = old
    assert torch.equal(y, c.gy)
    G.gptq_lora_apply(c.ad, c.plan, c.gx, y)


def test_wrapper_refusals():
    c = Case(10, 64, 48, 2, 4)
    ad, plan = c.ad, c.plan
    E = G.GptqError
    with pytest.raises(E):
        G.LowRankAdapters(c.A, c.B)                                   # on the CPU
    with pytest.raises(E):
        G.LowRankAdapters(ad.A, ad.B.float())                         # two types
    with pytest.raises(E):
        G.LowRankAdapters(ad.A, ad.B[:, :, :2])                       # two ranks
    with pytest.raises(E):
        G.LowRankAdapters(ad.A, ad.B, torch.zeros(2, device="cuda"))  # fp32 ranks
    with pytest.raises(E):
        G.LowRankAdapters(ad.A.half(), ad.B.half())
    with pytest.raises(E):
        G.LowRankAdapters(ad.A.expand(2, 4, 64)[:, :, ::2], ad.B[:, :, :4])
    with pytest.raises(E):
        G.LowRankAdapters(ad.A[:1].expand(2, 4, 64), ad.B)            # slots overlap
    with pytest.raises(E):
        G.LowRankAdapters(torch.zeros(1, 257, 8, device="cuda"),
                          torch.zeros(1, 8, 257, device="cuda"))      # rank past 256
    bad = [dict(x=c.gx[:, :32]), dict(y=c.gy[:9]), dict(y=c.gy.half()), dict(x=c.gx.t()),
           dict(x=c.gx.cpu()), dict(u=torch.zeros(10, 4, dtype=BF, device="cuda")),
           dict(u=torch.zeros(10, 3, device="cuda")), dict(plan=(plan[0][:9], plan[1])),
           dict(plan=(plan[0].long(), plan[1])), dict(plan=(plan[0], plan[1][:2])),
           dict(y=c.gy[:1].expand(10, 48))]
    for b in bad:
        k = {**dict(plan=plan, x=c.gx, y=c.gy), **b}
        with pytest.raises(E):
            G.gptq_lora_apply(ad, k["plan"], k["x"], k["y"], u=k.get("u"))
    u = torch.zeros(10, 4, device="cuda")
    q, s = G.gptq_quantize_act8(c.gx.nan_to_num(), 32)
    good = dict(dy=c.gdy, u=u, x=c.gx)
    for b in [dict(x=None), dict(codes=q, code_scales=s, group_size=32), dict(u=None),
              dict(x=None, codes=q, code_scales=s, group_size=64),
              dict(x=None, codes=q, code_scales=s.half(), group_size=32),
              dict(x=None, codes=q.int(), code_scales=s, group_size=32),
              dict(x=None, codes=q, code_scales=s, group_size=0),
              dict(dx=c.gdx[:9]), dict(dA=torch.zeros(2, 4, 63, device="cuda")),
              dict(dB=torch.zeros(2, 48, 4, dtype=BF, device="cuda")), dict(dy=c.gdy[:, :40])]:
        k = {**good, **b}
        with pytest.raises(E):
            G.gptq_lora_backward(ad, plan, k.pop("dy"), k.pop("u"), **k)
    with pytest.raises(E):
        G.gptq_lora_plan(torch.zeros(3, dtype=torch.int64, device="cuda"), 2)
    with pytest.raises(E):
        G.gptq_lora_plan(torch.zeros(3, dtype=torch.int32), 2)
    with pytest.raises(E):
        G.gptq_lora_plan(torch.zeros(3, dtype=torch.int32, device="cuda"), -1)
    with pytest.raises(E):
        G.AdaptedLinear(torch.zeros(47, 8, dtype=torch.int32, device="cuda"), 4, 64, None, None,
                        32, ad)


# ------------------------------------------------------------------ pieces of empty slots
@pytest.mark.parametrize("T,S,n,m", [(6000, 400, 64, 48), (3000, 300, 40, 2056), (40, 30, 24, 16)])
def test_tokens_of_empty_slots_where_a_cta_stands_alone(T, S, n, m):
    """So many pieces (or so short axes) that each has one CTA, and CTAs follow
    each other on an SM: tokens of slots of rank 0 get zeros in u, and no other
    token's u, v, y or dx is touched."""
    Case(T, n, m, S, 16, BF, BF, F32, mixed=True, idle=0.05, seed=T).check_apply()
    Case(T, n, m, S, 24, BF, BF, F32, mixed=True, idle=0.05, seed=T + 1).check_backward()


def test_calls_of_two_threads_at_once():
    """Two host threads with adapters of unlike ranks: the kernels' limits of
    shared memory belong to the device, not to a call."""
    import threading
    cases = [Case(2000, 256, 256, 1, r, F32, F32, F32, idle=0.0, seed=r) for r in (144, 256)]
    want = []
    for c in cases:
        assert c.ad.workspace_size(c.T) > 0
        u = torch.zeros(c.T, c.rmax, device="cuda")
        want.append((G.gptq_lora_apply(c.ad, c.plan, c.gx, c.gy.clone(), u=u), u))
    torch.cuda.synchronize()
    failed, streams = [], [torch.cuda.Stream() for _ in cases]

    def work(c, s, w):
        try:
            with torch.cuda.stream(s):
                for _ in range(2000):
                    G.gptq_lora_apply(c.ad, c.plan, c.gx, c.gy.clone(),
                                      u=torch.empty_like(w[1]))
                y, u = c.gy.clone(), torch.zeros_like(w[1])
                G.gptq_lora_apply(c.ad, c.plan, c.gx, y, u=u)
                s.synchronize()
                assert torch.equal(y, w[0]) and torch.equal(u, w[1])
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, streams, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# ------------------------------------------------------------------ strides of everything
def in_bank(t, rows, cols, pad, offset, between):
    """The same values as parts of a larger bank of NaN: rows `pad` apart from
    the columns' end, slots `between` elements apart."""
    S = t.shape[0]
    ld = cols + pad + offset
    step = rows * ld + between
    bank = torch.full((S * step + ld,), float("nan"), dtype=t.dtype, device="cuda")
    view = bank[offset:].as_strided((S, rows, cols), (step, ld, 1))
    view.copy_(t)
    return view


BANKS = [(8, 8, 0), (0, 0, 8), (8, 0, 48), (3, 1, 0), (0, 0, 1), (4, 4, 0)]


@pytest.mark.parametrize("pad,offset,between", BANKS)
@pytest.mark.parametrize("T,n,m,S,r,wt,yt,mixed", [
    (70, 160, 144, 3, 16, BF, F32, True), (70, 160, 144, 3, 40, F32, F32, False),
    (4700, 512, 520, 2, 64, BF, BF, True), (4700, 512, 520, 2, 32, BF, F32, False),
    (3000, 512, 520, 2, 128, BF, BF, True), (1400, 264, 136, 2, 16, BF, BF, False)])
def test_adapters_that_are_parts_of_a_bank(T, n, m, S, r, wt, yt, mixed, pad, offset, between):
    for check in ("check_apply", "check_backward"):
        c = Case(T, n, m, S, r, BF, wt, yt, mixed, seed=T + r, runs=True, idle=0.02)
        A, B = (in_bank(t, t.shape[1], t.shape[2], pad, offset, between)
                for t in (c.ad.A, c.ad.B))
        c.ad = G.LowRankAdapters(A, B, c.ad.ranks, c.ad.scales)
        getattr(c, check)()


@pytest.mark.parametrize("pad,offset", [(4, 4), (8, 0), (3, 0), (0, 1)])
@pytest.mark.parametrize("T,n,m,r,xt", [(40, 128, 96, 16, BF), (300, 128, 96, 12, F32),
                                        (1400, 264, 136, 16, BF), (1400, 264, 136, 40, BF),
                                        (4700, 512, 520, 64, BF), (4700, 512, 520, 64, F32)])
def test_u_as_rows_of_a_wider_buffer(T, n, m, r, xt, pad, offset):
    """Written by the forward pass, read by the backward pass, and the same bits
    as a dense u gives; nothing beside it is touched."""
    c = Case(T, n, m, 2, r, xt, BF, F32, mixed=True, runs=True, idle=0.02, seed=T)
    wide = torch.full((T, r + pad + offset), 7.0, device="cuda")
    u, dense = wide[:, offset:offset + r], torch.full((T, r), 7.0, device="cuda")
    y0, y1 = c.gy.clone(), c.gy.clone()
    G.gptq_lora_apply(c.ad, c.plan, c.gx, y0, u=dense)
    G.gptq_lora_apply(c.ad, c.plan, c.gx, y1, u=u)
    assert torch.equal(u, dense) and torch.equal(y0, y1)
    edge = torch.ones(r + pad + offset, dtype=torch.bool, device="cuda")
    edge[offset:offset + r] = False
    assert torch.all(wide[:, edge] == 7.0)
    wide[:, edge] = float("nan")
    g0 = G.gptq_lora_backward(c.ad, c.plan, c.gdy, dense, x=c.gx)
    g1 = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u, x=c.gx)
    assert torch.equal(g0[1], g1[1]) and torch.equal(g0[2], g1[2])


@pytest.mark.parametrize("pad,offset", [(16, 16), (8, 8), (5, 0), (1, 3)])
@pytest.mark.parametrize("T,group", [(70, 32), (70, 128), (1400, 64), (1400, 128), (1400, -1)])
def test_codes_as_rows_of_a_wider_buffer(T, group, pad, offset):
    """The oracle of dense codes: the columns beside them hold other codes."""
    n, m, r = 392, 136, 16
    c = Case(T, n, m, 2, r, runs=True, idle=0.0, seed=T)
    q, s = G.gptq_quantize_act8(c.gx, group)
    wide = torch.full((T, n + pad + offset), 77, dtype=torch.int8, device="cuda")
    wide[:, offset:offset + n] = q
    u = torch.randn(T, r, generator=gen(3))
    _, dA, dB = G.gptq_lora_backward(c.ad, c.plan, c.gdy, u.cuda(),
                                     codes=wide[:, offset:offset + n], code_scales=s,
                                     group_size=group)
    xo = LO.dequant_act8(q.cpu().numpy(), s.cpu().numpy(), group).astype(np.float64)
    o = LO.backward(f64(c.dy), f64(u), xo, f64(c.A), f64(c.B), c.ids.numpy(), c.ranks,
                    c.oracle_scales(), f64(c.dx))
    ca = c_of(m) + c_of(T) + 2.0 ** -24
    assert np.all(np.abs(f64(dA) - o["dA"]) <= ca * o["mdA"])
    assert np.all(np.abs(f64(dB) - o["dB"]) <= c_of(T) * o["mdB"])


@pytest.mark.parametrize("T,S", [(200003, 3000), (3001, 65536)])
def test_plan_of_very_many_slots(T, S):
    ids = torch.randint(-1, S, (T,), generator=gen(T), dtype=torch.int32)
    order, start = G.gptq_lora_plan(ids.cuda(), S)
    wo, ws = LO.plan(ids.numpy(), S)
    assert np.array_equal(order.cpu().numpy(), wo) and np.array_equal(start.cpu().numpy(), ws)


# ------------------------------------------------------------------ unlike types in one call
@pytest.mark.parametrize("T,n,m,r", [(50, 160, 136, 16), (1100, 264, 136, 40), (4700, 512, 520, 64)])
@pytest.mark.parametrize("xt,dyt,dxt,group", [(BF, F32, BF, None), (F32, BF, F32, None),
                                              (F32, BF, BF, 128), (BF, F32, F32, 64),
                                              (BF, BF, F32, -1)])
def test_x_and_dy_of_unlike_types(T, n, m, r, xt, dyt, dxt, group):
    c = Case(T, n, m, 2, r, xt, BF, dxt, mixed=True, runs=True, idle=0.02, seed=T + r)
    c.dy = c.dy.to(dyt)
    c.gdy = c.dy.cuda()
    c.check_backward(group)


@pytest.mark.parametrize("T,n,m,r", [(3000, 512, 520, 256), (3000, 512, 520, 200), (1300, 136, 264, 256)])
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F32, F32)])
def test_the_largest_ranks_with_many_tokens(T, n, m, r, xt, wt):
    Case(T, n, m, 2, r, xt, wt, BF, mixed=True, runs=True, idle=0.02, seed=r).check_apply()
    Case(T, n, m, 2, r, xt, wt, F32, mixed=True, runs=True, idle=0.02, seed=r).check_backward()
