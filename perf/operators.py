"""Cases that measure the low-rank adapter and 8-bit activation operators.

Each case is one pass through one operator (or, for ``kind = "step"``, one
training step of an adapted linear) at sizes that a user of the library meets:

* ``apply``     y += scale_a (x A_a^T) B_a^T for the adapter a of every token,
                beside the frozen projection's product that is already in y;
* ``backward``  dx += v A, dA = v^T x, dB = scale dy^T u with v = scale dy B,
                from x itself or from the 8-bit codes saved in its place;
* ``act8``      8-bit codes and scales of x, and x restored from them;
* ``step``      token plan, apply, 8-bit codes of x, backward from the codes.

``own = False`` computes the plain forms with elementary torch operations;
``own = True`` calls the library.
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SZ = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request's next token through one adapter of a 4096 x 4096 projection
        dict(name="decode_one", kind="apply", ntok=1, n=4096, rows=4096, slots=1, rank=16,
             mixed=False, runs=False, idle=False, xt="bf16", wt="bf16", yt="f32"),
        # the next tokens of 64 requests with 32 adapters of unlike ranks, gate projection
        dict(name="decode_mixed", kind="apply", ntok=64, n=4096, rows=11008, slots=32, rank=64,
             mixed=True, runs=False, idle=True, xt="bf16", wt="bf16", yt="f32"),
        # the prompts of several requests with 8 adapters, down projection
        dict(name="prompt_mixed", kind="apply", ntok=2048, n=11008, rows=4096, slots=8, rank=16,
             mixed=True, runs=True, idle=True, xt="bf16", wt="bf16", yt="f32"),
        # a full training or prefill batch on the widest layer, one adapter
        dict(name="long_wide", kind="apply", ntok=8192, n=28672, rows=8192, slots=1, rank=32,
             mixed=False, runs=True, idle=False, xt="bf16", wt="bf16", yt="bf16"),
        # float32 throughout, sizes that divide nothing
        dict(name="ragged_f32", kind="apply", ntok=777, n=1001, rows=515, slots=5, rank=24,
             mixed=True, runs=True, idle=True, xt="f32", wt="f32", yt="f32"),
        # a short fine-tuning example
        dict(name="grad_short", kind="backward", ntok=96, n=4096, rows=4096, slots=1, rank=8,
             mixed=False, runs=True, idle=False, xt="bf16", wt="bf16", yt="bf16", group=0),
        # a micro-batch at a large rank, up projection
        dict(name="grad_rank64", kind="backward", ntok=4096, n=4096, rows=11008, slots=1, rank=64,
             mixed=False, runs=True, idle=False, xt="bf16", wt="bf16", yt="bf16", group=0),
        # several adapters trained side by side, float32 parameters and gradients
        dict(name="grad_mixed_f32", kind="backward", ntok=1500, n=2048, rows=2056, slots=6,
             rank=16, mixed=True, runs=True, idle=True, xt="f32", wt="f32", yt="f32", group=0),
        # the down projection's backward pass from inputs saved in 8 bits
        dict(name="grad_codes", kind="backward", ntok=8192, n=11008, rows=4096, slots=1, rank=16,
             mixed=False, runs=True, idle=False, xt="bf16", wt="bf16", yt="bf16", group=128),
        # one short sequence's inputs, one scale a token
        dict(name="act8_token", kind="act8", ntok=48, n=4096, xt="bf16", group=-1),
        # a batch of the widest layer's inputs, groups of 128
        dict(name="act8_wide", kind="act8", ntok=8192, n=28672, xt="bf16", group=128),
        # one training step of one adapted 4096 x 4096 projection
        dict(name="step_4096", kind="step", ntok=4096, n=4096, rows=4096, slots=1, rank=16,
             mixed=False, runs=True, idle=False, xt="bf16", wt="bf16", yt="bf16", group=128),
    ]


def _log(rng, lo, hi):
    import math
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    w = _log(rng, lo, hi)
    step = rng.choice([128, 128, 64, 32, 8, 1])
    return max(lo, w // step * step)


def draw(rng):
    kind = rng.choice(["apply", "apply", "apply", "backward", "backward", "act8", "step"])
    most = work(dict(listed()[3]))["bytes"]
    while True:
        if kind == "act8":
            c = dict(kind=kind, ntok=_log(rng, 1, 8192), n=_width(rng, 64, 28672),
                     xt=rng.choice(["bf16", "bf16", "f32"]), group=rng.choice([-1, 32, 64, 128, 128, 256]))
        else:
            decode = kind == "apply" and rng.random() < 0.5
            slots = _log(rng, 1, 64) if decode else _log(rng, 1, 12)
            rank = rng.choice([4, 8, 16, 16, 24, 32, 64, 96, 128])
            if slots * rank > (2048 if decode else 256):
                continue
            f32 = rng.random() < 0.2
            c = dict(kind=kind, ntok=_log(rng, 1, 256) if decode else _log(rng, 16, 8192),
                     n=_width(rng, 256, 28672), rows=_width(rng, 256, 11008), slots=slots,
                     rank=rank, mixed=rng.random() < 0.5, runs=not decode,
                     idle=rng.random() < 0.5, xt="f32" if f32 else "bf16",
                     wt="f32" if f32 or rng.random() < 0.25 else "bf16",
                     yt="f32" if f32 or rng.random() < 0.5 else "bf16")
            if kind == "backward":
                c["group"] = rng.choice([0, 0, -1, 32, 64, 128])
            if kind == "step":
                c["group"] = rng.choice([-1, 64, 128])
        if work(c)["bytes"] <= most and c["ntok"] * c["n"] <= 8192 * 28672 // 2:
            return c


# ------------------------------------------------------------------ inputs
def _ranks(case):
    """The slots' ranks: all alike, or halves, an odd one and an empty slot among them."""
    r = case["rank"]
    if not case["mixed"]:
        return [r] * case["slots"]
    kinds = [r, max(1, r // 2), max(1, r // 4), max(1, r // 2 - 1), 0]
    return [kinds[a % 5] for a in range(case["slots"])]


def _ids(case, g):
    """The adapter of each token: requests of consecutive tokens, or one token a request."""
    T, S = case["ntok"], case["slots"]
    if case["runs"]:
        pieces = min(T, max(S, 3 * S if S > 1 else 1))
        cut = torch.sort(torch.randint(0, T, (pieces - 1,), generator=g, device="cuda")).values
        req = torch.searchsorted(cut, torch.arange(T, device="cuda"), right=True)
        slot = torch.randint(0, S, (pieces,), generator=g, device="cuda")
        ids = slot[req]
    else:
        ids = torch.randint(0, S, (T,), generator=g, device="cuda")
    if case["idle"]:
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.06, -1, ids)
    return ids.to(torch.int32)


def _act(g, T, n, dt):
    """Activations: normal values with a few outlier channels."""
    x = torch.randn(T, n, generator=g, device="cuda")
    if n >= 128:
        x[:, torch.randperm(n, generator=g, device="cuda")[: n // 512 + 1]] *= 20.0
    return x.to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, n = case["ntok"], case["n"]
    s = {"case": dict(case), "x": _act(g, T, n, _DT[case["xt"]])}
    if case["kind"] == "act8":
        return s
    m, S, r = case["rows"], case["slots"], case["rank"]
    wt, yt = _DT[case["wt"]], _DT[case["yt"]]
    s["A"] = (torch.randn(S, r, n, generator=g, device="cuda") * n ** -0.5).to(wt)
    s["B"] = (torch.randn(S, m, r, generator=g, device="cuda") * 0.05).to(wt)
    s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
    s["scales"] = torch.rand(S, generator=g, device="cuda") + 0.5
    s["ids"] = _ids(case, g)
    # the tokens by adapter, which a serving or training program keeps for all its layers
    key = torch.where(s["ids"] < 0, S, s["ids"]).long()
    s["order"] = torch.argsort(key, stable=True).to(torch.int32)
    s["slot_start"] = torch.searchsorted(
        torch.sort(key).values, torch.arange(S + 1, device="cuda")).to(torch.int32)
    if case["kind"] in ("apply", "step"):
        s["y"] = torch.randn(T, m, generator=g, device="cuda").to(yt)
    if case["kind"] in ("backward", "step"):
        s["dy"] = (torch.randn(T, m, generator=g, device="cuda") * 0.02).to(_DT[case["xt"]])
        s["dx"] = (torch.randn(T, n, generator=g, device="cuda") * 0.02).to(yt)
    if case["kind"] == "backward":
        s["u"] = _project(s)
        if case["group"]:
            s["codes"], s["code_scales"] = _quantize(s["x"], case["group"])
            del s["x"]
    return s


# ------------------------------------------------------------------ plain forms
def _mask(s):
    """(ntok, slots, rank): the places of each token's own adapter."""
    S, r, _ = s["A"].shape
    dev = s["A"].device
    mine = s["ids"].long()[:, None] == torch.arange(S, device=dev)
    real = torch.arange(r, device=dev) < s["ranks"][:, None]
    return mine[:, :, None] & real


def _project(s):
    """u = x A^T of each token's own adapter, (ntok, rank); zeros where there is none."""
    S, r, n = s["A"].shape
    U = (s["x"].float() @ s["A"].float().reshape(S * r, n).t()).reshape(-1, S, r)
    return torch.where(_mask(s), U, 0.0).sum(1)


def _spread(s, u):
    """scale u in the places of each token's own adapter, (ntok, slots rank)."""
    v = torch.where(_mask(s), (u[:, None, :] * s["scales"][:, None]), 0.0)
    return v.reshape(u.shape[0], -1)


def _flat_b(s):
    """B of all slots as (slots rank, rows)."""
    S, m, r = s["B"].shape
    return s["B"].float().permute(0, 2, 1).reshape(S * r, m)


def _apply(s, u):
    s["y"].copy_((s["y"].float() + _spread(s, u) @ _flat_b(s)).to(s["y"].dtype))


def _backward(s, u, x):
    S, r, n = s["A"].shape
    m = s["B"].shape[1]
    dy = s["dy"].float()
    v = (dy @ _flat_b(s).t()).reshape(-1, S, r) * s["scales"][:, None]
    v = torch.where(_mask(s), v, 0.0).reshape(-1, S * r)
    s["dx"].copy_((s["dx"].float() + v @ s["A"].float().reshape(S * r, n)).to(s["dx"].dtype))
    dA = (v.t() @ x).reshape(S, r, n)
    dB = (dy.t() @ _spread(s, u)).reshape(m, S, r).permute(1, 0, 2).contiguous()
    return {"dx": s["dx"], "dA": dA, "dB": dB}


def _groups(x, group):
    """x as (ntok, groups, group), zeros behind a ragged last group."""
    T, n = x.shape
    g = n if group < 0 else group
    G = (n + g - 1) // g
    return torch.nn.functional.pad(x, (0, G * g - n)).reshape(T, G, g)


def _quantize(x, group):
    """codes = round to even of x / scale, scale = max |x| of the group / 127 in float32.
    The quotient is next to a border often enough that it is taken in 64 bits."""
    T, n = x.shape
    xg = _groups(x, group)
    s = (xg.abs().amax(-1).double() / 127.0).float().clamp(min=2.0 ** -126)
    q = torch.round(xg.double() / s.double()[:, :, None]).clamp(-127, 127).to(torch.int8)
    return q.reshape(T, -1)[:, :n].contiguous(), s


def _restore(codes, scales, group):
    """float32 values that the codes stand for."""
    T, n = codes.shape
    return (_groups(codes, group).float() * scales[:, :, None]).reshape(T, -1)[:, :n]


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case = s["case"]
    if case["kind"] == "apply":
        _apply(s, _project(s))
        return {"y": s["y"]}
    if case["kind"] == "backward":
        x = _restore(s["codes"], s["code_scales"], case["group"]) if case["group"] else s["x"].float()
        return _backward(s, s["u"], x)
    q, qs = _quantize(s["x"], case["group"])
    if case["kind"] == "act8":
        return {"codes": q, "scales": qs, "x": _restore(q, qs, case["group"]).to(s["x"].dtype)}
    u = _project(s)
    _apply(s, u)
    return {"y": s["y"], **_backward(s, u, _restore(q, qs, case["group"]))}


def _run_own(s):
    import post_weight_quantization_25_b200 as G
    case = s["case"]
    if case["kind"] == "act8":
        q, qs = G.gptq_quantize_act8(s["x"], case["group"])
        return {"codes": q, "scales": qs,
                "x": G.gptq_dequant_act8(q, qs, case["group"], out_dtype=s["x"].dtype)}
    ad = s.get("adapters")
    if ad is None:
        ad = s["adapters"] = G.LowRankAdapters(s["A"], s["B"], s["ranks"], s["scales"])
    if case["kind"] == "apply":
        return {"y": G.gptq_lora_apply(ad, (s["order"], s["slot_start"]), s["x"], s["y"])}
    if case["kind"] == "backward":
        if case["group"]:
            saved = dict(codes=s["codes"], code_scales=s["code_scales"], group_size=case["group"])
        else:
            saved = dict(x=s["x"])
        dx, dA, dB = G.gptq_lora_backward(ad, (s["order"], s["slot_start"]), s["dy"], s["u"],
                                          dx=s["dx"], **saved)
        return {"dx": dx, "dA": dA, "dB": dB}
    plan = G.gptq_lora_plan(s["ids"], case["slots"])
    u = torch.empty(case["ntok"], case["rank"], dtype=torch.float32, device=s["x"].device)
    G.gptq_lora_apply(ad, plan, s["x"], s["y"], u=u)
    q, qs = G.gptq_quantize_act8(s["x"], case["group"])
    dx, dA, dB = G.gptq_lora_backward(ad, plan, s["dy"], u, codes=q, code_scales=qs,
                                      group_size=case["group"], dx=s["dx"])
    return {"y": s["y"], "dx": dx, "dA": dA, "dB": dB}


# ------------------------------------------------------------------ in 64 bits
def _exact_quantize(x, group):
    T, n = x.shape
    g = n if group < 0 else group
    codes, scales = torch.empty(T, n, dtype=torch.int8, device=x.device), []
    for c in range(0, n, g):
        w = x[:, c:c + g].double()
        sc = (w.abs().max(dim=1).values / 127.0).to(torch.float32)
        sc = torch.maximum(sc, torch.full_like(sc, 2.0 ** -126))
        scales.append(sc)
        codes[:, c:c + g] = torch.round(w / sc.double()[:, None]).to(torch.int8)
    return codes, torch.stack(scales, 1)


def _exact_values(codes, scales, group):
    n = codes.shape[1]
    g = n if group < 0 else group
    return codes.double() * scales.double().repeat_interleave(g, dim=1)[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "act8":
        q, qs = _exact_quantize(s["x"], case["group"])
        return {"codes": q, "scales": qs.double(), "x": _exact_values(q, qs, case["group"])}
    out = {}
    y = s["y"].double() if "y" in s else None
    dx = s["dx"].double() if "dx" in s else None
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    if kind == "step":
        xs = _exact_values(*_exact_quantize(s["x"], case["group"]), case["group"])
    elif kind == "backward" and case["group"]:
        xs = _exact_values(s["codes"], s["code_scales"], case["group"])
    else:
        xs = None
    for a, r in enumerate(_ranks(case)):
        t = torch.nonzero(s["ids"] == a).flatten()
        if r == 0 or t.numel() == 0:
            continue
        A, B = s["A"][a, :r].double(), s["B"][a, :, :r].double()
        sc = float(s["scales"][a])
        u = s["x"][t].double() @ A.t() if kind != "backward" else s["u"][t, :r].double()
        if y is not None:
            y[t] += sc * (u @ B.t())
        if dx is not None:
            dy = s["dy"][t].double()
            v = sc * (dy @ B)
            dx[t] += v @ A
            dA[a, :r] = v.t() @ (xs[t] if xs is not None else s["x"][t].double())
            dB[a, :, :r] = sc * (dy.t() @ u)
    if y is not None:
        out["y"] = y
    if dx is not None:
        out.update(dx=dx, dA=dA, dB=dB)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, n, x = case["ntok"], case["n"], _SZ[case["xt"]]
    if case["kind"] == "act8":
        G = 1 if case["group"] < 0 else -(-n // case["group"])
        # x in, codes and scales out; codes and scales in, x out
        return {"bytes": 2 * T * (n * (x + 1) + 4 * G), "flops": 4 * T * n}
    m, w, y = case["rows"], _SZ[case["wt"]], _SZ[case["yt"]]
    live = T * (0.94 if case["idle"] else 1.0)
    ranks = _ranks(case)
    # adapters that at least one token uses, and the tokens' mean rank
    used = case["slots"] * (1.0 - (1.0 - 1.0 / case["slots"]) ** live)
    rank = sum(ranks) / len(ranks)
    params = used * rank * (n + m)
    flops = 2 * live * rank * (n + m)
    fwd = live * (n * x + 2 * m * y) + params * w
    if case["kind"] == "apply":
        return {"bytes": fwd, "flops": flops}
    code = 1 + 4.0 / (n if case["group"] < 0 else case["group"]) if case["group"] else x
    grads = 4 * case["slots"] * case["rank"] * (n + m)
    bwd = live * (m * x + n * code + 2 * n * y + 4 * case["rank"]) + params * w + grads
    if case["kind"] == "backward":
        return {"bytes": bwd, "flops": 2 * flops}
    # the step reads x for the forward product and writes its codes, which stay out of both sums
    return {"bytes": fwd + bwd + live * n * code, "flops": 3 * flops}
