"""Cases of the routed-expert layer's operators around the grouped product.

Four operators, each timed as one call (or one forward and backward) of a
user's program:

* ``route``    -- scores, balance bias, expert groups, top-k and weights of a router;
* ``dispatch`` -- the grouped order of the routed slots and the rows gathered into it
  (as they are, or as the fp8 operand of the W4A8 product);
* ``combine``  -- the weighted sum that brings the experts' rows back to their tokens;
* ``swiglu``   -- the experts' activation with its input kept in 8 bits for the backward.

``run`` computes them in plain torch operations, or with the framework's
kernels where ``own`` is true.  ``exact`` computes the same from the
definitions in 64 bits, written apart from the plain forms.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32          # columns that share a scale, in the fp8 operand and in the 8-bit checkpoint
FP8_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of four sequences: grouped sigmoid router, latency only
        dict(name="route_decode", op="route", tokens=4, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, mask=False, dtype="f32", grad=False),
        # a long prompt through the same router
        dict(name="route_prompt", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, mask=False, dtype="f32", grad=False),
        # training step of a softmax router without renormalised weights (every logit has a gradient), odd sizes
        dict(name="route_train_softmax", op="route", tokens=8191, experts=60, top_k=4, score="softmax", bias=False,
             groups=1, top_groups=1, renorm=False, scale=1.0, mask=False, dtype="bf16", grad=True),
        # training step of a biased sigmoid router on a padded batch
        dict(name="route_train_padded", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=1, top_groups=1, renorm=True, scale=1.0, mask=True, dtype="f32", grad=True),
        # one decoding step: eight tokens to their experts
        dict(name="dispatch_decode", op="dispatch", tokens=8, hidden=7168, experts=256, first=0, local=256, top_k=8,
             mask=False, dtype="bf16", form="rows", grad=False),
        # training step of the routed-expert layer share: all 32 experts are here
        dict(name="dispatch_train", op="dispatch", tokens=8192, hidden=7168, experts=32, first=0, local=32, top_k=8,
             mask=False, dtype="bf16", form="rows", grad=True),
        # a prompt's rows quantized on their way to the W4A8 product, half of the experts here, padded tokens among them
        dict(name="dispatch_fp8", op="dispatch", tokens=2047, hidden=2048, experts=64, first=16, local=32, top_k=6,
             mask=True, dtype="bf16", form="fp8", grad=False),
        # one decoding step: eight tokens' expert rows summed
        dict(name="combine_decode", op="combine", tokens=8, hidden=7168, experts=256, first=0, local=256, top_k=8,
             mask=False, dtype="bf16", grad=False),
        # training step: the sum, the rows' gradients and the router weights' gradients
        dict(name="combine_train", op="combine", tokens=8192, hidden=7168, experts=32, first=0, local=32, top_k=8,
             mask=False, dtype="bf16", grad=True),
        # one decoding step's rows between the two products
        dict(name="swiglu_decode", op="swiglu", rows=64, inter=2048, tail=0, dtype="bf16", grad=False),
        # training step over the rows of the routed-expert layer share, gate and up kept in 8 bits
        dict(name="swiglu_train", op="swiglu", rows=65536, inter=2048, tail=0, dtype="bf16", grad=True),
        # the same in 16-bit halves with a smaller, odd layer and rows behind the last expert
        dict(name="swiglu_train_ragged", op="swiglu", rows=4099, inter=1408, tail=517, dtype="f16", grad=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "swiglu"])
    if op == "route":
        experts, groups = rng.choice([(8, 1), (60, 1), (64, 1), (64, 4), (96, 1), (128, 1), (160, 8), (256, 8), (256, 1), (384, 1)])
        top_groups = rng.randint(1, groups)
        score = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, groups=groups, top_groups=top_groups,
                    top_k=rng.randint(1, min(8, experts // groups * top_groups)), score=score, bias=rng.random() < 0.6,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), mask=rng.random() < 0.3,
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), grad=rng.random() < 0.5)
    if op == "swiglu":
        tokens = _log_int(rng, 1, 32768)
        return dict(op=op, rows=tokens, inter=32 * _log_int(rng, 2, 64), tail=rng.choice([0, 0, tokens // 7]),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), grad=rng.random() < 0.6)
    experts = rng.choice([8, 32, 60, 64, 128, 160, 256])
    local = rng.choice([experts, experts, experts // 2])
    case = dict(op=op, tokens=_log_int(rng, 1, 4096), hidden=0, experts=experts, local=local,
                first=rng.randint(0, experts - local), top_k=rng.randint(1, 8), mask=rng.random() < 0.3,
                dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), grad=rng.random() < 0.5)
    case["hidden"] = 32 * _log_int(rng, 8, 224)
    if op == "dispatch":
        case["form"] = rng.choice(["rows", "rows", "fp8"])
        if case["form"] == "fp8":
            case.update(grad=False, hidden=512 * rng.randint(1, 14))
    if rng.random() < 0.25 and case.get("form") != "fp8":
        case["hidden"] += rng.choice([1, 3, 8, 20])        # a hidden size of no particular multiple
    return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _assignment(case, g):
    """Experts that a router gave each token (distinct, skewed over the experts); padded tokens have none (-1)."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    liked = _randn(g, E) - torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_min(1e-9)))
    experts = torch.topk(liked, k, dim=1).indices.to(torch.int32)
    if case["mask"]:
        experts[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    return experts


def _order(experts, first, local):
    """The grouped order of the slots: cumulative counts, each slot's row (its complement if not served here), each row's slot."""
    key = experts.reshape(-1).long() - first
    key = torch.where((key >= 0) & (key < local), key, local)
    slots = torch.sort(key, stable=True).indices
    offs = torch.cumsum(torch.bincount(key, minlength=local + 1)[:local], 0)
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=slots.device)
    rows = torch.where(key < local, rows, -1 - rows)
    return offs.to(torch.int32), rows.to(torch.int32).view(experts.shape), slots.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "route":
        T, E = case["tokens"], case["experts"]
        # logits of a router: a part that all tokens share (some experts are liked more) and a token's own
        s["logits"] = (0.5 * _randn(g, E) + 1.5 * _randn(g, T, E)).to(dt)
        s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= 0.1 if case["mask"] else None
        s["grad"] = _randn(g, T, case["top_k"]) if case["grad"] else None
    elif case["op"] == "dispatch":
        T, H, k = case["tokens"], case["hidden"], case["top_k"]
        s["x"] = (_randn(g, T, H) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device="cuda"))).to(dt)
        s["experts"] = _assignment(case, g)
        s["grad"] = _randn(g, T * k, H).to(dt) if case["grad"] else None
    elif case["op"] == "combine":
        T, H, k = case["tokens"], case["hidden"], case["top_k"]
        s["y"] = _randn(g, T * k, H).to(dt)
        s["weights"] = torch.softmax(_randn(g, T, k), 1)
        s["offs"], s["rows"], s["slots"] = _order(_assignment(case, g), case["first"], case["local"])
        s["grad"] = (0.1 * _randn(g, T, H)).to(dt) if case["grad"] else None
    else:
        R, I = case["rows"], case["inter"]
        s["gate_up"] = _randn(g, R, 2 * I).to(dt)
        # eight experts' rows, and `tail` rows that belong to none
        cut = torch.sort(torch.randint(0, R - case["tail"] + 1, (7,), generator=g, device="cuda")).values
        s["offs"] = torch.cat([cut, cut.new_full((1,), R - case["tail"])]).to(torch.int32)
        s["grad"] = (0.1 * _randn(g, R, I)).to(dt) if case["grad"] else None
    return s


# -------------------------------------------------------------- plain forms
def _plain_route(s):
    """Scores, order and weights in 64 bits: which expert comes next is decided by values that lie close together."""
    c, logits = s["case"], s["logits"].double()
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.exp(logits - logits.max(1, keepdim=True).values)
    if c["score"] == "softmax":
        score = score / score.sum(1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        best = torch.sort(key.view(T, c["groups"], -1), dim=2, descending=True).values[:, :, :2].sum(2)
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=key.device).scatter_(1, chosen, True)
        keep = keep.unsqueeze(2).expand(T, c["groups"], E // c["groups"]).reshape(T, E)
        key = torch.where(keep, key, -math.inf)
    index = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    picked = torch.gather(score, 1, index)
    total = picked.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(picked[:, :1])
    weights, experts = c["scale"] * picked / total, index.to(torch.int32)
    if s["mask"] is not None:
        weights = torch.where(s["mask"][:, None], weights, 0.0)
        experts = torch.where(s["mask"][:, None], experts, -1)
    out = [weights.float(), experts]
    if s["grad"] is not None:
        gw = s["grad"].double() if s["mask"] is None else s["grad"].double() * s["mask"][:, None]
        gs = c["scale"] * gw / total
        if c["renorm"]:
            gs = gs - (gs * picked).sum(1, keepdim=True) / total
        full = torch.zeros_like(score).scatter_(1, index, gs)
        if c["score"] == "sigmoid":
            grad = full * score * (1 - score)
        else:
            grad = score * (full - (full * score).sum(1, keepdim=True))
        out.append(grad.to(s["logits"].dtype))
    return out


def _fp8_blocks(x):
    """Columns in blocks of 32 as E4M3 values under a power of two: (values, scales), float32 throughout."""
    b = x.float().view(*x.shape[:-1], -1, BLOCK)
    ratio = (b.abs().amax(-1, keepdim=True) / FP8_MAX).clamp_min(2.0 ** -126)
    mant, expo = torch.frexp(ratio)
    scale = torch.exp2((expo - (mant == 0.5).to(expo.dtype)).float())
    return (b / scale).to(torch.float8_e4m3fn), scale


def _plain_dispatch(s):
    c = s["case"]
    offs, rows, slots = _order(s["experts"], c["first"], c["local"])
    served = torch.arange(slots.numel(), device=slots.device)[:, None] < offs[-1]
    grouped = torch.where(served, s["x"][slots.long() // c["top_k"]], 0)
    if c["form"] == "fp8":
        values, scale = _fp8_blocks(grouped)
        return [offs, rows, slots, values.view(grouped.shape), scale.squeeze(-1).to(torch.float8_e8m0fnu)]
    if s["grad"] is None:
        return [offs, rows, slots, grouped]
    take = torch.where(rows >= 0, rows, 0).long()
    back = torch.where((rows >= 0)[..., None], s["grad"][take].float(), 0.0).sum(1)
    return [offs, rows, slots, grouped, back.to(s["x"].dtype)]


def _plain_combine(s):
    rows, slots, y, w = s["rows"], s["slots"].long(), s["y"], s["weights"]
    live = rows >= 0
    parts = torch.where(live[..., None], y[torch.where(live, rows, 0).long()].float(), 0.0)
    out = [(w[..., None] * parts).sum(1).to(y.dtype)]
    if s["grad"] is not None:
        g = s["grad"].float()
        served = torch.arange(slots.numel(), device=slots.device) < s["offs"][-1]
        gy = torch.where(served, w.reshape(-1)[slots], 0.0)[:, None] * g[slots // rows.shape[1]]
        out += [gy.to(y.dtype), (g[:, None, :] * parts).sum(2)]
    return out


def _plain_swiglu(s):
    gate_up, I = s["gate_up"], s["case"]["inter"]
    live = (torch.arange(gate_up.shape[0], device=gate_up.device) < s["offs"][-1])[:, None]
    g, u = gate_up.float().split(I, 1)
    out = [torch.where(live, g * torch.sigmoid(g) * u, 0.0).to(gate_up.dtype)]
    if s["grad"] is not None:
        values, scale = _fp8_blocks(gate_up)
        g, u = (values.float() * scale).view(gate_up.shape).split(I, 1)
        gh, sg = s["grad"].float(), torch.sigmoid(g)
        grad = torch.cat([gh * u * sg * (1 + g * (1 - sg)), gh * g * sg], 1)
        out.append(torch.where(live, grad, 0.0).to(gate_up.dtype))
    return out


_PLAIN = {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine, "swiglu": _plain_swiglu}


# ---------------------------------------------------------- framework's calls
def _own_route(mxq, s):
    c, grad = s["case"], s["grad"]
    logits = s["logits"] if grad is None else s["logits"].detach().requires_grad_(True)
    weights, experts = mxq.moe_route(logits, c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                     top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"],
                                     token_mask=s["mask"])
    if grad is None:
        return [weights, experts]
    return [weights.detach(), experts, torch.autograd.grad(weights, logits, grad)[0]]


def _own_dispatch(mxq, s):
    c, grad = s["case"], s["grad"]
    plan = mxq.moe_plan(s["experts"], c["experts"], first_expert=c["first"], local_experts=c["local"])
    if c["form"] == "fp8":
        codes, scales = mxq.moe_dispatch_quantized(s["x"], plan, "fp8")
        return [*plan, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)]
    if grad is None:
        return [*plan, mxq.moe_dispatch(s["x"], plan)]
    x = s["x"].detach().requires_grad_(True)
    grouped = mxq.moe_dispatch(x, plan)
    return [*plan, grouped.detach(), torch.autograd.grad(grouped, x, grad)[0]]


def _own_combine(mxq, s):
    plan, grad = mxq.MoEPlan(s["offs"], s["rows"], s["slots"]), s["grad"]
    if grad is None:
        return [mxq.moe_combine(s["y"], s["weights"], plan)]
    y, w = s["y"].detach().requires_grad_(True), s["weights"].detach().requires_grad_(True)
    out = mxq.moe_combine(y, w, plan)
    return [out.detach(), *torch.autograd.grad(out, (y, w), grad)]


def _own_swiglu(mxq, s):
    if s["grad"] is None:
        return [mxq.swiglu(s["gate_up"], s["offs"])]
    x = s["gate_up"].detach().requires_grad_(True)
    h = mxq.swiglu(x, s["offs"], checkpoint="fp8")
    return [h.detach(), torch.autograd.grad(h, x, s["grad"])[0]]


_OWN = {"route": _own_route, "dispatch": _own_dispatch, "combine": _own_combine, "swiglu": _own_swiglu}


def run(state):
    op = state["case"]["op"]
    if own:
        import nvfp4_quantization_grouped_amd as mxq
        return _OWN[op](mxq, state)
    return _PLAIN[op](state)


# --------------------------------------------------------------------- work
def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        fwd, bwd = T * E * b + T * k * 8, T * k * 4 + T * E * b
        return {"bytes": fwd + (bwd if case["grad"] else 0), "flops": T * E * (12 if case["grad"] else 6)}
    if case["op"] == "swiglu":
        n = (case["rows"] - case["tail"]) * case["inter"]
        h, gate_up = case["rows"] * case["inter"] * b, 2 * n * b
        if not case["grad"]:
            return {"bytes": gate_up + h, "flops": 6 * n}
        kept = 2 * n * (1 + 1 / BLOCK)                # the checkpoint is written by the forward and read by the backward
        return {"bytes": gate_up + h + 2 * kept + n * b + 2 * case["rows"] * case["inter"] * b, "flops": 20 * n}
    T, H, N = case["tokens"], case["hidden"], case["tokens"] * case["top_k"]
    live = N * case["local"] / case["experts"] * (0.9 if case["mask"] else 1.0)      # rows that belong here, on average
    if case["op"] == "dispatch":
        row = H * b if case["form"] == "rows" else H + H // BLOCK
        grad = live * H * b + T * H * b if case["grad"] else 0
        return {"bytes": T * H * b + N * row + 12 * N + grad, "flops": live * H if case["grad"] else N}
    fwd = live * H * b + T * H * b + 8 * N
    grad = T * H * b + N * H * b + 4 * N if case["grad"] else 0
    return {"bytes": fwd + grad, "flops": live * H * (5 if case["grad"] else 2)}


# ------------------------------------------------------- definitions, 64 bits
def _ranked(value, count):
    """The `count` largest along the last axis, equal ones by their place: each one's rank is the number of those before it."""
    rank = torch.argsort(torch.argsort(-value, dim=-1, stable=True), dim=-1)
    return rank < count, rank


def _exact_route(s):
    c = s["case"]
    x = s["logits"].to(torch.float64)
    p = 1 / (1 + torch.exp(-x)) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    key = p + s["bias"].to(torch.float64) if c["bias"] else p
    ok = torch.ones_like(key, dtype=torch.bool)
    if c["groups"] > 1:
        shape = (c["tokens"], c["groups"], c["experts"] // c["groups"])
        two, _ = _ranked(key.view(shape), 2)
        chosen, _ = _ranked(torch.where(two, key.view(shape), 0).sum(2), c["top_groups"])
        ok = chosen.repeat_interleave(shape[2], 1)
    if c["mask"]:
        alive = s["mask"][:, None].to(torch.float64)
    else:
        alive = torch.ones_like(x[:, :1])
    taken, rank = _ranked(torch.where(ok, key, -torch.inf), c["top_k"])
    index = torch.argsort(torch.where(taken, rank, c["experts"]), dim=1)[:, : c["top_k"]]
    inside = p * taken
    norm = inside.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(alive)
    all_w = c["scale"] * inside / norm * alive
    out = [all_w.gather(1, index), torch.where(alive > 0, index, -1).to(torch.int32)]
    if c["grad"]:
        g = torch.zeros_like(x).scatter_add_(1, index, s["grad"].to(torch.float64)) * alive
        # through w = scale p / norm, then through p
        dp = taken * (c["scale"] * g - ((g * all_w).sum(1, keepdim=True) if c["renorm"] else 0)) / norm
        out.append(dp * p * (1 - p) if c["score"] == "sigmoid" else dp * p - p * (dp * p).sum(1, keepdim=True))
    return out


def _exact_e4m3(v):
    """Nearest E4M3 value of v (|v| <= 448), ties to even: a multiple of 2^-3 of its own power of two, of 2^-9 below 2^-6."""
    power = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    power = torch.where(torch.exp2(power) > v.abs().clamp_min(2.0 ** -6), power - 1, power)
    step = torch.exp2(power - 3)
    return torch.round(v / step) * step


def _exact_blocks(x):
    v = x.to(torch.float64).unflatten(-1, (-1, BLOCK))
    top = v.abs().max(-1, keepdim=True).values
    power = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / FP8_MAX)).clamp_min(-126)
    power = torch.where(torch.exp2(power - 1) * FP8_MAX >= top, (power - 1).clamp_min(-126), power)
    scale = torch.exp2(power)
    return _exact_e4m3(v / scale), scale


def _exact_order(experts, first, local):
    flat = experts.reshape(-1).to(torch.int64)
    here = (flat >= first) & (flat < first + local)
    place = torch.where(here, flat - first, local) * flat.numel() + torch.arange(flat.numel(), device=flat.device)
    slots = torch.argsort(place)
    row = torch.argsort(slots)
    upto = torch.arange(1, local + 1, device=flat.device) * flat.numel()
    offs = torch.searchsorted(place[slots], upto)
    return offs.to(torch.int32), torch.where(here, row, ~row).to(torch.int32).view(experts.shape), slots.to(torch.int32)


def _exact_dispatch(s):
    c = s["case"]
    offs, rows, slots = _exact_order(s["experts"], c["first"], c["local"])
    grouped = s["x"].to(torch.float64).repeat_interleave(c["top_k"], 0)[slots.long()]
    grouped[int(offs[-1]):] = 0
    if c["form"] == "fp8":
        values, scale = _exact_blocks(grouped)
        return [offs, rows, slots, values.flatten(-2), scale.squeeze(-1)]
    if not c["grad"]:
        return [offs, rows, slots, grouped]
    back = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=grouped.device)
    n = int(offs[-1])
    back.index_add_(0, slots[:n].long() // c["top_k"], s["grad"][:n].to(torch.float64))
    return [offs, rows, slots, grouped, back]


def _exact_combine(s):
    T, k = s["rows"].shape
    n, H = int(s["offs"][-1]), s["y"].shape[1]
    slot = s["slots"][:n].long()
    w = s["weights"].to(torch.float64).reshape(-1)[slot]
    y = s["y"][:n].to(torch.float64)
    out = [torch.zeros(T, H, dtype=torch.float64, device=y.device).index_add_(0, slot // k, w[:, None] * y)]
    if s["grad"] is not None:
        g = s["grad"].to(torch.float64)[slot // k]
        gy = torch.zeros(T * k, H, dtype=torch.float64, device=y.device)
        gy[:n] = w[:, None] * g
        gw = torch.zeros(T * k, dtype=torch.float64, device=y.device)
        gw[slot] = (g * y).sum(1)
        out += [gy, gw.view(T, k)]
    return out


def _exact_swiglu(s):
    x, n = s["gate_up"], int(s["offs"][-1])
    I = s["case"]["inter"]
    v = x.to(torch.float64)
    h = v[:, :I] / (1 + torch.exp(-v[:, :I])) * v[:, I:]
    h[n:] = 0
    if s["grad"] is None:
        return [h]
    values, scale = _exact_blocks(x)
    v = (values * scale).flatten(-2)
    gate, up, gh = v[:, :I], v[:, I:], s["grad"].to(torch.float64)
    e = torch.exp(-gate)
    grad = torch.empty_like(v)
    grad[:, :I] = gh * up * (1 + e + gate * e) / (1 + e) ** 2
    grad[:, I:] = gh * gate / (1 + e)
    grad[n:] = 0
    return [h, grad]


_EXACT = {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine, "swiglu": _exact_swiglu}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
