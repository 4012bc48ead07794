"""The operators around a routed MoE layer, case by case: rows sorted by
expert and back with their gradients, the router's gradient, and products in
8-bit integers with a scale per token and per channel.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through block_quantized_expert_amd.  Common notation: token t has top_k slots,
f = t*top_k + i is the flat index of slot i; slots sorted by expert (stably)
are rows p, perm[p] = f, inv_perm[f] = p; a dropped slot (expert id -1) has no
row, and the rows behind the last expert's are zero.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
ROUTED_SCALE = 1.5


# ---------------------------------------------------------------- cases


def listed():
    return [
        # prefill of 4096 tokens through 256 experts, top-6: rows copied into
        # expert order (one read of a token, six writes)
        dict(name="dispatch_4096", kind="dispatch", back=False, n=4096, k=6, e=256, used=256,
             drop=0, hidden=4096, dtype="bf16"),
        # its gradient at sizes that divide nothing, fp32 as in a check of a
        # training run, with slots dropped by tail pruning
        dict(name="dispatch_back_odd", kind="dispatch", back=True, n=1237, k=5, e=37, used=33,
             drop=611, hidden=2059, dtype="f32"),
        # the end of a layer for one decoded token: six expert outputs and the
        # shared expert's, where only latency counts
        dict(name="combine_1", kind="combine", back=False, n=1, k=6, e=256, used=6, drop=0,
             hidden=4096, dtype="bf16", base=True),
        # a training batch of 4096 tokens: gradients of the expert outputs and
        # of the routing weights in one pass
        dict(name="combine_back_4096", kind="combine", back=True, n=4096, k=6, e=256, used=256,
             drop=0, hidden=4096, dtype="bf16", base=False),
        # the same in fp32 at odd sizes with dropped slots
        dict(name="combine_back_odd", kind="combine", back=True, n=777, k=3, e=19, used=17,
             drop=200, hidden=1001, dtype="f32", base=False),
        # router gradient of the training batch, and of a small odd one
        dict(name="route_back_4096", kind="route_back", n=4096, k=6, e=256),
        dict(name="route_back_13", kind="route_back", n=13, k=3, e=101),
        # one decoded token through int8 gate and up of its six experts: the
        # weights stream from memory
        dict(name="gate_up_1", kind="gate_up", n=1, k=6, e=256, used=6, drop=0, cols=4096,
             out=2048, dtype="bf16"),
        # prefill of 4096 tokens through the gate and up of 256 experts
        dict(name="gate_up_4096", kind="gate_up", n=4096, k=6, e=256, used=256, drop=0,
             cols=4096, out=2048, dtype="bf16"),
        # 32 decoded tokens through the down projection of the experts that
        # they reach, a few rows for each
        dict(name="down_32", kind="down", n=32, k=6, e=256, used=120, drop=0, cols=2048,
             out=4096, dtype="bf16"),
        # a dense projection over a prefill batch: bound by the matrix cores
        dict(name="linear_4096", kind="linear", n=4096, cols=4096, out=4096, dtype="bf16"),
        # a dense projection of a ragged batch at sizes that fill no tile, fp32 in and out
        dict(name="linear_odd", kind="linear", n=333, cols=2064, out=1235, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _routing(rng, n):
    e = _log_int(rng, 8, 256)
    k = rng.randint(1, min(8, e))
    used = rng.randint(k, max(k, min(e, n * k)))
    drop = rng.randint(0, n * (k - 1) // 2) if rng.random() < 0.4 else 0
    return e, k, used, drop


def draw(rng):
    """One more case of the listed ones' ranges."""
    kind = rng.choice(["dispatch", "combine", "route_back", "gate_up", "down", "linear"])
    dtype = rng.choice(["bf16", "f32"])
    n = _log_int(rng, 1, 4096)
    e, k, used, drop = _routing(rng, n)
    if kind == "route_back":
        return dict(kind=kind, n=n, k=k, e=e)
    if kind in ("dispatch", "combine"):
        hidden = _log_int(rng, 64, 4096)
        if rng.random() < 0.5:
            hidden -= hidden % 64
        case = dict(kind=kind, back=rng.random() < 0.5, n=n, k=k, e=e, used=used, drop=drop,
                    hidden=hidden, dtype=dtype)
        if kind == "combine":
            case["base"] = not case["back"] and rng.random() < 0.5
        return case
    cols = 16 * _log_int(rng, 8, 256)  # rows of int8 are whole 16-byte words
    out = _log_int(rng, 64, 4096 if kind == "linear" else 2048)
    if rng.random() < 0.5:
        out -= out % 64
    if kind == "linear":
        return dict(kind=kind, n=n, cols=cols, out=out, dtype=dtype)
    k = min(k, 6)
    return dict(kind=kind, n=n, k=k, e=e, used=max(k, min(used, n * k)),
                drop=min(drop, n * (k - 1) // 2), cols=cols, out=out, dtype=dtype)


def work(case):
    """Bytes and operations that a pass cannot do without: every input read
    once and every output written once; only the experts with rows count."""
    kind, n = case["kind"], case["n"]
    if kind == "route_back":
        return {"bytes": 4 * n * case["e"] + 12 * n * case["k"], "flops": 20 * n * case["k"]}
    s = SIZE[case["dtype"]]
    if kind in ("dispatch", "combine"):
        h, slots = case["hidden"], n * case["k"]
        kept = slots - case["drop"]
        if kind == "dispatch":
            if case["back"]:
                return {"bytes": (kept + n) * h * s + 4 * slots, "flops": kept * h}
            return {"bytes": (n + slots) * h * s + 4 * slots, "flops": 0}
        if case["back"]:
            return {"bytes": (n + kept + slots) * h * s + 12 * slots, "flops": 3 * kept * h}
        return {"bytes": (kept + n * (2 if case["base"] else 1)) * h * s + 8 * slots,
                "flops": 2 * kept * h}
    c, r = case["cols"], case["out"]
    if kind == "linear":
        return {"bytes": n * c * s + r * (c + 4) + n * r * s, "flops": 2 * n * c * r}
    slots = n * case["k"]
    kept = slots - case["drop"]
    mats = 2 if kind == "gate_up" else 1
    rows_in = n if kind == "gate_up" else slots
    return {"bytes": rows_in * c * s + mats * case["used"] * r * (c + 4) + slots * r * s + 4 * slots,
            "flops": 2 * mats * kept * c * r}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _grouping(case, g):
    """Expert ids of every slot (distinct within a token, every one of `used`
    experts reached, popularity falling with rank; exactly `drop` slots
    without an expert) and the sorted order."""
    n, k, e, used, drop = (case[i] for i in ("n", "k", "e", "used", "drop"))
    pool = torch.randperm(e, generator=g, device="cuda")[:used]
    rank = torch.arange(1, used + 1, device="cuda", dtype=torch.float32)
    score = -0.33 * rank.log() - (-torch.rand(n, used, generator=g, device="cuda").clamp(
        1e-7, 1 - 1e-6).log()).log()
    pick = score.topk(k, dim=1).indices
    first = min(n, -(-used // k))  # tokens that reach the pool one expert after the other
    turn = torch.arange(first * k, device="cuda").reshape(first, k) % used
    pick[:first] = turn
    ids = pool[pick][torch.randperm(n, generator=g, device="cuda")]
    if drop:  # never a token's first slot
        slots = torch.arange(n * k, device="cuda").reshape(n, k)[:, 1:].reshape(-1)
        gone = slots[torch.randperm(slots.numel(), generator=g, device="cuda")[:drop]]
        ids.view(-1)[gone] = -1
    flat = ids.reshape(-1)
    order = torch.where(flat < 0, e, flat).argsort(stable=True)
    total = n * k - drop
    counts = torch.bincount(flat[flat >= 0], minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    inv = torch.full((n * k,), -1, dtype=torch.int64, device="cuda")
    inv[order[:total]] = torch.arange(total, device="cuda")
    perm = order.clone()
    perm[total:] = 0
    return ids.int(), tuple(t.int() for t in (counts, offsets, perm, inv)), offsets.tolist()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, n, c, dtype):
    """Normal values with a few channels an order of magnitude larger, as
    hidden states have them."""
    x = _normal(g, n, c)
    x[:, torch.randint(0, c, (max(1, c // 256),), generator=g, device="cuda")] *= 12
    return x.to(DTYPES[dtype])


def _weight(g, e, r, c):
    """int8 rows spread like a normal's, largest value 127, a scale per row."""
    q = torch.empty(e, r, c, dtype=torch.int8, device="cuda")
    for i in range(0, e, 32):
        part = q[i:i + 32]
        part.copy_(_normal(g, *part.shape).mul_(30).round_().clamp_(-127, 127))
    scale = (1 + torch.rand(e, r, generator=g, device="cuda")) / (60 * math.sqrt(c))
    return q, scale


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    kind, n = case["kind"], case["n"]
    if kind == "route_back":
        st["logits"] = _normal(g, n, case["e"]) * 1.5
        st["ids"] = st["logits"].topk(case["k"], dim=1).indices.int()
        st["dw"] = _normal(g, n, case["k"])
    elif kind == "linear":
        st["x"] = _activations(g, n, case["cols"], case["dtype"])
        st["weights"] = [_weight(g, 1, case["out"], case["cols"])]
    else:
        k = case["k"]
        st["ids"], st["grouping"], st["bounds"] = _grouping(case, g)
        w = torch.rand(n, k, generator=g, device="cuda") + 0.05
        w = w.masked_fill(st["ids"] < 0, 0)
        st["w"] = ROUTED_SCALE * w / w.sum(1, keepdim=True)
        if kind in ("dispatch", "combine"):
            dt, h = DTYPES[case["dtype"]], case["hidden"]
            st["tokens"] = _normal(g, n, h).to(dt)  # x or dy
            st["rows"] = _normal(g, n * k, h).to(dt)  # expert outputs or their gradients
            st["base"] = _normal(g, n, h).to(dt) if case.get("base") else None
        else:
            rows = n if kind == "gate_up" else n * k
            st["x"] = _activations(g, rows, case["cols"], case["dtype"])
            st["weights"] = [_weight(g, case["e"], case["out"], case["cols"])
                             for _ in range(2 if kind == "gate_up" else 1)]
    if own and "weights" in st:
        from block_quantized_expert_amd import binding as B

        st["handles"] = [B.Int8Weight(q, s) for q, s in st["weights"]]
    return st


# ---------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from block_quantized_expert_amd import binding as B

    case = st["case"]
    kind = case["kind"]
    if kind == "route_back":
        return B.moe_route_backward(st["logits"], st["ids"], st["dw"], ROUTED_SCALE)
    if kind == "dispatch":
        if case["back"]:
            return B.moe_dispatch_backward(st["rows"], st["grouping"], case["k"])
        return B.moe_dispatch(st["tokens"], st["grouping"], case["k"])
    if kind == "combine":
        if case["back"]:
            return B.moe_combine_backward(st["tokens"], st["rows"], st["w"], st["grouping"])
        return B.moe_combine(st["rows"], st["w"], st["grouping"], base=st["base"])
    q, scale = B.moe_quantize_int8(st["x"])
    dt = DTYPES[case["dtype"]]
    if kind == "linear":
        return B.moe_product_int8(st["handles"][0], q, scale, out_dtype=dt)
    if kind == "down":
        return B.moe_product_int8(st["handles"][0], q, scale, st["grouping"], out_dtype=dt)
    return B.moe_swiglu_int8(st["handles"][0], st["handles"][1], q, scale, st["grouping"],
                             top_k=case["k"], out_dtype=dt)


def _quantize(x):
    """Whole numbers q (ties to even, taken in 64 bits: they lie next to a
    border) and fp32 scales with x ~ q * scale."""
    x = x.float()
    a = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(a > 0, (x.double() * 127 / a.double()).round(), 0.0).float()
    return q, a / 127


def _run_plain(st):
    case = st["case"]
    kind, n = case["kind"], case["n"]
    if kind == "route_back":  # 64 bits, as the router's own weights
        c, ids = ROUTED_SCALE, st["ids"].long()
        l = st["logits"].gather(1, ids).double()
        s = (l.clamp_min(0) + torch.log1p((-l.abs()).exp())).sqrt()
        total = s.sum(1, keepdim=True)
        dw = st["dw"].double()
        # sum_j s_j (dw_i - dw_j): nothing is left to cancel, and one slot gives zero
        ds = c / total**2 * sum(s[:, j:j + 1] * (dw - dw[:, j:j + 1]) for j in range(case["k"]))
        dl = ds / (1 + (-l).exp()) / (2 * s)
        return torch.zeros_like(st["logits"]).scatter_(1, ids, dl.float())
    if kind in ("dispatch", "combine"):
        return _plain_rows(st)
    dt = DTYPES[case["dtype"]]
    q, scale = _quantize(st["x"])
    if kind == "linear":
        wq, ws = st["weights"][0]
        return ((q @ wq[0].float().t()) * scale * ws[0]).to(dt)
    perm, bounds = st["grouping"][2].long(), st["bounds"]
    out = torch.zeros(n * case["k"], case["out"], dtype=dt, device="cuda")
    for e in range(case["e"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        r = perm[a:b] // case["k"] if kind == "gate_up" else slice(a, b)
        ye = [(q[r] @ wq[e].float().t()) * scale[r] * ws[e] for wq, ws in st["weights"]]
        if kind == "gate_up":
            out[a:b] = (ye[0] / (1 + (-ye[0]).exp()) * ye[1]).to(dt)
        else:
            out[a:b] = ye[0].to(dt)
    return out


def _plain_rows(st):
    case = st["case"]
    n, k, h = case["n"], case["k"], case["hidden"]
    dt = DTYPES[case["dtype"]]
    _, offsets, perm, inv = st["grouping"]
    live = (torch.arange(n * k, device="cuda") < offsets[-1]).unsqueeze(1)
    f = perm.long()
    if case["kind"] == "dispatch" and not case["back"]:
        return torch.where(live, st["tokens"].float()[f // k], 0.0).to(dt)
    if case["kind"] == "combine" and case["back"]:
        dy = st["tokens"].float()
        drows = torch.where(live, st["w"].reshape(-1, 1)[f] * dy[f // k], 0.0).to(dt)
        at = inv.long().clamp_min(0)
        dots = (st["rows"].float()[at].reshape(n, k, h) * dy.unsqueeze(1)).sum(2)
        return drows, torch.where(inv.reshape(n, k) >= 0, dots, 0.0)
    y = torch.zeros(n, h, device="cuda") if st["base"] is None else st["base"].float()
    inv = inv.reshape(n, k).long()
    for i in range(k):
        rows = st["rows"].float()[inv[:, i].clamp_min(0)]
        if case["kind"] == "combine":
            rows = rows * st["w"][:, i:i + 1]
        y = y + torch.where(inv[:, i:i + 1] >= 0, rows, 0.0)
    return y.to(dt)


# ---------------------------------------------------------------- exact values


def exact(case, seed):
    """The definitions in 64 bits, from the expert ids alone."""
    st = prepare(case, seed)
    kind, n = case["kind"], case["n"]
    if kind == "route_back":  # Jacobian of the weights times that of the scores
        l = st["logits"].double()
        s = (1 + l.exp()).log().sqrt()
        slope = 0.5 * (1 + torch.tanh(l / 2)) / (2 * s)
        ids = st["ids"].long()
        si, d = s.gather(1, ids), st["dw"].double()
        p = si / si.sum(1, keepdim=True)
        # d w_i / d s_j = c/S (delta_ij - p_i), with delta_ij = delta_ij sum_m p_m
        pull = ((d.unsqueeze(2) - d.unsqueeze(1)) * p.unsqueeze(1)).sum(2)
        ds = ROUTED_SCALE * pull / si.sum(1, keepdim=True)
        return torch.zeros_like(l).scatter_(1, ids, ds * slope.gather(1, ids))

    def quantized(x):
        x = x.double()
        step = x.abs().amax(1, keepdim=True) / 127
        top = step * 127
        return torch.round(torch.where(top > 0, x * 127 / x.abs().amax(1, keepdim=True), 0)), step

    if kind == "linear":
        q, step = quantized(st["x"])
        wq, ws = st["weights"][0]
        return torch.mm(q, wq[0].double().t().contiguous()) * step * ws[0].double()
    k = case["k"]
    flat = st["ids"].reshape(-1).tolist()
    order = sorted((e, f) for f, e in enumerate(flat) if e >= 0)  # row p -> (expert, slot)
    slot = torch.tensor([f for _, f in order], device="cuda")
    live = len(order)
    if kind in ("dispatch", "combine"):
        h = case["hidden"]
        tokens, rows = st["tokens"].double(), st["rows"].double()
        w = st["w"].double().reshape(-1)
        if kind == "dispatch" and not case["back"]:
            out = torch.zeros(n * k, h, dtype=torch.float64, device="cuda")
            out[:live] = tokens[slot // k]
            return out
        if case["back"] and kind == "combine":
            out = torch.zeros(n * k, h, dtype=torch.float64, device="cuda")
            dw = torch.zeros(n * k, dtype=torch.float64, device="cuda")
            for a in range(0, live, 4096):
                s = slot[a:a + 4096]
                out[a:a + 4096][:s.numel()] = tokens[s // k] * w[s].unsqueeze(1)
                dw[s] = (tokens[s // k] * rows[a:a + s.numel()]).sum(1)
            return out, dw.reshape(n, k)
        y = torch.zeros(n, h, dtype=torch.float64, device="cuda")
        if kind == "combine" and st["base"] is not None:
            y += st["base"].double()
        factor = w[slot].unsqueeze(1) if kind == "combine" else 1.0
        return y.index_add_(0, slot // k, rows[:live] * factor)
    q, step = quantized(st["x"])
    out = torch.zeros(n * k, case["out"], dtype=torch.float64, device="cuda")
    a = 0
    while a < live:
        e = order[a][0]
        b = a
        while b < live and order[b][0] == e:
            b += 1
        r = slot[a:b] // k if kind == "gate_up" else torch.arange(a, b, device="cuda")
        y = [torch.mm(q[r], wq[e].double().t().contiguous()) * step[r] * ws[e].double()
             for wq, ws in st["weights"]]
        out[a:b] = y[0] * torch.sigmoid(y[0]) * y[1] if kind == "gate_up" else y[0]
        a = b
    return out
