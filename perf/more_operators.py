"""The operators in front of a layer's products and in 4 bits, case by case:
the root-mean-square norm with the residual's addition (its outputs in 16 or 32
bits, in int8 with a scale per row, in MXFP4), its gradients, rounding to MXFP4
and back, and products of MXFP4 rows by MXFP4 weights, dense and grouped by
expert.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through block_quantized_expert_amd.  MXFP4: E2M1 values in blocks of 32 under a
power of two, 2^(byte - 127); two codes a byte, the first in the low bits.  A
row's scale bytes are padded to whole 16-byte words.  Slots sorted by expert
(stably) are rows p, perm[p] = f = t*top_k + i; a dropped slot (expert id -1)
has no row, and the rows behind the last expert's are zero.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decoded token between two layers: the residual's addition and the
        # norm in front of the router, where only latency counts
        dict(name="norm_1", kind="norm", n=1, h=4096, dtype="bf16", residual=True, out="same"),
        # the same for a prefill or training batch of 4096 tokens
        dict(name="norm_4096", kind="norm", n=4096, h=4096, dtype="bf16", residual=True,
             out="same"),
        # the norm in front of int8 products, a ragged batch in fp32
        dict(name="norm_int8_777", kind="norm", n=777, h=2064, dtype="f32", residual=True,
             out="int8"),
        # the training batch's gradients, the residual stream's added
        dict(name="norm_back_4096", kind="norm_back", n=4096, h=4096, dtype="bf16", total=True),
        # gradients at sizes that divide nothing, fp32 as in a check of a training run
        dict(name="norm_back_odd", kind="norm_back", n=1001, h=2059, dtype="f32", total=False),
        # weights rounded to MXFP4 and looked at again: a matrix of an expert, twice over
        dict(name="cast_8192", kind="cast", n=8192, c=4096, dtype="bf16"),
        # a small ragged batch of activations
        dict(name="cast_odd", kind="cast", n=333, c=2080, dtype="f32"),
        # 32 decoded tokens: norm, rounding and a dense projection
        dict(name="linear_32", kind="linear", n=32, c=4096, out=4096, dtype="bf16", norm=True),
        # a dense projection of a prefill batch: bound by the matrix cores
        dict(name="linear_4096", kind="linear", n=4096, c=4096, out=4096, dtype="bf16",
             norm=False),
        # a ragged batch at sizes that fill no tile, fp32 in and out
        dict(name="linear_odd", kind="linear", n=333, c=2080, out=1235, dtype="f32", norm=False),
        # one decoded token through gate and up of its six experts: the weights
        # stream from memory
        dict(name="gate_up_1", kind="gate_up", n=1, k=6, e=256, used=6, drop=0, c=4096, out=2048,
             dtype="bf16"),
        # prefill of 4096 tokens through the gate and up of 256 experts
        dict(name="gate_up_4096", kind="gate_up", n=4096, k=6, e=256, used=256, drop=0, c=4096,
             out=2048, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    kind = rng.choice(["norm", "norm", "norm_back", "cast", "linear", "linear", "gate_up", "down"])
    dtype = rng.choice(["bf16", "f32"])
    n = _log_int(rng, 1, 4096)
    if kind in ("norm", "norm_back"):
        h = _log_int(rng, 64, 8192)
        if kind == "norm_back":
            return dict(kind=kind, n=n, h=h, dtype=dtype, total=rng.random() < 0.5)
        out = rng.choice(["same", "int8"])
        if out == "int8" or rng.random() < 0.5:
            h -= h % 16  # rows of int8 are whole 16-byte words
        return dict(kind=kind, n=n, h=h, dtype=dtype, residual=rng.random() < 0.6, out=out)
    c = 32 * _log_int(rng, 2, 128)
    if kind == "cast":
        return dict(kind=kind, n=_log_int(rng, 1, 8192), c=c, dtype=dtype)
    out = _log_int(rng, 64, 4096 if kind == "linear" else 2048)
    if rng.random() < 0.5:
        out -= out % 64
    if kind == "linear":
        return dict(kind=kind, n=n, c=c, out=out, dtype=dtype, norm=rng.random() < 0.4)
    e = _log_int(rng, 8, 256)
    k = rng.randint(1, 6)
    used = rng.randint(k, max(k, min(e, n * k)))
    drop = rng.randint(0, n * (k - 1) // 2) if rng.random() < 0.4 else 0
    return dict(kind=kind, n=n, k=k, e=e, used=used, drop=drop, c=c, out=out, dtype=dtype)


def work(case):
    """Bytes and operations that a pass cannot do without: every input read
    once and every output written once; only the experts with rows count."""
    kind, n, s = case["kind"], case["n"], SIZE[case["dtype"]]
    if kind == "norm":
        h = case["h"]
        out = s if case["out"] == "same" else 1
        return {"bytes": n * h * (s + (2 * s if case["residual"] else 0) + out) + 4 * h,
                "flops": 6 * n * h}
    if kind == "norm_back":
        h = case["h"]
        return {"bytes": n * h * s * (4 if case["total"] else 3) + 8 * h, "flops": 12 * n * h}
    c = case["c"]
    packed = c // 2 + c // 32  # a row in MXFP4
    if kind == "cast":
        return {"bytes": n * (2 * c * s + packed), "flops": 4 * n * c}
    r = case["out"]
    if kind == "linear":
        return {"bytes": n * c * s + r * packed + n * r * s, "flops": 2 * n * c * r}
    slots = n * case["k"]
    kept = slots - case["drop"]
    mats = 2 if kind == "gate_up" else 1
    rows_in = n if kind == "gate_up" else slots
    return {"bytes": rows_in * c * s + mats * case["used"] * r * packed + slots * r * s + 4 * slots,
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
    pick[:first] = torch.arange(first * k, device="cuda").reshape(first, k) % used
    ids = pool[pick][torch.randperm(n, generator=g, device="cuda")]
    if drop:  # never a token's first slot
        slots = torch.arange(n * k, device="cuda").reshape(n, k)[:, 1:].reshape(-1)
        ids.view(-1)[slots[torch.randperm(slots.numel(), generator=g, device="cuda")[:drop]]] = -1
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
    return tuple(t.int() for t in (counts, offsets, perm, inv)), ids, offsets.tolist()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, n, c, dtype):
    """Normal values with a few channels an order of magnitude larger, as
    hidden states have them."""
    x = _normal(g, n, c)
    x[:, torch.randint(0, c, (max(1, c // 256),), generator=g, device="cuda")] *= 12
    return x.to(DTYPES[dtype])


def _codes_of_normals():
    """256 bytes -> E2M1 codes spread like a normal's in a block whose largest
    value is about 5."""
    v = torch.special.ndtri((torch.arange(256, dtype=torch.float64) + 0.5) / 256) * 2.2
    mags = torch.tensor(E2M1, dtype=torch.float64)
    code = torch.bucketize(v.abs(), (mags[1:] + mags[:-1]) / 2)
    return (code + 8 * (v < 0)).to(torch.uint8).cuda()


def _weight(g, e, r, c):
    """MXFP4 rows: codes uint8 [e][r][c/2], scale bytes uint8 [e][r][c/32
    padded to 16]; values of about 1/sqrt(c)."""
    lut = _codes_of_normals()
    codes = torch.empty(e, r, c // 2, dtype=torch.uint8, device="cuda")
    for i in range(0, e, 16):
        part = codes[i:i + 16]
        lo, hi = (lut[torch.randint(0, 256, part.shape, generator=g, device="cuda",
                                    dtype=torch.int32)] for _ in range(2))
        part.copy_(lo | (hi << 4))
    mid = 127 + int(round(math.log2(1 / (2.2 * math.sqrt(c)))))
    scales = torch.zeros(e, r, 16 * -(-c // 512), dtype=torch.uint8, device="cuda")
    scales[..., :c // 32] = torch.randint(mid - 1, mid + 2, (e, r, c // 32), generator=g,
                                          device="cuda", dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    kind, n = case["kind"], case["n"]
    if kind in ("norm", "norm_back"):
        h, dt = case["h"], DTYPES[case["dtype"]]
        st["w"] = 1 + 0.2 * _normal(g, h)
        st["x"] = _activations(g, n, h, case["dtype"])
        if kind == "norm":
            st["residual"] = (_normal(g, n, h) * 2).to(dt) if case["residual"] else None
        else:
            st["dy"] = _normal(g, n, h).to(dt)
            st["dtotal"] = _normal(g, n, h).to(dt) if case["total"] else None
        return st
    c = case["c"]
    if kind == "cast":
        st["x"] = _activations(g, n, c, case["dtype"])
        return st
    if kind == "linear":
        st["x"] = _activations(g, n, c, case["dtype"])
        st["weights"] = [_weight(g, 1, case["out"], c)]
        st["w"] = 1 + 0.2 * _normal(g, c)
    else:
        st["grouping"], st["ids"], st["bounds"] = _grouping(case, g)
        rows = n if kind == "gate_up" else n * case["k"]
        st["x"] = _activations(g, rows, c, case["dtype"])
        st["weights"] = [_weight(g, case["e"], case["out"], c)
                         for _ in range(2 if kind == "gate_up" else 1)]
    if own:
        from block_quantized_expert_amd import binding as B

        st["handles"] = [B.Mxfp4Weight(*w) for w in st["weights"]]
    return st


# ---------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from block_quantized_expert_amd import binding as B

    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        if case["out"] == "same":
            return B.moe_rmsnorm(st["x"], st["w"], EPS, residual=st["residual"])
        q, scale, *total = B.moe_rmsnorm_int8(st["x"], st["w"], EPS, residual=st["residual"])
        return (q * scale.unsqueeze(1), *total)
    if kind == "norm_back":
        return B.moe_rmsnorm_backward(st["dy"], st["x"], st["w"], EPS, dtotal=st["dtotal"])
    dt = DTYPES[case["dtype"]]
    if kind == "cast":
        return B.moe_dequantize_mxfp4(*B.moe_quantize_mxfp4(st["x"]), dtype=dt)
    if case.get("norm"):
        rows = B.moe_rmsnorm_mxfp4(st["x"], st["w"], EPS)
    else:
        rows = B.moe_quantize_mxfp4(st["x"])
    if kind == "linear":
        return B.moe_product_mxfp4(st["handles"][0], *rows, out_dtype=dt)
    if kind == "down":
        return B.moe_product_mxfp4(st["handles"][0], *rows, st["grouping"], out_dtype=dt)
    return B.moe_swiglu_mxfp4(*st["handles"], *rows, st["grouping"], top_k=case["k"],
                              out_dtype=dt)


def _normed(s, w):
    """The norm in 64 bits, rounded to fp32: what is rounded further lies next
    to borders."""
    s = s.double()
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
    return (s * r * w.double()).float()


def _mxfp4(x):
    """fp32 values of x rounded to MXFP4: a block's scale is 2^(floor(log2 of
    its largest magnitude) - 2), values go to the nearest of E2M1 (ties to
    even), those past 6 to 6."""
    blocks = x.float().reshape(x.shape[0], -1, 32)
    top = torch.frexp(blocks.abs().amax(2, keepdim=True)).exponent - 3
    scale = torch.ldexp(torch.ones_like(blocks[..., :1]), top.clamp(-125, 125))
    v = blocks / scale
    m = v.abs().clamp_max(6)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (m / step).round() * step
    return (torch.copysign(m, v) * scale).reshape(x.shape)


def _table():
    """Byte -> its two values."""
    v = torch.tensor(E2M1 + [-m for m in E2M1], device="cuda")
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b & 15], v[b >> 4]], 1)


def _values(codes, scales, table):
    """fp32 values of one matrix in MXFP4."""
    v = table[codes.int()].reshape(codes.shape[0], -1, 32)
    s = torch.exp2(scales[:, :v.shape[1]].float() - 127)
    return (v * s.unsqueeze(2)).reshape(codes.shape[0], -1)


def _run_plain(st):
    case = st["case"]
    kind, n = case["kind"], case["n"]
    dt = DTYPES[case["dtype"]]
    if kind == "norm":
        s, total = st["x"], ()
        if st["residual"] is not None:
            s = (s.float() + st["residual"].float()).to(dt)
            total = (s,)
        if case["out"] == "int8":
            y = _normed(s, st["w"])
            a = y.abs().amax(1, keepdim=True)
            q = (y.double() * 127 / a.double()).round().float()
            return (q * (a / 127), *total)
        f = s.float()
        y = (f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * st["w"]).to(dt)
        return (y, *total) if total else y
    if kind == "norm_back":
        s, dy = st["x"].float(), st["dy"].float()
        r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
        g = dy * st["w"]
        ds = r * g - s * (r * r * r * (s * g).mean(1, keepdim=True))
        if st["dtotal"] is not None:
            ds = ds + st["dtotal"].float()
        return ds.to(dt), (dy * s * r).sum(0)
    if kind == "cast":
        return _mxfp4(st["x"]).to(dt)
    x = _mxfp4(_normed(st["x"], st["w"]) if case.get("norm") else st["x"])
    table = _table()
    if kind == "linear":
        codes, scales = st["weights"][0]
        return (x @ _values(codes[0], scales[0], table).t()).to(dt)
    perm, bounds = st["grouping"][2].long(), st["bounds"]
    out = torch.zeros(n * case["k"], case["out"], dtype=dt, device="cuda")
    for e in range(case["e"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        r = x[perm[a:b] // case["k"]] if kind == "gate_up" else x[a:b]
        ye = [r @ _values(codes[e], scales[e], table).t() for codes, scales in st["weights"]]
        if kind == "gate_up":
            out[a:b] = (ye[0] / (1 + (-ye[0]).exp()) * ye[1]).to(dt)
        else:
            out[a:b] = ye[0].to(dt)
    return out


# ---------------------------------------------------------------- exact values


def _nearest_e2m1(v):
    """The nearest value of E2M1 in 64 bits by comparison with the borders
    between neighbours; a value on a border goes to the neighbour whose last
    bit is 0."""
    out = torch.zeros_like(v)
    m = v.abs()
    for i in range(7):
        border = (E2M1[i] + E2M1[i + 1]) / 2
        past = m > border if i % 2 == 0 else m >= border
        out = torch.where(past, E2M1[i + 1], out)
    return torch.where(v < 0, -out, out)


def _exact_mxfp4(x):
    b = x.double().reshape(x.shape[0], -1, 32)
    a = b.abs().amax(2, keepdim=True).clamp_min(2.0 ** -123)
    e = torch.floor(torch.log2(a))  # put right where the logarithm rounds to a whole number
    e = e - (2.0 ** e > a).double() + (2.0 ** (e + 1) <= a).double()
    scale = 2.0 ** (e - 2)
    return (_nearest_e2m1(b / scale) * scale).reshape(x.shape)


def _exact_weight(codes, scales):
    lo, hi = (codes & 15).int(), (codes >> 4).int()
    nib = torch.stack([lo, hi], -1).reshape(codes.shape[0], -1)
    e, m = (nib >> 1) & 3, nib & 1  # exponent (bias 1) and mantissa bits
    v = torch.where(e == 0, 0.5 * m.double(), 2.0 ** (e - 1).double() * (1 + 0.5 * m.double()))
    v = torch.where(nib >= 8, -v, v)
    s = 2.0 ** (scales[:, :v.shape[1] // 32].double() - 127)
    return v * s.repeat_interleave(32, dim=1)


def exact(case, seed):
    """The definitions in 64 bits, from the expert ids alone."""
    st = prepare(case, seed)
    kind, n = case["kind"], case["n"]
    dt = DTYPES[case["dtype"]]

    def norm(s):
        s = s.double()
        d = s.square().sum(1, keepdim=True) / s.shape[1] + EPS
        return s * st["w"].double() / d.sqrt()

    if kind == "norm":
        s, total = st["x"].double(), ()
        if st["residual"] is not None:
            s = (s + st["residual"].double()).float().to(dt)  # the definition rounds the sum
            total = (s.double(),)
        y = norm(s)
        if case["out"] == "int8":  # of the values in fp32
            y = y.float().double()
            a = y.abs().amax(1, keepdim=True)
            y = torch.round(y * 127 / a) * a / 127
        return (y, *total) if total or case["out"] == "int8" else y
    if kind == "norm_back":
        s, dy, w = st["x"].double(), st["dy"].double(), st["w"].double()
        h = case["h"]
        d = s.square().sum(1, keepdim=True) / h + EPS
        # y_j = w_j s_j d^(-1/2);  dd/ds_i = 2 s_i / h
        ds = w * dy / d.sqrt() - (w * dy * s).sum(1, keepdim=True) * s / (h * d * d.sqrt())
        if st["dtotal"] is not None:
            ds = ds + st["dtotal"].double()
        return ds, (dy * s / d.sqrt()).sum(0)
    if kind == "cast":
        return _exact_mxfp4(st["x"])
    x = _exact_mxfp4(norm(st["x"]).float() if case.get("norm") else st["x"])
    if kind == "linear":
        codes, scales = st["weights"][0]
        return torch.mm(x, _exact_weight(codes[0], scales[0]).t().contiguous())
    k = case["k"]
    order = sorted((e, f) for f, e in enumerate(st["ids"].reshape(-1).tolist()) if e >= 0)
    slot = torch.tensor([f for _, f in order], device="cuda", dtype=torch.int64)
    out = torch.zeros(n * k, case["out"], dtype=torch.float64, device="cuda")
    a = 0
    while a < len(order):
        e = order[a][0]
        b = a
        while b < len(order) and order[b][0] == e:
            b += 1
        r = slot[a:b] // k if kind == "gate_up" else torch.arange(a, b, device="cuda")
        y = [torch.mm(x[r], _exact_weight(codes[e], scales[e]).t().contiguous())
             for codes, scales in st["weights"]]
        out[a:b] = y[0] * torch.sigmoid(y[0]) * y[1] if kind == "gate_up" else y[0]
        a = b
    return out
