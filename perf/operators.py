"""The operators around the sequence mixer, as cases: the gated norm of the mixer's readout,
the norms around a residual block, the embedding lookup with its gradient, and the AdamW step.

``run`` computes a case in a plain form (elementary torch operations in fp32, rounded once at
the end) or, where ``own`` is true, through this package's entry points.  ``exact`` computes
the same from the definitions in fp64.

Every case names its operator and direction:

* ``gated_norm``: rows of one head's readout, y = o / sqrt(mean(o^2) + eps) * weight * act(gate).
* ``block_norm``: x_out = x + res_scale * scale * z, z = y or its RMSNorm with post_weight;
  h = RMSNorm(x_out) with weight.  Forward, or the backward of both outputs.
* ``embed``: out[n] = scale * table[ids[n]], or the gradient of the table.
* ``adamw``: one step over a list of tensors, states in 32 bits, or in 8 (e4m3 with one fp32
  scale per 256 elements; the second moment is held as its square root).

Rows t >= lengths[b] of a right-padded batch are padding: outputs there are zero, and they add
nothing to any gradient.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 256         # elements under one scale of the 8-bit optimiser states
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest normal fp32 number: the least scale of a block
BETAS, ADAM_EPS, LR, DECAY, STEP = (0.9, 0.95), 1e-8, 3e-4, 0.1, 100

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("silu", "sigmoid")


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 16 sequences on the 130M-LM layer: 96 short rows, latency only
        dict(name="gated_norm_decode", op="gated_norm", bwd=False, B=16, T=1, H=6, d=128, dtype="bf16", act="silu",
             gate="dense", ragged=0),
        # the readout norm of the 130M-LM layer; the gate is a slice of a fused projection
        dict(name="gated_norm_lm", op="gated_norm", bwd=False, B=16, T=2048, H=6, d=128, dtype="bf16", act="silu",
             gate="slice", ragged=0),
        # its training pass on the recommendation layer: right-padded user sequences
        dict(name="gated_norm_recsys_bwd", op="gated_norm", bwd=True, B=128, T=1024, H=2, d=64, dtype="bf16",
             act="silu", gate="dense", ragged=200),
        # the block boundary of the 130M LM with an fp32 residual stream, post-norm and layer scale
        dict(name="block_norm_lm", op="block_norm", bwd=False, B=16, T=2048, D=768, stream="fp32", dtype="bf16",
             delta=True, post=True, scale=True, ragged=0),
        # an odd width in fp32: a plain pre-norm with its residual add
        dict(name="block_norm_odd", op="block_norm", bwd=False, B=3, T=997, D=1001, stream="fp32", dtype="fp32",
             delta=True, post=False, scale=False, ragged=0),
        # the training pass of the block boundary, everything in bf16
        dict(name="block_norm_lm_bwd", op="block_norm", bwd=True, B=16, T=2048, D=768, stream="bf16", dtype="bf16",
             delta=True, post=True, scale=True, ragged=0),
        # item embeddings of the recommendation batch: a table far larger than the cache
        dict(name="embed_recsys", op="embed", bwd=False, B=128, T=1024, D=128, V=1000003, table="fp32",
             dtype="bf16", ids="int32", ragged=200, accumulate=False),
        # the dense gradient of a language model's token table
        dict(name="embed_lm_bwd", op="embed", bwd=True, B=16, T=2048, D=768, V=32000, table="fp32", dtype="bf16",
             ids="int64", ragged=0, accumulate=False),
        # the item table's gradient, added to what is there: only the rows of the batch move
        dict(name="embed_recsys_bwd", op="embed", bwd=True, B=128, T=1024, D=128, V=1000003, table="fp32",
             dtype="fp32", ids="int32", ragged=200, accumulate=True),
        # the small parameters of one mixer layer: ShortConv taps, norm weights, a gate projection
        dict(name="adamw_small", op="adamw", bits=32, param="fp32", grad="fp32", copies=False, layers=0, D=768, F=0,
             V=0),
        # every tensor of a 12-layer model of width 768, fp32 master weights with bf16 working copies
        dict(name="adamw_lm", op="adamw", bits=32, param="fp32", grad="fp32", copies=True, layers=12, D=768, F=2048,
             V=32000),
        # the same with 8-bit states and bf16 gradients
        dict(name="adamw_lm_8bit", op="adamw", bits=8, param="fp32", grad="bf16", copies=True, layers=12, D=768,
             F=2048, V=32000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated_norm", "block_norm", "embed", "adamw"))
    bwd = rng.random() < 0.5
    if op == "gated_norm":
        H, d = rng.choice((1, 2, 3, 5, 6, 8, 16)), rng.choice((16, 32, 64, 128))
        rows = _log(rng, 1, 50_000_000 // (H * d))
        B = min(rows, _log(rng, 1, 128))
        T = max(1, rows // B)
        return dict(op=op, bwd=bwd, B=B, T=T, H=H, d=d, dtype=rng.choice(("bf16", "fp32")), act=rng.choice(ACTS),
                    gate=rng.choice(("dense", "slice", "none")), ragged=rng.choice((0, 1 + T // 5)))
    if op == "block_norm":
        D = _log(rng, 1, 8192)
        if rng.random() < 0.6:
            D = max(8, D - D % 8)
        rows = _log(rng, 1, max(2, 50_000_000 // max(D, 64)))
        B = min(rows, _log(rng, 1, 128))
        T = max(1, rows // B)
        stream, dtype = rng.choice((("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")))
        delta = rng.random() < 0.8
        return dict(op=op, bwd=bwd, B=B, T=T, D=D, stream=stream, dtype=dtype, delta=delta,
                    post=delta and rng.random() < 0.5, scale=delta and rng.random() < 0.5,
                    ragged=rng.choice((0, 1 + T // 5)))
    if op == "embed":
        D = _log(rng, 8, 2048)
        if rng.random() < 0.7:
            D -= D % 8
        V = _log(rng, 2, 200_000_000 // max(D, 100))
        rows = _log(rng, 1, max(2, 40_000_000 // max(D, 64)))
        B = min(rows, _log(rng, 1, 128))
        T = max(1, rows // B)
        table, dtype = rng.choice((("fp32", "bf16"), ("bf16", "bf16"), ("fp32", "fp32")))
        return dict(op=op, bwd=bwd, B=B, T=T, D=D, V=V, table=table, dtype=dtype, ids=rng.choice(("int32", "int64")),
                    ragged=rng.choice((0, 1 + T // 5)), accumulate=bwd and rng.random() < 0.5)
    D = _log(rng, 17, 768)
    F = 0 if rng.random() < 0.3 else _log(rng, D, 2048)
    layers = rng.choice((0, 1, 2, 5, 12))
    param = rng.choice(("fp32", "fp32", "bf16"))
    return dict(op=op, bits=rng.choice((8, 32)), param=param, grad=rng.choice(("fp32", "bf16")),
                copies=param == "fp32" and rng.random() < 0.5, layers=layers, D=D, F=F,
                V=0 if layers == 0 or rng.random() < 0.3 else _log(rng, 100, 32000))


def _shapes(case):
    """The parameter tensors of an ``adamw`` case: a mixer's small ones, then per layer its
    projections, norms and taps (and an MLP of width F), and a table of V rows."""
    D, F, H = case["D"], case["F"], 6
    small = [(H, 128, 4), (D,), (128,), (D,), (D, 2 * H)]
    layer = small + [(D, D)] * 4 + ([(D, F), (D, F), (F, D)] if F else [])
    return (layer * case["layers"] if case["layers"] else small) + ([(case["V"], D)] if case["V"] else [])


# ----------------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, g):
    if not case["ragged"]:
        return None
    return torch.randint(case["ragged"], case["T"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = _gen(seed)

    def randn(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        x = torch.randn(shape, generator=g, device="cuda")
        return x.mul_(std).add_(mean).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "gated_norm":
        B, T, H, d, dt = case["B"], case["T"], case["H"], case["d"], DTYPES[case["dtype"]]
        s["lengths"] = _lengths(case, g)
        s["o"] = randn(B, T, H, d, dtype=dt, std=0.5)
        s["gate"] = None
        if case["gate"] == "dense":
            s["gate"] = randn(B, T, H, d, dtype=dt)
        elif case["gate"] == "slice":  # the second half of a fused projection's output
            s["gate"] = randn(B, T, 2 * H * d, dtype=dt)[..., H * d:].unflatten(-1, (H, d))
        s["weight"] = randn(d, mean=1.0, std=0.1)
        if case["bwd"]:
            s["dy"] = randn(B, T, H, d, dtype=dt)
    elif op == "block_norm":
        B, T, D = case["B"], case["T"], case["D"]
        xt, dt = DTYPES[case["stream"]], DTYPES[case["dtype"]]
        s["lengths"] = _lengths(case, g)
        s["x"] = randn(B, T, D, dtype=xt, std=2.0)
        s["weight"] = randn(D, mean=1.0, std=0.1)
        s["y"] = randn(B, T, D, dtype=dt, std=0.7) if case["delta"] else None
        s["post_weight"] = randn(D, mean=1.0, std=0.1) if case["post"] else None
        s["scale"] = randn(D, mean=0.5, std=0.1) if case["scale"] else None
        s["res_scale"] = 1.0 if case["scale"] or not case["delta"] else 0.5
        if case["bwd"]:
            s["dh"] = randn(B, T, D, dtype=dt)
            s["dx_out"] = randn(B, T, D, dtype=xt)
    elif op == "embed":
        B, T, D, V, dt = case["B"], case["T"], case["D"], case["V"], DTYPES[case["dtype"]]
        s["lengths"] = _lengths(case, g)
        # popularity falls with the rank as in a text or a catalogue; a fixed map spreads the ranks
        u = torch.rand((B, T), generator=g, device="cuda", dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
        ids = (rank * 2654435761 + 12345) % V
        if s["lengths"] is not None:  # what a loader leaves behind a sequence
            ids = torch.where(_valid(s["lengths"], B, T)[..., 0], ids, -1)
        s["ids"] = ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)
        s["factor"] = math.sqrt(D)
        if case["bwd"]:
            s["d_out"] = randn(B, T, D, dtype=dt)
            s["d_table"] = randn(V, D) if case["accumulate"] else None
        else:
            s["table"] = randn(V, D, dtype=DTYPES[case["table"]], std=0.02)
    else:
        # flat buffers with a view for each tensor, as a trainer keeps them; every tensor starts on a
        # multiple of 256 elements and what lies between two of them is zero
        shapes = _shapes(case)
        sizes = [math.prod(n) for n in shapes]
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + n + -n % BLOCK)
        used = torch.zeros(starts[-1], device="cuda")
        for at, n in zip(starts, sizes):
            used[at:at + n] = 1.0

        def views(flat):
            return [flat[at:at + n].view(shape) for at, n, shape in zip(starts, sizes, shapes)]

        def blocks(flat):
            return [flat[at // BLOCK:-(-(at + n) // BLOCK)] for at, n in zip(starts, sizes)]

        flat = {"params": (randn(starts[-1], std=0.02) * used).to(DTYPES[case["param"]])}
        grads = (randn(starts[-1], std=1e-3) * used).to(DTYPES[case["grad"]])
        m = randn(starts[-1], std=3e-4) * used
        v = (randn(starts[-1], std=1e-3) * used).square_()
        if case["copies"]:
            flat["copies"] = flat["params"].to(torch.bfloat16)
        if case["bits"] == 32:
            flat |= {"exp_avg": m, "exp_avg_sq": v}
        else:
            flat["exp_avg"], flat["exp_avg_scale"] = _encode(m)
            flat["exp_avg_sq"], flat["exp_avg_sq_scale"] = _encode(v.sqrt())
        s["flat"], s["flat_grads"] = flat, grads
        s["params"], s["grads"] = views(flat["params"]), views(grads)
        s["copies"] = views(flat["copies"]) if case["copies"] else None
        s["grad_scale"] = torch.full((1,), 0.5, device="cuda")  # a clip factor that stays on the device
        s["state"] = {n: (blocks if n.endswith("scale") else views)(x) for n, x in flat.items() if n.startswith("exp")}
    return s


# ------------------------------------------------------------------------------- the plain forms
def _valid(lengths, B, T):
    """[B, T, 1]: the rows that are not padding."""
    t = torch.arange(T, device=lengths.device)
    return (t < lengths[:, None])[..., None]


def _masked(x, valid):
    return x if valid is None else torch.where(valid, x, 0.0)


def _rstd(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_gated_norm(s):
    case = s["case"]
    valid = None if s["lengths"] is None else _valid(s["lengths"], case["B"], case["T"])[..., None]
    o, w = s["o"].float(), s["weight"]
    r = _rstd(o)
    xhat = o * r
    n = xhat * w
    if s["gate"] is not None:
        gate = s["gate"].float()
        sg = torch.sigmoid(gate)
        a = gate * sg if case["act"] == "silu" else sg
    if not case["bwd"]:
        y = n if s["gate"] is None else n * a
        return _masked(y, valid).to(s["o"].dtype)
    dy = _masked(s["dy"].float(), valid)
    out = {}
    if s["gate"] is not None:
        slope = sg * (1 + gate * (1 - sg)) if case["act"] == "silu" else sg * (1 - sg)
        out["gate"] = (dy * n * slope).to(s["o"].dtype)
        dy = dy * a
    out["weight"] = (dy * xhat).sum((0, 1, 2))
    dxhat = dy * w
    out["o"] = (r * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))).to(s["o"].dtype)
    return out


def _plain_block_norm(s):
    case = s["case"]
    valid = None if s["lengths"] is None else _valid(s["lengths"], case["B"], case["T"])
    x, w = s["x"].float(), s["weight"]
    k = s["res_scale"] if s["scale"] is None else s["res_scale"] * s["scale"]
    if s["y"] is not None:
        z = s["y"].float()
        if s["post_weight"] is not None:
            ry = _rstd(z)
            yhat = z * ry
            z = yhat * s["post_weight"]
    if not case["bwd"]:
        if s["y"] is None:
            return {"h": _masked(x * _rstd(x) * w, valid).to(DTYPES[case["dtype"]])}
        x = x + k * z
        h = x * _rstd(x) * w
        return {"x": _masked(x, valid).to(s["x"].dtype), "h": _masked(h, valid).to(s["y"].dtype)}
    dh = _masked(s["dh"].float(), valid)
    r = _rstd(x)
    xhat = x * r
    out = {"weight": (dh * xhat).sum((0, 1))}
    dxhat = dh * w
    dx = _masked(s["dx_out"].float(), valid) + r * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))
    out["x"] = dx.to(s["x"].dtype)
    if s["y"] is not None:
        if s["scale"] is not None:
            out["scale"] = (dx * z).sum((0, 1)) * s["res_scale"]
        dz = dx * k
        if s["post_weight"] is not None:
            out["post_weight"] = (dz * yhat).sum((0, 1))
            dyhat = dz * s["post_weight"]
            dz = ry * (dyhat - yhat * (dyhat * yhat).mean(-1, keepdim=True))
        out["y"] = dz.to(s["y"].dtype)
    return out


def _plain_embed(s):
    case = s["case"]
    valid = None if s["lengths"] is None else _valid(s["lengths"], case["B"], case["T"])
    ids = s["ids"] if valid is None else torch.where(valid[..., 0], s["ids"], 0)
    if not case["bwd"]:
        return _masked(s["table"][ids].float() * s["factor"], valid).to(DTYPES[case["dtype"]])
    d = s["d_table"] if case["accumulate"] else torch.zeros((case["V"], case["D"]), device=ids.device)
    rows = _masked(s["d_out"].float() * s["factor"], valid)
    return d.index_add_(0, ids.reshape(-1), rows.reshape(-1, case["D"]))


def _blocks(x):
    """x as rows of BLOCK elements, the last one filled with zeros."""
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _encode(x):
    """(codes in e4m3, one scale for each block of 256): the block's largest magnitude is 448."""
    b = _blocks(x)
    scale = (b.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    codes = (b * (1 / scale)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(-1)[:x.numel()].view(x.shape), scale


def _decode(codes, scale):
    b = _blocks(codes.float()) * scale[:, None]
    return b.view(-1)[:codes.numel()].view(codes.shape)


def _plain_adamw_one(s, i, c1, c2):
    st, (b1, b2) = s["state"], BETAS
    p = s["params"][i]
    g = s["grads"][i].float() * s["grad_scale"]
    if s["case"]["bits"] == 32:
        m = st["exp_avg"][i].mul_(b1).add_(g * (1 - b1))
        v = st["exp_avg_sq"][i].mul_(b2).add_(g * g * (1 - b2))
    else:
        m = _decode(st["exp_avg"][i], st["exp_avg_scale"][i]) * b1 + g * (1 - b1)
        v = _decode(st["exp_avg_sq"][i], st["exp_avg_sq_scale"][i]).square() * b2 + g * g * (1 - b2)
    root = v.sqrt()
    new = p.float() * (1 - LR * DECAY) - (LR / c1) * m / (root / math.sqrt(c2) + ADAM_EPS)
    p.copy_(new)
    if s["copies"] is not None:
        s["copies"][i].copy_(new)
    if s["case"]["bits"] == 8:
        codes, scale = _encode(m)
        st["exp_avg"][i].copy_(codes)
        st["exp_avg_scale"][i].copy_(scale)
        codes, scale = _encode(root)
        # a moment that is not zero is not held as zero
        least = torch.full((), 2.0 ** -9, device=p.device).to(torch.float8_e4m3fn).view(torch.uint8)
        raised = (codes.view(torch.uint8) == 0) & (root > 0)
        codes = torch.where(raised, least, codes.view(torch.uint8)).view(torch.float8_e4m3fn)
        st["exp_avg_sq"][i].copy_(codes)
        st["exp_avg_sq_scale"][i].copy_(scale)


def _plain_adamw(s):
    c1, c2 = 1 - BETAS[0] ** STEP, 1 - BETAS[1] ** STEP
    for i in range(len(s["params"])):  # one parameter tensor after another
        _plain_adamw_one(s, i, c1, c2)
    return s["flat"]


PLAIN = {"gated_norm": _plain_gated_norm, "block_norm": _plain_block_norm, "embed": _plain_embed,
         "adamw": _plain_adamw}


# -------------------------------------------------------------------------------- the entry points
def _own(s):
    import linear_attention_sequence_shortconv_b200 as prism

    case = s["case"]
    if case["op"] == "gated_norm":
        if case["bwd"]:
            g = prism.gated_norm_bwd(s["o"], s["gate"], s["weight"], s["dy"], lengths=s["lengths"], eps=EPS,
                                     act=case["act"])
            return {n: x for n, x in g.items() if x is not None}
        return prism.gated_norm_fwd(s["o"], s["gate"], s["weight"], lengths=s["lengths"], eps=EPS, act=case["act"])
    if case["op"] == "block_norm":
        block = dict(y=s["y"], post_weight=s["post_weight"], scale=s["scale"], res_scale=s["res_scale"],
                     lengths=s["lengths"], eps=EPS)
        if case["bwd"]:
            g = prism.block_norm_bwd(s["x"], s["weight"], s["dh"], dx_out=s["dx_out"], **block)
            return {n: x for n, x in g.items() if x is not None}
        x, h = prism.block_norm_fwd(s["x"], s["weight"], h_dtype=DTYPES[case["dtype"]], **block)
        return {"h": h} if s["y"] is None else {"x": x, "h": h}
    if case["op"] == "embed":
        if case["bwd"]:
            return prism.embed_bwd(s["ids"], s["d_out"], case["V"], scale=s["factor"], lengths=s["lengths"],
                                   d_table=s["d_table"], accumulate=case["accumulate"])
        return prism.embed_fwd(s["ids"], s["table"], scale=s["factor"], lengths=s["lengths"],
                               dtype=DTYPES[case["dtype"]])
    prism.adamw_step(s["params"], s["grads"], step=STEP, lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY,
                     grad_scale=s["grad_scale"], copies=s["copies"], **s["state"])
    return s["flat"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- the work
def _count(case):
    """Rows that are not padding, as far as the sizes alone tell: lengths are even over their range."""
    n = case["B"] * case["T"]
    return n if not case["ragged"] else case["B"] * (case["ragged"] + case["T"]) / 2


def work(case):
    size = {"bf16": 2, "fp32": 4}
    op = case["op"]
    if op == "gated_norm":
        e, n, all_n = size[case["dtype"]], _count(case) * case["H"] * case["d"], case["B"] * case["T"] * case["H"] * case["d"]
        gate = case["gate"] != "none"
        if case["bwd"]:
            return {"bytes": e * (n * (2 + gate) + all_n * (1 + gate)) + 8 * case["d"], "flops": 20 * n}
        return {"bytes": e * (n * (1 + gate) + all_n) + 4 * case["d"], "flops": 10 * n}
    if op == "block_norm":
        ex, e, D = size[case["stream"]], size[case["dtype"]], case["D"]
        n, all_n, y = _count(case) * D, case["B"] * case["T"] * D, case["delta"]
        vectors = 4 * D * (1 + case["post"] + case["scale"])
        if case["bwd"]:
            reads = 2 * ex + e + e * (y and (case["post"] or case["scale"]))
            return {"bytes": reads * n + (ex + e * y) * all_n + 2 * vectors, "flops": 25 * n}
        return {"bytes": (ex + e * y) * n + (e + ex * y) * all_n + vectors, "flops": 12 * n}
    if op == "embed":
        n, D, V = _count(case), case["D"], case["V"]
        ids = (4 if case["ids"] == "int32" else 8) * n
        if not case["bwd"]:
            # each row of the table that the batch names is read once
            return {"bytes": ids + _distinct(n, V) * D * size[case["table"]] + case["B"] * case["T"] * D * size[case["dtype"]],
                    "flops": n * D}
        rows = 2 * _distinct(n, V) if case["accumulate"] else V
        return {"bytes": ids + n * D * size[case["dtype"]] + rows * D * 4, "flops": 2 * n * D}
    n = sum(math.prod(x) for x in _shapes(case))
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + states + 2 * case["copies"]), "flops": 20 * n}


def _distinct(n, V):
    """How many different ids n draws of prepare() name, on average."""
    # rank r has the probability log((r + 2) / (r + 1)) / log(V + 1): summed over the ranks, coarsely for the far ones
    total, lo = 0.0, 1.0
    while lo < V + 1:
        hi = min(V + 1.0, max(lo + 1, lo * 1.05))
        p = math.log(hi / lo) / math.log(V + 1) / (hi - lo)
        total += (hi - lo) * (1 - (1 - p) ** n if p < 1 else 1)
        lo = hi
    return min(total, n, V)


# ---------------------------------------------------------------------------- the 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s, case)


def _rows(x, lengths):
    """x [B, T, ...] in 64 bits with the padding's rows set to zero."""
    x = x.double()
    if lengths is not None:
        keep = torch.arange(x.shape[1], device=x.device)[None, :] < lengths.long()[:, None]
        x = x.masked_fill(~keep.view(keep.shape + (1,) * (x.dim() - 2)), 0.0)
    return x


def _rms64(x, w):
    """RMSNorm of the rows of x and what leads back from its cotangent: (value, function)."""
    n = x.shape[-1]
    norm = ((x * x).sum(-1, keepdim=True) / n + EPS).sqrt()

    def back(d):
        t = d * w
        along = (t * x).sum(-1, keepdim=True) / n
        return t / norm - x * along / norm ** 3, (d * x / norm).reshape(-1, n).sum(0)

    return x / norm * w, back


def _exact_gated_norm(s, case):
    o, w = _rows(s["o"], s["lengths"]), s["weight"].double()
    value, back = _rms64(o, w)
    if s["gate"] is None:
        act = slope = None
    else:
        gate = _rows(s["gate"], s["lengths"])
        e = 1 / (1 + torch.exp(-gate))
        act = gate * e if case["act"] == "silu" else e
        slope = e + gate * e * (1 - e) if case["act"] == "silu" else e * (1 - e)
    if not case["bwd"]:
        return value if act is None else value * act
    dy = _rows(s["dy"], s["lengths"])
    d_o, d_w = back(dy if act is None else dy * act)
    out = {"o": d_o, "weight": d_w}
    if act is not None:
        out["gate"] = dy * value * slope
    return out


def _exact_block_norm(s, case):
    x, w = _rows(s["x"], s["lengths"]), s["weight"].double()
    y = None if s["y"] is None else _rows(s["y"], s["lengths"])
    k = s["res_scale"] * (torch.ones_like(w) if s["scale"] is None else s["scale"].double())
    z, back_z = y, None
    if s["post_weight"] is not None:
        z, back_z = _rms64(y, s["post_weight"].double())
    if not case["bwd"]:
        if y is None:
            return {"h": _rms64(x, w)[0]}
        x = x + k * z
        return {"x": x, "h": _rms64(x, w)[0]}
    _, back = _rms64(x, w)
    d_x, d_w = back(_rows(s["dh"], s["lengths"]))
    d_x = d_x + _rows(s["dx_out"], s["lengths"])
    out = {"x": d_x, "weight": d_w}
    if y is not None:
        if s["scale"] is not None:
            out["scale"] = s["res_scale"] * (d_x * z).sum((0, 1))
        out["y"] = k * d_x
        if back_z is not None:
            out["y"], out["post_weight"] = back_z(k * d_x)
    return out


def _exact_embed(s, case):
    B, T, D, V = case["B"], case["T"], case["D"], case["V"]
    ids = s["ids"].long().reshape(-1)
    if s["lengths"] is not None:
        t = torch.arange(T, device=ids.device).repeat(B)
        keep = t < s["lengths"].long().repeat_interleave(T)
    else:
        keep = torch.ones_like(ids, dtype=torch.bool)
    where = keep.nonzero()[:, 0]
    if not case["bwd"]:
        out = torch.zeros((B * T, D), dtype=torch.float64, device=ids.device)
        out[where] = s["table"].index_select(0, ids[where]).double() * s["factor"]
        return out.view(B, T, D)
    d = torch.zeros((V, D), dtype=torch.float64, device=ids.device)
    d.index_add_(0, ids[where], s["d_out"].reshape(-1, D)[where].double() * s["factor"])
    return d + s["d_table"].double() if case["accumulate"] else d


def _held(x):
    """What 8 bits hold of x (64 bits), as (codes, scales)."""
    b = _blocks(x)
    scale = (b.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    q = b / scale[:, None]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)  # 3 bits after the first
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX).view(-1)[:x.numel()].view(x.shape), scale


def _exact_adamw(s, case):
    # element by element, so the flat buffers in one piece: a zero between two tensors stays zero
    b1, b2 = BETAS
    f = {n: x.double() for n, x in s["flat"].items()}
    g = s["flat_grads"].double() * s["grad_scale"].double()
    m, v = f["exp_avg"], f["exp_avg_sq"]
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * f["exp_avg_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * f["exp_avg_sq_scale"][:, None]).view(-1) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    update = (m / (1 - b1 ** STEP)) / ((v / (1 - b2 ** STEP)) ** 0.5 + ADAM_EPS)
    out = {"params": f["params"] - LR * (DECAY * f["params"] + update)}
    if case["copies"]:
        out["copies"] = out["params"]
    if case["bits"] == 32:
        out["exp_avg"], out["exp_avg_sq"] = m, v
        return out
    out["exp_avg"], out["exp_avg_scale"] = _held(m)
    codes, out["exp_avg_sq_scale"] = _held(v ** 0.5)
    out["exp_avg_sq"] = torch.where((codes == 0) & (v > 0), 2.0 ** -9, codes)
    return out


EXACT = {"gated_norm": _exact_gated_norm, "block_norm": _exact_block_norm, "embed": _exact_embed,
         "adamw": _exact_adamw}
