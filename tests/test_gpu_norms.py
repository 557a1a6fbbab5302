"""The gated norm and the block norm on the GPU (through the C ABI) against their fp64
statements (oracle/layer_oracle.py).

Tolerances.  An output is rounded once, by at most half a step of its type: 2^-8 (bf16) or
2^-24 (fp32) of its value.  Before that it is a sum of a few products of fp32 numbers; each
factor and sum carries a relative error of k 2^-24, where k counts the roundings on its way:
a mean over D elements adds up at most 16 numbers per thread, 5 shuffle steps and 16 warps
(37, halved by the root), the fast sigmoid of a bf16 gate errs by at most 2 + 1.2 |g| units of
2^-23 in the exponential and 2 in the division (24 for |g| < 6), and products add one each.
K = 128 covers their sum with room; it multiplies the sum of the magnitudes of an output's
terms.  A weight's gradient is a sum over n rows in fp32: at most n more roundings per term.
"""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import linear_attention_sequence_shortconv_b200 as prism
from oracle import layer_oracle as ref

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
K = 128
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(seed, *shape, dtype=torch.float32, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _close(got, want, magnitude, roundings=K):
    """|got - want| <= half a step of the output's type + roundings * 2^-24 * magnitude."""
    got64 = got.double().cpu()
    bound = HALF[got.dtype] * want.abs() + roundings * U * magnitude + 2.0 ** -126
    worst = ((got64 - want).abs() / bound).max().item() if want.numel() else 0.0
    assert torch.isfinite(got64).all() and worst <= 1.0, worst


def _cuda(t):
    return None if t is None else t.cuda()


def _f64(t):
    return None if t is None else t.double()


def _gated_inputs(B, T, H, d, dtype, gate, seed=0):
    o, dy = _randn(seed + 1, B, T, H, d, dtype=dtype, std=0.7), _randn(seed + 2, B, T, H, d, dtype=dtype)
    w = 1 + 0.1 * _randn(seed + 3, d)
    g = None
    if gate == "dense":
        g = _randn(seed + 4, B, T, H, d, dtype=dtype)
    elif gate == "slice":  # the middle of a projection three times as wide
        g = _randn(seed + 4, B, T, 3 * H * d, dtype=dtype)[..., H * d:2 * H * d].unflatten(-1, (H, d))
    return o, g, w, dy


def _gated_magnitudes(o, g, w, dy, lengths, act):
    """Magnitudes of the terms of y, d_o and d_gate, and the sum over rows of those of d_weight."""
    keep = ref.valid_rows(lengths, *o.shape[:2])[..., None, None].double()
    o, dy = o * keep, dy * keep
    r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5)
    xh = (o * r).abs()
    if g is None:
        a, slope = torch.ones_like(o), None
    else:
        g = torch.where(keep > 0, g, 0.0)
        s = torch.sigmoid(g)
        a = s * (g.abs() if act == "silu" else 1)
        slope = s * (1 + g.abs()) if act == "silu" else s
    t = dy.abs() * a * w.abs()
    return {"y": xh * w.abs() * a * keep, "o": r * (t + xh * (t * xh).mean(-1, keepdim=True)),
            "gate": None if g is None else dy.abs() * xh * w.abs() * slope,
            "weight": (dy.abs() * a * xh).sum((0, 1, 2))}


GATED = [
    # B, T, H, d, dtype, gate, act, lengths
    (1, 1, 1, 16, "bf16", "dense", "silu", None),
    (1, 1, 1, 128, "fp32", "none", "silu", None),
    (3, 37, 5, 32, "bf16", "slice", "silu", [37, 0, 11]),
    (2, 65, 2, 64, "fp32", "dense", "sigmoid", [1, 64]),
    (4, 129, 6, 128, "bf16", "dense", "silu", None),
    (4, 129, 6, 128, "bf16", "slice", "sigmoid", [129, 128, 1, 0]),
    (2, 33, 3, 16, "fp32", "slice", "silu", [20, 33]),
    (2, 700, 16, 128, "bf16", "none", "silu", [700, 3]),
    (1, 5000, 2, 64, "bf16", "dense", "silu", None),
]


@pytest.mark.parametrize("B,T,H,d,dtype,gate,act,lengths", GATED)
def test_gated_norm_matches_fp64(B, T, H, d, dtype, gate, act, lengths):
    o, g, w, dy = _gated_inputs(B, T, H, d, DT[dtype], gate)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    gc = None
    if g is not None:  # a strided gate keeps its strides on the device
        gc = torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda")
        gc.copy_(g)
    leaves = [t.double().requires_grad_(True) for t in (o, g, w) if t is not None]
    y64 = ref.gated_norm(leaves[0], leaves[1] if g is not None else None, leaves[-1], lengths, act=act)
    grads = torch.autograd.grad((y64 * dy.double()).sum(), leaves)
    mag = _gated_magnitudes(o.double(), _f64(g), w.double(), dy.double(), lengths, act)

    y = prism.gated_norm_fwd(o.cuda(), gc, w.cuda(), lengths=_cuda(lens), act=act)
    got = prism.gated_norm_bwd(o.cuda(), gc, w.cuda(), dy.cuda(), lengths=_cuda(lens), act=act)
    assert prism.stream_status() == 0
    _close(y, y64.detach(), mag["y"])
    _close(got["o"], grads[0], mag["o"])
    if g is not None:
        _close(got["gate"], grads[1], mag["gate"])
    else:
        assert got["gate"] is None
    _close(got["weight"], grads[-1], mag["weight"], K + B * T * H)
    pad = ~ref.valid_rows(lengths, B, T)
    for t in (y, got["o"], got["gate"]):
        assert t is None or not t.cpu()[pad].any()


def test_gated_norm_of_a_decoded_token_is_that_of_its_row():
    o, g, w, dy = _gated_inputs(5, 1, 6, 128, torch.bfloat16, "slice")
    oc, wc, dyc = o.cuda(), w.cuda(), dy.cuda()
    gc = torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda").copy_(g)
    y = prism.gated_norm_fwd(oc, gc, wc)
    assert torch.equal(prism.gated_norm_fwd(oc[:, 0], gc[:, 0], wc), y[:, 0])
    a, b = prism.gated_norm_bwd(oc, gc, wc, dyc), prism.gated_norm_bwd(oc[:, 0], gc[:, 0], wc, dyc[:, 0])
    assert torch.equal(a["o"][:, 0], b["o"]) and torch.equal(a["gate"][:, 0], b["gate"])
    assert torch.equal(a["weight"], b["weight"])


def test_gated_norm_padding_is_not_read_and_buffers_may_be_reused():
    B, T, H, d = 3, 50, 4, 64
    o, g, w, dy = (t.cuda() for t in _gated_inputs(B, T, H, d, torch.bfloat16, "dense"))
    lens = torch.tensor([50, 7, 0], dtype=torch.int32, device="cuda")
    pad = ~ref.valid_rows(lens.cpu(), B, T).cuda()
    y, grads = prism.gated_norm_fwd(o, g, w, lengths=lens), prism.gated_norm_bwd(o, g, w, dy, lengths=lens)
    for bad in (float("nan"), float("inf")):
        o2, g2, dy2 = (t.clone() for t in (o, g, dy))
        for t in (o2, g2, dy2):
            t[pad] = bad
        assert torch.equal(prism.gated_norm_fwd(o2, g2, w, lengths=lens), y)
        again = prism.gated_norm_bwd(o2, g2, w, dy2, lengths=lens)
        assert all(torch.equal(again[n], grads[n]) for n in grads)
    # y over o; lengths above T and below zero
    o3 = o.clone()
    assert prism.gated_norm_fwd(o3, g, w, lengths=lens, y=o3) is o3 and torch.equal(o3, y)
    odd = torch.tensor([T + 9, 7, -3], dtype=torch.int32, device="cuda")
    assert torch.equal(prism.gated_norm_fwd(o, g, w, lengths=odd), y)


def test_a_nan_stays_in_its_row():
    o, g, w, _ = (t.cuda() for t in _gated_inputs(2, 9, 3, 32, torch.float32, "dense"))
    y = prism.gated_norm_fwd(o, g, w)
    o[1, 4, 2, 5] = float("nan")
    y2 = prism.gated_norm_fwd(o, g, w)
    assert torch.isnan(y2[1, 4, 2]).all()
    y2[1, 4, 2] = y[1, 4, 2]
    assert torch.equal(y, y2)


def test_gate_offsets_beyond_32_bits():
    # three tokens whose gates stand 2^30 elements apart
    o, g, w, dy = (t.cuda() for t in _gated_inputs(1, 3, 2, 64, torch.bfloat16, "dense"))
    wide = torch.empty(2 * (1 << 30) + 128, dtype=torch.bfloat16, device="cuda")
    far = wide.as_strided((1, 3, 2, 64), (3 << 30, 1 << 30, 64, 1))
    far.copy_(g)
    assert torch.equal(prism.gated_norm_fwd(o, far, w), prism.gated_norm_fwd(o, g, w))
    a, b = prism.gated_norm_bwd(o, far, w, dy), prism.gated_norm_bwd(o, g, w, dy)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_zero_rows():
    o = torch.zeros(2, 3, 2, 64, device="cuda")
    w, dy = torch.ones(64, device="cuda"), torch.ones(2, 3, 2, 64, device="cuda")
    assert not prism.gated_norm_fwd(o, None, w).any()
    g = prism.gated_norm_bwd(o, None, w, dy)
    assert torch.allclose(g["o"], torch.full_like(o, 1e-5 ** -0.5), rtol=1e-6) and not g["weight"].any()
    x_out, h = prism.block_norm_fwd(torch.zeros(2, 3, 40, device="cuda"), torch.ones(40, device="cuda"))
    assert not h.any() and not x_out.any()


# ------------------------------------------------------------------------------- block norm
BLOCK = [
    # B, T, D, stream, dtype, y, post, scale, res_scale, lengths
    (1, 1, 1, "fp32", "fp32", True, True, True, 1.0, None),
    (1, 1, 768, "bf16", "bf16", True, True, True, 1.0, None),
    (2, 3, 2, "bf16", "bf16", True, False, False, 0.5, None),
    (3, 19, 8, "fp32", "bf16", True, True, False, 1.0, [19, 0, 5]),
    (2, 70, 24, "fp32", "fp32", True, False, True, 1.0, [70, 69]),
    (2, 33, 129, "bf16", "bf16", True, True, True, 0.25, [1, 33]),
    (2, 100, 256, "fp32", "bf16", False, False, False, 1.0, [100, 4]),
    (2, 100, 264, "bf16", "bf16", False, False, False, 1.0, None),
    (3, 131, 768, "fp32", "bf16", True, True, True, 1.0, [131, 0, 64]),
    (2, 997, 768, "bf16", "bf16", True, True, True, 1.0, None),
    (3, 97, 1001, "fp32", "fp32", True, False, False, 1.0, [97, 1, 96]),
    (2, 60, 12, "fp32", "bf16", True, True, True, 1.0, [60, 7]),
    (2, 60, 100, "fp32", "fp32", True, True, True, 1.0, None),
    (2, 60, 100, "bf16", "bf16", True, False, True, 1.0, [3, 60]),
    (1, 50, 1028, "fp32", "bf16", True, True, True, 1.0, [49]),
    (1, 30, 1536, "bf16", "bf16", True, True, True, 1.0, None),
    (1, 200, 8192, "bf16", "bf16", True, True, True, 1.0, [199]),
    (1, 180, 5120, "fp32", "fp32", True, True, True, 1.0, None),
    (1, 400, 2048, "bf16", "bf16", True, True, False, 0.5, None),
    (1, 40, 1024, "bf16", "bf16", True, False, False, 1.0, None),
    (1, 21, 2056, "fp32", "bf16", True, True, True, 1.0, [20]),
    (1, 9, 4095, "fp32", "bf16", True, True, True, 1.0, None),
    (1, 13, 4104, "bf16", "bf16", True, True, True, 1.0, [12]),
    (1, 7, 8191, "fp32", "fp32", True, True, True, 1.0, None),
    (1, 6, 8192, "fp32", "bf16", True, False, True, 1.0, None),
]


def _block_inputs(B, T, D, stream, dtype, y, post, scale, seed=0):
    xt, at = DT[stream], DT[dtype]
    x = _randn(seed + 1, B, T, D, dtype=xt, std=2.0)
    vec = dict(y=_randn(seed + 2, B, T, D, dtype=at, std=0.7) if y else None,
               post_weight=1 + 0.1 * _randn(seed + 3, D) if post else None,
               scale=0.5 + 0.1 * _randn(seed + 4, D) if scale else None)
    w = 1 + 0.1 * _randn(seed + 5, D)
    return x, w, vec, _randn(seed + 6, B, T, D, dtype=at), _randn(seed + 7, B, T, D, dtype=xt)


@pytest.mark.parametrize("B,T,D,stream,dtype,y,post,scale,res,lengths", BLOCK)
def test_block_norm_matches_fp64(B, T, D, stream, dtype, y, post, scale, res, lengths):
    x, w, vec, dh, dxo = _block_inputs(B, T, D, stream, dtype, y, post, scale)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    keep = ref.valid_rows(lengths, B, T)[..., None]
    args = dict(res_scale=res, lengths=_cuda(lens), **{n: _cuda(t) for n, t in vec.items()})
    args64 = dict(res_scale=res, lengths=lengths, **{n: _f64(t) for n, t in vec.items()})

    x_out, h = prism.block_norm_fwd(x.cuda(), w.cuda(), h_dtype=DT[dtype], **args)
    xo64, h64 = ref.block_norm(x.double(), w.double(), **args64)
    # the terms of x_out: x and k z
    k = res * (1.0 if not scale else vec["scale"].double().abs())
    z = 0.0
    if y:
        z = torch.where(keep, vec["y"].double(), 0.0)
        ry = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-5)
        yh = (z * ry).abs()
        z = (yh * vec["post_weight"].double().abs()) if post else z.abs()
        mx = torch.where(keep, x.double().abs(), 0.0) + k * z
        _close(x_out, torch.where(keep, xo64, 0.0), mx)
    else:
        assert x_out.data_ptr() != 0 and torch.equal(x_out.cpu(), x)
        mx = torch.where(keep, x.double().abs(), 0.0)
    r = 1 / torch.sqrt((xo64 * xo64).mean(-1, keepdim=True) + 1e-5)
    # an error of x_out's terms enters h through the row's root mean square as well
    mr = torch.sqrt((mx * mx).mean(-1, keepdim=True)) * r
    _close(h, h64, (mx * r + (xo64 * r).abs() * mr) * w.double().abs())
    pad = ~ref.valid_rows(lengths, B, T)
    assert not h.cpu()[pad].any() and (not y or not x_out.cpu()[pad].any())

    # backward, from a stored x_out that both sides are given
    xs = torch.where(keep, x_out.cpu(), 0.0) if y else x
    got = prism.block_norm_bwd(xs.cuda(), w.cuda(), dh.cuda(), dx_out=dxo.cuda(), **args)
    want = ref.block_norm_grad(xs.double(), w.double(), dh.double(), dx_out=dxo.double(), **args64)
    assert prism.stream_status() == 0
    xk, dhk = torch.where(keep, xs.double(), 0.0), torch.where(keep, dh.double().abs(), 0.0)
    r = 1 / torch.sqrt((xk * xk).mean(-1, keepdim=True) + 1e-5)
    xh, t = (xk * r).abs(), dhk * w.double().abs()
    mdx = torch.where(keep, dxo.double().abs(), 0.0) + r * (t + xh * (t * xh).mean(-1, keepdim=True))
    _close(got["x"], want["x"], mdx)
    _close(got["weight"], want["weight"], (dhk * xh).sum((0, 1)), K + B * T)
    if y:
        if scale:
            _close(got["scale"], want["scale"], res * (mdx * z).sum((0, 1)), 2 * K + B * T)
        if post:
            _close(got["post_weight"], want["post_weight"], (k * mdx * yh).sum((0, 1)), 2 * K + B * T)
            u = k * mdx * vec["post_weight"].double().abs()
            _close(got["y"], want["y"], ry * (u + yh * (u * yh).mean(-1, keepdim=True)), 2 * K)
        else:
            _close(got["y"], want["y"], k * mdx)
    for n in ("y", "post_weight", "scale"):
        assert (got[n] is None) == (n not in want)
    assert not got["x"].cpu()[pad].any() and (got["y"] is None or not got["y"].cpu()[pad].any())


def test_block_norm_without_dx_out_is_with_zeros():
    x, w, vec, dh, dxo = _block_inputs(2, 40, 96, "fp32", "bf16", True, True, True)
    v = {n: t.cuda() for n, t in vec.items()}
    a = prism.block_norm_bwd(x.cuda(), w.cuda(), dh.cuda(), **v)
    b = prism.block_norm_bwd(x.cuda(), w.cuda(), dh.cuda(), dx_out=torch.zeros_like(dxo).cuda(), **v)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_block_norm_padding_is_not_read_and_buffers_may_be_reused():
    B, T, D = 3, 40, 200
    x, w, vec, dh, dxo = _block_inputs(B, T, D, "bf16", "bf16", True, True, True)
    x, w, dh, dxo = x.cuda(), w.cuda(), dh.cuda(), dxo.cuda()
    v = {n: t.cuda() for n, t in vec.items()}
    lens = torch.tensor([40, 0, 13], dtype=torch.int32, device="cuda")
    pad = ~ref.valid_rows(lens.cpu(), B, T).cuda()
    x_out, h = prism.block_norm_fwd(x, w, lengths=lens, **v)
    grads = prism.block_norm_bwd(x_out, w, dh, dx_out=dxo, lengths=lens, **v)
    bad = {"x": x.clone(), "dh": dh.clone(), "dxo": dxo.clone(), "xo": x_out.clone()}
    v2 = dict(v, y=v["y"].clone())
    for t in (*bad.values(), v2["y"]):
        t[pad] = float("nan")
    a, b = prism.block_norm_fwd(bad["x"], w, lengths=lens, **v2)
    assert torch.equal(a, x_out) and torch.equal(b, h)
    again = prism.block_norm_bwd(bad["xo"], w, bad["dh"], dx_out=bad["dxo"], lengths=lens, **v2)
    assert all(torch.equal(again[n], grads[n]) for n in grads)
    # x_out over x
    xi = x.clone()
    a, b = prism.block_norm_fwd(xi, w, lengths=lens, x_out=xi, **v)
    assert a is xi and torch.equal(a, x_out) and torch.equal(b, h)
    # a decoded token is a row
    a, b = prism.block_norm_fwd(x[:, 3].contiguous(), w, **dict(v, y=v["y"][:, 3].contiguous()))
    full = prism.block_norm_fwd(x, w, **v)
    assert torch.equal(a, full[0][:, 3]) and torch.equal(b, full[1][:, 3])


# ----------------------------------------------------------------- streams, graphs, repetition
def _train_calls(o, g, w, dy, x, wb, v, dh, dxo):
    y = prism.gated_norm_fwd(o, g, w)
    a = prism.gated_norm_bwd(o, g, w, dy)
    x_out, h = prism.block_norm_fwd(x, wb, **v)
    b = prism.block_norm_bwd(x_out, wb, dh, dx_out=dxo, **v)
    return [y, x_out, h, *a.values(), *b.values()]


def _train_inputs(seed):
    o, g, w, dy = (t.cuda() for t in _gated_inputs(4, 300, 6, 128, torch.bfloat16, "dense", seed))
    x, wb, vec, dh, dxo = _block_inputs(4, 300, 768, "fp32", "bf16", True, True, True, seed)
    return [o, g, w, dy, x.cuda(), wb.cuda(), {n: t.cuda() for n, t in vec.items()}, dh.cuda(), dxo.cuda()]


def test_results_repeat_bit_for_bit_also_on_another_stream():
    args = _train_inputs(0)
    first = _train_calls(*args)
    assert all(torch.equal(a, b) for a, b in zip(first, _train_calls(*args)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, g, w, dy = args[:4]
    y = prism.gated_norm_fwd(o, g, w, stream=s)
    a = prism.gated_norm_bwd(o, g, w, dy, stream=s)
    x_out, h = prism.block_norm_fwd(args[4], args[5], stream=s, **args[6])
    b = prism.block_norm_bwd(x_out, args[5], args[7], dx_out=args[8], stream=s, **args[6])
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, [y, x_out, h, *a.values(), *b.values()]))


def test_two_threads_call_at_once():
    # the same kernels with different amounts of shared memory, from two host threads
    sizes = [(("fp32", "bf16"), 768), (("fp32", "fp32"), 1024), (("bf16", "bf16"), 768), (("fp32", "fp32"), 640)]
    work, want = [], []
    for (stream, dtype), D in sizes:
        x, w, vec, dh, dxo = _block_inputs(2, 300, D, stream, dtype, True, True, True, D)
        args = (x.cuda(), w.cuda(), dh.cuda(), dxo.cuda(), {n: t.cuda() for n, t in vec.items()})
        work.append(args)
    torch.cuda.synchronize()

    def run(args, s=None):
        x, w, dh, dxo, v = args
        fwd = prism.block_norm_fwd(x, w, stream=s, **v)
        return [*fwd, *prism.block_norm_bwd(x, w, dh, dx_out=dxo, stream=s, **v).values()]

    want = [run(a) for a in work]
    torch.cuda.synchronize()

    def many(mine):
        s = torch.cuda.Stream()
        out = [[run(a, s) for a in mine] for _ in range(40)]
        s.synchronize()
        return out

    with ThreadPoolExecutor(2) as pool:
        jobs = [pool.submit(many, work[:2]), pool.submit(many, work[2:])]
        for k, job in enumerate(jobs):
            for out in job.result():
                for a, b in zip(out, want[2 * k:2 * k + 2]):
                    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_captured_graph_follows_its_inputs():
    args = _train_inputs(0)
    _train_calls(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _train_calls(*args)
    for seed in (50, 60):
        new = _train_inputs(seed)
        for old, t in zip(args, new):
            for a, b in zip(old.values(), t.values()) if isinstance(old, dict) else ((old, t),):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, _train_calls(*new)))


def test_refusals_name_the_argument():
    o, g, w, dy = (t.cuda() for t in _gated_inputs(2, 8, 2, 32, torch.bfloat16, "dense"))
    with pytest.raises(ValueError, match="weight"):
        prism.gated_norm_fwd(o, g, w[:16])
    with pytest.raises(TypeError, match="gate"):
        prism.gated_norm_fwd(o, g.float(), w)
    with pytest.raises(ValueError, match="gate"):
        prism.gated_norm_fwd(o, g[:, :4], w)
    with pytest.raises(ValueError, match="strides"):
        prism.gated_norm_fwd(o, g.transpose(1, 2).contiguous().transpose(1, 2), w)
    with pytest.raises(ValueError, match="strides"):
        prism.gated_norm_fwd(o, g[:, :1].expand(2, 8, 2, 32), w)
    with pytest.raises(ValueError, match="contiguous"):
        prism.gated_norm_fwd(o.transpose(1, 2), None, w)
    with pytest.raises(ValueError, match="lengths"):
        prism.gated_norm_fwd(o, g, w, lengths=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="float16"):
        prism.gated_norm_fwd(o.half(), None, w)
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.gated_norm_fwd(torch.zeros(1, 1, 1, 48, device="cuda"), None, torch.ones(48, device="cuda"))
    with pytest.raises(prism.PrismError, match="INVALID"):
        prism.gated_norm_fwd(o, g, w, eps=0.0)
    with pytest.raises(prism.PrismError, match="WORKSPACE"):
        prism.gated_norm_bwd(o, g, w, dy, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    x, wb = torch.zeros(2, 8, 40, device="cuda"), torch.ones(40, device="cuda")
    with pytest.raises(ValueError, match="post_weight"):
        prism.block_norm_fwd(x, wb, post_weight=wb)
    with pytest.raises(TypeError, match="h_dtype"):
        prism.block_norm_fwd(x, wb, y=x.clone(), h_dtype=torch.bfloat16)
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.block_norm_fwd(x.bfloat16(), wb, y=x.clone())
    with pytest.raises(prism.PrismError, match="INVALID"):
        prism.block_norm_fwd(x, wb, y=x.clone(), h=x)


def test_c_entry_points_take_gradients_in_place():
    # d_o over dy and dx over dx_out, which the C interface allows
    o, g, w, dy, x, wb, v, dh, dxo = _train_inputs(3)
    want, want_b = prism.gated_norm_bwd(o, g, w, dy), prism.block_norm_bwd(x, wb, dh, dx_out=dxo, **v)
    L, s = prism.lib(), torch.cuda.current_stream().cuda_stream
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    dg, dw = torch.empty_like(o), torch.empty_like(w)
    p = [t.data_ptr() for t in (o, g, w, dy)]
    assert L.prism_gated_norm_bwd(*p, None, 4, 300, 6, 128, 768, 1e-5, 0, 0, p[3], dg.data_ptr(), dw.data_ptr(),
                                  ws.data_ptr(), ws.numel(), s) == 0
    assert torch.equal(dy, want["o"]) and torch.equal(dg, want["gate"]) and torch.equal(dw, want["weight"])
    dyy, sums = torch.empty_like(dh), torch.empty(3, 768, device="cuda")
    assert L.prism_block_norm_bwd(x.data_ptr(), v["y"].data_ptr(), v["post_weight"].data_ptr(), v["scale"].data_ptr(),
                                  wb.data_ptr(), dh.data_ptr(), dxo.data_ptr(), None, 4, 300, 768, 1.0, 1e-5, 1, 0,
                                  dxo.data_ptr(), dyy.data_ptr(), *(t.data_ptr() for t in sums), ws.data_ptr(),
                                  ws.numel(), s) == 0
    assert torch.equal(dxo, want_b["x"]) and torch.equal(dyy, want_b["y"])
    assert all(torch.equal(a, want_b[n]) for a, n in zip(sums, ("weight", "post_weight", "scale")))


def test_sizes_beyond_32_bits_are_refused():
    x, w = torch.zeros(1, 1, device="cuda").expand((1 << 32) + 8, 1), torch.ones(1, device="cuda")
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.block_norm_fwd(x, w)
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.block_norm_bwd(x, w, x)
    o = torch.zeros(1, 1, 1, 16, device="cuda").expand(1, (1 << 32) + 8, 1, 16)
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.gated_norm_fwd(o, None, torch.ones(16, device="cuda"))


# ------------------------------------------------------------- padding under weights that are not finite
BAD = [float("inf"), float("nan")]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("d,dtype,gate", [(16, "bf16", "dense"), (32, "fp32", "none"), (64, "bf16", "none"),
                                          (64, "fp32", "dense"), (128, "bf16", "slice"), (128, "fp32", "dense")])
def test_gated_norm_padding_is_zero_whatever_the_weight(bad, d, dtype, gate):
    B, T, H = 3, 37, 5
    o, g, w, dy = _gated_inputs(B, T, H, d, DT[dtype], gate)
    gc = None if g is None else torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda").copy_(g)
    w[3] = bad
    for lengths in ([T, 0, 11], [0, 0, 0]):
        lens = torch.tensor(lengths, dtype=torch.int32).cuda()
        y = prism.gated_norm_fwd(o.cuda(), gc, w.cuda(), lengths=lens)
        got = prism.gated_norm_bwd(o.cuda(), gc, w.cuda(), dy.cuda(), lengths=lens)
        pad = ~ref.valid_rows(lengths, B, T)
        for t in (y, got["o"], got["gate"]):
            assert t is None or t.cpu()[pad].eq(0).all()
        assert any(lengths) or got["weight"].eq(0).all()
        # a valid row is what it was: not finite where the weight is not
        assert not any(lengths) or not torch.isfinite(y[0, :, :, 3]).any()


PADDED = [
    (8, "bf16", "bf16", True, True), (40, "fp32", "bf16", True, True), (77, "bf16", "bf16", True, True),
    (77, "fp32", "fp32", False, True), (768, "bf16", "bf16", True, True), (768, "fp32", "bf16", True, False),
    (1001, "fp32", "fp32", True, True), (2056, "bf16", "bf16", True, True), (2056, "fp32", "bf16", False, True),
    (4099, "bf16", "bf16", True, True)
]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("D,stream,dtype,post,scale,which",
                         [(*c, n) for c in PADDED for n, given in (("weight", True), ("post_weight", c[3]), ("scale", c[4]))
                          if given])
def test_block_norm_padding_is_zero_whatever_the_vectors(bad, D, stream, dtype, post, scale, which):
    B, T = 3, 37
    x, w, vec, dh, dxo = _block_inputs(B, T, D, stream, dtype, True, post, scale)
    vec["weight"] = w
    vec[which][3] = bad
    w = vec.pop("weight").cuda()
    v = {n: _cuda(t) for n, t in vec.items()}
    for lengths in ([T, 0, 11], [0, 0, 0]):
        lens = torch.tensor(lengths, dtype=torch.int32).cuda()
        pad = ~ref.valid_rows(lengths, B, T)
        outs = list(prism.block_norm_fwd(x.cuda(), w, lengths=lens, **v))
        got = prism.block_norm_bwd(x.cuda(), w, dh.cuda(), dx_out=dxo.cuda(), lengths=lens, **v)
        outs += [got["x"], got["y"]]
        if which == "weight":  # without y there is only h
            outs += [prism.block_norm_fwd(x.cuda(), w, lengths=lens)[1],
                     prism.block_norm_bwd(x.cuda(), w, dh.cuda(), lengths=lens)["x"]]
        for t in outs:
            assert t.cpu()[pad].eq(0).all()
        if not any(lengths):  # padding adds nothing to any vector's gradient
            assert all(got[n].eq(0).all() for n in ("weight", "post_weight", "scale") if got[n] is not None)


def test_places_behind_the_last_row_add_nothing_to_the_vectors_gradients():
    # fewer rows than a block has places for, and an infinite scale: the sum of infinities of one sign
    # over the rows is that infinity, and becomes NaN if a place without a row adds 0 * inf
    D = 40
    x, w, vec, dh, dxo = _block_inputs(1, 5, D, "fp32", "fp32", True, True, True)
    v = {n: t.cuda() for n, t in vec.items()}
    dx = prism.block_norm_bwd(x.cuda(), w.cuda(), dh.cuda(), dx_out=dxo.cuda(), **v)["x"]  # depends on neither
    v["y"][..., 3] = torch.where(dx[..., 3] > 0, 0.5, -0.5)
    want = prism.block_norm_bwd(x.cuda(), w.cuda(), dh.cuda(), dx_out=dxo.cuda(), **v)
    v["scale"][3] = float("inf")
    got = prism.block_norm_bwd(x.cuda(), w.cuda(), dh.cuda(), dx_out=dxo.cuda(), **v)
    want["post_weight"][3] = float("inf")
    assert all(torch.equal(got[n], want[n]) for n in ("x", "weight", "scale", "post_weight"))
