"""The AdamW step on the GPU (through the C ABI) against its fp64 statement
(oracle/layer_oracle.py) and, for the 8-bit states, against separate fp32 operations.

Tolerances.  A new moment is the sum of two products: at most four roundings on each term
(the coefficient, the scaled gradient and its square, the product) and one of the sum.  The
new parameter adds to p (1 - lr wd), three roundings, the update: the moments' errors, the
root, the division and the coefficients, at most twenty roundings of the update's magnitude.
K = 32 covers each.  bf16 outputs add half a step, 2^-8.
"""

import pytest
import torch

import linear_attention_sequence_shortconv_b200 as prism
from linear_attention_sequence_shortconv_b200 import layer_ops
from oracle import layer_oracle as ref

pytestmark = pytest.mark.gpu

U, K = 2.0 ** -24, 32
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [(1,), (768,), (6, 128, 4), (37, 11), (4096,), (4097,), (100, 777), (255,), (256,), (257,), (0,), (2, 8192)]


def _randn(seed, shape, std=1.0, dtype=torch.float32):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _inputs(sizes, param, grad, seed=0):
    p = [_randn(seed + 10 * i, s, 0.02, DT[param]) for i, s in enumerate(sizes)]
    g = [_randn(seed + 10 * i + 1, s, 1e-3, DT[grad]) for i, s in enumerate(sizes)]
    m = [_randn(seed + 10 * i + 2, s, 3e-4) for i, s in enumerate(sizes)]
    v = [_randn(seed + 10 * i + 3, s, 1e-3) ** 2 for i, s in enumerate(sizes)]
    return p, g, m, v


def _cuda(ts):
    return [t.cuda() for t in ts]


def _check32(p, g, m, v, p0, g0, m0, v0, step, hyper, wd, scale=1.0, copies=None):
    b1, b2 = hyper["betas"]
    for i in range(len(p)):
        decay = wd[i]
        a, b, c = ref.adamw(p0[i].double(), g0[i].double(), m0[i].double(), v0[i].double(), step, hyper["lr"],
                            hyper["betas"], hyper["eps"], decay, scale)
        gs = (scale * g0[i].double()).abs()
        mm, mv = b1 * m0[i].double().abs() + (1 - b1) * gs, b2 * v0[i].double() + (1 - b2) * gs * gs
        root = torch.sqrt(c / (1 - b2 ** step)) + hyper["eps"]
        mp = p0[i].double().abs() + hyper["lr"] / (1 - b1 ** step) * mm / root
        tiny = 2.0 ** -140
        assert ((m[i].double().cpu() - b).abs() <= K * U * mm + tiny).all()
        assert ((v[i].double().cpu() - c).abs() <= K * U * mv + tiny).all()
        assert ((p[i].double().cpu() - a).abs() <= HALF[p[i].dtype] * a.abs() + K * U * mp + tiny).all()
        if copies is not None:
            assert ((copies[i].double().cpu() - a).abs() <= 2.0 ** -8 * a.abs() + K * U * mp + tiny).all()


@pytest.mark.parametrize("param,grad,copies", [("fp32", "fp32", True), ("fp32", "bf16", False), ("bf16", "fp32", False),
                                               ("bf16", "bf16", False)])
@pytest.mark.parametrize("step", [1, 1000])
def test_step_in_32_bits_matches_fp64(param, grad, copies, step):
    p0, g0, m0, v0 = _inputs(SIZES, param, grad)
    p, g, m, v = _cuda(p0), _cuda(g0), _cuda(m0), _cuda(v0)
    c = [torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for t in p] if copies else None
    wd = [0.1 * (i % 3) for i in range(len(p))]  # a decay of its own for each tensor
    scale = torch.tensor([0.25], device="cuda")
    prism.adamw_step(p, g, m, v, step=step, copies=c, grad_scale=scale, **dict(HYPER, weight_decay=wd))
    assert prism.stream_status() == 0
    _check32(p, g, m, v, p0, g0, m0, v0, step, HYPER, wd, 0.25, c)
    if copies:
        assert all(torch.equal(a, b.bfloat16()) for a, b in zip(c, p))


def test_many_tensors_take_more_than_one_launch():
    sizes = [(1 + (7 * i) % 600,) for i in range(1000)]
    p0, g0, m0, v0 = _inputs(sizes, "fp32", "fp32")
    p, g, m, v = _cuda(p0), _cuda(g0), _cuda(m0), _cuda(v0)
    prism.adamw_step(p, g, m, v, step=3, **HYPER)
    _check32(p, g, m, v, p0, g0, m0, v0, 3, HYPER, [0.1] * 1000)


def test_nothing_behind_a_tensor_is_touched():
    # views of flat buffers with guards between them
    sizes, starts, total = [1, 255, 257, 5000], [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // 256) * 256 + 256
    for bits in (32, 8):
        flat = {n: torch.full((total,), 7.0, device="cuda").to(torch.float32 if bits == 32 or n in "pg" else
                                                               torch.float8_e4m3fn) for n in "pgmv"}
        flat["c"] = torch.full((total,), 7.0, device="cuda").bfloat16()
        view = {n: [x[a:a + k] for a, k in zip(starts, sizes)] for n, x in flat.items()}
        more = {}
        if bits == 8:
            more = {n: [torch.ones(-(-k // 256), device="cuda") for k in sizes]
                    for n in ("exp_avg_scale", "exp_avg_sq_scale")}
        prism.adamw_step(view["p"], view["g"], view["m"], view["v"], step=2, copies=view["c"], **more, **HYPER)
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        for a, k in zip(starts, sizes):
            used[a:a + k] = True
        for n, x in flat.items():
            assert x.float()[~used].eq(7).all(), (bits, n)
            # every element inside has moved; a copy is the new parameter in bf16, whose step at 7
            # (2^-5) is above the parameter's change, so it is compared with that instead
            if n == "c":
                assert torch.equal(x[used], flat["p"][used].bfloat16())
            elif n != "g":
                assert not x.float()[used].eq(7).any(), (bits, n)


def _separate_fp32_step(p, g, mc, ms, vc, vs, step, hyper, wd):
    """The step in separate fp32 torch operations: (p, m, root) before the states are rounded."""
    b1, b2 = hyper["betas"]
    m = ref.decode(mc, ms) * b1 + g * (1 - b1)
    r0 = ref.decode(vc, vs)
    v = (r0 * r0) * b2 + (g * g) * (1 - b2)
    # correctly rounded: torch's fp32 square root on the CPU is not, the one in fp64 rounded to
    # fp32 is (53 >= 2 * 24 + 2 bits)
    return m, v.double().sqrt().float()


def _separate_encode(x, root):
    b = ref.state_blocks(x)
    scale = (b.abs().amax(1) * torch.tensor(1 / ref.E4M3_MAX)).clamp_min(2.0 ** -126)
    codes = (b * (1 / scale)[:, None]).to(torch.float8_e4m3fn).view(-1)[:x.numel()].view(x.shape)
    if root:
        raw = codes.view(torch.uint8)
        codes = torch.where((raw == 0) & (x > 0), 1, raw).to(torch.uint8).view(torch.float8_e4m3fn)
    return codes, scale


@pytest.mark.parametrize("param,grad", [("fp32", "fp32"), ("bf16", "bf16")])
def test_step_in_8_bits(param, grad):
    sizes = [s for s in SIZES if s != (0,)]
    p0, g0, _, _ = _inputs(sizes, param, grad)
    # gradients over many magnitudes in one block, and zeros
    g0 = [(t.float() * 10.0 ** (-6 * torch.rand(t.shape, generator=torch.Generator().manual_seed(5)))).to(t.dtype)
          for t in g0]
    for t in g0:
        t.view(-1)[::7] = 0
    p, g = _cuda(p0), _cuda(g0)
    state = prism.adamw_state(p, bits=8)
    for step in (1, 2, 3):
        before = {n: [t.cpu() for t in x] for n, x in state.items()}
        held = [t.cpu() for t in p]
        prism.adamw_step(p, g, step=step, **HYPER, **state)
        assert prism.stream_status() == 0
        for i in range(len(p)):
            old = [before[n][i] for n in ("exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale")]
            m, root = _separate_fp32_step(held[i], g0[i].float(), *old, step, HYPER, 0.1)
            for name, x, is_root in (("exp_avg", m, False), ("exp_avg_sq", root, True)):
                codes, scale = _separate_encode(x, is_root)
                assert torch.equal(state[name + "_scale"][i].cpu(), scale)
                assert torch.equal(state[name][i].cpu().view(torch.uint8), codes.view(torch.uint8))
                # what is held is within half a step of e4m3, or of its smallest number; a root
                # that is not zero is held as at least that number
                value = ref.decode(state[name][i].cpu(), scale.double())
                least = ref.decode(torch.ones_like(codes.float()), scale.double()) * 2.0 ** -9
                slack = torch.maximum(2.0 ** -4 * x.double().abs(), least * (1.0 if is_root else 0.5))
                assert ((value - x.double()).abs() <= (1 + 2.0 ** -20) * slack).all()
                assert not is_root or ((value > 0) == (x > 0)).all()
            m_old, r_old = ref.decode(old[0], old[1].double()), ref.decode(old[2], old[3].double())
            a, b, c = ref.adamw(held[i].double(), g0[i].double(), m_old, r_old ** 2, step, HYPER["lr"], HYPER["betas"],
                                HYPER["eps"], 0.1)
            mm = 0.9 * m_old.abs() + (1 - 0.9) * g0[i].double().abs()
            mp = held[i].double().abs() + HYPER["lr"] / (1 - 0.9 ** step) * mm / (
                torch.sqrt(c / (1 - 0.95 ** step)) + 1e-8)
            assert ((p[i].double().cpu() - a).abs() <= HALF[p[i].dtype] * a.abs() + K * U * mp + 2.0 ** -140).all()


def test_extreme_gradients_stay_in_their_block():
    n = 1024
    for bits in (32, 8):
        p, g = [torch.ones(n, device="cuda")], [torch.ones(n, device="cuda")]
        g[0][300], g[0][700] = float("nan"), float("inf")
        state = prism.adamw_state(p, bits=bits)
        prism.adamw_step(p, g, step=1, **HYPER, **state)
        bad = torch.zeros(n, dtype=torch.bool)
        bad[[300, 700]] = True
        assert torch.equal(~torch.isfinite(p[0].cpu()), bad)
        held = state["exp_avg"][0].float().cpu()
        if bits == 8:
            held = ref.decode(state["exp_avg"][0].cpu(), state["exp_avg_scale"][0].cpu())
            bad = torch.zeros(n, dtype=torch.bool)
            bad[256:768] = True
        assert torch.equal(~torch.isfinite(held), bad)
    # the smallest and the largest gradients
    p, g = [torch.zeros(512, device="cuda")], [torch.full((512,), 1e-38, device="cuda")]
    g[0][256:] = 1e18
    state = prism.adamw_state(p, bits=8)
    prism.adamw_step(p, g, step=1, **HYPER, **state)
    assert torch.isfinite(p[0]).all() and torch.isfinite(state["exp_avg_sq_scale"][0]).all()
    assert torch.allclose(p[0][256:], torch.full((256,), -3e-3, device="cuda"), rtol=1e-5)


def test_step_and_rate_on_the_device():
    p0, g0, m0, v0 = _inputs([(700,), (33, 5)], "fp32", "fp32")
    for step, lr in ((1, 1e-2), (7, 3e-3), (10 ** 6, 1e-5)):
        a = [_cuda(t) for t in (p0, g0, m0, v0)]
        b = [_cuda(t) for t in (p0, g0, m0, v0)]
        rate = torch.tensor([lr], device="cuda")
        prism.adamw_step(*a, step=step, **dict(HYPER, lr=rate.item()))
        prism.adamw_step(*b, step=torch.tensor([step], dtype=torch.int32, device="cuda"), **dict(HYPER, lr=rate))
        for x, y in zip(a, b):
            for s, t in zip(x, y):
                assert torch.allclose(s, t, rtol=2 * U, atol=0)  # the same factors, up to their rounding to fp32
    # a step below one counts as one
    a, b = [_cuda(t) for t in (p0, g0, m0, v0)], [_cuda(t) for t in (p0, g0, m0, v0)]
    prism.adamw_step(*a, step=torch.tensor([0], dtype=torch.int32, device="cuda"), **HYPER)
    prism.adamw_step(*b, step=torch.tensor([1], dtype=torch.int32, device="cuda"), **HYPER)
    assert all(torch.equal(s, t) for x, y in zip(a, b) for s, t in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_graph_follows_step_rate_and_gradients(bits):
    p0, g0, _, _ = _inputs([(900,), (40, 30)], "fp32", "bf16")
    runs = []
    for captured in (False, True):
        p, g = _cuda(p0), _cuda(g0)
        state = prism.adamw_state(p, bits=bits)
        step = torch.ones(1, dtype=torch.int32, device="cuda")
        lr = torch.tensor([1e-3], device="cuda")

        def one():
            prism.adamw_step(p, g, step=step, **dict(HYPER, lr=lr), **state)

        graph = None
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        for i in range(4):
            step.fill_(i + 1)
            lr.fill_(1e-3 / (i + 1))
            for k, t in enumerate(g):
                t.copy_(_randn(100 * i + k, t.shape, 1e-3, t.dtype))
            graph.replay() if captured else one()
        torch.cuda.synchronize()
        runs.append(p + [t.float() for x in state.values() for t in x])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_another_stream_and_repetition():
    p0, g0, m0, v0 = _inputs(SIZES, "fp32", "fp32")
    runs = []
    for k in range(3):
        a = [_cuda(t) for t in (p0, g0, m0, v0)]
        s = torch.cuda.Stream() if k == 2 else None
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        prism.adamw_step(*a, step=5, stream=s, **HYPER)
        torch.cuda.synchronize()
        runs.append(a)
    for other in runs[1:]:
        assert all(torch.equal(s, t) for x, y in zip(runs[0], other) for s, t in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
def test_both_ways_to_read_the_lists_agree(bits, monkeypatch):
    p0, g0, _, _ = _inputs(SIZES, "fp32", "bf16")
    runs = []
    for slow in (False, True):
        if slow:
            monkeypatch.setattr(layer_ops, "_dl_exchange", lambda: None)
        else:
            assert layer_ops._dl_exchange() is not None
        p = torch.nn.ParameterList([torch.nn.Parameter(t) for t in _cuda(p0)])
        c = tuple(torch.zeros_like(t, dtype=torch.bfloat16) for t in p)
        state = prism.adamw_state(list(p), bits=bits)
        with torch.no_grad():
            prism.adamw_step(p, _cuda(g0), step=1, copies=c, **HYPER, **state)
        runs.append([*p, *c] + [t.float() for x in state.values() for t in x])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_refusals_name_the_argument():
    t = [torch.zeros(600, device="cuda") for _ in range(4)]
    one = [[x] for x in t]
    with pytest.raises(ValueError, match="grads"):
        prism.adamw_step(one[0], [], one[2], one[3])
    with pytest.raises(TypeError, match="exp_avg_sq"):
        prism.adamw_step(one[0], one[1], one[2], [t[3].bfloat16()])
    with pytest.raises(ValueError, match="shapes"):
        prism.adamw_step(one[0], [t[1][:599]], one[2], one[3])
    with pytest.raises(ValueError, match="cpu"):
        prism.adamw_step(one[0], [t[1].cpu()], one[2], one[3])
    with pytest.raises(Exception):
        prism.adamw_step(one[0], [None], one[2], one[3])
    with pytest.raises(ValueError, match="contiguous"):
        prism.adamw_step([t[0].view(20, 30).t()], [t[1].view(30, 20)], [t[2].view(30, 20)], [t[3].view(30, 20)])
    with pytest.raises(ValueError, match="exp_avg_scale"):
        prism.adamw_step(one[0], one[1], [t[2].to(torch.float8_e4m3fn)], [t[3].to(torch.float8_e4m3fn)])
    s8 = prism.adamw_state(one[0], bits=8)
    with pytest.raises(ValueError, match="256"):
        prism.adamw_step(one[0], one[1], **dict(s8, exp_avg_scale=[torch.zeros(2, device="cuda")]))
    with pytest.raises(ValueError, match="scales"):
        prism.adamw_step(*one, exp_avg_scale=[t[0]])
    with pytest.raises(ValueError, match="copies"):
        prism.adamw_step([t[0].bfloat16()], one[1], one[2], one[3], copies=[t[0].bfloat16()])
    with pytest.raises(TypeError, match="step"):
        prism.adamw_step(*one, step=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="lr"):
        prism.adamw_step(*one, lr=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="weight_decay"):
        prism.adamw_step(*one, weight_decay=[0.1, 0.2])
    with pytest.raises(prism.PrismError, match="INVALID"):
        prism.adamw_step(*one, step=0)
    with pytest.raises(prism.PrismError, match="INVALID"):  # the same parameter twice
        prism.adamw_step([t[0], t[0]], [t[1], t[1]], [t[2], t[2].clone()], [t[3], t[3].clone()])
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):  # not on 16 bytes
        prism.adamw_step([t[0][1:]], [t[1][1:]], [t[2][1:]], [t[3][1:]])
    assert all(not x.any() for x in t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,wd", [(1e-4, 1e-4), (1e-4, 3e-4), (1e-4, 1e-3), (1e-4, 1e-2)])
def test_a_small_decay_is_the_one_asked_for(bits, lr, wd):
    """lr wd from 1e-8 to 1e-6, where 1 - lr wd in fp32 is up to 100% off: the mean change of many
    parameters against the one in fp64.

    Every parameter stands twice, with opposite gradients, so that what the mean change holds of
    the updates is their roundings, at most K 2^-24 of their mean magnitude.  A new parameter in
    (1, 2) is rounded to a step of 2^-23: over n mantissas and updates that spread over more than
    500 steps the mean rounding is below 8 standard deviations, 8 step / sqrt(12 n), and
    1/500 of a step.
    """
    n, eps = 1 << 20, 1.0
    gen = torch.Generator().manual_seed(4)
    p0 = (1.001 + 0.998 * torch.rand(n // 2, generator=gen)).repeat(2)
    g0 = 0.5 + 3.5 * torch.rand(n // 2, generator=gen)  # g / (g + eps) from 0.33 to 0.8
    g0 = torch.cat([g0, -g0])
    p, state = [p0.cuda()], prism.adamw_state([p0.cuda()], bits=bits)
    prism.adamw_step(p, [g0.cuda()], step=1, lr=lr, betas=(0.9, 0.95), eps=eps, weight_decay=wd, **state)
    zero = torch.zeros(n, dtype=torch.float64)
    want, _, _ = ref.adamw(p0.double(), g0.double(), zero, zero, 1, lr, (0.9, 0.95), eps, wd)
    update = (p0.double() * (1 - lr * wd) - want).abs().mean().item()
    step = 2.0 ** -23
    bound = K * U * (update + 2 * lr * wd) + 8 * step / (12 * n) ** 0.5 + step / 500
    assert abs((p[0].double().cpu() - want).mean().item()) <= bound


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_infinite_parameters_stay(bits, wd):
    # such as the entries of a bias that masks
    p, inf = [torch.full((700,), 0.5, device="cuda")], float("inf")
    p[0][3], p[0][300], p[0][699] = -inf, inf, -inf
    prism.adamw_step(p, [torch.zeros(700, device="cuda")], step=1, lr=0.1, weight_decay=wd,
                     **prism.adamw_state(p, bits=bits))
    want = torch.full((700,), 0.5 * (1 - 0.1 * wd))
    want[3], want[300], want[699] = -inf, inf, -inf
    assert torch.allclose(p[0].cpu(), want, rtol=2 * U, atol=0)


@pytest.mark.parametrize("slow", [False, True])
def test_what_is_no_tensor_is_named(slow, monkeypatch):
    # such as the gradient of a parameter that took no part
    if slow:
        monkeypatch.setattr(layer_ops, "_dl_exchange", lambda: None)
    p = [torch.ones(300, device="cuda") for _ in range(3)]
    g = [torch.ones(300, device="cuda"), None, torch.ones(300, device="cuda")]
    state = prism.adamw_state(p)
    with pytest.raises(TypeError, match="grads.*NoneType"):
        prism.adamw_step(p, g, **state)
    with pytest.raises(TypeError, match="params.*float"):
        prism.adamw_step([p[0], 1.0, p[2]], [g[0], g[2], g[0]], **state)
    with pytest.raises(TypeError, match="exp_avg_sq.*list"):
        prism.adamw_step(p[:2], g[::2], state["exp_avg"][:2], [state["exp_avg_sq"][0], [1.0]])
    assert all(t.eq(1).all() for t in p)
