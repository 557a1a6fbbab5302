"""The operators around the mixer together with it, as a model uses them: one training step of
a one-layer model (embedding, pre-norm, mixer, readout norm, block border; their backward; the
optimiser), and the same model served token by token.

Both run in fp32 and are held to the error bars of the mixer's own tests: 1e-4 forward, 2e-4
for gradients, relative to the largest value (the operators around the mixer add a few units
of 2^-24, far below).
"""
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import linear_attention_sequence_shortconv_b200 as prism
from oracle import layer_oracle as ref
from oracle.prism_grad import prism_seq_torch

pytestmark = pytest.mark.gpu

B, T, H, d, V, W = 3, 90, 2, 32, 41, 4
D = H * d
EPS, SCALE = 1e-5, math.sqrt(D)
LENGTHS = [90, 0, 33]
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def _params():
    g = torch.Generator().manual_seed(1)
    r = lambda *s, std: std * torch.randn(s, generator=g)  # noqa: E731
    return {"table": r(V, D, std=0.1), "norm1": 1 + r(D, std=0.1), "wq": r(D, D, std=0.1), "wk": r(D, D, std=0.1),
            "wv": r(D, D, std=0.1), "wg": r(D, D, std=0.1), "wb": r(D, 2 * H, std=0.1), "conv_w": r(H, d, W, std=0.5),
            "norm_o": 1 + r(d, std=0.1), "wo": r(D, D, std=0.1), "post": 1 + r(D, std=0.1),
            "scale": 0.5 + r(D, std=0.1), "norm2": 1 + r(D, std=0.1)}


def _batch():
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(0, V, (B, T), generator=g)
    keep = ref.valid_rows(LENGTHS, B, T)[..., None]
    return ids, torch.randn((B, T, D), generator=g) * keep, torch.randn((B, T, D), generator=g) * keep


def _gates(h, wb):
    s = torch.sigmoid(h @ wb)
    return (0.5 + 0.5 * s[..., :H]).contiguous(), s[..., H:].contiguous()  # decay, step size


def _heads(x):
    return x.view(*x.shape[:-1], H, d)


def _unit(x):
    """Keys and queries of unit length, as the mixer's callers make them: the state's transition
    gamma (I - beta k k^T) has the eigenvalue gamma (1 - beta |k|^2), which is stable for
    beta |k|^2 < 2; the projections here have |k|^2 near 20, and an error would grow by 7 a token."""
    return x / x.square().sum(-1, keepdim=True).add(1e-12).sqrt()


def _unit_grad(x, g):
    n, u = x.square().sum(-1, keepdim=True).add(1e-12).sqrt(), _unit(x)
    return (g - u * (u * g).sum(-1, keepdim=True)) / n


def _reference(p, ids, dh, dx):
    """Loss and gradients in fp64 by automatic differentiation."""
    p = {n: t.double().requires_grad_(True) for n, t in p.items()}
    x = ref.embed(ids, p["table"], SCALE, LENGTHS)
    _, h = ref.block_norm(x, p["norm1"], lengths=LENGTHS, eps=EPS)
    q, k, v, g = (_heads(h @ p[n]) for n in ("wq", "wk", "wv", "wg"))
    gamma, beta = _gates(h, p["wb"])
    o, _ = prism_seq_torch(_unit(q), _unit(k), v, gamma, beta, None, None, None, p["conv_w"], lengths=LENGTHS)
    y = ref.gated_norm(o, g, p["norm_o"], LENGTHS, EPS)
    x2, h2 = ref.block_norm(x, p["norm2"], y.reshape(B, T, D) @ p["wo"], p["post"], p["scale"], 1.0, LENGTHS, EPS)
    loss = (h2 * dh.double()).sum() + (x2 * dx.double()).sum()
    grads = torch.autograd.grad(loss, list(p.values()), allow_unused=True)
    return h2.detach(), {n: torch.zeros_like(t) if gr is None else gr for (n, t), gr in zip(p.items(), grads)}


def _rel(got, want):
    return ((got.double().cpu() - want).abs().max() / want.abs().max().clamp_min(1e-12)).item()


def _forward(p, ids, lens):
    x = prism.embed_fwd(ids, p["table"], scale=SCALE, lengths=lens)
    _, h = prism.block_norm_fwd(x, p["norm1"], lengths=lens, eps=EPS)
    q, k, v = (_heads(h @ p[n]) for n in ("wq", "wk", "wv"))
    gate = _heads(h @ p["wg"])
    gamma, beta = _gates(h, p["wb"])
    o, _ = prism.scan_fwd(_unit(q), _unit(k), v, gamma, beta, None, None, None, p["conv_w"], L=1, chunk=16, lengths=lens)
    y = prism.gated_norm_fwd(o, gate, p["norm_o"], lengths=lens, eps=EPS)
    z = y.view(B, T, D) @ p["wo"]
    x2, h2 = prism.block_norm_fwd(x, p["norm2"], y=z, post_weight=p["post"], scale=p["scale"], lengths=lens, eps=EPS)
    return x, h, (q, k, v, gamma, beta), gate, o, y, z, x2, h2


def _flat(x):
    return x.reshape(-1, x.shape[-1])


@pytest.fixture(autouse=True)
def full_fp32_products():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


def test_training_step():
    p0 = _params()
    ids0, dh0, dx0 = _batch()
    h64, want = _reference(p0, ids0, dh0, dx0)
    p = {n: t.cuda() for n, t in p0.items()}
    ids, dh, dx = ids0.cuda(), dh0.cuda(), dx0.cuda()
    lens = torch.tensor(LENGTHS, dtype=torch.int32).cuda()
    x, h, (q, k, v, gamma, beta), gate, o, y, z, x2, h2 = _forward(p, ids, lens)
    assert _rel(h2, h64) <= 1e-4

    g = {}
    b2 = prism.block_norm_bwd(x2, p["norm2"], dh, y=z, post_weight=p["post"], scale=p["scale"], dx_out=dx,
                              lengths=lens, eps=EPS)
    g["norm2"], g["post"], g["scale"] = b2["weight"], b2["post_weight"], b2["scale"]
    g["wo"] = _flat(y.view(B, T, D)).t() @ _flat(b2["y"])
    dy = _heads(b2["y"] @ p["wo"].t())
    gn = prism.gated_norm_bwd(o, gate, p["norm_o"], dy, lengths=lens, eps=EPS)
    g["norm_o"] = gn["weight"]
    s = prism.scan_bwd(_unit(q), _unit(k), v, gamma, beta, None, None, None, p["conv_w"], gn["o"], L=1, lengths=lens)
    g["conv_w"] = s["conv_w"]
    dh1 = torch.zeros_like(h)
    for n, t in (("wq", _unit_grad(q, s["q"])), ("wk", _unit_grad(k, s["k"])), ("wv", s["v"]), ("wg", gn["gate"])):
        t = t.reshape(B, T, D)
        g[n] = _flat(h).t() @ _flat(t)
        dh1 += t @ p[n].t()
    sg, sb = 2 * gamma - 1, beta  # gamma = (1 + sigmoid) / 2
    db = torch.cat([0.5 * s["gamma"] * sg * (1 - sg), s["beta"] * sb * (1 - sb)], -1)
    g["wb"] = _flat(h).t() @ _flat(db)
    dh1 += db @ p["wb"].t()
    b1 = prism.block_norm_bwd(x, p["norm1"], dh1, dx_out=b2["x"], lengths=lens, eps=EPS)
    g["norm1"] = b1["weight"]
    g["table"] = prism.embed_bwd(ids, b1["x"], V, scale=SCALE, lengths=lens)
    assert prism.stream_status() == 0
    for n in p:  # conv_w has no gradient where there is no residual write
        assert (_rel(g[n], want[n]) <= 2e-4) if want[n].any() else not g[n].any(), n

    # the optimiser, on the gradients as they are
    names = list(p)
    before = {n: p[n].cpu().double() for n in names}
    for bits in (32, 8):
        params = [p0[n].cuda() for n in names]
        state = prism.adamw_state(params, bits=bits)
        prism.adamw_step(params, [g[n] for n in names], step=1, **HYPER, **state)
        for t, n in zip(params, names):
            zero = torch.zeros_like(before[n])
            new, _, _ = ref.adamw(before[n], g[n].cpu().double(), zero, zero, 1, HYPER["lr"], HYPER["betas"],
                                  HYPER["eps"], HYPER["weight_decay"])
            # the first step moves every parameter by at most lr: 32 roundings of |p| + lr
            assert ((t.cpu().double() - new).abs() <= 32 * 2.0 ** -24 * (before[n].abs() + 2 * HYPER["lr"])).all(), n


def test_serving_token_by_token_is_the_forward():
    p = {n: t.cuda() for n, t in _params().items()}
    ids = _batch()[0].cuda()
    steps = 20
    *_, h2 = _forward(p, ids, None)
    S = torch.zeros((B, H, d, d), device="cuda")
    hist = torch.zeros((B, H, W - 1, d), device="cuda")
    worst = 0.0
    for t in range(steps):
        x = prism.embed_fwd(ids[:, t].contiguous(), p["table"], scale=SCALE)
        _, h = prism.block_norm_fwd(x, p["norm1"], eps=EPS)
        q, k, v, gate = (_heads(h @ p[n]) for n in ("wq", "wk", "wv", "wg"))
        gamma, beta = _gates(h, p["wb"])
        o = prism.decode_step(_unit(q), _unit(k), v, gamma, beta, None, None, None, p["conv_w"], hist, S, L=1)
        y = prism.gated_norm_fwd(o, gate, p["norm_o"], eps=EPS)
        _, out = prism.block_norm_fwd(x, p["norm2"], y=y.view(B, D) @ p["wo"], post_weight=p["post"],
                                      scale=p["scale"], eps=EPS)
        worst = max(worst, ((out - h2[:, t]).abs().max() / h2.abs().max()).item())
    assert prism.stream_status() == 0 and worst <= 1e-4


def test_training_step_replayed_from_a_graph():
    # forward, backward of the operators and the optimiser in one captured graph, with the step
    # and the rate on the device: as the same calls made one by one
    p0 = _params()
    ids0, dh0, dx0 = _batch()
    lens = torch.tensor(LENGTHS, dtype=torch.int32).cuda()
    dh, dx = dh0.cuda(), dx0.cuda()
    names = ["table", "norm1", "post", "scale", "norm2"]
    runs = []
    for captured in (False, True):
        p = {n: p0[n].cuda() for n in names}
        state = prism.adamw_state([p[n] for n in names], bits=8)
        ids = ids0.cuda()
        step, lr = torch.ones(1, dtype=torch.int32, device="cuda"), torch.full((1,), 1e-2, device="cuda")

        def one():
            x = prism.embed_fwd(ids, p["table"], scale=SCALE, lengths=lens)
            _, z = prism.block_norm_fwd(x, p["norm1"], lengths=lens)
            x2, _ = prism.block_norm_fwd(x, p["norm2"], y=z, post_weight=p["post"], scale=p["scale"], lengths=lens)
            b2 = prism.block_norm_bwd(x2, p["norm2"], dh, y=z, post_weight=p["post"], scale=p["scale"], dx_out=dx,
                                      lengths=lens)
            b1 = prism.block_norm_bwd(x, p["norm1"], b2["y"], dx_out=b2["x"], lengths=lens)
            dt = prism.embed_bwd(ids, b1["x"], V, scale=SCALE, lengths=lens)
            prism.adamw_step([p[n] for n in names],
                             [dt, b1["weight"], b2["post_weight"], b2["scale"], b2["weight"]],
                             **dict(HYPER, step=step, lr=lr), **state)

        graph = None
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        for i in range(4):
            step.fill_(i + 1)
            ids.copy_(torch.roll(ids0, i, 1))
            graph.replay() if captured else one()
        torch.cuda.synchronize()
        runs.append([p[n] for n in names] + [t.float() for x in state.values() for t in x])
    assert prism.stream_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_autograd_sees_what_a_call_writes():
    # a graph that still needs the old values fails instead of taking the new ones
    r = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    w = torch.nn.Parameter(r(300))
    for bits in (32, 8):
        state = prism.adamw_state([w], bits=bits)
        loss = (w * w).sum()
        with torch.no_grad():
            prism.adamw_step([w], [r(300)], **state)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()

    def bumps(written, call):
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before))

    p, g = [r(300)], [r(300)]
    for bits in (32, 8):
        state, copies = prism.adamw_state(p, bits=bits), [torch.zeros(300, dtype=torch.bfloat16, device="cuda")]
        bumps([*p, *copies, *(t for x in state.values() for t in x)],
              lambda: prism.adamw_step(p, g, copies=copies, **state))
    assert g[0]._version == 0
    o, x, y, h, out, dt = r(2, 3, H, d), r(2, 3, D), r(2, 3, D), r(2, 3, D), r(2, 3, D), r(V, D)
    ids = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    bumps([o], lambda: prism.gated_norm_fwd(o, None, r(d), y=o))
    bumps([x, h], lambda: prism.block_norm_fwd(x, r(D), y=y, x_out=x, h=h))
    bumps([h], lambda: prism.block_norm_fwd(x, r(D), h=h))
    bumps([out], lambda: prism.embed_fwd(ids, dt, out=out))
    bumps([dt], lambda: prism.embed_bwd(ids, out, V, d_table=dt, accumulate=True))
    assert y._version == 0 and ids._version == 0
    # the mixer's calls as well
    S, hist, ob = r(2, H, d, d), r(2, H, W - 1, d), r(2, H, d)
    q, gamma = r(2, H, d), torch.rand((2, H), device="cuda")
    bumps([S, hist, ob], lambda: prism.decode_step(q, q, q, gamma, gamma, None, None, None, r(H, d, W), hist, S, L=1,
                                                   o=ob))
    q, gamma, os = r(2, 3, H, d), torch.rand((2, 3, H), device="cuda"), r(2, 3, H, d)
    for scan in (prism.scan_fwd, prism.scan_fwd_static):
        bumps([S, os], lambda: scan(q, q, q, gamma, gamma, None, None, None, r(H, d, W), L=1, chunk=16, o=os, S_final=S))
    bumps([S], lambda: prism.state_affine(S, r(2, H, d, d), out=S))
    assert q._version == 0 and gamma._version == 0
    # inference tensors have no version and are written as before
    with torch.inference_mode():
        t = torch.zeros(300, device="cuda")
        prism.adamw_step([t], [torch.ones(300, device="cuda")], lr=0.5, **prism.adamw_state([t]))
    assert torch.allclose(t, torch.full_like(t, -0.5))


def test_two_threads_call_at_once():
    # the gated norm, the lookup and the AdamW step from two host threads, each on a stream of its own
    def inputs(k):
        g = torch.Generator().manual_seed(k)
        r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        ids = torch.randint(0, 500, (2, 300), generator=g).cuda()
        return dict(o=r(2, 300, 3, 64 << k), gate=r(2, 300, 3, 64 << k), w=r(64 << k), dy=r(2, 300, 3, 64 << k), ids=ids,
                    table=r(500, 40 + k), p=[r(700 + k), r(3, 5000)], g=[r(700 + k), r(3, 5000)])

    def run(x, s):
        p = [t.clone() for t in x["p"]]
        state = prism.adamw_state(p, bits=8)
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        out = [prism.gated_norm_fwd(x["o"], x["gate"], x["w"], stream=s),
               *prism.gated_norm_bwd(x["o"], x["gate"], x["w"], x["dy"], stream=s).values(),
               prism.embed_fwd(x["ids"], x["table"], stream=s)]
        for step in (1, 2):
            prism.adamw_step(p, x["g"], step=step, stream=s, **state)
        return out + p + [t.float() if s is None else t for n in state for t in state[n]]

    work = [inputs(k) for k in (0, 1)]
    want = [run(x, None) for x in work]
    torch.cuda.synchronize()

    def many(x):
        s = torch.cuda.Stream()
        out = [run(x, s) for _ in range(20)]
        s.synchronize()
        return out

    with ThreadPoolExecutor(2) as pool:
        for outs, first in zip(pool.map(many, work), want):
            for out in outs:
                assert all(torch.equal(a.float(), b) for a, b in zip(out, first))
    assert prism.stream_status() == 0


def test_a_refused_type_names_its_argument():
    o, x, w = torch.zeros(2, 3, H, d, device="cuda"), torch.zeros(2, 3, D, device="cuda"), torch.ones(D, device="cuda")
    ids, table = torch.zeros((2, 3), dtype=torch.int64, device="cuda"), torch.zeros(V, D, device="cuda")
    p = [torch.zeros(300, device="cuda")]
    half = torch.float16
    for name, call in (("^o ", lambda: prism.gated_norm_fwd(o.to(half), None, w[:d])),
                       ("^o ", lambda: prism.gated_norm_bwd(o.to(half), None, w[:d], o)),
                       ("^x ", lambda: prism.block_norm_fwd(x.to(half), w)),
                       ("^x_out ", lambda: prism.block_norm_bwd(x.to(half), w, x)),
                       ("^dh ", lambda: prism.block_norm_bwd(x, w, x.to(half))),
                       ("^table ", lambda: prism.embed_fwd(ids, table.to(half))),
                       ("^d_out ", lambda: prism.embed_bwd(ids, x.to(half), V)),
                       ("^params ", lambda: prism.adamw_step([p[0].to(half)], p, p, p)),
                       ("^grads ", lambda: prism.adamw_step(p, [p[0].to(half)], p, p))):
        with pytest.raises(TypeError, match=name + ".*float16"):
            call()
