"""Pins of the fp64 statements of the operators around the mixer (CPU): hand-computed values,
and gradients against central differences of the forward statements."""
import math

import pytest
import torch

from oracle import layer_oracle as ref

F64 = torch.float64


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_gated_norm_by_hand():
    # mean(3^2, 4^2) = 12.5, eps = 3.5: r = 1/4
    o = torch.tensor([[[[3.0, 4.0]]]], dtype=F64)
    w = torch.tensor([2.0, 1.0], dtype=F64)
    g = torch.tensor([[[[0.0, math.log(3.0)]]]], dtype=F64)  # sigmoid: 1/2, 3/4
    assert torch.allclose(ref.gated_norm(o, None, w, eps=3.5), torch.tensor([1.5, 1.0], dtype=F64))
    assert torch.allclose(ref.gated_norm(o, g, w, eps=3.5, act="sigmoid"), torch.tensor([0.75, 0.75], dtype=F64))
    assert torch.allclose(ref.gated_norm(o, g, w, eps=3.5), torch.tensor([0.0, 0.75 * math.log(3.0)], dtype=F64))


def test_block_norm_by_hand():
    x, y = torch.tensor([[[1.0, 2.0]]], dtype=F64), torch.tensor([[[2.0, 2.0]]], dtype=F64)
    w, s = torch.ones(2, dtype=F64), torch.tensor([1.0, 0.5], dtype=F64)
    x_out, h = ref.block_norm(x, w, y=y, scale=s, res_scale=2.0, eps=11.5)  # x_out = (5, 4), mean square 20.5
    assert torch.allclose(x_out, torch.tensor([5.0, 4.0], dtype=F64))
    assert torch.allclose(h, torch.tensor([5.0, 4.0], dtype=F64) / math.sqrt(32.0))


def test_adamw_first_step_by_hand():
    # the first step moves by lr * sign(g) (eps = 0), after the decay
    p, g = torch.tensor([1.0, -2.0], dtype=F64), torch.tensor([0.3, -5.0], dtype=F64)
    z = torch.zeros(2, dtype=F64)
    new, m, v = ref.adamw(p, g, z, z, 1, 0.1, (0.9, 0.99), 0.0, 0.5)
    assert torch.allclose(new, torch.tensor([0.95 - 0.1, -1.9 + 0.1], dtype=F64))
    assert torch.allclose(m, 0.1 * g) and torch.allclose(v, 0.01 * g * g)


def _differences(f, x, at, h=1e-5):
    out = []
    for i in at:
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        out.append((f(a) - f(b)) / (2 * h))
    return torch.stack(out)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_norm_gradients_are_the_differences(act):
    o, g, w, dy = _randn(1, 2, 3, 2, 16), _randn(2, 2, 3, 2, 16), _randn(3, 16), _randn(4, 2, 3, 2, 16)
    lengths = [3, 1]
    leaves = [t.clone().requires_grad_(True) for t in (o, g, w)]
    grads = torch.autograd.grad((ref.gated_norm(*leaves, lengths, act=act) * dy).sum(), leaves)
    for k, x in enumerate((o, g, w)):
        at = [0, 5, x.numel() // 2, x.numel() - 1]
        args = [o, g, w]

        def loss(t):
            return (ref.gated_norm(*args[:k], t, *args[k + 1:], lengths, act=act) * dy).sum()

        assert torch.allclose(grads[k].view(-1)[at], _differences(loss, x, at), rtol=1e-7, atol=1e-8)


def test_block_norm_gradients_are_the_differences():
    x, y, w, wp, s = _randn(1, 2, 3, 9), _randn(2, 2, 3, 9), _randn(3, 9), _randn(4, 9), _randn(5, 9)
    dh, dxo, lengths = _randn(6, 2, 3, 9), _randn(7, 2, 3, 9), [2, 3]
    x_out, _ = ref.block_norm(x, w, y, wp, s, 0.7, lengths)
    got = ref.block_norm_grad(x_out, w, dh, y, wp, s, 0.7, dxo, lengths)
    args = {"x": x, "weight": w, "y": y, "post_weight": wp, "scale": s}
    keep = ref.valid_rows(lengths, 2, 3)[..., None]

    for name, value in args.items():
        def loss(t):
            a = dict(args, **{name: t})
            xo, h = ref.block_norm(a["x"], a["weight"], a["y"], a["post_weight"], a["scale"], 0.7, lengths)
            return (torch.where(keep, dxo, 0.0) * xo).sum() + (dh * h).sum()

        at = [0, 4, value.numel() // 2, value.numel() - 1]
        assert torch.allclose(got[name].reshape(-1)[at], _differences(loss, value, at), rtol=1e-6, atol=1e-7), name


def test_embedding_gradient_is_the_sum_over_its_tokens():
    ids = torch.tensor([[1, 4, 1], [0, 1, 2]])
    table = _randn(1, 5, 3).requires_grad_(True)
    d = _randn(2, 2, 3, 3)
    (ref.embed(ids, table, 2.0, [3, 2]) * d).sum().backward()
    want = torch.zeros(5, 3, dtype=F64)
    for b, t, v in ((0, 0, 1), (0, 1, 4), (0, 2, 1), (1, 0, 0), (1, 1, 1)):
        want[v] += 2.0 * d[b, t]
    assert torch.allclose(table.grad, want)
