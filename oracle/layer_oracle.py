"""The operators around the mixer for the CPU oracle (PyTorch, fp64, CPU).

TEST INFRASTRUCTURE, like prism_oracle.py: the library never imports it.

Each operator is stated once, from its definition in include/prism.h, with differentiable
torch operations; gradients are taken by reverse-mode automatic differentiation of that
statement (tests/test_oracle_layer.py pins them to central differences).
"""
from __future__ import annotations

import torch

E4M3_MAX = 448.0
STATE_BLOCK = 256


def valid_rows(lengths, B, T):
    """[B, T] bool: the steps that are not padding."""
    if lengths is None:
        return torch.ones((B, T), dtype=torch.bool)
    return torch.arange(T)[None, :] < torch.as_tensor(lengths)[:, None]


def rms_norm(x, weight, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def gated_norm(o, gate, weight, lengths=None, eps=1e-5, act="silu"):
    """o, gate [B,T,H,d] (gate may be None); padding rows give zero."""
    keep = valid_rows(lengths, *o.shape[:2])[..., None, None]
    y = rms_norm(torch.where(keep, o, 0.0), weight, eps)
    if gate is not None:
        g = torch.where(keep, gate, 0.0)
        y = y * torch.sigmoid(g) * (g if act == "silu" else 1.0)
    return torch.where(keep, y, 0.0)


def block_norm(x, weight, y=None, post_weight=None, scale=None, res_scale=1.0, lengths=None, eps=1e-5):
    """x, y [B,T,D]; returns (x_out, h)."""
    keep = valid_rows(lengths, *x.shape[:2])[..., None]
    x = torch.where(keep, x, 0.0)
    if y is not None:
        z = torch.where(keep, y, 0.0)
        if post_weight is not None:
            z = rms_norm(z, post_weight, eps)
        x = x + res_scale * (1.0 if scale is None else scale) * z
    return x, torch.where(keep, rms_norm(x, weight, eps), 0.0)


def block_norm_of_x_out(x_out, weight, lengths=None, eps=1e-5):
    """h as a function of the stored x_out (what the backward pass differentiates)."""
    keep = valid_rows(lengths, *x_out.shape[:2])[..., None]
    return torch.where(keep, rms_norm(torch.where(keep, x_out, 0.0), weight, eps), 0.0)


def block_norm_grad(x_out, weight, dh, y=None, post_weight=None, scale=None, res_scale=1.0, dx_out=None,
                    lengths=None, eps=1e-5):
    """Gradients of <x_out, dx_out> + <h, dh> at the stored x_out: through h to x_out, then
    through x_out = x + res_scale * scale * z to x, y and the vectors."""
    keep = valid_rows(lengths, *x_out.shape[:2])[..., None]
    xo = x_out.clone().requires_grad_(True)
    w = weight.clone().requires_grad_(True)
    h = block_norm_of_x_out(xo, w, lengths, eps)
    d_xo, d_w = torch.autograd.grad((h * torch.where(keep, dh, 0.0)).sum(), [xo, w])
    if dx_out is not None:
        d_xo = d_xo + torch.where(keep, dx_out, 0.0)
    out = {"x": d_xo, "weight": d_w}
    if y is not None:
        leaves = {"y": y, "post_weight": post_weight, "scale": scale}
        leaves = {n: t.clone().requires_grad_(True) for n, t in leaves.items() if t is not None}
        z = torch.where(keep, leaves["y"], 0.0)
        if post_weight is not None:
            z = rms_norm(z, leaves["post_weight"], eps)
        join = (res_scale * leaves.get("scale", torch.ones((), dtype=z.dtype)) * z * d_xo).sum()
        out.update(zip(leaves, torch.autograd.grad(join, list(leaves.values()))))
    return out


def embed(ids, table, scale=1.0, lengths=None):
    """ids [B,T]; ids outside the table and padding give zero rows."""
    keep = valid_rows(lengths, *ids.shape) & (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(keep, ids, 0).long()]
    return torch.where(keep[..., None], scale * rows, 0.0)


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after one step."""
    b1, b2 = betas
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    update = m / (1 - b1 ** step) / (torch.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * update, m, v


def state_blocks(x):
    """x as rows of STATE_BLOCK elements, filled with zeros."""
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % STATE_BLOCK)).view(-1, STATE_BLOCK)


def decode(codes, scale):
    """The values that e4m3 codes and their blocks' scales stand for (in scale's precision)."""
    return (state_blocks(codes.to(scale.dtype)) * scale[:, None]).view(-1)[:codes.numel()].view(codes.shape)
