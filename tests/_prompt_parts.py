"""Prompts whose level sums are nothing but the small parts of their operands, and what they must come to.

A bucket of four tokens.  The first is x = f k with f = exp(log_a), as an fp32 product, times v; the others,
with f = 1, take away the products of the rounded bf16 parts, so that what is left is 2^-18 and less of
the terms: x - x0 - x1 times v for bf16 v (x0 = bf16(x), x1 = bf16(x - x0)), and x v - x0 v0 - x1 v0 - x0 v1
for fp32 v.  Sums that hold all of fp32's bits keep it; sums of fewer parts are off by all of it.

The bound, of the terms' absolute sum A (at least twice |x v|): exp 2^-23 |x v| (one unit of the last
place), x rounded 2^-24, the matrix product's sum cut off at 2^-23, and for fp32 v the products of second
and third parts that are left out, 2^-26: 2.75 * 2^-23 |x v| < 2^-22 A.  Then half a step of the code.
"""
import numpy as np
import torch

LENGTH = 4
BOUND = 2.0 ** -22


def _parts(x):
    """x (fp32) as three bf16 values, each the rounded rest."""
    out = []
    for _ in range(3):
        p = x.bfloat16().float()
        out.append(p)
        x = x - p
    return out


def make(dtype, B, H, dk, dv, seed):
    """k, v, log_a of [B, 4, H, .], the exact level [B, H, dk, dv] and its bound."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((B, H, w), generator=g) for w in (dk, dv))
    la = torch.zeros((B, LENGTH, H))
    la[:, 1] = -0.05 - 0.6 * torch.rand((B, H), generator=g)      # gates the first token alone
    if dtype == torch.bfloat16:
        k, v = k.bfloat16().float(), v.bfloat16().float()
    x0, x1, _ = _parts(torch.exp(la[:, 1])[..., None] * k)
    v0, v1, _ = _parts(v)
    zero = torch.zeros_like(x0)
    ks = [k, -x0, -x1, zero if dtype == torch.bfloat16 else -x0]
    vs = [v, v0, v0, v1]
    k, v = torch.stack(ks, 1), torch.stack(vs, 1)
    f = torch.ones((B, LENGTH, H)).double()
    f[:, 0] = torch.exp(la[:, 1].double())
    terms = (f[..., None] * k.double())[..., None] * v.double()[..., None, :]
    return k.to(dtype), v.to(dtype), la, terms.sum(1), BOUND * terms.abs().sum(1)


def sums(k, v, la, products):
    """The level as sums of the given products of parts (q of f k, w of v), in 64 bits."""
    f = torch.ones(la.shape)
    f[:, 0] = torch.from_numpy(np.exp(la[:, 1].numpy()))
    x, y = _parts(f[..., None] * k.float()), _parts(v.float())
    return sum((x[q].double()[..., None] * y[w].double()[..., None, :]).sum(1) for q, w in products)


def rounded(S):
    """S as held in 8 bits, and the step of each value's block."""
    b = S.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    step = torch.exp2((e - 7 + (m > 127.0 / 128.0).int()).double())
    step = torch.where(m > 0, step, torch.zeros_like(step))
    val = torch.where(m > 0, torch.round(b / step.clamp_min(1e-300)) * step, torch.zeros_like(b))
    return val.flatten(-2), step.expand_as(b).flatten(-2)


def off(val, step, exact, err):
    """Whether held values are further from the exact level than their bound."""
    return not bool(((val - exact).abs() <= 0.5 * step + err).all())
