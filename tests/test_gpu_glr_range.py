"""The gated linear recurrence where products of its gates leave fp32's range although the states do
not: growing gates over states that are zero or small, and starts afresh behind them.

Bounds (u = 2^-24).  As in the other tests of the recurrence a step costs 16 u of M_t, M_t = a_t M_{t-1}
+ |x_t|.  The gates of a part of a walk are summed as logarithms and its product is 2 to that sum, so a
rounding of the sum, at most u times the sum of the |log_a| in it, is one of the product by as much.  A
gate is in at most 35 such sums (32 steps of a thread, 4 warps; 8, 2 and 8 in the wide form) and in
one rounding of log_a log2 e (1.25 u |log_a|): 48 u |log_a_t| M_t per step in all.  Results below fp32's
normal numbers are off by less than 2^-126, and later gates multiply that as they do every error.
"""
import math

import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 2.0 ** -126
DEV = "cuda:0"
SHAPES = [(1, 17, 32), (2, 128, 64), (1, 128, 33), (1, 300, 5), (2, 700, 36), (1, 1500, 40), (130, 300, 36)]


def _reference(x, la, h0):
    """h of [B, T, D] in 64 bits and its bound."""
    a, x = la.double().exp(), x.double()
    y = torch.zeros_like(x[:, 0]) if h0 is None else h0.double()
    m, err = y.abs(), torch.zeros_like(y)
    h, E = torch.empty_like(a), torch.empty_like(a)
    cost = 16 * U + 48 * U * torch.where(a > 0, la.double().abs(), 0.0)
    for t in range(a.shape[1]):
        y, m = a[:, t] * y + x[:, t], a[:, t] * m + x[:, t].abs()
        err = a[:, t] * (err + TINY) + cost[:, t] * m
        h[:, t], E[:, t] = y, err + TINY
    return h, E


def _reference_backward(la, h, dh, h0, dh_last):
    a, h, dh = la.double().exp(), h.double(), dh.double()
    c = torch.zeros_like(dh[:, 0]) if dh_last is None else dh_last.double()
    m, err = c.abs(), torch.zeros_like(c)
    first = torch.zeros_like(c) if h0 is None else h0.double()
    cost = 16 * U + 48 * U * torch.where(a > 0, la.double().abs(), 0.0)
    dx, dla, E, Ela = (torch.empty_like(a) for _ in range(4))
    for t in reversed(range(a.shape[1])):
        g, m = dh[:, t] + c, dh[:, t].abs() + m
        err = err + 16 * U * m + TINY
        dx[:, t], E[:, t] = g, err
        past = h[:, t - 1] if t else first
        c, m, err = a[:, t] * g, a[:, t] * m, a[:, t] * (err + cost[:, t] * m)
        dla[:, t], Ela[:, t] = c * past, (err + 8 * U * m + TINY) * past.abs() + TINY
    return {"x": dx, "log_a": dla, "h0": c}, {"x": E, "log_a": Ela, "h0": err + TINY}


def _near(got, ref, tol, what):
    got = got.double().cpu()
    assert bool(got.isfinite().all()), what
    bad = (got - ref).abs() - tol
    assert bool((bad <= 0).all()), f"{what}: {bad.max():.3e} beyond its bound"


def _both(x, la, h0=None, dh=None, dh_last=None):
    dev = [None if t is None else t.to(DEV) for t in (x, la, h0, dh, dh_last)]
    last = torch.empty_like(x[:, 0]).float().to(DEV)
    h = binding.glr_forward(dev[0], dev[1], h0=dev[2], h_last=last)
    ref, E = _reference(x, la, h0)
    _near(h, ref, E, "h")
    _near(last, ref[:, -1], E[:, -1], "h_last")   # (through the map of the last tile: other roundings)
    if dh is None:
        return
    got = binding.glr_backward(dev[1], h, dev[3], h0=dev[2], dh_last=dev[4])
    want, tol = _reference_backward(la, h.cpu(), dh, h0, dh_last)
    for n in got:
        _near(got[n], want[n], tol[n], n)


@pytest.mark.parametrize("B,T,D", SHAPES)
def test_zeros_stay_zeros(B, T, D):
    x, la = torch.zeros((B, T, D)), torch.ones((B, T, D))
    last, d0 = torch.full((B, D), math.nan, device=DEV), torch.zeros((B, D), device=DEV)
    h = binding.glr_forward(x.to(DEV), la.to(DEV), h_last=last)
    assert bool((h == 0).all()) and bool((last == 0).all())
    got = binding.glr_backward(la.to(DEV), h, x.to(DEV), h0=d0)
    assert all(bool((t == 0).all()) for t in got.values())


@pytest.mark.parametrize("B,T,D", SHAPES)
def test_a_small_state_that_grows(B, T, D):
    """e^150 over the sequence, from 1e-30 up to 1e35, and the gradient the same way back."""
    g = torch.Generator().manual_seed(T + D)
    la = (150.0 / T) * (0.5 + torch.rand((B, T, D), generator=g))
    la *= 150.0 / la.sum(1, keepdim=True)
    h0 = 1e-30 * (1 + torch.rand((B, D), generator=g))
    zero = torch.zeros((B, T, D))
    _both(zero, la, h0=h0)
    _both(zero, la, h0=h0, dh=zero, dh_last=1e-35 * torch.randn((B, D), generator=g))


@pytest.mark.parametrize("B,T,D", [s for s in SHAPES if s[1] >= 128])
def test_a_start_afresh_behind_growth(B, T, D):
    """100 steps of e on zeros, a gate of 0, then growth of 1 by e^(1/8): inside a tile and over tiles."""
    g = torch.Generator().manual_seed(D)
    x, la = torch.zeros((B, T, D)), torch.ones((B, T, D))
    la[:, 100], x[:, 100] = -math.inf, 1.0
    la[:, 101:128] = 0.125
    la[:, 128:] = -torch.exp(-3 + 0.5 * torch.randn((B, T - 128, D), generator=g))
    x[:, 128:] = torch.randn((B, T - 128, D), generator=g)
    dh = torch.randn((B, T, D), generator=g)
    dh[:, :100] = 0.0
    _both(x, la, dh=dh)


@pytest.mark.parametrize("B,T,D", SHAPES)
def test_growth_and_decay_by_turns(B, T, D):
    """Log gates whose sums wander by 30 and more: products from 1e-30 to 1e30.  Inputs are scaled so
    that every sum of absolute terms is below 1e15 and the gradients' products stay in range too."""
    g = torch.Generator().manual_seed(3 * T + D)
    la = 30.0 / math.sqrt(T) * torch.randn((B, T, D), generator=g)
    x, dh = (torch.randn((B, T, D), generator=g) for _ in range(2))
    h0, dl = (torch.randn((B, D), generator=g) for _ in range(2))

    def size(x, la, s):
        m, top = s.double().abs(), s.double().abs()
        for t in range(T):
            m = la[:, t].double().exp() * m + x[:, t].double().abs()
            top = torch.maximum(top, m)
        return (top / 1e15).clamp_min(1.0)

    fwd = size(x, la, h0)
    back = size(dh.flip(1), torch.cat([torch.zeros_like(la[:, :1]), la.flip(1)[:, :-1]], 1), dl)
    scale = lambda t, f: (t.double() / f).float()  # noqa: E731
    _both(scale(x, fwd[:, None]), la, scale(h0, fwd), scale(dh, back[:, None]), scale(dl, back))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D", [(3, 1, 8), (2, 9, 33)] + SHAPES)
def test_nothing_crosses_a_start_afresh(B, T, D, dtype):
    """Infinities and NaN in x, h0, dh and dh_last, and states that overflow, with log gates of -inf
    behind (before) them: the rest of the channel is as if they were not there."""
    g = torch.Generator().manual_seed(T * D)
    x, dh = (torch.randn((B, T, D), generator=g) for _ in range(2))
    la = -torch.exp(-2 + 0.5 * torch.randn((B, T, D), generator=g))
    h0, dl = (torch.randn((B, D), generator=g) for _ in range(2))
    u = torch.rand((B, T, D), generator=g)
    cut = u < 4.0 / (T + 4)
    la[cut] = -math.inf
    la[:, 0, ::2] = -math.inf
    bad = [math.inf, -math.inf, math.nan]
    for t in (x, dh):
        at = torch.rand((B, T, D), generator=g) < 1.0 / (T + 4)
        t[at] = torch.tensor(bad)[torch.randint(3, (int(at.sum()),), generator=g)]
    h0[:, ::3], dl[:, 1::3] = math.nan, math.inf
    if T > 100:
        la[:, 20:60, 2] = 4.0                  # e^160, then afresh
        la[:, 60, 2], x[:, 20:61, 2] = -math.inf, 1.0
    x = x.to(dtype)
    a = la.double().exp()

    def join(a, y, add, m, err, la):
        zero = a == 0
        cost = 16 * U + 48 * U * torch.where(zero, 0.0, la.double().abs())
        y = torch.where(zero, 0.0, a * y) + add
        m = torch.where(zero, 0.0, a * m) + add.abs()
        err = torch.where(zero, 0.0, a * (err + TINY)) + cost * m
        return y, m, err

    def check(got, ref, tol, what):
        got = got.double().cpu()
        fits = ref.abs() < 2.0 ** 127          # (not for NaN)
        assert bool(got[fits].isfinite().all()), what
        assert bool(((got - ref).abs() <= tol + TINY)[fits].all()), what
        assert not bool(got[ref.isnan()].isfinite().any()), what

    last = torch.empty((B, D), device=DEV)
    h = binding.glr_forward(x.to(DEV), la.to(DEV), h0=h0.to(DEV), h_last=last)
    y, ref, E = h0.double(), torch.empty_like(a), torch.empty_like(a)
    m, err = y.abs(), torch.zeros_like(y)
    for t in range(T):
        y, m, err = join(a[:, t], y, x[:, t].double(), m, err, la[:, t])
        ref[:, t], E[:, t] = y, err
    check(h, ref, E, "h")
    check(last, ref[:, -1], E[:, -1], "h_last")

    got = binding.glr_backward(la.to(DEV), h, dh.to(DEV), h0=h0.to(DEV), dh_last=dl.to(DEV))
    hd, c = h.double().cpu(), dl.double()
    m, err = c.abs(), torch.zeros_like(c)
    dx, dla, Ex, Ela = (torch.empty_like(a) for _ in range(4))
    for t in reversed(range(T)):
        gt, m = dh[:, t].double() + c, dh[:, t].double().abs() + m
        err = err + 16 * U * m + TINY
        dx[:, t], Ex[:, t] = gt, err
        past = hd[:, t - 1] if t else h0.double()
        c, m, err = join(a[:, t], gt, torch.zeros_like(gt), m, err, la[:, t])
        err = err + 48 * U * torch.where(a[:, t] == 0, 0.0, la[:, t].double().abs()) * m
        zero = a[:, t] == 0
        dla[:, t] = torch.where(zero, 0.0, c * past)
        Ela[:, t] = torch.where(zero, 0.0, (err + 8 * U * m + TINY) * past.abs())
    check(got["x"], dx, Ex, "dx")
    check(got["log_a"], dla, Ela, "dlog_a")
    check(got["h0"], c, err + 8 * U * m, "dh0")
