"""Norms of queries and keys with the position rotation on the GPU, forward and backward.

The reference is the formula in 64 bits on the CPU, on exactly the values the device sees; the
backward pass is checked against it differentiated by torch, and against central differences.

Bounds (u = 2^-24, half a step of fp32).  A sum of d <= 128 squares in any order is off by at most
127 u of itself, its reciprocal square root by half of that and its own 2 steps (4 u); three
roundings of products and the weight add 4 u.  An angle's fraction of a turn is rounded once
(at most 2 u radians after the factor 2 pi), sine and cosine by 2 steps each (4 u), their products
and the sum by 3 u: so an output differs by at most 84 u of its pair's |a| + |b|; 96 u is used.
Outputs in bf16 are rounded once more, by half a step, 2^-8 of the value.
Backward: z w - u t collects the same errors of inv twice and those of z (rotation and up to 32
summed heads, 32 u), and the sum t adds 127 u and one more inv: at most 512 u of
inv (sum of |dy| over heads and pair * |w| + |u| sum |z w u|).
dw: a sum of products over all rows whose longest chain of additions is at most 2048 long in any of
the tested shapes (a lane adds the rows of its turns, at most 40000 / 64 here, then 64 lanes, then
partial sums of at most 296 CTAs), each product off by at most 128 u: 2304 u of sum |z u|.
"""
import math

import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pair_partner(rot, d, layout):
    """Each element's place in its pair: pair number, partner element, sign of the sine term."""
    i = torch.arange(d)
    if layout == "half":
        first = i < rot // 2
        pair = torch.where(first, i, i - rot // 2)
        partner = torch.where(first, i + rot // 2, i - rot // 2)
    else:
        first = i % 2 == 0
        pair, partner = i // 2, torch.where(first, i + 1, i - 1)
    inside = i < rot
    return torch.where(inside, pair, 0), torch.where(inside, partner, i), torch.where(first, -1.0, 1.0).double(), inside


def _turn(y, pos, freq, rot, layout):
    """Rotation of [N, G, d] in 64 bits."""
    if rot == 0:
        return y
    pair, partner, sign, inside = _pair_partner(rot, y.shape[-1], layout)
    ang = (pos.double()[:, None] * freq.double())[:, pair][:, None]
    return torch.where(inside, y * ang.cos() + sign * y[..., partner] * ang.sin(), y)


def _forward(x, w, pos, freq, rot, H, layout, norm, eps):
    sq = (x * x).sum(-1, keepdim=True)
    y = x / torch.sqrt((sq / x.shape[-1] if norm == "rms" else sq) + eps)
    y = y if w is None else y * w
    y = _turn(y, pos, freq, rot, layout)
    return y.repeat_interleave(H // x.shape[1], 1)


def _pair_size(y, rot, layout):
    """|a| + |b| of each element's pair (the element itself where it is not turned)."""
    if rot == 0:
        return y.abs()
    _, partner, _, inside = _pair_partner(rot, y.shape[-1], layout)
    return torch.where(inside, y.abs() + y[..., partner].abs(), y.abs())


class Case:
    def __init__(self, N, Gq, Gk, H, d, rot, layout, norm, weights, dtype, fused, eps=1e-6, seed=0,
                 max_pos=1 << 20, lead=None):
        g = torch.Generator().manual_seed(seed + 31 * N + d)
        self.N, self.G, self.H, self.d, self.rot, self.eps = N, (Gq, Gk), H, d, rot, eps
        self.layout, self.norm, self.dtype = layout, norm, DT[dtype]
        lead = lead or (N,)
        assert math.prod(lead) == N
        row = torch.randn((N, (Gq + Gk) * d + 64), generator=g).to(self.dtype)
        if fused:   # q and k are columns of one wider row
            dev = row.to(DEV).view(*lead, -1)
            self.q = dev[..., :Gq * d].unflatten(-1, (Gq, d))
            self.k = dev[..., Gq * d:(Gq + Gk) * d].unflatten(-1, (Gk, d))
            assert N == 1 or not self.q.is_contiguous()
        else:
            self.q = row[:, :Gq * d].contiguous().to(DEV).view(*lead, Gq, d)
            self.k = row[:, Gq * d:(Gq + Gk) * d].contiguous().to(DEV).view(*lead, Gk, d)
        self.x = [t.reshape(N, -1, d).double().cpu() for t in (self.q, self.k)]
        self.w = [None, None]
        if weights:
            self.w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)]
        self.pos = torch.randint(-max_pos, max_pos, (N,), generator=g, dtype=torch.int64).int()
        self.freq = (10000.0 ** (-2 * torch.arange(rot // 2).double() / max(rot, 1))).float()
        self.dy = [torch.randn((N, H, d), generator=g) for _ in range(2)]
        self.lead = lead

    def how(self):
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return dict(wq=dev(self.w[0]), wk=dev(self.w[1]), pos=dev(self.pos) if self.rot else None,
                    inv_freq=dev(self.freq) if self.rot else None, norm=self.norm, layout=self.layout,
                    eps=self.eps)

    def ref(self, side, x=None, w=None):
        x = self.x[side] if x is None else x
        w = w if w is not None else (None if self.w[side] is None else self.w[side].double())
        return _forward(x, w, self.pos, self.freq, self.rot, self.H, self.layout, self.norm, self.eps)

    def bounds(self, side):
        """Reference gradients of x and w, and the bounds on their errors."""
        x = self.x[side].clone().requires_grad_(True)
        w = None if self.w[side] is None else self.w[side].double().requires_grad_(True)
        y = self.ref(side, x, w)
        got = torch.autograd.grad(y, [x] + ([] if w is None else [w]), self.dy[side].double())
        x, d, G = x.detach(), self.d, self.G[side]
        w = torch.ones(d).double() if w is None else w.detach()
        dy = self.dy[side].double().unflatten(1, (G, -1))
        z = _turn(dy.sum(2), -self.pos, self.freq, self.rot, self.layout)
        size = _pair_size(dy.abs().sum(2), self.rot, self.layout)
        sq = (x * x).sum(-1, keepdim=True)
        inv = ((sq / d if self.norm == "rms" else sq) + self.eps) ** -0.5
        u = x * inv
        t = (size * w.abs() * u.abs()).sum(-1, keepdim=True) / (d if self.norm == "rms" else 1)
        return got, 512 * U * inv * (size * w.abs() + u.abs() * t), 2304 * U * (size * u.abs()).sum((0, 1)), z, u


CASES = [
    # N  Gq  Gk  H   d  rot  layout         norm  weights dtype  fused
    (1, 1, 1, 1, 32, 0, "half", "l2", False, "bf16", False),
    (1, 4, 4, 4, 64, 64, "half", "l2", False, "bf16", True),
    (7, 3, 1, 6, 64, 32, "interleaved", "rms", True, "bf16", True),
    (64, 32, 32, 32, 64, 64, "half", "l2", False, "bf16", True),
    (130, 16, 4, 16, 128, 32, "interleaved", "rms", True, "bf16", True),
    (129, 2, 8, 8, 128, 128, "half", "l2", True, "f32", False),
    (33, 5, 5, 5, 32, 8, "half", "rms", False, "f32", True),
    (50, 6, 2, 6, 32, 24, "half", "rms", True, "bf16", False),
    (61, 1, 2, 4, 128, 40, "half", "l2", True, "bf16", True),
    (1000, 4, 1, 4, 64, 48, "interleaved", "l2", True, "f32", True),
    (3001, 8, 8, 8, 64, 64, "half", "rms", True, "bf16", False),
    (5, 64, 1, 64, 128, 128, "interleaved", "l2", False, "f32", False),
    (20000, 2, 1, 2, 32, 16, "half", "l2", True, "bf16", True),      # many batches for each CTA
    (2, 600, 300, 600, 32, 32, "half", "l2", False, "bf16", False),  # one token to a batch
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    c = Case(*case)
    got = binding.qk_norm_rope(c.q, c.k, heads=c.H, **c.how())
    for side in (0, 1):
        y, ref = got[side].double().cpu(), c.ref(side)
        assert got[side].dtype == c.dtype and tuple(y.shape) == (c.N, c.H, c.d)
        tol = 96 * U * _pair_size(ref, c.rot, c.layout)
        if c.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert bool(((y - ref).abs() <= tol).all()), ((y - ref).abs() / tol).max()


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    c = Case(*case)
    got = binding.qk_norm_rope_backward(c.q, c.k, c.dy[0].to(DEV), c.dy[1].to(DEV), **c.how())
    again = binding.qk_norm_rope_backward(c.q, c.k, c.dy[0].to(DEV), c.dy[1].to(DEV), **c.how())
    assert set(got) == ({"q", "k", "wq", "wk"} if c.w[0] is not None else {"q", "k"})
    for n in got:
        assert torch.equal(got[n], again[n]), n
    for side, n in ((0, "q"), (1, "k")):
        ref, tol, tol_w, _, _ = c.bounds(side)
        dx = got[n].double().cpu()
        assert bool(((dx - ref[0]).abs() <= tol).all()), ((dx - ref[0]).abs() / tol).max()
        if c.w[0] is not None:
            dw = got["w" + n].double().cpu()
            assert bool(((dw - ref[1]).abs() <= tol_w).all()), ((dw - ref[1]).abs() / tol_w).max()


def test_gradient_against_differences():
    """The device's dq against central differences of the formula, along random directions.  The
    difference of step h is off by h^2/6 of the third derivative (h = 1e-4: below 1e-7 of the
    gradient for unit-size rows) and by 2^-53 / h of the sum's terms (about 1e-10)."""
    c = Case(9, 2, 1, 4, 64, 32, "half", "rms", True, "f32", False, seed=3)
    got = binding.qk_norm_rope_backward(c.q, c.k, c.dy[0].to(DEV), c.dy[1].to(DEV), **c.how())
    g = torch.Generator().manual_seed(4)
    for side, n in ((0, "q"), (1, "k")):
        for what in ("x", "w"):
            base = c.x[side] if what == "x" else c.w[side].double()
            dirn = torch.randn(base.shape, generator=g).double()
            h = 1e-4
            f = [(c.ref(side, **{what: base + s * h * dirn}) * c.dy[side].double()).sum() for s in (1, -1)]
            want = (f[0] - f[1]) / (2 * h)
            dev = got[n if what == "x" else "w" + n].double().cpu()
            have = (dev * dirn).sum()
            scale = (dev * dirn).abs().sum()
            assert abs(have - want) <= 1e-5 * scale


def test_leading_dimensions_and_preallocated_outputs():
    c = Case(24, 4, 2, 4, 64, 16, "half", "l2", False, "bf16", True, lead=(2, 12))
    assert c.q.dim() == 4
    c.pos = c.pos.view(2, 12)
    out = tuple(torch.empty((2, 12, 4, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    got = binding.qk_norm_rope(c.q, c.k, out=out, **c.how())
    assert got[0] is out[0] and got[1] is out[1]
    c.pos = c.pos.view(-1)
    for side in (0, 1):
        ref = c.ref(side)
        tol = 2.0 ** -8 * ref.abs() + 100 * U * _pair_size(ref, c.rot, c.layout)
        assert bool(((out[side].view(24, 4, 64).double().cpu() - ref).abs() <= tol).all())


def test_gradients_into_one_buffer_leave_the_rest():
    """dq and dk as columns of a projection's gradient: equal to the separate ones bit for bit, and
    nothing else of the buffer is written."""
    c = Case(37, 4, 2, 4, 32, 32, "interleaved", "l2", False, "bf16", True)
    dy = [t.to(DEV) for t in c.dy]
    want = binding.qk_norm_rope_backward(c.q, c.k, *dy, **c.how())
    buf = torch.full((37, 8 * 32), 7.0, device=DEV)
    grads = {"q": buf[:, :128].unflatten(1, (4, 32)), "k": buf[:, 128:192].unflatten(1, (2, 32))}
    binding.qk_norm_rope_backward(c.q, c.k, *dy, grads=grads, **c.how())
    assert torch.equal(grads["q"], want["q"]) and torch.equal(grads["k"], want["k"])
    assert bool((buf[:, 192:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_rows_of_zeros_and_of_no_numbers(dtype, norm):
    """A row of zeros gives zeros (and finite gradients), a row with an infinity or NaN gives NaN;
    every other row keeps its bits."""
    c = Case(16, 4, 4, 4, 64, 32, "half", norm, True, dtype, False)
    clean = binding.qk_norm_rope(c.q, c.k, **c.how())
    q, k = c.q.clone(), c.k.clone()
    q[3, 1], k[0, 0] = 0, 0
    q[5, 2, 7], k[15, 3, 63] = float("inf"), float("nan")
    got = binding.qk_norm_rope(q, k, **c.how())
    assert bool((got[0][3, 1] == 0).all()) and bool((got[1][0, 0] == 0).all())
    assert bool(got[0][5, 2, :32].isnan().any()) and bool(got[1][15, 3, 63].isnan())
    for g, want, rows in ((got[0], clean[0], [(3, 1), (5, 2)]), (got[1], clean[1], [(0, 0), (15, 3)])):
        same = (g == want).all(-1).cpu()
        for r in rows:
            same[r] = True
        assert bool(same.all())
    q[5, 2, 7], k[15, 3, 63] = 0, 0
    grads = binding.qk_norm_rope_backward(q, k, c.dy[0].to(DEV), c.dy[1].to(DEV), **c.how())
    assert all(bool(t.isfinite().all()) for t in grads.values())


def test_far_positions():
    """Positions up to 2^31 - 1 and below 0: angles reach 2^31 radians, where a 32-bit product would
    be off by many turns.  (The product in 64 bits is off by 2^-22 radians there: 4 u.)"""
    c = Case(64, 2, 2, 2, 64, 64, "half", "l2", False, "f32", False, max_pos=(1 << 31) - 1)
    c.pos[0], c.pos[1] = (1 << 31) - 1, -(1 << 31)
    got = binding.qk_norm_rope(c.q, c.k, **c.how())
    for side in (0, 1):
        ref = c.ref(side)
        assert bool(((got[side].double().cpu() - ref).abs() <= 104 * U * _pair_size(ref, c.rot, c.layout)).all())


def test_no_rows():
    c = Case(4, 2, 2, 2, 64, 64, "half", "rms", True, "bf16", False)
    how = c.how()
    how["pos"] = how["pos"][:0]
    q, k = c.q[:0], c.k[:0]
    out = binding.qk_norm_rope(q, k, **how)
    assert tuple(out[0].shape) == (0, 2, 64)
    dy = torch.empty((0, 2, 64), device=DEV)
    got = binding.qk_norm_rope_backward(q, k, dy, dy.clone(), **how)
    assert bool((got["wq"] == 0).all()) and bool((got["wk"] == 0).all())


def test_other_stream_and_graph_replay():
    """Calls on a side stream and replayed from a graph on new inputs give the bits of a direct
    call; two graphs with workspaces of their own replay side by side."""
    a, b = (Case(300, 8, 2, 8, 64, 32, "half", "rms", True, "bf16", False, seed=s) for s in (1, 2))
    how, dy = a.how(), [t.to(DEV) for t in b.dy]
    want = [binding.qk_norm_rope(c.q, c.k, **how) for c in (a, b)]
    want_g = [binding.qk_norm_rope_backward(c.q, c.k, *dy, **how) for c in (a, b)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = binding.qk_norm_rope(a.q, a.k, stream=s, **how)
    s.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    n = binding.qk_norm_rope_bwd_workspace_bytes(64)
    graphs = []
    for c in (a, b):
        q, k, ws = c.q.clone(), c.k.clone(), torch.empty(n, dtype=torch.uint8, device=DEV)
        out = tuple(torch.empty((300, 8, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        grads = {m: torch.empty_like(t) for m, t in want_g[0].items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.qk_norm_rope(q, k, out=out, **how)
            binding.qk_norm_rope_backward(q, k, *dy, grads=grads, workspace=ws, **how)
        graphs.append((g, q, k, out, grads, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for swap in (0, 1):
        for i, (g, q, k, *_rest) in enumerate(graphs):
            src = (a, b)[i ^ swap]
            q.copy_(src.q)
            k.copy_(src.k)
        torch.cuda.synchronize()
        for (g, *_rest), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, _, _, out, grads, _) in enumerate(graphs):
            w, wg = want[i ^ swap], want_g[i ^ swap]
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
            for m in wg:
                assert torch.equal(grads[m], wg[m]), m


def test_binding_refusals():
    c = Case(8, 4, 4, 4, 64, 32, "half", "l2", False, "bf16", False)
    how = c.how()
    for bad in (dict(k=c.k.float()),):
        with pytest.raises(TypeError):
            binding.qk_norm_rope(c.q, bad["k"], **how)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(c.q, c.k[:7], **how)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(c.q.transpose(1, 2), c.k.transpose(1, 2), **how)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(c.q, c.k, **dict(how, pos=how["pos"][:7]))
    with pytest.raises(ValueError):
        binding.qk_norm_rope(c.q, c.k, **dict(how, pos=None))
    with pytest.raises(TypeError):
        binding.qk_norm_rope(c.q, c.k, **dict(how, pos=how["pos"].long()))
    with pytest.raises(ValueError):
        binding.qk_norm_rope(c.q, c.k, **dict(how, norm="max"))
    with pytest.raises(binding.LLAttnError):
        binding.qk_norm_rope(c.q, c.k, heads=6, **how)
    with pytest.raises(binding.LLAttnError):
        binding.qk_norm_rope(c.q, c.k, **dict(how, eps=0.0))
    with pytest.raises(binding.LLAttnError):      # a workspace that is too small
        c2 = Case(8, 4, 4, 4, 64, 32, "half", "l2", True, "bf16", False)
        binding.qk_norm_rope_backward(c2.q, c2.k, c2.dy[0].to(DEV), c2.dy[1].to(DEV),
                                      workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **c2.how())
