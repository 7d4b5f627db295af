"""The gated linear recurrence on the GPU, forward and backward, against the recurrence in 64 bits.

Bounds (u = 2^-24).  Each step multiplies by exp(log_a), off by at most 2 steps (4 u) and, as
2^(log_a log2 e), by the roundings of the exponent's product and of log2 e: an error d of the exponent
x log2 e is one of d ln 2 relative, and |d| <= |x| log2 e (u + 0.23 u), so 1.25 |x| u.  It rounds the
product and the sum; where a walk is split, the parts' gates are products (one more rounding of
u per step) and joining them adds a rounding or two per part.  So with M_t = a_t M_{t-1} + |x_t|
(M_{-1} = |h0|), an error grows as E_t = a_t E_{t-1} + 16 u M_t, whatever the split (the exponent's part
is 1.25 |x| e^x u M_{t-1} <= 0.46 u M_{t-1}, and no part for a gate above 1: those are below e^0.1).
The backward recurrence is the same with the gates one step on; dlog_a = g a h_{t-1} adds 8 u and the
exponent's 1.25 |log_a| u of itself.

Those are relative errors, which hold for results of at least 2^-126, fp32's smallest normal number.
Below it a result is off by up to half of 2^-149, or by all of itself where it is flushed to zero,
so by less than 2^-126 in each case, and that error is multiplied by later factors: a gate (below 2
but for a handful of steps of the growing ones, whose products stay below e^(0.01 * 6 * 513^(1/2)) < 4)
and, for dlog_a, |g| or |h|, below 2^12 in every case here (sums of at most 4100 terms of size 1).  At
most 4100 such errors add up along a sequence: 2^-126 * 2^2 * 2^12 * 2^13 < 2^-98.
"""
import math

import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SEQ_TOO_LONG, BAD_CU = 1, 4


def _gates(shape, mode, g):
    z = torch.randn(shape, generator=g)
    la = {"dist": -torch.exp(-2 + 0.5 * z), "slow": -torch.exp(-7 + 0.5 * z), "strong": -torch.exp(1 + z),
          "zero": torch.zeros(shape), "grow": 0.01 * z}[mode]
    if mode == "strong":   # and some that start afresh
        la = torch.where(torch.rand(shape, generator=g) < 0.1, torch.tensor(-math.inf), la)
    return la


class Case:
    def __init__(self, lengths, D, dtype="f32", gates="dist", state=True, packed=False, seed=0):
        g = torch.Generator().manual_seed(seed + D + 17 * len(lengths) + sum(lengths))
        self.lengths, self.D, self.packed, self.B, self.T = lengths, D, packed, len(lengths), max(lengths)
        total = sum(lengths)
        self.x = torch.randn((total, D), generator=g).to(DT[dtype])
        self.la = _gates((total, D), gates, g)
        self.dh = torch.randn((total, D), generator=g)
        self.h0 = torch.randn((self.B, D), generator=g) if state else None
        self.dl = torch.randn((self.B, D), generator=g) if state else None
        cu = torch.tensor([0] + lengths).cumsum(0).int()
        self.cu = cu.to(DEV) if packed else None
        self.spans = [(int(cu[i]), int(cu[i + 1])) for i in range(self.B)]

    def dev(self, t):
        if t is None:
            return None
        t = t.to(DEV)
        return t if self.packed or t.shape[0] == self.B else t.view(self.B, self.T, self.D)

    def rows(self, t):
        return self.dev(t) if self.packed else t.to(DEV).view(self.B, self.T, self.D)

    def forward(self, **kw):
        last = torch.full((self.B, self.D), math.nan, device=DEV)
        h0 = None if self.h0 is None else self.h0.to(DEV)
        h = binding.glr_forward(self.rows(self.x), self.rows(self.la), h0=h0, h_last=last,
                                cu_seqlens=self.cu, T=self.T, **kw)
        return h, last

    def reference(self):
        """h, h_last and the bounds of both."""
        a, x = self.la.double().exp(), self.x.double()
        h, E = torch.empty_like(a), torch.empty_like(a)
        last = torch.zeros((self.B, self.D)).double() if self.h0 is None else self.h0.double().clone()
        elast = torch.zeros_like(last)
        for b, (s, e) in enumerate(self.spans):
            y, m, err = last[b], last[b].abs(), elast[b]
            for t in range(s, e):
                y, m = a[t] * y + x[t], a[t] * m + x[t].abs()
                err = a[t] * err + 16 * U * m
                h[t], E[t] = y, err
            last[b], elast[b] = y, err
        return h, last, E, elast

    def reference_backward(self, h):
        """Gradients with the given h (fp32, as the device reads it), and their bounds."""
        a, dh, h = self.la.double().exp(), self.dh.double(), h.double()
        dx, dla, E, Ela = (torch.empty_like(a) for _ in range(4))
        d0, e0 = torch.empty((self.B, self.D)).double(), torch.empty((self.B, self.D)).double()
        for b, (s, e) in enumerate(self.spans):
            c = torch.zeros(self.D).double() if self.dl is None else self.dl[b].double()
            m, err = c.abs(), torch.zeros(self.D).double()
            h0 = torch.zeros(self.D).double() if self.h0 is None else self.h0[b].double()
            for t in reversed(range(s, e)):
                g, m = dh[t] + c, dh[t].abs() + m
                err = err + 16 * U * m
                past = a[t] * (h[t - 1] if t > s else h0)
                dx[t], dla[t], E[t] = g, g * past, err
                off = 8 * U + torch.where(a[t] > 0, 1.25 * U * self.la[t].double().abs(), 0.0)
                Ela[t] = (err + off * g.abs()) * past.abs()
                c, m, err = a[t] * g, a[t] * m, a[t] * err
            d0[b], e0[b] = c, err + 8 * U * m   # a_0 g_0: its exponent's part as in E
        return dx, dla, d0, E, Ela, e0


def _near(got, ref, tol, what):
    got = got.double().cpu().reshape(ref.shape)
    tol = tol + 2.0 ** -98   # results below the normal numbers
    bad = (got - ref).abs() - tol
    assert bool((bad <= 0).all()), f"{what}: {bad.max():.3e} beyond its bound, {((got - ref).abs() / tol.clamp_min(1e-300)).max():.2f} of it"


CASES = [
    dict(lengths=[1], D=1), dict(lengths=[1] * 64, D=96, dtype="bf16"), dict(lengths=[2, 2, 2], D=7),
    dict(lengths=[5], D=64, gates="strong"), dict(lengths=[33, 33], D=128, dtype="bf16", gates="slow"),
    dict(lengths=[300], D=3, state=False), dict(lengths=[257, 257], D=130, dtype="bf16", gates="strong"),
    dict(lengths=[1000], D=64, gates="zero"), dict(lengths=[1025], D=40, dtype="bf16"),
    dict(lengths=[513, 513], D=31, gates="grow"), dict(lengths=[3000], D=36, dtype="bf16", gates="slow"),
    dict(lengths=[4099], D=12), dict(lengths=[20, 0, 1, 333, 64, 0, 7], D=72, packed=True, dtype="bf16"),
    dict(lengths=[0, 700, 129], D=33, packed=True, gates="strong"),
    dict(lengths=[2050, 5], D=256, packed=True, state=False, dtype="bf16"),
    dict(lengths=[700, 700], D=520, dtype="f32", gates="dist"),
]
IDS = [f"{i}-{len(c['lengths'])}x{max(c['lengths'])}x{c['D']}" for i, c in enumerate(CASES)]


@pytest.mark.parametrize("kw", CASES, ids=IDS)
def test_forward(kw):
    c = Case(**kw)
    binding.device_status(clear=True)
    h, last = c.forward()
    ref, rl, E, el = c.reference()
    assert h.dtype == torch.float32
    _near(h, ref, E, "h")
    _near(last, rl, el, "h_last")
    assert binding.device_status(clear=True) == 0


@pytest.mark.parametrize("kw", CASES, ids=IDS)
def test_backward(kw):
    c = Case(**kw)
    h, _ = c.forward()
    args = dict(h0=None if c.h0 is None else c.h0.to(DEV), dh_last=None if c.dl is None else c.dl.to(DEV),
                cu_seqlens=c.cu, T=c.T)
    got = binding.glr_backward(c.rows(c.la), h, c.rows(c.dh), **args)
    assert set(got) == ({"x", "log_a", "h0"} if c.h0 is not None else {"x", "log_a"})
    dx, dla, d0, E, Ela, e0 = c.reference_backward(h.cpu().reshape(c.la.shape))
    _near(got["x"], dx, E, "dx")
    _near(got["log_a"], dla, Ela, "dlog_a")
    if c.h0 is not None:
        _near(got["h0"], d0, e0, "dh0")
    again = binding.glr_backward(c.rows(c.la), h, c.rows(c.dh), **args)
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_gradients_against_differences():
    """Central differences (h = 1e-4) of sum(h dh) + sum(h_last dh_last) in 64 bits along random
    directions; the device's h differs from the exact one by about 1e-6, and so dlog_a."""
    c = Case([40, 40], 6)
    h, _ = c.forward()
    got = binding.glr_backward(c.rows(c.la), h, c.rows(c.dh), h0=c.h0.to(DEV), dh_last=c.dl.to(DEV))

    def loss(x, la, h0):
        y = h0
        out = 0.0
        for t in range(40):
            y = la[:, t].exp() * y + x[:, t]
            out = out + (y * c.dh.view(2, 40, 6)[:, t].double()).sum()
        return out + (y * c.dl.double()).sum()

    base = dict(x=c.x.double().view(2, 40, 6), la=c.la.double().view(2, 40, 6), h0=c.h0.double())
    g = torch.Generator().manual_seed(1)
    for n, m in (("x", "x"), ("la", "log_a"), ("h0", "h0")):
        d = torch.randn(base[n].shape, generator=g).double()
        f = [loss(**{**base, n: base[n] + s * 1e-4 * d}) for s in (1, -1)]
        dev = got[m].double().cpu().view(base[n].shape)
        assert abs((f[0] - f[1]) / 2e-4 - (dev * d).sum()) <= 2e-5 * (dev * d).abs().sum()


@pytest.mark.parametrize("B,T,D", [(1, 65536, 64), (3, 9000, 1000), (1, 30000, 6), (160, 50, 260), (40, 1500, 132),
                                   (50, 1100, 131), (2, 4000, 4099)])
def test_long_and_wide(B, T, D):
    """Split walks over long sequences, sampled channels against the recurrence in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((B, T, D), generator=g, device=DEV).bfloat16()
    la = -torch.exp(-4 + torch.randn((B, T, D), generator=g, device=DEV))
    dh = torch.randn((B, T, D), generator=g, device=DEV)
    h = binding.glr_forward(x, la)
    got = binding.glr_backward(la, h, dh)
    pick = [(0, 0), (B - 1, D - 1), (B // 2, D // 2), (B - 1, 1)]
    cb, cd = torch.tensor([p[0] for p in pick]), torch.tensor([p[1] for p in pick])
    col = lambda t: t[cb.to(DEV), :, cd.to(DEV)].T.cpu().contiguous()  # noqa: E731
    c = Case([T], len(pick), state=False)
    c.x, c.la, c.dh = col(x), col(la), col(dh)
    ref, _, E, _ = c.reference()
    _near(col(h), ref, E, "h")
    dx, dla, _, E, Ela, _ = c.reference_backward(col(h))
    _near(col(got["x"]), dx, E, "dx")
    _near(col(got["log_a"]), dla, Ela, "dlog_a")


@pytest.mark.parametrize("D", [64, 35])
def test_many_packed_sequences(D):
    """150 sequences of 0 to 600 tokens: more chains of tiles than are handed out by turns."""
    g = torch.Generator().manual_seed(D)
    c = Case(torch.randint(0, 601, (150,), generator=g).tolist(), D, dtype="bf16", packed=True)
    h, last = c.forward()
    ref, rl, E, el = c.reference()
    _near(h, ref, E, "h")
    _near(last, rl, el, "h_last")
    got = binding.glr_backward(c.rows(c.la), h, c.rows(c.dh), h0=c.h0.to(DEV), dh_last=c.dl.to(DEV),
                               cu_seqlens=c.cu, T=c.T)
    dx, dla, d0, E, Ela, e0 = c.reference_backward(h.cpu())
    _near(got["x"], dx, E, "dx")
    _near(got["log_a"], dla, Ela, "dlog_a")
    _near(got["h0"], d0, e0, "dh0")


def test_the_librarys_buffer_and_a_callers_workspace():
    """The C entry points without a workspace (the library's buffer, grown between the calls) and with
    one full of noise give the bits of the binding's call; one that is too small or off a 256-byte
    boundary is refused."""
    import ctypes
    lib, P = binding.lib(), lambda t: t.data_ptr()  # noqa: E731
    for T in (300, 5000):
        c = Case([T] * 3, 68, seed=T)
        x, la, dh, h0 = c.rows(c.x), c.rows(c.la), c.rows(c.dh), c.h0.to(DEV)
        want = binding.glr_forward(x, la, h0=h0)
        grads = binding.glr_backward(la, want, dh, h0=h0)
        n = binding.glr_workspace_bytes(3, T, 68)
        noise = torch.randint(0, 256, (n + 256,), device=DEV).to(torch.uint8)
        assert noise.data_ptr() % 256 == 0
        s = torch.cuda.current_stream().cuda_stream
        for ws, size in ((None, 0), (P(noise), n)):
            h, g = torch.empty_like(want), [torch.empty_like(t) for t in (la, la, h0)]
            assert lib.llattn_glr_fwd(binding.F32, P(x), P(la), P(h0), P(h), None, 3, T, 68, None, ws, size, s) == 0
            assert lib.llattn_glr_bwd(P(la), P(h), P(h0), P(dh), None, P(g[0]), P(g[1]), P(g[2]), 3, T, 68, None,
                                      ws, size, s) == 0
            assert torch.equal(h, want)
            for t, m in zip(g, ("x", "log_a", "h0")):
                assert torch.equal(t, grads[m]), m
        assert lib.llattn_glr_fwd(binding.F32, P(x), P(la), None, P(want), None, 3, T, 68, None, P(noise), n - 1, s) == 7
        assert lib.llattn_glr_fwd(binding.F32, P(x), P(la), None, P(want), None, 3, T, 68, None,
                                  ctypes.c_void_p(P(noise) + 16), n, s) == 7


def test_calls_side_by_side():
    """Four calls on four streams at once, each with scratch of its own: the bits of calls alone."""
    cases = [Case([2500] * 4, 100 + 4 * i, seed=i) for i in range(4)]
    dev = [(c.rows(c.x), c.rows(c.la), c.rows(c.dh), c.h0.to(DEV)) for c in cases]
    want = [binding.glr_forward(x, la, h0=h0) for x, la, _, h0 in dev]
    want_g = [binding.glr_backward(la, h, dh, h0=h0) for (x, la, dh, h0), h in zip(dev, want)]
    streams = [torch.cuda.Stream() for _ in dev]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for (x, la, dh, h0), s in zip(dev, streams):
            with torch.cuda.stream(s):
                h = binding.glr_forward(x, la, h0=h0)
                got.append((h, binding.glr_backward(la, h, dh, h0=h0)))
        torch.cuda.synchronize()
        for (h, g), w, wg in zip(got, want, want_g):
            assert torch.equal(h, w)
            for n in wg:
                assert torch.equal(g[n], wg[n]), n


def test_steps_continue_a_prompt_in_place():
    """T = 1 calls with one state buffer, after a prompt's h_last: within the bounds of the whole."""
    c = Case([150] * 5, 200, dtype="bf16")
    ref, rl, E, el = c.reference()
    x, la = c.rows(c.x), c.rows(c.la)
    state = c.h0.to(DEV)
    out = torch.empty((5, 150, 200), device=DEV)
    out[:, :120] = binding.glr_forward(x[:, :120].contiguous(), la[:, :120].contiguous(), h0=state, h_last=state)
    for t in range(120, 150):
        out[:, t:t + 1] = binding.glr_forward(x[:, t:t + 1].contiguous(), la[:, t:t + 1].contiguous(),
                                              h0=state, h_last=state)
    _near(out, ref, E, "h")
    _near(state, rl, el, "state")


def test_rows_behind_the_last_sequence_and_the_bound():
    """Rows that no sequence has are neither read nor written; a sequence above the bound is cut
    there and reported."""
    c = Case([50, 90], 24, packed=True)
    pad = torch.full((30, 24), math.nan)
    x, la, dh = (torch.cat([t.float(), pad]).to(DEV) for t in (c.x, c.la, c.dh))
    out = torch.full((170, 24), 7.0, device=DEV)
    last = torch.empty((2, 24), device=DEV)
    binding.glr_forward(x, la, h0=c.h0.to(DEV), h_last=last, cu_seqlens=c.cu, T=90, out=out)
    ref, rl, E, el = c.reference()
    _near(out[:140], ref, E, "h")
    _near(last, rl, el, "h_last")
    assert bool((out[140:] == 7.0).all())
    grads = {n: torch.full((170, 24), 7.0, device=DEV) for n in ("x", "log_a")}
    grads["h0"] = torch.empty((2, 24), device=DEV)
    binding.glr_backward(la, out, dh, h0=c.h0.to(DEV), dh_last=c.dl.to(DEV), cu_seqlens=c.cu, T=90, grads=grads)
    dx, dla, d0, E, Ela, e0 = c.reference_backward(out[:140].cpu())
    _near(grads["x"][:140], dx, E, "dx")
    _near(grads["log_a"][:140], dla, Ela, "dlog_a")
    assert bool((grads["x"][140:] == 7.0).all()) and bool((grads["log_a"][140:] == 7.0).all())
    assert binding.device_status(clear=True) == 0
    cut = Case([50, 60], 24, packed=True)
    out.fill_(7.0)
    binding.glr_forward(x, la, h0=c.h0.to(DEV), h_last=last, cu_seqlens=c.cu, T=60, out=out)
    assert binding.device_status(clear=True) == SEQ_TOO_LONG
    cut.x, cut.la, cut.h0 = c.x[:110], c.la[:110], c.h0
    ref, rl, E, el = cut.reference()
    _near(out[:110], ref, E, "h")
    _near(last, rl, el, "h_last")
    assert bool((out[110:] == 7.0).all())


def test_values_that_are_no_numbers_stay_in_their_channel():
    c = Case([400, 400], 48)
    clean, _ = c.forward()
    c.x[100, 5], c.x[450, 9] = math.inf, math.nan
    h, _ = c.forward()
    h, clean = h.view(800, 48), clean.view(800, 48)
    assert bool(h[100:400, 5].isinf().all() or h[100:400, 5].isnan().any())
    assert bool(h[450:, 9].isnan().all())
    same = h == clean
    same[100:400, 5] = True
    same[450:, 9] = True
    assert bool(same.all())
    c.la[150, 5] = c.la[500, 9] = 0.0   # and a finite gate does not stop them
    h, _ = c.forward()
    assert bool(h.view(800, 48)[500:, 9].isnan().all())


def test_no_rows():
    x = torch.empty((3, 0, 16), device=DEV)
    h0, last = torch.randn((3, 16), device=DEV), torch.empty((3, 16), device=DEV)
    assert binding.glr_forward(x, x.clone(), h0=h0, h_last=last).numel() == 0
    assert torch.equal(h0, last)
    got = binding.glr_backward(x, x.clone(), x.clone(), h0=h0, dh_last=h0)
    assert torch.equal(got["h0"], h0)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.empty((0, 16), device=DEV)
    last.fill_(5.0)
    binding.glr_forward(x, x.clone(), h_last=last, cu_seqlens=cu, T=9)
    assert bool((last == 0).all())


@pytest.mark.parametrize("shape", [(2, 700, 256), (64, 1, 512), (1, 5000, 64)])
def test_other_stream_graph_and_unaligned_rows(shape):
    """A side stream, a replayed graph on new inputs, and tensors that start off a 16-byte boundary:
    each within the bounds; stream and graph give the direct call's bits."""
    B, T, D = shape
    c = [Case([T] * B, D, dtype="bf16", seed=s) for s in (1, 2)]
    dev = [[t.to(DEV).view(B, T, D) for t in (k.x, k.la, k.dh)] + [k.h0.to(DEV)] for k in c]
    want = [binding.glr_forward(x, la, h0=h0) for x, la, _, h0 in dev]
    want_g = [binding.glr_backward(la, h, dh, h0=h0) for (x, la, dh, h0), h in zip(dev, want)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = binding.glr_forward(dev[0][0], dev[0][1], h0=dev[0][3], stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])
    buf = [t.clone() for t in dev[0]]
    out = torch.empty((B, T, D), device=DEV)
    grads = {n: torch.empty_like(t) for n, t in want_g[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.glr_forward(buf[0], buf[1], h0=buf[3], out=out)
        binding.glr_backward(buf[1], out, buf[2], h0=buf[3], grads=grads)
    for i in (1, 0):
        for t, src in zip(buf, dev[i]):
            t.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        for n in grads:
            assert torch.equal(grads[n], want_g[i][n]), n
    if T <= 700:
        odd = []
        for t in dev[0][:3]:
            b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
            odd.append(b.copy_(t))
        ref, _, E, _ = c[0].reference()
        h = binding.glr_forward(odd[0], odd[1], h0=dev[0][3])
        _near(h, ref, E, "unaligned h")
        h2 = torch.empty(h.numel() + 1, device=DEV)[1:].view(h.shape).copy_(want[0])
        got = binding.glr_backward(odd[1], h2, odd[2], h0=dev[0][3])
        c[0].dl = None
        dx, dla, d0, E, Ela, e0 = c[0].reference_backward(want[0].cpu().view(-1, D))
        _near(got["x"], dx, E, "unaligned dx")
        _near(got["log_a"], dla, Ela, "unaligned dlog_a")
        _near(got["h0"], d0, e0, "unaligned dh0")


def test_binding_refusals():
    x = torch.zeros((2, 8, 16), device=DEV)
    with pytest.raises(ValueError):
        binding.glr_forward(x.transpose(1, 2), x.transpose(1, 2))
    with pytest.raises(ValueError):
        binding.glr_forward(x, x[:, :4])
    with pytest.raises(TypeError):
        binding.glr_forward(x, x.bfloat16())
    with pytest.raises(ValueError):
        binding.glr_forward(x, x.clone(), h0=torch.zeros((2, 8), device=DEV))
    with pytest.raises(ValueError):
        binding.glr_forward(x[0], x[0].clone(), cu_seqlens=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        binding.glr_forward(x[0], x[0].clone(), cu_seqlens=torch.zeros(2, dtype=torch.int64, device=DEV), T=8)
    with pytest.raises(binding.LLAttnError):      # in place
        binding.glr_forward(x, x.clone(), out=x)


def test_results_belong_to_the_stream_that_writes_them():
    """A call on a side stream takes no memory that the current stream may still be writing; a
    workspace of the host is refused."""
    x, la = torch.randn((2, 700, 256), device=DEV), -torch.rand((2, 700, 256), device=DEV)
    want = binding.glr_forward(x, la)
    torch.cuda.synchronize()
    s, busy = torch.cuda.Stream(), torch.empty_like(x)
    at = busy.data_ptr()
    for _ in range(50):
        busy.fill_(1.0)
    del busy                       # free for the current stream, whose fills are not done
    h = binding.glr_forward(x, la, stream=s)
    grads = binding.glr_backward(la, want, x, stream=s)
    s.synchronize()
    assert at not in (h.data_ptr(), grads["x"].data_ptr(), grads["log_a"].data_ptr())
    assert torch.equal(h, want)
    with pytest.raises(ValueError):
        binding.glr_forward(x, la, workspace=torch.empty(1 << 20))


@pytest.mark.parametrize("start", [0, 1])
@pytest.mark.parametrize("T,D", [(17, 33), (333, 33), (1025, 1)])
def test_lone_bf16_values_at_both_ends_of_a_word(start, T, D):
    """Odd counts of bf16, from either half of a word: the first value, the last and those between."""
    c = Case([T], D, dtype="bf16")
    x = torch.full((T * D + 2,), float("nan"), dtype=torch.bfloat16, device=DEV)[start:start + T * D].view(1, T, D)
    x.copy_(c.x.view(1, T, D))
    la, h0 = c.la.to(DEV).view(1, T, D), c.h0.to(DEV)
    h = binding.glr_forward(x, la, h0=h0)
    assert torch.equal(h, binding.glr_forward(x.float(), la, h0=h0))   # bf16 values in fp32: the same
