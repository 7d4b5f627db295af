"""The 8-bit decoding state on the GPU: written by a step and by a prompt, read by a step, read back.

Reference: the definition in 64 bits on the CPU, from the held codes.  Bounds (u = 2^-24):
  * a read-out is a sum over at most 128 rows of at most 17 levels with weights exp(gate + log_a)
    (the sum of two logarithms below 32: 64 u, exp 4 u) and a few products: 256 u of the sum of the
    terms' absolute values;
  * a carried value differs from the exact one by 128 u of the same kind of sum, and is then rounded
    by half a step of its block's power of two;
  * a prompt's sum: operands split into bf16 parts (off by 2^-16 at most), products and sums over a
    bucket in fp32, decays from log sums below 32 (about 2^-15): 2^-13 of the sum of the terms'
    absolute values, then half a step;
  * a block's power of two is the smallest that holds it: checked on its exact largest value, but
    for values within 2^-12 of a border, where a rounding may take either.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from hierarchical_fenwick_state_b200 import binding
from hierarchical_fenwick_state_b200 import inputs as I

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DECODE_POS, SEQ_TOO_LONG = 8, 1


def _views(state, B, H, L, dk, dv):
    n = B * H * (L - 1)
    a, b = n * dk * dv, n * dk * dv + n * 8
    return (state[:a].view(torch.int8).view(B, H, L - 1, dk, dv), state[a:b].view(torch.float32).view(B, H, 2, L - 1),
            state[b:].view(B, H, L - 1, dk, dv // 32))


def _buffer(B, H, L, dk, dv, fill=0xA5):
    s = torch.full((binding.decode_q8_state_bytes(B, H, L, dk, dv),), fill, dtype=torch.uint8, device=DEV)
    return s, _views(s, B, H, L, dk, dv)


def _values(codes, exps):
    """Held values in 64 bits: 2^(e - 127) per 32 columns; 0 a block of zeros, 255 none."""
    e = exps.double().cpu()
    scale = torch.where(e == 0, 0.0, torch.where(e == 255, math.nan, torch.exp2(e - 127)))
    return (codes.double().cpu().unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def _steps(exps):
    e = exps.double().cpu()
    return torch.where(e == 0, 0.0, torch.exp2(e - 127)).repeat_interleave(32, -1)


def _check_rounded(codes, exps, exact, err, what):
    """Held values against the exact ones: half a step and `err` apart, in the smallest power of two."""
    val, step = _values(codes, exps), _steps(exps)
    assert bool(((val - exact).abs() <= 0.5 * step + err).all()), what
    top = exact.abs().unflatten(-1, (-1, 32)).amax(-1)
    s = torch.exp2(exps.double().cpu() - 127)
    live = top > 2.0 ** -119          # above the smallest exponent code
    slack = 1 + 2.0 ** -12
    assert bool((top[live] <= 127 * s[live] * slack).all()), what
    assert bool((top[live] * slack >= 63.5 * s[live]).all()), what
    assert int(codes.min()) >= -127


def _step_ref(q, k, v, la, lam, pos, S, gate, L):
    """out, carry and their terms' absolute sums for every (sequence, head), in 64 bits."""
    B, H, dk = q.shape
    w = torch.exp(gate[torch.arange(B), :, (pos & 1).long()] + la[..., None])
    j = torch.arange(L - 1)
    held = ((pos[:, None].long() >> j) & 1).double()[:, None]
    m = torch.tensor([(~int(n) & (int(n) + 1)).bit_length() - 1 for n in pos])
    merged = held * (j < m[:, None])[:, None].double()
    S = torch.where(held[..., None, None] > 0, S, 0.0)
    wl = lam[..., 1:] * w * held
    own = lam[..., :1] * (q * k).sum(-1, True) * v
    out = own + torch.einsum("bhl,bhi,bhlij->bhj", wl, q, S)
    size = (lam[..., :1] * (q * k).abs().sum(-1, True) * v.abs()
            + torch.einsum("bhl,bhi,bhlij->bhj", wl.abs(), q.abs(), S.abs()))
    carry = k[..., None] * v[..., None, :] + torch.einsum("bhl,bhlij->bhij", w * merged, S)
    csize = k.abs()[..., None] * v.abs()[..., None, :] + torch.einsum("bhl,bhlij->bhij", w * merged, S.abs())
    return out, size, carry, csize, m


POSITIONS = {
    2: [0, 1, 0], 5: [0, 1, 7, 8, 14, 15], 14: [0, 1, 2, 3, 4095, 4096, 8190, 8191, 5000],
    17: [65535, 65534, 32767, 32768, 43690], 32: [0, 1023, (1 << 31) - 1, (1 << 31) - 2],
}


@pytest.mark.parametrize("H,L,dk,dv,dtype", [
    (3, 14, 64, 64, "bf16"), (2, 17, 128, 128, "bf16"), (5, 5, 32, 32, "f32"), (1, 2, 64, 128, "f32"),
    (2, 14, 128, 32, "bf16"), (4, 5, 32, 128, "bf16"), (1, 32, 32, 32, "f32"),
    # large batches, whose slots go through rings of 11, and (the smaller states) more CTAs than run at once
    (64, 14, 64, 64, "bf16"), (60, 17, 128, 128, "bf16"), (50, 5, 32, 32, "f32"), (100, 2, 64, 128, "f32"),
    (33, 14, 128, 32, "bf16"), (50, 5, 32, 128, "f32"), (75, 32, 32, 32, "f32"), (33, 14, 64, 32, "f32"),
    (50, 5, 32, 64, "bf16"), (60, 17, 128, 64, "bf16"), (60, 14, 128, 32, "bf16"), (110, 5, 32, 128, "f32"),
    (128, 32, 64, 64, "f32"),
])
def test_one_step(H, L, dk, dv, dtype):
    pos = torch.tensor(POSITIONS[L], dtype=torch.int32)
    B, nslot = len(pos), L - 1
    g = torch.Generator().manual_seed(L + dk + dv)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v = (rnd(B, H, n).to(DT[dtype]) for n in (dk, dk, dv))
    la, lam = -torch.exp(rnd(B, H) - 2), torch.nn.functional.softplus(rnd(B, H, L))
    state, (codes, gate, exps) = _buffer(B, H, L, dk, dv)
    codes.copy_(torch.randint(-127, 128, codes.shape, generator=g).to(torch.int8))
    e = torch.randint(110, 130, exps.shape, generator=g).to(torch.uint8)
    e[torch.rand(e.shape, generator=g) < 0.02] = 0     # some blocks of zeros
    exps.copy_(e)
    codes.masked_fill_((exps == 0).repeat_interleave(32, -1), 0)
    gate.copy_(-30 * torch.rand(gate.shape, generator=g) ** 4)
    before = state.clone()
    S, gate0 = _values(codes, exps), gate.cpu().clone()
    out = torch.full((B, H, dv), math.nan, device=DEV)
    binding.device_status(clear=True)
    args = [t.to(DEV) for t in (q, k, v, la, lam, pos)]
    binding.decode_step_q8(*args, state, out, B, H, L, dk, dv)
    assert binding.device_status(clear=True) == 0
    ref, size, carry, csize, m = _step_ref(q.double(), k.double(), v.double(), la.double(), lam.double(), pos, S,
                                           gate0.double(), L)
    got = out.double().cpu()
    assert bool(((got - ref).abs() <= 256 * U * size).all()), ((got - ref).abs() / (U * size)).max()
    bc, bg, be = _views(before, B, H, L, dk, dv)
    for b in range(B):
        n, mb = int(pos[b]), int(m[b])
        if mb < nslot:
            _check_rounded(codes[b, :, mb], exps[b, :, mb], carry[b], 128 * U * csize[b], f"position {n}")
        for j in range(nslot):     # everything else as it was
            if j != mb:
                assert torch.equal(codes[b, :, j], bc[b, :, j]) and torch.equal(exps[b, :, j], be[b, :, j])
            row = gate[b, :, :, j].cpu()
            assert torch.equal(row[:, n & 1], gate0[b, :, n & 1, j])
            want = gate0[b, :, 1 - (n & 1), j]
            if (n + 1) >> j & 1:
                want = torch.zeros(H) if j == mb else gate0[b, :, n & 1, j] + la[b]
            assert torch.equal(row[:, 1 - (n & 1)], want)
    again = torch.empty_like(out)     # the step reads none of what it wrote: once more, the same bits
    binding.decode_step_q8(*args, state, again, B, H, L, dk, dv)
    assert torch.equal(out, again)


def test_blocks_at_the_borders_of_the_numbers():
    """Position 0 carries k v^T alone: block maxima just at, above and below 127 powers of two, far
    out of fp32's middle, zeros, infinities and NaN, against the definition."""
    B, H, L, d = 1, 1, 3, 32
    state, (codes, gate, exps) = _buffer(B, H, L, d, d)
    k = torch.ones((B, H, d))
    tops = [127.0, 127.0001, 126.9999, 63.5, 64.0, 1.0, 2.0 ** -118, 2.0 ** -126, 2.0 ** -140, 0.0, 3e38, 1e-30,
            math.inf, math.nan, -127.0, -1.9843751, 1.984375]
    k[0, 0, :len(tops)] = torch.tensor(tops)
    v = torch.linspace(-1, 1, d).view(B, H, d).clone()
    v[..., 0] = 1.0
    v[..., 1] = 0.5 / 127
    v[..., 2] = 1.5 / 127
    out = torch.empty((B, H, d), device=DEV)
    zeros = torch.zeros((B, H, d), device=DEV)
    binding.decode_step_q8(zeros, k.to(DEV), v.to(DEV), torch.zeros((B, H), device=DEV),
                           torch.zeros((B, H, L), device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV),
                           state, out, B, H, L, d, d)
    S = (k[0, 0, :, None] * v[0, 0]).double()        # products as the device rounds them (fp32)
    c, e = codes[0, 0, 0].cpu().double(), exps[0, 0, 0, :, 0].cpu().long()
    for r in range(d):
        top = S[r].abs().max().item()
        if not math.isfinite(top):
            assert int(e[r]) == 255 and bool((c[r] == 0).all())
            continue
        if top == 0:
            assert int(e[r]) == 0 and bool((c[r] == 0).all())
            continue
        want = max(math.ceil(math.log2(top / 127) - 1e-12) + 127, 1)
        assert int(e[r]) == want, (r, top)
        step = 2.0 ** (want - 127)
        assert torch.equal(c[r], (S[r] / step).round()), r
    back = binding.read_state_q8(state, B, H, L, d, d, dtype=torch.float32)[0, 0, 0].cpu().double()
    assert torch.equal(torch.nan_to_num(back, nan=1e9), torch.nan_to_num(_values(codes, exps)[0, 0, 0], nan=1e9))


@pytest.mark.parametrize("dtype,T", [("bf16", 300), ("f32", 130)])
def test_whole_sequences(dtype, T):
    """Sequences decoded from a buffer of noise against the exact recurrence: each carried value is
    rounded by at most 1/127 of its block's largest, which for these draws is about 1% of a level's
    spread; 9 levels in turn and the read-out's sums of independent errors stay below 3% of the
    output's size (rms), a third of what any slot read wrongly costs."""
    w = I.shrink(I.WORKLOADS["t2k_d64_bf16" if dtype == "bf16" else "t256_d32_f32"], B=3, H=2, T=T)
    inp = I.make_inputs(w, seed=5, log_a_mode="slow")
    ref = torch.from_numpy(O.llattn_recurrent(inp))
    B, H, L, dk, dv = inp.B, inp.H, inp.L, inp.dk, inp.dv
    q, k, v = (torch.from_numpy(x).to(DEV).to(DT[dtype]) for x in (inp.q, inp.k, inp.v))
    la, lam = torch.from_numpy(inp.log_a).to(DEV), torch.from_numpy(inp.lam).to(DEV)
    state, _ = _buffer(B, H, L, dk, dv)
    got = torch.empty((B, T, H, dv), device=DEV)
    out = torch.empty((B, H, dv), device=DEV)
    for n in range(T):
        pos = torch.full((B,), n, dtype=torch.int32, device=DEV)
        binding.decode_step_q8(*(x[:, n].contiguous() for x in (q, k, v, la, lam)), pos, state, out, B, H, L, dk, dv)
        got[:, n] = out
    err = (got.double().cpu() - ref).square().mean().sqrt() / ref.square().mean().sqrt()
    assert err <= 0.03, err


def _prompt(lengths, H, dk, dv, dtype, gates, packed, seed=0, mu=-2.0):
    g = torch.Generator().manual_seed(seed + sum(lengths) + dk)
    total = sum(lengths)
    k = torch.randn((total, H, dk), generator=g)
    k = (k / k.norm(dim=-1, keepdim=True)).to(DT[dtype])
    v = torch.randn((total, H, dv), generator=g).to(DT[dtype])
    z = torch.randn((total, H), generator=g)
    la = {"dist": -torch.exp(mu + 0.5 * z), "zero": 0 * z, "slow": -torch.exp(-7 + 0.5 * z),
          "strong": -torch.exp(1 + 0.5 * z)}[gates]
    cu = torch.tensor([0] + lengths).cumsum(0).int()
    lead = (len(lengths), lengths[0])
    dev = [t.to(DEV) if packed else t.to(DEV).view(*lead, *t.shape[1:]) for t in (k, v, la)]
    return k.double(), v.double(), la.double(), cu, dev


def _prompt_levels(k, v, la, s, n, lvl):
    """Exact slot of level lvl of the sequence [s, s + n), its terms' absolute sum and its gate."""
    lo = (n >> lvl) << lvl
    hi = lo + (1 << (lvl - 1))
    a = la[s + lo:s + hi]
    f = torch.exp(a.flip(0).cumsum(0).flip(0) - a)[..., None]
    kk, vv = k[s + lo:s + hi] * f, v[s + lo:s + hi]
    return (torch.einsum("thi,thj->hij", kk, vv), torch.einsum("thi,thj->hij", kk.abs(), vv.abs()),
            la[s + hi:s + n].sum(0), la[s + hi:s + n].abs().sum(0))


@pytest.mark.parametrize("lengths,H,L,dk,dv,dtype,gates,packed", [
    ([1], 1, 2, 32, 32, "f32", "dist", False), ([0, 1, 2, 3], 2, 5, 64, 64, "bf16", "dist", True),
    ([15, 15], 3, 5, 64, 64, "bf16", "slow", False), ([255], 2, 14, 64, 64, "bf16", "dist", False),
    ([1023], 2, 11, 128, 128, "bf16", "slow", False), ([700, 0, 33, 129], 2, 14, 64, 64, "f32", "zero", True),
    ([517], 1, 12, 32, 128, "f32", "strong", False), ([2047, 1], 2, 12, 128, 32, "bf16", "zero", True),
    ([4100, 97], 1, 17, 64, 128, "bf16", "slow", True), ([64, 64, 64], 5, 8, 32, 32, "bf16", "strong", False),
    ([9000], 2, 15, 64, 64, "bf16", "slow", False),
    ([66000], 1, 18, 32, 32, "bf16", "slow", False),        # a bucket of 512 pieces
    ([2048, 1500, 2047, 512], 64, 13, 32, 32, "bf16", "slow", True),   # pieces of 512
    ([5000, 4096], 1, 14, 64, 64, "f32", "slow", True),
    # tiles of 64 tokens: buckets shorter than one, of one, of several; more tokens than a segment of factors
    ([0, 1, 63, 64, 65, 127, 700], 2, 14, 128, 128, "bf16", "dist", True),
    ([9000, 3000], 3, 15, 64, 128, "bf16", "slow", True), ([20000], 1, 16, 128, 128, "bf16", "slow", False),
    ([33, 2047], 5, 12, 128, 128, "bf16", "strong", True),
])
def test_prompt(lengths, H, L, dk, dv, dtype, gates, packed):
    k, v, la, cu, dev = _prompt(lengths, H, dk, dv, dtype, gates, packed)
    B = len(lengths)
    state, (codes, gate, exps) = _buffer(B, H, L, dk, dv)
    before = state.clone()
    binding.device_status(clear=True)
    binding.prefill_state_q8(*dev, state, B, H, max(lengths), L, dk, dv, cu_seqlens=cu.to(DEV) if packed else None)
    assert binding.device_status(clear=True) == 0
    bc, _, be = _views(before, B, H, L, dk, dv)
    for b, n in enumerate(lengths):
        for j in range(L - 1):
            if not n >> j & 1:
                assert torch.equal(codes[b, :, j], bc[b, :, j]) and torch.equal(exps[b, :, j], be[b, :, j])
                assert bool((gate[b, :, :, j] == 0).all())
                continue
            S, size, rest, rsize = _prompt_levels(k, v, la, int(cu[b]), n, j + 1)
            _check_rounded(codes[b, :, j], exps[b, :, j], S, 2.0 ** -13 * size, (n, j))
            got = gate[b, :, :, j].double().cpu()
            assert torch.equal(got[:, 0], got[:, 1])
            assert bool(((got[:, 0] - rest).abs() <= 256 * U * rsize).all())
    again = before.clone()
    binding.prefill_state_q8(*dev, again, B, H, max(lengths), L, dk, dv, cu_seqlens=cu.to(DEV) if packed else None)
    assert torch.equal(again, state)


def test_prompt_then_steps_as_they_are_used():
    """A packed batch of prompts: norms and rotation, the forward, the hand-off; then steps from it.
    Outputs against the exact operation on the normalised, rotated values: the prompt within the
    forward's 2e-2 bound, the steps within 3% (rms) of it."""
    lengths, K, H, d = [70, 133, 8], 12, 4, 64
    B, T = len(lengths), max(lengths) + K
    L = binding.num_levels(T)
    g = torch.Generator().manual_seed(9)
    full = [n + K for n in lengths]
    cu_full = torch.tensor([0] + full).cumsum(0)
    total = int(cu_full[-1])
    row = torch.randn((total, (H + 2 + H) * d), generator=g).bfloat16()   # q of 4 heads, k of 2 groups, v
    la = -torch.exp(-4 + 0.5 * torch.randn((total, H), generator=g))
    lam = torch.nn.functional.softplus(torch.randn((total, H, L), generator=g))
    pos = torch.cat([torch.arange(n) for n in full]).int()
    freq = (10000.0 ** (-2 * torch.arange(16).double() / 32)).float().to(DEV)

    def prep(rows, p):
        return binding.qk_norm_rope(rows[:, :H * d].unflatten(1, (H, d)), rows[:, H * d:(H + 2) * d].unflatten(1, (2, d)),
                                    pos=p, inv_freq=freq, heads=H, norm="l2")

    rdev, pdev = row.to(DEV), pos.to(DEV)
    q, k = prep(rdev, pdev)
    v = rdev[:, (H + 2) * d:].unflatten(1, (H, d))
    ref = []
    for b in range(B):     # exact outputs of every sequence, from the rounded q and k
        sl = slice(int(cu_full[b]), int(cu_full[b + 1]))
        f = lambda t: np.ascontiguousarray(t[sl].float().cpu().numpy()[None])  # noqa: E731
        Lb = I.num_levels(full[b])
        ref.append(torch.from_numpy(O.llattn_recurrent(I.Inputs(
            q=f(q), k=f(k), v=f(v), log_a=f(la), lam=f(lam[..., :Lb]), cu_seqlens=None, B=1, H=H, T=full[b],
            dk=d, dv=d, dtype="bf16")))[0])
    keep = torch.cat([torch.arange(int(cu_full[b]), int(cu_full[b]) + n) for b, n in enumerate(lengths)]).to(DEV)
    cu = torch.tensor([0] + lengths).cumsum(0).int().to(DEV)
    qp, kp = prep(rdev[keep], pdev[keep])
    assert torch.equal(qp, q[keep]) and torch.equal(kp, k[keep])
    vp, lap, lamp = v[keep].contiguous(), la.to(DEV)[keep].contiguous(), lam.to(DEV)[keep].contiguous()
    Lp = binding.num_levels(max(lengths))
    out = binding.forward(qp, kp, vp, lap, lamp[..., :Lp].contiguous(), cu_seqlens=cu, T=max(lengths))
    state, _ = _buffer(B, H, L, d, d)
    binding.prefill_state_q8(kp, vp, lap, state, B, H, max(lengths), L, d, d, cu_seqlens=cu)
    want = torch.cat([ref[b][:n] for b, n in enumerate(lengths)])
    assert O.rel_max_err(out.double().cpu().numpy(), want.numpy()) <= 2e-2
    err, size = 0.0, 0.0
    step = torch.empty((B, H, d), device=DEV)
    for t in range(K):
        at = torch.tensor([int(cu_full[b]) + n + t for b, n in enumerate(lengths)], device=DEV)
        p = pdev[at]
        qs, ks = prep(rdev[at], p)
        binding.decode_step_q8(qs, ks, v[at].contiguous(), la.to(DEV)[at].contiguous(), lam.to(DEV)[at].contiguous(), p,
                               state, step, B, H, L, d, d)
        for b, n in enumerate(lengths):
            err += (step[b].double().cpu() - ref[b][n + t]).square().sum().item()
            size += ref[b][n + t].square().sum().item()
    assert math.sqrt(err / size) <= 0.03, math.sqrt(err / size)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 32)])
def test_read_back(dk, dv, dtype):
    B, H, L = 4, 3, 6
    g = torch.Generator().manual_seed(dk)
    state, (codes, gate, exps) = _buffer(B, H, L, dk, dv)
    codes.copy_(torch.randint(-127, 128, codes.shape, generator=g).to(torch.int8))
    exps.copy_(torch.randint(0, 250, exps.shape, generator=g).to(torch.uint8))
    codes.masked_fill_((exps == 0).repeat_interleave(32, -1), 0)
    want = _values(codes, exps)
    # Exponents up to 249 are drawn here for any code: 127 * 2^(249 - 127) = 6.8e38 is above the range
    # of fp32 and bf16 (3.4e38), and reads as an infinity, as its conversion gives; what is in range
    # (all that a step or a prompt writes) is held exactly by both types.
    inside = want.abs() <= torch.finfo(torch.bfloat16).max
    assert torch.equal(want.to(dtype).double()[inside], want[inside]) and bool((~inside).any())
    want = want.to(dtype).double()
    got = binding.read_state_q8(state, B, H, L, dk, dv, dtype=dtype)
    assert got.dtype == dtype and torch.equal(got.double().cpu(), want)
    slot = torch.tensor([0, 4, 2, 3], dtype=torch.int32)
    got = binding.read_state_q8(state, B, H, L, dk, dv, slot=slot.to(DEV), dtype=dtype)
    assert torch.equal(got.double().cpu(), want[torch.arange(B), :, slot.long()])
    binding.device_status(clear=True)
    out = torch.full((B, H, dk, dv), 7.0, dtype=dtype, device=DEV)
    bad = torch.tensor([-1, 1, 5, 2 ** 31 - 1], dtype=torch.int32)
    binding.read_state_q8(state, B, H, L, dk, dv, slot=bad.to(DEV), out=out)
    assert binding.device_status(clear=True) == DECODE_POS
    assert bool((out[[0, 2, 3]] == 7.0).all()) and torch.equal(out[1].double().cpu(), want[1, :, 1])


def test_positions_and_lengths_out_of_range():
    B, H, L, d = 4, 2, 5, 64
    state, _ = _buffer(B, H, L, d, d)
    g = torch.Generator().manual_seed(1)
    state.copy_(torch.randint(0, 128, state.shape, generator=g).to(torch.uint8))
    before = state.clone()
    x = [torch.randn((B, H, d), generator=g).to(DEV) for _ in range(3)]
    la, lam = torch.zeros((B, H), device=DEV), torch.ones((B, H, L), device=DEV)
    out = torch.full((B, H, d), 7.0, device=DEV)
    pos = torch.tensor([-1, 16, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    binding.device_status(clear=True)
    binding.decode_step_q8(*x, la, lam, pos, state, out, B, H, L, d, d)
    assert binding.device_status(clear=True) == DECODE_POS
    assert torch.equal(state, before) and bool((out == 7.0).all())
    k, v, la, cu, dev = _prompt([16, 3], 2, d, d, "bf16", "dist", True)
    state, _ = _buffer(2, 2, L, d, d)
    before = state.clone()
    binding.prefill_state_q8(*dev, state, 2, 2, 16, L, d, d, cu_seqlens=cu.to(DEV))
    assert binding.device_status(clear=True) == DECODE_POS
    (c, ga, e), (bc, bg, be) = _views(state, 2, 2, L, d, d), _views(before, 2, 2, L, d, d)
    # (compared as bytes: the buffer's fill is no number as fp32 in general)
    assert torch.equal(c[0], bc[0]) and torch.equal(e[0], be[0])
    assert torch.equal(ga[0].view(torch.int32), bg[0].view(torch.int32))
    assert bool((ga[1] == ga[1]).all())
    binding.prefill_state_q8(*dev, state, 2, 2, 8, L, d, d, cu_seqlens=cu.to(DEV))   # cut at T = 8
    assert binding.device_status(clear=True) == SEQ_TOO_LONG
    S, size, _, _ = _prompt_levels(k, v, la, 0, 8, 4)
    _check_rounded(c[0, :, 3], e[0, :, 3], S, 2.0 ** -13 * size, "cut")


@pytest.mark.parametrize("B,H,d", [(3, 4, 64), (20, 40, 64), (12, 16, 128)])
def test_other_stream_and_graph_replay(B, H, d):
    """A decoding loop replayed from a graph (its position advanced on the device), beside the same
    loop on a stream: the same bits, for few heads and sequences and for many."""
    L, T = 8, 40
    g = torch.Generator().manual_seed(2)
    toks = [torch.randn((T, B, H, d), generator=g).to(DEV).bfloat16() for _ in range(3)]
    la = -torch.rand((T, B, H), generator=g).to(DEV)
    lam = torch.rand((T, B, H, L), generator=g).to(DEV)
    s = torch.cuda.Stream()
    a, _ = _buffer(B, H, L, d, d)
    b = a.clone()
    want = torch.empty((T, B, H, d), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for t in range(T):
            pos = torch.full((B,), t, dtype=torch.int32, device=DEV)
            binding.decode_step_q8(*(x[t] for x in toks), la[t], lam[t], pos, a, want[t], B, H, L, d, d)
    torch.cuda.synchronize()
    cur = [torch.empty_like(x[0]) for x in toks] + [torch.empty_like(la[0]), torch.empty_like(lam[0])]
    pos, out = torch.zeros(B, dtype=torch.int32, device=DEV), torch.empty((B, H, d), device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.decode_step_q8(*cur, pos, b, out, B, H, L, d, d)
        pos += 1
    for t in range(T):
        for c, x in zip(cur, toks + [la, lam]):
            c.copy_(x[t])
        graph.replay()
        assert torch.equal(out, want[t]), t


def test_the_librarys_buffer_and_a_callers_workspace():
    """llattn_prefill_state_q8 without a workspace and with one full of noise: the same bytes."""
    k, v, la, cu, dev = _prompt([3000, 1111], 4, 64, 64, "bf16", "slow", True)
    B, H, T, L, d = 2, 4, 3000, 13, 64
    want, _ = _buffer(B, H, L, d, d)
    blank = want.clone()
    c = cu.to(DEV)
    binding.prefill_state_q8(*dev, want, B, H, T, L, d, d, cu_seqlens=c)
    n = binding.prefill_q8_workspace_bytes(B, H, T, L, d, d)
    noise = torch.randint(0, 256, (n,), device=DEV).to(torch.uint8)
    s = torch.cuda.current_stream().cuda_stream
    args = [binding.BF16] + [t.data_ptr() for t in dev]
    for ws, size in ((None, 0), (noise.data_ptr(), n)):
        state = blank.clone()
        assert binding.lib().llattn_prefill_state_q8(*args, state.data_ptr(), B, H, T, L, d, d, c.data_ptr(), ws, size,
                                                     s) == 0
        assert torch.equal(state, want)
    assert binding.lib().llattn_prefill_state_q8(*args, want.data_ptr(), B, H, T, L, d, d, c.data_ptr(), noise.data_ptr(),
                                                 n - 1, s) == 7


@pytest.mark.parametrize("B,H,d", [(2, 3, 32), (32, 20, 64)])
def test_no_levels(B, H, d):
    """L = 1: the token alone, no state."""
    x = [torch.randn((B, H, d), device=DEV) for _ in range(3)]
    state = torch.empty(16, dtype=torch.uint8, device=DEV)
    out = torch.empty((B, H, d), device=DEV)
    lam = torch.rand((B, H, 1), device=DEV)
    zero = torch.zeros((B, H), device=DEV)
    binding.decode_step_q8(*x, zero, lam, torch.zeros(B, dtype=torch.int32, device=DEV), state, out, B, H, 1, d, d)
    q, k, v = (t.double() for t in x)
    ref = lam.double() * (q * k).sum(-1, True) * v
    assert bool(((out - ref).abs() <= 64 * U * lam * (q * k).abs().sum(-1, True) * v.abs()).all())
    assert binding.read_state_q8(state, B, H, 1, d, d).numel() == 0


def test_binding_refusals():
    B, H, L, d = 1, 1, 4, 32
    state, _ = _buffer(B, H, L, d, d)
    x = torch.zeros((B, H, d), device=DEV)
    la, lam = torch.zeros((B, H), device=DEV), torch.zeros((B, H, L), device=DEV)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    out = torch.empty((B, H, d), device=DEV)
    with pytest.raises(ValueError):
        binding.decode_step_q8(x, x, x, la, lam, pos, state[:-1], out, B, H, L, d, d)
    with pytest.raises(TypeError):
        binding.decode_step_q8(x, x, x, la, lam, pos.long(), state, out, B, H, L, d, d)
    with pytest.raises(ValueError):
        binding.decode_step_q8(x, x, x, la, lam[..., :2], pos, state, out, B, H, L, d, d)
    with pytest.raises(TypeError):
        binding.decode_step_q8(x, x.bfloat16(), x, la, lam, pos, state, out, B, H, L, d, d)
    with pytest.raises(ValueError):
        binding.prefill_state_q8(torch.zeros((B, 4, H, d), device=DEV), torch.zeros((B, 5, H, d), device=DEV),
                                 torch.zeros((B, 4, H), device=DEV), state, B, H, 4, L, d, d)
    with pytest.raises(TypeError):
        binding.read_state_q8(state, B, H, L, d, d, dtype=torch.float16)


@pytest.mark.parametrize("B,H,dk,dv", [(43, 64, 64, 64), (30, 60, 32, 128), (41, 70, 32, 32), (9, 75, 128, 128)])
def test_more_pairs_than_fit_the_machine(B, H, dk, dv):
    """Sequences of every position, some out of range (left as they are), beyond what runs at once."""
    L = 5
    nslot = L - 1
    g = torch.Generator().manual_seed(B)
    pos = torch.arange(B, dtype=torch.int32) % 18 - 1      # -1 and 16 are out of range
    good = (pos >= 0) & (pos < 16)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v = (rnd(B, H, n).to(torch.bfloat16) for n in (dk, dk, dv))
    la, lam = -torch.exp(rnd(B, H) - 2), torch.nn.functional.softplus(rnd(B, H, L))
    state, (codes, gate, exps) = _buffer(B, H, L, dk, dv)
    codes.copy_(torch.randint(-127, 128, codes.shape, generator=g).to(torch.int8))
    exps.copy_(torch.randint(110, 130, exps.shape, generator=g).to(torch.uint8))
    gate.copy_(-30 * torch.rand(gate.shape, generator=g) ** 4)
    before = state.clone()
    S, gate0 = _values(codes, exps), gate.cpu().clone()
    out = torch.full((B, H, dv), 7.0, device=DEV)
    binding.device_status(clear=True)
    binding.decode_step_q8(*[t.to(DEV) for t in (q, k, v, la, lam, pos)], state, out, B, H, L, dk, dv)
    assert binding.device_status(clear=True) == DECODE_POS
    ref, size, carry, csize, m = _step_ref(q[good].double(), k[good].double(), v[good].double(), la[good].double(),
                                           lam[good].double(), pos[good], S[good], gate0[good].double(), L)
    got = out.double().cpu()
    assert bool(((got[good] - ref).abs() <= 256 * U * size).all())
    assert bool((got[~good] == 7.0).all())
    bc, _, be = _views(before, B, H, L, dk, dv)
    for i, b in enumerate(torch.nonzero(good).flatten().tolist()):
        if int(m[i]) < nslot:
            _check_rounded(codes[b, :, m[i]], exps[b, :, m[i]], carry[i], 128 * U * csize[i], f"sequence {b}")
    for b in torch.nonzero(~good).flatten().tolist():
        assert torch.equal(codes[b], bc[b]) and torch.equal(exps[b], be[b]) and torch.equal(gate[b].cpu(), gate0[b])


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, "bf16"), (128, 128, "bf16"), (64, 128, "bf16"), (128, 128, "f32")])
def test_prompts_do_not_reach_into_their_neighbours(dk, dv, dtype):
    """A sequence between two of infinities and NaN holds the same levels as between two of numbers."""
    lengths, H, L = [70, 37, 90], 2, 8
    k, v, la, cu, dev = _prompt(lengths, H, dk, dv, dtype, "dist", True)
    want, _ = _buffer(3, H, L, dk, dv)
    got = want.clone()
    binding.prefill_state_q8(*dev, want, 3, H, 90, L, dk, dv, cu_seqlens=cu.to(DEV))
    at = torch.ones(sum(lengths), dtype=torch.bool, device=DEV)
    at[70:107] = False
    for t, bad in zip(dev, (math.nan, math.inf, math.nan)):
        t[at] = bad
    binding.prefill_state_q8(*dev, got, 3, H, 90, L, dk, dv, cu_seqlens=cu.to(DEV))
    for x, y in zip(_views(got, 3, H, L, dk, dv), _views(want, 3, H, L, dk, dv)):
        assert torch.equal(x[1].view(torch.uint8), y[1].view(torch.uint8))


def test_steps_and_prompts_side_by_side():
    """Steps of large batches, prompts and forwards of the attention on three streams at once: each the
    bits that it gives alone."""
    d, L, T = 128, 10, 500
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g).to(DEV).bfloat16()  # noqa: E731
    B, H = 16, 20                                                       # the steps'
    toks = [rnd(6, B, H, d) for _ in range(3)]
    la1, lam1 = -torch.rand((6, B, H), generator=g).to(DEV), torch.rand((6, B, H, L), generator=g).to(DEV)
    pos = torch.arange(B, dtype=torch.int32, device=DEV) * 17
    k, v, la = rnd(4, T, 8, d), rnd(4, T, 8, d), -torch.rand((4, T, 8), generator=g).to(DEV)
    lam = torch.rand((4, T, 8, binding.num_levels(T)), generator=g).to(DEV)
    q = (k / k.float().norm(dim=-1, keepdim=True)).bfloat16()

    def steps(state, out):
        for t in range(6):
            binding.decode_step_q8(*(x[t] for x in toks), la1[t], lam1[t], pos + t, state, out[t], B, H, L, d, d)

    def prompt(state):
        for _ in range(6):
            binding.prefill_state_q8(k, v, la, state, 4, 8, T, L, d, d)

    def attention(out):
        ws = torch.empty(binding.workspace_bytes(binding.BF16, "auto", 0, 4, 8, T, d, d, False), dtype=torch.uint8, device=DEV)
        for _ in range(6):
            binding.forward(q, q, v, la, lam, out=out, workspace=ws if ws.numel() else None)

    held = torch.zeros(binding.decode_q8_state_bytes(B, H, L, d, d), dtype=torch.uint8, device=DEV)
    empty = torch.zeros(binding.decode_q8_state_bytes(4, 8, L, d, d), dtype=torch.uint8, device=DEV)
    res = []
    for streams in ([torch.cuda.current_stream()] * 3, [torch.cuda.Stream() for _ in range(3)]):
        a, b = held.clone(), empty.clone()
        o1, o2 = torch.zeros((6, B, H, d), device=DEV), torch.zeros((4, T, 8, d), device=DEV)
        torch.cuda.synchronize()
        for st, f in zip(streams, (lambda: steps(a, o1), lambda: prompt(b), lambda: attention(o2))):
            with torch.cuda.stream(st):
                f()
        torch.cuda.synchronize()
        res.append((a, b, o1, o2))
    assert binding.device_status(clear=True) == 0
    for x, y in zip(*res):
        assert torch.equal(x, y)
