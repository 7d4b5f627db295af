"""A prompt's hand-off to decoding with log gates of -inf and -1e5 among ordinary ones, inside buckets and
behind them: on the 8-bit state (both of its kernels) and on the fp32 state, and a step from there.

Bounds (u = 2^-24), in the terms' absolute values.  A term's decay is exp of a sum of at most 16 + 5 + 16
roundings, each at most u of the sum D of the |log_a| behind the term (tokens in its bucket, up to the next gate of 0), and
exp itself 4 u: (64 D + 4) u.  Products and sums: buckets of at most 1024 tokens are summed 16 at a
time in pieces of at most 512, each time cut off at 2 u of the sum so far, at most 32 + 8 times, and the
operands' parts leave 2^-24: 2^-17 in all.  fp32 sums of the terms one by one, 128 or fewer to a
CTA of a cluster, stay in that too.  A bucket's terms before a gate of 0 (exp of -inf or of -1e5) add
nothing.  Held values are then rounded by half a step.
"""
import math

import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _prompt(lengths, H, dk, dv, dtype, mode):
    g = torch.Generator().manual_seed(sum(lengths) + dk + dv + len(mode))
    total = sum(lengths)
    k = torch.randn((total, H, dk), generator=g)
    k = (k / k.norm(dim=-1, keepdim=True)).to(DT[dtype])
    v = torch.randn((total, H, dv), generator=g).to(DT[dtype])
    la = -torch.exp(-2 + 0.5 * torch.randn((total, H), generator=g))
    at = torch.rand((total, H), generator=g) < 0.06
    la[at] = {"cut": torch.tensor([-math.inf]), "deep": torch.tensor([-1e5]),
              "both": torch.tensor([-math.inf, -1e5])}[mode][torch.randint(1 + (mode == "both"), (int(at.sum()),), generator=g)]
    return k, v, la, torch.tensor([0] + lengths).cumsum(0).int()


def _level(k, v, la, s, n, lvl):
    """Exact slot of level lvl of the sequence [s, s + n), its bound, and its pending gate with its bound."""
    lo = (n >> lvl) << lvl
    hi = lo + (1 << (lvl - 1))
    a = la[s + lo:s + hi].double()
    behind = torch.cat([a[1:], torch.zeros_like(a[:1])])           # of the tokens after each
    D = behind.flip(0).cumsum(0).flip(0)
    f = torch.exp(D)
    err = torch.where(f > 0, f * (2.0 ** -17 + 4 * U + 64 * U * torch.where(f > 0, -D, 0.0)), 0.0)
    kk, vv = k[s + lo:s + hi].double(), v[s + lo:s + hi].double()
    rest = la[s + hi:s + n].double()
    return (torch.einsum("thi,th,thj->hij", kk, f, vv), torch.einsum("thi,th,thj->hij", kk.abs(), err, vv.abs()),
            rest.sum(0), 256 * U * rest.abs().sum(0))


SHAPES = [("bf16", 64, 64), ("bf16", 128, 32), ("bf16", 32, 128), ("f32", 64, 64), ("f32", 128, 128),
          ("bf16", 64, 128), ("bf16", 128, 128)]
LENGTHS = [1023, 3, 64, 257, 600]


@pytest.mark.parametrize("mode", ["cut", "deep", "both"])
@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
def test_8_bit_state(dtype, dk, dv, mode):
    B, H, L = len(LENGTHS), 2, 12
    k, v, la, cu = _prompt(LENGTHS, H, dk, dv, dtype, mode)
    state = torch.zeros(binding.decode_q8_state_bytes(B, H, L, dk, dv), dtype=torch.uint8, device=DEV)
    n = B * H * (L - 1)
    gate = state[n * dk * dv:n * (dk * dv + 8)].view(torch.float32).view(B, H, 2, L - 1)
    exps = state[n * (dk * dv + 8):].view(B, H, L - 1, dk, dv // 32)
    binding.prefill_state_q8(k.to(DEV), v.to(DEV), la.to(DEV), state, B, H, max(LENGTHS), L, dk, dv,
                             cu_seqlens=cu.to(DEV))
    held = binding.read_state_q8(state, B, H, L, dk, dv, dtype=torch.float32).double().cpu()
    step = torch.exp2(exps.double().cpu() - 127).repeat_interleave(32, -1)
    for b, m in enumerate(LENGTHS):
        for j in range(L - 1):
            if m >> j & 1:
                S, err, rest, rerr = _level(k, v, la, int(cu[b]), m, j + 1)
                assert bool(held[b, :, j].isfinite().all()), (m, j)
                assert bool(((held[b, :, j] - S).abs() <= 0.5 * step[b, :, j] + err).all()), (m, j)
                got = gate[b, :, 0, j].double().cpu()
                assert bool(((got == rest) | ((got - rest).abs() <= rerr)).all()), (m, j)
    # a step from there: levels behind a gate of 0 add nothing
    g = torch.Generator().manual_seed(7)
    q, k1 = (torch.randn((B, H, dk), generator=g).to(DT[dtype]) for _ in range(2))
    v1, lam = torch.randn((B, H, dv), generator=g).to(DT[dtype]), torch.rand((B, H, L), generator=g)
    la1, pos = -torch.rand((B, H), generator=g), torch.tensor(LENGTHS, dtype=torch.int32)
    w = torch.exp(gate.double().cpu()[torch.arange(B), :, (pos & 1).long()] + la1.double()[..., None])
    on = ((pos[:, None] >> torch.arange(L - 1)) & 1).double()[:, None]
    qd, kd, vd = q.double(), k1.double(), v1.double()
    parts = torch.einsum("bhi,bhlij,bhl->bhlj", qd, held * on[..., None, None], w * lam[..., 1:].double())
    size = torch.einsum("bhi,bhlij,bhl->bhj", qd.abs(), held.abs() * on[..., None, None], w * lam[..., 1:].double())
    want = parts.sum(2) + lam[..., :1].double() * (qd * kd).sum(-1, True) * vd
    size = size + lam[..., :1].double() * (qd * kd).abs().sum(-1, True) * vd.abs()
    out = torch.empty((B, H, dv), device=DEV)
    binding.decode_step_q8(*(t.to(DEV) for t in (q, k1, v1, la1, lam, pos)), state, out, B, H, L, dk, dv)
    assert bool(((out.double().cpu() - want).abs() <= 256 * U * size).all())
    assert binding.device_status(clear=True) == 0


@pytest.mark.parametrize("mode", ["cut", "deep", "both"])
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 64), ("f32", 32, 128)])
def test_fp32_state(dtype, dk, dv, mode):
    B, H, L = len(LENGTHS), 2, 12
    k, v, la, cu = _prompt(LENGTHS, H, dk, dv, dtype, mode)
    state = torch.zeros(binding.decode_state_bytes(B, H, L, dk, dv) // 4, device=DEV)
    n = B * H * (L - 1)
    levels, gate = state[:n * dk * dv].view(B, H, L - 1, dk, dv), state[n * dk * dv:].view(B, H, 2, L - 1)
    binding.prefill_state(k.to(DEV), v.to(DEV), la.to(DEV), state, B, H, max(LENGTHS), L, dk, dv,
                          cu_seqlens=cu.to(DEV))
    for b, m in enumerate(LENGTHS):
        for j in range(L - 1):
            if m >> j & 1:
                S, err, rest, rerr = _level(k, v, la, int(cu[b]), m, j + 1)
                got = levels[b, :, j].double().cpu()
                assert bool(got.isfinite().all()) and bool(((got - S).abs() <= err + 2.0 ** -126).all()), (m, j)
                got = gate[b, :, 0, j].double().cpu()
                assert bool(((got == rest) | ((got - rest).abs() <= rerr)).all()), (m, j)
    assert binding.device_status(clear=True) == 0
