"""Packed batches of the gated linear recurrence whose bound T says little about them: bounds far above every
length, and one long sequence among many short ones.  The scratch follows the rows, and the results are
the bits of a call with the exact bound."""
import math

import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SEQ_TOO_LONG, BAD_CU, WORKSPACE = 1, 4, 32


def _batch(lengths, D, dtype=torch.bfloat16, behind=0):
    g = torch.Generator(device=DEV).manual_seed(sum(lengths) + D)
    n = sum(lengths) + behind
    x = torch.randn((n, D), generator=g, device=DEV).to(dtype)
    la = -torch.exp(-3 + 0.5 * torch.randn((n, D), generator=g, device=DEV))
    dh = torch.randn((n, D), generator=g, device=DEV)
    h0, dl = (torch.randn((len(lengths), D), generator=g, device=DEV) for _ in range(2))
    return x, la, dh, h0, dl, torch.tensor([0] + lengths).cumsum(0).int().to(DEV)


def _both(x, la, dh, h0, dl, cu, T, **kw):
    last = torch.full_like(h0, math.nan)
    h = binding.glr_forward(x, la, h0=h0, h_last=last, cu_seqlens=cu, T=T, **kw)
    return {"h": h, "last": last, **binding.glr_backward(la, h, dh, h0=h0, dh_last=dl, cu_seqlens=cu, T=T, **kw)}


LENGTHS = [[100, 0, 300, 17, 1, 65], [3] * 40 + [5000] + [60] * 40, [700] * 5, [0, 0, 4000, 0], [200] * 150 + [3000]]


@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("lengths", LENGTHS, ids=[f"{len(n)}x{max(n)}" for n in LENGTHS])
def test_any_bound_gives_the_same_bits(lengths, D):
    args = _batch(lengths, D, behind=1000)      # rows behind the last sequence, which only loosen the rows' bound
    n, cu = sum(lengths), args[-1].tolist()
    binding.device_status(clear=True)
    base = torch.cuda.memory_allocated()
    want = _both(*args, max(lengths))
    for T in (max(lengths) + 1, 65536, 1 << 24):
        torch.cuda.reset_peak_memory_stats()
        got = _both(*args, T)
        assert torch.cuda.max_memory_allocated() - base < 40 * (n + 1000) * D + (1 << 24)
        for m in want:
            a, b = (got[m][:n], want[m][:n]) if m in ("h", "x", "log_a") else (got[m], want[m])
            assert torch.equal(a, b), (T, m)
    # and those of its sequences one by one
    x, la, dh, h0, dl, _ = args
    for b in {0, len(lengths) // 2, len(lengths) - 1, lengths.index(max(lengths))}:
        s, e = cu[b], cu[b + 1]
        if e - s <= 16:                         # another form
            continue
        one = _both(x[None, s:e].contiguous(), la[None, s:e].contiguous(), dh[None, s:e].contiguous(), h0[b:b + 1],
                    dl[b:b + 1], None, None)
        for m in want:
            if m in ("h", "x", "log_a"):
                assert torch.equal(one[m][0], want[m][s:e]), (b, m)
            else:
                name = {"last": "last", "h0": "h0"}[m]
                assert torch.equal(one[m][0], want[name][b]), (b, m)
    assert binding.device_status(clear=True) == 0


@pytest.mark.parametrize("D", [64, 33])
def test_workspaces_of_either_size(D):
    lengths = [400, 20, 1900, 0, 65]
    args = _batch(lengths, D)
    B, T, n = len(lengths), 2000, sum(lengths)
    small, big = binding.glr_packed_workspace_bytes(B, T, n, D), binding.glr_workspace_bytes(B, T, D)
    assert small < big
    want = _both(*args, T)
    for size in (small, big):
        ws = torch.randint(0, 256, (size,), device=DEV).to(torch.uint8)
        got = _both(*args, T, workspace=ws)
        for m in want:
            assert torch.equal(got[m], want[m]), (size, m)
    # room for a slot of each sequence and no more: taken, and refused by the kernel
    binding.device_status(clear=True)
    tiny = torch.empty(binding.glr_packed_workspace_bytes(B, T, 0, D), dtype=torch.uint8, device=DEV)
    out = torch.full_like(args[1], 7.0)
    binding.glr_forward(args[0], args[1], cu_seqlens=args[-1], T=T, out=out, workspace=tiny)
    assert binding.device_status(clear=True) == WORKSPACE and bool((out == 7.0).all())
    with pytest.raises(binding.LLAttnError):    # not even that
        binding.glr_forward(args[0], args[1], cu_seqlens=args[-1], T=T, out=out, workspace=tiny[:-1])


def test_offsets_that_do_not_start_at_zero_or_decrease():
    """A batch that is a part of a longer one keeps its rows' numbers; decreasing offsets are reported."""
    lengths = [300, 50, 1000, 64]
    x, la, dh, h0, dl, cu = _batch(lengths, 64)
    want = _both(x, la, dh, h0, dl, cu, 4096)
    binding.device_status(clear=True)
    out = torch.full_like(la, 7.0)
    last = torch.empty_like(h0[1:])
    binding.glr_forward(x, la, h0=h0[1:], h_last=last, cu_seqlens=cu[1:], T=4096, out=out)
    assert torch.equal(out[300:], want["h"][300:]) and bool((out[:300] == 7.0).all())
    assert torch.equal(last, want["last"][1:])
    assert binding.device_status(clear=True) == 0
    bad = torch.tensor([0, 300, 200, 1350, 1414], dtype=torch.int32, device=DEV)
    binding.glr_forward(x, la, h0=h0, h_last=torch.empty_like(h0), cu_seqlens=bad, T=1200, out=out,
                        workspace=torch.empty(binding.glr_workspace_bytes(4, 1200, 64), dtype=torch.uint8, device=DEV))
    assert binding.device_status(clear=True) == BAD_CU
