"""A prompt's 8-bit levels where only the operands' small parts are left (see _prompt_parts): that the sums
of all parts meet the bound and that those without any one of them do not (CPU), and the kernels (GPU)."""
import pytest
import torch

import _prompt_parts as P
from hierarchical_fenwick_state_b200 import binding

BF16, F32 = torch.bfloat16, torch.float32
ALL = {BF16: [(0, 0), (1, 0), (2, 0)], F32: [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0)]}


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_bound_tells_a_missing_part(dtype):
    k, v, la, exact, err = P.make(dtype, 1, 2, 64, 64, 3)
    assert not P.off(*P.rounded(P.sums(k, v, la, ALL[dtype])), exact, err)
    for drop in ALL[dtype]:
        assert P.off(*P.rounded(P.sums(k, v, la, [p for p in ALL[dtype] if p != drop])), exact, err), drop


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 32, 32), (BF16, 64, 64), (BF16, 128, 64), (BF16, 32, 128), (F32, 64, 64),
                                         (F32, 32, 128), (F32, 128, 128), (BF16, 64, 128), (BF16, 128, 128)])
def test_every_part_is_in_the_sum(dtype, dk, dv):
    B, H, L, dev = 3, 4, 4, "cuda:0"
    k, v, la, exact, err = P.make(dtype, B, H, dk, dv, dk + dv)
    state = torch.zeros(binding.decode_q8_state_bytes(B, H, L, dk, dv), dtype=torch.uint8, device=dev)
    binding.prefill_state_q8(k.to(dev), v.to(dev), la.to(dev), state, B, H, P.LENGTH, L, dk, dv)
    n = B * H * (L - 1)
    exps = state[n * (dk * dv + 8):].view(B, H, L - 1, dk, dv // 32)[:, :, 2]
    held = binding.read_state_q8(state, B, H, L, dk, dv, dtype=F32)[:, :, 2].double().cpu()
    step = torch.exp2(exps.double().cpu() - 127).repeat_interleave(32, -1)
    assert not P.off(held, step, exact, err), ((held - exact).abs() - 0.5 * step).div(err).max()
    assert binding.device_status(clear=True) == 0
