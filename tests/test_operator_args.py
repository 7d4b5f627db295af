"""Refusals of the layer operators (norms with rotation, gated recurrence, 8-bit decoding state)
before any CUDA call, and their size queries.  No GPU: the pointers are made up and never read."""
import ctypes

import pytest

from hierarchical_fenwick_state_b200 import binding

OK, ARG, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
M = 1 << 20   # far enough apart for every size below
F32, BF16 = binding.F32, binding.BF16


def _call(name, order, defaults, kw):
    a = dict(defaults, **kw)
    assert set(a) == set(order.split()), set(a) ^ set(order.split())
    return getattr(binding.lib(), name)(*[a[n] for n in order.split()])


QK = dict(in_dtype=BF16, q=1 * M, k=2 * M, qs=512, ks=512, wq=None, wk=None, pos=3 * M, freq=4 * M,
          qo=5 * M, ko=6 * M, N=16, Gq=4, Gk=2, H=4, d=64, rot=32, layout=0, norm=0, eps=1e-6,
          stream=None)
QK_ORDER = "in_dtype q k qs ks wq wk pos freq qo ko N Gq Gk H d rot layout norm eps stream"

QK_BAD = [
    (dict(in_dtype=2), DTYPE), (dict(d=48), SHAPE), (dict(d=256), SHAPE), (dict(N=-1), SHAPE),
    (dict(H=0), SHAPE), (dict(H=65536), SHAPE), (dict(Gq=0), SHAPE), (dict(Gq=3), SHAPE),
    (dict(Gk=8), SHAPE), (dict(rot=12), SHAPE), (dict(rot=72), SHAPE), (dict(rot=-8), SHAPE),
    (dict(layout=2), ARG), (dict(norm=2), ARG), (dict(norm=-1), ARG), (dict(eps=0.0), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(qs=255), SHAPE), (dict(ks=64), SHAPE), (dict(N=1 << 40), SHAPE),
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(pos=None), ARG), (dict(freq=None), ARG),
    (dict(q=M + 8), ALIGN), (dict(k=2 * M + 2), ALIGN), (dict(qs=260), ALIGN),
    (dict(wq=7 * M + 2), ALIGN), (dict(pos=3 * M + 1), ALIGN),
]


@pytest.mark.parametrize("kw,status", QK_BAD + [
    (dict(qo=None), ARG), (dict(ko=6 * M + 8), ALIGN),
    (dict(qo=1 * M), ARG),                       # in place
    (dict(qo=1 * M + 15 * 1024), ARG),           # over q's last token
    (dict(ko=5 * M + 16), ARG),                  # over the other output
    (dict(qo=3 * M - 16), ARG),                  # over pos
])
def test_qk_refusals(kw, status):
    assert _call("llattn_qk_norm_rope", QK_ORDER, QK, kw) == status


QKB = {**{n: v for n, v in QK.items() if n not in ("qo", "ko", "stream")}, "wq": 7 * M, "wk": 8 * M,
       "dqo": 5 * M, "dko": 6 * M, "dq": 9 * M, "dk": 10 * M, "dqs": 512, "dks": 512, "dwq": 11 * M,
       "dwk": 12 * M, "ws": 13 * M, "wsn": 1 << 30, "stream": None}
QKB_ORDER = ("in_dtype q k qs ks wq wk pos freq dqo dko dq dk dqs dks dwq dwk N Gq Gk H d rot layout norm "
             "eps ws wsn stream")


@pytest.mark.parametrize("kw,status", QK_BAD + [
    (dict(dqo=None), ARG), (dict(dk=None), ARG), (dict(wq=None), ARG), (dict(dqs=255), SHAPE),
    (dict(dks=126), SHAPE), (dict(dq=9 * M + 4), ALIGN), (dict(dqs=513), ALIGN),
    (dict(dwk=12 * M + 1), ALIGN), (dict(dwq=12 * M), ARG), (dict(dq=5 * M), ARG),
    (dict(dk=9 * M + 64 * 4), ARG),              # dk's columns on dq's, same stride
    (dict(dk=9 * M + 448 * 4), ARG),             # dk's columns reach into dq's next token
])
def test_qk_backward_refusals(kw, status):
    assert _call("llattn_qk_norm_rope_bwd", QKB_ORDER, QKB, kw) == status


def test_qk_empty_calls_and_workspace():
    assert _call("llattn_qk_norm_rope", QK_ORDER, QK, dict(N=0)) == OK
    assert _call("llattn_qk_norm_rope", QK_ORDER, QK, dict(N=0, q=None, qo=None, pos=None)) == OK
    assert _call("llattn_qk_norm_rope_bwd", QKB_ORDER, QKB, dict(N=0, dwq=None, dwk=None)) == OK
    assert binding.qk_norm_rope_bwd_workspace_bytes(64, False) == 0
    for d in (32, 64, 128):          # what the binding allocates without asking
        assert binding.qk_norm_rope_bwd_workspace_bytes(d, True) == 148 * 2 * 2 * d * 4
    with pytest.raises(binding.LLAttnError):
        binding.qk_norm_rope_bwd_workspace_bytes(48)


GLR = dict(in_dtype=BF16, x=1 * M, log_a=2 * M, h0=None, h=3 * M, h_last=None, B=2, T=16, D=64,
           cu=None, ws=None, wsn=0, stream=None)
GLR_ORDER = "in_dtype x log_a h0 h h_last B T D cu ws wsn stream"


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=7), DTYPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=-1), SHAPE),
    (dict(B=65536), SHAPE), (dict(D=65536), SHAPE), (dict(T=(1 << 24) + 1), SHAPE),
    (dict(B=65535, T=1 << 24, D=64), SHAPE),
    (dict(x=None), ARG), (dict(log_a=None), ARG), (dict(h=None), ARG),
    (dict(x=M + 1), ALIGN), (dict(in_dtype=F32, x=M + 2), ALIGN), (dict(log_a=2 * M + 2), ALIGN),
    (dict(h=3 * M + 1), ALIGN), (dict(h_last=4 * M + 2), ALIGN), (dict(cu=4 * M + 1), ALIGN),
    (dict(h=2 * M), ARG), (dict(h=2 * M + 2 * 16 * 64 * 4 - 4), ARG), (dict(h=1 * M), ARG),
    (dict(h_last=3 * M), ARG), (dict(h0=4 * M, h_last=4 * M + 4), ARG), (dict(h0=3 * M), ARG),
    (dict(cu=5 * M, h_last=5 * M + 4), ARG),
])
def test_glr_refusals(kw, status):
    assert _call("llattn_glr_fwd", GLR_ORDER, GLR, kw) == status


GLRB = dict(log_a=1 * M, h=2 * M, h0=None, dh=3 * M, dh_last=None, dx=4 * M, dlog_a=5 * M, dh0=None,
            B=2, T=16, D=64, cu=None, ws=None, wsn=0, stream=None)
GLRB_ORDER = "log_a h h0 dh dh_last dx dlog_a dh0 B T D cu ws wsn stream"


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=65536), SHAPE), (dict(dh=None), ARG),
    (dict(dx=None), ARG), (dict(dlog_a=None), ARG), (dict(h=None), ARG), (dict(dx=4 * M + 2), ALIGN),
    (dict(dh0=6 * M + 1), ALIGN), (dict(dx=3 * M), ARG), (dict(dx=5 * M), ARG), (dict(dx=2 * M), ARG),
    (dict(dh_last=6 * M, dh0=6 * M), ARG), (dict(h0=6 * M, dh0=6 * M + 508), ARG),
])
def test_glr_backward_refusals(kw, status):
    assert _call("llattn_glr_bwd", GLRB_ORDER, GLRB, kw) == status


def test_glr_workspace():
    assert binding.glr_workspace_bytes(64, 1, 2048) == 0
    assert binding.glr_workspace_bytes(0, 5000, 64) == 0
    for shape in ((1, 64, 7), (1, 65, 7), (64, 1, 2048), (3, 1000, 33), (0, 100, 4), (5, 16384, 1024)):
        assert binding.glr_workspace_bytes(*shape) == binding._glr_need(*shape), shape
    n = binding.glr_workspace_bytes(1, 65536, 2048)
    assert 0 < n < 65536 * 2048      # small beside the 10 bytes per element of a call
    for bad in ((-1, 1, 1), (1, 1 << 25, 1), (1, 1, 65536), (65535, 1 << 24, 64)):
        with pytest.raises(binding.LLAttnError):
            binding.glr_workspace_bytes(*bad)


def test_glr_empty_calls():
    for kw in (dict(B=0), dict(D=0), dict(T=0)):
        assert _call("llattn_glr_fwd", GLR_ORDER, GLR, kw) == OK
        assert _call("llattn_glr_bwd", GLRB_ORDER, GLRB, kw) == OK


STEP = dict(in_dtype=BF16, q=1 * M, k=2 * M, v=3 * M, log_a=4 * M, lam=5 * M, pos=6 * M, state=64 * M,
            out=7 * M, B=2, H=3, L=14, dk=64, dv=64, stream=None)
STEP_ORDER = "in_dtype q k v log_a lam pos state out B H L dk dv stream"


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), DTYPE), (dict(dk=48), SHAPE), (dict(L=0), SHAPE), (dict(L=33), SHAPE),
    (dict(B=-1), SHAPE), (dict(H=65536), SHAPE), (dict(q=None), ARG), (dict(pos=None), ARG),
    (dict(state=None), ARG), (dict(out=None), ARG), (dict(q=M + 8), ALIGN), (dict(state=64 * M + 8), ALIGN),
    (dict(lam=5 * M + 2), ALIGN), (dict(out=64 * M), ARG), (dict(out=5 * M), ARG), (dict(state=6 * M), ARG),
])
def test_step_q8_refusals(kw, status):
    assert _call("llattn_decode_step_q8", STEP_ORDER, STEP, kw) == status


PRE = dict(in_dtype=BF16, k=1 * M, v=2 * M, log_a=3 * M, state=64 * M, B=2, H=3, T=100, L=14, dk=64, dv=64,
           cu=None, ws=None, wsn=0, stream=None)
PRE_ORDER = "in_dtype k v log_a state B H T L dk dv cu ws wsn stream"


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), DTYPE), (dict(dv=48), SHAPE), (dict(L=0), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=(1 << 24) + 1), SHAPE), (dict(k=None), ARG), (dict(state=None), ARG), (dict(v=2 * M + 8), ALIGN),
    (dict(log_a=3 * M + 2), ALIGN), (dict(cu=4 * M + 2), ALIGN), (dict(state=2 * M), ARG),
    (dict(state=2 * M - 16), ARG),
])
def test_prefill_q8_refusals(kw, status):
    assert _call("llattn_prefill_state_q8", PRE_ORDER, PRE, kw) == status


READ = dict(state=64 * M, slot=None, out=1 * M, out_dtype=BF16, B=2, H=3, L=14, dk=64, dv=64, stream=None)
READ_ORDER = "state slot out out_dtype B H L dk dv stream"


@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=2), DTYPE), (dict(dk=16), SHAPE), (dict(L=33), SHAPE), (dict(state=None), ARG),
    (dict(out=None), ARG), (dict(out=M + 8), ALIGN), (dict(slot=2 * M + 2), ALIGN), (dict(out=64 * M), ARG),
    (dict(slot=1 * M), ARG),
])
def test_read_q8_refusals(kw, status):
    assert _call("llattn_read_state_q8", READ_ORDER, READ, kw) == status


def test_prefill_q8_workspace():
    assert binding.prefill_q8_workspace_bytes(0, 4, 100, 14, 64, 64) == 0
    assert binding.prefill_q8_workspace_bytes(2, 4, 100, 1, 64, 64) == 0
    for B, H, T, dk, dv in ((8, 16, 16384, 64, 64), (32, 32, 8192, 64, 64), (1, 1, 1 << 24, 128, 128)):
        assert 0 < binding.prefill_q8_workspace_bytes(B, H, T, 25, dk, dv) <= (64 << 20) + (1 << 18)
    for bad in ((-1, 1, 1, 14, 64, 64), (1, 1, 1 << 25, 14, 64, 64), (1, 1, 1, 33, 64, 64), (1, 1, 1, 14, 48, 64)):
        with pytest.raises(binding.LLAttnError):
            binding.prefill_q8_workspace_bytes(*bad)


def test_q8_empty_calls_and_state_bytes():
    for kw in (dict(B=0), dict(H=0)):
        assert _call("llattn_decode_step_q8", STEP_ORDER, STEP, kw) == OK
        assert _call("llattn_prefill_state_q8", PRE_ORDER, PRE, kw) == OK
        assert _call("llattn_read_state_q8", READ_ORDER, READ, kw) == OK
    assert _call("llattn_read_state_q8", READ_ORDER, READ, dict(L=1)) == OK
    for B, H, L, dk, dv in ((1, 1, 1, 32, 32), (64, 32, 14, 64, 64), (3, 5, 17, 128, 32)):
        n = B * H * (L - 1)
        assert binding.decode_q8_state_bytes(B, H, L, dk, dv) == n * (dk * dv + 8 + dk * dv // 32)
    with pytest.raises(binding.LLAttnError):
        binding.decode_q8_state_bytes(1, 1, 14, 48, 64)
    assert binding.lib().llattn_decode_q8_state_bytes(1, 1, 2, 32, 32, ctypes.POINTER(ctypes.c_size_t)()) == ARG


def test_binding_refuses_what_it_cannot_pass_on():
    import torch
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(x, x)                       # not on the GPU
    with pytest.raises(TypeError):
        binding.qk_norm_rope(x.double(), x.double())
    with pytest.raises(TypeError):
        binding.glr_forward(x.half(), x)
    with pytest.raises(ValueError):
        binding.glr_forward(x, x)
    with pytest.raises(ValueError):
        binding.read_state_q8(torch.zeros(8, dtype=torch.uint8), 1, 1, 2, 32, 32)


def test_workspace_is_checked():
    import torch
    like = torch.empty(4)
    ws, at, size = binding._workspace(torch.empty(8), 16, like, None)
    assert (at, size) == (ws.data_ptr(), 32)
    for bad in (torch.empty(16)[::2], torch.empty(16, device="meta")):   # strided; of another device
        with pytest.raises(ValueError):
            binding._workspace(bad, 16, like, None)


def test_glr_packed_workspace():
    """What the binding allocates without asking; never more than for any batch of the bound."""
    for B, T, rows, D in ((64, 65536, 71836, 2048), (3, 64, 100, 33), (3, 65, 100, 33), (8, 16384, 92526, 1024),
                          (5, 1 << 24, 7, 1), (65535, 1 << 24, 1 << 21, 64), (0, 100, 0, 4), (2, 1000, 0, 4)):
        n = binding.glr_packed_workspace_bytes(B, T, rows, D)
        assert n == binding._glr_need(B, T, D, rows), (B, T, rows, D)
        if B * T * D < 1 << 40:
            assert n <= binding.glr_workspace_bytes(B, T, D)
    for bad in ((-1, 1, 1, 1), (1, 1 << 25, 1, 1), (1, 1, 1, 65536), (1, 1, -1, 1), (1, 1, 1 << 31, 1)):
        with pytest.raises(binding.LLAttnError):
            binding.glr_packed_workspace_bytes(*bad)


def test_glr_packed_bounds():
    """A packed call's B * T * D is no limit, its rows are; a workspace without a slot per sequence is refused."""
    big = dict(B=64, T=1 << 24, D=2048, cu=6 * M)
    assert _call("llattn_glr_fwd", GLR_ORDER, GLR, dict(big, ws=7 * M, wsn=256 + 64 * 64 * 512 - 1, x=None)) == ARG
    assert _call("llattn_glr_fwd", GLR_ORDER, GLR, dict(big, cu=None)) == SHAPE
    assert _call("llattn_glr_bwd", GLRB_ORDER, GLRB, dict(big, cu=None)) == SHAPE
