"""A stack of two layers as a user runs it: log-linear attention on normalised, rotated q and k, and the gated
recurrence over what it gives.  A packed training step against the same formulas differentiated in 64 bits, and
prompts that are carried on token by token through both layers' states.

Bounds: the attention is held to 1e-4 of its output's RMS (fp32 inputs), and so are its gradients.  The
recurrence passes errors on with weights that sum to 1 / (1 - a), about 8 here, where the values themselves,
of random signs, grow by 1 / sqrt(1 - a^2), about 2; its own rounding and that of the norms are below 1e-5.  So
1e-4 becomes at most about 4e-4 of the RMS at either end: 1e-3 is asked for.
"""
import pytest
import torch

from hierarchical_fenwick_state_b200 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, D, G = 2, 32, 1
LENGTHS = [33, 1, 70, 0, 9]


def _inputs(total, L, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(xq=r(total, H, D), xk=r(total, G, D), v=r(total, H, D), la=-torch.exp(-2 + 0.5 * r(total, H)),
                lam=torch.nn.functional.softplus(r(total, H, L)), gate=-torch.exp(-2 + 0.5 * r(total, H * D)),
                w=1 + 0.1 * r(D))


def _norm_rope(x, pos, freq, w, heads):
    y = x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6) * w
    a = (pos.double()[:, None] * freq.double())[:, None]
    n = freq.numel()
    y = torch.cat([y[..., :n] * a.cos() - y[..., n:2 * n] * a.sin(), y[..., :n] * a.sin() + y[..., n:2 * n] * a.cos(),
                   y[..., 2 * n:]], -1)
    return y.repeat_interleave(heads // x.shape[1], 1)


def _stack(p, n, freq):
    """Both layers' outputs of one sequence of n tokens, in 64 bits."""
    pos = torch.arange(n)
    q, k = _norm_rope(p["xq"], pos, freq, p["w"], H), _norm_rope(p["xk"], pos, freq, p["w"], H)
    c = p["la"].cumsum(0)
    t, s = torch.meshgrid(pos, pos, indexing="ij")
    level = torch.where(t == s, 0, 1 + torch.floor(torch.log2((t ^ s).clamp_min(1).double())).long())
    seen = (s <= t)[..., None]
    decay = torch.exp(torch.where(seen, c[:, None] - c[None], 0.0)) * seen
    lam = torch.gather(p["lam"][:, None].expand(n, n, H, -1), 3, level[..., None, None].expand(n, n, H, 1))[..., 0]
    y = torch.einsum("tsh,shd->thd", torch.einsum("thd,shd->tsh", q, k) * decay * lam, p["v"])
    h, hs = torch.zeros(H * D).double(), []
    for i in range(n):
        h = p["gate"][i].exp() * h + y[i].flatten()
        hs.append(h)
    return y, torch.stack(hs) if hs else y.reshape(0, H * D)


def _near(got, ref, what):
    err = (got.double().cpu().reshape(ref.shape) - ref).abs().max() / ref.square().mean().sqrt()
    assert err <= 1e-3, f"{what}: {err:.2e}"


def test_training_step():
    T, B, total = max(LENGTHS), len(LENGTHS), sum(LENGTHS)
    p = _inputs(total, binding.num_levels(T), 0)
    cu = torch.tensor([0] + LENGTHS).cumsum(0)
    freq = (100.0 ** (-2 * torch.arange(8).double() / 16)).float()
    dh = torch.randn((total, H * D), generator=torch.Generator().manual_seed(1))

    d = {n: t.to(DEV) for n, t in p.items()}
    cud, pos = cu.int().to(DEV), torch.cat([torch.arange(n) for n in LENGTHS]).int().to(DEV)
    how = dict(wq=d["w"], wk=d["w"], pos=pos, inv_freq=freq.to(DEV))
    q, k = binding.qk_norm_rope(d["xq"], d["xk"], heads=H, **how)
    y = binding.forward(q, k, d["v"], d["la"], d["lam"], cu_seqlens=cud, T=T)
    h = binding.glr_forward(y.view(total, H * D), d["gate"], cu_seqlens=cud, T=T)
    g1 = binding.glr_backward(d["gate"], h, dh.to(DEV), cu_seqlens=cud, T=T)
    g2 = binding.backward(q, k, d["v"], d["la"], d["lam"], g1["x"].view(total, H, D), cu_seqlens=cud, T=T)
    g3 = binding.qk_norm_rope_backward(d["xq"], d["xk"], g2["q"], g2["k"], **how)

    ref = {n: t.double().requires_grad_(True) for n, t in p.items()}
    ys, hs = [], []
    for b, n in enumerate(LENGTHS):
        s = slice(int(cu[b]), int(cu[b + 1]))
        yb, hb = _stack({m: t if m == "w" else t[s] for m, t in ref.items()}, n, freq)
        ys.append(yb)
        hs.append(hb)
    want = torch.cat(hs)
    names = list(ref)
    grads = dict(zip(names, torch.autograd.grad(want, [ref[n] for n in names], dh.double())))
    _near(y, torch.cat(ys).detach(), "attention")
    _near(h, want.detach(), "stack")
    got = dict(xq=g3["q"], xk=g3["k"], v=g2["v"], la=g2["log_a"], lam=g2["lam"], gate=g1["log_a"], w=g3["wq"] + g3["wk"])
    for n in names:
        _near(got[n], grads[n], "gradient of " + n)
    assert binding.device_status(clear=True) == 0


def test_prompt_and_steps():
    """Prompts of 21 and 40 tokens, then 9 tokens for each: outputs of both layers as for the whole."""
    prompts, K = [21, 40], 9
    B, T = 2, max(prompts) + K
    L = binding.num_levels(T)
    full = [n + K for n in prompts]
    p = _inputs(sum(full), L, 2)
    at = torch.tensor([0] + full).cumsum(0).tolist()
    freq = (100.0 ** (-2 * torch.arange(8).double() / 16)).float()
    ref = [_stack({m: t.double() if m == "w" else t[at[b]:at[b + 1]].double() for m, t in p.items()}, full[b], freq)
           for b in range(B)]
    d = {n: t.to(DEV) for n, t in p.items()}
    fd = freq.to(DEV)

    def prep(rows, pos):
        return binding.qk_norm_rope(d["xq"][rows], d["xk"][rows], wq=d["w"], wk=d["w"], pos=pos, inv_freq=fd, heads=H)

    keep = torch.cat([torch.arange(at[b], at[b] + n) for b, n in enumerate(prompts)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in prompts]).int().to(DEV)
    cu = torch.tensor([0] + prompts).cumsum(0).int().to(DEV)
    q, k = prep(keep, pos)
    v, la, lam, gate = (d[n][keep].contiguous() for n in ("v", "la", "lam", "gate"))
    Lp, Tp = binding.num_levels(max(prompts)), max(prompts)
    y = binding.forward(q, k, v, la, lam[..., :Lp].contiguous(), cu_seqlens=cu, T=Tp)
    states = torch.empty(binding.decode_state_bytes(B, H, L, D, D) // 4, device=DEV)
    binding.prefill_state(k, v, la, states, B, H, Tp, L, D, D, cu_seqlens=cu)
    carried = torch.empty((B, H * D), device=DEV)
    h = binding.glr_forward(y.view(-1, H * D), gate, h_last=carried, cu_seqlens=cu, T=Tp)
    _near(h, torch.cat([ref[b][1][:n] for b, n in enumerate(prompts)]), "prompts")
    got, out = torch.empty((K, B, H * D), device=DEV), torch.empty((B, H, D), device=DEV)
    for i in range(K):
        rows = torch.tensor([at[b] + n + i for b, n in enumerate(prompts)], device=DEV)
        pos = torch.tensor([n + i for n in prompts], dtype=torch.int32, device=DEV)
        q, k = prep(rows, pos)
        binding.decode_step(q, k, d["v"][rows].contiguous(), d["la"][rows].contiguous(), d["lam"][rows].contiguous(),
                            pos, states, out, B, H, L, D, D)
        got[i] = binding.glr_forward(out.view(B, 1, H * D), d["gate"][rows].view(B, 1, H * D), h0=carried,
                                     h_last=carried)[:, 0]
    for b, n in enumerate(prompts):
        _near(got[:, b], ref[b][1][n:], "steps")
    assert binding.device_status(clear=True) == 0
