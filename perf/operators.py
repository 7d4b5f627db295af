"""The layer operators around log-linear attention, as measured cases.

Three operators, each in the form a user's program calls it:

  qk     norms of queries and keys for each head, with the position rotation in the same pass,
         forward and backward: what turns a projection's output into the unit-norm q, k that the
         attention forward takes, and the gradients that its backward writes into those of the
         projection;
  glr    the gated linear recurrence h_t = exp(log_a_t) h_{t-1} + x_t over long sequences, with
         carried states, forward and backward, and its single-token step;
  q8     the decoding state held in 8 bits: written by a prompt (``prefill``) and by a decoding
         step (``decode``), and read back.

``run`` computes them from elementary torch operations in 32 bits (64 where said) where ``own``
is false, and through the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one decoding step of 64 sequences: 32 heads of 64 out of a fused projection, whole head rotated
        dict(name="qk_step_b64_h32_d64", op="qk_fwd", N=64, Gq=32, Gk=32, H=32, d=64, rot=64, layout="half",
             norm="l2", weights=False, dtype="bf16", max_pos=8192, fused=True),
        # a 65536-token prompt at head size 128: 4 key groups for 16 heads, a quarter of the head rotated in
        # interleaved pairs, learned weights
        dict(name="qk_t64k_h16_d128_gqa", op="qk_fwd", N=65536, Gq=16, Gk=4, H=16, d=128, rot=32,
             layout="interleaved", norm="rms", weights=True, dtype="bf16", max_pos=65536, fused=True),
        # the training batch of 4 x 8192 tokens and 32 heads, its gradients
        dict(name="qk_bwd_4x8k_h32_d64", op="qk_bwd", N=32768, Gq=32, Gk=32, H=32, d=64, rot=64, layout="half",
             norm="l2", weights=False, dtype="bf16", max_pos=8192, fused=True),
        # a ragged packed batch in fp32 with shared key groups and weight gradients
        dict(name="qk_bwd_n2999_h16_d32_f32", op="qk_bwd", N=2999, Gq=16, Gk=2, H=16, d=32, rot=16,
             layout="interleaved", norm="rms", weights=True, dtype="f32", max_pos=16384, fused=False),
        # one token for each of 64 sequences, state carried over from the last
        dict(name="glr_step_b64_d2048", op="glr_fwd", B=64, T=1, D=2048, packed=False, state=True, dtype="bf16",
             mu=-2.0),
        # one sequence of 65536 tokens, long memory
        dict(name="glr_t64k_d2048", op="glr_fwd", B=1, T=65536, D=2048, packed=False, state=True, dtype="bf16",
             mu=-3.0),
        # gradients of a batch of two 2048-token sequences, 16 heads of 64
        dict(name="glr_bwd_2x2k_d1024", op="glr_bwd", B=2, T=2048, D=1024, packed=False, state=False, dtype="bf16",
             mu=-2.0),
        # gradients of eight packed sequences of 1024 to 16384 tokens
        dict(name="glr_bwd_varlen8_d1024", op="glr_bwd", B=8, T=16384, D=1024, packed=True, state=True, dtype="bf16",
             mu=-2.0),
        # one sequence far into a 65536-token context: few heads, where latency counts
        dict(name="q8_step_b1_h16_d128", op="decode", B=1, H=16, L=17, dk=128, dv=128, dtype="bf16", mu=-3.0),
        # a serving batch of 64 sequences at positions over [0, 8192)
        dict(name="q8_step_b64_h32_d64", op="decode", B=64, H=32, L=14, dk=64, dv=64, dtype="bf16", mu=-2.0),
        # two prompts of 2047 tokens: a bucket at every level
        dict(name="q8_prompt_2x2047_h16_d64", op="prefill", B=2, H=16, T=2047, L=14, dk=64, dv=64, packed=False,
             dtype="bf16", mu=-2.0),
        # eight packed prompts of 1024 to 16384 tokens
        dict(name="q8_prompt_varlen8_h16_d64", op="prefill", B=8, H=16, T=16384, L=16, dk=64, dv=64, packed=True,
             dtype="bf16", mu=-2.0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "glr_fwd", "glr_bwd", "decode", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk_fwd", "qk_bwd"):
        d, H = rng.choice([32, 64, 128]), rng.choice([1, 2, 4, 6, 8, 16, 32])
        groups = [g for g in range(1, H + 1) if H % g == 0]
        N = _log(rng, 1, max(1, (1 << 25) // (H * d)))
        return dict(op=op, N=N, Gq=rng.choice([H, rng.choice(groups)]), Gk=rng.choice(groups), H=H, d=d,
                    rot=rng.choice([0, 8, d // 2, d, d]), layout=rng.choice(["half", "interleaved"]),
                    norm=rng.choice(["l2", "rms"]), weights=rng.random() < 0.5, dtype=dtype,
                    max_pos=_log(rng, 1, 1 << 20), fused=rng.random() < 0.5)
    if op in ("glr_fwd", "glr_bwd"):
        D = _log(rng, 1, 4096)
        T = _log(rng, 1, min(65536, (1 << 26) // D))
        B = _log(rng, 1, max(1, min(64, (1 << 25) // (D * T))))
        return dict(op=op, B=B, T=T, D=D, packed=rng.random() < 0.4, state=rng.random() < 0.5, dtype=dtype,
                    mu=rng.choice([-2.0, -3.0]))
    dk, dv = rng.choice([(32, 32), (64, 64), (64, 64), (128, 128), (64, 128), (128, 32)])
    H, L = rng.choice([1, 3, 8, 16, 32]), rng.randint(2, 17)
    if op == "decode":
        B = _log(rng, 1, max(1, min(64, (1 << 26) // (H * (L - 1) * dk * dv))))
        return dict(op=op, B=B, H=H, L=L, dk=dk, dv=dv, dtype=dtype, mu=-2.0)
    T = _log(rng, 1, min((1 << (L - 1)) - 1, 16384))
    B = _log(rng, 1, max(1, min(16, (1 << 18) // (H * T))))
    return dict(op=op, B=B, H=H, T=T, L=L, dk=dk, dv=dv, packed=rng.random() < 0.4, dtype=dtype, mu=-2.0)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """Sequence lengths of a packed batch, the same for every seed: 1/16 of the bound to the bound, the last one at the
    bound."""
    g = torch.Generator()
    g.manual_seed(7919 + case["B"] + 64 * case["T"])
    n = torch.randint(max(1, case["T"] // 16), case["T"] + 1, (case["B"],), generator=g)
    n[-1] = case["T"]
    return n.tolist()


def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _gates(shape, mu, g):
    """log a = -exp(N(mu, 0.5))"""
    return -torch.exp(mu + 0.5 * torch.randn(shape, generator=g, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    op = case["op"]
    if op in ("qk_fwd", "qk_bwd"):
        N, Gq, Gk, H, d, rot = (case[n] for n in ("N", "Gq", "Gk", "H", "d", "rot"))
        if case["fused"]:  # one projection's output: q, k and v beside one another in each row
            row = normal(N, (Gq + Gk + H) * d)
            s["q"] = row[:, :Gq * d].unflatten(1, (Gq, d))
            s["k"] = row[:, Gq * d:(Gq + Gk) * d].unflatten(1, (Gk, d))
        else:
            s["q"], s["k"] = normal(N, Gq, d), normal(N, Gk, d)
        s["wq"] = 1 + 0.1 * normal(d, dtype=F32) if case["weights"] else None
        s["wk"] = 1 + 0.1 * normal(d, dtype=F32) if case["weights"] else None
        s["pos"] = torch.randint(0, case["max_pos"], (N,), generator=g, device=DEV).int() if rot else None
        i = torch.arange(rot // 2, dtype=F64, device=DEV)
        s["inv_freq"] = (10000.0 ** (-2 * i / rot)).float() if rot else None
        s["eps"] = 1e-6
        if op == "qk_bwd":
            s["dqo"], s["dko"] = normal(N, H, d, dtype=F32), normal(N, H, d, dtype=F32)
        return s
    if op in ("glr_fwd", "glr_bwd"):
        B, T, D = case["B"], case["T"], case["D"]
        lengths = _lengths(case) if case["packed"] else None
        lead = (sum(lengths),) if lengths else (B, T)
        s["lengths"] = lengths or [T] * B
        s["cu"] = _cu(lengths) if lengths else None
        s["x"] = normal(*lead, D)
        s["log_a"] = _gates(lead + (D,), case["mu"], g)
        s["h0"] = normal(B, D, dtype=F32) if case["state"] else None
        first = torch.zeros(lead, dtype=torch.bool, device=DEV)  # the sequences' first rows
        first.view(-1)[_starts(s)] = True
        s["first"] = first.view(-1, 1)
        if op == "glr_bwd":
            s["h"] = _scan(s).view(lead + (D,))
            s["dh"] = normal(*lead, D, dtype=F32)
            s["dh_last"] = normal(B, D, dtype=F32) if case["state"] else None
        return s
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    nslot, sizes = L - 1, _state_sizes(B, H, L, dk, dv)
    s["state"] = torch.zeros(sum(sizes), dtype=torch.uint8, device=DEV)
    s["codes"], s["gate"], s["exps"] = _state_views(s["state"], B, H, L, dk, dv)
    if op == "prefill":
        lengths = _lengths(case) if case["packed"] else None
        lead = (sum(lengths),) if lengths else (B, case["T"])
        s["lengths"] = lengths or [case["T"]] * B
        s["cu"] = _cu(lengths) if lengths else None
        k = torch.randn(lead + (H, dk), generator=g, device=DEV)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"], s["log_a"] = normal(*lead, H, dv), _gates(lead + (H,), case["mu"], g)
        return s
    pos = torch.randint(0, (1 << nslot) - 1 if nslot > 1 else 1, (B,), generator=g, device=DEV)
    s["pos"] = pos.int()
    s["m"] = _trailing_ones(pos).int()  # the slot that the step writes
    for n, w in (("q", dk), ("k", dk)):
        x = torch.randn(B, H, w, generator=g, device=DEV)
        s[n] = (x / x.norm(dim=-1, keepdim=True)).to(dt)
    s["v"], s["log_a"] = normal(B, H, dv), _gates((B, H), case["mu"], g)
    s["lam"] = torch.nn.functional.softplus(torch.randn(B, H, L, generator=g, device=DEV))
    for j in range(nslot):  # level states as earlier steps have written them
        c, e = _quantise(0.3 * torch.randn(B, H, dk, dv, generator=g, device=DEV))
        s["codes"][:, :, j], s["exps"][:, :, j] = c, e
    s["gate"].copy_(-3.0 * torch.rand(B, H, 2, nslot, generator=g, device=DEV))
    return s


# ---------------------------------------------------------------- the 8-bit state: its layout and its numbers

def _state_sizes(B, H, L, dk, dv):
    """Bytes of the codes, the pending gates and the block exponents."""
    n = B * H * (L - 1)
    return n * dk * dv, n * 2 * 4, n * dk * (dv // 32)


def _state_views(state, B, H, L, dk, dv):
    a, b, _ = _state_sizes(B, H, L, dk, dv)
    return (state[:a].view(torch.int8).view(B, H, L - 1, dk, dv), state[a:a + b].view(F32).view(B, H, 2, L - 1),
            state[a + b:].view(B, H, L - 1, dk, dv // 32))


def _trailing_ones(n):
    low = (~n) & (n + 1)  # the lowest zero bit
    return torch.log2(low.double()).round().long()


def _quantise(x):
    """Codes in -127..127 and one power of two for 32 adjacent columns: the smallest that holds them (biased by 127;
    0: a block of zeros)."""
    b = x.unflatten(-1, (x.shape[-1] // 32, 32))
    top = b.abs().amax(-1)
    f, e = torch.frexp(top)  # top = f 2^e, f in [1/2, 1)
    e = e.long() - 7 + (f > 127.0 / 128.0).long()
    e = e.clamp(-126, 127)
    c = torch.ldexp(b, -e.unsqueeze(-1).to(b.dtype)).round()
    code = torch.where(top > 0, e + 127, torch.zeros_like(e))
    return c.flatten(-2).to(torch.int8), code.to(torch.uint8)


def _values(codes, exps, dtype=F32):
    scale = torch.where(exps > 0, torch.exp2(exps.to(F64) - 127), 0.0).to(dtype)
    return (codes.unflatten(-1, (codes.shape[-1] // 32, 32)).to(dtype) * scale.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------- the gated recurrence

def _starts(s):
    """The first row of each sequence (none is empty here)."""
    n = torch.tensor(s["lengths"])
    return (n.cumsum(0) - n).to(DEV)


def _ends(s):
    return (torch.tensor(s["lengths"]).cumsum(0) - 1).to(DEV)


def _doubling(a, x, reverse=False):
    """y_t = a_t y_{t-1} + x_t over the rows, by recursive doubling (reverse: y_t = a_t y_{t+1} + x_t).  Takes a and x."""
    d, n = 1, a.shape[0]
    while d < n:
        lo, hi = (slice(d, None), slice(None, -d)) if reverse else (slice(None, -d), slice(d, None))
        x[hi] += a[hi] * x[lo].clone()
        a[hi] *= a[lo].clone()
        d *= 2
    return x


def _scan(s):
    D = s["case"]["D"]
    a = torch.exp(s["log_a"].view(-1, D))
    x = s["x"].view(-1, D).float().clone()
    if s["h0"] is not None:
        r = _starts(s)
        x[r] += a[r] * s["h0"]
    return _doubling(a.masked_fill(s["first"], 0.0), x)


def _glr_backward(s):
    D = s["case"]["D"]
    a, h = torch.exp(s["log_a"].view(-1, D)), s["h"].view(-1, D)
    first, last = _starts(s), _ends(s)
    g = s["dh"].view(-1, D).clone()
    if s["dh_last"] is not None:
        g[last] += s["dh_last"]
    after = torch.zeros_like(a)  # the next row's gate, where it is the same sequence's
    after[:-1] = a.masked_fill(s["first"], 0.0)[1:]
    g = _doubling(after, g, reverse=True)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = s["h0"] if s["h0"] is not None else 0.0
    lead = s["dh"].shape
    out = {"x": g.view(lead), "log_a": (g * a * before).view(lead)}
    if s["h0"] is not None:
        out["h0"] = a[first] * g[first]
    return out


# ---------------------------------------------------------------- norms and rotation of q and k

def _angles(s):
    """Cosine and sine by (token, pair); positions times frequencies in 64 bits."""
    t = s["pos"].double()[:, None] * s["inv_freq"].double()
    return t.cos().float()[:, None], t.sin().float()[:, None]


def _pairs(y, case):
    """The two halves of the rotated pairs, and the rest."""
    r = case["rot"]
    if case["layout"] == "half":
        return y[..., :r // 2], y[..., r // 2:r], y[..., r:]
    return y[..., 0:r:2], y[..., 1:r:2], y[..., r:]


def _joined(a, b, rest, case):
    if case["layout"] == "half":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _rotated(y, s, back=False):
    case = s["case"]
    if not case["rot"]:
        return y
    c, n = _angles(s)
    n = -n if back else n
    a, b, rest = _pairs(y, case)
    return _joined(a * c - b * n, a * n + b * c, rest, case)


def _inverse_norm(x, s):
    sq = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((sq / x.shape[-1] if s["case"]["norm"] == "rms" else sq) + s["eps"])


def _qk_one(x, w, s):
    y = x.float()
    y = y * _inverse_norm(y, s)
    y = _rotated(y * w if w is not None else y, s)
    return y.repeat_interleave(s["case"]["H"] // x.shape[1], 1).to(x.dtype)


def _qk_one_backward(x, w, dy, s):
    G, d = x.shape[1:]
    x = x.float()
    dy = _rotated(dy.unflatten(1, (G, -1)).sum(2), s, back=True)
    inv = _inverse_norm(x, s)
    u = x * inv
    du = dy * w if w is not None else dy
    along = (du * u).sum(-1, keepdim=True)
    dx = inv * (du - u * (along / d if s["case"]["norm"] == "rms" else along))
    return dx, (dy * u).sum((0, 1)) if w is not None else None


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    if op == "qk_fwd":
        return {"q": _qk_one(s["q"], s["wq"], s), "k": _qk_one(s["k"], s["wk"], s)}
    if op == "qk_bwd":
        dq, dwq = _qk_one_backward(s["q"], s["wq"], s["dqo"], s)
        dk, dwk = _qk_one_backward(s["k"], s["wk"], s["dko"], s)
        return {n: t for n, t in (("q", dq), ("k", dk), ("wq", dwq), ("wk", dwk)) if t is not None}
    if op == "glr_fwd":
        h = _scan(s)
        return {"h": h.view(s["x"].shape), "h_last": h[_ends(s)]}
    if op == "glr_bwd":
        return _glr_backward(s)
    return _prefill(s) if op == "prefill" else _decode(s)


def _decode(s):
    n, nslot = s["pos"].long(), s["case"]["L"] - 1
    j = torch.arange(nslot, device=DEV)
    held = ((n[:, None] >> j) & 1).float()[:, None]  # [B, 1, slots]
    merged = held * (j < s["m"][:, None])[:, None].float()
    parity = n & 1
    row = s["gate"][torch.arange(len(n), device=DEV), :, parity]  # [B, H, slots]
    w = torch.exp(row + s["log_a"][..., None])
    S = _values(s["codes"], s["exps"])
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    read = (q[:, :, None, :, None] * S).sum(3)  # [B, H, slots, dv]
    out = ((s["lam"][..., 1:] * w * held)[..., None] * read).sum(2) + (s["lam"][..., :1] * (q * k).sum(-1, True)) * v
    carry = k[..., None] * v[..., None, :] + ((w * merged)[..., None, None] * S).sum(2)
    after = (((n + 1)[:, None] >> j) & 1).bool()[:, None]
    new = torch.where(j == s["m"][:, None, None], torch.zeros_like(row), row + s["log_a"][..., None])
    gate = s["gate"].clone()
    at = (torch.arange(len(n), device=DEV), slice(None), 1 - parity)
    gate[at] = torch.where(after, new, gate[at])
    return {"out": out, "slot": _values(*_quantise(carry), BF16), "gate": gate}


def _prefill(s):
    case = s["case"]
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    k, v = s["k"].view(-1, H, dk), s["v"].view(-1, H, dv)
    la = s["log_a"].view(-1, H).double()
    levels = torch.zeros(B, H, L - 1, dk, dv, dtype=BF16, device=DEV)
    gate = torch.zeros(B, H, 2, L - 1, device=DEV)
    start = 0
    for b, n in enumerate(s["lengths"]):
        after = la[start:start + n].flip(0).cumsum(0).flip(0)  # the log gates from each token to the end
        after = torch.cat([after, torch.zeros_like(after[:1])])
        for j in range(L - 1):
            if not n >> j & 1:
                continue
            lo = n >> (j + 1) << (j + 1)
            hi = lo + (1 << j)
            f = torch.exp(after[lo + 1:hi + 1] - after[hi]).float()
            kk = (k[start + lo:start + hi].float() * f[..., None]).transpose(0, 1)
            S = kk.transpose(1, 2) @ v[start + lo:start + hi].float().transpose(0, 1)
            levels[b, :, j] = _values(*_quantise(S), BF16)
            gate[b, :, :, j] = after[hi].float()[:, None]
        start += n
    return {"levels": levels, "gate": gate}


def _run_own(s):
    from hierarchical_fenwick_state_b200 import binding
    case, op = s["case"], s["case"]["op"]
    if op in ("qk_fwd", "qk_bwd"):
        how = dict(wq=s["wq"], wk=s["wk"], pos=s["pos"], inv_freq=s["inv_freq"], norm=case["norm"], eps=s["eps"],
                   layout=case["layout"])
        if op == "qk_fwd":
            q, k = binding.qk_norm_rope(s["q"], s["k"], heads=case["H"], **how)
            return {"q": q, "k": k}
        return binding.qk_norm_rope_backward(s["q"], s["k"], s["dqo"], s["dko"], **how)
    if op == "glr_fwd":
        last = torch.empty(case["B"], case["D"], device=DEV)
        h = binding.glr_forward(s["x"], s["log_a"], h0=s["h0"], h_last=last, cu_seqlens=s["cu"], T=case["T"])
        return {"h": h, "h_last": last}
    if op == "glr_bwd":
        return binding.glr_backward(s["log_a"], s["h"], s["dh"], h0=s["h0"], dh_last=s["dh_last"],
                                    cu_seqlens=s["cu"], T=case["T"])
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    if op == "prefill":
        binding.prefill_state_q8(s["k"], s["v"], s["log_a"], s["state"], B, H, case["T"], L, dk, dv,
                                 cu_seqlens=s["cu"])
        return {"levels": binding.read_state_q8(s["state"], B, H, L, dk, dv), "gate": s["gate"]}
    out = torch.empty(B, H, dv, device=DEV)
    binding.decode_step_q8(s["q"], s["k"], s["v"], s["log_a"], s["lam"], s["pos"], s["state"], out, B, H, L, dk, dv)
    return {"out": out, "slot": binding.read_state_q8(s["state"], B, H, L, dk, dv, slot=s["m"]), "gate": s["gate"]}


# ---------------------------------------------------------------- the work of one pass

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("qk_fwd", "qk_bwd"):
        N, G, H, d = case["N"], case["Gq"] + case["Gk"], case["H"], case["d"]
        angles = N * 4 if case["rot"] else 0
        if op == "qk_fwd":
            return {"bytes": N * G * d * e + 2 * N * H * d * e + angles, "flops": N * G * d * 8}
        return {"bytes": N * G * d * (e + 4) + 2 * N * H * d * 4 + angles, "flops": N * (G * 16 + 2 * H) * d}
    if op in ("glr_fwd", "glr_bwd"):
        n = sum(_lengths(case)) if case["packed"] else case["B"] * case["T"]
        n, ends = n * case["D"], case["B"] * case["D"] * 4
        if op == "glr_fwd":
            return {"bytes": n * (e + 8) + ends * (2 if case["state"] else 1), "flops": 3 * n}
        return {"bytes": n * 20 + ends * (3 if case["state"] else 0), "flops": 5 * n}
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    slot = dk * dv + dk * dv // 32 + 4
    if op == "decode":  # half of the slots hold a level at a position drawn from all; one is written
        held = (L - 1) / 2
        token = (2 * dk + dv) * e + dv * 4 + (L + 1) * 4
        return {"bytes": B * H * (held * slot + slot + token), "flops": B * H * dk * dv * (2 * held + 4)}
    lengths = _lengths(case) if case["packed"] else [case["T"]] * B
    n, levels = sum(lengths), sum(bin(x).count("1") for x in lengths)
    return {"bytes": n * H * ((dk + dv) * e + 4) + H * levels * slot, "flops": n * H * dk * dv * 2}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("qk_fwd", "qk_bwd"):
        return _exact_qk(s)
    if op in ("glr_fwd", "glr_bwd"):
        return _exact_glr(s)
    return _exact_decode(s) if op == "decode" else _exact_prefill(s)


def _exact_qk(s):
    """The formula with pairs as complex numbers; gradients by differentiating it."""
    case = s["case"]
    H, rot = case["H"], case["rot"]
    back = case["op"] == "qk_bwd"
    out = {}
    for n in ("q", "k"):
        x = s[n].double().requires_grad_(back)
        w = s["w" + n].double().requires_grad_(back) if s["w" + n] is not None else None
        with torch.set_grad_enabled(back):
            size = x.square().mean(-1) if case["norm"] == "rms" else x.square().sum(-1)
            y = x / (size + s["eps"]).sqrt()[..., None]
            y = y * w if w is not None else y
            if rot:
                at = torch.arange(rot, device=DEV)
                at = at.view(2, -1).T if case["layout"] == "half" else at.view(-1, 2)
                turn = torch.polar(torch.ones(1, dtype=F64, device=DEV),
                                   s["pos"].double()[:, None] * s["inv_freq"].double())
                z = torch.view_as_real(torch.view_as_complex(y[..., at].contiguous()) * turn[:, None])
                y = torch.cat([z.flatten(-2)[..., torch.argsort(at.flatten())], y[..., rot:]], -1)
            y = y[:, torch.arange(H, device=DEV) // (H // x.shape[1])]
        if back:
            g = torch.autograd.grad(y, [x] + ([w] if w is not None else []), s["d%so" % n].double())
            out[n] = g[0]
            if w is not None:
                out["w" + n] = g[1]
        else:
            out[n] = y
    return out


def _exact_glr(s):
    """The recurrence token by token."""
    case = s["case"]
    B, D = case["B"], case["D"]
    n = torch.tensor(s["lengths"], device=DEV)
    start = n.cumsum(0) - n
    la = s["log_a"].view(-1, D)
    zero = torch.zeros(B, D, dtype=F64, device=DEV)
    dense = not case["packed"]

    def rows(t):
        return start + t if dense else (start + t)[n > t]

    if case["op"] == "glr_fwd":
        x = s["x"].view(-1, D)
        h = s["h0"].double() if s["h0"] is not None else zero.clone()
        out = torch.empty(x.shape, dtype=F64, device=DEV)
        for t in range(max(s["lengths"])):
            r = rows(t)
            if dense:
                h = torch.addcmul(x[r].double(), la[r].double().exp_(), h)
                out[r] = h
            else:
                live = n > t
                h[live] = la[r].double().exp_() * h[live] + x[r].double()
                out[r] = h[live]
        return {"h": out.view(s["x"].shape), "h_last": h}
    h, dh = s["h"].view(-1, D), s["dh"].view(-1, D)
    c = s["dh_last"].double() if s["dh_last"] is not None else zero.clone()
    dx, dla = (torch.empty(dh.shape, dtype=F64, device=DEV) for _ in range(2))
    for t in reversed(range(max(s["lengths"]))):
        r, live = rows(t), n > t
        g = dh[r].double() + c[live]
        past = h[r - 1].double() if t else (s["h0"][live].double() if s["h0"] is not None else zero[live])
        cc = la[r].double().exp_() * g
        dx[r], dla[r] = g, cc * past
        c[live] = cc
    out = {"x": dx.view(s["dh"].shape), "log_a": dla.view(s["dh"].shape)}
    if s["h0"] is not None:
        out["h0"] = c
    return out


def _exact_round(S):
    """The 8-bit values of S: the block's power of two from its logarithm, whole steps by rounding to even."""
    b = S.unflatten(-1, (S.shape[-1] // 32, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 127.0)).clamp(-126, 127)
    return (torch.round(b / torch.exp2(e)) * torch.exp2(e)).flatten(-2).to(BF16)


def _exact_decode(s):
    """Sequence by sequence and level by level."""
    case = s["case"]
    outs, slots, gates = [], [], s["gate"].double()
    for b, n in enumerate(s["pos"].tolist()):
        q, k, v = (s[i][b].double() for i in ("q", "k", "v"))
        la, lam = s["log_a"][b].double(), s["lam"][b].double()
        carry = torch.einsum("hi,hj->hij", k, v)
        o = lam[:, :1] * torch.einsum("hi,hij->hj", q, carry)
        m = 0
        while n >> m & 1:
            m += 1
        for j in range(case["L"] - 1):
            if n >> j & 1:
                w = torch.exp(s["gate"][b, :, n & 1, j].double() + la)
                S = _values(s["codes"][b, :, j], s["exps"][b, :, j], F64) * w[:, None, None]
                o = o + lam[:, j + 1, None] * torch.einsum("hi,hij->hj", q, S)
                if j < m:
                    carry = carry + S
            if (n + 1) >> j & 1:
                gates[b, :, 1 - (n & 1), j] = 0.0 if j == m else s["gate"][b, :, n & 1, j].double() + la
        outs.append(o)
        slots.append(_exact_round(carry))
    return {"out": torch.stack(outs), "slot": torch.stack(slots), "gate": gates}


def _exact_prefill(s):
    """Every bucket's sum with the decay products taken from its own end."""
    case = s["case"]
    B, H, L, dk, dv = (case[n] for n in ("B", "H", "L", "dk", "dv"))
    k, v, la = s["k"].view(-1, H, dk), s["v"].view(-1, H, dv), s["log_a"].view(-1, H)
    levels = torch.zeros(B, H, L - 1, dk, dv, dtype=BF16, device=DEV)
    gate = torch.zeros(B, H, 2, L - 1, dtype=F64, device=DEV)
    start = 0
    for b, n in enumerate(s["lengths"]):
        done = 0
        for j in reversed(range(L - 1)):
            if n >> j & 1:  # the buckets follow one another, the largest first
                r = slice(start + done, start + done + (1 << j))
                done += 1 << j
                a = la[r].double()
                f = torch.exp(a.sum(0) - a.cumsum(0))
                levels[b, :, j] = _exact_round(torch.einsum("thi,th,thj->hij", k[r].double(), f, v[r].double()))
                gate[b, :, :, j] = la[start + done:start + n].double().sum(0)[:, None]
        start += n
    return {"levels": levels, "gate": gate}
