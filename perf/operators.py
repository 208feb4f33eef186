"""Measured cases of the decayed linear attention and rotary position operators.

Each case runs one operator once. `run` makes the calls a user makes of the package where `own` is
true, and computes the same in elementary torch operations, in 32 bits, where it is false.

  attend   out_t = S_t^T q_t with S_t = lambda_h S_{t-1} + k_t v_t^T: prompts, state in and out
  grad     its gradients dq, dk, dv (and of the incoming state)
  step     one token per head against the carried state, which is updated in place
  rotary   rotary positions of q and k, with the d^-1/4 pre-scale of both
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 128


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt: latency counts
        dict(name="attend-short", op="attend", B=1, H=8, L=256, d=64, dtype="bf16", rows="bhld", ragged=False,
             state=False),
        # a training or prefill batch at the package's long-sequence shape
        dict(name="attend-batch", op="attend", B=4, H=8, L=4096, d=64, dtype="bf16", rows="bhld", ragged=False,
             state=False),
        # one very long document
        dict(name="attend-long", op="attend", B=1, H=16, L=65536, d=64, dtype="bf16", rows="bhld", ragged=False,
             state=True),
        # continued prompts of different lengths, token-major projections, wide heads
        dict(name="attend-ragged", op="attend", B=6, H=16, L=1999, d=128, dtype="bf16", rows="blhd", ragged=True,
             state=True),
        # the accuracy path
        dict(name="attend-f32", op="attend", B=2, H=8, L=1023, d=64, dtype="f32", rows="bhld", ragged=False,
             state=True),
        # a training step's gradients
        dict(name="grad-batch", op="grad", B=4, H=8, L=4096, d=64, dtype="bf16", rows="bhld", ragged=False,
             state=False),
        # gradients through carried states, padded batch, wide heads
        dict(name="grad-ragged", op="grad", B=2, H=12, L=2049, d=128, dtype="bf16", rows="blhd", ragged=True,
             state=True),
        # a small fp32 gradient
        dict(name="grad-f32", op="grad", B=1, H=8, L=777, d=64, dtype="f32", rows="bhld", ragged=False, state=False),
        # one sequence served token by token
        dict(name="step-one", op="step", B=1, H=8, d=64, dtype="bf16"),
        # a full serving batch
        dict(name="step-many", op="step", B=512, H=8, d=64, dtype="bf16"),
        # q and k of a training batch, positions scaled for a longer context
        dict(name="rotary-batch", op="rotary", B=4, H=8, Hk=8, L=4096, d=64, rot=64, dtype="bf16", rows="bhld",
             interleaved=False, inverse=False, far=False),
        # one token of each served sequence, far positions, part of the head
        dict(name="rotary-step", op="rotary", B=64, H=16, Hk=4, L=1, d=128, rot=64, dtype="bf16", rows="blhd",
             interleaved=True, inverse=False, far=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "grad", "grad", "step", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128, _log_int(rng, 1, 128)])
    H = rng.choice([1, 2, 4, 8, 8, 12, 16])
    if op == "step":
        top = max(1, 4096 * 64 * 64 // (H * d * d))
        return dict(op=op, B=_log_int(rng, 1, min(1024, top)), H=H, d=d, dtype=dtype)
    cap = {"attend": 16 * 65536 * 64, "grad": 4 * 8 * 4096 * 64, "rotary": 4 * 8 * 4096 * 64}[op]
    if dtype == "f32":
        cap //= 4
    B = _log_int(rng, 1, 16)
    while B * H * d * 16 > cap:
        B = max(1, B // 2)
        H = max(1, H // 2)
    L = _log_int(rng, 1, max(1, min(65536, cap // (B * H * d))))
    rows = rng.choice(["bhld", "blhd"])
    if op == "rotary":
        rot = 2 * rng.randint(1, d // 2) if rng.random() < 0.5 and d > 1 else 2 * (d // 2)
        return dict(op=op, B=B, H=H, Hk=rng.choice([h for h in (1, 2, 4, 8, H) if h <= H]), L=L, d=max(2, d),
                    rot=max(2, rot), dtype=dtype, rows=rows, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, far=rng.random() < 0.5)
    return dict(op=op, B=B, H=H, L=L, d=d, dtype=dtype, rows=rows, ragged=rng.random() < 0.4,
                state=rng.random() < 0.6)


def _lengths(case):
    """Valid tokens per sequence: from L down to about a third of it in a ragged batch."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    return [max(1, L - (b * (2 * L // 3)) // max(1, B - 1)) for b in range(B)]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, H, d = case["B"], case["H"], case["d"]
    if case["op"] == "step":
        return {"bytes": 8 * B * H * d * d + 4 * B * H * d * es + 4 * H, "flops": 5 * B * H * d * d}
    if case["op"] == "rotary":
        heads = (H + case["Hk"]) * B * case["L"]
        return {"bytes": 2 * heads * d * es + 4 * B * case["L"] + 4 * case["rot"], "flops": 4 * heads * case["rot"]}
    n = sum(_lengths(case)) * H
    state = 8 * B * H * d * d if case["state"] else 0
    if case["op"] == "attend":
        return {"bytes": 4 * n * d * es + state, "flops": 4 * n * d * d}
    return {"bytes": 7 * n * d * es + state + state // 2, "flops": 10 * n * d * d}


# ------------------------------------------------------------------------------------ inputs
def _rows(case, heads, g, scale, dtype):
    """A [B, heads, L, d] tensor, stored head-major or token-major."""
    B, L, d = case["B"], case["L"], case["d"]
    if case["rows"] == "bhld":
        return (torch.randn(B, heads, L, d, generator=g, device="cuda") * scale).to(dtype)
    return (torch.randn(B, L, heads, d, generator=g, device="cuda") * scale).to(dtype).transpose(1, 2)


def _zeros_like(x):
    return torch.empty_like(x).zero_()


def _slopes(H, g):
    """log lambda_h: half-lives from about a token to about a thousand, jittered by the seed."""
    e = 1.0 + 9.0 * torch.arange(H, device="cuda", dtype=torch.float32) / max(1, H - 1)
    return -torch.exp2(-e) * (1.0 + 0.2 * torch.rand(H, generator=g, device="cuda"))


def _frequencies(rot, scaled):
    """Angle per position of each pair, in 64 bits; scaled: the slow half is interpolated by 4."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / rot)
    if scaled:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 4.0)
    return f


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DT[case["dtype"]]
    B, H, d = case["B"], case["H"], case["d"]
    op = case["op"]
    st = dict(op=op)
    if op == "rotary":
        st["q"] = _rows(case, H, g, 1.0, dtype)
        st["k"] = _rows(case, case["Hk"], g, 1.0, dtype)
        start = torch.randint(0, 1000000 if case["far"] else 64, (B, 1), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(case["L"], device="cuda")).to(torch.int32).contiguous()
        st["freq"] = _frequencies(case["rot"], case["far"])
        st["scale"] = d ** -0.25
        st["rot_scale"] = 0.1 * math.log(4.0) + 1.0 if case["far"] else 1.0
        st["interleaved"], st["inverse"] = case["interleaved"], case["inverse"]
        return st
    st["g"] = _slopes(H, g)
    s = d ** -0.25
    if op == "step":
        st["q"], st["k"], st["v"] = ((torch.randn(B, H, d, generator=g, device="cuda") * x).to(dtype)
                                     for x in (s, s, 1.0))
        st["S"] = torch.randn(B, H, d, d, generator=g, device="cuda")
        return st
    st["q"], st["k"], st["v"] = _rows(case, H, g, s, dtype), _rows(case, H, g, s, dtype), _rows(case, H, g, 1.0, dtype)
    st["S"] = torch.randn(B, H, d, d, generator=g, device="cuda") if case["state"] else None
    st["lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None)
    if op == "attend":
        st["out"] = _zeros_like(st["q"])
    else:
        st["do"] = _rows(case, H, g, 1.0, dtype)
        st["dS"] = torch.randn(B, H, d, d, generator=g, device="cuda") if case["state"] else None
        st["dq"], st["dk"], st["dv"] = _zeros_like(st["q"]), _zeros_like(st["k"]), _zeros_like(st["v"])
    return st


# ------------------------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return {"attend": _attend, "grad": _grad, "step": _step, "rotary": _rotary}[st["op"]](st)


def _run_own(st):
    import linear_kernelized_attention_b200 as F
    op = st["op"]
    if op == "attend":
        return F.favor_decay_attention(st["q"], st["k"], st["v"], st["g"], state=st["S"], lengths=st["lengths"],
                                       out=st["out"], return_state=True)
    if op == "grad":
        return F.favor_decay_attention_backward(st["q"], st["k"], st["v"], st["g"], st["do"], state=st["S"],
                                                dstate=st["dS"], lengths=st["lengths"], dq=st["dq"], dk=st["dk"],
                                                dv=st["dv"])
    if op == "step":
        return F.favor_decay_step(st["q"], st["k"], st["v"], st["g"], st["S"]), st["S"]
    return F.favor_rotary(st["q"], st["k"], st["freq"], positions=st["positions"], interleaved=st["interleaved"],
                          inverse=st["inverse"], scale=st["scale"], rot_scale=st["rot_scale"])


# ------------------------------------------------------------------------------------ plain forms
def _pow(g, n):
    """lambda^n in 32 bits, the exponent in 64: g [H], n any shape -> [H, ...]."""
    gv = g.double().view(-1, *([1] * n.dim()))
    e = torch.where(n == 0, torch.zeros_like(gv * n), gv * n)
    return torch.exp(e).float()


def _scan(a, b, c, g, reverse):
    """sum over j <= i (j >= i) of lambda^|i-j| (a_i . b_j) c_j, in chunks; a, b, c [B, H, L, d] fp32."""
    B, H, L, d = a.shape
    n = -(-L // _CHUNK)
    C = _CHUNK if n > 1 else L
    pad = n * C - L
    if pad:
        a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (a, b, c))
    a, b, c = (x.reshape(B, H, n, C, d) for x in (a, b, c))
    i = torch.arange(C, device=a.device)
    gap = (i[:, None] - i[None, :]) * (-1 if reverse else 1)
    D = torch.where(gap >= 0, _pow(g, gap.clamp(min=0)), torch.zeros((), device=a.device))
    out = ((a @ b.transpose(-1, -2)) * D[:, None]) @ c
    if n > 1:
        to_end = _pow(g, i if reverse else C - 1 - i)[:, None, :, None]
        U = (b * to_end).transpose(-1, -2) @ c
        lc = _pow(g, torch.tensor(C, device=a.device)).view(H, 1, 1)
        S, X = torch.zeros_like(U[:, :, 0]), torch.empty_like(U)
        for t in (reversed(range(n)) if reverse else range(n)):
            X[:, :, t] = S
            S = S * lc + U[:, :, t]
        out = out + (a * _pow(g, C - i if reverse else i + 1)[:, None, :, None]) @ X
    return out.reshape(B, H, n * C, d)[:, :, :L]


def _valid(st, L):
    """[B, 1, L, 1] truth values of the tokens inside each sequence, and the lengths [B]."""
    B = st["q"].shape[0]
    n = st["lengths"].long() if st["lengths"] is not None else torch.full((B,), L, device="cuda")
    t = torch.arange(L, device="cuda")
    return (t[None, :] < n[:, None])[:, None, :, None], n


def _masked(x, ok):
    return torch.where(ok, x.float(), torch.zeros((), device=x.device))


def _weights(g, n, L, shift):
    """lambda^(len - 1 + shift - t) for the tokens inside, [B, H, L, 1]."""
    e = (n[:, None] - 1 + shift - torch.arange(L, device=g.device)[None, :]).clamp(min=0)
    return _pow(g, e).transpose(0, 1)[..., None]


def _attend(st):
    L = st["q"].shape[2]
    ok, n = _valid(st, L)
    q, k, v = (_masked(st[x], ok) for x in ("q", "k", "v"))
    g, S = st["g"], st["S"]
    out = _scan(q, k, v, g, False)
    new = (k * _weights(g, n, L, 0)).transpose(-1, -2) @ v
    if S is not None:
        t = torch.arange(L, device="cuda")
        out = out + _pow(g, t + 1)[None, :, :, None] * (q @ S)
        new = new + _pow(g, n).transpose(0, 1)[..., None, None] * S
    return torch.where(ok, out, torch.zeros((), device="cuda")).to(st["q"].dtype), new


def _grad(st):
    L = st["q"].shape[2]
    ok, n = _valid(st, L)
    q, k, v, do = (_masked(st[x], ok) for x in ("q", "k", "v", "do"))
    g, S, dS = st["g"], st["S"], st["dS"]
    dq = _scan(do, v, k, g, False)
    dk = _scan(v, do, q, g, True)
    dv = _scan(k, q, do, g, True)
    dnew = None
    if S is not None:
        t = torch.arange(L, device="cuda")
        dq = dq + _pow(g, t + 1)[None, :, :, None] * (do @ S.transpose(-1, -2))
        w = _weights(g, n, L, 0)
        dk = dk + w * (v @ dS.transpose(-1, -2))
        dv = dv + w * (k @ dS)
        dnew = (q * _pow(g, t + 1)[None, :, :, None]).transpose(-1, -2) @ do
        dnew = dnew + _pow(g, n).transpose(0, 1)[..., None, None] * dS
    dt = st["q"].dtype
    zero = torch.zeros((), device="cuda")
    dq, dk, dv = (torch.where(ok, x, zero).to(dt) for x in (dq, dk, dv))
    return (dq, dk, dv, dnew) if dnew is not None else (dq, dk, dv)


def _step(st):
    q, k, v = (st[x].float() for x in ("q", "k", "v"))
    S = st["S"]
    S.mul_(torch.exp(st["g"]).view(1, -1, 1, 1)).add_(k[..., :, None] * v[..., None, :])
    return (q[..., None, :] @ S)[..., 0, :].to(st["q"].dtype), S


def _rotary(st):
    f = st["freq"]
    angle = st["positions"].double()[:, None, :, None] * f
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    if st["inverse"]:
        s = -s
    h = f.numel()
    c, s = c * st["rot_scale"] * st["scale"], s * st["rot_scale"] * st["scale"]

    def turn(x):
        y = x.float()
        r, rest = y[..., :2 * h], y[..., 2 * h:] * st["scale"]
        if st["interleaved"]:
            x1, x2 = r[..., 0::2], r[..., 1::2]
            r = torch.stack((x1 * c - x2 * s, x1 * s + x2 * c), dim=-1).flatten(-2)
        else:
            x1, x2 = r[..., :h], r[..., h:]
            r = torch.cat((x1 * c - x2 * s, x1 * s + x2 * c), dim=-1)
        return torch.cat((r, rest), dim=-1).to(x.dtype)

    return turn(st["q"]), turn(st["k"])


# ------------------------------------------------------------------------------------ 64 bits
def _quadratic(a, b, c, g, n, later):
    """Rows sum_j lambda^|i-j| (a_i . b_j) c_j over the sequence's n tokens, j <= i or (later) j >= i:
    one head, float64, the full matrix in row blocks."""
    out = torch.zeros_like(a)
    pos = torch.arange(n, device=a.device, dtype=torch.float64)
    for i0 in range(0, n, 2048):
        i1 = min(n, i0 + 2048)
        j0, j1 = (i0, n) if later else (0, i1)
        gap = pos[i0:i1, None] - pos[None, j0:j1]
        if later:
            gap = -gap
        m = torch.exp(g * gap.clamp_(min=0)).masked_fill_(
            (pos[None, j0:j1] < pos[i0:i1, None]) if later else (pos[None, j0:j1] > pos[i0:i1, None]), 0.0)
        out[i0:i1] = (m * (a[i0:i1] @ b[j0:j1].T)) @ c[j0:j1]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(st)
    g = st["g"].double()
    if case["op"] == "step":
        q, k, v = (st[x].double() for x in ("q", "k", "v"))
        S = g.exp()[None, :, None, None] * st["S"].double() + torch.einsum("bhm,bhn->bhmn", k, v)
        return torch.einsum("bhm,bhmn->bhn", q, S), S
    names = ("q", "k", "v") + (("do",) if case["op"] == "grad" else ())
    x = {name: st[name].double() for name in names}
    B, H, L, d = x["q"].shape
    outs = [torch.zeros(B, H, L, d, dtype=torch.float64, device="cuda") for _ in range(1 if case["op"] == "attend" else 3)]
    states = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        t = torch.arange(n, device="cuda", dtype=torch.float64)
        for h in range(H):
            gh = g[h]
            up, down = torch.exp(gh * (t + 1))[:, None], torch.exp(gh * (n - 1 - t))[:, None]
            q, k, v = (x[name][b, h] for name in ("q", "k", "v"))
            S = st["S"][b, h].double() if st["S"] is not None else None
            if case["op"] == "attend":
                o = _quadratic(q, k, v, gh, n, False)
                states[b, h] = torch.einsum("tm,tn->mn", down * k[:n], v[:n])
                if S is not None:
                    o[:n] += up * (q[:n] @ S)
                    states[b, h] += torch.exp(gh * n) * S
                outs[0][b, h] = o
                continue
            do = x["do"][b, h]
            dq = _quadratic(do, v, k, gh, n, False)
            dk = _quadratic(v, do, q, gh, n, True)
            dv = _quadratic(k, q, do, gh, n, True)
            if S is not None:
                dS = st["dS"][b, h].double()
                dq[:n] += up * (do[:n] @ S.T)
                dk[:n] += down * (v[:n] @ dS.T)
                dv[:n] += down * (k[:n] @ dS)
                states[b, h] = torch.einsum("tm,tn->mn", up * q[:n], do[:n]) + torch.exp(gh * n) * dS
            for dst, val in zip(outs, (dq, dk, dv)):
                dst[b, h] = val
    if case["op"] == "attend" or case["state"]:
        return (*outs, states)
    return tuple(outs)


def _exact_rotary(st):
    h = st["freq"].numel()
    a = st["positions"].double()[:, None, :, None] * st["freq"] * (-1.0 if st["inverse"] else 1.0)
    z = torch.polar(torch.full_like(a, st["rot_scale"]), a)

    def turn(x):
        y = x.double()
        lo, hi = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if st["interleaved"] else (y[..., :h], y[..., h:2 * h])
        w = torch.complex(lo.contiguous(), hi.contiguous()) * z
        r = y.clone()
        if st["interleaved"]:
            r[..., 0:2 * h:2], r[..., 1:2 * h:2] = w.real, w.imag
        else:
            r[..., :h], r[..., h:2 * h] = w.real, w.imag
        return r * st["scale"]

    return turn(st["q"]), turn(st["k"])
