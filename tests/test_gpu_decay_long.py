"""Decayed linear attention over chains of many chunks: segments of several chunks with a ragged last one, walks and
stand-alone states of dozens of chunks, scans of 64 segments and more, forward and reverse. Decays near 1 and inputs
with a mean, so that a rounding with a sign (tensor cores truncate) adds up instead of cancelling.

Each case names the plan it is for, which the scratch a call takes tells: a change of plan fails here and wants another
size. The reference is decay_cases.scan64 on the GPU in float64; tolerances are those of decay_cases."""
import numpy as np
import pytest

import decay_cases as C

pytestmark = pytest.mark.gpu

# B, H, L, d, type, segments (tensor cores: chunks of 128 tokens; fp32: every chunk of 64 is one)
FORWARD = [
    (1, 16, 15000, 64, "bf16", 9),    # 14 chunks a segment
    (1, 32, 4000, 128, "bf16", 4),    # 8
    (1, 1, 18000, 64, "bf16", 141),   # the scan with 32 loads in flight
    (1, 74, 4200, 64, "bf16", 1),     # 33 chunks a walk, 33 a state
    (1, 128, 2200, 128, "bf16", 1),   # 18
    (1, 2, 8300, 64, "f32", 130),
    (1, 1, 5000, 128, "f32", 79),
]
BACKWARD = [
    (1, 8, 16000, 64, "bf16", 6),     # 21
    (1, 4, 8100, 128, "bf16", 11),    # 6
    (1, 40, 4200, 64, "bf16", 1),     # 33
    (1, 48, 4200, 128, "bf16", 1),    # 33
    (1, 1, 169570, 64, "bf16", 148),  # the reverse scan with 32 loads in flight
    (1, 2, 4300, 64, "f32", 68),
    (1, 1, 4200, 100, "f32", 66),
]
SLOPES = (-1e-5, 0.0, -2e-4, -1e-2, -0.3)


def _inputs(B, H, L, d, name, n):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[name]
    gen = torch.Generator(device="cuda").manual_seed(L + d)
    s = d ** -0.25
    x = [((torch.randn(B, H, L, d, generator=gen, device="cuda") + 0.5) * (s if i < 2 else 1.0)).to(dt) for i in range(n)]
    S = [torch.randn(B, H, d, d, generator=gen, device="cuda") + 0.5 for _ in range(2)]
    g = np.array([SLOPES[h % len(SLOPES)] for h in range(H)], dtype=np.float32)
    return x, S, g, torch.from_numpy(g).cuda()


def _check(got, ref, mag, d, L, what, bf16_out, f32_operands):
    """decay_cases.check, on the GPU."""
    import torch
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    a = (d + 266 + -(-L // 128)) * C.U32 * mag + 1e-37
    if bf16_out:
        a += C.UBF * ref.abs() + (C.UBF + C.UBF ** 2) * mag
    elif not f32_operands:
        a += 2.0 ** -26 * mag
    err = (got - ref).abs()
    assert float((err / a).max()) <= 1.0, (what, float((err / a).max()))
    e, rms = float(err.square().mean().sqrt()), float(ref.square().mean().sqrt())
    lim = 2 * np.sqrt(2 / 3) * C.UBF if bf16_out else 2.0 ** -19
    print(what, "of the allowance", float((err / a).max()), "rms", e / rms)
    assert e <= lim * rms, (what, e / rms)


def _plan(F, B, H, L, d, name, backward, nseg):
    n = 2 if backward else 1
    want = n * B * H * nseg * d * d * 4 if nseg > 1 else 0
    assert F.favor_decay_workspace_bytes(B, H, L, d, int(name == "bf16"), backward) == want


@pytest.mark.parametrize("B,H,L,d,name,nseg", FORWARD)
def test_forward_chains(B, H, L, d, name, nseg):
    import linear_kernelized_attention_b200 as F
    _plan(F, B, H, L, d, name, False, nseg)
    (q, k, v), (S, _), g, gg = _inputs(B, H, L, d, name, 3)
    out, new = F.favor_decay_attention(q, k, v, gg, state=S, return_state=True)
    assert F.favor_sync_status() == 0
    ref = C.forward64(q, k, v, g, S)
    mag = C.forward64(q.abs(), k.abs(), v.abs(), g, S.abs())
    _check(out, ref[0], mag[0], d, L, "out", name == "bf16", name == "f32")
    _check(new, ref[1], mag[1], d, L, "state", False, name == "f32")


@pytest.mark.parametrize("B,H,L,d,name,nseg", BACKWARD)
def test_backward_chains(B, H, L, d, name, nseg):
    import linear_kernelized_attention_b200 as F
    _plan(F, B, H, L, d, name, True, nseg)
    (q, k, v, do), (S, dS), g, gg = _inputs(B, H, L, d, name, 4)
    got = F.favor_decay_attention_backward(q, k, v, gg, do, state=S, dstate=dS)
    assert F.favor_sync_status() == 0
    ref = C.backward64(q, k, v, g, do, S, dS)
    mag = C.backward64(q.abs(), k.abs(), v.abs(), g, do.abs(), S.abs(), dS.abs())
    for what, x, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        _check(x, r, m, d, L, what, name == "bf16", name == "f32")
    _check(got[3], ref[3], mag[3], d, L, "dstate_in", False, name == "f32")


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_chains(d):
    """Sequences that end in the first, a middle and the last segment of a plan of several chunks each."""
    import torch
    import linear_kernelized_attention_b200 as F
    B, H, L = 4, 4, 15000 if d == 64 else 9000
    lens = [L, 300, L // 2 + 77, L - 1]
    (q, k, v, do), (S, dS), g, gg = _inputs(B, H, L, d, "bf16", 4)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert F.favor_decay_workspace_bytes(B, H, L, d) // (B * H * d * d * 4) in range(4, 17)  # segments of 8 chunks and up
    out, new = F.favor_decay_attention(q, k, v, gg, state=S, lengths=n, return_state=True)
    grads = F.favor_decay_attention_backward(q, k, v, gg, do, state=S, dstate=dS, lengths=n)
    assert F.favor_sync_status() == 0
    for b, m in enumerate(lens):
        x = [t[b:b + 1, :, :m] for t in (q, k, v, do)]
        s, ds = S[b:b + 1], dS[b:b + 1]
        ab = [t.abs() for t in x]
        ref, mag = C.forward64(*x[:3], g, s), C.forward64(*ab[:3], g, s.abs())
        _check(out[b:b + 1, :, :m], ref[0], mag[0], d, m, "out", True, False)
        _check(new[b:b + 1], ref[1], mag[1], d, m, "state", False, False)
        ref, mag = C.backward64(*x[:3], g, x[3], s, ds), C.backward64(*ab[:3], g, ab[3], s.abs(), ds.abs())
        for i in range(3):
            _check(grads[i][b:b + 1, :, :m], ref[i], mag[i], d, m, "dq dk dv".split()[i], True, False)
        _check(grads[3][b:b + 1], ref[3], mag[3], d, m, "dstate_in", False, False)
        assert not out[b, :, m:].any() and not any(t[b, :, m:].any() for t in grads[:3])
