"""The single-token form of the decayed linear attention, and a run of the operators as they are served: rotary
positions, a prompt, then tokens one by one."""
import numpy as np
import pytest

import decay_cases as C
from oracle import decay_oracle as D

pytestmark = pytest.mark.gpu


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _tol(ref, mag, d, bf16):
    # two roundings in the state's element (its fused updates), one in the product, d in the sum
    return (d + 6) * C.U32 * mag + (C.UBF * np.abs(ref) if bf16 else 0.0) + 1e-37


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (1, 8, 64), (3, 5, 16), (2, 2, 128), (1, 3, 33), (2, 3, 100), (40, 16, 64),
                                   (5, 2, 6), (30, 20, 32), (64, 8, 128)])
def test_step(B, H, d, name):
    import torch
    import linear_kernelized_attention_b200 as F
    dt = _dtype(name)
    (q, qn), (k, kn), (v, vn) = (C.draw((B, H, 1, d), 3 + i, dt) for i in range(3))
    S, Sn = C.draw((B, H, d, d), 9, torch.float32)
    g = C.slopes(H, d)
    ref, refS = D.decay_attention(qn, kn, vn, g, Sn)
    mag, magS = D.decay_attention(abs(qn), abs(kn), abs(vn), g, abs(Sn))
    state = S.cuda()
    got = F.favor_decay_step(*(x.cuda()[:, :, 0] for x in (q, k, v)), torch.from_numpy(g).cuda(), state)
    assert F.favor_sync_status() == 0
    err = np.abs(got.double().cpu().numpy() - ref[:, :, 0])
    assert (err <= _tol(ref, mag, d, name == "bf16")[:, :, 0]).all()
    assert (np.abs(state.double().cpu().numpy() - refS) <= 6 * C.U32 * magS + 1e-37).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_step_reads_fused_projections_in_place(name):
    import torch
    import linear_kernelized_attention_b200 as F
    x = torch.randn(4, 3, 5, 64, device="cuda").to(_dtype(name))  # [B, 3, H, d]
    g = torch.from_numpy(C.slopes(5)).cuda()
    s1, s2 = torch.zeros(2, 4, 5, 64, 64, device="cuda")
    a = F.favor_decay_step(x[:, 0], x[:, 1], x[:, 2], g, s1)
    b = F.favor_decay_step(*(x[:, i].contiguous() for i in range(3)), g, s2)
    assert torch.equal(a, b) and torch.equal(s1, s2)


def test_steps_equal_prompt():
    """300 single tokens in fp32 stay on the float64 recurrence (lambda near 1: its rounding must not grow)."""
    import torch
    import linear_kernelized_attention_b200 as F
    T, H, d = 300, 3, 32
    (q, qn), (k, kn), (v, vn) = (C.draw((1, H, T, d), 13 + i, torch.float32) for i in range(3))
    g = np.array([-1e-4, -0.05, 0.0], dtype=np.float32)
    ref, refS = D.decay_attention(qn, kn, vn, g)
    mag, magS = D.decay_attention(abs(qn), abs(kn), abs(vn), g)
    S = torch.zeros(1, H, d, d, device="cuda")
    gg = torch.from_numpy(g).cuda()
    rows = [F.favor_decay_step(q[:, :, t].cuda(), k[:, :, t].cuda(), v[:, :, t].cuda(), gg, S) for t in range(T)]
    got = torch.stack(rows, 2).double().cpu().numpy()
    # each product is rounded at most twice a step it is carried over
    assert (np.abs(got - ref) <= (d + 4 + 2 * T) * C.U32 * mag).all()
    assert (np.abs(S.double().cpu().numpy() - refS) <= (4 + 2 * T) * C.U32 * magS).all()


def test_step_state_past_32_bit_offsets():
    """More than 2^31 state elements: the last heads as a small call gives them."""
    import torch
    import linear_kernelized_attention_b200 as F
    B, H, d = 1030, 128, 128
    S = torch.zeros(B, H, d, d, device="cuda")
    S[-1].normal_()
    q, k, v = (torch.randn(B, H, d, device="cuda").bfloat16() for _ in range(3))
    g = torch.full((H,), -0.1, device="cuda")
    last = S[-1:].clone()
    out = F.favor_decay_step(q, k, v, g, S)
    ref = F.favor_decay_step(q[-1:], k[-1:], v[-1:], g, last)
    assert torch.equal(S[-1:], last) and torch.equal(out[-1:], ref)


def test_step_in_a_graph_advances_the_state():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v = (torch.randn(2, 4, 64, device="cuda").bfloat16() for _ in range(3))
    g = torch.from_numpy(C.slopes(4)).cuda()
    S, ref = torch.zeros(2, 2, 4, 64, 64, device="cuda")
    out = torch.empty_like(q)
    F.favor_decay_step(q, k, v, g, ref, out=out)
    ref.zero_()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        F.favor_decay_step(q, k, v, g, S, out=out)
    for _ in range(5):
        q.normal_(), k.normal_(), v.normal_()
        gr.replay()
        want = F.favor_decay_step(q, k, v, g, ref)
        assert torch.equal(out, want) and torch.equal(S, ref)


def test_step_refusals():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v = (torch.randn(2, 2, 64, device="cuda") for _ in range(3))
    g = torch.zeros(2, device="cuda")
    S = torch.zeros(2, 2, 64, 64, device="cuda")
    with pytest.raises(TypeError):
        F.favor_decay_step(q, k, v, g, None)
    with pytest.raises(TypeError):
        F.favor_decay_step(q, k, v, g, S.bfloat16())
    with pytest.raises(ValueError):
        F.favor_decay_step(q, k, v, g, S[:1])
    with pytest.raises(ValueError):
        F.favor_decay_step(q, k[:1], v, g, S)
    with pytest.raises(F.FavorError):
        F.favor_decay_step(q, k, v, g, S, out=q)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_rotary_prompt_then_tokens(name):
    """As served: positions turned, a ragged prompt, then tokens against the carried state, each step from the
    kernels' own rounded q and k, against the float64 operators on the same values."""
    import torch
    import linear_kernelized_attention_b200 as F
    B, H, L, d, T = 3, 4, 150, 64, 6
    dt = _dtype(name)
    lens = [150, 129, 64]
    (q, qn), (k, kn), (v, vn) = (C.draw((B, H, L + T, d), 50 + i, dt) for i in range(3))
    g = np.array([-0.5, -0.05, -0.005, 0.0], dtype=np.float32)
    gg = torch.from_numpy(g).cuda()
    freq, rs = F.favor_rotary_frequencies(d, scaling=F.FAVOR_ROTARY_PARTS, factor=4, trained_length=128, device="cuda")
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qr, kr = F.favor_rotary(q[:, :, :L], k[:, :, :L], freq, scale=d ** -0.25, rot_scale=rs)
    S = torch.empty(B, H, d, d, device="cuda")
    out, _ = F.favor_decay_attention(qr, kr, v[:, :, :L], gg, lengths=n, state_out=S)
    f64 = lambda t: t.double().cpu().numpy()
    pos = np.tile(np.arange(L), (B, 1))
    want = D.rotary(f64(q[:, :, :L]), freq.cpu().numpy(), pos, scale=d ** -0.25, rot_scale=rs)
    # relative to the pair: x1 c - x2 s cancels, and a bound on |want| alone is below one fp32 rounding there
    a = C.rotary_allowed(want, f64(q[:, :, :L]), d // 2, False, d ** -0.25, rs, name == "bf16")
    assert (np.abs(f64(qr) - want) <= a).all()
    ref, refS = D.decay_attention(f64(qr), f64(kr), f64(v[:, :, :L]), g, None, lens)
    mag, magS = D.decay_attention(*(abs(f64(x)) for x in (qr, kr, v[:, :, :L])), g, None, lens)
    C.check(out, ref, mag, d, L, name == "bf16", "prompt", name == "f32")
    C.check(S, refS, magS, d, L, False, "prompt state", name == "f32")
    for t in range(T):
        p = (n + t).view(B, 1).contiguous()
        at = lambda x: torch.stack([x[b, :, lens[b] + t] for b in range(B)])[:, :, None]
        q1, k1 = F.favor_rotary(at(q), at(k), freq, positions=p, scale=d ** -0.25, rot_scale=rs)
        before = f64(S)
        row = F.favor_decay_step(q1[:, :, 0], k1[:, :, 0], at(v)[:, :, 0], gg, S)
        o, s = D.decay_attention(f64(q1), f64(k1), f64(at(v)), g, before)
        m, _ = D.decay_attention(*(abs(f64(x)) for x in (q1, k1, at(v))), g, abs(before))
        assert (np.abs(f64(row) - o[:, :, 0]) <= _tol(o, m, d, name == "bf16")[:, :, 0]).all()
    assert F.favor_sync_status() == 0


def test_rotary_feeds_favor_attention_and_its_decode():
    """The rotated, pre-scaled q and k as the FAVOR entry points take them: one causal prompt, and the same rows
    token by token."""
    import torch
    import linear_kernelized_attention_b200 as F
    B, H, L, d, M = 1, 2, 40, 64, 64
    q, k, v = (torch.randn(B, H, L, d, device="cuda").bfloat16() for _ in range(3))
    om = F.favor_orf_omega_seeded(3, H, M, d)
    freq, _ = F.favor_rotary_frequencies(d, device="cuda")
    qr, kr = F.favor_rotary(q, k, freq, scale=d ** -0.25)
    ref = F.favor_attention(qr, kr, v, om, feature_kind=F.FAVOR_RELU, causal=True)
    st = F.favor_decode_new_state(B, H, d, M, F.FAVOR_RELU)
    for t in range(L):
        p = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        q1, k1 = F.favor_rotary(q[:, :, t:t + 1], k[:, :, t:t + 1], freq, positions=p, scale=d ** -0.25)
        assert torch.equal(q1[:, :, 0], qr[:, :, t]) and torch.equal(k1[:, :, 0], kr[:, :, t])
        o = F.favor_decode_step(q1[:, :, 0].contiguous(), k1[:, :, 0].contiguous(), v[:, :, t].contiguous(), om, st,
                                feature_kind=F.FAVOR_RELU)
        e = (o.float() - ref[:, :, t].float()).abs().amax(-1) / ref[:, :, t].float().abs().amax(-1)
        assert float(e.max()) < 2e-2 + 5e-3


def test_stream_handle_of_the_default_stream():
    """Handle 0: the call runs on the default stream itself, behind the work already there."""
    import torch
    import linear_kernelized_attention_b200 as F
    dev = torch.device("cuda", torch.cuda.current_device())
    assert torch.cuda.default_stream().cuda_stream == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        with F._elsewhere(dev, 0):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with F._elsewhere(dev, torch.cuda.current_stream().cuda_stream):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    q, k, v = (torch.randn(2, 4, 64, device="cuda") for _ in range(3))
    g = torch.from_numpy(C.slopes(4)).cuda()
    S, ref = torch.zeros(2, 2, 4, 64, 64, device="cuda")
    want = F.favor_decay_step(q, k, v, g, ref)
    assert torch.equal(F.favor_decay_step(q, k, v, g, S, stream=0), want) and torch.equal(S, ref)


def test_a_call_refused_for_scratch_leaves_no_error_behind():
    """2^22 heads of one token at d = 128 want 64 KB of chunk states each, 275 GB: refused before any launch. The
    next calls, here a token step that updates its state in place, must not report it."""
    import torch
    import linear_kernelized_attention_b200 as F
    B, d = 2 ** 22, 128
    assert F.favor_decay_workspace_bytes(B, 1, 1, d, 0) > torch.cuda.get_device_properties(0).total_memory
    x = torch.zeros(1, 1, 1, d, device="cuda").expand(B, 1, 1, d)
    out = torch.empty(B, 1, 1, d, device="cuda")
    g = torch.full((1,), -0.1, device="cuda")
    with pytest.raises(F.FavorError) as e:
        F.favor_decay_attention(x, x, x, g, out=out)
    assert e.value.code == -6
    q = torch.randn(2, 1, 64, device="cuda")
    S = torch.zeros(2, 1, 64, 64, device="cuda")
    row = F.favor_decay_step(q, q, q, g, S)
    freq, _ = F.favor_rotary_frequencies(64, device="cuda")
    F.favor_rotary(q[:, :, None], None, freq)
    assert torch.allclose(row, q * (q * q).sum(-1, keepdim=True), rtol=1e-5) and F.favor_sync_status() == 0


@pytest.mark.parametrize("d", [64, 33])
def test_step_decay_does_not_drift(d):
    """4096 tokens with k = 0: the state is lambda^4096 of the first one's. lambda rounded to fp32 would shift every
    element to one side by 4096 roundings (the CPU test beside the oracle shows it past the bound)."""
    import torch
    import linear_kernelized_attention_b200 as F
    T, g = 4096, C.coarse_slope()
    S, Sn = C.draw((2, 2, d, d), 5, torch.float32)
    S, gg = S.cuda(), torch.tensor([g, g], device="cuda")
    q, v = (torch.randn(2, 2, d, device="cuda") for _ in range(2))
    k, out = torch.zeros_like(q), torch.empty_like(q)
    F.favor_decay_step(q, k, v, gg, torch.zeros_like(S), out=out)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        for _ in range(64):
            F.favor_decay_step(q, k, v, gg, S, out=out)
    for _ in range(T // 64):
        gr.replay()
    rel = S.double().cpu().numpy() / (Sn * np.exp(g * T)) - 1
    assert abs(rel.mean()) <= C.drift_allowed(T)
    assert np.abs(rel).max() <= T * C.U32
