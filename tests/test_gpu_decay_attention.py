"""Decayed linear attention on the GPU (prompts and gradients) against the float64 recurrence; tolerances in
decay_cases."""
import numpy as np
import pytest

import decay_cases as C
from oracle import decay_oracle as D

pytestmark = pytest.mark.gpu

# one token, chunk borders (64 and 128 tokens), segments, odd head sizes, every route
SHAPES = [
    (1, 1, 1, 1), (2, 3, 1, 64), (1, 2, 2, 128), (2, 2, 63, 16), (1, 2, 64, 64), (1, 3, 65, 32), (2, 2, 127, 64),
    (1, 2, 128, 128), (1, 2, 129, 64), (1, 3, 200, 48), (1, 2, 257, 100), (2, 2, 300, 17), (1, 2, 385, 80),
    (1, 2, 640, 128), (3, 2, 1023, 64), (1, 1, 2049, 64), (1, 2, 1500, 8),
]


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _inputs(B, H, L, d, dtype, seed, n=3):
    s = d ** -0.25
    return [C.draw((B, H, L, d), seed + i, dtype, s if i < 2 else 1.0) for i in range(n)]


def _state(B, H, d, seed):
    import torch
    return C.draw((B, H, d, d), seed, torch.float32)


def _forward_case(B, H, L, d, name, state, lengths=None, rows="bhld", g=None, seed=0):
    import torch
    import linear_kernelized_attention_b200 as F
    dt = _dtype(name)
    (q, qn), (k, kn), (v, vn) = _inputs(B, H, L, d, dt, seed + 10)
    g = C.slopes(H, seed + L) if g is None else np.asarray(g, dtype=np.float32)
    S, Sn = _state(B, H, d, seed + 90) if state else (None, None)
    ref, refS = D.decay_attention(qn, kn, vn, g, Sn, lengths)
    mag, magS = D.decay_attention(abs(qn), abs(kn), abs(vn), g, None if Sn is None else abs(Sn), lengths)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full((B, H, L, d), 7.0, dtype=dt, device="cuda")
    got, gotS = F.favor_decay_attention(*(C.place(x, rows) for x in (q, k, v)), torch.from_numpy(g).cuda(),
                                        state=None if S is None else S.cuda(), lengths=n, out=out, return_state=True)
    assert F.favor_sync_status() == 0
    what = f"{B}x{H}x{L} d={d} {name} {rows} state={state} lengths={lengths}"
    assert got is out
    if lengths is not None:
        for b, m in enumerate(np.clip(lengths, 0, L)):
            assert bool((out[b, :, m:] == 7.0).all()), f"{what}: rows past the length were written"
            out[b, :, m:] = 0.0
    w = C.check(got, ref, mag, d, L, name == "bf16", what, f32_operands=name == "f32")
    ws = C.check(gotS, refS, magS, d, L, False, what + " state", f32_operands=name == "f32")
    print(what, f"{w:.3f} {ws:.3f}")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,L,d", SHAPES)
def test_forward(B, H, L, d, name):
    _forward_case(B, H, L, d, name, state=(L + d) % 2 == 0)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ["blhd", "fused"])
@pytest.mark.parametrize("B,H,L,d", [(2, 3, 200, 64), (1, 2, 130, 128), (2, 2, 70, 24)])
def test_forward_strides(B, H, L, d, rows, name):
    _forward_case(B, H, L, d, name, state=True, rows=rows)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("L,d,lengths", [
    (300, 64, [0, 1, 300, 128, 129]), (129, 128, [127, 128, 129, 64, 0]), (700, 32, [700, 65, 513, 1, 699]),
    (50, 64, [-3, 60, 50, 49, 2]),  # held to [0, L]
])
def test_forward_lengths(L, d, lengths, name):
    _forward_case(5, 2, L, d, name, state=True, lengths=lengths, rows="blhd")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("g", [0.0, -np.inf, -100.0, -1e-6, 0.01])
def test_forward_decays(g, name):
    _forward_case(1, 1, 400, 64, name, state=True, g=[g])


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_many_heads(name):
    """More heads than SMs: no segments."""
    _forward_case(20, 10, 150, 64, name, state=True)


@pytest.mark.parametrize("d", [64, 128, 40])
def test_forward_segments_of_ragged_sequences(d):
    """Few heads, long sequences: several segments a sequence, some of them behind its end."""
    _forward_case(3, 1, 5000, d, "bf16", state=True, lengths=[5000, 1, 3071], rows="blhd", g=[-2e-3])


def test_long_sequence_many_segments():
    _forward_case(1, 1, 9000, 64, "bf16", state=True, g=[-1e-3])


def _backward_case(B, H, L, d, name, state, lengths=None, rows="bhld", g=None, seed=0):
    import torch
    import linear_kernelized_attention_b200 as F
    dt = _dtype(name)
    (q, qn), (k, kn), (v, vn), (do, don) = _inputs(B, H, L, d, dt, seed + 40, 4)
    g = C.slopes(H, seed + L) if g is None else np.asarray(g, dtype=np.float32)
    S, Sn = _state(B, H, d, seed + 91) if state else (None, None)
    dS, dSn = _state(B, H, d, seed + 92) if state else (None, None)
    ref = D.decay_backward(qn, kn, vn, g, don, Sn, dSn, lengths)
    mag = D.decay_backward(abs(qn), abs(kn), abs(vn), g, abs(don), None if Sn is None else abs(Sn),
                           None if dSn is None else abs(dSn), lengths)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    outs = [torch.full((B, H, L, d), 7.0, dtype=dt, device="cuda") for _ in range(3)]
    dsi = torch.empty(B, H, d, d, device="cuda")
    got = F.favor_decay_attention_backward(
        *(C.place(x, rows) for x in (q, k, v)), torch.from_numpy(g).cuda(), C.place(do, rows),
        state=None if S is None else S.cuda(), dstate=None if dS is None else dS.cuda(), lengths=n, dq=outs[0],
        dk=outs[1], dv=outs[2], dstate_in=dsi)
    assert F.favor_sync_status() == 0
    what = f"{B}x{H}x{L} d={d} {name} {rows} state={state} lengths={lengths}"
    worst = []
    for i, part in enumerate(("dq", "dk", "dv")):
        if lengths is not None:
            for b, m in enumerate(np.clip(lengths, 0, L)):
                assert bool((outs[i][b, :, m:] == 7.0).all()), f"{what}: {part} rows past the length were written"
                outs[i][b, :, m:] = 0.0
        worst.append(C.check(got[i], ref[i], mag[i], d, L, name == "bf16", f"{what} {part}", name == "f32"))
    worst.append(C.check(got[3], ref[3], mag[3], d, L, False, f"{what} dstate_in", name == "f32"))
    print(what, " ".join(f"{x:.3f}" for x in worst))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,L,d", SHAPES)
def test_backward(B, H, L, d, name):
    _backward_case(B, H, L, d, name, state=(L + d) % 2 == 1)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ["blhd", "fused"])
@pytest.mark.parametrize("B,H,L,d", [(2, 3, 200, 64), (1, 2, 130, 128), (2, 2, 70, 24)])
def test_backward_strides(B, H, L, d, rows, name):
    _backward_case(B, H, L, d, name, state=True, rows=rows)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("L,d,lengths", [
    (300, 64, [0, 1, 300, 128, 129]), (129, 128, [127, 128, 129, 64, 0]), (700, 32, [700, 65, 513, 1, 699]),
])
def test_backward_lengths(L, d, lengths, name):
    _backward_case(5, 2, L, d, name, state=True, lengths=lengths, rows="blhd")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("g", [0.0, -np.inf, -100.0, -1e-6])
def test_backward_decays(g, name):
    _backward_case(1, 1, 400, 64, name, state=True, g=[g])


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_backward_many_heads(name):
    _backward_case(20, 10, 150, 64, name, state=True)


@pytest.mark.parametrize("d", [64, 128])
def test_backward_segments_of_ragged_sequences(d):
    _backward_case(3, 1, 4500, d, "bf16", state=True, lengths=[4500, 0, 2305], rows="blhd", g=[-2e-3])


def test_backward_long_sequence():
    _backward_case(1, 1, 5000, 64, "bf16", state=True, g=[-1e-3])


# ------------------------------------------------------------------ beyond values
def _simple(B=2, H=3, L=260, d=64, name="bf16", seed=5):
    import torch
    dt = _dtype(name)
    q, k, v, do = (x[0].cuda() for x in _inputs(B, H, L, d, dt, seed, 4))
    return q, k, v, do, torch.from_numpy(C.slopes(H)).cuda()


def _same(got, ref, mag):
    """Equal, but where the kernel sums an element again in another order and with unrounded weights: weights in
    bf16 are within 2^-8 of their products, two fp32 sums of at most 128 products differ by at most 2 x 128 x 2^-24
    of their magnitudes' sum, and their bf16 roundings by one step of 2^-7."""
    got, ref, mag = got.float(), ref.float(), mag.float()
    return bool(((got - ref).abs() <= 2.0 ** -7 * ref.abs() + (2.0 ** -8 + 2.0 ** -16) * mag).all())


@pytest.mark.parametrize("name,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 20)])
@pytest.mark.parametrize("where", ["v", "k", "q"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_later_non_finite_tokens_do_not_reach_earlier_rows(name, d, where, bad):
    """A NaN or an infinity in token t of q reaches row t alone, in k or v the rows from t on."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, _, g = _simple(1, 2, 300, d, name)
    clean = F.favor_decay_attention(q, k, v, g)
    mag = F.favor_decay_attention(q.abs(), k.abs(), v.abs(), g)
    x = dict(q=q.clone(), k=k.clone(), v=v.clone())
    for t, c in ((77, 3), (200, d - 1)):
        x[where][0, 0, t, c] = float(bad)
    got = F.favor_decay_attention(x["q"], x["k"], x["v"], g)
    assert torch.equal(got[0, 1], clean[0, 1])
    if where == "q":
        keep = [t for t in range(300) if t not in (77, 200)]
        assert torch.equal(got[0, 0, keep], clean[0, 0, keep])
        assert not torch.isfinite(got[0, 0, 77]).any()
        return
    others = [c for c in range(d) if c not in (3, d - 1)]
    assert torch.equal(got[0, 0, :77][:, others], clean[0, 0, :77][:, others])
    assert _same(got[0, 0, :77], clean[0, 0, :77], mag[0, 0, :77])
    if where == "v":  # only the token's column
        assert not torch.isfinite(got[0, 0, 77:, 3]).any()
        assert not torch.isfinite(got[0, 0, 200:, d - 1]).any()
        assert _same(got[0, 0, 77:200, d - 1], clean[0, 0, 77:200, d - 1], mag[0, 0, 77:200, d - 1])
        assert torch.equal(got[0, 0][:, others], clean[0, 0][:, others])
    else:
        assert not torch.isfinite(got[0, 0, 77:]).any()


@pytest.mark.parametrize("name,d", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 20)])
def test_tokens_past_the_length_are_never_read_into_results(name, d):
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(3, 2, 270, d, name)
    n = torch.tensor([140, 0, 129], dtype=torch.int32, device="cuda")
    clean = F.favor_decay_attention(q, k, v, g, lengths=n, return_state=True)
    cgrad = F.favor_decay_attention_backward(q, k, v, g, do, lengths=n)
    for b, m in enumerate((140, 0, 129)):
        for t in (q, k, v, do):
            t[b, :, m:] = float("nan")
    got = F.favor_decay_attention(q, k, v, g, lengths=n, return_state=True)
    ggrad = F.favor_decay_attention_backward(q, k, v, g, do, lengths=n)
    for a, b in zip((*clean, *cgrad), (*got, *ggrad)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name,d,where", [("f32", 64, "do"), ("bf16", 64, "do"), ("bf16", 128, "q"), ("bf16", 64, "k")])
def test_gradients_keep_non_finite_tokens_to_their_rows(name, d, where):
    """A NaN in token t: of dout or q it reaches dk, dv of rows up to t; of k it reaches dq from t on."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(1, 1, 300, d, name)
    clean = F.favor_decay_attention_backward(q, k, v, g, do)
    mag = F.favor_decay_attention_backward(q.abs(), k.abs(), v.abs(), g, do.abs())
    t = 150
    {"q": q, "k": k, "do": do}[where][0, 0, t, 2] = float("nan")
    dq, dk, dv = F.favor_decay_attention_backward(q, k, v, g, do)
    if where == "k":
        assert _same(dq[:, :, :t], clean[0][:, :, :t], mag[0][:, :, :t]) and torch.equal(dk, clean[1])
        others = [i for i in range(300) if i != t]
        assert torch.equal(dv[:, :, others], clean[2][:, :, others])
    else:
        assert _same(dk[:, :, t + 1:], clean[1][:, :, t + 1:], mag[1][:, :, t + 1:])
        assert _same(dv[:, :, t + 1:], clean[2][:, :, t + 1:], mag[2][:, :, t + 1:])
        if where == "do":
            others = [i for i in range(300) if i != t]
            assert torch.equal(dq[:, :, others], clean[0][:, :, others])
        else:
            assert torch.equal(dq, clean[0])


@pytest.mark.parametrize("name,L", [("bf16", 64), ("bf16", 2000), ("f32", 500)])
def test_state_in_place_and_split_prompt(name, L):
    """state_out = state_in's tensor; two calls carry the state; equal to one call within the tolerance of the
    operands' rounding (the cut moves the chunk borders)."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, _, g = _simple(1, 2, L, 64, name)
    S0 = torch.randn(1, 2, 64, 64, device="cuda")
    _, ref = F.favor_decay_attention(q, k, v, g, state=S0, return_state=True)
    S = S0.clone()
    out, same = F.favor_decay_attention(q, k, v, g, state=S, state_out=S)
    assert same is S and torch.equal(S, ref)
    m = L // 3
    S = S0.clone()
    F.favor_decay_attention(q[:, :, :m], k[:, :, :m], v[:, :, :m], g, state=S, state_out=S)
    F.favor_decay_attention(q[:, :, m:], k[:, :, m:], v[:, :, m:], g, state=S, state_out=S)
    assert float((S - ref).norm() / ref.norm()) < 2.0 ** -16


@pytest.mark.parametrize("name,L,d", [("bf16", 300, 64), ("bf16", 6000, 64), ("bf16", 300, 128), ("f32", 500, 64),
                                      ("bf16", 200, 20)])
def test_gradient_state_in_place(name, L, d):
    """dstate_in = dstate's tensor: two of the three gradients read it."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(1, 2, L, d, name)
    S, dS = torch.randn(2, 1, 2, d, d, device="cuda")
    ref = F.favor_decay_attention_backward(q, k, v, g, do, state=S, dstate=dS)
    got = F.favor_decay_attention_backward(q, k, v, g, do, state=S, dstate=dS, dstate_in=dS)
    assert got[3] is dS
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("d", [64, 128])
def test_overlapping_input_rows(d):
    """A window sliding over one buffer: rows of an input may overlap."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(1, 2, 400, d)
    buf = torch.randn(2, 399 * 8 + d, device="cuda").bfloat16() * 0.3
    w = buf.as_strided((1, 2, 400, d), (0, buf.stride(0), 8, 1))
    out, S = F.favor_decay_attention(q, w, v, g, return_state=True)
    ref, rS = F.favor_decay_attention(q, w.contiguous(), v, g, return_state=True)
    assert torch.equal(out, ref) and torch.equal(S, rS)
    for a, b in zip(F.favor_decay_attention_backward(q, w, v, g, do),
                    F.favor_decay_attention_backward(q, w.contiguous(), v, g, do)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name,d", [("bf16", 64), ("bf16", 20), ("f32", 64)])
def test_offsets_past_32_bits(name, d):
    """Batch entries more than 2^32 bytes apart, inputs and outputs."""
    import torch
    import linear_kernelized_attention_b200 as F
    dt = _dtype(name)
    far = (2 ** 32 // torch.empty((), dtype=dt).element_size()) + 64
    big = [torch.empty(far + 200 * d, dtype=dt, device="cuda") for _ in range(2)]
    x, o = (b.as_strided((2, 1, 200, d), (far, 200 * d, d, 1)) for b in big)
    q = _simple(2, 1, 200, d, name)[0]
    x.copy_(q)
    g = torch.tensor([-0.05], device="cuda")
    ref, rS = F.favor_decay_attention(q, q, q, g, return_state=True)
    out, S = F.favor_decay_attention(x, x, x, g, out=o, return_state=True)
    assert torch.equal(out, ref) and torch.equal(S, rS)
    rg = F.favor_decay_attention_backward(q, q, q, g, q)
    assert torch.equal(F.favor_decay_attention_backward(x, x, x, g, x, dq=o)[0], rg[0])
    freq, _ = F.favor_rotary_frequencies(d, device="cuda")
    F.favor_rotary(x, None, freq, q_out=o)
    assert torch.equal(o, F.favor_rotary(q, None, freq)[0])


def test_same_tensor_as_query_key_and_value():
    import torch
    import linear_kernelized_attention_b200 as F
    q, _, _, do, g = _simple(1, 2, 300, 64)
    ref = F.favor_decay_attention(q, q.clone(), q.clone(), g, return_state=True)
    assert all(torch.equal(a, b) for a, b in zip(F.favor_decay_attention(q, q, q, g, return_state=True), ref))
    ref = F.favor_decay_attention_backward(q, q.clone(), q.clone(), g, do)
    assert all(torch.equal(a, b) for a, b in zip(F.favor_decay_attention_backward(q, q, q, g, do), ref))


def test_graphs_replayed_at_once_do_not_share_scratch():
    """Two captured calls that each take scratch (several segments), replayed on two streams together."""
    import torch
    import linear_kernelized_attention_b200 as F
    sets = [_simple(1, 1, 6000, 64, seed=s) for s in (41, 42)]
    assert F.favor_decay_workspace_bytes(1, 1, 6000, 64) > 0
    refs = [F.favor_decay_attention(*x[:3], x[4], return_state=True) for x in sets]
    outs = [(torch.zeros_like(x[0]), torch.zeros(1, 1, 64, 64, device="cuda")) for x in sets]
    torch.cuda.synchronize()
    graphs, streams = [torch.cuda.CUDAGraph() for _ in sets], [torch.cuda.Stream() for _ in sets]
    for gr, x, o in zip(graphs, sets, outs):
        with torch.cuda.graph(gr):
            F.favor_decay_attention(*x[:3], x[4], out=o[0], state_out=o[1])
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(refs, outs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeated_calls_are_identical():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(2, 4, 1100, 64)
    a = (*F.favor_decay_attention(q, k, v, g, return_state=True), *F.favor_decay_attention_backward(q, k, v, g, do))
    for _ in range(3):
        b = (*F.favor_decay_attention(q, k, v, g, return_state=True), *F.favor_decay_attention_backward(q, k, v, g, do))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_broadcast_head(name):
    """One k and v head shared by every query head through stride 0."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(2, 3, 200, 64, name)
    k1, v1 = k[:, :1].expand_as(q), v[:, :1].expand_as(q)
    got = F.favor_decay_attention(q, k1, v1, g)
    ref = F.favor_decay_attention(q, k1.contiguous(), v1.contiguous(), g)
    tol = 2.0 ** -7 if name == "bf16" else 2.0 ** -16
    assert float((got.float() - ref.float()).norm()) <= tol * float(ref.float().norm())
    got = F.favor_decay_attention_backward(q, k1, v1, g, do)
    ref = F.favor_decay_attention_backward(q, k1.contiguous(), v1.contiguous(), g, do)
    for a, b in zip(got, ref):
        assert float((a.float() - b.float()).norm()) <= tol * float(b.float().norm())


def test_graph_capture_and_replay():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(1, 3, 900, 64)
    S = torch.zeros(1, 3, 64, 64, device="cuda")
    F.favor_decay_attention(q, k, v, g, state=S, return_state=True)
    F.favor_decay_attention_backward(q, k, v, g, do)
    out, so = torch.empty_like(q), torch.empty_like(S)
    grads = [torch.empty_like(q) for _ in range(3)]
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        F.favor_decay_attention(q, k, v, g, state=S, out=out, state_out=so)
    with torch.cuda.graph(g2):
        F.favor_decay_attention_backward(q, k, v, g, do, dq=grads[0], dk=grads[1], dv=grads[2])
    for seed in (21, 22):
        fresh = _simple(1, 3, 900, 64, seed=seed)
        for a, b in zip((q, k, v, do), fresh):
            a.copy_(b)
        S.normal_()
        g2.replay()
        g1.replay()
        ref = F.favor_decay_attention(q, k, v, g, state=S, return_state=True)
        rg = F.favor_decay_attention_backward(q, k, v, g, do)
        assert torch.equal(out, ref[0]) and torch.equal(so, ref[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, rg))


def test_two_streams_at_once():
    import torch
    import linear_kernelized_attention_b200 as F
    sets = [_simple(2, 4, 700, 64, seed=s) for s in (31, 32)]
    refs = [F.favor_decay_attention(*x[:3], x[4], return_state=True) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = [F.favor_decay_attention(*x[:3], x[4], return_state=True, stream=s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(refs, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_new_outputs_are_zero_past_the_length():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(2, 2, 100, 64)
    n = torch.tensor([40, 0], dtype=torch.int32, device="cuda")
    out = F.favor_decay_attention(q, k, v, g, lengths=n)
    assert not out[0, :, 40:].any() and not out[1].any()
    for x in F.favor_decay_attention_backward(q, k, v, g, do, lengths=n):
        assert not x[0, :, 40:].any() and not x[1].any()


def test_refusals():
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(1, 2, 20, 64)
    with pytest.raises(TypeError):
        F.favor_decay_attention(q.half(), k.half(), v.half(), g)
    with pytest.raises(TypeError):
        F.favor_decay_attention(q, k.float(), v, g)
    with pytest.raises(TypeError):
        F.favor_decay_attention(q, k, v, g.double())
    with pytest.raises(TypeError):
        F.favor_decay_attention(q, k, v, None)
    with pytest.raises(ValueError):
        F.favor_decay_attention(q, k[:, :1], v, g)
    with pytest.raises(ValueError):
        F.favor_decay_attention(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), g)
    with pytest.raises(TypeError):
        F.favor_decay_attention(q, k, v, g, lengths=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        F.favor_decay_attention(q, k, v, g, state=torch.zeros(1, 2, 64, 32, device="cuda"))
    with pytest.raises(F.FavorError):
        F.favor_decay_attention(q, k, v, g, out=v)
    with pytest.raises(F.FavorError):
        F.favor_decay_attention(q, k, v, g, out=q[:, :1].expand_as(q).contiguous()[:, :1].expand_as(q))
    with pytest.raises(ValueError):
        F.favor_decay_attention_backward(q, k, v, g, do[:, :, :5])
    S = torch.zeros(1, 2, 64, 64, device="cuda")
    with pytest.raises(F.FavorError):
        F.favor_decay_attention_backward(q, k, v, g, do, state=S, dstate_in=S)
    wide = torch.zeros(1, 1, 4, 136, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(F.FavorError) as e:
        F.favor_decay_attention(wide, wide, wide, g[:1])
    assert e.value.code == -5
    torch.cuda.synchronize()
    assert F.favor_sync_status() == 0


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("H,d", [(2, 20), (2, 33), (1, 20), (3, 100)])
def test_slices_of_rows_that_are_not_whole_pieces(H, d, name):
    """Token slices, split prompts and fused projections of odd heads start anywhere: the same results as their
    copies, bit for bit."""
    import torch
    import linear_kernelized_attention_b200 as F
    x = torch.randn(2, 90, 3, H, d, device="cuda").to(_dtype(name)) * 0.5  # fused [B, L, 3, H, d]
    do = torch.randn(2, H, 90, d, device="cuda").to(_dtype(name))
    g = torch.from_numpy(C.slopes(H)).cuda()
    q, k, v = (x[:, :, i].transpose(1, 2) for i in range(3))
    c = [t.contiguous() for t in (q, k, v)]
    if d * x.element_size() % 16:
        assert any(t.data_ptr() % 16 for t in (q, k, v, x[:, 1:], do[:, :, 41:]))
    ref = F.favor_decay_attention(*c, g, return_state=True)
    got = F.favor_decay_attention(q, k, v, g, return_state=True)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for a, b in zip(F.favor_decay_attention_backward(q, k, v, g, do), F.favor_decay_attention_backward(*c, g, do)):
        assert torch.equal(a, b)
    # the prompt in two parts, outputs and gradients into slices too
    cut = lambda t, a, b: t[:, :, a:b]
    S1, S2 = torch.zeros(2, 2, H, d, d, device="cuda")
    out = torch.empty_like(c[0])
    dq, dk, dv = (torch.empty_like(t) for t in c)
    for a, b in ((0, 41), (41, 90)):
        part, whole = [cut(t, a, b) for t in c], [cut(t, a, b).contiguous() for t in c]
        F.favor_decay_attention(*part, g, state=S1, out=cut(out, a, b), state_out=S1)
        ref, _ = F.favor_decay_attention(*whole, g, state=S2, state_out=S2)
        assert torch.equal(cut(out, a, b), ref) and torch.equal(S1, S2)
        F.favor_decay_attention_backward(*part, g, cut(do, a, b), dq=cut(dq, a, b), dk=cut(dk, a, b), dv=cut(dv, a, b))
        for t, w in zip((dq, dk, dv), F.favor_decay_attention_backward(*whole, g, cut(do, a, b).contiguous())):
            assert torch.equal(cut(t, a, b), w)
    # single tokens of the contiguous prompt
    S1, S2 = torch.zeros(2, 2, H, d, d, device="cuda")
    for t in range(9):
        row = F.favor_decay_step(*(y[:, :, t] for y in c), g, S1, out=out[:, :, t])
        assert torch.equal(row, F.favor_decay_step(*(y[:, :, t].contiguous() for y in c), g, S2))
    assert torch.equal(S1, S2)
    freq, _ = F.favor_rotary_frequencies(d // 2 * 2, device="cuda")
    for a, b in zip(F.favor_rotary(q[:, :, 3:], k[:, :, 3:], freq),
                    F.favor_rotary(q[:, :, 3:].contiguous(), k[:, :, 3:].contiguous(), freq)):
        assert torch.equal(a, b)
    assert F.favor_sync_status() == 0


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_rows_of_whole_pieces_between_odd_strides(name):
    """d = 64 in rows of 67 elements, from an odd element on."""
    import torch
    import linear_kernelized_attention_b200 as F
    wide = [torch.randn(2, 3, 150, 67, device="cuda").to(_dtype(name)) for _ in range(4)]
    q, k, v, do = (t[..., 1:65] for t in wide)
    g = torch.from_numpy(C.slopes(3)).cuda()
    c = [t.contiguous() for t in (q, k, v, do)]
    # the copies of bf16 rows go to the tensor cores, these to the CUDA cores: within twice the norms that
    # decay_cases.check allows each, 2 x 2 sqrt(2 / 3) 2^-8 < 2^-6 and 2 x 2^-19
    (r, rS), (o, S) = (F.favor_decay_attention(*t[:3], g, return_state=True) for t in (c, (q, k, v)))
    tol = 2.0 ** -6 if name == "bf16" else 0.0
    assert float((o.float() - r.float()).norm()) <= tol * float(r.float().norm())
    assert float((S - rS).norm()) <= (2.0 ** -18 if name == "bf16" else 0.0) * float(rS.norm())
    for a, b in zip(F.favor_decay_attention_backward(q, k, v, g, do), F.favor_decay_attention_backward(*c[:3], g, c[3])):
        assert float((a.float() - b.float()).norm()) <= tol * float(b.float().norm())


# ------------------------------------------------------------------ non-finite tokens, many of them
def _spoil(x, spots):
    for name, t, c, val in spots:
        x[name][0, 0, t, slice(None) if c is None else c] = float(val)


SPOTS = {
    "every chunk": [("v", t, None, "nan") for t in range(127, 600, 128)],
    "first of every chunk": [("v", t, 5, "inf") for t in range(0, 600, 128)],
    "key then values": [("k", 200, 3, "inf"), ("v", 260, None, "nan"), ("v", 20, 6, "-inf")],
    "dout": [("do", 400, None, "nan"), ("do", 130, 2, "inf"), ("q", 300, 1, "nan")],
    "all keys": [("k", t, None, "nan") for t in range(600)],
    "all": [(n, t, None, "nan") for n in ("q", "k", "v", "do") for t in range(600)],
}


@pytest.mark.parametrize("name,d", [("bf16", 64), ("bf16", 128), ("bf16", 40), ("f32", 64)])
@pytest.mark.parametrize("spots", list(SPOTS))
def test_non_finite_tokens_reach_what_the_recurrence_takes_them_to(name, d, spots):
    """Which elements are finite is the float64 recurrence's, rows and gradients; the finite ones keep their bounds."""
    import torch
    import linear_kernelized_attention_b200 as F
    dt = _dtype(name)
    x = {n: t for n, (t, _) in zip(("q", "k", "v", "do"), _inputs(1, 1, 600, d, dt, 77, 4))}
    _spoil(x, SPOTS[spots])
    f = {n: t.double().numpy() for n, t in x.items()}
    clean = {n: np.where(np.isfinite(a), a, 0.0) for n, a in f.items()}
    g = np.array([-0.01], dtype=np.float32)
    gg = torch.from_numpy(g).cuda()
    c = {n: t.cuda() for n, t in x.items()}
    out, S = F.favor_decay_attention(c["q"], c["k"], c["v"], gg, return_state=True)
    grads = F.favor_decay_attention_backward(c["q"], c["k"], c["v"], gg, c["do"])
    assert F.favor_sync_status() == 0
    with np.errstate(invalid="ignore"):
        want = [*D.decay_attention(f["q"], f["k"], f["v"], g), *D.decay_backward(f["q"], f["k"], f["v"], g, f["do"])[:3]]
    a = {n: np.abs(v) for n, v in clean.items()}
    mag = [*D.decay_attention(a["q"], a["k"], a["v"], g), *D.decay_backward(a["q"], a["k"], a["v"], g, a["do"])[:3]]
    for i, (got, ref, m) in enumerate(zip((out, S, *grads), want, mag)):
        got = got.double().cpu().numpy()
        ok = np.isfinite(ref)
        assert np.array_equal(np.isfinite(got), ok), ("out", "state", "dq", "dk", "dv")[i]
        # an element summed again carries weights and scores in fp32: inside the bounds of the rounded ones
        assert (np.abs(got[ok] - ref[ok]) <= C.allowed(np.where(ok, ref, 0.0), m, d, 600, name == "bf16" and i != 1)[ok]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("names", [("q", "k", "v", "do"), ("k",), ("v",), ("do",)])
def test_a_call_on_nan_takes_about_as_long_as_any_other(d, names):
    """A diverged training step: every element of some operand is NaN. Where each element was summed again over
    its own tokens, such calls took 35 to 450 times as long as clean ones; 10 leaves room for noise."""
    import torch
    import linear_kernelized_attention_b200 as F
    x = dict(zip(("q", "k", "v", "do"), _simple(1, 8, 2048, d)[:4]))
    g = torch.full((8,), -0.05, device="cuda")

    def us(x):
        best = 1e9
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            F.favor_decay_attention(x["q"], x["k"], x["v"], g)
            F.favor_decay_attention_backward(x["q"], x["k"], x["v"], g, x["do"])
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3)
        return best

    clean = us(x)
    bad = us({n: torch.full_like(t, float("nan")) if n in names else t for n, t in x.items()})
    assert bad <= 10 * clean, (clean, bad)


@pytest.mark.parametrize("name,d", [("bf16", 64), ("bf16", 128), ("bf16", 20), ("f32", 64)])
def test_broadcast_head_is_its_copies(name, d):
    """Heads shared through stride 0 pass through the same arithmetic as copies of them: equal bit for bit."""
    import torch
    import linear_kernelized_attention_b200 as F
    q, k, v, do, g = _simple(2, 3, 200, d, name)
    k1, v1 = k[:, :1].expand_as(q), v[:1, :1].expand_as(q)
    got = (*F.favor_decay_attention(q, k1, v1, g, return_state=True), *F.favor_decay_attention_backward(q, k1, v1, g, do))
    k2, v2 = k1.contiguous(), v1.contiguous()
    ref = (*F.favor_decay_attention(q, k2, v2, g, return_state=True), *F.favor_decay_attention_backward(q, k2, v2, g, do))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("L,g", [(600, 0.1), (40, 2.0)])
def test_growing_states_up_to_the_documented_limit(L, g, name):
    """Positive log decays with exp(L g) within fp32, exp(128 g) beyond it for the short one."""
    _forward_case(1, 1, L, 64, name, state=True, g=[g])
    _backward_case(1, 1, L, 64, name, state=True, g=[g])


FIRST_CALL = """
import torch
import linear_kernelized_attention_b200 as F
q = (torch.randn(1, 2, 3000, 64, device="cuda") * 0.3).{dtype}()
g = torch.full((2,), -0.05, device="cuda")
out = torch.zeros_like(q)
om = torch.randn(2, 64, 64, device="cuda").{dtype}()
call = lambda: {call}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = out.clone()
assert got.any()
call()
assert torch.equal(got, out) and F.favor_sync_status() == 0
print("captured")
"""


@pytest.mark.parametrize("dtype,call", [
    ("bfloat16", "F.favor_decay_attention(q, q, q, g, out=out)"), ("float", "F.favor_decay_attention(q, q, q, g, out=out)"),
    ("bfloat16", "F.favor_decay_attention_backward(q, q, q, g, q, dq=out)"),
    ("bfloat16", "F.favor_attention(q, q, q, om, out=out)"),
])
def test_first_call_of_a_process_may_be_captured(dtype, call):
    """The library's scratch pool is made on first use, also where that is inside a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(dtype=dtype, call=call)], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
