"""The float64 oracle of the decayed linear attention, pinned on the CPU: the recurrence equals the masked
quadratic form, gradients equal central differences and torch's, rotary equals its matrices; and the
host-only frequency table equals its formulas."""
import math

import numpy as np
import pytest

from oracle import decay_oracle as D


def _inputs(B, H, L, d, seed, n=4):
    r = np.random.default_rng(seed)
    return [r.standard_normal((B, H, L, d)) for _ in range(n)]


@pytest.mark.parametrize("g", [-0.4, 0.0, -np.inf, -40.0])
def test_recurrence_equals_quadratic_form(g):
    q, k, v = _inputs(1, 1, 9, 5, 1, 3)
    S = np.random.default_rng(2).standard_normal((1, 1, 5, 5))
    out, new = D.decay_attention(q, k, v, [g], S)
    lam = math.exp(g)
    assert np.allclose(out[0, 0], D.decay_quadratic_head(q[0, 0], k[0, 0], v[0, 0], lam, S[0, 0]), atol=1e-12)
    w = np.array([lam ** (8 - j) for j in range(9)])
    assert np.allclose(new[0, 0], (k[0, 0] * w[:, None]).T @ v[0, 0] + lam ** 9 * S[0, 0], atol=1e-12)


def test_split_prompt_equals_whole():
    q, k, v = _inputs(2, 3, 11, 4, 3, 3)
    g = [-0.1, -0.7, 0.0]
    out, S = D.decay_attention(q, k, v, g)
    o1, s1 = D.decay_attention(q[:, :, :4], k[:, :, :4], v[:, :, :4], g)
    o2, s2 = D.decay_attention(q[:, :, 4:], k[:, :, 4:], v[:, :, 4:], g, s1)
    assert np.allclose(out, np.concatenate([o1, o2], 2)) and np.allclose(S, s2)


def test_lengths_stop_the_recurrence():
    q, k, v = _inputs(3, 2, 6, 3, 4, 3)
    S0 = np.random.default_rng(5).standard_normal((3, 2, 3, 3))
    out, S = D.decay_attention(q, k, v, [-0.2, 0.0], S0, [0, 4, 6])
    assert np.array_equal(S[0], S0[0]) and not out[0].any() and not out[1, :, 4:].any()
    o4, s4 = D.decay_attention(q[1:2, :, :4], k[1:2, :, :4], v[1:2, :, :4], [-0.2, 0.0], S0[1:2])
    assert np.allclose(out[1, :, :4], o4[0]) and np.allclose(S[1], s4[0])


@pytest.mark.parametrize("g", [-0.3, 0.0, -np.inf])
def test_gradients_equal_differences(g):
    q, k, v, do = _inputs(1, 1, 5, 3, 6)
    r = np.random.default_rng(7)
    S, dS = r.standard_normal((2, 1, 1, 3, 3))
    lens = [4]

    def loss(q, k, v, S):
        o, s = D.decay_attention(q, k, v, [g], S, lens)
        return (o * do)[:, :, :4].sum() + (s * dS).sum()

    grads = D.decay_backward(q, k, v, [g], do, S, dS, lens)
    base = [q, k, v, S]
    for i, x in enumerate(base):
        for idx in np.ndindex(x.shape):
            hi, lo = x.copy(), x.copy()
            hi[idx] += 1e-5
            lo[idx] -= 1e-5
            args = list(base)
            args[i] = hi
            up = loss(*args)
            args[i] = lo
            assert abs((up - loss(*args)) / 2e-5 - grads[i][idx]) < 1e-7


def test_gradients_equal_autograd():
    import torch
    q, k, v, do = (torch.tensor(x, requires_grad=True) for x in _inputs(2, 2, 7, 4, 8))
    g = torch.tensor([-0.2, -1.5], dtype=torch.float64)
    i = torch.arange(7)
    gap = (i[:, None] - i[None, :]).double()
    w = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), torch.zeros((), dtype=torch.float64))
    ((((q @ k.transpose(-1, -2)) * w) @ v) * do.detach()).sum().backward()
    dq, dk, dv, _ = D.decay_backward(*(t.detach().numpy() for t in (q, k, v)), g.numpy(), do.detach().numpy())
    for a, b in zip((dq, dk, dv), (q, k, v)):
        assert np.allclose(a, b.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_equals_its_matrices_and_inverse(interleaved):
    x = np.random.default_rng(9).standard_normal((1, 2, 3, 6))
    freq, pos = np.array([0.7, 0.01]), np.array([[0, 5, 1000]])
    y = D.rotary(x, freq, pos, interleaved, scale=0.5, rot_scale=1.5)
    for t in range(3):
        R = np.eye(6) * 0.5
        for i, f in enumerate(freq):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 2)
            c, s = math.cos(pos[0, t] * f), math.sin(pos[0, t] * f)
            R[np.ix_([a, b], [a, b])] = 0.75 * np.array([[c, -s], [s, c]])
        assert np.allclose(y[0, :, t], x[0, :, t] @ R.T)
        back = D.rotary(y, freq, pos, interleaved, inverse=True, scale=0.5, rot_scale=1.5)
        assert np.allclose(back[0, :, t], y[0, :, t] @ R)


def test_rotary_frequencies_follow_their_formulas():
    import linear_kernelized_attention_b200 as F
    i = np.arange(16)
    plain = 10000.0 ** (-2.0 * i / 32)
    f, m = F.favor_rotary_frequencies(32)
    assert np.allclose(f.numpy(), plain, rtol=1e-14) and m == 1.0
    f, m = F.favor_rotary_frequencies(32, scaling=F.FAVOR_ROTARY_LINEAR, factor=8)
    assert np.allclose(f.numpy(), plain / 8, rtol=1e-14) and m == 1.0
    f, m = F.favor_rotary_frequencies(32, scaling=F.FAVOR_ROTARY_BASE, factor=8)
    assert np.isclose(f[0], 1.0) and np.isclose(f[-1], plain[-1] / 8, rtol=1e-12) and m == 1.0
    f, m = F.favor_rotary_frequencies(32, scaling=F.FAVOR_ROTARY_PARTS, factor=4, trained_length=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(f.numpy()[turns >= 32], plain[turns >= 32], rtol=1e-14)
    assert np.allclose(f.numpy()[turns <= 1], plain[turns <= 1] / 4, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    ramp = (turns[mid] - 1) / 31
    assert mid.any() and np.allclose(f.numpy()[mid], plain[mid] * (ramp + (1 - ramp) / 4), rtol=1e-14)
    assert np.isclose(m, 0.1 * math.log(4) + 1)


@pytest.mark.parametrize("args,kw,code", [
    ((0,), {}, -3), ((3,), {}, -3), ((8,), dict(base=1.0), -3), ((8,), dict(base=float("nan")), -3),
    ((8,), dict(scaling=4), -4), ((8,), dict(scaling=-1), -4),
    ((8,), dict(scaling=1, factor=0.5), -3), ((2,), dict(scaling=2, factor=2.0), -3),
    ((8,), dict(scaling=3, factor=2.0, trained_length=0), -3),
    ((8,), dict(scaling=3, factor=2.0, trained_length=128, beta_fast=1.0, beta_slow=1.0), -3),
])
def test_rotary_frequencies_refuse(args, kw, code):
    import linear_kernelized_attention_b200 as F
    with pytest.raises(F.FavorError) as e:
        F.favor_rotary_frequencies(*args, **kw)
    assert e.value.code == code


@pytest.mark.parametrize("block", [1, 7, 16, 64])
def test_blocked_reference_equals_recurrence(block, monkeypatch):
    """The 64-bit reference of the long tests, against the recurrence: forward, gradients, states, every kind of decay."""
    import torch

    import decay_cases as C
    monkeypatch.setattr(C.scan64, "__defaults__", (None, False, block))
    g = np.array([-0.3, 0.0, -np.inf, -40.0])
    q, k, v, do = _inputs(2, 4, 33, 5, 11)
    S, dS = np.random.default_rng(12).standard_normal((2, 2, 4, 5, 5))
    t = [torch.from_numpy(x) for x in (q, k, v, do, S, dS)]
    got = [*C.forward64(*t[:3], g, t[4]), *C.backward64(*t[:3], g, t[3], t[4], t[5])]
    want = [*D.decay_attention(q, k, v, g, S), *D.decay_backward(q, k, v, g, do, S, dS)]
    for a, b in zip(got, want):
        assert np.allclose(a.numpy(), b, atol=1e-11)
    assert np.allclose(C.forward64(*t[:3], g)[0].numpy(), D.decay_attention(q, k, v, g)[0], atol=1e-11)


def test_drift_bound_tells_a_rounded_decay_from_an_exact_one():
    """4096 steps of a decaying state in fp32 on the CPU: with lambda as one fp32 value the mean error is past the
    bound, with its remainder carried well inside it."""
    import decay_cases as C
    T, g = 4096, C.coarse_slope()
    lam = math.exp(g)
    lh = np.float32(lam)
    ll = np.float32(lam - float(lh))
    s0 = np.random.default_rng(3).standard_normal(4096).astype(np.float32)
    one, two = s0.copy(), s0.copy()
    for _ in range(T):
        one = one * lh
        two = (two.astype(np.float64) * lh + (two * ll).astype(np.float64)).astype(np.float32)  # a fused update
    mean = lambda s: abs(np.mean(s.astype(np.float64) / (s0.astype(np.float64) * lam ** T) - 1))
    assert mean(two) <= 0.1 * C.drift_allowed(T) and mean(one) >= 5 * C.drift_allowed(T)
