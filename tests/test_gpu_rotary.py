"""Rotary positions on the GPU against the float64 rotation.

The tolerance is derived in decay_cases.rotary_allowed.
"""
import numpy as np
import pytest

import decay_cases as C
from oracle import decay_oracle as D

pytestmark = pytest.mark.gpu


def _check(got, x, freq, pos, inter, inv, scale, rs, bf16):
    ref = D.rotary(x, freq, pos, inter, inv, scale, rs)
    a = C.rotary_allowed(ref, x, len(freq), inter, scale, rs, bf16)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= a).all(), float((err / a).max())


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,L,d,rot", [
    (1, 1, 1, 1, 2, 2), (2, 4, 1, 37, 64, 64), (1, 3, 2, 130, 128, 64), (2, 2, 2, 9, 48, 16), (1, 2, 5, 21, 33, 10),
    (1, 8, 0, 5, 80, 80), (3, 40, 8, 1, 128, 128), (1, 2, 2, 1000, 256, 96), (2, 1, 1, 12, 40, 24),
])
def test_rotary(B, Hq, Hk, L, d, rot, interleaved, name):
    import torch
    import linear_kernelized_attention_b200 as F
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[name]
    q, qn = C.draw((B, Hq, L, d), 1, dt)
    k, kn = C.draw((B, max(Hk, 1), L, d), 2, dt)
    freq, rs = F.favor_rotary_frequencies(rot, scaling=F.FAVOR_ROTARY_PARTS, factor=2, trained_length=512)
    pos = np.random.default_rng(4).integers(0, 5000, (B, L)).astype(np.int32)
    inv = (L + d) % 2 == 0
    qo, ko = F.favor_rotary(q.cuda(), k.cuda() if Hk else None, freq.cuda(), positions=torch.from_numpy(pos).cuda(),
                            interleaved=interleaved, inverse=inv, scale=d ** -0.25, rot_scale=rs)
    assert F.favor_sync_status() == 0
    _check(qo, qn, freq.numpy(), pos, interleaved, inv, d ** -0.25, rs, name == "bf16")
    if Hk:
        _check(ko, kn, freq.numpy(), pos, interleaved, inv, d ** -0.25, rs, name == "bf16")
    else:
        assert ko is None


@pytest.mark.parametrize("first", [0, 1, 123456789, 2 ** 31 - 40])
def test_far_positions_keep_their_angle(first):
    import torch
    import linear_kernelized_attention_b200 as F
    q, qn = C.draw((1, 2, 30, 64), 5, torch.float32)
    freq, _ = F.favor_rotary_frequencies(64)
    qo, _ = F.favor_rotary(q.cuda(), None, freq.cuda(), first_position=first)
    pos = first + np.arange(30, dtype=np.int64)[None]
    _check(qo, qn, freq.numpy(), pos, False, False, 1.0, 1.0, False)


def test_negative_positions():
    import torch
    import linear_kernelized_attention_b200 as F
    q, qn = C.draw((1, 1, 8, 32), 6, torch.float32)
    freq, _ = F.favor_rotary_frequencies(32)
    pos = -np.arange(8, dtype=np.int32)[None] * 77
    qo, _ = F.favor_rotary(q.cuda(), None, freq.cuda(), positions=torch.from_numpy(pos).cuda())
    _check(qo, qn, freq.numpy(), pos, False, False, 1.0, 1.0, False)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strided(interleaved, name):
    import torch
    import linear_kernelized_attention_b200 as F
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[name]
    x = torch.randn(2, 50, 3, 4, 64, device="cuda").to(dt)  # [B, L, 3, H, d]
    freq, _ = F.favor_rotary_frequencies(32, device="cuda")
    q, k = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
    ref = F.favor_rotary(q.contiguous(), k.contiguous(), freq, interleaved=interleaved)
    keep = x[:, :, 2].clone()
    a, b = F.favor_rotary(q, k, freq, interleaved=interleaved)
    assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])
    a, b = F.favor_rotary(q, k, freq, interleaved=interleaved, q_out=q, k_out=k)
    assert a is q and torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and torch.equal(x[:, :, 2], keep)


def test_inverse_is_the_gradient():
    import torch
    import linear_kernelized_attention_b200 as F
    (q, qn), (w, wn) = (C.draw((1, 2, 20, 64), s, torch.float32) for s in (7, 8))
    freq, _ = F.favor_rotary_frequencies(48, device="cuda")
    y, _ = F.favor_rotary(q.cuda(), None, freq, scale=0.5, rot_scale=1.25, first_position=9)
    dx, _ = F.favor_rotary(w.cuda(), None, freq, scale=0.5, rot_scale=1.25, first_position=9, inverse=True)
    lhs = float((y.double().cpu().numpy() * wn).sum())
    rhs = float((dx.double().cpu().numpy() * qn).sum())
    # both sides are the same sum of 2560 products, each within 2^-21 of its pair's magnitude
    assert abs(lhs - rhs) <= 2 * 2.0 ** -21 * np.sum(C.pair_mag(qn.copy(), 24, False, 0.5, 1.25) * np.abs(wn))


def test_refusals():
    import torch
    import linear_kernelized_attention_b200 as F
    q = torch.randn(1, 2, 8, 64, device="cuda")
    freq = torch.ones(16, dtype=torch.float64, device="cuda")
    with pytest.raises(TypeError):
        F.favor_rotary(q, q, freq.float())
    with pytest.raises(TypeError):
        F.favor_rotary(q, q, [1.0] * 16)
    with pytest.raises(TypeError):
        F.favor_rotary(q, q.bfloat16(), freq)
    with pytest.raises(TypeError):
        F.favor_rotary(q, None, freq, positions=torch.zeros(1, 8, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        F.favor_rotary(q, None, freq, positions=torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        F.favor_rotary(q, None, freq, k_out=q)
    with pytest.raises(ValueError):
        F.favor_rotary(q, None, freq, first_position=2 ** 31)
    with pytest.raises(F.FavorError):
        F.favor_rotary(q, None, torch.ones(33, dtype=torch.float64, device="cuda"))
    with pytest.raises(F.FavorError):
        F.favor_rotary(q, q.clone(), freq, q_out=q, k_out=q)
    torch.cuda.synchronize()
    assert F.favor_sync_status() == 0
