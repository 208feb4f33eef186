"""Seeded inputs and derived tolerances for the decayed linear attention tests.

Tolerances. Every output is a sum of products; `mag` is the oracle run on absolute values, the sum of
their magnitudes, so a relative error e in every product's chain of roundings moves an output by at most
e mag.
  fp32: a product passes at most d roundings in a score or state product, 2 x 128 in chunk sums, one
    for each 128-token chunk it is carried over (`hops`), and ten in weights and joins:
    (d + 266 + hops) 2^-24 mag.
  fp32 states of bf16 operands, on the tensor cores: the decayed operand in three bf16 terms, 2^-26 of a
    product; a chunk's sum is accumulated 24 times with truncation (2^-23 each), below the 256 roundings above.
  bf16 outputs: one rounding of the result (2^-8 |o|), and on the tensor cores one of the weighted scores
    inside a chunk, or one of the carried state's image; the decayed operand of the state's update keeps 16 bits
    there (2^-16): 2^-8 |o| + (2^-8 + 2^-16) mag, plus the fp32 terms.
  The elementwise bound is a worst case. Roundings have independent signs, each with a variance of at
    most 2^-16 / 3 of its product's square, so for random inputs the root mean square of the error over
    a tensor stays within sqrt(2 / 3) 2^-8 of the root mean square of the outputs: the norm test allows
    twice that for bf16. fp32 values: sums of some 128 terms with independent roundings, 0.6 sqrt(128) 2^-24 =
    2^-21.2, and up to 24 truncations of one sign, half a step each, 2^-20.4: the norm test allows 2^-19.
"""
import numpy as np

U32, UBF = 2.0 ** -24, 2.0 ** -8
SLOPES = (-0.3, 0.0, -2.0 ** -7, -np.inf, -30.0, -1e-4)


def slopes(H, first=0):
    return np.array([SLOPES[(first + h) % len(SLOPES)] for h in range(H)], dtype=np.float32)


def draw(shape, seed, dtype, scale=1.0):
    """(CPU tensor in dtype, its float64 values)."""
    import torch
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale))
    x = x.to(dtype)
    return x, x.double().numpy()


def place(t, rows="bhld"):
    """The tensor on the GPU: [B, H, L, d] contiguous, token-major, or a slice of a fused projection."""
    import torch
    t = t.cuda()
    if rows == "bhld":
        return t
    if rows == "blhd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    B, H, L, d = t.shape  # "fused": the middle third of [B, L, 3, H, d]
    x = torch.full((B, L, 3, H, d), float("nan"), dtype=t.dtype, device="cuda")
    x[:, :, 1] = t.transpose(1, 2)
    return x[:, :, 1].transpose(1, 2)


def allowed(ref, mag, d, L, bf16_out, tensor_cores=True):
    hops = -(-L // 128)
    a = (d + 266 + hops) * U32 * mag
    if bf16_out:
        a = a + UBF * np.abs(ref) + ((UBF + UBF * UBF) * mag if tensor_cores else 0.0)
    else:
        a = a + 2.0 ** -26 * mag  # states of bf16 operands; fp32 ones keep the first term alone
    return a + 1e-37


def check(got, ref, mag, d, L, bf16_out, what, f32_operands=False):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    a = allowed(ref, mag, d, L, bf16_out)
    if f32_operands:
        a = (d + 266 + -(-L // 128)) * U32 * mag + 1e-37
    err = np.abs(got - ref)
    worst = float((err / a).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"
    rms = np.sqrt(np.mean(ref ** 2)) if ref.size else 0.0
    if ref.size >= 256:
        e = np.sqrt(np.mean(err ** 2))
        lim = 2 * np.sqrt(2 / 3) * UBF if bf16_out else 2.0 ** -19
        # values below 2^-126 = 1.2e-38 are not normal numbers of either type and flush to zero: the elementwise
        # bound's 1e-37 holds for the norm too (e^-100 times a product is of 1e-44, its fp32 value 0)
        assert e <= lim * rms + 1e-37, f"{what}: rms error {e / rms:.3g}"
    return worst


def pair_mag(x, h, interleaved, scale, rot_scale):
    """scale (|x1| + |x2|) of each element's pair (times rot_scale), scale |x| of unrotated columns."""
    m = np.abs(x) * scale
    if interleaved:
        s = m[..., 0:2 * h:2] + m[..., 1:2 * h:2]
        m[..., 0:2 * h:2] = m[..., 1:2 * h:2] = s * rot_scale
    else:
        s = m[..., :h] + m[..., h:2 * h]
        m[..., :h] = m[..., h:2 * h] = s * rot_scale
    return m


def rotary_allowed(ref, x, h, interleaved, scale, rot_scale, bf16):
    """An output x1 c - x2 s may cancel, so its error is relative to the pair, not to itself. sin and cos are
    within 2^-22 of their values (an fp32 argument in [-1, 1] half turns, rounded once: pi 2^-25, and the
    function's own rounding); their scale, the scales' product and the two products take one rounding each
    (6 x 2^-24 of the pair with the sum's); then one rounding of the result to its type."""
    mag = pair_mag(x, h, interleaved, scale, rot_scale)
    return (6 * U32 + 2.0 ** -22) * mag + (UBF if bf16 else U32) * np.abs(ref) * (1 + 2.0 ** -7) + 1e-37


def scan64(a, b, c, g, X=None, reverse=False, block=256):
    """The scan job of all four outputs in 64 bits, a block of tokens at a time (the oracle's recurrence takes one token
    at a time, too slow for long sequences; it pins this one): y_i = sum over j <= i (reverse: j >= i) of lambda^|i-j|
    (a_i . b_j) c_j + lambda^(distance to X) a_i X, and the X handed on. Torch tensors [B, H, L, d] on any device."""
    import torch
    a, b, c = (x.double().flip(2) if reverse else x.double() for x in (a, b, c))
    B, H, L, d = a.shape
    g = torch.as_tensor(np.asarray(g), dtype=torch.float64, device=a.device)[:, None]
    e0 = 0 if reverse else 1  # X is handed over before (reverse: after) the decay of the step it crosses
    pw = lambda n: torch.where(n == 0, torch.ones_like(g * n), torch.exp(g * n))
    X = torch.zeros(B, H, d, c.shape[-1], dtype=torch.float64, device=a.device) if X is None else X.double().clone()
    y = torch.empty(B, H, L, c.shape[-1], dtype=torch.float64, device=a.device)
    for t in range(0, L, block):
        n = min(block, L - t)
        r = torch.arange(n, device=a.device, dtype=torch.float64)
        x, z, w = a[:, :, t:t + n], b[:, :, t:t + n], c[:, :, t:t + n]
        gap = r[:, None] - r[None, :]
        D = torch.where(gap >= 0, pw(gap.clamp(min=0).reshape(-1)).reshape(H, n, n), torch.zeros((), dtype=torch.float64,
                                                                                                 device=a.device))
        y[:, :, t:t + n] = ((x @ z.transpose(-1, -2)) * D) @ w + pw(r + e0)[..., None] * (x @ X)
        X = pw(torch.full((1,), float(n), device=a.device, dtype=torch.float64))[..., None] * X \
            + (pw(n - r - e0)[..., None] * z).transpose(-1, -2) @ w
    return (y.flip(2) if reverse else y), X


def forward64(q, k, v, g, S=None):
    return scan64(q, k, v, g, S)


def backward64(q, k, v, g, do, S=None, dS=None):
    """(dq, dk, dv, dstate_in)."""
    T = lambda x: None if x is None else x.transpose(-1, -2)
    dq, _ = scan64(do, v, k, g, T(S))
    dk, _ = scan64(v, do, q, g, T(dS), reverse=True)
    dv, G = scan64(k, q, do, g, dS, reverse=True)
    return dq, dk, dv, G


def coarse_slope():
    """A log decay whose exp lies far from the fp32 values beside it: rounding it is off by a quarter of a step at least."""
    g = np.float32(-1e-3) - np.arange(200, dtype=np.float32) * np.float32(1e-6)
    lam = np.exp(g.astype(np.float64))
    off = np.abs(lam.astype(np.float32).astype(np.float64) / lam - 1)
    i = int(off.argmax())
    assert off[i] >= 2.0 ** -26
    return float(g[i])


def drift_allowed(steps):
    """The mean signed relative error of decaying elements, over many of them: each step rounds each once, by at most
    2^-24 and to either side, so one element has a standard deviation of sqrt(steps / 3) 2^-24 and the mean of N a
    sqrt(N)-th of it. A decay rounded to fp32 moves all elements to one side, steps times."""
    return np.sqrt(steps) * U32
