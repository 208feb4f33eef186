"""B200 (sm_100a) FAVOR attention forward pass: Python binding of libfavor.so.

The binding only marshals arguments. Every step of the computation runs in the CUDA kernels
of ``libfavor.so``, and PyTorch supplies device memory and streams. There is no CPU fallback:
if the library is missing or a call fails, an exception is raised.

Entry points mirror the C ABI in include/favor.h:
    favor_attention, favor_attention_chunked, favor_attention_f32, favor_orf_omega,
    favor_attention_host, favor_sync_status, favor_status_string, favor_workspace_bytes,
    favor_selftest_timeout, favor_selftest_sincos, favor_attention_f32_noalloc,
    favor_noalloc_scratch_bytes,
    favor_decode_state_bytes, favor_decode_init, favor_decode_step, favor_orf_omega_seeded,
    favor_orf_gaussians_seeded, favor_philox4x64, favor_attention_backward_f32,
    favor_decay_attention, favor_decay_attention_backward, favor_decay_step,
    favor_decay_workspace_bytes, favor_rotary, favor_rotary_frequencies
"""
from __future__ import annotations

import ctypes
import os

FAVOR_TRIG = 0
FAVOR_RELU = 1
FAVOR_ROTARY_PLAIN, FAVOR_ROTARY_LINEAR, FAVOR_ROTARY_BASE, FAVOR_ROTARY_PARTS = 0, 1, 2, 3
STATUS = {
    0: "FAVOR_OK", -1: "FAVOR_ERR_NULL", -2: "FAVOR_ERR_ALIGN", -3: "FAVOR_ERR_SHAPE",
    -4: "FAVOR_ERR_KIND", -5: "FAVOR_ERR_UNSUPPORTED", -6: "FAVOR_ERR_CUDA",
    -7: "FAVOR_ERR_TIMEOUT", -8: "FAVOR_ERR_DEVICE",
}
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfavor.so")

_vp, _i, _ll, _sz, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_uint64
_f, _d = ctypes.c_float, ctypes.c_double
_SIGS = {
    "favor_attention": (_i, [_vp] * 5 + [_i] * 7 + [_vp]),
    "favor_attention_chunked": (_i, [_vp] * 5 + [_i] * 8 + [_vp]),
    "favor_attention_f32": (_i, [_vp] * 5 + [_i] * 7 + [_vp]),
    "favor_orf_omega": (_i, [_vp] * 3 + [_i] * 4 + [_vp]),
    "favor_attention_host": (_i, [_vp] * 5 + [_i] * 8 + [_vp]),
    "favor_sync_status": (_i, [_vp]),
    "favor_status_string": (ctypes.c_char_p, [_i]),
    "favor_selftest_timeout": (_i, [_ll, _vp]),
    "favor_selftest_sincos": (_i, [_vp] * 3 + [_i, _vp]),
    "favor_workspace_bytes": (_sz, [_i] * 7),
    "favor_attention_f32_noalloc": (_i, [_vp] * 5 + [_i] * 7 + [_vp]),
    "favor_noalloc_scratch_bytes": (_sz, []),
    "favor_decode_state_bytes": (_sz, [_i] * 5),
    "favor_decode_init": (_i, [_vp] + [_i] * 5 + [_vp]),
    "favor_decode_step": (_i, [_vp] * 6 + [_i] * 5 + [_vp]),
    "favor_orf_omega_seeded": (_i, [_u64, _vp] + [_i] * 4 + [_vp]),
    "favor_orf_gaussians_seeded": (_i, [_u64, _vp, _vp] + [_i] * 3 + [_vp]),
    "favor_philox4x64": (_i, [_u64, _u64, _u64, _vp, _vp]),
    "favor_attention_backward_f32": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "favor_decay_attention": (_i, [_vp] * 8 + [_i] * 5 + [_vp, _vp]),
    "favor_decay_attention_backward": (_i, [_vp] * 12 + [_i] * 5 + [_vp, _vp]),
    "favor_decay_step": (_i, [_vp] * 6 + [_i] * 4 + [_vp, _vp]),
    "favor_decay_workspace_bytes": (_sz, [_i] * 6),
    "favor_rotary": (_i, [_vp] * 6 + [_i] * 9 + [_f, _f, _i, _vp, _vp]),
    "favor_rotary_frequencies": (_i, [_vp, _vp, _i, _d, _i] + [_d] * 4),
}
_LIB = None


class FavorError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({favor_status_string(code)})")


def lib() -> ctypes.CDLL:
    """Load libfavor.so (built in-tree). Raises ImportError if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m linear_kernelized_attention_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _LIB = L
    return _LIB


def favor_status_string(code: int) -> str:
    return lib().favor_status_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise FavorError(rc, where)


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check_qkv(q, k, v, omega, dtype):
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("omega", omega)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share the shape [B, H, L, d]")
    B, H, L, d = q.shape
    if omega.dim() != 3 or omega.shape[0] != H or omega.shape[2] != d:
        raise ValueError("omega must have shape [H, M, d]")
    return B, H, L, d, omega.shape[1]


def _check_out(out, like, name="out"):
    """An output tensor must match `like` in shape, dtype and device, and be contiguous: the C
    layer sees only a pointer and writes B*H*L*d elements through it."""
    import torch
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, dtype {like.dtype} and device "
                         f"{like.device}; got {tuple(out.shape)}, {out.dtype}, {out.device}")
    if not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def favor_attention(q, k, v, omega, out=None, feature_kind=FAVOR_TRIG, causal=False, chunk=0,
                    stream=None):
    """bf16 FAVOR forward. q, k, v: [B,H,L,d]; omega: [H,M,d]. Tensor-core kernels for the shapes
    they cover; other shapes up to d = 128, M = 512 run the fp32 CUDA-core kernels on widened
    copies (favor_attention in include/favor.h)."""
    import torch
    B, H, L, d, M = _check_qkv(q, k, v, omega, torch.bfloat16)
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    rc = lib().favor_attention_chunked(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                       out.data_ptr(), B, H, L, d, M, int(feature_kind), int(causal),
                                       int(chunk), _stream(stream))
    _check(rc, "favor_attention")
    return out


def favor_attention_chunked(q, k, v, omega, out=None, feature_kind=FAVOR_TRIG, causal=False,
                            chunk=0, stream=None):
    return favor_attention(q, k, v, omega, out, feature_kind, causal, chunk, stream)


def favor_attention_f32(q, k, v, omega, out=None, feature_kind=FAVOR_TRIG, causal=False,
                        stream=None):
    """fp32 FAVOR forward on the accuracy path."""
    import torch
    B, H, L, d, M = _check_qkv(q, k, v, omega, torch.float32)
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    rc = lib().favor_attention_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                   out.data_ptr(), B, H, L, d, M, int(feature_kind), int(causal),
                                   _stream(stream))
    _check(rc, "favor_attention_f32")
    return out


def _check_omega_out(out, H, M, d):
    import torch
    if not isinstance(out, torch.Tensor) or not out.is_cuda or not out.is_contiguous():
        raise TypeError("out must be a contiguous CUDA tensor")
    if tuple(out.shape) != (H, M, d) or out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out must have shape {(H, M, d)} and dtype float32 or bfloat16")


def favor_orf_omega(gauss_blocks, gauss_norms, M, dtype=None, out=None, stream=None):
    """Build ORF Omega [H, M, d] on the device from fp64 Gaussian draws (see include/favor.h)."""
    import torch
    dtype = dtype or torch.bfloat16
    H, nb, d, d2 = gauss_blocks.shape
    if d != d2 or gauss_norms.shape != (H, M, d) or nb != -(-M // d):
        raise ValueError("gauss_blocks must be [H, ceil(M/d), d, d] and gauss_norms [H, M, d]")
    for t in (gauss_blocks, gauss_norms):
        if t.dtype != torch.float64 or not t.is_cuda or not t.is_contiguous():
            raise TypeError("Gaussian draws must be contiguous float64 CUDA tensors")
    if out is None:
        out = torch.empty((H, M, d), dtype=dtype, device=gauss_blocks.device)
    _check_omega_out(out, H, M, d)
    code = {torch.float32: 0, torch.bfloat16: 1}[out.dtype]
    rc = lib().favor_orf_omega(gauss_blocks.data_ptr(), gauss_norms.data_ptr(), out.data_ptr(), H, M,
                               d, code, _stream(stream))
    _check(rc, "favor_orf_omega")
    return out


def favor_attention_host(q, k, v, omega, out, feature_kind=FAVOR_TRIG, causal=False, stream=None):
    """Host-buffer entry: q, k, v, omega, out are CPU tensors (pinned for async copies)."""
    import torch
    for t in (q, k, v, omega, out):
        if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_contiguous():
            raise TypeError("favor_attention_host takes contiguous CPU tensors")
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("favor_attention_host takes float32 or bfloat16 tensors")
    code = {torch.float32: 0, torch.bfloat16: 1}[q.dtype]
    if q.dim() != 4:
        raise ValueError("q must have shape [B, H, L, d]")
    B, H, L, d = q.shape
    for name, t in (("k", k), ("v", v), ("out", out)):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must match q in shape {tuple(q.shape)} and dtype {q.dtype}")
    if omega.dim() != 3 or omega.shape[0] != H or omega.shape[2] != d or omega.dtype != q.dtype:
        raise ValueError("omega must have shape [H, M, d] and q's dtype")
    M = omega.shape[1]
    rc = lib().favor_attention_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                    out.data_ptr(), B, H, L, d, M, int(feature_kind), int(causal),
                                    code, _stream(stream))
    _check(rc, "favor_attention_host")
    return out


def favor_sync_status(stream=None) -> int:
    return lib().favor_sync_status(_stream(stream))


def favor_workspace_bytes(B, H, L, d, M, feature_kind=FAVOR_TRIG, causal=False) -> int:
    return lib().favor_workspace_bytes(B, H, L, d, M, int(feature_kind), int(causal))


def favor_selftest_timeout(limit_cycles: int, stream=None) -> int:
    return lib().favor_selftest_timeout(int(limit_cycles), _stream(stream))


def favor_selftest_sincos(u, stream=None):
    """FMA-pipe (sin(u), cos(u)) of a contiguous float32 CUDA tensor, as two new tensors."""
    import torch
    if u.dtype != torch.float32 or not u.is_cuda or not u.is_contiguous():
        raise ValueError("u must be a contiguous float32 CUDA tensor")
    s, c = torch.empty_like(u), torch.empty_like(u)
    rc = lib().favor_selftest_sincos(u.data_ptr(), s.data_ptr(), c.data_ptr(), u.numel(), _stream(stream))
    if rc != 0:
        raise FavorError(rc, "favor_selftest_sincos")
    return s, c


def favor_attention_f32_noalloc(q, k, v, omega, out=None, feature_kind=FAVOR_TRIG, causal=False,
                                stream=None):
    """fp32 forward with its workspace in the library's static device array (no allocation by
    the library; `out` is allocated here only if not given). Calls that overlap in time race on
    the shared workspace: see include/favor.h."""
    import torch
    B, H, L, d, M = _check_qkv(q, k, v, omega, torch.float32)
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    rc = lib().favor_attention_f32_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                           out.data_ptr(), B, H, L, d, M, int(feature_kind), int(causal),
                                           _stream(stream))
    _check(rc, "favor_attention_f32_noalloc")
    return out


def favor_noalloc_scratch_bytes() -> int:
    return lib().favor_noalloc_scratch_bytes()


# ---------------------------------------------------------------- causal decode (carried state)
def favor_decode_state_bytes(B, H, d, M, feature_kind=FAVOR_TRIG) -> int:
    return lib().favor_decode_state_bytes(B, H, d, M, int(feature_kind))


def favor_decode_init(state, B, H, d, M, feature_kind=FAVOR_TRIG, stream=None):
    """Set `state` (a CUDA tensor of favor_decode_state_bytes bytes) to the empty state."""
    rc = lib().favor_decode_init(state.data_ptr(), B, H, d, M, int(feature_kind), _stream(stream))
    _check(rc, "favor_decode_init")
    return state


def favor_decode_new_state(B, H, d, M, feature_kind=FAVOR_TRIG, device="cuda", stream=None):
    """Allocate (with torch) and initialise an empty decode state: a flat float32 tensor."""
    import torch
    n = favor_decode_state_bytes(B, H, d, M, feature_kind)
    if n == 0:
        raise FavorError(-5, "favor_decode_state_bytes")
    state = torch.empty(n // 4, dtype=torch.float32, device=device)
    return favor_decode_init(state, B, H, d, M, feature_kind, stream)


def favor_decode_state_views(state, B, H, d, M, feature_kind=FAVOR_TRIG):
    """Views (S [B*H, F, d], z [B*H, F], c [B*H]) of a decode state, per include/favor.h."""
    F = 2 * M if feature_kind == FAVOR_TRIG else M
    BH = B * H
    S = state[:BH * F * d].view(BH, F, d)
    z = state[BH * F * d:BH * F * (d + 1)].view(BH, F)
    c = state[BH * F * (d + 1):BH * F * (d + 1) + BH]
    return S, z, c


def favor_decode_step(q, k, v, omega, state, out=None, feature_kind=FAVOR_TRIG, stream=None):
    """One causal decode step. q, k, v: [B, H, d] bf16 (one token per head); omega: [H, M, d]
    bf16; state: from favor_decode_new_state, updated in place. Returns out [B, H, d] bf16."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("omega", omega)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share the shape [B, H, d]")
    B, H, d = q.shape
    if omega.dim() != 3 or omega.shape[0] != H or omega.shape[2] != d:
        raise ValueError("omega must have shape [H, M, d]")
    M = omega.shape[1]
    need = favor_decode_state_bytes(B, H, d, M, feature_kind)
    if not state.is_cuda or state.numel() * state.element_size() < need:
        raise ValueError(f"state must be a CUDA tensor of at least {need} bytes")
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    rc = lib().favor_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                 state.data_ptr(), out.data_ptr(), B, H, d, M, int(feature_kind),
                                 _stream(stream))
    _check(rc, "favor_decode_step")
    return out


# ---------------------------------------------------------------- ORF redrawn from a seed
def favor_orf_omega_seeded(seed, H, M, d, dtype=None, out=None, device="cuda", stream=None):
    """ORF Omega [H, M, d] drawn on the device from `seed` (Philox4x64-10; see include/favor.h)."""
    import torch
    dtype = dtype or torch.bfloat16
    if out is None:
        out = torch.empty((H, M, d), dtype=dtype, device=device)
    _check_omega_out(out, H, M, d)
    code = {torch.float32: 0, torch.bfloat16: 1}[out.dtype]
    rc = lib().favor_orf_omega_seeded(int(seed) & (2**64 - 1), out.data_ptr(), H, M, d, code, _stream(stream))
    _check(rc, "favor_orf_omega_seeded")
    return out


def favor_orf_gaussians_seeded(seed, H, M, d, device="cuda", stream=None):
    """The draws behind favor_orf_omega_seeded: (G [H, ceil(M/d), d, d], R [H, M, d]) float64."""
    import torch
    nb = -(-M // d)
    G = torch.empty((H, nb, d, d), dtype=torch.float64, device=device)
    R = torch.empty((H, M, d), dtype=torch.float64, device=device)
    rc = lib().favor_orf_gaussians_seeded(int(seed) & (2**64 - 1), G.data_ptr(), R.data_ptr(), H, M, d,
                                          _stream(stream))
    _check(rc, "favor_orf_gaussians_seeded")
    return G, R


def favor_philox4x64(key, first_counter, n_blocks, device="cuda", stream=None):
    """Raw Philox4x64-10 blocks: an int64 tensor [n_blocks, 4] holding the uint64 words' bits."""
    import torch
    out = torch.empty((n_blocks, 4), dtype=torch.int64, device=device)
    rc = lib().favor_philox4x64(int(key) & (2**64 - 1), int(first_counter) & (2**64 - 1), int(n_blocks),
                                out.data_ptr(), _stream(stream))
    _check(rc, "favor_philox4x64")
    return out


# ---------------------------------------------------------------- backward
def favor_attention_backward_f32(q, k, v, omega, dout, feature_kind=FAVOR_TRIG, causal=False, stream=None):
    """fp32 gradients (dq, dk, dv) of sum(dout * out) for out = favor_attention_f32(q, k, v, omega)."""
    import torch
    B, H, L, d, M = _check_qkv(q, k, v, omega, torch.float32)
    if dout.shape != q.shape or dout.dtype != torch.float32 or not dout.is_cuda or not dout.is_contiguous():
        raise ValueError("dout must be a contiguous float32 CUDA tensor shaped like q")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    rc = lib().favor_attention_backward_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(), omega.data_ptr(),
                                            dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                            B, H, L, d, M, int(feature_kind), int(causal), _stream(stream))
    _check(rc, "favor_attention_backward_f32")
    return dq, dk, dv


# ---------------------------------------------------------------- linear attention with a decay
# A single-token call costs a few microseconds on the device, so the checks below stay on the few
# attributes that decide, and errors are worded only once one fails.
def _operands(shape, dtype, device, names, *ts):
    """Pointers of operands [B, H, L, d] (or [B, H, d]) read in place (any strides, d contiguous), and whether
    all are contiguous."""
    ptrs, whole, index = [], True, device.index
    try:
        for t in ts:
            if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
                break
            if not t.is_contiguous():
                whole = False
                if t.stride(-1) != 1 and shape[-1] > 1:
                    raise ValueError(f"{names[len(ptrs)]} must be contiguous in its last dimension")
            ptrs.append(t.data_ptr())
        else:
            return ptrs, whole
    except AttributeError:
        raise TypeError(f"{names[len(ptrs)]} must be a CUDA tensor") from None
    name = names[len(ptrs)]
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")


def _aux(name, t, shape, dtype, device):
    """A contiguous companion tensor (decays, lengths, states, positions), or None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == device.index:
            if t.shape == shape and t.is_contiguous():
                return t.data_ptr()
            raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")
    except AttributeError:
        pass
    raise TypeError(f"{name} must be a {dtype} tensor on {device}")


def _strides(*ts):
    """favor_strides of the operands."""
    a = []
    for t in ts:
        a += (0, 0, 0) if t is None else (*t.stride()[:-1], 0)[:3]
    return (_ll * len(a))(*a)


def _dims(shape):
    """Sizes as the C layer takes them (int)."""
    if max(shape) > 0x7fffffff:
        raise ValueError(f"a dimension of {tuple(shape)} exceeds 2^31 - 1")
    return shape


def _first(name, t, dims):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dt = t.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dt}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have shape {'[B, H, L, d]' if dims == 4 else '[B, H, d]'}")
    return 1 if dt is torch.bfloat16 else 0


def _elsewhere(device, stream):
    """A context that makes `stream` (a stream or its handle; None: the device's current one) and the device of
    the call's tensors current, or None where they are. Tensors made inside belong to that stream."""
    import torch
    if stream is None:
        if torch._C._cuda_getDevice() == device.index:
            return None
        return torch.cuda.device(device)
    if isinstance(stream, int):  # 0 is the default stream; torch would wrap it as a new stream of its pool
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    return torch.cuda.stream(stream)


def _handle(device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _new(like, zero):
    import torch
    make = torch.zeros_like if zero else torch.empty_like
    return make(like) if like.is_contiguous() else make(like, memory_format=torch.contiguous_format)


def favor_decay_attention(q, k, v, log_decay, state=None, lengths=None, out=None, state_out=None,
                          return_state=False, stream=None):
    """Causal linear attention with a decay per head: S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,
    out_t = S_t^T q_t (favor_decay_attention in include/favor.h). q, k, v: [B, H, L, d] bf16 or float32,
    any strides with d contiguous (a tensor whose rows are whole 16-byte pieces starts on one); log_decay: float32 [H]; state: float32 [B, H, d, d] carried in, or
    None; lengths: int32 [B] or None. Returns out, or (out, state_out) where return_state is true or
    state_out is given. Rows past a sequence's length are left as they were in a given `out`, and zero
    in a new one. state_out may be `state`."""
    import torch
    code = _first("q", q, 4)
    dev = q.device
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return favor_decay_attention(q, k, v, log_decay, state, lengths, out, state_out, return_state)
    shape, dt = q.shape, q.dtype
    B, H, L, d = _dims(shape)
    if log_decay is None:
        raise TypeError("log_decay must be a float32 tensor")
    g = _aux("log_decay", log_decay, (H,), torch.float32, dev)
    s_in = _aux("state", state, (B, H, d, d), torch.float32, dev)
    n = _aux("lengths", lengths, (B,), torch.int32, dev)
    if out is None:
        out = _new(q, lengths is not None)
    (pq, pk, pv, po), whole = _operands(shape, dt, dev, ("q", "k", "v", "out"), q, k, v, out)
    if state_out is None and return_state:
        state_out = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
    s_out = _aux("state_out", state_out, (B, H, d, d), torch.float32, dev)
    rc = lib().favor_decay_attention(pq, pk, pv, g, s_in, n, po, s_out, B, H, L, d, code,
                                     None if whole else _strides(q, k, v, out), _handle(dev))
    if rc != 0:
        raise FavorError(rc, "favor_decay_attention")
    return out if state_out is None else (out, state_out)


def favor_decay_attention_backward(q, k, v, log_decay, dout, state=None, dstate=None, lengths=None, dq=None, dk=None,
                                   dv=None, dstate_in=None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out) + sum(dstate * state_out) for the outputs of
    favor_decay_attention on the same arguments; with `state`, `dstate` or `dstate_in` given, (dq, dk, dv,
    dstate_in). dstate: float32 [B, H, d, d] or None (zeros). Rows past a sequence's length are left
    as they were in given outputs, and zero in new ones. log_decay gets no gradient."""
    import torch
    code = _first("q", q, 4)
    dev = q.device
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return favor_decay_attention_backward(q, k, v, log_decay, dout, state, dstate, lengths, dq, dk, dv,
                                                  dstate_in)
    shape, dt = q.shape, q.dtype
    B, H, L, d = _dims(shape)
    if log_decay is None:
        raise TypeError("log_decay must be a float32 tensor")
    g = _aux("log_decay", log_decay, (H,), torch.float32, dev)
    s_in = _aux("state", state, (B, H, d, d), torch.float32, dev)
    ds = _aux("dstate", dstate, (B, H, d, d), torch.float32, dev)
    n = _aux("lengths", lengths, (B,), torch.int32, dev)
    zero = lengths is not None
    dq, dk, dv = (_new(q, zero) if t is None else t for t in (dq, dk, dv))
    (pq, pk, pv, pdo, pdq, pdk, pdv), whole = _operands(shape, dt, dev, ("q", "k", "v", "dout", "dq", "dk", "dv"),
                                                        q, k, v, dout, dq, dk, dv)
    if dstate_in is None and (state is not None or dstate is not None):
        dstate_in = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
    ds_in = _aux("dstate_in", dstate_in, (B, H, d, d), torch.float32, dev)
    rc = lib().favor_decay_attention_backward(
        pq, pk, pv, g, s_in, n, pdo, ds, pdq, pdk, pdv, ds_in, B, H, L, d, code,
        None if whole else _strides(q, k, v, dout, dq, dk, dv), _handle(dev))
    if rc != 0:
        raise FavorError(rc, "favor_decay_attention_backward")
    return (dq, dk, dv) if dstate_in is None else (dq, dk, dv, dstate_in)


def favor_decay_step(q, k, v, log_decay, state, out=None, stream=None):
    """One token per head against the carried state, updated in place: S = exp(log_decay[h]) S + k v^T,
    out = S^T q. q, k, v: [B, H, d] bf16 or float32 (slices of fused projections are read in place, strides and
    alignment as for favor_decay_attention); state: float32 [B, H, d, d]. Returns out [B, H, d]."""
    import torch
    code = _first("q", q, 3)
    dev = q.device
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return favor_decay_step(q, k, v, log_decay, state, out)
    shape, dt = q.shape, q.dtype
    B, H, d = _dims(shape)
    if log_decay is None or state is None:
        raise TypeError("log_decay and state must be float32 tensors")
    g = _aux("log_decay", log_decay, (H,), torch.float32, dev)
    s = _aux("state", state, (B, H, d, d), torch.float32, dev)
    if out is None:
        out = _new(q, False)
    (pq, pk, pv, po), whole = _operands(shape, dt, dev, ("q", "k", "v", "out"), q, k, v, out)
    rc = lib().favor_decay_step(pq, pk, pv, g, s, po, B, H, d, code, None if whole else _strides(q, k, v, out),
                                _handle(dev))
    if rc != 0:
        raise FavorError(rc, "favor_decay_step")
    return out


def favor_decay_workspace_bytes(B, H, L, d, dtype_code=1, backward=False) -> int:
    if max(B, H, L, d) > 0x7fffffff:
        return 0  # not a size the calls take
    return lib().favor_decay_workspace_bytes(B, H, L, d, int(dtype_code), int(backward))


# ---------------------------------------------------------------- rotary positions
def favor_rotary_frequencies(rot, base=10000.0, scaling=FAVOR_ROTARY_PLAIN, factor=1.0, trained_length=0,
                             beta_fast=32.0, beta_slow=1.0, device=None):
    """(freq, rot_scale): float64 [rot/2] radians per position, on `device` (CPU if None), and the scale of
    the rotated columns to pass to favor_rotary. Scalings: favor_rotary_frequencies in include/favor.h."""
    import torch
    _dims((rot,))
    freq = torch.empty(max(int(rot) // 2, 1), dtype=torch.float64)
    rs = ctypes.c_double(1.0)
    rc = lib().favor_rotary_frequencies(freq.data_ptr(), ctypes.addressof(rs), int(rot), float(base), int(scaling),
                                        float(factor), float(trained_length), float(beta_fast), float(beta_slow))
    _check(rc, "favor_rotary_frequencies")
    return (freq if device is None else freq.to(device)), rs.value


def favor_rotary(q, k, freq, positions=None, first_position=0, interleaved=False, inverse=False, scale=1.0,
                 rot_scale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [B, Hq, L, d] and k [B, Hk, L, d] (or None) in one launch: the first
    2 len(freq) columns turn by positions * freq, all are multiplied by `scale`, the rotated ones by
    rot_scale too. Strides and alignment as for favor_decay_attention. freq: float64 [rot/2]; positions: int32 [B, L], or None for first_position + t.
    inverse=True is the gradient of the same call. q_out / k_out may be q / k (in place). Returns
    (q_out, k_out)."""
    import torch
    code = _first("q", q, 4)
    dev = q.device
    on = _elsewhere(dev, stream)
    if on is not None:
        with on:
            return favor_rotary(q, k, freq, positions, first_position, interleaved, inverse, scale, rot_scale, q_out,
                                k_out)
    shape, dt = q.shape, q.dtype
    B, Hq, L, d = _dims(shape)
    Hk, pk, pko, wk = 0, None, None, True
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise TypeError("k must be a CUDA tensor of shape [B, Hk, L, d]")
        Hk = _dims(k.shape)[1]
        if k_out is None:
            k_out = _new(k, False)
        (pk, pko), wk = _operands((B, Hk, L, d), dt, dev, ("k", "k_out"), k, k_out)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if not -0x80000000 <= first_position <= 0x7fffffff:
        raise ValueError("first_position must fit 32 bits")
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise TypeError("freq must be a float64 tensor of shape [rot/2]")
    (rot,) = _dims((2 * freq.shape[0],))
    f = _aux("freq", freq, freq.shape, torch.float64, dev)
    pos = _aux("positions", positions, (B, L), torch.int32, dev)
    if q_out is None:
        q_out = _new(q, False)
    (pq, pqo), wq = _operands(shape, dt, dev, ("q", "q_out"), q, q_out)
    rc = lib().favor_rotary(pq, pk, f, pos, pqo, pko, B, Hq, Hk, L, d, rot, int(interleaved), int(inverse),
                            int(first_position), scale, rot_scale, code,
                            None if wq and wk else _strides(q, k, q_out, k_out), _handle(dev))
    if rc != 0:
        raise FavorError(rc, "favor_rotary")
    return q_out, k_out
