"""Host checks of the decayed linear attention and rotary entry points: bad arguments are refused before any
CUDA call (the pointers are made up and never read)."""
import ctypes

import pytest

import linear_kernelized_attention_b200 as F

vp = ctypes.c_void_p


def _strides(rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


def _attend(**o):
    a = dict(q=16, k=32, v=48, g=64, s_in=0, n=0, out=80, s_out=0, B=2, H=2, L=8, d=64, dt=1, st=None)
    a.update(o)
    return F.lib().favor_decay_attention(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["g"]), vp(a["s_in"]), vp(a["n"]),
                                         vp(a["out"]), vp(a["s_out"]), a["B"], a["H"], a["L"], a["d"], a["dt"],
                                         a["st"], None)


OK = (1024, 512, 64)
COMMON = [
    ({"q": 0}, -1), ({"k": 0}, -1), ({"v": 0}, -1), ({"g": 0}, -1),
    ({"k": 34}, -2), ({"g": 66}, -2),
    ({"B": 0}, -3), ({"H": -1}, -3), ({"d": 0}, -3), ({"B": 1 << 20, "H": 1 << 20}, -3),
    ({"d": 129}, -5), ({"dt": 2}, -5), ({"dt": -1}, -5),
]


@pytest.mark.parametrize("over,code", COMMON + [
    ({"out": 0}, -1), ({"s_in": 20}, -2), ({"s_out": 8}, -2), ({"n": 3}, -2), ({"out": 16}, -5), ({"out": 48}, -5),
    ({"L": 0}, -3),
    ({"st": [OK, OK, OK, (1024, 512, 32)]}, -3),     # rows of the output overlap
    ({"st": [OK, OK, OK, (1024, 0, 64)]}, -3),       # heads of the output overlap
    ({"st": [OK, OK, OK, (512, 512, 64)]}, -3),
    ({"st": [OK, (-1024, 512, 64), OK, OK]}, -3),
    ({"st": [OK, OK, (1 << 43, 512, 64), OK]}, -3),
])
def test_attention_refuses(over, code):
    if isinstance(over.get("st"), list):
        over = dict(over, st=_strides(over["st"]))
    assert _attend(**over) == code


def _backward(**o):
    a = dict(q=16, k=32, v=48, g=64, s_in=0, n=0, do=80, ds=0, dq=96, dk=112, dv=128, ds_in=0, B=2, H=2, L=8, d=64,
             dt=1, st=None)
    a.update(o)
    return F.lib().favor_decay_attention_backward(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["g"]), vp(a["s_in"]), vp(a["n"]), vp(a["do"]), vp(a["ds"]),
        vp(a["dq"]), vp(a["dk"]), vp(a["dv"]), vp(a["ds_in"]), a["B"], a["H"], a["L"], a["d"], a["dt"], a["st"], None)


@pytest.mark.parametrize("over,code", COMMON + [
    ({"do": 0}, -1), ({"dq": 0}, -1), ({"dk": 0}, -1), ({"dv": 0}, -1), ({"ds": 4}, -2), ({"ds_in": 24}, -2),
    ({"L": 0}, -3), ({"dq": 16}, -5), ({"dk": 96}, -5), ({"dv": 112}, -5), ({"dv": 80}, -5),
    ({"s_in": 160, "ds_in": 160}, -5),  # dstate_in over the state still being read
    ({"st": [OK] * 6 + [(1024, 512, 0)]}, -3), ({"st": [OK] * 4 + [(0, 512, 64)] + [OK] * 2}, -3),
])
def test_backward_refuses(over, code):
    if isinstance(over.get("st"), list):
        over = dict(over, st=_strides(over["st"]))
    assert _backward(**over) == code


def _step(**o):
    a = dict(q=16, k=32, v=48, g=64, s=80, out=96, B=2, H=2, d=64, dt=1, st=None)
    a.update(o)
    return F.lib().favor_decay_step(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["g"]), vp(a["s"]), vp(a["out"]), a["B"],
                                    a["H"], a["d"], a["dt"], a["st"], None)


@pytest.mark.parametrize("over,code", COMMON + [
    ({"s": 0}, -1), ({"out": 0}, -1), ({"s": 84}, -2), ({"out": 16}, -5),
    ({"st": [OK, OK, OK, (64, 64, 0)]}, -3),
])
def test_step_refuses(over, code):
    if isinstance(over.get("st"), list):
        over = dict(over, st=_strides(over["st"]))
    assert _step(**over) == code


def _rotary(**o):
    a = dict(q=16, k=32, f=64, n=0, qo=80, ko=96, B=2, Hq=2, Hk=1, L=8, d=64, rot=32, dt=1, st=None)
    a.update(o)
    return F.lib().favor_rotary(vp(a["q"]), vp(a["k"]), vp(a["f"]), vp(a["n"]), vp(a["qo"]), vp(a["ko"]), a["B"],
                                a["Hq"], a["Hk"], a["L"], a["d"], a["rot"], 0, 0, 0, 1.0, 1.0, a["dt"], a["st"], None)


@pytest.mark.parametrize("over,code", [
    ({"q": 0}, -1), ({"k": 0}, -1), ({"f": 0}, -1), ({"qo": 0}, -1), ({"ko": 0}, -1),
    ({"q": 18}, -2), ({"ko": 97}, -2), ({"f": 68}, -2), ({"n": 6}, -2),
    ({"B": 0}, -3), ({"Hq": 0}, -3), ({"Hk": -1}, -3), ({"L": -2}, -3), ({"rot": 0}, -3), ({"rot": 7}, -3),
    ({"rot": 66}, -3), ({"dt": 3}, -5), ({"Hq": 65535}, -5),
    ({"qo": 32}, -5), ({"ko": 16}, -5), ({"ko": 80}, -5),
    ({"st": [OK, OK, (1024, 512, 0), OK]}, -3),
    ({"qo": 16, "st": [OK, OK, (2048, 1024, 128), OK]}, -5),  # in place with other strides
])
def test_rotary_refuses(over, code):
    if isinstance(over.get("st"), list):
        over = dict(over, st=_strides(over["st"]))
    assert _rotary(**over) == code


def test_workspace_is_host_only():
    assert F.favor_decay_workspace_bytes(1, 1, 0, 64) == 0
    assert F.favor_decay_workspace_bytes(1, 1, 8, 129) == 0
    assert F.favor_decay_workspace_bytes(1, 1, 8, 64, 2) == 0
    assert F.favor_decay_workspace_bytes(2, 3, 1000, 40, 0) > 0
    assert F.favor_decay_workspace_bytes(2, 3, 1000, 40, 0, True) >= F.favor_decay_workspace_bytes(2, 3, 1000, 40, 0)


def test_binding_refuses_sizes_past_int():
    with pytest.raises(ValueError):
        F._dims((1, 1, 2 ** 32 + 5, 8))
    assert F._dims((2, 3, 2 ** 31 - 1, 8)) == (2, 3, 2 ** 31 - 1, 8)


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(1, 1, 4, 8)
    g = torch.zeros(1)
    with pytest.raises(TypeError):
        F.favor_decay_attention(x, x, x, g)
    with pytest.raises(TypeError):
        F.favor_decay_attention_backward(x, x, x, g, x)
    with pytest.raises(TypeError):
        F.favor_decay_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, torch.zeros(1, 1, 8, 8))
    with pytest.raises(TypeError):
        F.favor_rotary(x, x, torch.zeros(4, dtype=torch.float64))


def test_stream_handle_zero_is_the_default_stream(monkeypatch):
    """torch.cuda.current_stream().cuda_stream is 0 on the default stream; wrapped as an external stream, 0 gives
    another stream of torch's pool, which runs beside the caller's work."""
    import types

    import torch
    dev = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: types.SimpleNamespace(device=device, of=h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: types.SimpleNamespace(device=device, of="default"))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert F._elsewhere(dev, 0).of == "default"
    assert F._elsewhere(dev, 64).of == 64


def test_every_entry_refuses_sizes_past_int(monkeypatch):
    """The C layer takes int: 2^32 + 5 would arrive as 5, and most of the batch would be left out without a word.
    Expanded tensors without storage stand in for the operands; the checks before the sizes are let through."""
    import torch
    monkeypatch.setattr(F, "_first", lambda name, t, dims: 1)
    monkeypatch.setattr(F, "_elsewhere", lambda device, stream: None)
    big, none = 2 ** 32 + 5, torch.empty(1, device="meta")
    x = torch.empty(1, 1, 8, device="meta", dtype=torch.bfloat16)
    for shape in ((big, 1, 8), (1, big, 8)):
        t = x.expand(shape)
        with pytest.raises(ValueError, match="exceeds 2"):
            F.favor_decay_step(t, t, t, none, none)
    q = x[:, :, None]
    for shape in ((1, big, 1, 8), (big, 1, 1, 8)):
        with pytest.raises(ValueError, match="exceeds 2"):
            F.favor_rotary(q, q.expand(shape), torch.empty(4, device="meta", dtype=torch.float64))
    with pytest.raises(ValueError, match="exceeds 2"):
        F.favor_rotary(q, None, torch.empty(2 ** 31 + 4, device="meta", dtype=torch.float64))
    with pytest.raises(ValueError, match="exceeds 2"):
        F.favor_rotary_frequencies(2 ** 32 + 8)
    assert F.favor_decay_workspace_bytes(1, 1, big, 64) == 0 == F.favor_decay_workspace_bytes(big, 1, 8, 64, 0)


# operands that are not whole 16-byte pieces need their element's alignment alone: the call gets as far as the
# output that is an input (-5), which the host refuses before any CUDA call
@pytest.mark.parametrize("dt,off,d,st,code", [
    (1, 2, 20, None, -5), (1, 8, 33, None, -5), (1, 1, 20, None, -2), (0, 4, 33, None, -5), (0, 2, 33, None, -2),
    (1, 2, 64, None, -2), (0, 4, 64, None, -2),                           # whole pieces: as before
    (1, 2, 64, (1028, 512, 64), -5), (0, 4, 64, (1026, 512, 64), -5),    # rows of whole pieces, odd strides
])
def test_alignment_follows_the_rows(dt, off, d, st, code):
    o = dict(q=4096 + off, k=8192 + off, v=12288 + off, out=4096 + off, d=d, dt=dt)
    n = lambda i: None if st is None else _strides([st] * i)
    assert _attend(**o, st=n(4)) == code
    assert _step(**o, st=n(4)) == code
    g = dict(q=4096 + off, k=8192 + off, v=12288 + off, do=16384 + off, dq=4096 + off, dk=20480 + off, dv=24576 + off)
    assert _backward(**g, d=d, dt=dt, st=n(7)) == code
    r = dict(q=4096 + off, k=8192 + off, qo=12288 + off, ko=4096 + off, d=d, rot=16, dt=dt)
    assert _rotary(**r, st=n(4)) == code


def test_states_stay_on_16_bytes():
    assert _attend(d=20, s_in=20) == -2 and _attend(d=33, s_out=40) == -2
    assert _step(d=33, s=84) == -2
    assert _backward(d=20, ds=4) == -2 and _backward(d=20, ds_in=24) == -2
