"""The calls around the expert FFN refuse bad arguments on the host, before
anything is launched (no GPU is touched: the addresses are never read)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def m():
    from moe_expert_layer_02_gb300 import build
    build.build()
    import moe_expert_layer_02_gb300 as mm
    mm.load_library()
    return mm


def P(v):
    return ctypes.c_void_p(v)


A = P(4096)  # an aligned address; never dereferenced
BIG = 1 << 40


def calls(m, T=4, H=64, E=8, k=2, dtype=0, nH=None, eps=1e-6):
    """name -> (function, description, positional tensor arguments, has workspace)."""
    lib = m.load_library()
    r, n = m.make_rows(T, H, E, k, dtype), m.make_norm(T, nH or H, dtype, eps)
    return {
        "dispatch": (lib.moe_dispatch, r, [A, A, None, A, A, A, A, A, None], True),
        "dispatch_backward": (lib.moe_dispatch_backward, r, [A, A, None, A], False),
        "combine": (lib.moe_combine, r, [A, A, A, None, A], False),
        "combine_backward": (lib.moe_combine_backward, r, [A] * 7, False),
        "add_rmsnorm": (lib.moe_add_rmsnorm, n, [A, None, A, None, A, None, None], False),
        "add_rmsnorm_backward": (lib.moe_add_rmsnorm_backward, n, [A, A, A, None, A, A], True),
    }


def call(entry, args=None, ws=A, ws_bytes=BIG, desc=True):
    fn, d, tensors, has_ws = entry
    args = tensors if args is None else args
    return fn(ctypes.byref(d) if desc else None, *args, *([ws, ws_bytes] if has_ws else []), None)


NAMES = ("dispatch", "dispatch_backward", "combine", "combine_backward", "add_rmsnorm",
         "add_rmsnorm_backward")
# arguments that may be NULL in the lists above, by position
OPTIONAL = {"dispatch": {2, 8}, "dispatch_backward": {2}, "combine": {3}, "combine_backward": set(),
            "add_rmsnorm": {1, 3, 5, 6}, "add_rmsnorm_backward": {3, 5}}


@pytest.mark.parametrize("name", NAMES)
def test_descriptions(m, name):
    assert call(calls(m)[name], desc=False) == INVALID
    for bad in (dict(T=-1), dict(H=0), dict(H=(1 << 20) + 1), dict(dtype=4), dict(dtype=-1)):
        assert call(calls(m, **bad)[name]) == INVALID, bad
    if "norm" in name:
        for eps in (-1e-6, float("nan"), float("inf")):
            assert call(calls(m, eps=eps)[name]) == INVALID
    else:
        for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(T=(1 << 30) // 2 + 1)):
            assert call(calls(m, **bad)[name]) == INVALID, bad
    if name != "dispatch":  # 8-bit rows are moved, not summed
        assert call(calls(m, dtype=3)[name]) == UNSUPPORTED


@pytest.mark.parametrize("name", NAMES)
def test_null_and_misaligned_pointers(m, name):
    for dtype in (0, 2):
        entry = calls(m, dtype=dtype)[name]
        for i, v in enumerate(entry[2]):
            if v is not None and i not in OPTIONAL[name]:
                args = list(entry[2])
                args[i] = None
                assert call(entry, args) == INVALID, i
            # one byte off no element's boundary holds (the codes q alone are bytes)
            args = list(entry[2])
            args[i] = P(4097)
            if name == "dispatch" and i in (2, 8):
                args[2], args[8] = (P(4097), A) if i == 2 else (A, P(4097))
            if name == "add_rmsnorm" and i in (5, 6):
                args[5], args[6] = A, P(4097)
            assert call(entry, args) == INVALID, i


def test_dispatch_scales_come_in_pairs(m):
    for dtype in range(4):
        entry = calls(m, dtype=dtype)["dispatch"]
        for x_scale, scale_rows in ((A, None), (None, A)):
            args = list(entry[2])
            args[2], args[8] = x_scale, scale_rows
            assert call(entry, args) == INVALID
    assert call(calls(m, dtype=3)["dispatch"]) == INVALID  # 8-bit rows need theirs


def test_norm_outputs(m):
    entry = calls(m)["add_rmsnorm"]
    for y, q, s in ((None, None, None), (A, A, None), (A, None, A), (None, A, None)):
        args = list(entry[2])
        args[4:] = [y, q, s]
        assert call(entry, args) == INVALID


@pytest.mark.parametrize("name", ("dispatch", "add_rmsnorm_backward"))
def test_workspaces(m, name):
    need = (m.moe_rows_workspace_bytes(m.make_rows(4, 64, 8, 2)) if name == "dispatch"
            else m.moe_norm_workspace_bytes(m.make_norm(4, 64)))
    assert need > 0
    entry = calls(m)[name]
    assert call(entry, ws=None) == WORKSPACE
    assert call(entry, ws=P(4096 + 128)) == WORKSPACE
    assert call(entry, ws_bytes=need - 1) == WORKSPACE
    assert m.moe_rows_workspace_bytes(m.make_rows(4, 64, 8, 33)) == 0
    assert m.moe_norm_workspace_bytes(m.make_norm(4, 0)) == 0


def test_route_backward(m):
    lib = m.load_library()
    p = m.make_problem(4, 128, 128, 8, 2)
    args = [None, A, A, A, A]
    assert lib.moe_route_backward(None, *args, None) == INVALID
    assert lib.moe_route_backward(ctypes.byref(m.make_problem(4, 128, 128, 8, 9)), *args, None) == INVALID
    for i in range(1, 5):
        for v in (None, P(4098)):
            bad = list(args)
            bad[i] = v
            assert lib.moe_route_backward(ctypes.byref(p), *bad, None) == INVALID
    s = m.make_problem(4, 128, 128, 8, 2, flags=m.F_SIGMOID_ROUTING)
    assert lib.moe_route_backward(ctypes.byref(s), *args, None) == INVALID  # needs the logits


def test_empty_calls_are_no_ops(m):
    c = calls(m, T=0)
    for name in ("dispatch_backward", "combine", "combine_backward", "add_rmsnorm"):
        assert call(c[name], [None] * len(c[name][2])) == 0, name
    # without dgamma there is nothing to set to zero
    assert call(c["add_rmsnorm_backward"], [None] * 6, ws=None, ws_bytes=0) == 0
    p = m.make_problem(0, 128, 128, 8, 2)
    assert m.load_library().moe_route_backward(ctypes.byref(p), *[None] * 5, None) == 0


def test_binding_checks_types_sizes_and_layout(m):
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    r = m.make_rows(4, 64, 8, 2, bf)
    rows, perm, w, out = (torch.empty(8, 64, dtype=bf), torch.zeros(4, 2, dtype=i32),
                          torch.zeros(4, 2), torch.empty(4, 64, dtype=bf))
    for bad in ((rows.float(), perm, w, None, out), (rows, perm.long(), w, None, out),
                (rows, perm, w.double(), None, out), (rows[:7], perm, w, None, out),
                (rows, perm, w, None, torch.empty(64, 4, dtype=bf).t()), (rows, perm, w, out[:3], out),
                (rows, perm, w, None, out)):  # the last: not on the device
        with pytest.raises(ValueError):
            m.moe_combine(r, *bad, stream=0)
    with pytest.raises(ValueError):
        m.make_rows(4, 64, 8, 2, torch.float64)
    n = m.make_norm(4, 64, f32)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(n, torch.empty(4, 64), None, torch.empty(32), None, torch.empty(4, 64),
                          None, None, stream=0)


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_current_stream_without_the_private_lookup(m, monkeypatch, missing):
    # every entry point takes the current stream; torch's private names for it may go
    stream = type("Stream", (), {"cuda_stream": 0x1230})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: stream)
    monkeypatch.delattr(torch._C, missing)
    monkeypatch.setattr(m, "_stream_of", None)
    monkeypatch.setattr(m, "_device", None)
    assert m._stream(None) == 0x1230
    stream.cuda_stream = 0x4560  # looked up at every call
    assert m._stream(None) == 0x4560
    assert m._stream(stream) == 0x4560 and m._stream(0x20) == 0x20


def test_current_stream_by_the_private_lookup(m, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x100 + d, raising=False)
    monkeypatch.setattr(m, "_stream_of", None)
    monkeypatch.setattr(m, "_device", None)
    assert m._stream(None) == 0x103
