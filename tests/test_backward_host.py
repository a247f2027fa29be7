"""Backward pass without a GPU: the oracle against differences of the layer as
a function, the 8-bit form against its stated bounds, sizes, and every refusal
(validation returns before any HIP call)."""
import ctypes
import os

import numpy as np
import pytest

from grouped_gemm_gemv_amd import _lib
from grouped_gemm_gemv_amd._lib import MoeBackwardSizes, MoeDispatch, MoeSaved8, MoeShape
from oracle import backward as B
from oracle import moe_oracle as O

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmoe.so not built")


def _rows(ids, E, capacity=0):
    d = O.dispatch(ids, E, capacity, 16)
    T, k = ids.shape
    R = d["token_of"].shape[0]
    entry_of, expert_of = np.full(R, -1), np.full(R, -1)
    for f, r in enumerate(d["row_of"]):
        entry_of[r], expert_of[r] = f, ids.reshape(-1)[f]
    return d, entry_of, expert_of


@pytest.mark.parametrize("capacity", [0, 2])
def test_oracle_gradients_match_differences(capacity):
    rng = np.random.default_rng(3)
    T, d, E, k, F = 5, 6, 4, 2, 16
    x, dout = rng.standard_normal((2, T, d))
    wr, bias = rng.standard_normal((E, d)), rng.standard_normal(E)
    wg, wu = rng.standard_normal((2, E, F, d)) * 0.5
    wd = rng.standard_normal((E, d, F)) * 0.5
    ids = np.argsort(-(x @ wr.T + bias), axis=1)[:, :k]
    disp, entry_of, expert_of = _rows(ids, E, capacity)

    def loss(x=x, wr=wr, bias=bias, wg=wg, wu=wu, wd=wd):
        return (B.layer(x, ids, lambda v: v @ wr.T + bias, wg, wu, wd) * dout).sum()

    z = np.take_along_axis(x @ wr.T + bias, ids, axis=1)
    w = np.exp(z) / np.exp(z).sum(axis=1, keepdims=True)
    R = disp["token_of"].shape[0]
    g, u, y = np.zeros((R, F)), np.zeros((R, F)), np.zeros((R, d))
    for r in np.flatnonzero(expert_of >= 0):
        e, t = expert_of[r], disp["token_of"][r]
        g[r], u[r] = wg[e] @ x[t], wu[e] @ x[t]
        y[r] = wd[e] @ (g[r] / (1 + np.exp(-g[r])) * u[r])
    got = B.ffn_backward(x, dout, w, wg, wu, wd, g, u, disp["token_of"], entry_of, expert_of, "f32")
    # the routing weights' gradient by the other route, <dout, y>
    _, _, dw_y, _ = B.combine_backward(dout, y, w, disp["row_of"], "f32")
    dw = got["dw"][0].reshape(T, k)
    assert np.allclose(dw, dw_y, rtol=1e-10, atol=1e-12)
    (dxr, _), (dwr, _), (db, _) = B.route_backward(x, wr, ids, w, dw, "f32")
    dx = B.permute_backward(got["dx_perm"][0], disp["row_of"], T, k, "f32")[0] + dxr
    for name, val, grad in (("x", x, dx), ("wr", wr, dwr), ("bias", bias, db), ("wg", wg, got["dwg"][0]),
                            ("wu", wu, got["dwu"][0]), ("wd", wd, got["dwd"][0])):
        flat = val.reshape(-1)
        for i in rng.choice(flat.size, min(flat.size, 12), replace=False):
            h = 1e-5
            hi, lo = val.copy(), val.copy()
            hi.reshape(-1)[i] += h
            lo.reshape(-1)[i] -= h
            diff = (loss(**{name: hi}) - loss(**{name: lo})) / (2 * h)
            # central differences: h^2 times a third derivative of order 100, and 1e-16 / h of rounding
            assert abs(diff - grad.reshape(-1)[i]) <= 1e-7 * max(1.0, abs(diff)), (name, i)


def test_eight_bit_form_error_and_exactness():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((64, 64)).astype(np.float32).astype(np.float64)
    v *= 2.0 ** rng.integers(-60, 60, (64, 1))
    v[3, :16] = 0.0
    v[4, 5] = v[4, :16].max() * 255.9  # one value dominates its block
    codes, b = B.pack8(v)
    back = B.value8(codes, b)
    step = np.repeat(2.0 ** (b.astype(np.float64) - 133), 16, axis=-1)
    full = np.abs(codes.astype(int)) == 127
    assert (np.abs(back - v) <= np.where(full, 1.0, 0.5) * step).all()
    assert (np.abs(back - v) <= np.repeat(np.abs(v).reshape(64, 4, 16).max(-1), 16, axis=-1) * 2.0 ** -6).all()
    as_bf16 = (back.astype(np.float32).view(np.uint32) & 0xffff) == 0  # exact in the upper 16 bits
    assert as_bf16.all()
    again, b2 = B.pack8(back)
    assert np.array_equal(B.value8(again, b2), back)


# ---- sizes and refusals of the library ----

def _shape(T=64, d=128, E=8, k=2, F=256, C=0, dt=1, bm=0, layout=0):
    return MoeShape(T, d, E, k, F, C, dt, bm, layout)


def _sizes(s):
    out = MoeBackwardSizes()
    st = _lib.lib().moe_backward_query(ctypes.byref(s), ctypes.byref(out))
    return st, out


@built
@pytest.mark.parametrize("over", [dict(), dict(C=7), dict(dt=0), dict(T=1, k=1), dict(E=256, k=64, T=2048)])
def test_sizes(over):
    s = _shape(**over)
    st, q = _sizes(s)
    R = O.row_space(s.T, s.k, s.E, s.capacity)
    eb = 2 if s.dtype == 1 else 4
    assert st == 0
    assert q.saved8_bytes >= 2 * R * s.F * 17 // 16
    assert q.ffn_ws_bytes >= R * (2 * s.d + 3 * s.F) * eb
    assert q.route_ws_bytes >= 4 * s.T * s.k + 4 * s.E * s.d
    assert q.backward_ws_bytes >= max(q.ffn_ws_bytes, q.route_ws_bytes) + R * s.d * eb
    saved = MoeSaved8()
    f = _lib.lib().moe_saved8_carve
    assert f(ctypes.byref(s), 1 << 20, q.saved8_bytes, ctypes.byref(saved)) == 0
    spans = sorted([(saved.gate, R * s.F), (saved.up, R * s.F), (saved.gate_exp, R * s.F // 16),
                    (saved.up_exp, R * s.F // 16)])
    for (a, n), (b, _) in zip(spans, spans[1:]):
        assert a % 256 == 0 and a + n <= b
    assert spans[-1][0] + spans[-1][1] <= (1 << 20) + q.saved8_bytes
    assert f(ctypes.byref(s), 1 << 20, q.saved8_bytes - 1, ctypes.byref(saved)) == 3
    assert f(ctypes.byref(s), (1 << 20) + 16, q.saved8_bytes, ctypes.byref(saved)) == 1
    assert f(ctypes.byref(s), None, q.saved8_bytes, ctypes.byref(saved)) == 2


A = 1 << 20  # an aligned address; nothing here is dereferenced


def _dispatch(s):
    from grouped_gemm_gemv_amd._lib import MoeSizes
    q = MoeSizes()
    assert _lib.lib().moe_query(ctypes.byref(s), ctypes.byref(q)) == 0
    d = MoeDispatch()
    assert _lib.lib().moe_dispatch_carve(ctypes.byref(s), A, q.dispatch_bytes, ctypes.byref(d)) == 0
    return d


def _calls(s):
    """{entry point: (arguments without shape and stream, positions of required pointers)}"""
    d, v = _dispatch(s), MoeSaved8(A, A, A, A)
    big = 1 << 50
    D, V = ctypes.byref(d), ctypes.byref(v)
    return {
        "moe_ffn_gate_up_save8": ([A, A, A, D, 0, A, V], [0, 1, 2, 3, 5, 6], [0, 1, 2, 5]),
        "moe_saved8_unpack": ([V, D, A, A], [0, 1, 2, 3], [2, 3]),
        "moe_combine_backward": ([A, A, A, D, A, A], [0, 1, 2, 3, 4, 5], [0, 1, 4]),
        "moe_permute_backward": ([A, D, A], [0, 1, 2], [0, 2]),
        "moe_route_backward": ([A, A, A, A, A, A, A, A, A, big], [0, 1, 2, 3, 4, 5, 6, 8], [0, 1, 5, 6]),
        "moe_grouped_ffn_backward": ([A, A, A, A, A, A, D, V, A, A, A, A, A, A, big],
                                     [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 13], [0, 1, 3, 4, 5, 8, 10, 11, 12]),
        "moe_forward_save8": ([A, A, A, A, A, A, A, A, A, D, V, A, big], [0, 3, 4, 5, 6, 7, 8, 9, 10, 11],
                              [0, 1, 5, 6, 7, 8]),
        "moe_backward": ([A, A, A, A, A, A, A, D, V, A, A, A, A, A, A, A, A, A, big],
                         [0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 17], [0, 1, 4, 5, 6, 9, 10, 12, 14, 15, 16]),
    }


NAMES = ["moe_ffn_gate_up_save8", "moe_saved8_unpack", "moe_combine_backward", "moe_permute_backward",
         "moe_route_backward", "moe_grouped_ffn_backward", "moe_forward_save8", "moe_backward"]


@built
@pytest.mark.parametrize("name", NAMES)
def test_refusals(name):
    s = _shape()
    f = getattr(_lib.lib(), name)
    args, required, aligned = _calls(s)[name]

    def call(a, shape=s):
        return f(ctypes.byref(shape) if shape is not None else None, *a, None)

    assert call(args, None) == 2
    for i in required:
        assert call(args[:i] + [None] + args[i + 1:]) == 2, i
    for i in aligned:
        assert call(args[:i] + [A + 8] + args[i + 1:]) == 1, i
    # nothing of this reaches a launch: a shape that is out of range
    for bad, code in ((dict(T=0), 1), (dict(k=9), 1), (dict(E=257), 1), (dict(d=96), 4), (dict(F=100), 4),
                      (dict(dt=5), 1), (dict(layout=3), 1), (dict(bm=17), 4)):
        assert call(args, _shape(**bad)) == code, bad
    if name in ("moe_route_backward", "moe_grouped_ffn_backward", "moe_forward_save8", "moe_backward"):
        assert call(args[:-1] + [16]) == 3
        assert call(args[:-2] + [A + 16, args[-1]]) == 1
    v = MoeSaved8(A, A, None, A)
    if "saved" in name or "ffn" in name or name in ("moe_forward_save8", "moe_backward"):
        at = {"moe_ffn_gate_up_save8": 6, "moe_saved8_unpack": 0, "moe_grouped_ffn_backward": 7,
              "moe_forward_save8": 10, "moe_backward": 8}[name]
        assert call(args[:at] + [ctypes.byref(v)] + args[at + 1:]) == 2
        v = MoeSaved8(A, A + 4, A, A)
        assert call(args[:at] + [ctypes.byref(v)] + args[at + 1:]) == 1


@built
def test_refused_combinations():
    s = _shape()
    lib = _lib.lib()
    S = ctypes.byref(s)
    a = _calls(s)["moe_grouped_ffn_backward"][0]
    assert lib.moe_grouped_ffn_backward(S, *a[:10], None, a[11], a[12], *a[13:], None) == 1  # dw_up without dw_gate
    a = _calls(s)["moe_backward"][0]
    assert lib.moe_backward(S, a[0], None, *a[2:], None) == 1                 # router gradients without a router
    assert lib.moe_backward(S, *a[:14], None, *a[15:], None) == 1             # dw_up without dw_gate
    a = _calls(s)["moe_ffn_gate_up_save8"][0]
    assert lib.moe_ffn_gate_up_save8(S, *a[:4], 3, *a[5:], None) == 1         # no such pass
    wide = _shape(T=1 << 20, d=4096, dt=0)                                    # x past the gather's 32-bit offsets
    d = _dispatch(wide)
    assert lib.moe_ffn_gate_up_save8(ctypes.byref(wide), *a[:3], ctypes.byref(d), *a[4:], None) == 4


def test_python_checks_shapes_before_the_library():
    torch = pytest.importorskip("torch")
    import grouped_gemm_gemv_amd as M
    s = M.Shape(4, 64, 2, 1, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dx must be"):
        M.api._in(x[:3], "dx", (4, 64), s.dtype, x.device)
    with pytest.raises(ValueError, match="dx must be"):
        M.api._in(x.float(), "dx", (4, 64), s.dtype, x.device)
    with pytest.raises(ValueError, match="device tensors"):
        M.api._in(x, "x", (4, 64), s.dtype, x.device)
    with pytest.raises(ValueError, match="is on"):
        M.api._in(x, "x", (4, 64), s.dtype, torch.device("cuda", 0))


@built
def test_a_shape_that_was_used_still_copies():
    import copy
    import pickle

    import grouped_gemm_gemv_amd as M
    s = M.Shape(3, 64, 4, 2, 64, capacity=1)
    n = M.backward_workspace_size(s)
    for c in (copy.copy(s), copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
        assert c == s and hash(c) == hash(s) and M.backward_workspace_size(c) == n


def test_a_stream_of_another_device_is_refused():
    import types

    import torch

    from grouped_gemm_gemv_amd import api
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        api._call("moe_permute_backward", torch.device("cuda", 0), other)
