"""The operators around the layer and the layer for a few tokens, without a GPU: the oracle against differences and
published numbers, sizes, and every refusal (validation returns before any HIP call)."""
import ctypes
import math
import os

import numpy as np
import pytest

from grouped_gemm_gemv_amd import _lib
from grouped_gemm_gemv_amd._lib import MoeResidual, MoeShape
from oracle import block as K

built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmoe.so not built")


# ---- the oracle ----


@pytest.mark.parametrize("ctr,key,want", [
    # known-answer vectors published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_known_answers(ctr, key, want):
    block = np.array([ctr[0] | ctr[1] << 32], dtype=np.uint64)
    got = K.philox(block, ctr[2] | ctr[3] << 32, key[0] | key[1] << 32)[0]
    assert tuple(int(v) for v in got) == want


def test_share_of_kept_elements():
    n = 1 << 14
    for p in (0.1, 0.5, 0.9):
        kept = K.keep(p, 77, 3, n).mean()
        assert abs(kept - (1 - p)) < 5 * math.sqrt(p * (1 - p) / n)  # five standard deviations


@pytest.mark.parametrize("post,gate,drop,nxt", [(1, "token", 1, 1), (1, "full", 0, 1), (0, "token", 1, 0),
                                                (0, None, 0, 1), (1, None, 1, 0), (0, "full", 1, 1)])
def test_oracle_gradients_match_differences(post, gate, drop, nxt):
    rng = np.random.default_rng(5)
    T, d, eps, scale = 3, 16, 1e-3, 0.7
    v = {"res": rng.standard_normal((T, d)), "y": rng.standard_normal((T, d))}
    if post:
        v["post"] = rng.standard_normal(d)
    if gate:
        v["gate"] = rng.standard_normal((T, 1 if gate == "token" else d))
    if nxt:
        v["next"] = rng.standard_normal(d)
    mask = np.where(K.keep(0.4, 9, 1, T * d).reshape(T, d), 1 / 0.6, 0.0) if drop else None
    dout, dn = rng.standard_normal((2, T, d))

    def forward(v):
        return K.residual(v["res"], v["y"], v.get("post"), v.get("gate"), mask, v.get("next"), eps, scale, "f32")

    def loss(v):
        o = forward(v)
        return (o["out"][0] * dout).sum() + ((o["n"][0] * dn).sum() if nxt else 0.0)

    got = K.residual_backward(forward(v)["out"][0], v["y"], v.get("post"), v.get("gate"), mask, v.get("next"), dout,
                              dn if nxt else None, eps, scale, "f32")
    names = {"res": "dres", "y": "dy", "post": "dpost", "gate": "dgate", "next": "dnext"}
    for name, val in v.items():
        grad = got[names[name]][0].reshape(val.shape)
        for i in rng.choice(val.size, min(val.size, 10), replace=False):
            at = np.unravel_index(i, val.shape)
            step = []
            for h in (1e-5, -1e-5):
                moved = dict(v, **{name: val.copy()})
                moved[name][at] += h
                step.append(loss(moved))
            assert abs((step[0] - step[1]) / 2e-5 - grad[at]) <= 1e-6 * (1 + abs(grad[at])), (name, at)


# ---- sizes and refusals ----

FAKE = 0x100000  # an address no call gets as far as using


def _shape(T=4, d=128, E=8, k=2, F=256, C=0, dt=1, layout=0):
    return MoeShape(T, d, E, k, F, C, dt, 0, layout)


def _size(name, s):
    n = ctypes.c_size_t()
    return getattr(_lib.lib(), name)(ctypes.byref(s), ctypes.byref(n)), n.value


@built
def test_residual_workspace_size():
    st, n = _size("moe_residual_workspace_size", _shape(T=4096, d=4096))
    assert st == 0 and n >= 2 * 4096 * 4
    assert _size("moe_residual_workspace_size", _shape(T=1, d=64))[0] == 0
    assert _size("moe_residual_workspace_size", _shape(d=16384))[0] == 0
    assert _size("moe_residual_workspace_size", _shape(d=16384 + 64))[0] == 4
    assert _size("moe_residual_workspace_size", _shape(T=0))[0] == 1
    lib = _lib.lib()
    assert lib.moe_residual_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == 2
    assert lib.moe_residual_workspace_size(ctypes.byref(_shape()), None) == 2


@built
@pytest.mark.parametrize("kw,code", [
    (dict(T=16, d=4096, E=8), 0), (dict(T=16, d=4096, E=80), 0), (dict(T=16, d=4096, E=81), 4),
    (dict(T=8, d=7168, E=256), 0), (dict(T=9, d=7168, E=256), 4), (dict(T=17, d=64), 4), (dict(T=8, d=4096, dt=0), 0),
    (dict(T=16, d=4096, dt=0), 4), (dict(T=0), 1), (dict(d=96), 4), (dict(T=1, d=65536, E=8), 0),
    (dict(T=16, d=4096, C=3), 0),
])
def test_decode_workspace_size(kw, code):
    s = _shape(**kw)
    st, n = _size("moe_decode_workspace_size", s)
    assert st == code
    if code == 0:
        active = min(s.E, s.T * s.k)
        assert n >= active * s.T * s.F * (2 if s.dtype else 4) + active * 16 * 4


def _norm_args(**over):
    a = dict(s=_shape(), x=FAKE, w=FAKE, eps=1e-6, n=FAKE)
    a.update(over)
    return [ctypes.byref(a["s"]) if a["s"] is not None else None, a["x"], a["w"], a["eps"], a["n"], None]


@built
@pytest.mark.parametrize("over,code", [
    (dict(s=None), 2), (dict(s=_shape(T=0)), 1), (dict(s=_shape(d=16448)), 4), (dict(x=None), 2), (dict(w=None), 2),
    (dict(n=None), 2), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=math.inf), 1), (dict(eps=math.nan), 1),
    (dict(x=FAKE + 8), 1), (dict(n=FAKE + 2), 1), (dict(w=FAKE + 4), 1),
])
def test_norm_refusals(over, code):
    assert _lib.lib().moe_norm(*_norm_args(**over)) == code


@built
@pytest.mark.parametrize("over,code", [
    (dict(s=None), 2), (dict(x=None), 2), (dict(w=None), 2), (dict(dn=None), 2), (dict(dx=None), 2), (dict(ws=None), 2),
    (dict(n=0), 3), (dict(eps=0.0), 1), (dict(ws=FAKE + 16), 1), (dict(dw=FAKE + 4), 1), (dict(dres=FAKE + 4), 1),
    (dict(s=_shape(d=20480)), 4),
])
def test_norm_backward_refusals(over, code):
    a = dict(s=_shape(), x=FAKE, w=FAKE, eps=1e-6, dn=FAKE, dres=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 40)
    a.update(over)
    s = ctypes.byref(a["s"]) if a["s"] is not None else None
    assert _lib.lib().moe_norm_backward(s, a["x"], a["w"], a["eps"], a["dn"], a["dres"], a["dx"], a["dw"], a["ws"],
                                        a["n"], None) == code


RESIDUAL = [
    (dict(s=None), 2), (dict(r=None), 2), (dict(s=_shape(d=16448)), 4), (dict(y=None), 2), (dict(gate=None), 2),
    (dict(rng=None), 2), (dict(r=MoeResidual(1e-6, 1.0, 0.1, 0)), 1), (dict(r=MoeResidual(1e-6, 1.0, 0.1, 3)), 1),
    (dict(r=MoeResidual(1e-6, 1.0, 1.0, 1)), 1), (dict(r=MoeResidual(1e-6, 1.0, -0.1, 1)), 1),
    (dict(r=MoeResidual(1e-6, 1.0, math.nan, 1)), 1), (dict(r=MoeResidual(0.0, 1.0, 0.1, 1)), 1),
    (dict(r=MoeResidual(1e-6, math.inf, 0.1, 1)), 1), (dict(r=MoeResidual(1e-6, math.nan, 0.1, 1)), 1),
    (dict(next_w=None), 1), (dict(y=FAKE + 8), 1), (dict(rng=FAKE + 4), 1), (dict(gate=FAKE + 1), 1),
    (dict(r=MoeResidual(1e-6, 1.0, 0.1, 2), gate=FAKE + 8), 1), (dict(post_w=FAKE + 8), 1),
]


@built
@pytest.mark.parametrize("over,code", RESIDUAL + [(dict(res=None), 2), (dict(out=None), 2), (dict(n=None), 1)])
def test_residual_refusals(over, code):
    a = dict(s=_shape(), r=MoeResidual(1e-6, 1.0, 0.1, 1), res=FAKE, y=FAKE, post_w=FAKE, gate=FAKE, rng=FAKE,
             next_w=FAKE, out=FAKE, n=FAKE)
    a.update(over)
    ref = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    assert _lib.lib().moe_residual(ref(a["s"]), ref(a["r"]), *[a[n] for n in (
        "res", "y", "post_w", "gate", "rng", "next_w", "out", "n")], None) == code


@built
@pytest.mark.parametrize("over,code", RESIDUAL + [
    (dict(out=None), 2), (dict(dn=None), 1), (dict(dres=None), 2), (dict(dy=None), 2), (dict(ws=None), 2),
    (dict(bytes=16), 3), (dict(ws=FAKE + 16), 1), (dict(post_w=None), 1), (dict(next_w=None, dn=None), 1),
    (dict(next_w=None, dn=None, dnext_w=None, dout=None), 2), (dict(dgate=FAKE + 1), 1), (dict(dy=FAKE + 8), 1),
    (dict(r=MoeResidual(1e-6, 1.0, 0.1, 0), gate=None), 1),
])
def test_residual_backward_refusals(over, code):
    a = dict(s=_shape(), r=MoeResidual(1e-6, 1.0, 0.1, 1), out=FAKE, y=FAKE, post_w=FAKE, gate=FAKE, rng=FAKE,
             next_w=FAKE, dout=FAKE, dn=FAKE, dres=FAKE, dy=FAKE, dgate=FAKE, dpost_w=FAKE, dnext_w=FAKE, ws=FAKE,
             bytes=1 << 40)
    a.update(over)
    ref = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    assert _lib.lib().moe_residual_backward(ref(a["s"]), ref(a["r"]), *[a[n] for n in (
        "out", "y", "post_w", "gate", "rng", "next_w", "dout", "dn", "dres", "dy", "dgate", "dpost_w", "dnext_w", "ws",
        "bytes")], None) == code


@built
@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(dtype=2), 1), (dict(p=1.0), 1), (dict(p=-0.5), 1), (dict(p=math.nan), 1), (dict(x=None), 2),
    (dict(out=None), 2), (dict(rng=None), 2), (dict(x=FAKE + 2), 1), (dict(out=FAKE + 8), 1), (dict(rng=FAKE + 4), 1),
    (dict(n=0, x=None, out=None, rng=None), 0),  # nothing to do, and nothing is launched
])
def test_dropout_refusals(over, code):
    a = dict(x=FAKE, n=100, dtype=1, p=0.1, rng=FAKE, out=FAKE)
    a.update(over)
    assert _lib.lib().moe_dropout(a["x"], a["n"], a["dtype"], a["p"], a["rng"], a["out"], None) == code


DECODE = [
    (dict(s=None), 2), (dict(s=_shape(T=17)), 4), (dict(s=_shape(T=16, d=8192)), 4), (dict(x=None), 2),
    (dict(wg=None), 2), (dict(wu=None), 2), (dict(wd=None), 2), (dict(out=None), 2), (dict(ws=None), 2),
    (dict(bytes=64), 3), (dict(wr=None, ids=None), 2), (dict(wr=None, w=None), 2), (dict(wr=None), 1),
    (dict(eps=0.0), 1), (dict(eps=math.nan), 1), (dict(scale=math.inf), 1), (dict(x=FAKE + 8), 1),
    (dict(wd=FAKE + 8), 1), (dict(ws=FAKE + 16), 1), (dict(ids=FAKE + 2), 1), (dict(bias=FAKE + 2), 1),
    (dict(res=FAKE + 8), 1), (dict(norm=FAKE + 8), 1),
]


@built
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over,code", DECODE)
def test_decode_refusals(over, code, fp8):
    a = dict(s=_shape(), x=FAKE, norm=FAKE, eps=1e-6, wr=FAKE, bias=FAKE, ids=FAKE, w=FAKE, wg=FAKE, wu=FAKE, wd=FAKE,
             sg=FAKE, su=FAKE, sd=FAKE, res=FAKE, scale=1.0, out=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(over)
    s = ctypes.byref(a["s"]) if a["s"] is not None else None
    scales = [a[n] for n in ("sg", "su", "sd")] if fp8 else []
    fn = _lib.lib().moe_decode_fp8 if fp8 else _lib.lib().moe_decode
    assert fn(s, a["x"], a["norm"], a["eps"], a["wr"], a["bias"], a["ids"], a["w"], a["wg"], a["wu"], a["wd"], *scales,
              a["res"], a["scale"], a["out"], a["ws"], a["bytes"], None) == code


@built
def test_decode_fp8_refuses_fp32_and_missing_scales():
    fn = _lib.lib().moe_decode_fp8
    args = [FAKE, FAKE, 1e-6, FAKE, None, None, None, FAKE, FAKE, FAKE]
    tail = [None, 1.0, FAKE, FAKE, 1 << 40, None]
    assert fn(ctypes.byref(_shape(dt=0)), *args, FAKE, FAKE, FAKE, *tail) == 4
    for i in range(3):
        scales = [FAKE] * 3
        scales[i] = None
        assert fn(ctypes.byref(_shape()), *args, *scales, *tail) == 2


@built
def test_binding_refuses_wrong_tensors():
    import torch

    import grouped_gemm_gemv_amd as M
    s = M.Shape(4, 64, 2, 1, 64)
    t = lambda *n, dt=torch.bfloat16: torch.zeros(n, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="device tensors"):
        M.moe_norm(s, t(4, 64), t(64), t(4, 64))
    with pytest.raises(ValueError, match="x must be"):
        M.moe_norm(s, t(4, 128), t(64), t(4, 64))
    with pytest.raises(ValueError, match="fp32 or bf16"):
        M.moe_dropout(t(8, dt=torch.float16), 0.1, t(2, dt=torch.int64), t(8, dt=torch.float16))
    with pytest.raises(ValueError, match="gate must be"):
        M.moe_residual(s, M.Residual(), t(4, 64), t(4, 64), None, t(3), None, None, t(4, 64), None)
    with pytest.raises(ValueError, match="dgate must have"):
        M.moe_residual_backward(s, M.Residual(), None, t(4, 64), None, None, None, None, t(4, 64), None, t(4, 64),
                                t(4, 64), t(4), None, None, t(64, dt=torch.uint8))
