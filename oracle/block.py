"""The operators around the layer and the layer for a few tokens, in float64 from their definitions, with bounds of
what a kernel's fp32 arithmetic and one rounding of each output may be off by.

Inputs are float64 arrays that hold the device's values.  A function returns (value, bound) for each output.  Bounds:
`S` fp32 operations lie on any path from an input to a sum over a row (up to 16 elements of a thread, 6 exchanges of a
wavefront, up to 16 wavefronts one after another, which is 38, and twice as many for the square root, division,
exponential and products around them, each at most 2^-24, the exponential at most 4 of those), so each term of such a sum
is off by at most S 2^-24 of its magnitude.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative
TINY = 2.0 ** -120  # below it a magnitude is in nobody's way
S = 80 * U32
# The experts' SwiGLU takes the fast exponential, whose argument is rounded in another base: |g| 2^-24 / ln 2 of its
# value, below 100 for |g| <= 60, past which nothing is left of it.
EXP = 128 * U32


def philox(block: np.ndarray, step: int, seed: int) -> np.ndarray:
    """The four 32-bit words of Philox 4x32-10 for counter {block, step} and key {seed}: [..., 4] uint32.  Written with
    Python integers, a word at a time, so that nothing can wrap unseen."""
    out = np.empty(block.shape + (4,), dtype=np.uint32)
    m = 0xFFFFFFFF
    for at in np.ndindex(block.shape):
        b = int(block[at])
        c = [b & m, b >> 32, step & m, step >> 32]
        k = [seed & m, seed >> 32]
        for _ in range(10):
            p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(q >> 32) ^ c[1] ^ k[0], q & m, (p >> 32) ^ c[3] ^ k[1], p & m]
            k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
        out[at] = c
    return out


def threshold(p: float) -> int:
    return min(65535, int(np.floor(float(np.float32(p)) * 65536.0 + 0.5)))


def keep(p: float, seed: int, step: int, n: int) -> np.ndarray:
    """Which of n elements are kept."""
    words = philox(np.arange((n + 7) // 8, dtype=np.uint64), step, seed)
    halves = np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)[:n]
    return halves >= threshold(p)


def sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def norm(x, w, eps, dtype):
    n = x * rms(x, eps) * w
    return n, (U[dtype] + S) * np.abs(n) + TINY


def residual(res, y, post_w, gate, mask, next_w, eps, scale, dtype):
    """mask: keep over 1 - p, or None; gate [T, 1] or [T, d] or None.  {name: (value, bound)}."""
    v = y * rms(y, eps) * post_w if post_w is not None else y
    v = v * scale
    if gate is not None:
        v = v * sigmoid(gate)
    if mask is not None:
        v = np.where(mask > 0, v * mask, 0.0)
    out = res + v
    e = S * np.abs(v) + U32 * np.abs(out)
    outs = {"out": (out, e + U[dtype] * np.abs(out) + TINY)}
    if next_w is not None:
        r = rms(out, eps)
        n = out * r * next_w
        # r moves by half of what the mean square does
        e_r = (np.abs(out) * e).mean(axis=1, keepdims=True) * r * r + S
        outs["n"] = (n, e * r * np.abs(next_w) + (e_r + U[dtype] + S) * np.abs(n) + TINY)
    return outs


def _norm_grad(x, w, dn, e_dn, eps):
    """Gradient of the norm towards x with its bound, and dn x r with its own (to be summed over rows)."""
    r = rms(x, eps)
    z, e_z = dn * w, e_dn * np.abs(w)
    zx, a_zx = (z * x).mean(axis=1, keepdims=True), (np.abs(z * x)).mean(axis=1, keepdims=True)
    dx = r * (z - x * r * r * zx)
    e = r * (e_z + np.abs(x) * r * r * (e_z * np.abs(x)).mean(axis=1, keepdims=True))
    e = e + 2 * S * r * (np.abs(z) + np.abs(x) * r * r * a_zx)
    return dx, e, dn * x * r, np.abs(x) * r * (e_dn + S * np.abs(dn))


def _column(terms, e_terms, dtype):
    """A sum over tokens: a workgroup's rows one after another, then the workgroups'."""
    depth = (terms.shape[0] / 256 + 100) * U32
    v = terms.sum(axis=0)
    return v, e_terms.sum(axis=0) + depth * np.abs(terms).sum(axis=0) + U[dtype] * np.abs(v) + TINY


def residual_backward(x, y, post_w, gate, mask, next_w, dout, dn, eps, scale, dtype):
    """x: what the forward pass left in out.  y None: the norm alone ("dres" is then its dx)."""
    outs = {}
    shape = x if x is not None else dout
    D = dout if dout is not None else np.zeros_like(shape)
    e = np.zeros_like(D)
    if next_w is not None:
        dx, e, terms, e_terms = _norm_grad(x, next_w, dn, np.zeros_like(dn), eps)
        outs["dnext"] = _column(terms, e_terms, dtype)
        D = D + dx
        e = e + U32 * np.abs(D)
    outs["dres"] = (D, e + U[dtype] * np.abs(D) + TINY)
    if y is None:
        return outs
    m = scale * (mask if mask is not None else 1.0)
    q, e = D * m, e * np.abs(m)
    e = e + S * np.abs(q)
    if gate is not None:
        v = y * rms(y, eps) * post_w if post_w is not None else y
        if mask is not None:
            v = np.where(mask > 0, v, 0.0)
        sg = sigmoid(gate)
        slope = sg * (1.0 - sg)
        t, e_t = q * v * slope, (e + 2 * S * np.abs(q)) * np.abs(v) * slope
        if gate.shape[1] == 1:
            t, e_t = t.sum(axis=1), e_t.sum(axis=1)
        outs["dgate"] = (t, e_t + U[dtype] * np.abs(t) + TINY)
        q, e = q * sg, e * sg + S * np.abs(q * sg)
    if post_w is not None:
        dy, e, terms, e_terms = _norm_grad(y, post_w, q, e, eps)
        outs["dpost"] = _column(terms, e_terms, dtype)
    else:
        dy = q
    outs["dy"] = (dy, e + (U[dtype] + S) * np.abs(dy) + TINY)
    return outs


def decode(x, norm_w, eps, ids, w, wg, wu, wd, res, scale, dtype, e_w=0.0, terms=1):
    """out and its bound for a routing (ids [T, k] and weights [T, k], each off by at most e_w of itself); weights
    [E, F, d], [E, F, d], [E, d, F].  m and h are kept in `terms` numbers of the type, each of which takes what rounding
    left of the one before (half a step of it at most): 1 is the bound of a layer that rounds both, 2 of one that does not."""
    T, d = x.shape
    F = wg.shape[1]
    u = U[dtype]
    u_in = u ** terms
    m = x * rms(x, eps) * norm_w if norm_w is not None else x
    e_m = (u_in + S) * np.abs(m) if norm_w is not None else np.zeros_like(m)
    out = np.zeros((T, d))
    bound = np.zeros((T, d))
    # products added one after another; those of second terms are as many again, and 2^-8 of the first ones'
    k_up, k_down = [(n + (terms - 1) * (1 + 2 * u) * n + 64) * U32 for n in (d, F * ids.shape[1])]
    for t in range(T):
        for j, expert in enumerate(ids[t]):
            if not 0 <= expert < wg.shape[0] or w[t, j] == 0:
                continue
            ag, au, ad = np.abs(wg[expert]), np.abs(wu[expert]), np.abs(wd[expert])
            g, up = wg[expert] @ m[t], wu[expert] @ m[t]
            e_g = ag @ (e_m[t] + k_up * np.abs(m[t]))
            e_u = au @ (e_m[t] + k_up * np.abs(m[t]))
            sg = sigmoid(g)
            h = g * sg * up
            # |silu'| is at most 1.1
            e_h = 1.1 * e_g * (np.abs(up) + e_u) + np.abs(g * sg) * e_u + (u_in + EXP) * np.abs(h)
            y = wd[expert] @ h
            e_y = ad @ (e_h + k_down * np.abs(h))
            out[t] += w[t, j] * y
            bound[t] += np.abs(w[t, j]) * (e_y + (e_w + 4 * U32) * np.abs(y))
    out, bound = out * scale, bound * abs(scale)
    if res is not None:
        out = out + res
    return out, bound + (u + 2 * U32) * np.abs(out) + TINY
