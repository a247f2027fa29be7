"""CPU oracle of the layer's backward pass (test infrastructure only).

Plain float64 NumPy from the definitions, given the inputs as float64 arrays.
Where a result is compared with the GPU, a bound on the GPU's error comes with
it, carried through the formulas from the roundings it makes: u (half a step of
the element type, relative) at each value stored between two steps, and
n 2^-24 of the sum of magnitudes for an fp32 sum of n terms in any order.
"""
from __future__ import annotations

import numpy as np

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24
# Relative error of the GPU's sigmoid and products with it in fp32.  exp2's
# argument carries |g| 2^-24 / ln 2 of rounding, its result 2^-23, the division
# 2^-23; for |g| <= 60, past which sg or 1 - sg no longer matters, that is
# below 100 * 2^-24 with the few multiplications behind it.
EXP = 128 * U32


# ---- 8-bit projections ----

def pack8(v: np.ndarray):
    """(codes, exponents) of float64 values [..., F]: the format's definition."""
    blocks = v.reshape(v.shape[:-1] + (v.shape[-1] // 16, 16))
    top = np.abs(blocks).max(axis=-1)
    # exponent field of the fp32 magnitude: floor(log2) + 127
    b = np.maximum(np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] + 126, 0), 7)
    codes = np.clip(np.rint(blocks * 2.0 ** (133 - b)[..., None]), -127, 127)
    return codes.reshape(v.shape).astype(np.int8), b.astype(np.uint8)


def value8(codes: np.ndarray, b: np.ndarray) -> np.ndarray:
    return codes.astype(np.float64) * np.repeat(2.0 ** (b.astype(np.float64) - 133), 16, axis=-1)


# ---- row steps ----

def combine_backward(dout, y, w, row_of, dtype):
    """dy [R, d] (0 in rows without a token) and dw [T, k], each with its bound."""
    T, k = w.shape
    R, d = y.shape
    dy, dw = np.zeros((R, d)), np.zeros((T, k))
    bound = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_of[t * k + j]
            if r >= 0:
                dy[r] = w[t, j] * dout[t]
                dw[t, j] = dout[t] @ y[r]
                bound[t, j] = (d + 4) * U32 * (np.abs(dout[t]) @ np.abs(y[r]))
    return dy, (U[dtype] + U32) * np.abs(dy), dw, bound


def permute_backward(dx_perm, row_of, T, k, dtype):
    dx, mag = np.zeros((T, dx_perm.shape[1])), np.zeros((T, dx_perm.shape[1]))
    for f in range(T * k):
        if row_of[f] >= 0:
            dx[f // k] += dx_perm[row_of[f]]
            mag[f // k] += np.abs(dx_perm[row_of[f]])
    return dx, U[dtype] * np.abs(dx) + 2 * k * U32 * mag


def route_backward(x, wr, ids, w, dw, dtype):
    """dx, dw_router, dbias with bounds.  dz = w (dw - <w, dw>) over the slots that have an expert."""
    T, k = w.shape
    E, d = wr.shape
    live = (ids >= 0) & (ids < E)
    w, dw = np.where(live, w, 0.0), np.where(live, dw, 0.0)
    dz = w * (dw - (w * dw).sum(axis=1, keepdims=True))
    e_dz = (k + 4) * U32 * np.abs(w) * (np.abs(dw) + (np.abs(w) * np.abs(dw)).sum(axis=1, keepdims=True))
    dense, e_dense, n = np.zeros((T, E)), np.zeros((T, E)), np.zeros(E)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                dense[t, e] += dz[t, j]
                e_dense[t, e] += e_dz[t, j] + U32 * np.abs(dz[t, j])
                n[e] += 1
    mag = np.abs(dense)
    dx, dwr, db = dense @ wr, dense.T @ x, dense.sum(axis=0)
    e_dx = e_dense @ np.abs(wr) + 2 * (k + 2) * U32 * (mag @ np.abs(wr))
    # bf16 carries dz as two terms: what is left after both is u^2 of it
    split = U["bf16"] ** 2 if dtype == "bf16" else 0.0
    terms = (2 * T + 80) * U32
    e_dwr = (e_dense + (split + terms) * mag).T @ np.abs(x)
    e_db = e_dense.sum(axis=0) + (n + 16) * U32 * mag.sum(axis=0)
    return ((dx, e_dx + U[dtype] * np.abs(dx)), (dwr, e_dwr + U[dtype] * np.abs(dwr)), (db, e_db))


# ---- experts ----

def ffn_backward(x, dout, w, wg, wu, wd, g, u, token_of, entry_of, expert_of, dtype):
    """Gradients of the experts' products from saved projections g, u [R, F].

    token_of, entry_of, expert_of: per row, -1 where the row holds no token.
    Returns {name: (value, bound)} for dx_perm [R, d], dw [T k], dwg, dwu [E, F, d]
    and dwd [E, d, F]."""
    E, F, d = wg.shape
    R = token_of.shape[0]
    un = U[dtype]
    out = {"dx_perm": [np.zeros((R, d)), np.zeros((R, d))], "dw": [np.zeros(w.size), np.zeros(w.size)]}
    for n, sh in (("dwg", (E, F, d)), ("dwu", (E, F, d)), ("dwd", (E, d, F))):
        out[n] = [np.zeros(sh), np.zeros(sh)]
    for e in range(E):
        rows = np.flatnonzero(expert_of == e)
        if rows.size == 0:
            continue
        t, f = token_of[rows], entry_of[rows]
        X, Y, W = x[t], dout[t], w.reshape(-1)[f][:, None]
        G, V = g[rows], u[rows]
        D = Y @ wd[e]
        e_D = (d + 8) * U32 * (np.abs(Y) @ np.abs(wd[e]))
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-G))
        a, h = G * s, G * s * V
        out["dw"][0][f] = (D * h).sum(axis=1)
        out["dw"][1][f] = (e_D * np.abs(h) + np.abs(D * h) * (EXP + (F + 16) * U32)).sum(axis=1)
        q = V * s * (1 + G * (1 - s))          # d(g s u) / dg
        q_mag = np.abs(V) * s * (1 + np.abs(G) * (1 - s))
        dG, dU, H = W * D * q, W * D * a, W * h
        aW = np.abs(W)
        # stored between the products: one rounding of the type each
        e_G = aW * (e_D * np.abs(q) + np.abs(D) * EXP * q_mag) + un * np.abs(dG)
        e_U = aW * (e_D * np.abs(a) + np.abs(D) * EXP * np.abs(a)) + un * np.abs(dU)
        e_H = (EXP + un) * np.abs(H)
        dxp = dG @ wg[e] + dU @ wu[e]
        mag = np.abs(dG) @ np.abs(wg[e]) + np.abs(dU) @ np.abs(wu[e])
        out["dx_perm"][0][rows] = dxp
        out["dx_perm"][1][rows] = (e_G @ np.abs(wg[e]) + e_U @ np.abs(wu[e]) + (2 * F + 8) * U32 * mag
                                   + un * np.abs(dxp))
        n32 = (rows.size + 64) * U32
        for name, P, Q, e_P, e_Q in (("dwg", dG, X, e_G, 0.0), ("dwu", dU, X, e_U, 0.0), ("dwd", Y, H, 0.0, e_H)):
            val = P.T @ Q
            bound = n32 * (np.abs(P).T @ np.abs(Q)) + un * np.abs(val)
            if np.ndim(e_P):
                bound += e_P.T @ np.abs(Q)
            if np.ndim(e_Q):
                bound += np.abs(P).T @ e_Q
            out[name][0][e], out[name][1][e] = val, bound
    return {n: tuple(v) for n, v in out.items()}


# ---- the layer as a function, for differences ----

def layer(x, ids, logits_of, wg, wu, wd):
    """out [T, d] of the SwiGLU layer for fixed ids; weights = softmax over the chosen logits logits_of(x) [T, E]."""
    z = np.take_along_axis(logits_of(x), ids, axis=1)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    w = p / p.sum(axis=1, keepdims=True)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            g, v = wg[e] @ x[t], wu[e] @ x[t]
            out[t] += w[t, j] * (wd[e] @ (g / (1 + np.exp(-g)) * v))
    return out
