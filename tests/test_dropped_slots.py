"""Slots without an expert (an id outside [0, E)) of tokens that have others: they
contribute nothing to any gradient, whatever their routing weight and its
gradient hold."""
import numpy as np
import pytest

from oracle import backward as B

HOLD = (0.0, 3.0, float("inf"), float("nan"))


def _routing(rng, T, E, k):
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    drop = rng.random((T, k)) < 0.4
    drop[:, 0] = False  # every token keeps a slot
    drop[0] = False
    ids[drop] = np.where(rng.random(int(drop.sum())) < 0.5, -1, E)
    w = rng.random((T, k)).astype(np.float32)
    return ids, drop, w / w.sum(axis=1, keepdims=True)


def test_oracle_router_gradient_matches_differences_over_the_live_slots():
    """The weights are the softmax over the slots that have an expert; the others' weights enter nothing."""
    rng = np.random.default_rng(4)
    T, d, E, k = 6, 5, 7, 4
    ids, drop, _ = _routing(rng, T, E, k)
    x, wr, dw = rng.standard_normal((T, d)), rng.standard_normal((E, d)), rng.standard_normal((T, k))

    def weights(x, wr):
        z = np.where(drop, -np.inf, np.take_along_axis(x @ wr.T, np.where(drop, 0, ids), axis=1))
        p = np.exp(z - z.max(axis=1, keepdims=True))
        return p / p.sum(axis=1, keepdims=True)

    w = weights(x, wr)
    for v in HOLD:
        w[drop], dw[drop] = v, v
        (dx, _), (dwr, _), _ = B.route_backward(x, wr, ids, w, dw, "f32")
        for name, val, grad in (("x", x, dx), ("wr", wr, dwr)):
            for i in range(val.size):
                h, loss = 1e-5, []
                for sign in (1, -1):
                    p = {"x": x.copy(), "wr": wr.copy()}
                    p[name].reshape(-1)[i] += sign * h
                    loss.append((weights(**p) * np.where(drop, 0.0, dw)).sum())
                # central differences: h^2 times a third derivative of order 100, and 1e-16 / h of rounding
                assert abs((loss[0] - loss[1]) / (2 * h) - grad.reshape(-1)[i]) <= 1e-7, (name, i, v)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(T=50, d=128, E=8, k=3, F=64), dict(T=33, d=64, E=130, k=6, F=64, dtype="f32"),
    dict(T=300, d=192, E=16, k=4, F=64, cap=30),
], ids=str)
def test_router_gradient_does_not_look_at_dropped_slots(kw):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests.gpu_helpers import bits, host64
    from tests.test_gpu_backward import Case, close
    print(f"\n[gpu] dropped slots {kw}", flush=True)
    c = Case(**kw)
    M = c.M
    ids, drop, w = _routing(np.random.default_rng(6), c.T, c.E, c.k)
    c.ids.copy_(torch.from_numpy(ids))
    M.moe_permute(c.shape, c.x, c.ids, c.disp, c.empty(c.R, c.d), M.workspace(M.query(c.shape).permute_ws_bytes))
    m = torch.from_numpy(drop).cuda()
    dw = torch.randn(c.T, c.k, device="cuda")
    saved, _, _ = c.saved()
    ws = M.workspace(M.backward_workspace_size(c.shape))
    runs = []
    for v in HOLD:
        c.w.copy_(torch.from_numpy(w))
        c.w[m], dw[m] = v, v
        r = {"dx": c.empty(c.T, c.d), "dwr": c.empty(c.E, c.d), "db": c.empty(c.E, dt=torch.float32)}
        M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, dw, r["dx"], r["dwr"], r["db"], ws)
        want = B.route_backward(host64(c.x), host64(c.wr), ids, host64(c.w), host64(dw), c.dtype)
        for n, (value, bound) in zip(("dx", "dwr", "db"), want):
            close(n, host64(r[n]), value, bound)
        a = {"dx": c.empty(c.T, c.d), "dw": c.empty(c.T, c.k, dt=torch.float32), "dwr": c.empty(c.E, c.d),
             "db": c.empty(c.E, dt=torch.float32), "dwg": torch.empty_like(c.wg), "dwu": torch.empty_like(c.wu),
             "dwd": torch.empty_like(c.wd)}
        M.moe_backward(c.shape, c.x, c.wr, c.ids, c.w, c.wg, c.wu, c.wd, c.disp, saved, c.dout, a["dx"], a["dw"],
                       a["dwr"], a["db"], a["dwg"], a["dwu"], a["dwd"], ws)
        assert (a["dw"][m] == 0).all() and all(torch.isfinite(t).all() for t in a.values())
        runs.append([bits(t) for t in (*r.values(), *a.values())])
    for other in runs[1:]:
        assert all(np.array_equal(p, q) for p, q in zip(runs[0], other))
