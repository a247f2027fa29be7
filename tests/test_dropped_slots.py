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


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(T=40, d=576, E=16, k=9, F=64), dict(T=21, d=64, E=12, k=5, F=64, dtype="f32")],
                         ids=str)
def test_combine_gradient_where_groups_of_slots_have_no_row(kw):
    """The kernel works four slots at a time: whole groups of them without a row, and tokens without any, whose dout
    and weights hold NaN."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests.gpu_helpers import host64
    from tests.test_gpu_backward import Case, _t, close
    print(f"\n[gpu] combine gradient, groups without a row {kw}", flush=True)
    c = Case(**kw)
    rng = np.random.default_rng(8)
    drop = np.zeros((c.T, c.k), dtype=bool)
    drop[::3, :4], drop[1::3, 4:], drop[[2, 5, c.T - 1]] = True, True, True
    pad = drop.all(axis=1)
    ids = np.where(drop, -1, c.ids_np).astype(np.int32)
    c.ids.copy_(torch.from_numpy(ids))
    c.M.moe_permute(c.shape, c.x, c.ids, c.disp, c.empty(c.R, c.d),
                    c.M.workspace(c.M.query(c.shape).permute_ws_bytes))
    y = _t(rng.standard_normal((c.R, c.d)), c.dt)
    want, e, dww, ew = B.combine_backward(host64(c.dout), host64(y), host64(c.w),
                                          c.disp.arrays()["row_of"].cpu().numpy(), c.dtype)
    c.dout[torch.from_numpy(pad).cuda()] = float("nan")
    c.w[torch.from_numpy(drop).cuda()] = float("nan")
    dy, dw = c.empty(c.R, c.d), c.empty(c.T, c.k, dt=torch.float32)
    c.M.moe_combine_backward(c.shape, c.dout, y, c.w, c.disp, dy, dw)
    live = c.disp.arrays()["token_of"].cpu().numpy() >= 0
    close("dy", host64(dy)[live], want[live], e[live])
    assert np.isnan(host64(dy)[~live]).all()  # rows without a token stay as they were
    close("dw", host64(dw), dww, ew)
    assert (host64(dw)[drop] == 0).all()
