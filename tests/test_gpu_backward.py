"""The backward pass on the GPU against float64, element by element within
bounds carried through the formulas (oracle/backward.py), over both types,
both weight orders, capacity, experts without rows, dropped entries, one
token, column tails of every tile and every row-tile height; then the pieces
together, replayed from a graph, repeated bitwise, and on another stream."""
import numpy as np
import pytest

from oracle import backward as B
from oracle import moe_oracle as O
from tests.gpu_helpers import bits, host64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _t(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dt).cuda()


class Case:
    """Inputs of a layer on the device with their float64 values."""

    def __init__(self, T, d, E, k, F, cap=0, dtype="bf16", layout=0, drop=0.0, hot=None, tile_rows=0, seed=0):
        import grouped_gemm_gemv_amd as M
        self.M = M
        rng = np.random.default_rng(seed)
        dt = self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.T, self.d, self.E, self.k, self.F, self.dtype = T, d, E, k, F, dtype
        self.shape = M.Shape(T, d, E, k, F, cap, dt, tile_rows, layout)
        self.rows = M.Shape(T, d, E, k, F, cap, dt, tile_rows, 0)
        self.x, self.dout = _t(rng.standard_normal((T, d)), dt), _t(rng.standard_normal((T, d)), dt)
        self.wr = _t(rng.standard_normal((E, d)) / np.sqrt(d), dt)
        self.wg = _t(rng.standard_normal((E, F, d)) * 1.5 / np.sqrt(d), dt)
        self.wu = _t(rng.standard_normal((E, F, d)) * 1.5 / np.sqrt(d), dt)
        self.wd = _t(rng.standard_normal((E, d, F)) / np.sqrt(F), dt)
        pool = E if hot is None else hot  # hot: only that many experts are used
        ids = np.argsort(rng.random((T, pool)), axis=1)[:, :k].astype(np.int32)
        if drop:
            ids[rng.random((T, k)) < drop] = -1
        self.ids_np = ids
        self.ids = torch.from_numpy(ids).cuda()
        w = rng.random((T, k)).astype(np.float32)
        self.w = torch.from_numpy(w / w.sum(axis=1, keepdims=True)).cuda()
        self.R = M.query(self.shape).rows
        self.disp = M.Dispatch(self.shape)
        xp = torch.empty(self.R, d, dtype=dt, device="cuda")
        M.moe_permute(self.shape, self.x, self.ids, self.disp, xp, M.workspace(M.query(self.shape).permute_ws_bytes))
        arr = self.disp.arrays()
        self.row_of = arr["row_of"].cpu().numpy()
        self.token_of = arr["token_of"].cpu().numpy()
        self.entry_of, self.expert_of = np.full(self.R, -1), np.full(self.R, -1)
        for f, r in enumerate(self.row_of):
            if r >= 0:
                self.entry_of[r], self.expert_of[r] = f, ids.reshape(-1)[f]
        self.live = self.token_of >= 0

    def weight(self, w):
        """A weight in the shape's storage order."""
        return self.M.moe_pack_blocked16(w) if self.shape.weight_layout else w

    def unweight(self, w):
        """A gradient that came in the storage order, as rows (the inverse byte permutation, on the host)."""
        a = w.float().cpu().numpy().astype(np.float64)
        if not self.shape.weight_layout:
            return a
        e, n, m = a.shape
        per = 32 if self.dtype == "bf16" else 16
        return a.reshape(e, n // 16, m // per, 16, per).swapaxes(2, 3).reshape(e, n, m)

    def empty(self, *n, dt=None):
        return torch.full(n, float("nan"), dtype=dt or self.dt, device="cuda")

    def saved(self, seed=5):
        """Saved projections as a forward pass could have left them, and their values."""
        rng = np.random.default_rng(seed)
        s = self.M.Saved8(self.shape)
        a = s.arrays()
        vals = []
        for n in ("gate", "up"):
            codes, b = B.pack8(rng.standard_normal((self.R, self.F)) * 1.5)
            a[n].copy_(torch.from_numpy(codes))
            a[n + "_exp"].copy_(torch.from_numpy(b))
            vals.append(B.value8(codes, b))
        return s, vals[0], vals[1]


def close(name, got, want, bound):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(err / np.maximum(bound, 1e-300))))


ROW_CASES = [
    dict(T=1, d=64, E=2, k=1, F=64), dict(T=7, d=192, E=5, k=3, F=64, drop=0.3),
    dict(T=65, d=576, E=16, k=9, F=64, cap=5), dict(T=33, d=4096, E=8, k=2, F=64, dtype="f32"),
    dict(T=9, d=64, E=64, k=64, F=64, dtype="f32", cap=2, drop=0.1), dict(T=300, d=1024, E=4, k=4, F=64),
]


@pytest.mark.parametrize("kw", ROW_CASES, ids=str)
def test_combine_and_permute_backward(kw):
    _need_gpu()
    print(f"\n[gpu] combine/permute backward {kw}", flush=True)
    c = Case(**kw)
    rng = np.random.default_rng(1)
    y = _t(rng.standard_normal((c.R, c.d)), c.dt)
    dy, dw = c.empty(c.R, c.d), c.empty(c.T, c.k, dt=torch.float32)
    c.M.moe_combine_backward(c.shape, c.dout, y, c.w, c.disp, dy, dw)
    dx = c.empty(c.T, c.d)
    c.M.moe_permute_backward(c.shape, y, c.disp, dx)
    want, e, dww, ew = B.combine_backward(host64(c.dout), host64(y), host64(c.w), c.row_of, c.dtype)
    got = host64(dy)
    close("dy", got[c.live], want[c.live], e[c.live])
    assert np.isnan(got[~c.live]).all()  # rows without a token stay as they were
    close("dw", host64(dw), dww, ew)
    want, e = B.permute_backward(host64(y), c.row_of, c.T, c.k, c.dtype)
    close("dx", host64(dx), want, e)


@pytest.mark.parametrize("kw", [
    dict(T=1, d=64, E=2, k=1, F=64), dict(T=31, d=192, E=5, k=3, F=64), dict(T=333, d=320, E=70, k=6, F=64),
    dict(T=2100, d=128, E=8, k=2, F=64), dict(T=50, d=128, E=8, k=2, F=64, dtype="f32"),
    dict(T=700, d=192, E=130, k=5, F=64, dtype="f32"), dict(T=20, d=64, E=256, k=64, F=64, drop=0.2),
], ids=str)
def test_route_backward(kw):
    _need_gpu()
    print(f"\n[gpu] route backward {kw}", flush=True)
    c = Case(**kw)
    rng = np.random.default_rng(2)
    dw = torch.from_numpy(rng.standard_normal((c.T, c.k)).astype(np.float32)).cuda()
    dx, dwr, db = c.empty(c.T, c.d), c.empty(c.E, c.d), c.empty(c.E, dt=torch.float32)
    ws = c.M.workspace(c.M.backward_query(c.shape).route_ws_bytes)
    c.M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, dw, dx, dwr, db, ws)
    want = B.route_backward(host64(c.x), host64(c.wr), c.ids_np, host64(c.w), host64(dw), c.dtype)
    for name, got, (v, e) in zip(("dx", "dwr", "db"), (dx, dwr, db), want):
        close(name, host64(got), v, e)
    again = torch.empty_like(dwr)
    c.M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, dw, dx, again, None, ws)
    assert np.array_equal(bits(again), bits(dwr))


def test_route_backward_counts_a_repeated_id_twice():
    _need_gpu()
    c = Case(T=40, d=64, E=6, k=3, F=64)
    c.ids_np[:, 1] = c.ids_np[:, 0]
    c.ids.copy_(torch.from_numpy(c.ids_np))
    dw = torch.randn(c.T, c.k, device="cuda")
    dx, dwr, db = c.empty(c.T, c.d), c.empty(c.E, c.d), c.empty(c.E, dt=torch.float32)
    c.M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, dw, dx, dwr, db,
                           c.M.workspace(c.M.backward_workspace_size(c.shape)))
    want = B.route_backward(host64(c.x), host64(c.wr), c.ids_np, host64(c.w), host64(dw), c.dtype)
    for name, got, (v, e) in zip(("dx", "dwr", "db"), (dx, dwr, db), want):
        close(name, host64(got), v, e)


@pytest.mark.parametrize("tile_rows", [0, 16, 32, 48, 64, 96, 128, 160, 192, 384])
@pytest.mark.parametrize("kw", [
    dict(T=150, d=128, E=3, k=2, F=320), dict(T=90, d=64, E=4, k=2, F=192, cap=20, layout=1),
    dict(T=70, d=128, E=3, k=2, F=192, dtype="f32"),
], ids=str)
def test_gate_up_save8(kw, tile_rows):
    """h bitwise that of the plain gate+up; every code within half a step (a full one where clamped) of float64."""
    _need_gpu()
    print(f"\n[gpu] save8 {kw} {tile_rows}", flush=True)
    c = Case(tile_rows=tile_rows, **kw)
    h, ref = c.empty(c.R, c.F), c.empty(c.R, c.F)
    saved = c.M.Saved8(c.shape)
    for a in saved.arrays().values():
        a.fill_(77)
    wg, wu = c.weight(c.wg), c.weight(c.wu)
    c.M.moe_ffn_gate_up_save8(c.shape, c.x, wg, wu, c.disp, c.M.PASS_BOTH, h, saved)
    c.M.moe_ffn_gate_up_gather(c.shape, c.x, wg, wu, c.disp, c.M.PASS_BOTH, ref)
    assert np.array_equal(bits(h), bits(ref))
    out = [c.empty(c.R, c.F, dt=torch.bfloat16) for _ in range(2)]
    c.M.moe_saved8_unpack(c.shape, saved, c.disp, *out)
    arr = {n: v.cpu().numpy() for n, v in saved.arrays().items()}
    x = host64(c.x)
    for name, w, o in (("gate", c.wg, out[0]), ("up", c.wu, out[1])):
        codes, b, w = arr[name], arr[name + "_exp"], host64(w)
        assert (codes[~c.live] == 77).all() and (b[~c.live] == 77).all() and np.isnan(host64(o)[~c.live]).all()
        val = B.value8(codes, b)
        assert np.array_equal(host64(o)[c.live], val[c.live])
        for r in np.flatnonzero(c.live):
            e, t = c.expert_of[r], c.token_of[r]
            v = w[e] @ x[t]
            acc = (c.d + 8) * B.U32 * (np.abs(w[e]) @ np.abs(x[t]))
            step = np.repeat(2.0 ** (b[r].astype(np.float64) - 133), 16)
            lim = np.where(np.abs(codes[r].astype(int)) == 127, 1.0, 0.5) * step + acc
            assert (np.abs(val[r] - v) <= lim).all(), (name, r)
            # the block's exponent is that of its largest magnitude, up to the sum's rounding
            top, et = np.abs(v).reshape(-1, 16).max(1), acc.reshape(-1, 16).max(1)
            lo, hi = 2.0 ** (b[r].astype(np.float64) - 127), 2.0 ** (b[r].astype(np.float64) - 126)
            assert ((top + et >= lo) & (top - et < hi)).all(), (name, r)


def test_save8_marks_blocks_that_hold_no_number():
    _need_gpu()
    c = Case(T=8, d=64, E=2, k=1, F=64)
    wg = c.wg.clone()
    wg[:, 5, 0], wg[:, 40, 0], wg[:, 20:36, :] = float("nan"), float("inf"), 0.0
    saved, h = c.M.Saved8(c.shape), c.empty(c.R, c.F)
    c.M.moe_ffn_gate_up_save8(c.shape, c.x, wg, c.wu, c.disp, 0, h, saved)
    out = [c.empty(c.R, c.F, dt=torch.bfloat16) for _ in range(2)]
    c.M.moe_saved8_unpack(c.shape, saved, c.disp, *out)
    g = host64(out[0])
    assert np.isnan(g[:, 0:16]).all() and np.isnan(g[:, 32:48]).all()
    assert not np.isnan(g[:, 16:32]).any() and not np.isnan(g[:, 48:]).any() and not np.isnan(host64(out[1])).any()
    assert (g[:, 20:32] == 0).all()


FFN_CASES = [
    dict(T=1, d=64, E=2, k=1, F=64),
    dict(T=5, d=128, E=8, k=2, F=192, layout=1),
    dict(T=64, d=320, E=8, k=2, F=448),                      # column tails of every tile width
    dict(T=100, d=192, E=4, k=2, F=320, cap=30),             # rows in two runs
    dict(T=90, d=64, E=16, k=3, F=128, cap=9, layout=1, drop=0.1),
    dict(T=200, d=192, E=6, k=2, F=576, hot=3),              # experts without rows
    dict(T=130, d=256, E=2, k=1, F=320),                     # 65 mean rows: 128-row tiles
    dict(T=500, d=320, E=2, k=1, F=576, layout=1),           # 250: 256-row tiles
    dict(T=700, d=256, E=3, k=1, F=256, cap=230),
    dict(T=64, d=128, E=8, k=2, F=256, dtype="f32"),
    dict(T=70, d=192, E=5, k=2, F=320, dtype="f32", cap=20, layout=1, drop=0.1),
    dict(T=300, d=64, E=2, k=1, F=192, dtype="f32", hot=1),
    # more tiles than workgroups, which take several in turn: wide, narrow, low
    # and fp32 tiles of the first data gradient, wide ones of the second, with the
    # weight gradients' in each
    dict(T=2060, d=64, E=4, k=1, F=12288, cap=300),
    dict(T=2060, d=64, E=4, k=1, F=6144),
    dict(T=1600, d=64, E=8, k=1, F=3200, cap=100),
    dict(T=640, d=64, E=64, k=1, F=2048, drop=0.1),
    dict(T=1500, d=64, E=8, k=1, F=4096, dtype="f32"),
    dict(T=2060, d=12288, E=4, k=1, F=64),
    dict(T=600, d=192, E=16, k=1, F=1536, cap=30, layout=1),
    dict(T=160, d=8192, E=16, k=1, F=64, dtype="f32"),
    # tiles of 192 rows, in the first data gradient and in the second
    dict(T=2060, d=64, E=4, k=1, F=9216), dict(T=1300, d=64, E=4, k=1, F=12480, cap=260, layout=1),
    dict(T=1000, d=12288, E=6, k=1, F=64),
    # of 128
    dict(T=560, d=320, E=8, k=1, F=448, layout=1), dict(T=1150, d=64, E=12, k=1, F=2688, cap=60, drop=0.1),
]


def _ffn(c, saved, dwn=("dwg", "dwu", "dwd"), ws=None):
    o = {"dx_perm": c.empty(c.R, c.d), "dw": c.empty(c.T, c.k, dt=torch.float32), "dwg": c.empty(c.E, c.F, c.d),
         "dwu": c.empty(c.E, c.F, c.d), "dwd": c.empty(c.E, c.d, c.F)}
    g = [o[n] if n in dwn else None for n in ("dwg", "dwu", "dwd")]
    ws = ws if ws is not None else c.M.workspace(c.M.backward_query(c.shape).ffn_ws_bytes)
    c.M.moe_grouped_ffn_backward(c.shape, c.x, c.dout, c.w, c.weight(c.wg), c.weight(c.wu), c.weight(c.wd), c.disp,
                                 saved, o["dx_perm"], o["dw"], *g, ws)
    return o


@pytest.mark.parametrize("kw", FFN_CASES, ids=str)
def test_grouped_ffn_backward(kw):
    _need_gpu()
    print(f"\n[gpu] ffn backward {kw}", flush=True)
    c = Case(**kw)
    saved, g, u = c.saved()
    o = _ffn(c, saved)
    want = B.ffn_backward(host64(c.x), host64(c.dout), host64(c.w), host64(c.wg), host64(c.wu), host64(c.wd), g, u,
                          c.token_of, c.entry_of, c.expert_of, c.dtype)
    dxp = host64(o["dx_perm"])
    close("dx_perm", dxp[c.live], want["dx_perm"][0][c.live], want["dx_perm"][1][c.live])
    assert np.isnan(dxp[~c.live]).all()
    close("dw", host64(o["dw"]).reshape(-1), *want["dw"])
    for n in ("dwg", "dwu", "dwd"):
        close(n, c.unweight(o[n]), *want[n])
    again = _ffn(c, saved)
    for n in o:
        assert np.array_equal(bits(o[n]), bits(again[n])), n


@pytest.mark.parametrize("kw", [
    dict(T=100, d=192, E=8, k=1, F=320), dict(T=300, d=64, E=4, k=2, F=192, cap=90, layout=1),
    dict(T=90, d=64, E=4, k=2, F=128, dtype="f32"), dict(T=2060, d=64, E=4, k=1, F=9216),
], ids=str)
def test_padding_may_hold_anything(kw):
    """Tokens without an expert: whatever x, dout and the weights hold there, every gradient is bitwise the same."""
    _need_gpu()
    print(f"\n[gpu] padding {kw}", flush=True)
    c = Case(**kw, drop=0.0)
    pad = np.zeros(c.T, dtype=bool)
    pad[[1, 2, c.T // 2]] = True
    pad[-7:] = True
    m = torch.from_numpy(pad).cuda()
    c.ids[m] = -1
    M = c.M
    xp = torch.empty(c.R, c.d, dtype=c.dt, device="cuda")
    M.moe_permute(c.shape, c.x, c.ids, c.disp, xp, M.workspace(M.query(c.shape).permute_ws_bytes))
    saved, _, _ = c.saved()
    ws = M.workspace(M.backward_workspace_size(c.shape))
    wts = [c.weight(w) for w in (c.wg, c.wu, c.wd)]
    dw_in = torch.randn(c.T, c.k, device="cuda")
    runs = []
    for v in (0.0, float("nan"), float("inf")):
        c.x[m], c.dout[m], c.w[m], dw_in[m] = v, v, v, v
        o = _ffn(c, saved)
        r = {"dx": c.empty(c.T, c.d), "dwr": c.empty(c.E, c.d), "db": c.empty(c.E, dt=torch.float32)}
        M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, dw_in, r["dx"], r["dwr"], r["db"], ws)
        a = {"dx": c.empty(c.T, c.d), "dw": c.empty(c.T, c.k, dt=torch.float32), "dwr": c.empty(c.E, c.d),
             "db": c.empty(c.E, dt=torch.float32), **{n: torch.empty_like(o[n]) for n in ("dwg", "dwu", "dwd")}}
        M.moe_backward(c.shape, c.x, c.wr, c.ids, c.w, *wts, c.disp, saved, c.dout, a["dx"], a["dw"], a["dwr"],
                       a["db"], a["dwg"], a["dwu"], a["dwd"], ws)
        for n in ("dwr", "db", "dx"):
            assert torch.isfinite(r[n]).all() and torch.isfinite(a[n]).all(), (n, v)
        assert (r["dx"][m] == 0).all() and (a["dx"][m] == 0).all() and (a["dw"][m] == 0).all()
        runs.append([bits(t) for t in (*o.values(), *r.values(), *a.values())])
    for other in runs[1:]:
        assert all(np.array_equal(p, q) for p, q in zip(runs[0], other))


def test_gradients_that_are_not_asked_for():
    _need_gpu()
    c = Case(T=60, d=128, E=4, k=2, F=192)
    saved, _, _ = c.saved()
    full = _ffn(c, saved)
    for asked in ((), ("dwd",), ("dwg", "dwu")):
        part = _ffn(c, saved, asked)
        for n in full:
            if n in asked or n in ("dx_perm", "dw"):
                assert np.array_equal(bits(full[n]), bits(part[n])), n
            else:
                assert torch.isnan(part[n]).all(), n


def test_extreme_projections():
    """Saturated and vanishing gates: 1 + exp(-g) overflows to infinity, sg is 0 or 1, nothing turns into NaN."""
    _need_gpu()
    c = Case(T=20, d=64, E=2, k=1, F=64)
    saved, _, _ = c.saved()
    a = saved.arrays()
    a["gate"].copy_(torch.randint(-127, 128, (c.R, c.F)).to(torch.int8))
    a["gate_exp"].copy_(torch.tensor([7, 100, 130, 138]).repeat(c.R, 1))  # from 2^-126 to about 4000
    g = B.value8(a["gate"].cpu().numpy(), a["gate_exp"].cpu().numpy())
    u = B.value8(a["up"].cpu().numpy(), a["up_exp"].cpu().numpy())
    o = _ffn(c, saved)
    want = B.ffn_backward(host64(c.x), host64(c.dout), host64(c.w), host64(c.wg), host64(c.wu), host64(c.wd), g, u,
                          c.token_of, c.entry_of, c.expert_of, c.dtype)
    for n in ("dwg", "dwu", "dwd"):
        # where |g| > 60 the sigmoid's own error is up to |g| 2^-23 of a value below 2^-86: nothing beside the rest
        close(n, host64(o[n]), want[n][0], want[n][1] + 1e-20)


# ---- together ----

def _train(c, router=True, disp=None, saved=None, ws=None, bufs=None, stream=None):
    M = c.M
    n = dict(out=(c.T, c.d), dx=(c.T, c.d), dwg=(c.E, c.F, c.d), dwu=(c.E, c.F, c.d), dwd=(c.E, c.d, c.F))
    if router:
        n["dwr"] = (c.E, c.d)
    o = bufs or {k: c.empty(*v) for k, v in n.items()}
    if bufs is None:
        o["dw"] = c.empty(c.T, c.k, dt=torch.float32)
        if router:
            o["db"] = c.empty(c.E, dt=torch.float32)
    wr = c.wr if router else None
    args = [c.weight(w) for w in (c.wg, c.wu, c.wd)] if not hasattr(c, "packed") else c.packed
    M.moe_forward_save8(c.shape, c.x, wr, c.bias if router else None, c.ids, c.w, *args, o["out"], disp, saved, ws,
                        stream=stream)
    M.moe_backward(c.shape, c.x, wr, c.ids, c.w, *args, disp, saved, c.dout, o["dx"], o["dw"], o.get("dwr"),
                   o.get("db"), o["dwg"], o["dwu"], o["dwd"], ws, stream=stream)
    return o


def _kit(c):
    return dict(disp=c.M.Dispatch(c.shape), saved=c.M.Saved8(c.shape),
                ws=c.M.workspace(max(c.M.workspace_size(c.shape), c.M.backward_workspace_size(c.shape))))


@pytest.mark.parametrize("router", [True, False])
@pytest.mark.parametrize("kw", [
    dict(T=1, d=64, E=8, k=2, F=128), dict(T=12, d=256, E=8, k=2, F=192), dict(T=200, d=256, E=8, k=2, F=320),
    dict(T=300, d=128, E=16, k=4, F=192, cap=40, layout=1), dict(T=64, d=128, E=8, k=2, F=256, dtype="f32"),
    dict(T=900, d=128, E=2, k=1, F=192),
    dict(T=1000, d=12288, E=6, k=1, F=64), dict(T=2060, d=12288, E=4, k=1, F=64),  # the tall tiles, into fp32
], ids=str)
def test_layer_forward_then_backward(kw, router):
    """out is bitwise moe_forward's; the gradients follow, in float64, from the codes that the forward pass left."""
    _need_gpu()
    print(f"\n[gpu] layer {kw} router {router}", flush=True)
    c = Case(**kw)
    c.bias = torch.linspace(-0.5, 0.5, c.E, device="cuda")
    kit = _kit(c)
    o = _train(c, router, **kit)
    ref = c.empty(c.T, c.d)
    ws = c.M.workspace(c.M.workspace_size(c.shape))
    wts = [c.weight(w) for w in (c.wg, c.wu, c.wd)]
    v = c.M.moe_forward(c.shape, c.x, c.wr if router else None, c.bias if router else None,
                        None if router else c.ids, None if router else c.w, *wts, ref, ws)
    assert np.array_equal(bits(o["out"]), bits(ref))
    assert np.array_equal(c.ids.cpu().numpy(), v.topk_ids.cpu().numpy())
    assert np.array_equal(bits(c.w), bits(v.topk_w))
    ids = c.ids.cpu().numpy()
    arr = kit["disp"].arrays()
    row_of, token_of = arr["row_of"].cpu().numpy(), arr["token_of"].cpu().numpy()
    entry_of, expert_of = np.full(c.R, -1), np.full(c.R, -1)
    for f, r in enumerate(row_of):
        entry_of[r], expert_of[r] = f, ids.reshape(-1)[f]
    a = {n: t.cpu().numpy() for n, t in kit["saved"].arrays().items()}
    live = token_of >= 0
    g, u = np.zeros((c.R, c.F)), np.zeros((c.R, c.F))
    g[live] = B.value8(a["gate"], a["gate_exp"])[live]
    u[live] = B.value8(a["up"], a["up_exp"])[live]
    x, w = host64(c.x), host64(c.w)
    want = B.ffn_backward(x, host64(c.dout), w, host64(c.wg), host64(c.wu), host64(c.wd), g, u, token_of, entry_of,
                          expert_of, c.dtype)
    for n in ("dwg", "dwu", "dwd"):
        close(n, c.unweight(o[n]), *want[n])
    dw, e_dw = (z.reshape(c.T, c.k) for z in want["dw"])
    close("dw", host64(o["dw"]), dw, e_dw)
    # dx: rows of dx_perm, here without their own rounding, summed and rounded; the router's part from the GPU's own dw
    dx, e = B.permute_backward(want["dx_perm"][0], row_of, c.T, c.k, c.dtype)
    for f, r in enumerate(row_of):
        e[f // c.k] += want["dx_perm"][1][r] - B.U[c.dtype] * np.abs(want["dx_perm"][0][r])
    if router:
        (dxr, er), (dwr, ew), (db, eb) = B.route_backward(x, host64(c.wr), ids, w, host64(o["dw"]), c.dtype)
        e += er + B.U[c.dtype] * np.abs(dxr) + 4 * c.k * B.U32 * (np.abs(dx) + np.abs(dxr))
        dx = dx + dxr
        close("dwr", host64(o["dwr"]), dwr, ew)
        close("db", host64(o["db"]), db, eb)
    close("dx", host64(o["dx"]), dx, e)


@pytest.mark.parametrize("kw", [
    dict(T=200, d=256, E=8, k=2, F=320), dict(T=300, d=128, E=16, k=4, F=192, cap=40, layout=1),
    dict(T=3, d=64, E=8, k=2, F=128), dict(T=64, d=128, E=8, k=2, F=256, dtype="f32"),
    dict(T=600, d=192, E=16, k=2, F=1536),  # several tiles for each workgroup
], ids=str)
def test_graph_replays_match_eager(kw):
    """Both passes captured into one graph; two graphs share the workspace; eager work in between."""
    _need_gpu()
    print(f"\n[gpu] backward graph {kw}", flush=True)
    c = Case(**kw)
    c.bias = torch.linspace(-0.5, 0.5, c.E, device="cuda")
    c.packed = [c.weight(w) for w in (c.wg, c.wu, c.wd)]
    xs = [c.x.clone(), torch.randn_like(c.x)]
    kit = _kit(c)
    refs = []
    for x in xs:
        c.x.copy_(x)
        refs.append({n: bits(t) for n, t in _train(c, **kit).items()})
    assert not np.array_equal(refs[0]["dx"], refs[1]["dx"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bufs = [_train(c, **kit), _train(c, **kit)]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs = []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _train(c, bufs=b, **kit)
        graphs.append(g)
    torch.cuda.synchronize()
    for rep in range(6):
        which = rep % 2
        c.x.copy_(xs[which])
        for t in bufs[rep // 2 % 2].values():
            t.fill_(float("nan"))
        graphs[rep // 2 % 2].replay()
        torch.cuda.synchronize()
        for n, t in bufs[rep // 2 % 2].items():
            assert np.array_equal(bits(t), refs[which][n]), (rep, n)
        eager = _train(c, **kit)
        assert np.array_equal(bits(eager["dwd"]), refs[which]["dwd"])
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)


def test_stream_argument_and_current_stream():
    _need_gpu()
    c = Case(T=64, d=128, E=4, k=2, F=192)
    c.bias = None
    kit = _kit(c)
    ref = {n: bits(t) for n, t in _train(c, **kit).items()}
    s = torch.cuda.Stream()
    b = _train(c, **kit)
    torch.cuda.synchronize()
    for t in b.values():
        t.zero_()
    torch.cuda.synchronize()
    _train(c, bufs=b, stream=s, **kit)
    s.synchronize()
    for n, t in b.items():
        assert np.array_equal(bits(t), ref[n]), n


def test_two_calls_at_once_with_their_own_buffers():
    _need_gpu()
    cs = [Case(T=150, d=256, E=4, k=2, F=320, seed=s) for s in (0, 1)]
    for c in cs:
        c.bias = None
    kits = [_kit(c) for c in cs]
    refs = [{n: bits(t) for n, t in _train(c, **k).items()} for c, k in zip(cs, kits)]
    bufs = [_train(c, **k) for c, k in zip(cs, kits)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, k, b, s in zip(cs, kits, bufs, streams):
            _train(c, bufs=b, stream=s, **k)
    torch.cuda.synchronize()
    for b, r in zip(bufs, refs):
        for n, t in b.items():
            assert np.array_equal(bits(t), r[n]), n
