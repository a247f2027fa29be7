"""Backward calls at the ends of their ranges: arrays past 2^31 elements, 256
experts, a single expert and token, no live entry at all, the two passes of a
capacity one at a time, a dispatch of another tile height."""
import numpy as np
import pytest

from oracle import backward as B
from tests.gpu_helpers import bits, host64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _check_ffn(c, saved, g, u, o):
    from tests.test_gpu_backward import close
    want = B.ffn_backward(host64(c.x), host64(c.dout), host64(c.w), host64(c.wg), host64(c.wu), host64(c.wd), g, u,
                          c.token_of, c.entry_of, c.expert_of, c.dtype)
    close("dx_perm", host64(o["dx_perm"])[c.live], want["dx_perm"][0][c.live], want["dx_perm"][1][c.live])
    close("dw", host64(o["dw"]).reshape(-1), *want["dw"])
    for n in ("dwg", "dwu", "dwd"):
        close(n, c.unweight(o[n]), *want[n])


@pytest.mark.parametrize("kw", [
    dict(T=300, d=64, E=256, k=4, F=128), dict(T=90, d=64, E=256, k=2, F=64, dtype="f32", cap=1),
    dict(T=1, d=64, E=1, k=1, F=64), dict(T=1, d=64, E=1, k=1, F=64, dtype="f32"),
    dict(T=70, d=64, E=1, k=1, F=64, cap=33, layout=1), dict(T=3, d=64, E=64, k=64, F=64),
], ids=str)
def test_most_and_fewest_experts(kw):
    _need_gpu()
    from tests.test_gpu_backward import Case, _ffn
    print(f"\n[gpu] reach {kw}", flush=True)
    c = Case(**kw)
    saved, g, u = c.saved()
    _check_ffn(c, saved, g, u, _ffn(c, saved))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_live_entry(dtype):
    """Every id is invalid: gradients of all weights, of x and of the routing weights are zeros."""
    _need_gpu()
    from tests.test_gpu_backward import Case, _kit, _train
    print(f"\n[gpu] no live entry {dtype}", flush=True)
    c = Case(T=37, d=128, E=4, k=2, F=192, dtype=dtype)
    c.ids.fill_(-1)
    for t in (c.x, c.dout, c.w):
        t.fill_(float("nan"))
    kit = _kit(c)
    o = _train(c, router=False, **kit)
    for n in ("dx", "dw", "dwg", "dwu", "dwd"):
        assert (o[n] == 0).all(), n
    g = {"dx": c.empty(c.T, c.d), "dwr": c.empty(c.E, c.d), "db": c.empty(c.E, dt=torch.float32)}
    c.M.moe_route_backward(c.shape, c.x, c.wr, c.ids, c.w, c.w, g["dx"], g["dwr"], g["db"], kit["ws"])
    for n, t in g.items():
        assert (t == 0).all(), n


def test_save8_one_pass_at_a_time():
    """Pass 0 writes the rows of the fixed region, pass 1 those behind it; together they are both passes in one."""
    _need_gpu()
    from tests.test_gpu_backward import Case
    print("\n[gpu] save8, pass by pass", flush=True)
    c = Case(T=200, d=128, E=6, k=2, F=192, cap=25)
    M, first = c.M, c.E * 25
    h, ref = c.empty(c.R, c.F), c.empty(c.R, c.F)
    one, both = M.Saved8(c.shape), M.Saved8(c.shape)
    for s in (one, both):
        for a in s.arrays().values():
            a.fill_(77)
    M.moe_ffn_gate_up_save8(c.shape, c.x, c.wg, c.wu, c.disp, M.PASS_BOTH, ref, both)
    M.moe_ffn_gate_up_save8(c.shape, c.x, c.wg, c.wu, c.disp, 0, h, one)
    assert torch.isnan(h[first:]).all() and (one.arrays()["gate"][first:] == 77).all()
    M.moe_ffn_gate_up_save8(c.shape, c.x, c.wg, c.wu, c.disp, 1, h, one)
    assert np.array_equal(bits(h), bits(ref))
    for n, a in one.arrays().items():
        assert torch.equal(a, both.arrays()[n]), n


def test_backward_with_a_dispatch_of_another_tile_height():
    _need_gpu()
    from tests.test_gpu_backward import Case, _ffn
    print("\n[gpu] other tile height", flush=True)
    c = Case(T=120, d=128, E=4, k=2, F=192)
    saved, _, _ = c.saved()
    ref = _ffn(c, saved)
    tall = c.M.Dispatch(c.M.Shape(c.T, c.d, c.E, c.k, c.F, 0, c.dt, tile_rows=384))
    c.M.moe_permute(c.shape, c.x, c.ids, tall, c.empty(c.R, c.d), c.M.workspace(c.M.query(c.shape).permute_ws_bytes))
    c.disp = tall
    o = _ffn(c, saved)
    for n in o:
        assert np.array_equal(bits(o[n]), bits(ref[n])), n


def test_arrays_past_32_bits():
    """2.4 10^9 codes of each projection, and as many values in every array of [R, F]: the last rows, whose offsets
    pass 2^31, against float64; the rows before them have routing weight 0 and contribute exact zeros."""
    _need_gpu()
    import grouped_gemm_gemv_amd as M
    from tests.test_gpu_backward import close
    print("\n[gpu] past 32 bits", flush=True)
    T, d, E, F, n = 146000, 64, 2, 16448, 96
    s = M.Shape(T, d, E, 1, F)
    assert T * F > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    x, dout = rnd(T, d), rnd(T, d)
    wg, wu, wd = rnd(E, F, d, std=0.2), rnd(E, F, d, std=0.2), rnd(E, d, F, std=0.01)
    ids = torch.ones(T, 1, dtype=torch.int32, device="cuda")
    ids[0] = 0  # one row of expert 0, so that expert 1's do not start at 0
    w = torch.zeros(T, 1, device="cuda")
    w[-n:] = torch.rand(n, 1, generator=gen, device="cuda") + 0.5
    out, disp, saved = torch.empty_like(x), M.Dispatch(s), M.Saved8(s)
    ws = M.workspace(max(M.workspace_size(s), M.backward_workspace_size(s)))
    M.moe_forward_save8(s, x, None, None, ids, w, wg, wu, wd, out, disp, saved, ws)
    val = [torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    M.moe_saved8_unpack(s, saved, disp, *val)
    xs = host64(x[-n:])
    kept = []
    for wt, v, name in ((wg, val[0], "gate"), (wu, val[1], "up")):
        p, mag = xs @ host64(wt[1]).T, np.abs(xs) @ np.abs(host64(wt[1])).T
        b = saved.arrays()[name + "_exp"][-n:].cpu().numpy().astype(np.float64)
        codes = saved.arrays()[name][-n:].cpu().numpy().astype(int)
        step = np.repeat(2.0 ** (b - 133), 16, axis=1)
        kept.append(host64(v[-n:]))
        assert np.array_equal(kept[-1], codes * step)
        # half a step, a whole one where clamped, and the fp32 sum's rounding
        assert (np.abs(kept[-1] - p) <= np.where(np.abs(codes) == 127, 1.0, 0.5) * step + (d + 8) * B.U32 * mag).all()
    del val
    dx, dw = torch.full_like(x, float("nan")), torch.full((T, 1), float("nan"), device="cuda")
    g = [torch.full_like(t, float("nan")) for t in (wg, wu, wd)]
    M.moe_backward(s, x, None, ids, w, wg, wu, wd, disp, saved, dout, dx, dw, None, None, *g, ws)
    assert (dx[:-n] == 0).all() and all((t[0] == 0).all() for t in g)
    one = np.ones(n, dtype=int)
    want = B.ffn_backward(xs, host64(dout[-n:]), host64(w[-n:]), host64(wg), host64(wu), host64(wd), *kept,
                          np.arange(n), np.arange(n), one, "bf16")
    close("dx", host64(dx[-n:]), *want["dx_perm"])
    close("dw", host64(dw[-n:]).reshape(-1), *want["dw"])
    # sums over T rows of which all but n are exact zeros
    for name, t in zip(("dwg", "dwu", "dwd"), g):
        close(name, host64(t[1]), want[name][0][1], want[name][1][1])
