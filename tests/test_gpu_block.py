"""The operators around the layer on the GPU: norms, gate, dropout and residual scale and their gradients against
float64 within bounds carried through the formulas (oracle/block.py), over both types, every kind of gate, one row to
many, and widths of every kernel's range; what dropped and odd values may reach; graphs, streams and repeated calls."""
import numpy as np
import pytest

from oracle import block as K
from tests.gpu_helpers import bits, host64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _t(a, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dt).cuda()


def _nan(t):
    return torch.full_like(t, float("nan"))


def close(name, got, value_bound):
    want, bound = value_bound
    got = host64(got).reshape(want.shape)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(err / bound)), np.argwhere(bad)[:4].tolist())


class Case:
    def __init__(self, T, d, dtype="bf16", post=True, gate=None, p=0.0, nxt=True, scale=1.0, seed=0):
        import grouped_gemm_gemv_amd as M
        self.M, self.T, self.d, self.dtype, self.p, self.scale = M, T, d, dtype, p, scale
        rng = np.random.default_rng(seed)
        self.shape = M.Shape(T, d, 1, 1, 64, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
        self.r = M.Residual(EPS, scale, p)
        # rows of very different size, as a residual stream has them
        size = np.exp(rng.uniform(-4, 4, (T, 1)))
        self.res = _t(rng.standard_normal((T, d)) * size, dtype)
        self.y = _t(rng.standard_normal((T, d)) * size[::-1], dtype)
        self.post = _t(1 + 0.3 * rng.standard_normal(d), dtype) if post else None
        self.next = _t(1 + 0.3 * rng.standard_normal(d), dtype) if nxt else None
        self.gate = None if gate is None else _t(rng.standard_normal(T if gate == "token" else (T, d)) * 3, dtype)
        self.dout = _t(rng.standard_normal((T, d)), dtype)
        self.dn = _t(rng.standard_normal((T, d)), dtype) if nxt else None
        self.seed, self.step = (1 << 40) + 12345 + seed, (1 << 33) + 7
        self.rng = torch.tensor([self.seed, self.step], device="cuda") if p else None

    def mask(self):
        if not self.p:
            return None
        t = K.threshold(self.p)
        keep = K.keep(self.p, self.seed, self.step, self.T * self.d).reshape(self.T, self.d)
        return np.where(keep, 65536.0 / (65536 - t), 0.0)

    def h(self, t):
        return None if t is None else host64(t)

    def hgate(self):
        return None if self.gate is None else host64(self.gate).reshape(self.T, -1)

    def forward(self, stream=None):
        out, n = _nan(self.res), _nan(self.res) if self.next is not None else None
        self.M.moe_residual(self.shape, self.r, self.res, self.y, self.post, self.gate, self.rng, self.next, out, n,
                            stream=stream)
        return out, n

    def backward(self, x, stream=None):
        g = {"dres": _nan(self.res), "dy": _nan(self.res),
             "dgate": _nan(self.gate) if self.gate is not None else None,
             "dpost": _nan(self.post) if self.post is not None else None,
             "dnext": _nan(self.next) if self.next is not None else None}
        ws = self.M.workspace(self.M.residual_workspace_size(self.shape))
        self.M.moe_residual_backward(self.shape, self.r, x, self.y, self.post, self.gate, self.rng, self.next,
                                     self.dout, self.dn, *g.values(), ws, stream=stream)
        return {k: v for k, v in g.items() if v is not None}

    def check(self):
        out, n = self.forward()
        want = K.residual(self.h(self.res), self.h(self.y), self.h(self.post), self.hgate(), self.mask(),
                          self.h(self.next), EPS, float(np.float32(self.scale)), self.dtype)
        close("out", out, want["out"])
        if n is not None:
            close("n", n, want["n"])
        got = self.backward(out)
        want = K.residual_backward(self.h(out), self.h(self.y), self.h(self.post), self.hgate(), self.mask(),
                                   self.h(self.next), self.h(self.dout), self.h(self.dn), EPS,
                                   float(np.float32(self.scale)), self.dtype)
        assert set(got) == set(want)
        for name in got:
            close(name, got[name], want[name])


# every width's kernel: 64, 256 and 512 threads of a row, with one to four vectors each, full and not
WIDTHS = [64, 128, 448, 512, 576, 1024, 1088, 2048, 2112, 3584, 4096, 4160, 8192, 8256, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_every_width(d, dtype):
    print(f"\n[gpu] residual d={d} {dtype}", flush=True)
    Case(7, d, dtype, gate="token", p=0.25 if d <= 512 else 0.0, scale=0.5, seed=d).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,gate,p,nxt", [
    (True, None, 0.0, True), (False, None, 0.0, False), (True, "token", 0.5, True), (False, "token", 0.1, False),
    (True, "full", 0.1, False), (False, "full", 0.9, True), (False, "token", 0.0, True), (True, "full", 0.0, True),
    (False, None, 0.3, True),
])
@pytest.mark.parametrize("T,d", [(1, 320), (33, 128), (3, 1216)])
def test_every_combination(T, d, post, gate, p, nxt, dtype):
    print(f"\n[gpu] residual T={T} d={d} post={post} gate={gate} p={p} next={nxt} {dtype}", flush=True)
    Case(T, d, dtype, post, gate, p, nxt, scale=-0.75, seed=T).check()


@pytest.mark.parametrize("T,d", [(2049, 64), (4099, 64), (1500, 1088), (515, 2048)])
def test_many_rows_for_a_workgroup(T, d):
    # more rows than the gradient has workgroups: each sums several, unevenly
    print(f"\n[gpu] residual T={T} d={d}", flush=True)
    Case(T, d, "bf16", gate="full", seed=1).check()
    Case(T, d, "f32", post=False, gate="token", seed=2).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 64), (5, 512), (700, 640), (1030, 2048), (3, 16384)])
def test_norm_and_its_gradient(T, d, dtype):
    print(f"\n[gpu] norm T={T} d={d} {dtype}", flush=True)
    import grouped_gemm_gemv_amd as M
    c = Case(T, d, dtype, seed=4)
    n = _nan(c.res)
    M.moe_norm(c.shape, c.res, c.next, n, eps=EPS)
    close("n", n, K.norm(host64(c.res), host64(c.next), EPS, dtype))
    ws = M.workspace(M.residual_workspace_size(c.shape))
    for dres in (None, c.dout):
        dx, dw = _nan(c.res), _nan(c.next)
        M.moe_norm_backward(c.shape, c.res, c.next, c.dn, dres, dx, dw, ws, eps=EPS)
        want = K.residual_backward(host64(c.res), None, None, None, None, host64(c.next), c.h(dres), host64(c.dn), EPS,
                                   1.0, dtype)
        close("dx", dx, want["dres"])
        close("dw", dw, want["dnext"])
        again = _nan(c.res)
        M.moe_norm_backward(c.shape, c.res, c.next, c.dn, dres, again, None, ws, eps=EPS)  # no weight gradient
        assert np.array_equal(bits(dx), bits(again))


def test_rows_of_zeros_have_norm_zero():
    import grouped_gemm_gemv_amd as M
    c = Case(4, 256)
    c.y[1], c.res[1] = 0, 0  # a padded row
    out, n = c.forward()
    assert (out[1] == 0).all() and (n[1] == 0).all() and torch.isfinite(n.float()).all()
    g = c.backward(out)
    assert all(torch.isfinite(v.float()).all() for v in g.values())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
def test_dropped_elements_reach_nothing(bad):
    """What a dropped element holds is in no output, without a norm that reads the whole row."""
    c = Case(5, 256, "f32", post=False, gate="token", p=0.5, seed=3)
    out, n = c.forward()
    g = c.backward(out)
    dropped = torch.from_numpy(c.mask() == 0).cuda()
    c.y = torch.where(dropped, torch.full_like(c.y, bad), c.y)
    out2, n2 = c.forward()
    g2 = c.backward(out)
    assert np.array_equal(bits(out), bits(out2)) and np.array_equal(bits(n), bits(n2))
    for name in g:
        assert np.array_equal(bits(g[name]), bits(g2[name])), name
    import grouped_gemm_gemv_amd as M
    z = _nan(c.y)
    M.moe_dropout(c.y, c.p, c.rng, z)
    assert (z[dropped] == 0).all() and torch.isfinite(z).all()


def test_a_bad_row_stays_in_its_row():
    c = Case(6, 512, gate="full", p=0.0)
    out, n = c.forward()
    c.y[2, 5] = float("nan")
    out2, n2 = c.forward()
    for a, b in ((out, out2), (n, n2)):
        rest = [0, 1, 3, 4, 5]
        assert np.array_equal(bits(a)[rest], bits(b)[rest])
    assert torch.isnan(out2[2].float()).all() and torch.isnan(n2[2].float()).all()


def test_closed_and_open_gates():
    # sigmoid at both ends, where its slope vanishes and nothing may overflow
    c = Case(4, 256, "f32", gate="full")
    c.gate[0], c.gate[1], c.gate[2], c.gate[3] = -200.0, 200.0, float("-inf"), float("inf")
    out, _ = c.forward()
    assert torch.equal(out[0], c.res[0]) and torch.equal(out[2], c.res[2])
    g = c.backward(out)
    assert (g["dgate"] == 0).all() and (g["dy"][[0, 2]] == 0).all()
    assert all(torch.isfinite(v).all() for v in g.values())


# ---- dropout alone ----


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,p", [(1, 0.5), (7, 0.5), (8, 0.3), (9, 0.9), (1000, 0.1), (4099, 0.0), (70001, 0.99999)])
def test_dropout_bitwise(n, p, dtype):
    """The products have one rounding each, so every bit is known."""
    import grouped_gemm_gemv_amd as M
    x = _t(np.random.default_rng(n).standard_normal(n), dtype)
    seed, step = 0x7abcdef012345678, 3
    rng = torch.tensor([seed, step], device="cuda")
    out = _nan(x)
    M.moe_dropout(x, p, rng, out)
    t = K.threshold(p)
    scale = np.float32(65536.0) / np.float32(65536 - t)
    want = torch.from_numpy(np.where(K.keep(p, seed, step, n), x.float().cpu().numpy() * scale, np.float32(0)))
    assert np.array_equal(bits(out), bits(want.to(x.dtype)))
    M.moe_dropout(x, p, rng, x)  # in place
    assert np.array_equal(bits(out), bits(x))
    empty = x[:0]
    M.moe_dropout(empty, p, rng, empty)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_of_odd_values(dtype):
    """Subnormal numbers, zeros of both signs, infinities and the largest values keep their bits' meaning."""
    import grouped_gemm_gemv_amd as M
    vals = [0.0, -0.0, 1e-38, -1e-39, 1e-40, 9.2e-41, 3.3e38, -3.38e38, float("inf"), float("-inf"), float("nan"), 1.0]
    x = _t(np.resize(np.array(vals), 6000), dtype)
    rng = torch.tensor([3, 4], device="cuda")
    out = _nan(x)
    M.moe_dropout(x, 0.25, rng, out)
    t = K.threshold(0.25)
    scale = np.float32(65536.0) / np.float32(65536 - t)
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(K.keep(0.25, 3, 4, x.numel()), x.float().cpu().numpy() * scale, np.float32(0))
    want = torch.from_numpy(want).to(x.dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    live = ~torch.isnan(want)
    assert np.array_equal(bits(got[live]), bits(want[live]))


def test_dropout_masks_differ_by_step_and_seed_and_agree_with_the_fused_one():
    import grouped_gemm_gemv_amd as M
    T, d, p = 16, 1024, 0.5
    x = torch.ones(T, d, device="cuda")
    masks = []
    for seed, step in ((1, 0), (1, 1), (2, 0), (1, 1 << 32), (1 << 32, 0)):
        out = _nan(x)
        M.moe_dropout(x, p, torch.tensor([seed, step], device="cuda"), out)
        masks.append(out != 0)
    n = T * d
    for i in range(5):
        for j in range(i):  # independent masks agree at half of the places: five standard deviations
            assert abs((masks[i] == masks[j]).sum().item() - n / 2) < 5 * (n / 4) ** 0.5
    shape = M.Shape(T, d, 1, 1, 64, dtype=torch.float32)
    out = _nan(x)
    M.moe_residual(shape, M.Residual(dropout=p), torch.zeros_like(x), x, None, None,
                   torch.tensor([1, 1], device="cuda"), None, out, None)
    assert torch.equal(out != 0, masks[1])


def test_dropout_past_2_31_elements():
    import grouped_gemm_gemv_amd as M
    n = (1 << 31) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    seed, step, p = 5, 6, 0.5
    M.moe_dropout(x, p, torch.tensor([seed, step], device="cuda"), x)
    for at in (0, (1 << 31) - 64, n - 88):
        words = K.philox(np.arange(at // 8, at // 8 + 11, dtype=np.uint64), step, seed)
        halves = np.stack([words & 0xFFFF, words >> 16], axis=-1).reshape(-1)[:88]
        assert np.array_equal(x[at:at + 88].float().cpu().numpy(), np.where(halves >= 32768, 2.0, 0.0)), at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_any_size_and_a_small_eps(dtype):
    """1 / rms of 1e-15 to 1e15, whose cube no fp32 number holds, and rows of zeros beside an eps of 1e-30."""
    import grouped_gemm_gemv_amd as M
    eps = 1e-30
    c = Case(7, 320, dtype, gate="token", scale=0.5, seed=8)
    c.r = M.Residual(eps, c.scale, 0.0)
    rng = np.random.default_rng(80)
    for t, (a, b) in enumerate([(1e15, 1e-15), (1e-15, 1e15), (1e15, 1e15), (1e-15, 1e-15), (0, 0), (1, 0), (0, 1)]):
        c.res[t], c.y[t] = _t(rng.standard_normal(320) * a, dtype), _t(rng.standard_normal(320) * b, dtype)
    out, n = c.forward()
    want = K.residual(c.h(c.res), c.h(c.y), c.h(c.post), c.hgate(), None, c.h(c.next), float(np.float32(eps)), 0.5, dtype)
    close("out", out, want["out"])
    close("n", n, want["n"])
    c.res[4] = 0
    x = c.res  # (any row may stand for the sum)
    got = c.backward(x)
    want = K.residual_backward(c.h(x), c.h(c.y), c.h(c.post), c.hgate(), None, c.h(c.next), c.h(c.dout), c.h(c.dn),
                               float(np.float32(eps)), 0.5, dtype)
    for name in ("dres", "dy", "dpost", "dnext"):
        assert torch.isfinite(got[name].float()).all(), name
        close(name, got[name], want[name])


def test_rows_past_2_31_elements():
    """The last rows of arrays of 4.4 GB are those of a small batch of their own; their masks those of the flat array."""
    import grouped_gemm_gemv_amd as M
    T, d, last = 270000, 8192, 3
    c, bf = Case(last, d, gate="token", seed=10), torch.bfloat16
    big = M.Shape(T, d, 1, 1, 64, dtype=bf)
    want, want_n = c.forward()
    g = c.backward(want)

    def grown(v):
        b = torch.ones((T,) + tuple(v.shape[1:]), dtype=bf, device="cuda")
        b[-last:] = v
        return b

    res, y, gate = grown(c.res), grown(c.y), grown(c.gate)
    out, n = torch.empty_like(res), torch.empty_like(res)
    M.moe_residual(big, c.r, res, y, c.post, gate, None, c.next, out, n)
    assert np.array_equal(bits(out[-last:]), bits(want)) and np.array_equal(bits(n[-last:]), bits(want_n))
    dout, dn = grown(c.dout), grown(c.dn)
    dres, dy, dgate = res, n, torch.empty_like(gate)
    M.moe_residual_backward(big, c.r, out, y, c.post, gate, None, c.next, dout, dn, dres, dy, dgate, None, None,
                            M.workspace(M.residual_workspace_size(big)))
    for name, v in (("dres", dres), ("dy", dy), ("dgate", dgate)):
        assert np.array_equal(bits(v[-last:]), bits(g[name])), name
    rng = torch.tensor([77, 3], device="cuda")
    M.moe_residual(big, M.Residual(dropout=0.5), dres.zero_(), y, None, None, rng, None, out, None)
    M.moe_dropout(y, 0.5, rng, dn)
    assert torch.equal(out[-2 * last:], dn[-2 * last:]) and torch.equal(out[131070:131075], dn[131070:131075])


# ---- how calls may be made ----


def test_in_place_results_are_the_same():
    c = Case(40, 2112, gate="token", p=0.2)
    out, n = c.forward()
    g = c.backward(out)
    res, dout = c.res.clone(), c.dout.clone()
    n2 = _nan(n)
    c.M.moe_residual(c.shape, c.r, res, c.y, c.post, c.gate, c.rng, c.next, res, n2)
    assert np.array_equal(bits(res), bits(out)) and np.array_equal(bits(n2), bits(n))
    dy = _nan(out)
    ws = c.M.workspace(c.M.residual_workspace_size(c.shape))
    c.M.moe_residual_backward(c.shape, c.r, out, c.y, c.post, c.gate, c.rng, c.next, dout, c.dn, dout, dy, None, None,
                              None, ws)
    assert np.array_equal(bits(dout), bits(g["dres"])) and np.array_equal(bits(dy), bits(g["dy"]))


@pytest.mark.parametrize("gate", ["token", "full"])
def test_arrays_at_their_least_alignment(gate):
    def shifted(t, by):
        b = torch.zeros(t.numel() * t.element_size() + by + 64, dtype=torch.uint8, device="cuda")
        return b[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape).copy_(t)

    c = Case(9, 448, gate=gate, p=0.3, seed=17)
    out, n = c.forward()
    g = c.backward(out)
    for name in ("res", "y", "post", "next", "dout", "dn"):
        setattr(c, name, shifted(getattr(c, name), 16))
    c.gate, c.rng = shifted(c.gate, 2 if gate == "token" else 16), shifted(c.rng, 8)
    out2, n2 = c.forward()
    g2 = c.backward(shifted(out2, 16))
    assert np.array_equal(bits(out), bits(out2)) and np.array_equal(bits(n), bits(n2))
    for name in g:
        assert np.array_equal(bits(g[name]), bits(g2[name])), name


def test_rows_behind_the_last_stay_as_they_were():
    import grouped_gemm_gemv_amd as M
    T, d = 5, 192
    c = Case(T, d)
    big = torch.full((T + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    M.moe_norm(c.shape, c.res, c.next, big[:T], eps=EPS)
    assert (big[T:] == 7).all() and not (big[:T] == 7).all()


def test_no_gradient_from_the_sum_is_a_gradient_of_zero():
    c = Case(9, 320, gate="full")
    out, _ = c.forward()
    c.dout = torch.zeros_like(c.dout)
    want = c.backward(out)
    c.dout = None
    got = c.backward(out)
    for name in want:
        assert np.array_equal(bits(got[name]), bits(want[name])), name


def test_repeats_streams_and_graph_replays_are_bitwise_equal():
    c = Case(600, 1088, gate="token", p=0.3)
    out, n = c.forward()
    g = c.backward(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, n2 = c.forward(stream=side)
    g2 = c.backward(out2, stream=side)
    side.synchronize()
    assert np.array_equal(bits(out), bits(out2)) and np.array_equal(bits(n), bits(n2))
    for name in g:
        assert np.array_equal(bits(g[name]), bits(g2[name])), name

    # a captured pass: another step of the generator and other inputs on each replay
    M = c.M
    ws = M.workspace(M.residual_workspace_size(c.shape))
    o, nn = _nan(out), _nan(n)
    gr = {k: _nan(v) for k, v in g.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_residual(c.shape, c.r, c.res, c.y, c.post, c.gate, c.rng, c.next, o, nn)
        M.moe_residual_backward(c.shape, c.r, o, c.y, c.post, c.gate, c.rng, c.next, c.dout, c.dn, gr["dres"], gr["dy"],
                                gr["dgate"], gr["dpost"], gr["dnext"], ws)
    for i in range(3):
        c.rng[1] = 100 + i
        c.y.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        out, n = c.forward()
        g = c.backward(out)
        torch.cuda.synchronize()
        assert np.array_equal(bits(o), bits(out)) and np.array_equal(bits(nn), bits(n)), i
        for name in g:
            assert np.array_equal(bits(gr[name]), bits(g[name])), (i, name)


def test_refusals_on_the_device():
    import grouped_gemm_gemv_amd as M
    c = Case(4, 128, gate="token")
    out = _nan(c.res)
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_norm(c.shape, torch.zeros(128, 4, dtype=torch.bfloat16, device="cuda").t(), c.next, out)
    with pytest.raises(ValueError, match="must be"):
        M.moe_norm(c.shape, c.res.float(), c.next, out)
    with pytest.raises(ValueError, match="rng must be"):
        M.moe_residual(c.shape, M.Residual(dropout=0.5), c.res, c.y, None, None, torch.zeros(2, device="cuda"), None,
                       out, None)
    with pytest.raises(RuntimeError, match="NULL"):
        M.moe_residual(c.shape, M.Residual(dropout=0.5), c.res, c.y, None, None, None, None, out, None)
    with pytest.raises(RuntimeError, match="INVALID"):  # a view that starts off a 16-byte boundary
        flat = torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")
        M.moe_norm(c.shape, flat[1:].view(4, 128), c.next, out)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        M.moe_norm_backward(c.shape, c.res, c.next, c.dn, None, out, None, torch.empty(16, dtype=torch.uint8, device="cuda"))
