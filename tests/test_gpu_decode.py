"""The layer for a few tokens on the GPU, against float64 within bounds carried through the formulas and against the
layer's own forward pass: both types and E4M3 weights, both storage orders, one token to sixteen, given and computed
routing, masked, repeated and missing experts, values that must not spread, graphs and streams."""
import numpy as np
import pytest

from oracle import block as K
from oracle import moe_oracle as O
from tests.gpu_helpers import bits, check_routing, host64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _t(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dt).cuda()


class Case:
    def __init__(self, T, d, E, k, F, dtype="bf16", norm=True, res=True, layout=0, fp8=False, bias=False, given=None,
                 scale=1.0, cap=0, seed=0):
        import grouped_gemm_gemv_amd as M
        self.M, self.dtype, self.fp8, self.scale = M, dtype, fp8, scale
        self.T, self.d, self.E, self.k, self.F = T, d, E, k, F
        rng = np.random.default_rng(seed)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.shape = M.Shape(T, d, E, k, F, cap, dt, 0, layout)
        self.x = _t(rng.standard_normal((T, d)) * 2, dt)
        self.norm = _t(1 + 0.3 * rng.standard_normal(d), dt) if norm else None
        self.wr = _t(rng.standard_normal((E, d)) * 1.5 / np.sqrt(d), dt)
        self.bias = _t(0.3 * rng.standard_normal(E), torch.float32) if bias else None
        self.res = _t(rng.standard_normal((T, d)), dt) if res else None
        raw = [rng.standard_normal((E, F, d)) * 1.2 / np.sqrt(d), rng.standard_normal((E, F, d)) * 1.2 / np.sqrt(d),
               rng.standard_normal((E, d, F)) / np.sqrt(F)]
        self.scales = None
        if fp8:
            self.scales = [_t(np.abs(w).max(axis=2) / 448 * rng.uniform(1, 2, w.shape[:2]), torch.float32) for w in raw]
            self.w = [(torch.from_numpy(w).float().cuda() / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
                      for w, s in zip(raw, self.scales)]
            self.w64 = [w.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64) *
                        host64(s)[:, :, None] for w, s in zip(self.w, self.scales)]
        else:
            self.w = [_t(w, dt) for w in raw]
            self.w64 = [host64(w) for w in self.w]
        self.ids = self.tw = None
        if given is not None:
            ids, w = given(rng)
            self.ids = torch.from_numpy(np.ascontiguousarray(ids, dtype=np.int32)).cuda()
            self.tw = torch.from_numpy(np.ascontiguousarray(w, dtype=np.float32)).cuda()
        self.ws = M.workspace(M.decode_workspace_size(self.shape))
        self.ws.fill_(0xFF)  # whatever an earlier call left

    def stored(self):
        return [self.M.moe_pack_blocked16(w) for w in self.w] if self.shape.weight_layout else self.w

    def run(self, ids=None, w=None, out=None, stream=None, weights=None, ws=None):
        M = self.M
        if out is None:
            out = torch.full_like(self.x, float("nan"))
        given = self.ids is not None
        args = (self.shape, self.x, self.norm, None if given else self.wr, self.bias, self.ids if given else ids,
                self.tw if given else w) + tuple(weights if weights is not None else self.stored())
        if self.fp8:
            args += tuple(self.scales)
        fn = M.moe_decode_fp8 if self.fp8 else M.moe_decode
        fn(*args, self.res, out, ws if ws is not None else self.ws, eps=EPS, scale=self.scale, stream=stream)
        return out

    def logits(self):
        x, wr = host64(self.x), host64(self.wr)
        m = x * K.rms(x, EPS) * host64(self.norm) if self.norm is not None else x
        z = m @ wr.T + (host64(self.bias) if self.bias is not None else 0.0)
        bound = (self.d + 80) * K.U32 * (np.abs(m) @ np.abs(wr).T) + 2 * K.U32 * np.abs(z)
        return z, bound

    def check(self):
        ids = torch.full((self.T, self.k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((self.T, self.k), float("nan"), device="cuda")
        got = self.run(ids, w)
        e_w = 0.0
        if self.ids is None:
            z, e_z = self.logits()
            gi, gw = ids.cpu().numpy(), w.cpu().numpy()
            check_routing(gi, gw, z, self.k)
            sel = np.take_along_axis(z, gi.astype(np.int64), axis=1)
            p = np.exp(sel - sel.max(axis=1, keepdims=True))
            ids, tw = gi, p / p.sum(axis=1, keepdims=True)
            e_w = 2.5 * float(e_z.max()) + 16 * K.U32  # a softmax weight moves by at most twice its logits' error
        else:
            ids, tw = self.ids.cpu().numpy(), host64(self.tw)
        want, bound = K.decode(host64(self.x), None if self.norm is None else host64(self.norm), EPS, ids, tw,
                               *self.w64, None if self.res is None else host64(self.res),
                               float(np.float32(self.scale)), self.dtype, e_w)
        err = np.abs(host64(got) - want)
        assert (err <= bound).all(), (int((~(err <= bound)).sum()), float(np.nanmax(err / bound)))
        # and over the whole output: the roundings of m (twice, for gate and up), h and out at half a step each,
        # which only add up in full where they all agree
        branch = want - (host64(self.res) if self.res is not None else 0.0)
        u = K.U[self.dtype] if self.dtype == "bf16" else 64 * K.U32
        assert np.linalg.norm(err) <= 3 * u * np.linalg.norm(branch) + u * np.linalg.norm(want)
        return got


SHAPES = [
    dict(T=1, d=64, E=1, k=1, F=64), dict(T=1, d=128, E=8, k=2, F=256), dict(T=2, d=192, E=3, k=3, F=192),
    dict(T=5, d=448, E=16, k=4, F=320), dict(T=8, d=512, E=17, k=5, F=128), dict(T=9, d=256, E=64, k=8, F=64),
    dict(T=16, d=320, E=5, k=2, F=448), dict(T=16, d=64, E=256, k=64, F=64), dict(T=3, d=1088, E=65, k=1, F=704),
    dict(T=13, d=128, E=40, k=40, F=192),
]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("kw", SHAPES, ids=str)
def test_shapes(kw, dtype, fp8, layout):
    print(f"\n[gpu] decode {kw} {dtype} fp8={fp8} layout={layout}", flush=True)
    Case(**kw, dtype=dtype, fp8=fp8, layout=layout, seed=kw["T"]).check()


@pytest.mark.parametrize("T", range(1, 17))
def test_every_number_of_tokens(T):
    print(f"\n[gpu] decode T={T}", flush=True)
    for dtype, fp8 in (("bf16", False), ("f32", False), ("bf16", True)):
        Case(T, 256, 8, 2, 192, dtype=dtype, fp8=fp8, seed=100 + T).check()


@pytest.mark.parametrize("norm,res,bias,scale", [(False, False, False, 1.0), (True, False, True, 1.0),
                                                 (False, True, True, 0.5), (True, True, True, -2.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts(norm, res, bias, scale, dtype):
    print(f"\n[gpu] decode norm={norm} res={res} bias={bias} scale={scale} {dtype}", flush=True)
    Case(6, 384, 12, 3, 256, dtype=dtype, norm=norm, res=res, bias=bias, scale=scale, seed=7).check()


@pytest.mark.parametrize("dtype,T,d,E,k,F", [
    ("bf16", 16, 4096, 4, 2, 640),   # x takes 128 KB of LDS
    ("f32", 8, 4096, 4, 2, 192), ("bf16", 1, 16384, 2, 1, 128), ("bf16", 2, 4096, 8, 2, 1408),
    ("bf16", 4, 2048, 64, 6, 704),
])
def test_wide_rows(dtype, T, d, E, k, F):
    print(f"\n[gpu] decode {dtype} T={T} d={d} E={E} k={k} F={F}", flush=True)
    Case(T, d, E, k, F, dtype=dtype, layout=1, seed=11).check()


@pytest.mark.parametrize("T,d,E,k,F,fp8,layout", [
    (16, 2304, 4, 2, 128, False, 0), (12, 3584, 4, 2, 192, True, 1),  # x once in LDS, routed beside the products
    (16, 4096, 80, 8, 64, True, 1), (16, 4096, 80, 8, 64, False, 0),  # all of LDS: 141312 bytes of x, logits and weights
    (9, 4096, 256, 16, 64, False, 1),                                 # four experts of a lane
    (1, 70592, 1, 1, 64, False, 0), (1, 70592, 2, 1, 64, True, 1),    # the widest row, four thousand tiles of columns
    (16, 2048, 20, 3, 64, False, 0),                                  # both terms in LDS, instructions of their own
])
def test_wide_rows_with_a_router(T, d, E, k, F, fp8, layout):
    print(f"\n[gpu] decode T={T} d={d} E={E} k={k} F={F} fp8={fp8} layout={layout}", flush=True)
    Case(T, d, E, k, F, fp8=fp8, layout=layout, bias=True, seed=T + E).check()


def _given(T, k, E, drop=0.2):
    def make(rng):
        ids = rng.integers(0, E, (T, k))  # the same expert may come twice
        ids[rng.random((T, k)) < drop] = rng.choice([-1, E, 1 << 30])
        return ids, rng.standard_normal((T, k))
    return make


@pytest.mark.parametrize("T,d,E,F", [(3, 256, 4, 192), (8, 1024, 4, 256), (9, 256, 4, 192), (16, 1024, 5, 320),
                                     (16, 2304, 4, 128), (16, 4096, 4, 192), (8, 6144, 4, 128), (1, 512, 4, 64)])
@pytest.mark.parametrize("layout,fp8", [(0, False), (1, False), (0, True), (1, True)])
@pytest.mark.parametrize("norm", [True, False])
def test_bf16_is_rounded_once(T, d, E, F, layout, fp8, norm):
    """p and h are kept in two terms each, wherever the second ones are, so all that is left is the output's rounding:
    even over a step, which is 2^-7 |v| at the most, that is a root mean square of 2^-7 |v| / sqrt(12) at the most
    (0.0023; over the values of a step about 0.0017).  One term of both comes to 0.0029."""
    print(f"\n[gpu] decode rounded once T={T} d={d} E={E} F={F} layout={layout} fp8={fp8} norm={norm}", flush=True)
    c = Case(T, d, E, 2, F, fp8=fp8, norm=norm, res=False, layout=layout, given=_given(T, 2, E, drop=0.0), seed=T + d)
    got = c.check()
    want, _ = K.decode(host64(c.x), None if c.norm is None else host64(c.norm), EPS, c.ids.cpu().numpy(), host64(c.tw),
                       *c.w64, None, 1.0, "bf16")
    err = np.linalg.norm(host64(got) - want) / np.linalg.norm(want)
    assert err <= 2.0**-7 / 12**0.5, err


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (7, 3, 3), (16, 100, 6)])
def test_given_routing_with_repeats_and_gaps(T, E, k, dtype, fp8):
    print(f"\n[gpu] decode given T={T} E={E} k={k} {dtype} fp8={fp8}", flush=True)
    Case(T, 192, E, k, 128, dtype=dtype, fp8=fp8, given=_given(T, k, E), seed=T).check()


def test_slots_without_an_expert_may_hold_anything():
    c = Case(5, 128, 6, 3, 64, given=_given(5, 3, 6, 0.4), seed=2)
    want = c.run()
    c.tw = torch.where((c.ids < 0) | (c.ids >= 6), torch.full_like(c.tw, float("nan")), c.tw)
    assert np.array_equal(bits(c.run()), bits(want))


@pytest.mark.parametrize("fp8", [False, True])
def test_no_expert_at_all(fp8):
    c = Case(4, 128, 4, 2, 64, fp8=fp8, given=lambda rng: (np.full((4, 2), -1), np.ones((4, 2))))
    assert np.array_equal(bits(c.run()), bits(c.res))
    c.res = None
    assert (c.run() == 0).all()


def test_bias_of_minus_infinity_masks_an_expert():
    c = Case(8, 256, 6, 2, 64, bias=True, seed=3)
    c.bias[1], c.bias[4] = float("-inf"), float("-inf")
    for w in c.w:  # not even read
        w[1], w[4] = float("nan"), float("nan")
    ids = torch.empty(8, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(8, 2, device="cuda")
    out = c.run(ids, w)
    assert not ((ids == 1) | (ids == 4)).any() and torch.isfinite(out.float()).all()
    # fewer experts left than slots: the rest have weight 0 and add nothing
    c.bias[:] = float("-inf")
    c.bias[2] = 0.0
    for m in c.w:
        m[[0, 1, 3, 4, 5]] = float("nan")
    out = c.run(ids, w)
    assert (ids[:, 0] == 2).all() and (w[:, 0] == 1).all() and (w[:, 1] == 0).all()
    assert torch.isfinite(out.float()).all()
    # none left
    c.bias[2] = float("-inf")
    out = c.run(ids, w)
    assert (w == 0).all() and np.array_equal(bits(out), bits(c.res))


def test_equal_logits_take_the_lower_expert():
    c = Case(3, 128, 20, 4, 64, seed=5)
    c.wr[:] = c.wr[0].clone()
    ids = torch.empty(3, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(3, 4, device="cuda")
    c.run(ids, w)
    assert (ids == torch.arange(4, device="cuda")).all() and torch.allclose(w, torch.full_like(w, 0.25), atol=1e-6)


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f32", False), ("bf16", True)])
def test_bad_values_stay_with_their_tokens(dtype, fp8):
    """A NaN in one token's x, or in the weights of an expert that some tokens did not choose."""
    T, E = 7, 5
    ids = np.array([[0, 1], [1, 2], [3, 4], [0, 2], [1, 4], [2, 3], [0, 4]])
    c = Case(T, 192, E, 2, 128, dtype=dtype, fp8=fp8, given=lambda rng: (ids, rng.random((T, 2)) + 0.1), seed=9)
    want = c.run()
    x = c.x.clone()
    c.x[4, 17] = float("nan")
    got = c.run()
    rest = [0, 1, 2, 3, 5, 6]
    assert np.array_equal(bits(got)[rest], bits(want)[rest]) and torch.isnan(got[4].float()).all()
    c.x = x
    for m in range(3):  # gate, up, down of expert 2 (E4M3 0x7f is NaN)
        keep = c.w[m].clone()
        c.w[m][2] = 0x7F if fp8 else float("nan")
        got = c.run()
        without = [t for t in range(T) if 2 not in ids[t]]
        assert np.array_equal(bits(got)[without], bits(want)[without]), m
        assert torch.isnan(got[[1, 3, 5]].float()).any(dim=1).all(), m
        c.w[m].copy_(keep)


def test_nan_in_x_with_a_router():
    c = Case(6, 256, 40, 4, 64, seed=6)
    want = c.run()
    c.x[3, 0] = float("nan")
    ids = torch.full((6, 4), -7, dtype=torch.int32, device="cuda")
    got = c.run(ids, torch.empty(6, 4, device="cuda"))
    rest = [0, 1, 2, 4, 5]
    assert np.array_equal(bits(got)[rest], bits(want)[rest]) and torch.isnan(got[3].float()).all()
    assert ids.min() >= 0 and ids.max() < 40
    # a router row of NaN is an expert nobody takes
    c = Case(6, 256, 40, 4, 64, seed=6)
    c.wr[5] = float("nan")
    c.run(ids)
    assert not (ids == 5).any()


def test_padded_batch_gives_the_same_rows():
    """Tokens that hold anything beside the live ones do not change them (rows are columns of the same products)."""
    c = Case(3, 256, 8, 2, 128, seed=12)
    want = c.run()
    p = Case(3, 256, 8, 2, 128, seed=12)
    pad = 16
    p.T = pad
    p.shape = p.M.Shape(pad, 256, 8, 2, 128)
    p.x = torch.cat([c.x, torch.full((pad - 3, 256), float("inf"), dtype=torch.bfloat16, device="cuda")])
    p.res = torch.cat([c.res, torch.zeros(pad - 3, 256, dtype=torch.bfloat16, device="cuda")])
    p.ws = p.M.workspace(p.M.decode_workspace_size(p.shape))
    got = p.run()
    a, b = host64(got[:3]), host64(want)
    assert np.linalg.norm(a - b) <= 4 * K.U["bf16"] * np.linalg.norm(b)  # two results, each within two half steps


def _shifted(t, by):
    """The same values `by` bytes into an allocation."""
    b = torch.zeros(t.numel() * t.element_size() + by + 64, dtype=torch.uint8, device="cuda")
    v = b[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("layout", [0, 1])
def test_arrays_at_their_least_alignment(dtype, fp8, layout):
    c = Case(5, 320, 6, 2, 192, dtype=dtype, fp8=fp8, layout=layout, bias=True, seed=16)
    ids, w = torch.empty(5, 2, dtype=torch.int32, device="cuda"), torch.empty(5, 2, device="cuda")
    want = c.run(ids, w)
    weights = [_shifted(v, 16) for v in c.stored()]
    c.x, c.norm, c.wr, c.res = (_shifted(v, 16) for v in (c.x, c.norm, c.wr, c.res))
    c.bias = _shifted(c.bias, 4)
    if fp8:
        c.scales = [_shifted(v, 16) for v in c.scales]
    ids2, w2, out = _shifted(ids, 4), _shifted(w, 4), _shifted(torch.zeros_like(want), 16)
    ids2.zero_(), w2.zero_()
    got = c.run(ids2, w2, out, weights=weights)
    assert np.array_equal(bits(got), bits(want)) and torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("layout", [0, 1])
def test_weights_past_2_31_elements(layout):
    """The last two of 40 experts of 58.7 M elements, against a layer of those two."""
    import grouped_gemm_gemv_amd as M
    E, d, F = 40, 4096, 14336
    print(f"\n[gpu] decode E={E} d={d} F={F} layout={layout}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape, std):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    two = [rand(2, F, d, std=d**-0.5), rand(2, F, d, std=d**-0.5), rand(2, d, F, std=F**-0.5)]
    if layout:
        two = [M.moe_pack_blocked16(w) for w in two]
    x, norm, w = rand(1, d, std=1.0), rand(d, std=1.0), torch.tensor([[0.75, -0.5]], device="cuda")
    outs = []
    for n in (2, E):
        shape = M.Shape(1, d, n, 2, F, 0, torch.bfloat16, 0, layout)
        big = two if n == 2 else [torch.empty((E,) + tuple(v.shape[1:]), dtype=v.dtype, device="cuda") for v in two]
        if n == E:
            for b, v in zip(big, two):
                b[-2:] = v
        ids = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device="cuda")
        out = torch.full_like(x, float("nan"))
        M.moe_decode(shape, x, norm, None, None, ids, w, *big, None, out, M.workspace(M.decode_workspace_size(shape)))
        outs.append(out)
    assert torch.isfinite(outs[0].float()).all() and np.array_equal(bits(outs[0]), bits(outs[1]))


@pytest.mark.parametrize("name,over", [("mixtral_decode_t8", dict(d=512, F=640)), ("tiny_f32", dict(T=16)),
                                       ("mixtral_decode_t8_fp8", dict(d=512, F=640))])
def test_agrees_with_the_layers_forward_pass(name, over):
    from tests.gpu_helpers import TOL, dev, rel_err, torch_dtype
    from workloads import get_workload, make_inputs
    import grouped_gemm_gemv_amd as M
    wl = get_workload(name, **over)
    inp = make_inputs(wl, 1)
    dt = torch_dtype(wl.dtype)
    shape = M.Shape(wl.T, wl.d, wl.E, wl.k, wl.F, 0, dt)
    fp8 = wl.weights == "e4m3"
    x, wr = dev(inp.x), dev(inp.wr)
    w = [dev(inp.wg), dev(inp.wu), dev(inp.wd)] + ([dev(inp.sg), dev(inp.su), dev(inp.sd)] if fp8 else [])
    a, b = torch.empty(wl.T, wl.d, dtype=dt, device="cuda"), torch.empty(wl.T, wl.d, dtype=dt, device="cuda")
    v = (M.moe_forward_fp8 if fp8 else M.moe_forward)(shape, x, wr, None, None, None, *w, a,
                                                      M.workspace(M.workspace_size(shape)))
    ids, tw = torch.empty_like(v.topk_ids), torch.empty_like(v.topk_w)
    (M.moe_decode_fp8 if fp8 else M.moe_decode)(shape, x, None, wr, None, ids, tw, *w, None, b,
                                                M.workspace(M.decode_workspace_size(shape)))
    assert torch.equal(ids, v.topk_ids) and (tw - v.topk_w).abs().max() <= 2e-6
    assert rel_err(host64(b), host64(a)) <= 2 * TOL[wl.dtype]


def test_capacity_and_tile_rows_do_not_matter():
    c = Case(16, 128, 4, 2, 64, seed=13)
    want = c.run()
    c.shape = c.M.Shape(16, 128, 4, 2, 64, 3, torch.bfloat16, 64)
    assert np.array_equal(bits(c.run()), bits(want))


def test_out_may_be_res_or_x():
    c = Case(7, 192, 6, 2, 128, seed=14)
    want = c.run()
    x, res = c.x.clone(), c.res.clone()
    assert np.array_equal(bits(c.run(out=c.res)), bits(want))
    c.res = res
    assert np.array_equal(bits(c.run(out=c.x)), bits(want))
    c.x = c.res = x.clone()
    c2 = c.run()
    c.x = c.res = x
    assert np.array_equal(bits(c.run(out=x)), bits(c2))


def test_repeats_streams_and_graph_replays_are_bitwise_equal():
    c = Case(11, 512, 16, 4, 320, layout=1, seed=15)
    weights = c.stored()
    want = c.run(weights=weights)
    for _ in range(3):
        assert np.array_equal(bits(c.run(weights=weights)), bits(want))
    # two calls at once, each with its workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [], [c.M.workspace(c.M.decode_workspace_size(c.shape)) for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    blank = [torch.full_like(want, float("nan")) for _ in range(8)]
    torch.cuda.synchronize()
    for i in range(8):
        outs.append(c.run(weights=weights, stream=streams[i % 2], ws=wss[i % 2], out=blank[i]))
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(bits(o), bits(want))
    ids, tw = torch.empty(11, 4, dtype=torch.int32, device="cuda"), torch.empty(11, 4, device="cuda")
    out = torch.full_like(want, float("nan"))
    c.run(ids, tw, out, weights=weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ids, tw, out, weights=weights)
    for i in range(3):
        c.x.copy_(torch.roll(c.x, 1, 0) * (1.0 + i))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), bits(c.run(weights=weights, ws=wss[0]))), i
        torch.cuda.synchronize()


def test_refusals_on_the_device():
    import grouped_gemm_gemv_amd as M
    c = Case(4, 128, 4, 2, 64)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        M.decode_workspace_size(M.Shape(17, 128, 4, 2, 64))
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        c.run(ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="w_gate must be"):
        M.moe_decode_fp8(c.shape, c.x, None, c.wr, None, None, None, *c.w, *([torch.ones(4, 64, device="cuda")] * 2),
                         torch.ones(4, 128, device="cuda"), None, c.x.clone(), c.ws)
    with pytest.raises(RuntimeError, match="NULL"):
        M.moe_decode(c.shape, c.x, None, None, None, None, None, *c.w, None, c.x.clone(), c.ws)
