"""The operators around the layer together with it, as a model uses them: a training step through norm, layer, post-norm,
gate, dropout and residual and back against 64-bit automatic differentiation and against differences; serving steps
through several blocks, eager and replayed; and the layer for a few tokens against the calls it stands for."""
import numpy as np
import pytest

from oracle import block as K
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _block(T, d, E, k, F, dt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*n, std=1.0, mean=0.0):
        return (torch.randn(*n, generator=g, device="cuda") * std + mean).to(dt)

    return dict(x=r(T, d), w_in=r(d, std=0.2, mean=1.0), wr=r(E, d, std=1.5 / d ** 0.5), wg=r(E, F, d, std=1.3 / d ** 0.5),
                wu=r(E, F, d, std=1.3 / d ** 0.5), wd=r(E, d, F, std=1.0 / F ** 0.5), post=r(d, std=0.2, mean=1.0),
                gate=r(T), w_next=r(d, std=0.2, mean=1.0), dout=r(T, d), dn=r(T, d))


def _reference(v, ids, mask, scale):
    """The block in 64 bits with the routing's choice given; loss = <out, dout> + <n, dn>."""
    def norm(a, w):
        return a / torch.sqrt((a * a).mean(1, keepdim=True) + EPS) * w

    m = norm(v["x"], v["w_in"])
    w = torch.softmax(torch.gather(m @ v["wr"].t(), 1, ids), dim=1)
    y = torch.zeros_like(m)
    for e in range(v["wr"].shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a, b = m[t] @ v["wg"][e].t(), m[t] @ v["wu"][e].t()
        y = y.index_add(0, t, w[t, j].unsqueeze(1) * ((a * torch.sigmoid(a) * b) @ v["wd"][e].t()))
    out = v["x"] + scale * torch.sigmoid(v["gate"]).unsqueeze(1) * mask * norm(y, v["post"])
    n = norm(out, v["w_next"])
    return out, n, (out * v["dout"]).sum() + (n * v["dn"]).sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_through_a_block(dtype):
    import grouped_gemm_gemv_amd as M
    T, d, E, k, F, p, scale = 48, 256, 6, 2, 192, 0.25, 0.5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    v = _block(T, d, E, k, F, dt, 3)
    shape, r = M.Shape(T, d, E, k, F, dtype=dt), M.Residual(EPS, scale, p)
    seed, step = 11, 5
    rng = torch.tensor([seed, step], device="cuda")
    new = lambda *n, t=dt: torch.full(n, float("nan"), dtype=t, device="cuda")  # noqa: E731
    disp, saved = M.Dispatch(shape), M.Saved8(shape)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    m, y, out, n = new(T, d), new(T, d), new(T, d), new(T, d)
    M.moe_norm(shape, v["x"], v["w_in"], m, eps=EPS)
    M.moe_forward_save8(shape, m, v["wr"], None, ids, w, v["wg"], v["wu"], v["wd"], y, disp, saved,
                        M.workspace(M.workspace_size(shape)))
    M.moe_residual(shape, r, v["x"], y, v["post"], v["gate"], rng, v["w_next"], out, n)
    dres, dy, dgate, dpost, dnext = new(T, d), new(T, d), new(T), new(d), new(d)
    rws = M.workspace(M.residual_workspace_size(shape))
    M.moe_residual_backward(shape, r, out, y, v["post"], v["gate"], rng, v["w_next"], v["dout"], v["dn"], dres, dy, dgate,
                            dpost, dnext, rws)
    dm, dw, dwr = new(T, d), new(T, k, t=torch.float32), new(E, d)
    dwg, dwu, dwd = new(E, F, d), new(E, F, d), new(E, d, F)
    M.moe_backward(shape, m, v["wr"], ids, w, v["wg"], v["wu"], v["wd"], disp, saved, dy, dm, dw, dwr, None, dwg, dwu, dwd,
                   M.workspace(M.backward_workspace_size(shape)))
    dx, dw_in = new(T, d), new(d)
    M.moe_norm_backward(shape, v["x"], v["w_in"], dm, dres, dx, dw_in, rws, eps=EPS)

    v64 = {name: t.double().requires_grad_(name not in ("dout", "dn")) for name, t in v.items()}
    t = K.threshold(p)
    mask = torch.from_numpy(np.where(K.keep(p, seed, step, T * d), 65536 / (65536 - t), 0.0)).cuda().view(T, d)
    ids64 = ids.long()
    o64, n64, loss = _reference(v64, ids64, mask, scale)
    loss.backward()
    # Forward: m, h, y (and out) rounded once each, and every later value carries those: four half steps, norm-wise
    u = K.U["bf16"] if dtype == "bf16" else 64 * K.U32
    for got, want in ((out, o64), (n, n64)):
        assert (got.double() - want).norm() <= 4 * u * want.norm()
    # Backward: the layer's projections are in 8 bits, each off by at most 2^-7 of its block's largest magnitude, and
    # every gradient has two of them (gate and up) as factors; the roundings between the calls come on top
    tol = 2 * 2.0 ** -7 + 4 * u
    for name, got in (("x", dx), ("w_in", dw_in), ("wr", dwr), ("wg", dwg), ("wu", dwu), ("wd", dwd), ("post", dpost),
                      ("gate", dgate), ("w_next", dnext)):
        want = v64[name].grad
        assert (got.double() - want).norm() <= tol * want.norm(), (name, float((got.double() - want).norm() / want.norm()))
    # and the whole gradient along one direction against the difference of the loss (the choice of experts held)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    with torch.no_grad():
        way = {name: torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) * t.abs().mean()
               for name, t in v64.items() if t.requires_grad}
        grads = dict(x=dx, w_in=dw_in, wr=dwr, wg=dwg, wu=dwu, wd=dwd, post=dpost, gate=dgate, w_next=dnext)
        slope = sum((grads[name].double() * way[name]).sum() for name in way)
        size = sum((grads[name].double() * way[name]).norm() ** 2 for name in way) ** 0.5
        h = 1e-4
        ends = [_reference({name: t + s * h * way[name] if name in way else t for name, t in v64.items()}, ids64, mask,
                           scale)[2] for s in (1, -1)]
        # the errors of the terms of this sum are independent of the direction: tol of its root sum of squares, thrice
        assert (slope - (ends[0] - ends[1]) / (2 * h)).abs() <= 3 * tol * size


def _weights(shape, v, fp8):
    import grouped_gemm_gemv_amd as M
    if not fp8:
        return [M.moe_pack_blocked16(v[n]) if shape.weight_layout else v[n] for n in ("wg", "wu", "wd")]
    codes, scales = [], []
    for n in ("wg", "wu", "wd"):
        s = v[n].float().abs().amax(2) / 448
        c = (v[n].float() / s.unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(M.moe_pack_blocked16(c) if shape.weight_layout else c)
        scales.append(s)
    return codes + scales


@pytest.mark.parametrize("dtype,fp8,layout", [("bf16", False, 1), ("f32", False, 0), ("bf16", True, 1)])
def test_serving_steps_through_blocks(dtype, fp8, layout):
    """Three blocks a step, each a decode call and the norms between them, replayed from a graph for several steps."""
    import grouped_gemm_gemv_amd as M
    T, d, E, k, F, blocks = 5, 512, 12, 3, 320, 3
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape, r = M.Shape(T, d, E, k, F, 0, dt, 0, layout), M.Residual(EPS, 0.5)
    vs = [_block(T, d, E, k, F, dt, 20 + b) for b in range(blocks)]
    ws = [_weights(shape, v, fp8) for v in vs]
    work = M.workspace(M.decode_workspace_size(shape))
    fn = M.moe_decode_fp8 if fp8 else M.moe_decode
    x = vs[0]["x"].clone()
    y, out = torch.empty_like(x), torch.empty_like(x)
    n = [torch.empty_like(x) for _ in range(2)]

    def step():
        M.moe_norm(shape, x, vs[0]["w_in"], n[0], eps=EPS)
        out.copy_(x)
        for b in range(blocks):
            v, nxt = vs[b], vs[(b + 1) % blocks]["w_in"]
            fn(shape, n[b % 2], None, v["wr"], None, None, None, *ws[b], None, y, work)
            M.moe_residual(shape, r, out, y, v["post"], v["gate"], None, nxt, out, n[(b + 1) % 2])

    step()
    first = out.clone()
    for _ in range(2):
        step()
        assert np.array_equal(bits(out), bits(first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(vs[1]["x"] * (i + 1))
        step()
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), bits(want)), i


@pytest.mark.parametrize("T", [1, 8, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_is_norm_layer_and_residual(T, dtype):
    import grouped_gemm_gemv_amd as M
    d, E, k, F = 256, 10, 3, 192
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    v = _block(T, d, E, k, F, dt, 40 + T)
    shape = M.Shape(T, d, E, k, F, dtype=dt)
    m, y, a, b = (torch.empty_like(v["x"]) for _ in range(4))
    M.moe_norm(shape, v["x"], v["w_in"], m, eps=EPS)
    views = M.moe_forward(shape, m, v["wr"], None, None, None, v["wg"], v["wu"], v["wd"], y,
                          M.workspace(M.workspace_size(shape)))
    M.moe_residual(shape, M.Residual(EPS, 0.5), v["x"], y, None, None, None, None, a, None)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    M.moe_decode(shape, v["x"], v["w_in"], v["wr"], None, ids, torch.empty(T, k, device="cuda"), v["wg"], v["wu"], v["wd"],
                 v["x"], b, M.workspace(M.decode_workspace_size(shape)), eps=EPS, scale=0.5)
    same = (ids == views.topk_ids).all(dim=1)  # the layer's router sees m rounded: a near tie may fall elsewhere
    assert same.float().mean() >= 0.75
    a, b = a[same].double(), b[same].double()
    u = K.U["bf16"] if dtype == "bf16" else 64 * K.U32
    # one side rounds m, h, y and out, the other m, h and out
    assert (a - b).norm() <= 7 * u * a.norm()


# Shapes whose units are dealt on the device: the router is a kernel of its own, and the workgroups have eight turns and
# more, active experts x F / (8 x 256 x groups), with one group of wavefronts (rows of 64 KB / 8 and more) to eight
@pytest.mark.parametrize("T,d,E,k,F,dtype,fp8,layout", [
    (3, 4096, 64, 8, 1024, "bf16", False, 1), (16, 4096, 8, 2, 2112, "bf16", False, 0),  # one group
    (16, 2048, 8, 2, 4096, "bf16", False, 1), (8, 1024, 32, 4, 2048, "f32", False, 0),   # two
    (16, 4096, 8, 2, 4096, "bf16", True, 1),                                             # two, with scales
    (16, 1024, 16, 4, 4096, "bf16", False, 1), (16, 2048, 8, 2, 8192, "bf16", True, 0),  # four
    (16, 1024, 16, 4, 8192, "bf16", True, 1),                                            # eight
])
def test_dealt_units_give_the_same_bits(T, d, E, k, F, dtype, fp8, layout):
    """The same routing, computed (dealt in the order workgroups come) and given (dealt evenly): who works a unit must
    not show, so both are equal to the bit, in every repeat.  And right, token by token, against 64 bits."""
    import grouped_gemm_gemv_amd as M
    print(f"\n[gpu] dealt T={T} d={d} E={E} k={k} F={F} {dtype} fp8={fp8} layout={layout}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = M.Shape(T, d, E, k, F, 0, dt, 0, layout)
    v = _block(T, d, E, k, F, dt, T + d)
    w = _weights(shape, v, fp8)
    fn = M.moe_decode_fp8 if fp8 else M.moe_decode
    ws = M.workspace(M.decode_workspace_size(shape))
    ws.fill_(0xFF)
    ids, tw = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    first = torch.full_like(v["x"], float("nan"))
    fn(shape, v["x"], v["w_in"], v["wr"], None, ids, tw, *w, v["x"], first, ws, eps=EPS)
    for i in range(4):
        out = torch.full_like(first, float("nan"))
        if i == 0:
            fn(shape, v["x"], v["w_in"], None, None, ids, tw, *w, v["x"], out, ws, eps=EPS)
        else:
            fn(shape, v["x"], v["w_in"], v["wr"], None, None, None, *w, v["x"], out, ws, eps=EPS)
        assert np.array_equal(bits(out), bits(first)), i
    x = v["x"].double()
    m = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * v["w_in"].double()
    y = torch.zeros_like(x)
    plain = [v[n] for n in ("wg", "wu", "wd")]
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        g, u, dn = (p[e].double() for p in plain)
        if fp8:
            g, u, dn = ((p[e].float() / s[e].unsqueeze(1)).to(torch.float8_e4m3fn).double() * s[e].double().unsqueeze(1)
                        for p, s in zip((q.float() for q in plain), w[3:]))
        a = m[t] @ g.t()
        y.index_add_(0, t, tw[t, j].double().unsqueeze(1) * ((a * torch.sigmoid(a) * (m[t] @ u.t())) @ dn.t()))
    err = (first.double() - (x + y)).norm(dim=1)
    half = K.U["bf16"] if dtype == "bf16" else 64 * K.U32
    assert (err <= 3 * half * y.norm(dim=1) + half * (x + y).norm(dim=1)).all(), err.max()


def test_captured_graphs_may_share_a_workspace():
    """Replays in turn on one stream, with eager calls on the same workspaces between them: none leaves anything that
    the next one needs or minds."""
    import grouped_gemm_gemv_amd as M
    bf = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(9)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(bf)

    shapes = [M.Shape(T, 256, E, 2, 192, 0, bf) for T, E in ((3, 4), (14, 20))]
    ws = M.workspace(max(M.decode_workspace_size(s) for s in shapes))
    gws = M.workspace(max(M.residual_workspace_size(s) for s in shapes))
    runs = []
    for s in shapes:
        T, d, E, F = s.T, s.d, s.E, s.F
        x, norm, wr = rand(T, d), rand(d), rand(E, d, std=0.1)
        w = [rand(E, F, d, std=d**-0.5), rand(E, F, d, std=d**-0.5), rand(E, d, F, std=F**-0.5)]
        out, dn, dx, dw = torch.empty_like(x), rand(T, d), torch.empty_like(x), torch.empty_like(norm)

        def call(s=s, x=x, norm=norm, wr=wr, w=w, out=out, dn=dn, dx=dx, dw=dw):
            M.moe_decode(s, x, norm, wr, None, None, None, *w, x, out, ws)
            M.moe_norm_backward(s, out, norm, dn, None, dx, dw, gws)

        call()
        torch.cuda.synchronize()
        want = [v.clone() for v in (out, dx, dw)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, call, (out, dx, dw), want))
    for i in (0, 1, 0, 0, 1, 1, 0):
        graph, call, got, want = runs[i]
        for v in got:
            v.fill_(float("nan"))
        graph.replay()
        runs[1 - i][1]()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
