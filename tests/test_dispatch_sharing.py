"""A dispatch carved for one layer and used with another of the same routing.  Its
one array that depends on the layer's widths holds the down GEMM's partial
sums, [2][R][d] of the carved shape: calls that write them there refuse planes
that are too small, and moe_forward_save8 keeps them in its own workspace."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")


def _shapes(**kw):
    import grouped_gemm_gemv_amd as M
    # 128 rows per expert: the down GEMM on 160-row tiles splits K
    return [M.Shape(512, d, 8, 2, 256, tile_rows=160, **kw) for d in (64, 512)]


def test_partial_sums_of_a_narrower_dispatch_are_too_small():
    """The sizes behind the refusal: the narrow layer's whole dispatch is smaller than the wide one's planes."""
    import grouped_gemm_gemv_amd as M
    narrow, wide = _shapes()
    assert M.query(narrow).dispatch_bytes < 2 * M.query(wide).rows * wide.d * 4
    assert M.workspace_size(wide) >= M.query(wide).dispatch_bytes + M.query(wide).rows * (wide.d + wide.F) * 2


@pytest.mark.parametrize("call", ["moe_ffn_down", "moe_grouped_ffn", "moe_ffn_down_fp8"])
def test_down_calls_refuse_a_dispatch_with_too_few_partial_sums(call):
    import grouped_gemm_gemv_amd as M
    narrow, wide = _shapes()
    x = torch.zeros(1)
    n = {"moe_ffn_down": 2, "moe_grouped_ffn": 4, "moe_ffn_down_fp8": 3}[call]  # tensors in front of disp
    tail = (x, x) if call == "moe_grouped_ffn" else (0, x)

    def run(disp, shape):
        getattr(M, call)(shape, *[x] * n, disp, *tail)

    with pytest.raises(ValueError, match="partial sums"):
        run(M.Dispatch(narrow, device="cpu"), wide)
    # wide enough, or a call that does not split K: on to the next check, here that the tensors are on the host
    for disp, shape in ((wide, wide), (wide, narrow), (narrow, M.Shape(512, 512, 8, 2, 256, dtype=torch.float32))):
        with pytest.raises(ValueError, match="device tensors"):
            run(M.Dispatch(disp, device="cpu"), shape)


def test_only_the_down_calls_ask_for_planes_of_partial_sums():
    """A dispatch carved without planes (F = 64 does not split K) for a layer of the same routing that splits: the down
    GEMM calls refuse it (a pointer is missing, 2), the calls that do not use the planes go on to their next check, here
    a workspace or a pointer that is not aligned (1).  No address is used."""
    import grouped_gemm_gemv_amd as M
    from grouped_gemm_gemv_amd._lib import MoeSaved8, lib
    _, wide = _shapes()
    disp = M.Dispatch(M.Shape(512, 512, 8, 2, 64, tile_rows=160), device="cpu")
    assert not disp.c.kpart and M.Dispatch(wide, device="cpu").c.kpart
    S, D, V = ctypes.byref(wide.c()), ctypes.byref(disp.c), ctypes.byref(MoeSaved8(*[1 << 20] * 4))
    A, big = 1 << 20, 1 << 50
    assert lib().moe_ffn_down(S, A, A, D, 0, A, None) == 2
    assert lib().moe_ffn_down_fp8(S, A, A, A, D, 0, A, None) == 2
    assert lib().moe_grouped_ffn(S, A, A, A, A, D, A, A, None) == 2
    assert lib().moe_ffn_gate_up_save8(S, A + 8, A, A, D, 0, A, V, None) == 1
    assert lib().moe_forward_save8(S, A, A, A, A, A, A, A, A, A, D, V, A + 8, big, None) == 1
    assert lib().moe_grouped_ffn_backward(S, *[A] * 6, D, V, *[A] * 5, A + 8, big, None) == 1
    assert lib().moe_backward(S, *[A] * 7, D, V, *[A] * 8, A + 8, big, None) == 1


@pytest.mark.gpu
def test_forward_save8_leaves_a_shared_dispatchs_partial_sums_alone():
    """Two layers of different width share a dispatch: nothing behind its other arrays is written, out is bitwise
    moe_forward's, and the gradients are those of a dispatch of the layer's own."""
    import grouped_gemm_gemv_amd as M
    from grouped_gemm_gemv_amd._lib import MoeDispatch, check, lib
    from tests.gpu_helpers import bits
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("\n[gpu] shared dispatch", flush=True)
    narrow, wide = _shapes()
    s = wide
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*n):
        return (torch.randn(*n, generator=gen, device="cuda") / n[-1] ** 0.5).bfloat16()

    x, dout, wr = rnd(s.T, s.d) * s.d ** 0.5, rnd(s.T, s.d), rnd(s.E, s.d)
    wg, wu, wd = rnd(s.E, s.F, s.d), rnd(s.E, s.F, s.d), rnd(s.E, s.d, s.F)
    ws = M.workspace(max(M.workspace_size(s), M.backward_workspace_size(s)))
    # the narrow layer's dispatch at the head of a buffer that also holds everything the wide one could write
    n = M.query(narrow).dispatch_bytes
    buf = torch.full((n + 2 * M.query(s).rows * s.d * 4 + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    c = MoeDispatch()
    base = (buf.data_ptr() + 255) // 256 * 256
    check("moe_dispatch_carve", lib().moe_dispatch_carve(ctypes.byref(narrow.c()), base, n, ctypes.byref(c)))
    assert c.kpart
    shared = M.Dispatch(narrow, c=c, owner=buf)
    res = []
    none = M.Dispatch(M.Shape(s.T, s.d, s.E, s.k, 64, tile_rows=160))  # carved without planes
    assert not none.c.kpart
    for disp in (shared, M.Dispatch(s), none):
        ids = torch.empty(s.T, s.k, dtype=torch.int32, device="cuda")
        w, dw = (torch.empty(s.T, s.k, device="cuda") for _ in range(2))
        out, dx = torch.empty_like(x), torch.empty_like(x)
        g = [torch.empty_like(t) for t in (wr, wg, wu, wd)]
        saved = M.Saved8(s)
        M.moe_forward_save8(s, x, wr, None, ids, w, wg, wu, wd, out, disp, saved, ws)
        M.moe_backward(s, x, wr, ids, w, wg, wu, wd, disp, saved, dout, dx, dw, g[0], None, *g[1:], ws)
        res.append([bits(t) for t in (ids, w, out, dx, dw, *g)])
    torch.cuda.synchronize()
    assert (buf[c.kpart - buf.data_ptr():] == 0x5A).all()
    for other in res[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(res[0], other))
    ref = torch.empty_like(x)
    M.moe_forward(s, x, wr, None, None, None, wg, wu, wd, ref, ws)
    assert np.array_equal(bits(ref), res[0][2])


@pytest.mark.gpu
def test_forward_save8_on_a_taller_dispatch_than_the_shapes_own():
    """The dispatch's 160-row tiles would split K, this shape's own 64-row ones do not, so the workspace has no place
    for partial sums: the down GEMM runs unsplit, and the dispatch's planes stay as they are."""
    import grouped_gemm_gemv_amd as M
    from tests.gpu_helpers import TOL, host64, rel_err
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("\n[gpu] taller dispatch", flush=True)
    s, tall = M.Shape(512, 64, 8, 2, 256), M.Shape(512, 64, 8, 2, 256, tile_rows=160)
    assert M.query(s).tile_rows != 160
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*n):
        return (torch.randn(*n, generator=gen, device="cuda") / n[-1] ** 0.5).bfloat16()

    x, wr = rnd(s.T, s.d) * 8, rnd(s.E, s.d)
    wg, wu, wd = rnd(s.E, s.F, s.d), rnd(s.E, s.F, s.d), rnd(s.E, s.d, s.F)
    disp, saved, ws = M.Dispatch(tall), M.Saved8(s), M.workspace(M.workspace_size(s))
    disp.buf.fill_(0x5A)
    ids, w = torch.empty(s.T, s.k, dtype=torch.int32, device="cuda"), torch.empty(s.T, s.k, device="cuda")
    out, ref = torch.full_like(x, float("nan")), torch.empty_like(x)
    M.moe_forward_save8(s, x, wr, None, ids, w, wg, wu, wd, out, disp, saved, ws)
    M.moe_forward(s, x, wr, None, None, None, wg, wu, wd, ref, ws)
    torch.cuda.synchronize()
    assert disp.c.kpart and (disp.buf[disp.c.kpart - disp.buf.data_ptr():] == 0x5A).all()
    assert rel_err(host64(out), host64(ref)) <= TOL["bf16"]
