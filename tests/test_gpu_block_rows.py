"""The operators around the layer where a workgroup works several rows, one after another: what it keeps from row to row
(column sums, the next row's loads, the places of its sums in LDS), against float64 (oracle/block.py)."""
import numpy as np
import pytest

from oracle import block as K
from tests.gpu_helpers import bits, host64
from tests.test_gpu_block import EPS, Case, close

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def workgroups(T, d, dtype=None):
    """Workgroups of the gradient: its workspace is their two rows of partial sums, up to the next 256 bytes."""
    import grouped_gemm_gemv_amd as M
    return M.residual_workspace_size(M.Shape(T, d, 1, 1, 64, dtype=dtype or torch.bfloat16)) // (8 * d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("T,d", [(1500, 1088), (600, 4096)])
def test_a_gate_a_token_without_norms(T, d, p, dtype):
    """One sum over a row and so one barrier: no wavefront may leave its part of a row's sum where another still reads
    the row before it.  A sum of two rows' parts is another gate's gradient, and another one on each call."""
    print(f"\n[gpu] residual gradient T={T} d={d} p={p} gate alone {dtype}", flush=True)
    assert T > workgroups(T, d)
    c = Case(T, d, dtype, post=False, gate="token", p=p, nxt=False, scale=0.5, seed=T)
    c.check()
    out, _ = c.forward()
    first = c.backward(out)
    for _ in range(4):
        again = c.backward(out)
        for name in first:
            assert np.array_equal(bits(first[name]), bits(again[name])), name


# one width or two for each number of threads of a row, 64 to 1024, and one past the next row's loads (16 elements of a thread)
WIDTHS = [64, 448, 640, 2048, 4096, 8192, 16384]


def many_rows(d):
    """Three rows for some workgroups and two for the others (forward and gradient launch equally many).  A workgroup of
    four wavefronts takes four rows of up to 512 elements at a time."""
    side = 4 if d <= 512 else 1
    most = workgroups(1 << 20, d)
    T = 2 * most * side + 3
    assert workgroups(T, d) == most and T > 2 * most * side
    return T


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("post,gate,nxt", [(True, "token", True), (False, "full", True), (True, None, False)])
def test_several_rows_of_a_workgroup(post, gate, nxt, d, dtype):
    T = many_rows(d)
    print(f"\n[gpu] residual T={T} d={d} post={post} gate={gate} next={nxt} {dtype}", flush=True)
    Case(T, d, dtype, post, gate, 0.0, nxt, scale=0.5, seed=d).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_several_rows_of_a_norm(d, dtype):
    import grouped_gemm_gemv_amd as M
    T = many_rows(d)
    print(f"\n[gpu] norm T={T} d={d} {dtype}", flush=True)
    c = Case(T, d, dtype, seed=d + 1)
    x, w = host64(c.res), host64(c.next)
    n, dx, dw = torch.empty_like(c.res), torch.empty_like(c.res), torch.empty_like(c.next)
    M.moe_norm(c.shape, c.res, c.next, n, eps=EPS)
    close("n", n, K.norm(x, w, EPS, dtype))
    M.moe_norm_backward(c.shape, c.res, c.next, c.dn, None, dx, dw, M.workspace(M.residual_workspace_size(c.shape)), eps=EPS)
    want = K.residual_backward(x, None, None, None, None, w, None, host64(c.dn), EPS, 1.0, dtype)
    close("dx", dx, want["dres"])
    close("dw", dw, want["dnext"])


@pytest.mark.parametrize("d", [640, 4096])
def test_several_rows_with_dropout(d):
    """The mask's numbers go on from row to row: a gradient of one pass has the forward pass's mask."""
    T = workgroups(1 << 20, d) + 5
    print(f"\n[gpu] residual T={T} d={d} dropout", flush=True)
    Case(T, d, "bf16", gate="token", p=0.1, scale=0.5, seed=d).check()
