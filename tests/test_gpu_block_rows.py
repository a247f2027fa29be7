"""Gradients of the operators around the layer where a workgroup works several rows, one after another: what it keeps from
row to row (column sums, the next row's loads, the places of its sums in LDS), against float64 (oracle/block.py)."""
import numpy as np
import pytest

from tests.gpu_helpers import bits
from tests.test_gpu_block import Case

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
