"""What the layer for a few tokens does with logits that are no numbers and with masked experts, wherever it routes: in its
first kernel or in one of its own, with x norm_w in LDS once, twice or as it is, one expert of a lane or four."""
import numpy as np
import pytest

from tests.gpu_helpers import bits
from tests.test_gpu_decode import Case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")
# T, d, E, F: routed in the first kernel by one tile of experts and by several, apart, four experts of a lane, x as it is in LDS
ROUTERS = [(5, 128, 8, 64), (3, 256, 40, 64), (4, 2048, 64, 64), (2, 128, 100, 64), (16, 4096, 6, 64), (16, 4096, 70, 64)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _routing(c):
    ids = torch.full((c.T, c.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((c.T, c.k), -7.0, device="cuda")
    out = c.run(ids, w)
    return out, ids.cpu().numpy(), w.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_a_nan_ranks_below_a_masked_expert(T, d, E, F, dtype):
    """Four slots and two experts with a number for a logit: masked ones, which have no weight, take the other slots, and
    none goes to the expert with a NaN, although its index is the lowest."""
    if dtype == "f32" and T * d * 4 > 131072:
        T = 131072 // 4 // d
    print(f"\n[gpu] decode NaN and masked T={T} d={d} E={E} {dtype}", flush=True)
    c = Case(T, d, E, 4, F, dtype=dtype, bias=True, seed=E)
    c.bias[:] = -INF
    c.bias[[0, 2, E - 1]] = 0.25
    c.wr[0] = NAN
    out, ids, w = _routing(c)
    assert np.array_equal(np.sort(ids[:, :2], axis=1), np.tile([2, E - 1], (T, 1)))
    assert (ids[:, 2:] == [1, 3]).all() and (w[:, 2:] == 0).all()
    assert np.isfinite(w).all() and torch.isfinite(out.float()).all()
    c.wr[0], c.bias[0] = 0.0, -INF  # that expert masked too: the same layer
    assert np.array_equal(bits(out), bits(c.run()))


@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_a_nan_has_the_slots_that_are_left(T, d, E, F):
    """Three experts with a number, six slots: these come first, then the experts without one, lowest first; a token that has
    such an expert has weights, and a row of out, that are no numbers."""
    print(f"\n[gpu] decode slots for NaN T={T} d={d} E={E}", flush=True)
    c = Case(T, d, E, 6, F, seed=E)
    live = [1, 3, E - 1]
    dead = [e for e in range(E) if e not in live]
    c.wr[dead] = NAN
    out, ids, w = _routing(c)
    assert np.array_equal(np.sort(ids[:, :3], axis=1), np.tile(live, (T, 1)))
    assert (ids[:, 3:] == dead[:3]).all()
    assert np.isnan(w).all() and torch.isnan(out.float()).all()
    c.wr[:] = NAN
    out, ids, w = _routing(c)
    assert (ids == np.arange(6)).all() and np.isnan(w).all() and torch.isnan(out.float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_a_masked_experts_router_row_may_hold_anything(T, d, E, F, dtype):
    """A bias of -inf masks an expert whatever its logit would have been: NaN and +inf plus -inf are NaN, and with fewer
    experts left than slots that would be chosen."""
    if dtype == "f32" and T * d * 4 > 131072:
        T = 131072 // 4 // d
    print(f"\n[gpu] decode masked rows T={T} d={d} E={E} {dtype}", flush=True)
    c = Case(T, d, E, 3, F, dtype=dtype, bias=True, seed=E)
    masked = [e for e in range(E) if e not in (2, E - 1)]
    c.bias[masked] = -INF
    want, wids, ww = _routing(c)
    assert (ww[:, 2] == 0).all() and (wids[:, 2] == 0).all() and torch.isfinite(want.float()).all()
    for bad in (NAN, INF, -INF):
        c.wr[masked] = bad
        out, ids, w = _routing(c)
        assert np.array_equal(ids, wids) and np.array_equal(w, ww), bad
        assert np.array_equal(bits(out), bits(want)), bad
    c.wr[masked[0]] = c.wr[2]
    c.wr[masked[0], 0], c.x[:, 0] = INF, 1.0  # a logit of +inf
    c.bias[:] = -INF
    out, ids, w = _routing(c)
    assert (w == 0).all() and np.array_equal(bits(out), bits(c.res))


@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_a_nan_in_x_shows_beside_masked_experts(T, d, E, F):
    """The experts that are not masked have a NaN for that token: masked ones fill its slots, but its row is a NaN."""
    print(f"\n[gpu] decode NaN in x and masked T={T} d={d} E={E}", flush=True)
    c = Case(T, d, E, 2, F, bias=True, seed=E)
    c.bias[:] = -INF
    c.bias[[1, E - 1]] = 0.5
    want = c.run()
    c.x[T - 1, 7] = NAN
    out, ids, w = _routing(c)
    assert torch.isnan(out[T - 1].float()).all() and np.isnan(w[T - 1]).all()
    assert ids.min() >= 0 and ids.max() < E
    assert np.array_equal(bits(out)[:T - 1], bits(want)[:T - 1]) and torch.isfinite(want.float()).all()
