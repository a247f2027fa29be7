"""The layer for a few tokens keeps x norm_w and h in two bf16 terms each, behind a routing of its own too: the router's
products and the experts' see both of them, wherever they are made."""
import numpy as np
import pytest

from oracle import block as K
from tests.gpu_helpers import host64
from tests.test_gpu_decode import EPS, Case, _t

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _run(c):
    ids = torch.full((c.T, c.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((c.T, c.k), float("nan"), device="cuda")
    return c.run(ids, w), ids.cpu().numpy(), host64(w)


# T, d, E, F: routed in the first kernel by one tile of experts and by several, with second terms in the instruction's idle
# columns and in instructions of their own; apart; four experts of a lane; x as it is in LDS, routed in the kernel and apart
ROUTERS = [(1, 512, 6, 192), (8, 1024, 8, 128), (13, 512, 8, 128), (3, 448, 40, 64), (12, 256, 100, 64), (4, 2048, 64, 128),
           (16, 4096, 3, 128), (16, 4096, 70, 64), (8, 6144, 4, 64)]


@pytest.mark.parametrize("fp8,layout", [(False, 0), (False, 1), (True, 0), (True, 1)])
@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_bf16_is_rounded_once_behind_a_router(T, d, E, F, fp8, layout):
    """Against float64 with the routing that the call gave: the bound with both terms, and over all of the output its one
    rounding, even over a step of at most 2^-7 |v|: a root mean square of 2^-7 |v| / sqrt(12) at the most (0.0023).
    One term of both comes to 0.0029."""
    print(f"\n[gpu] decode rounded once behind a router T={T} d={d} E={E} F={F} fp8={fp8} layout={layout}", flush=True)
    c = Case(T, d, E, 2, F, fp8=fp8, layout=layout, res=False, seed=T + E)
    got, ids, w = _run(c)
    want, bound = K.decode(host64(c.x), host64(c.norm), EPS, ids, w, *c.w64, None, 1.0, "bf16", terms=2)
    err = np.abs(host64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())
    assert np.linalg.norm(err) <= 2.0**-7 / 12**0.5 * np.linalg.norm(want), np.linalg.norm(err) / np.linalg.norm(want)


@pytest.mark.parametrize("T,d,E,F", ROUTERS)
def test_the_router_sees_both_terms(T, d, E, F):
    """x norm_w has 13 bits, a router row is plus and minus one power of two, and every sum is below 2^24 of its last bit:
    products and sums are exact, so a logit is off by what 1 / rms is, S of itself, and two logits that are equal stay
    so.  A first term alone would move a logit by about 2^-9 of itself."""
    print(f"\n[gpu] decode router terms T={T} d={d} E={E} F={F}", flush=True)
    k = min(E, 6)
    c = Case(T, d, E, k, F, seed=T + E + 1)
    rng = np.random.default_rng(T + d + E)
    x = rng.integers(-15, 16, (T, d)).astype(np.float64)
    norm = 1 + rng.integers(0, 128, d) / 128
    assert (np.abs(x * norm).sum(axis=1) * 128 < 2**24).all()
    row = 2.0 ** -np.round(np.log2(np.sqrt(d)) + 1)  # (logits of about a half)
    wr = rng.choice([-row, row], (E, d))
    c.x, c.norm, c.wr = (_t(v, torch.bfloat16) for v in (x, norm, wr))
    assert np.array_equal(host64(c.x), x) and np.array_equal(host64(c.norm), norm) and np.array_equal(host64(c.wr), wr)
    _, ids, w = _run(c)
    z = (x * norm) @ wr.T * K.rms(x, EPS)
    order = np.argsort(-((x * norm) @ wr.T), axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids, order)
    sel = np.take_along_axis(z, order, axis=1)
    p = np.exp(sel - sel.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    # each exponential's argument is off by two logits' errors, and a quotient of them by twice that; 16 roundings around it
    e_w = 4 * K.S * np.abs(sel).max() + 16 * K.U32
    assert (np.abs(w - p) <= e_w * p).all(), float((np.abs(w - p) / p).max() / e_w)
