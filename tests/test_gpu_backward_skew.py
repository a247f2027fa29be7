"""The experts' gradients under skewed routing: right where one expert holds most
rows and workgroups take several tiles in turn, and no slower than with the
rows spread evenly by more than the hot expert's own tiles explain."""
import numpy as np
import pytest

from oracle import backward as B
from tests.gpu_helpers import bits, host64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _zipf(c, share, seed=0):
    """Routes `share` of the tokens to expert 1, the rest evenly, and redoes the dispatch."""
    rng = np.random.default_rng(seed)
    ids = c.ids_np
    hot = rng.random(c.T) < share
    ids[hot, 0] = 1
    c.ids.copy_(torch.from_numpy(ids))
    c.M.moe_permute(c.shape, c.x, c.ids, c.disp, c.empty(c.R, c.d),
                    c.M.workspace(c.M.query(c.shape).permute_ws_bytes))
    arr = c.disp.arrays()
    c.row_of, c.token_of = arr["row_of"].cpu().numpy(), arr["token_of"].cpu().numpy()
    c.entry_of, c.expert_of = np.full(c.R, -1), np.full(c.R, -1)
    for f, r in enumerate(c.row_of):
        if r >= 0:
            c.entry_of[r], c.expert_of[r] = f, ids.reshape(-1)[f]
    c.live = c.token_of >= 0


@pytest.mark.parametrize("kw", [
    dict(T=700, d=64, E=8, k=1, F=6144), dict(T=600, d=192, E=24, k=1, F=1536, cap=20, layout=1),
    dict(T=500, d=64, E=8, k=1, F=4096, dtype="f32"),
], ids=str)
def test_gradients_with_a_hot_expert(kw):
    _need_gpu()
    from tests.test_gpu_backward import Case, _ffn, close
    print(f"\n[gpu] hot expert {kw}", flush=True)
    c = Case(**kw)
    _zipf(c, 0.85)
    saved, g, u = c.saved()
    o = _ffn(c, saved)
    want = B.ffn_backward(host64(c.x), host64(c.dout), host64(c.w), host64(c.wg), host64(c.wu), host64(c.wd), g, u,
                          c.token_of, c.entry_of, c.expert_of, c.dtype)
    close("dx_perm", host64(o["dx_perm"])[c.live], want["dx_perm"][0][c.live], want["dx_perm"][1][c.live])
    close("dw", host64(o["dw"]).reshape(-1), *want["dw"])
    for n in ("dwg", "dwu", "dwd"):
        close(n, c.unweight(o[n]), *want[n])
    again = _ffn(c, saved)
    for n in o:
        assert np.array_equal(bits(o[n]), bits(again[n])), n


def test_weight_gradients_do_not_wait_for_the_hot_experts_workgroups():
    """The products' work is the same however the rows are spread (one expert with three quarters of 2048 rows against
    an even spread, fp32, where the products are all there is): dealt evenly they take the same time, and 5 times as
    long if an eighth of the GPU has the hot expert to itself.  Time of the call with less that without weight
    gradients, least of several."""
    _need_gpu()
    from tests.test_gpu_backward import Case
    print("\n[gpu] weight gradients, time with a hot expert", flush=True)
    c = Case(T=2048, d=1024, E=8, k=1, F=2048, dtype="f32")
    saved = c.M.Saved8(c.shape)
    for a in saved.arrays().values():
        a.fill_(100)
    ws = c.M.workspace(c.M.backward_query(c.shape).ffn_ws_bytes)
    dx, dw = c.empty(c.R, c.d), c.empty(c.T, c.k, dt=torch.float32)
    grads = [torch.empty_like(t) for t in (c.wg, c.wu, c.wd)]

    def least(g):
        t = []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            c.M.moe_grouped_ffn_backward(c.shape, c.x, c.dout, c.w, c.wg, c.wu, c.wd, c.disp, saved, dx, dw, *g, ws)
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b))
        return min(t[2:])

    took = []
    for share in (0.0, 0.75):
        _zipf(c, share)
        took.append(least(grads) - least([None] * 3))
    assert took[1] < 2.0 * took[0], took
