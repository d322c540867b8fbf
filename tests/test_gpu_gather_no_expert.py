"""Rows gathered by the copy engine for pairs that name no expert (the permutation leaves their places unwritten)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_ffn_07_b200 as moe  # noqa: E402
from tests import _gpu  # noqa: E402
from tests.test_gpu_experts_formats import _experts  # noqa: E402
from tests.test_gpu_parity import make, spec  # noqa: E402


@pytest.mark.parametrize("T", [20, 300])
def test_gathered_rows_and_pairs_of_no_expert(T):
    """Rows gathered by the copy engine: the unwritten end of the pairs' order is read inside x, whatever it holds."""
    s = spec(T, 256, 8, 96, 2, dt="bf16", w_dt="bf16", r_dt="bf16")
    wl = make(s, seed=83)
    desc, w, x = _gpu.upload(wl)
    _, gids, gw, _ = _gpu.run_route(desc, w, x)
    ids, tw = gids.view(s.T, s.K).contiguous(), gw.view(s.T, s.K).contiguous()
    bad = ids.clone()
    bad[::3] = -1
    want = _experts(desc, x, w, bad, tw, None)
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    moe.set_tma_gather(True)
    try:
        got = _experts(desc, x, w, bad, tw, None)
    finally:
        moe.set_tma_gather(False)
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    assert torch.equal(got, want) and torch.all(got[::3] == 0)
