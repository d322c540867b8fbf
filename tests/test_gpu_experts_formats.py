"""moe_experts on the weight formats besides 8-bit floats: its output is moe_layer's on the layer's own routing, with a shared
expert and without, and pairs of no expert count nothing."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_ffn_07_b200 as moe  # noqa: E402
import oracle  # noqa: E402
import workloads  # noqa: E402
from tests import _gpu  # noqa: E402
from tests.test_gpu_kquant import kspec  # noqa: E402
from tests.test_gpu_parity import make, spec  # noqa: E402

CASES = {  # one token, a decode batch, a batch past the fused decode kernel; a shared expert, gated and not
    "q8_0_T1": spec(1, 512, 16, 256, 4, dt="f32", w_dt="q8_0", r_dt="f32"),
    "q8_0_T16_shared_gated": spec(16, 256, 16, 128, 4, dt="f32", w_dt="q8_0", r_dt="f32", shared=96, gated=True),
    "q8_0_T90_shared": spec(90, 256, 16, 128, 4, dt="bf16", w_dt="q8_0", r_dt="bf16", shared=64),
    "q4_k_T1": kspec(1, 512, 8, 256, 2, w_dt="q4_k"),
    "q4_k_T12_shared_gated": kspec(12, 512, 16, 256, 4, w_dt="q4_k", shared=256, gated=True),
    "q4_k_T80": kspec(80, 512, 16, 256, 4, w_dt="q4_k", dt="bf16"),
    "q4_k_q6_k_T1_shared": kspec(1, 768, 8, 256, 2, shared=256),
    "q4_k_q6_k_T9_shared_gated": kspec(9, 768, 16, 256, 2, shared=512, gated=True),
    "q4_k_q6_k_T80": kspec(80, 512, 16, 256, 4, act="gelu_tanh"),
    "f32_T7_shared_gated": spec(7, 256, 8, 96, 2, dt="f32", w_dt="f32", r_dt="f32", shared=64, gated=True),
    "f32_T100_shared": spec(100, 256, 8, 96, 2, dt="f32", w_dt="f32", r_dt="f32", shared=64),
    "bf16_T5_shared_gated": spec(5, 256, 8, 96, 2, dt="bf16", w_dt="bf16", r_dt="bf16", shared=64, gated=True),
    "bf16_T200_shared_gated": spec(200, 256, 8, 96, 2, dt="bf16", w_dt="bf16", r_dt="bf16", shared=96, gated=True),
}


def _experts(desc, x, w, ids, tw, sg):
    out = torch.full((desc.T, desc.H), float("nan"), dtype=x.dtype, device="cuda")
    ws = torch.full((moe.workspace_bytes(desc),), 0x7F, dtype=torch.uint8, device="cuda")
    moe.experts(desc, x, w, ids, tw, out, ws, shared_gate=sg)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("case", sorted(CASES))
def test_own_routing_gives_the_layer(case):
    s = CASES[case]
    wl = make(s, seed=81)
    desc, w, x = _gpu.upload(wl)
    _, gids, gw, sg = _gpu.run_route(desc, w, x)
    ids, tw = gids.view(s.T, s.K).contiguous(), gw.view(s.T, s.K).contiguous()
    sg = sg.view(-1)[:s.T].contiguous() if desc.shared_I and desc.has_shared_gate else None
    out = _experts(desc, x, w, ids, tw, sg)
    assert moe.last_device_status() == moe.MOE_OK
    exp, _ = _gpu.expected_layer(oracle.from_workload(wl), ids.cpu().numpy())
    _gpu.assert_close(_gpu.to_np(out), exp, s.act_dtype, case)
    # pairs of no expert: the token's other experts and its shared one are left, weighted as given
    bad = ids.clone()
    bad[0] = -1
    bad[-1, -1] = s.E
    got = _experts(desc, x, w, bad, tw, sg)
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    zero = tw.clone()
    zero[0], zero[-1, -1] = 0, 0
    want = _experts(desc, x, w, ids, zero, sg)
    assert moe.last_device_status() == moe.MOE_OK
    tol = _gpu.tolerance(exp, s.act_dtype)  # (the groups' rows, and with them the split of the sums, differ)
    assert np.max(np.abs(_gpu.to_np(got) - _gpu.to_np(want))) <= tol
