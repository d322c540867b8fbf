"""The stable permutation at the borders between its launch forms (1 to 8 pairs a thread of a cluster, one CTA beyond)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_ffn_07_b200 as moe  # noqa: E402


@pytest.mark.parametrize("T,K", [(1, 1), (1023, 1), (1025, 1), (8191, 1), (1024, 8), (8193, 1), (2048, 8), (16385, 1),
                                 (4096, 8), (32769, 1), (8192, 8), (65537, 1), (20000, 7)])
@pytest.mark.parametrize("E", [1, 7, 256])
def test_sizes(T, K, E):
    if K > E:
        K, T = 1, T * K
    ids = np.random.default_rng(T + K + E).integers(0, E, (T, K)).astype(np.int32)
    d = moe.Desc(T=T, H=256, E=E, I=64, top_k=K)
    counts, offsets = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    pairs, place = (torch.full((T * K,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.permute(d, torch.from_numpy(ids).cuda(), counts, offsets, pairs, place)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    order = np.argsort(ids.ravel(), kind="stable")
    n = np.bincount(ids.ravel(), minlength=E)
    assert np.array_equal(counts.cpu().numpy(), n)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(n)]))
    assert np.array_equal(pairs.cpu().numpy(), order)
    back = np.empty_like(order)
    back[order] = np.arange(order.size)
    assert np.array_equal(place.cpu().numpy(), back)
