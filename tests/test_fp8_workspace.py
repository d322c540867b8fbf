"""Workspace of layers with experts of 8-bit floats: what each form of the products needs, and no more (on the host)."""
import pytest

import mixture_experts_ffn_07_b200 as moe


@pytest.mark.parametrize("T,E,K", [(1, 128, 8), (16, 128, 8), (200, 256, 8), (500, 256, 8), (4096, 256, 8)])
@pytest.mark.parametrize("H,I", [(2048, 768), (7168, 2048), (160, 96)])
def test_regions(T, E, K, H, I):
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    n, P = moe.workspace_bytes(d), T * K
    mean = P / min(E, P)
    # up to 8 rows an expert f32 slot rows, many f16 ones with a power of two for each 128; x in expert order where it is
    # not gathered
    slots = P * H * 4 if mean <= 8 else P * (2 * H + 4 * -(-H // 128))
    x = T * H + (P * H if mean > 16 else 0)
    rest = P * I + 4 * (-(-H // 128) * T + -(-I // 128) * P) + 4 * (T * E + 8 * P + 2 * E)
    router = 20480 * E * 4 + 256 * E * 4  # split-K logits and counts, at most
    assert slots + x <= n <= slots + x + rest + router + 32 * 256
