"""Calls that read what the library's own launch before them wrote, back to back on changing inputs, give what they give
one by one."""
import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests.test_gpu_fp8 import _fp8_weights, _gen, _ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,I,K", [(8, 512, 32, 256, 4), (300, 512, 64, 96, 6), (700, 1024, 64, 256, 6)])
def test_training_step_back_to_back(T, H, E, I, K):
    """select -> permute -> expert_ffn -> combine_backward -> select_backward, its gradient and the experts' coded and
    multiplied on, and experts: every launch starts while the one before it still runs."""
    g = _gen(T)
    t = _fp8_weights(E, H, I, 0, T + 1)
    w = moe.Weights(**t)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    sd = moe.SelectDesc(T=T, E=E, top_k=K, scoring="sigmoid")
    n = 4
    xs = torch.randn((n, T, H), generator=g, device="cuda").to(torch.bfloat16)
    ls = torch.randn((n, T, E), generator=g, device="cuda")
    ds = torch.randn((n, T, H), generator=g, device="cuda")
    E4, i32 = torch.float8_e4m3fn, torch.int32

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    ids, tw, out = empty(T, K, dtype=i32), empty(T, K), empty(T, H, dtype=torch.bfloat16)
    counts, offs, sp, pp = empty(E, dtype=i32), empty(E + 1, dtype=i32), empty(T * K, dtype=i32), empty(T * K, dtype=i32)
    y, dy, dw, dl = empty(T * K, H), empty(T, K, H), empty(T, K), empty(T, E)
    oq, oqs = empty(T, H, dtype=E4), empty(H // 128, T)
    q, qs = empty(T * K, H, dtype=E4), empty(H // 128, T * K)
    lq, lqs, p = empty(T, E, dtype=E4), empty(-(-E // 128), T), empty(T, -(-T // 32) * 32)
    tall, tq, ts = empty(-(-T // 32) * 32, E), empty(-(-T // 32) * 32, E, dtype=E4), empty(-(-T // 128), -(-E // 128))
    tall.normal_(generator=g)
    ws = torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    one = torch.ones_like(tw)

    def step(i, sync):
        def call(f, *a, **kw):
            f(*a, **kw)
            if sync:
                torch.cuda.synchronize()

        call(moe.select, sd, ls[i], ids, tw)
        call(moe.experts, d, xs[i], w, ids, tw, out, ws)
        call(moe.fp8_quantize, out, oq, oqs)
        call(moe.permute, d, ids, counts, offs, sp, pp)
        call(moe.expert_ffn, d, xs[i], w, offs, sp, one, y, ws)
        call(moe.combine_backward, y.view(T, K, H), tw, ds[i], dy, dw)
        call(moe.fp8_quantize, dy.view(T * K, H), q, qs)
        call(moe.select_backward, sd, ls[i], ids, dw, dl)
        call(moe.fp8_quantize, dl, lq, lqs)
        call(moe.fp8_quantize_weights, tall, tq, ts)
        call(moe.fp8_gemm, lq, lqs, tq, ts, p)
        return [v.clone() for v in (ids, tw, out, oq.view(torch.uint8), oqs, y, dw, q.view(torch.uint8), qs, dl, lq.view(torch.uint8), lqs, p)]

    want = [step(i, True) for i in range(n)]
    got = [step(i % n, False) for i in range(6 * n)]
    _ok()
    for i, r in enumerate(got):
        for k, (a, b) in enumerate(zip(r, want[i % n])):
            assert torch.equal(a, b), (i, k)


@pytest.mark.parametrize("T,dtype,w_dtype", [(5, "bf16", "bf16"), (100, "bf16", "bf16"), (400, "bf16", "bf16"), (3, "f32", "f32"),
                                             (90, "f32", "f32"), (90, "bf16", "fp8"), (900, "bf16", "fp8")])
def test_layers_back_to_back(T, dtype, w_dtype):
    """A layer on the layer before it, and the gradient of its combine: each call reads what the one before it writes."""
    H, E, I, K = 256, 32, 96, 4
    g = _gen(T)
    at = torch.bfloat16 if dtype == "bf16" else torch.float32
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, act_dtype=dtype, w_dtype=w_dtype, router_dtype=dtype)
    layers = []
    for i in range(2):
        router = (torch.randn((E, H), generator=g, device="cuda") / 16).to(at)
        if w_dtype == "fp8":
            layers.append(moe.Weights(router=router, **_fp8_weights(E, H, I, 0, T + i)))
        else:
            layers.append(moe.Weights(router=router, **{n: (torch.randn(s, generator=g, device="cuda") / 8).to(at) for n, s in
                                                       dict(gate=(E, I, H), up=(E, I, H), down=(E, H, I)).items()}))
    n = 3
    xs = (torch.randn((n, T, H), generator=g, device="cuda")).to(at)
    a, b, ws = torch.empty_like(xs[0]), torch.empty_like(xs[0]), torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    logits, ids, tw = torch.empty((T, E), device="cuda"), torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    counts, offs = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp, pp = (torch.empty(T * K, dtype=torch.int32, device="cuda") for _ in range(2))
    y, dy, dw = torch.empty((T * K, H), device="cuda"), torch.empty((T, K, H), device="cuda"), torch.empty((T, K), device="cuda")
    z = torch.empty_like(a)

    def step(i, sync):
        def call(f, *args):
            f(*args)
            if sync:
                torch.cuda.synchronize()

        call(moe.layer, d, xs[i], layers[0], a, ws)
        call(moe.layer, d, a, layers[1], b, ws)
        call(moe.route, d, b, layers[0], logits, ids, tw, None, ws)
        call(moe.permute, d, ids, counts, offs, sp, pp)
        call(moe.expert_ffn, d, b, layers[0], offs, sp, tw, y, ws)
        call(moe.combine, d, y, b, layers[0], None, z, ws)
        call(moe.combine_backward, y.view(T, K, H), tw, y.view(T, K, H)[:, 0].contiguous(), dy, dw)
        return [v.clone() for v in (a, b, logits, ids, tw, offs, sp, y, z, dy, dw)]

    want = [step(i, True) for i in range(n)]
    got = [step(i % n, False) for i in range(8 * n)]
    _ok()
    for i, r in enumerate(got):
        for k, (p, q) in enumerate(zip(r, want[i % n])):
            assert torch.equal(p, q), (i, k)
