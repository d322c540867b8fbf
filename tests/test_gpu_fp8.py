"""Block-scaled 8-bit floats: quantisation, the grouped product and the experts against 64-bit references."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref

pytestmark = pytest.mark.gpu
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ok():
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK


# ------------------------------------------------------------------------------------------------ quantisation
def _quantize(x, fmt, pow2):
    R, C = x.shape
    q = torch.full((R, C), 0x7F, dtype=torch.uint8, device="cuda").view(FMT[fmt])
    s = torch.full((-(-C // 128), R), float("nan"), device="cuda")
    moe.fp8_quantize(x, q, s, pow2=pow2)
    _ok()
    return q, s


@pytest.mark.parametrize("R,C", [(1, 32), (1, 2816), (33, 704), (31, 1056), (16, 160), (300, 128), (65, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows_bit_exact(R, C, dtype, fmt, pow2):
    g = _gen(R + C)
    x = torch.randn((R, C + 16), generator=g, device="cuda") * torch.exp(4 * torch.randn((R, 1), generator=g, device="cuda"))
    x = x.to(dtype)[:, :C]  # padded rows
    if R > 5:
        x[1] = 0
        x[2] = 2.0 ** -120
        x[3] = 0.5
        x[4, ::2] = -448.0 / 16
        x[5] = torch.arange(C, device="cuda").to(dtype) / 16  # borders between codes
    q, s = _quantize(x, fmt, pow2)
    want, ws = ref.quantize(x.double(), fmt, pow2)
    assert torch.equal(s.t().double(), ws)
    assert torch.equal(q.double(), want)
    # every value is within half a step of its block's grid (plus the rounding of the product and the scale)
    back = ref.dequantize_rows(q, s)
    st = ref.step8(want, fmt) * ref.spread(ws, R, C, 1)
    assert torch.all((back - x.double()).abs() <= st / 2 * (1 + 2.0 ** -20) + x.double().abs() * 4 * ref.U32)


@pytest.mark.parametrize("pow2", [False, True])
def test_rows_nan_inf_stay_in_their_block(pow2):
    x = torch.randn((4, 384), generator=_gen(1), device="cuda")
    x[0, 5], x[1, 130], x[2, 300] = math.nan, math.inf, -math.inf
    q, s = _quantize(x, "e4m3", pow2)
    v = ref.dequantize_rows(q, s)
    bad = torch.zeros((4, 384), dtype=torch.bool, device="cuda")
    bad[0, :128] = bad[1, 128:256] = bad[2, 256:] = True
    assert torch.isnan(v[bad]).all() and torch.isfinite(v[~bad]).all()


def test_rows_extremes():
    """The largest finite values, and powers of two whose quotient sits on the border of the scale's exponent."""
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros((6, 256), device="cuda")
        x[0] = torch.finfo(dtype).max
        x[1] = torch.finfo(torch.float32).tiny
        x[2], x[3], x[4] = 448.0, 449.0 if dtype == torch.float32 else 450.0, 447.0
        x[5] = 2.0 ** 100
        x = x.to(dtype)
        for fmt in ("e4m3", "e5m2"):
            for pow2 in (False, True):
                q, s = _quantize(x, fmt, pow2)
                want, ws = ref.quantize(x.double(), fmt, pow2)
                assert torch.equal(s.t().double(), ws) and torch.equal(q.double(), want)


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (3, 200, 416), (2, 1, 32), (5, 130, 2048), (1, 33, 160)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("pow2", [False, True])
def test_weights_bit_exact(G, N, K, dtype, fmt, pow2):
    w = (torch.randn((G, N, K), generator=_gen(G + N + K), device="cuda") * 0.02).to(dtype)
    w[0, 0] = 0
    q = torch.full((G, N, K), 0x7F, dtype=torch.uint8, device="cuda").view(FMT[fmt])
    s = torch.full((G, -(-N // 128), -(-K // 128)), float("nan"), device="cuda")
    moe.fp8_quantize_weights(w, q, s, pow2=pow2)
    _ok()
    for i in range(G):
        want, ws = ref.quantize(w[i].double(), fmt, pow2, rows=128)
        assert torch.equal(s[i].double(), ws) and torch.equal(q[i].double(), want)
    q2, s2 = torch.empty_like(q[0]), torch.empty_like(s[0])
    moe.fp8_quantize_weights(w[0], q2, s2, pow2=pow2)
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


# ------------------------------------------------------------------------------------------------ product
def _operands(M, G, N, K, af, bf, seed):
    g = _gen(seed)
    a, sa = _quantize(torch.randn((M, K), generator=g, device="cuda"), af, False)
    w = torch.randn((G, N, K), generator=g, device="cuda") / math.sqrt(K)
    b = torch.empty((G, N, K), dtype=FMT[bf], device="cuda")
    sb = torch.empty((G, -(-N // 128), -(-K // 128)), device="cuda")
    moe.fp8_quantize_weights(w, b, sb)
    return a, sa, b, sb


def _product(a, sa, b, sb, off, out_dtype):
    M, N = a.shape[0], b.shape[-2]
    out = torch.full((M, N), float("nan"), dtype=out_dtype, device="cuda")
    off_d = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    moe.fp8_gemm(a, sa, b, sb, out, offsets=off_d)
    _ok()
    return out


def _check_product(out, a, sa, b, sb, off):
    M, K = a.shape
    A = ref.dequantize_rows(a, sa)
    covered = torch.zeros(M, dtype=torch.bool, device="cuda")
    for i in range(len(off) - 1):
        r0, r1 = off[i], off[i + 1]
        if r1 <= r0:
            continue
        covered[r0:r1] = True
        W = ref.dequantize_weights(b[i], sb[i])
        want = A[r0:r1] @ W.T
        tol = ref.sum_bound(K) * (A[r0:r1].abs() @ W.abs().T)
        if out.dtype == torch.bfloat16:
            tol = tol + ref.U16 * (want.abs() + tol)
        err = (out[r0:r1].double() - want).abs()
        assert torch.all(err <= tol), (i, float((err - tol).max()))
    assert torch.isnan(out[~covered].float()).all()  # rows of no group are left alone


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (1, 2048, 512), (3, 96, 160), (16, 128, 128), (17, 160, 1056),
                                   (33, 704, 2816), (128, 256, 384), (129, 32, 96), (300, 1056, 416), (700, 128, 2048)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product_dense(M, N, K, out):
    a, sa, b, sb = _operands(M, 1, N, K, "e4m3", "e4m3", M + N + K)
    _check_product(_product(a, sa, b, sb, None, out), a, sa, b, sb, [0, M])
    y = torch.empty((M, N), dtype=out, device="cuda")
    moe.fp8_gemm(a, sa, b[0], sb[0], y)  # a plain matrix
    assert torch.equal(y, _product(a, sa, b, sb, None, out))


@pytest.mark.parametrize("af,bf", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_product_formats(af, bf):
    a, sa, b, sb = _operands(70, 1, 224, 544, af, bf, 7)
    _check_product(_product(a, sa, b, sb, None, torch.float32), a, sa, b, sb, [0, 70])


@pytest.mark.parametrize("off", [[0, 5, 5, 40, 41, 60], [3, 3, 10, 10, 10, 10], [0, 0, 0, 0, 0, 0], [0, 64, 64, 64, 64, 64],
                                 [7, 20, 30, 31, 47, 63]])
@pytest.mark.parametrize("N,K", [(160, 288), (256, 128)])
def test_product_groups(off, N, K):
    a, sa, b, sb = _operands(64, 5, N, K, "e4m3", "e4m3", sum(off))
    _check_product(_product(a, sa, b, sb, off, torch.float32), a, sa, b, sb, off)


@pytest.mark.parametrize("M,G,seed", [(2000, 7, 1), (1500, 256, 2), (1000, 2, 3)])
def test_product_ragged(M, G, seed):
    rng = np.random.default_rng(seed)
    off = [0] + sorted(rng.integers(0, M - 10, G - 1).tolist()) + [M - 10]
    a, sa, b, sb = _operands(M, G, 224, 160, "e4m3", "e4m3", seed)
    _check_product(_product(a, sa, b, sb, off, torch.bfloat16), a, sa, b, sb, off)


def test_product_row_values_do_not_leak():
    """A NaN row of one group stays in its row."""
    a, sa, b, sb = _operands(40, 3, 96, 256, "e4m3", "e4m3", 4)
    off = [0, 11, 30, 40]
    clean = _product(a, sa, b, sb, off, torch.float32)
    a = a.clone()
    a.view(torch.uint8)[12, 100] = 0x7F
    sa[1, 35] = math.inf
    got = _product(a, sa, b, sb, off, torch.float32)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[12] = bad[35] = True
    assert not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], clean[~bad])


def test_product_offsets_are_checked():
    a, sa, b, sb = _operands(40, 3, 96, 256, "e4m3", "e4m3", 5)
    out = torch.full((40, 96), float("nan"), device="cuda")
    moe.fp8_gemm(a, sa, b, sb, out, offsets=torch.tensor([-5, 10, 30, 90], dtype=torch.int32, device="cuda"))
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    _check_product(out, a, sa, b, sb, [0, 10, 30, 40])


def test_product_gradient_is_the_product_with_the_transposed_stack():
    """d_a = d_out W: the same call on [K, N] matrices with transposed block scales."""
    a, sa, b, sb = _operands(50, 2, 160, 288, "e4m3", "e4m3", 6)
    off = [0, 21, 50]
    d_out, sd = _quantize(torch.randn((50, 160), generator=_gen(8), device="cuda"), "e5m2", False)
    bt, sbt = b.view(torch.uint8).transpose(1, 2).contiguous().view(b.dtype), sb.transpose(1, 2).contiguous()
    d_a = _product(d_out, sd, bt, sbt, off, torch.float32)
    D = ref.dequantize_rows(d_out, sd)
    for i in range(2):
        W = ref.dequantize_weights(b[i], sb[i])
        r = slice(off[i], off[i + 1])
        assert torch.all((d_a[r].double() - D[r] @ W).abs() <= ref.sum_bound(160) * (D[r].abs() @ W.abs()))


# ------------------------------------------------------------------------------------------------ experts
def _fp8_weights(E, H, I, Is, seed):
    g = _gen(seed)
    t = {}
    for n, (G, N, K) in dict(gate=(E, I, H), up=(E, I, H), down=(E, H, I), sh_gate=(1, Is, H), sh_up=(1, Is, H),
                             sh_down=(1, H, Is)).items():
        if N == 0 or K == 0:
            continue
        w = torch.randn((G, N, K), generator=g, device="cuda") / math.sqrt(K)
        q = torch.empty((G, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((G, -(-N // 128), -(-K // 128)), device="cuda")
        moe.fp8_quantize_weights(w, q, s)
        t[n], t[n + "_scale"] = (q[0], s[0]) if n.startswith("sh") else (q, s)
    return t


def _expected(x, ids, tw, sg, t, E, act):
    T, K = ids.shape
    H = x.shape[1]
    q, s = ref.quantize(x.double(), "e4m3", False)
    X = q * ref.spread(s, T, H, 1)
    out, tol = torch.zeros((T, H), dtype=torch.float64, device="cuda"), torch.zeros((T, H), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for e in range(E):
        for k in range(K):
            rows = torch.nonzero(ids[:, k] == e).flatten()
            if rows.numel():
                y, b = ref.ffn(X[rows], *[ref.dequantize_weights(t[n][e], t[n + "_scale"][e]) for n in ("gate", "up", "down")], act)
                w = tw[rows, k, None].double()
                out[rows] += w * y
                tol[rows] += w.abs() * b
                mag[rows] += w.abs() * y.abs()
    if "sh_gate" in t:
        y, b = ref.ffn(X, *[ref.dequantize_weights(t["sh_" + n], t["sh_" + n + "_scale"]) for n in ("gate", "up", "down")], act)
        g = sg.double()[:, None] if sg is not None else 1.0
        out += g * y
        tol += abs(g) * b if sg is None else g.abs() * b
        mag += (g * y).abs()
    half = ref.U16 if x.dtype == torch.bfloat16 else ref.U32
    tol = tol + half * (mag + tol) + (K + 2) * ref.U32 * mag   # slot rows, and the sum over the slots
    return out, tol + half * (out.abs() + tol)                 # the output's rounding


def _experts(d, x, t, ids, tw, sg=None, ws=None, out=None, **kw):
    w = moe.Weights(**t)
    out = torch.full((d.T, d.H), float("nan"), dtype=x.dtype, device="cuda") if out is None else out
    ws = torch.full((moe.workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    moe.experts(d, x, w, ids, tw, out, ws, shared_gate=sg, **kw)
    return out


SHAPES = [  # T, H, E, I, K, Is
    (1, 256, 4, 128, 2, 0), (1, 2816, 16, 704, 8, 0), (5, 160, 8, 96, 3, 64), (16, 512, 8, 160, 4, 96),
    (64, 288, 3, 224, 2, 0), (200, 256, 4, 256, 4, 160), (333, 544, 60, 96, 6, 0), (500, 128, 2, 32, 1, 32)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts(shape, act, dtype):
    T, H, E, I, K, Is = shape
    g = _gen(sum(shape))
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = _fp8_weights(E, H, I, Is, T + H)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    sg = torch.rand(T, generator=g, device="cuda") if Is else None
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, act=act, act_dtype=dtype, w_dtype="fp8", shared_I=Is, has_shared_gate=Is > 0)
    out = _experts(d, x, t, ids, tw, sg)
    _ok()
    want, tol = _expected(x, ids, tw, sg, t, E, act)
    err = (out.double() - want).abs()
    assert torch.all(err <= tol), float((err / tol).max())
    # two bf16 roundings, each at most 2^-8 / sqrt(3) of the values in the mean square, and rare code changes: 2^-8 / sqrt(3)
    # for f32 activations leaves the code changes alone (one element in a thousand by one step of at most 2^-3)
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= (ref.U16 if dtype == "bf16" else 2.0 ** -8 / math.sqrt(3)), rel


def test_experts_edge_routings():
    """All pairs on one expert, the same expert twice, zero and negative weights, ids of no expert."""
    T, H, E, I, K = 150, 256, 5, 160, 3
    g = _gen(31)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    t = _fp8_weights(E, H, I, 0, 32)
    tw = torch.randn((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    for kind in ("one", "twice", "zero", "none"):
        ids = torch.randint(0, E, (T, K), generator=g, device="cuda").to(torch.int32)
        w = tw.clone()
        if kind == "one":
            ids[:] = 3
        elif kind == "twice":
            ids[:, 1] = ids[:, 0]
        elif kind == "zero":
            w[::2] = 0
        else:
            ids[::3, 0], ids[1::3, 2], ids[7] = -1, E, 1 << 30
        out = _experts(d, x, t, ids, w)
        torch.cuda.synchronize()
        assert moe.last_device_status() == (moe.MOE_ERR_DEVICE_INDEX if kind == "none" else moe.MOE_OK)
        want, tol = _expected(x, ids, w, None, t, E, "silu")
        assert torch.all((out.double() - want).abs() <= tol), kind
        if kind == "none":
            assert torch.all(out[7] == 0)


def test_bad_token_stays_in_its_row():
    T, H, E, I, K = 40, 256, 4, 128, 2
    g = _gen(41)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    t = _fp8_weights(E, H, I, 0, 42)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.rand((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    clean = _experts(d, x, t, ids, tw)
    x = x.clone()
    x[9, 3], x[20, 200] = math.nan, math.inf
    got = _experts(d, x, t, ids, tw)
    _ok()
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[9] = bad[20] = True
    assert torch.isnan(got[bad].float()).all() and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("fmt,act_dtype,T", [("bf16", "bf16", 70), ("bf16", "bf16", 5), ("f32", "f32", 6), ("bf16", "f32", 6)])
def test_experts_of_the_other_formats(fmt, act_dtype, T):
    """moe_experts on moe_layer's own routing gives moe_layer's output, for formats it serves besides fp8."""
    H, E, I, K = 256, 8, 128, 2
    g = _gen(51)
    wt, at = (torch.bfloat16 if v == "bf16" else torch.float32 for v in (fmt, act_dtype))
    x = torch.randn((T, H), generator=g, device="cuda").to(at)
    t = {n: (torch.randn(s, generator=g, device="cuda") / 16).to(wt)
         for n, s in dict(gate=(E, I, H), up=(E, I, H), down=(E, H, I)).items()}
    router = (torch.randn((E, H), generator=g, device="cuda") / 16).to(wt)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, act_dtype=act_dtype, w_dtype=fmt, router_dtype=fmt)
    w = moe.Weights(router=router, **t)
    ws = torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, K), device="cuda")
    moe.route(d, x, w, torch.empty((T, E), device="cuda"), ids, tw, None, ws)
    want = torch.empty_like(x)
    moe.layer(d, x, w, want, ws)
    got = torch.full_like(x, float("nan"))
    ids2, tw2 = ids.clone(), tw.clone()
    moe.experts(d, x, w, ids2, tw2, got, ws)
    _ok()
    # same products; f32 sums may be taken in another order (streaming path): the layer's f32 tolerance
    tol = (2.0 ** -7 if act_dtype == "bf16" else 1e-5) * want.float().abs().max()
    assert torch.all((got.float() - want.float()).abs() <= tol)
    bad = ids2.clone()
    bad[0] = -1
    moe.experts(d, x, w, bad, tw2, got, ws)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    assert torch.all(got[0] == 0) and torch.all((got[1:].float() - want[1:].float()).abs() <= tol)


@pytest.mark.parametrize("T,router_dtype,shared", [(1, "f32", 0), (9, "bf16", 64), (100, "bf16", 64), (100, "f32", 0)])
def test_layer_and_steps(T, router_dtype, shared):
    """moe_layer with fp8 experts is moe_route + moe_experts, and the steps one by one give the same values."""
    H, E, I, K = 256, 32, 160, 4
    g = _gen(61)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    t = _fp8_weights(E, H, I, shared, 62)
    rt = torch.bfloat16 if router_dtype == "bf16" else torch.float32
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", router_dtype=router_dtype, shared_I=shared,
                 has_shared_gate=shared > 0)
    w = moe.Weights(router=(torch.randn((E, H), generator=g, device="cuda") / 16).to(rt),
                    sh_gate_w=(torch.randn(H, generator=g, device="cuda") / 16).to(rt) if shared else None, **t)
    ws = torch.full((moe.workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, float("nan"))
    moe.layer(d, x, w, out, ws)
    _ok()
    r = moe.workspace_regions(d)

    def region(name, n, dtype):
        return ws[r[name]:r[name] + 4 * n].view(dtype).clone()

    ids = region("topk_ids", T * K, torch.int32).view(T, K)
    tw = region("topk_w", T * K, torch.float32).view(T, K)
    sg = region("shared_gate", T, torch.float32) if shared else None
    got = _experts(d, x, t, ids, tw, sg)
    _ok()
    assert torch.equal(got, out)
    logits, ids2, tw2 = torch.empty((T, E), device="cuda"), torch.empty_like(ids), torch.empty_like(tw)
    sg2 = torch.empty(T, device="cuda")
    ws2 = torch.full_like(ws, 0xFF)
    moe.route(d, x, w, logits, ids2, tw2, sg2 if shared else None, ws2)
    counts, offs = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp, pp = torch.empty(T * K, dtype=torch.int32, device="cuda"), torch.empty(T * K, dtype=torch.int32, device="cuda")
    moe.permute(d, ids2, counts, offs, sp, pp)
    y = torch.full((T * K, H), float("nan"), device="cuda")
    moe.expert_ffn(d, x, w, offs, sp, tw2, y, ws2)
    step = torch.full_like(x, float("nan"))
    moe.combine(d, y, x, w, sg2 if shared else None, step, ws2)
    _ok()
    assert torch.equal(ids2, ids) and torch.equal(tw2, tw)
    want, tol = _expected(x, ids, tw, sg, t, E, "silu")
    assert torch.all((out.double() - want).abs() <= tol)
    assert torch.all((step.double() - want).abs() <= tol)
    if moe.workspace_bytes(d) < 32 << 20:
        na = torch.full_like(x, float("nan"))
        moe.layer_noalloc(d, x, w, na)
        assert torch.equal(na, out)


def test_routing_to_gradient_run():
    """A training step's router around the experts: select -> experts -> combine_backward -> select_backward."""
    T, H, E, I, K = 90, 256, 16, 128, 4
    g = _gen(71)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    t = _fp8_weights(E, H, I, 0, 72)
    sd = moe.SelectDesc(T=T, E=E, top_k=K, scoring="sigmoid", n_groups=4, topk_groups=2, group_score="top2", scale=2.5)
    ids, tw = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.select(sd, logits, ids, tw, bias=bias)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    out = _experts(d, x, t, ids, tw)
    rid, rw, _ = ref.select(logits, K, "sigmoid", bias, 4, 2, "top2", True, 2.5)
    assert torch.equal(ids.long(), rid)
    want, tol = _expected(x, ids, rw.float(), None, t, E, "silu")
    assert torch.all((out.double() - want).abs() <= tol * (1 + 1e-5))
    # gradient of sum(out * d_out) with respect to the logits through the weights
    d_out = torch.randn((T, H), generator=g, device="cuda")
    y = torch.empty((T * K, H), device="cuda")
    counts, offs = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp, pp = torch.empty(T * K, dtype=torch.int32, device="cuda"), torch.empty(T * K, dtype=torch.int32, device="cuda")
    moe.permute(d, ids, counts, offs, sp, pp)
    ws = torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    moe.expert_ffn(d, x, moe.Weights(**t), offs, sp, torch.ones_like(tw), y, ws)
    d_y, d_w = torch.empty((T, K, H), device="cuda"), torch.empty((T, K), device="cuda")
    moe.combine_backward(y.view(T, K, H), tw, d_out, d_y, d_w)
    d_logits = torch.empty_like(logits)
    moe.select_backward(sd, logits, ids, d_w, d_logits)
    _ok()
    rdw = (y.view(T, K, H).double() * d_out.double()[:, None]).sum(2)
    want, mag = ref.select_backward(logits, rid, rdw, None, "sigmoid", True, 2.5)
    dw_err = H * 2.0 ** -24 * (y.view(T, K, H).double() * d_out.double()[:, None]).abs().sum(2)
    _, more = ref.select_backward(logits, rid, dw_err, None, "sigmoid", True, 2.5)
    assert torch.all((d_logits.double() - want).abs() <= 400 * ref.U32 * mag + 2 * more)


def test_streams_graphs_and_two_calls_at_once():
    """Captured and replayed on new inputs, and two calls in flight on two streams with a workspace each."""
    T, H, E, I, K = 24, 512, 8, 256, 2
    t = _fp8_weights(E, H, I, 0, 81)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    sd = moe.SelectDesc(T=T, E=E, top_k=K)

    def inputs(seed):
        g = _gen(seed)
        return (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16),
                torch.randn((T, E), generator=g, device="cuda"))

    def run(x, l, ids, tw, out, ws):
        moe.select(sd, l, ids, tw)
        moe.experts(d, x, moe.Weights(**t), ids, tw, out, ws)

    def fresh():
        return (torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda"),
                torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
                torch.full((moe.workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda"))

    want = []
    for seed in (1, 2, 3):
        b = fresh()
        run(*inputs(seed), *b)
        torch.cuda.synchronize()
        want.append(b[2].clone())
    x, l = inputs(1)
    buf = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x, l, *buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(x, l, *buf)
    for i, seed in enumerate((1, 2, 3)):
        nx, nl = inputs(seed)
        x.copy_(nx)
        l.copy_(nl)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf[2], want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [fresh() for _ in streams]
    ins = [inputs(2), inputs(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, b, i in zip(streams, bufs, ins):
            with torch.cuda.stream(s):
                run(*i, *b)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][2], want[1]) and torch.equal(bufs[1][2], want[2])
    _ok()


def test_deterministic():
    T, H, E, I, K = 300, 512, 8, 256, 4
    g = _gen(91)
    t = _fp8_weights(E, H, I, 128, 92)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", shared_I=128)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.rand((T, K), generator=g, device="cuda")
    first = _experts(d, x, t, ids, tw)
    for _ in range(3):
        assert torch.equal(_experts(d, x, t, ids, tw), first)
    # a token's output does not depend on the tokens beside it
    d1 = moe.Desc(T=1, H=H, E=E, I=I, top_k=K, w_dtype="fp8", shared_I=128)
    for i in (0, 17, 299):
        one = _experts(d1, x[i:i + 1].contiguous(), t, ids[i:i + 1].contiguous(), tw[i:i + 1].contiguous())
        want, tol = _expected(x[i:i + 1], ids[i:i + 1], tw[i:i + 1], None, t, E, "silu")
        assert torch.all((one.double() - want).abs() <= tol)


@pytest.mark.parametrize("M,N,K", [(2, 64, 4128), (16, 352, 7200), (5, 32, 2048), (31, 96, 4992), (32, 32, 8192)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product_few_items_split_over_k(M, N, K, out):
    """Few tiles: the k-blocks are shared by CTAs of a cluster, in parts that do not divide evenly."""
    a, sa, b, sb = _operands(M, 1, N, K, "e4m3", "e4m3", M + N + K)
    first = _product(a, sa, b, sb, None, out)
    _check_product(first, a, sa, b, sb, [0, M])
    for _ in range(20):
        assert torch.equal(_product(a, sa, b, sb, None, out), first)


@pytest.mark.parametrize("M,off", [(300, None), (300, [0, 130, 131, 290]), (20, [0, 3, 9, 20])])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product_output_at_sixteen_bytes(M, off, out):
    """Outputs on a 16-byte boundary that is no 32-byte one, inside a larger buffer whose rest is left alone."""
    G = 1 if off is None else 3
    a, sa, b, sb = _operands(M, G, 160, 416, "e4m3", "e4m3", 9)
    pad = 16 // out.itemsize
    buf = torch.full((M * 160 + 2 * pad,), float("nan"), dtype=out, device="cuda")
    assert buf.data_ptr() % 32 == 0
    y = buf[pad:-pad].view(M, 160)
    off_d = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    moe.fp8_gemm(a, sa, b, sb, y, offsets=off_d)
    _ok()
    _check_product(y, a, sa, b, sb, off or [0, M])
    assert torch.isnan(buf[:pad].float()).all() and torch.isnan(buf[-pad:].float()).all()


def _spread_routing(T, E, K, seed):
    """Ids whose experts hold from none to many rows."""
    g = _gen(seed)
    lean = torch.exp(2 * torch.randn(E, generator=g, device="cuda"))
    return torch.multinomial(lean.expand(T, E), K, generator=g).to(torch.int32), torch.rand((T, K), generator=g, device="cuda")


@pytest.mark.parametrize("T,H,E,I,K", [(40, 512, 64, 384, 6), (100, 256, 60, 96, 6), (100, 1024, 128, 256, 8), (400, 512, 64, 512, 6)])
def test_many_passes_give_the_same_bits(T, H, E, I, K):
    """Every CTA works through items of groups of all sizes (one row to several tiles), over many passes: the pipelines'
    barriers are passed millions of times without a wait that expires or a sum that differs."""
    t = _fp8_weights(E, H, I, 0, T + E)
    ids, tw = _spread_routing(T, E, K, T)
    x = torch.randn((T, H), generator=_gen(T + 1), device="cuda").to(torch.bfloat16)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    ws = torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    w = moe.Weights(**t)
    first = _experts(d, x, t, ids, tw)
    _ok()
    want, tol = _expected(x, ids, tw, None, t, E, "silu")
    assert torch.all((first.double() - want).abs() <= tol)
    out = torch.empty_like(first)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        moe.experts(d, x, w, ids, tw, out, ws)
        differ += (out != first).sum()
    _ok()
    assert int(differ) == 0


@pytest.mark.parametrize("T,E,K", [(8, 4, 2), (24, 16, 4), (60, 4, 2), (300, 4, 2)])  # each form of the product
def test_wait_timeout_is_reported_and_context_survives(T, E, K):
    """One stage of CTA 0 is left unfilled: its waits run out, the error is reported and the next call is right."""
    H, I = 512, 256
    t = _fp8_weights(E, H, I, 0, 71)
    g = _gen(72)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.rand((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    clean = _experts(d, x, t, ids, tw)
    _ok()
    a, sa, b, sb = _operands(T, 1, H, I, "e4m3", "e4m3", 73)
    product = _product(a, sa, b, sb, None, torch.float32)
    out = torch.empty_like(clean)
    y = torch.empty_like(product)
    try:
        moe.debug_set_wait_limit(20_000_000)  # about 10 ms of SM cycles
        moe.debug_set_skip_stage(True)
        _experts(d, x, t, ids, tw, out=out)
        torch.cuda.synchronize()
        assert moe.last_device_status() == moe.MOE_ERR_TIMEOUT
        moe.fp8_gemm(a, sa, b, sb, y)
        torch.cuda.synchronize()
        assert moe.last_device_status() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.debug_set_skip_stage(False)
        moe.debug_set_wait_limit(0)
    assert torch.equal(_experts(d, x, t, ids, tw), clean)
    assert torch.equal(_product(a, sa, b, sb, None, torch.float32), product)
    _ok()


def test_layer_host():
    """The layer from and to pinned host memory, with fp8 experts."""
    T, H, E, I, K = 33, 256, 8, 128, 2
    g = _gen(75)
    t = _fp8_weights(E, H, I, 0, 76)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", router_dtype="f32")
    w = moe.Weights(router=(torch.randn((E, H), generator=g, device="cuda") / 16), **t)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ws = torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(x)
    moe.layer(d, x, w, want, ws)
    _ok()
    xh, oh = x.cpu().pin_memory(), torch.empty((T, H), dtype=torch.bfloat16).pin_memory()
    moe.layer_host(d, xh, w, oh, torch.empty_like(x), torch.empty_like(x), ws)
    _ok()
    assert torch.equal(oh, want.cpu())


def test_quantize_in_a_graph():
    x = torch.randn((40, 416), generator=_gen(77), device="cuda")
    w = torch.randn((2, 96, 416), generator=_gen(78), device="cuda")
    q, s = torch.empty((40, 416), dtype=FMT["e4m3"], device="cuda"), torch.empty((4, 40), device="cuda")
    qw, sw = torch.empty((2, 96, 416), dtype=FMT["e4m3"], device="cuda"), torch.empty((2, 1, 4), device="cuda")
    off = torch.tensor([0, 11, 40], dtype=torch.int32, device="cuda")
    y = torch.empty((40, 96), device="cuda")

    def run():
        moe.fp8_quantize(x, q, s)
        moe.fp8_quantize_weights(w, qw, sw)
        moe.fp8_gemm(q, s, qw, sw, y, offsets=off)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=_gen(79 + i), device="cuda"))
        w.copy_(torch.randn(w.shape, generator=_gen(89 + i), device="cuda"))
        graph.replay()
        _ok()
        got = y.clone()
        run()
        _ok()
        assert torch.equal(got, y)
        _check_product(got, q, s, qw, sw, [0, 11, 40])


@pytest.mark.parametrize("M,N,K", [(40, 512, 2080), (160, 256, 1056), (500, 32, 160), (600, 1024, 256), (1000, 544, 96)])
def test_product_of_one_matrix_by_rows(M, N, K):
    """From few items, that share k-blocks, to many rows: both forms of the product, on both sides of the crossover."""
    a, sa, b, sb = _operands(M, 1, N, K, "e4m3", "e5m2", M + N)
    _check_product(_product(a, sa, b, sb, None, torch.bfloat16), a, sa, b, sb, [0, M])
    _check_product(_product(a, sa, b, sb, None, torch.float32), a, sa, b, sb, [0, M])


def test_weights_are_checked():
    """Stacks and scales of another size, type or layout are refused before anything is launched."""
    T, H, E, I, K = 8, 256, 4, 160, 2
    t = _fp8_weights(E, H, I, 64, 95)
    g = _gen(96)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.rand((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", shared_I=64)
    launched = moe.launch_count()
    bad = [dict(gate=t["gate"][:3]), dict(up=t["up"].view(torch.uint8)), dict(down=t["up"]),
           dict(gate_scale=t["gate_scale"][:, :1].contiguous()), dict(up_scale=t["up_scale"].double()), dict(down_scale=None),
           dict(gate=t["gate"].view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn)),
           dict(sh_down=t["sh_down"][:, :32].contiguous()), dict(sh_gate=None), dict(up=t["up"].cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            _experts(d, x, {**t, **b}, ids, tw)
    with pytest.raises(ValueError):
        _experts(d, x, t, ids, tw, ws=torch.empty(moe.workspace_bytes(d), dtype=torch.uint8))
    assert moe.launch_count() == launched
    _experts(d, x, t, ids, tw)
    _ok()


@pytest.mark.parametrize("shape", [(100, 256, 60, 96, 6, 0), (20, 128, 40, 64, 32, 32), (70, 128, 33, 32, 17, 0), (900, 1056, 5, 96, 5, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_of_many_slots(shape, dtype):
    """Up to 32 experts a token, and batches past the single front launch whose rows are gathered or put in order."""
    test_experts(shape, "silu", dtype)


@pytest.mark.parametrize("T,H,E", [(12, 512, 16), (100, 512, 64), (400, 512, 8)])
def test_inputs_written_just_before(T, H, E):
    """x, ids and weights come from launches right before the call, on its stream, and change from call to call."""
    I, K = 128, 4
    t = _fp8_weights(E, H, I, 0, 97)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    w, ws = moe.Weights(**t), torch.empty(moe.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    g = _gen(98)
    xs = torch.randn((6, T, H), generator=g, device="cuda").to(torch.bfloat16)
    idss = torch.rand((6, T, E), generator=g, device="cuda").topk(K, 2).indices.to(torch.int32)
    tws = torch.rand((6, T, K), generator=g, device="cuda")
    want = [_experts(d, xs[i], t, idss[i], tws[i]) for i in range(6)]
    _ok()
    x, ids, tw = torch.empty_like(xs[0]), torch.empty_like(idss[0]), torch.empty_like(tws[0])
    slow = torch.randn((4096, 4096), device="cuda")
    outs = torch.empty((60, T, H), dtype=torch.bfloat16, device="cuda")
    for i in range(60):
        if i % 7 == 0:
            slow = torch.mm(slow, slow) * 1e-4  # a launch that takes longer than the call
        tw.copy_(tws[i % 6])
        ids.copy_(idss[i % 6])
        x.copy_(xs[i % 6])
        moe.experts(d, x, w, ids, tw, outs[i], ws)
    _ok()
    for i in range(60):
        assert torch.equal(outs[i], want[i % 6]), i
