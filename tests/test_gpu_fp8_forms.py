"""Which of the two kernels of the block-scaled product a call takes, and both of them over the shapes and forms that their
users meet."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref
from tests.test_gpu_fp8 import _check_product, _experts, _expected, _fp8_weights, _gen, _ok, _operands, _product

pytestmark = pytest.mark.gpu


def _names(run):
    """Names of the launches of run(), and what it returns."""
    moe.trace_enable(True)
    moe.trace_read()
    try:
        out = run()
        torch.cuda.synchronize()
        return [n for n, _ in moe.trace_read()], out
    finally:
        moe.trace_enable(False)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("M,N", [(128, 4096), (128, 4608), (96, 4096), (96, 6016), (64, 9472), (32, 18944), (33, 9472), (33, 9600),
                                 (160, 3584), (128, 4864), (8, 18944), (256, 2304), (256, 2432), (320, 4096)])
def test_a_single_matrix_fills_the_gpu_or_not(M, N):
    """Tiles of 32 rows x 128 outputs, no more of them than SMs: the few-row kernel, whatever M is a multiple of.  More of
    them and more than 8 rows: the other one."""
    K = 288
    a, sa, b, sb = _operands(M, 1, N, K, "e4m3", "e4m3", M + N)
    names, out = _names(lambda: _product(a, sa, b, sb, None, torch.float32))
    tiles = -(-M // 32) * -(-N // 128)
    assert names == ["fp8_gemm" if tiles <= _sms() or M <= 8 else "fp8_gemm_rows"], tiles
    _check_product(out, a, sa, b, sb, [0, M])


# ------------------------------------------------------------------------------------------------ many rows a group
MANY = [  # M, G, N, K: K and N that end inside blocks and tiles of weights, odd and even numbers of them
    (1000, 1, 1056, 416), (1100, 1, 2048, 32), (777, 3, 1184, 2080), (2500, 40, 1312, 288), (1024, 5, 1024, 1152)]


@pytest.mark.parametrize("M,G,N,K", MANY)
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_many_rows(M, G, N, K, af, bf, out):
    """Every pair of formats, both outputs, ragged groups (one of them empty) and rows of none."""
    a, sa, b, sb = _operands(M, G, N, K, af, bf, M + N)
    off = None
    if G > 1:
        rng = np.random.default_rng(M)
        off = [5] + sorted(rng.integers(5, M - 7, G - 1).tolist()) + [M - 7]
        off[2] = off[1]
    names, y = _names(lambda: _product(a, sa, b, sb, off, out))
    assert names == ["fp8_gemm_rows"]
    _check_product(y, a, sa, b, sb, off or [0, M])


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ragged", [False, True])
def test_many_rows_at_sixteen_bytes(out, ragged):
    """An output on a 16-byte boundary that is no 32-byte one."""
    M, N, K, G = 1000, 1056, 416, 3 if ragged else 1
    off = [0, 300, 301, 990] if ragged else None
    a, sa, b, sb = _operands(M, G, N, K, "e5m2", "e4m3", 3)
    pad = 16 // out.itemsize
    buf = torch.full((M * N + 2 * pad,), float("nan"), dtype=out, device="cuda")
    y = buf[pad:-pad].view(M, N)
    off_d = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    names, _ = _names(lambda: moe.fp8_gemm(a, sa, b, sb, y, offsets=off_d))
    _ok()
    assert names == ["fp8_gemm_rows"] and y.data_ptr() % 32 == 16
    _check_product(y, a, sa, b, sb, off or [0, M])
    assert torch.isnan(buf[:pad].float()).all() and torch.isnan(buf[-pad:].float()).all()


def _spread_ids(T, E, K, g):
    lean = torch.exp(torch.randn(E, generator=g, device="cuda"))
    return torch.multinomial(lean.expand(T, E), K, generator=g).to(torch.int32)


@pytest.mark.parametrize("T,H,E,I,K,Is", [(700, 256, 64, 416, 6, 0), (700, 1056, 64, 480, 6, 0), (1500, 288, 40, 96, 4, 160),
                                          (900, 160, 64, 352, 8, 1056)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_of_experts(T, H, E, I, K, Is, act, dtype):
    """Hidden rows and outputs that end inside a block of 128, K tails, both activations and types of x."""
    g = _gen(T + H)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = _fp8_weights(E, H, I, Is, T + I)
    ids = _spread_ids(T, E, K, g)
    tw = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    sg = torch.rand(T, generator=g, device="cuda") if Is else None
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, act=act, act_dtype=dtype, w_dtype="fp8", shared_I=Is, has_shared_gate=Is > 0)
    names, out = _names(lambda: _experts(d, x, t, ids, tw, sg))
    assert moe.last_device_status() == moe.MOE_OK
    assert "expert_gate_up_fp8_rows" in names and "expert_down_fp8_rows" in names
    want, tol = _expected(x, ids, tw, sg, t, E, act)
    err = (out.double() - want).abs()
    assert torch.all(err <= tol), float((err / tol).max())
    # one bf16 rounding (2^-8 / sqrt(3) of the values in the mean square, at most), f16 slot rows an eighth of that, and rare
    # code changes (2^-3 of one element in a thousand or fewer); f32 rows and outputs have the last alone
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= 2.0 ** -8 / math.sqrt(3) * (1.1 if dtype == "bf16" else 1.0), rel


@pytest.mark.parametrize("T,H,E,I,K", [(1024, 7168, 256, 256, 8), (600, 2304, 256, 1024, 8)])
def test_large_experts(T, H, E, I, K):
    """256 experts, rows of 7168, more k-blocks than the rings of either kernel hold."""
    g = _gen(T)
    t = _fp8_weights(E, H, I, 0, 5)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = _spread_ids(T, E, K, g)
    tw = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    names, out = _names(lambda: _experts(d, x, t, ids, tw))
    assert moe.last_device_status() == moe.MOE_OK
    assert "expert_gate_up_fp8_rows" in names and "expert_down_fp8_rows" in names
    q, s = ref.quantize(x.double(), "e4m3", False)
    X = q * ref.spread(s, T, H, 1)
    want, tol, mag = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(3))
    for e in range(E):
        rows, k = torch.nonzero(ids == e, as_tuple=True)  # (an expert once a token)
        if rows.numel():
            y, b = ref.ffn(X[rows], *[ref.dequantize_weights(t[n][e], t[n + "_scale"][e]) for n in ("gate", "up", "down")], "silu")
            w = tw[rows, k, None].double()
            want[rows] += w * y
            tol[rows] += w.abs() * (b + 2.0 ** -11 * (y.abs() + b))
            mag[rows] += w.abs() * y.abs()
    tol = tol + (K + 2) * ref.U32 * mag
    err = (out.double() - want).abs()
    assert torch.all(err <= tol + ref.U16 * (want.abs() + tol))
    assert float((out.double() - want).norm() / want.norm()) <= 1.1 * 2.0 ** -8 / math.sqrt(3)


def test_large_groups():
    """The product itself with 256 groups and 18 k-blocks."""
    M, G, N, K = 9000, 256, 1024, 2304
    rng = np.random.default_rng(1)
    off = [0] + sorted(rng.integers(0, M, G - 1).tolist()) + [M]
    a, sa, b, sb = _operands(M, G, N, K, "e4m3", "e4m3", 11)
    names, y = _names(lambda: _product(a, sa, b, sb, off, torch.bfloat16))
    assert names == ["fp8_gemm_rows"]
    _check_product(y, a, sa, b, sb, off)


@pytest.mark.parametrize("T,H,E,I,K", [(700, 512, 64, 416, 6)])
def test_expired_wait_of_many_rows(T, H, E, I, K):
    """One stage of CTA 0 is left unfilled in the gate/up product, in the down product that starts under it, and in a plain
    one: the waits run out, the error is reported, and the next call is right."""
    t = _fp8_weights(E, H, I, 0, 71)
    g = _gen(72)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = _spread_ids(T, E, K, g)
    tw = torch.rand((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    names, clean = _names(lambda: _experts(d, x, t, ids, tw))
    assert "expert_gate_up_fp8_rows" in names and "expert_down_fp8_rows" in names
    a, sa, b, sb = _operands(1000, 1, 1024, 416, "e4m3", "e4m3", 73)
    names, product = _names(lambda: _product(a, sa, b, sb, None, torch.float32))
    assert names == ["fp8_gemm_rows"]
    _ok()
    out, y = torch.empty_like(clean), torch.empty_like(product)
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
