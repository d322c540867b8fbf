"""Selection weights and their gradient where the chosen scores themselves are too small for f32 and their ratios are not."""
import math

import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref

pytestmark = pytest.mark.gpu


def _log_scores(l, scoring):
    """Logarithms of the scores in 64 bits, of softmax without the row's common term."""
    l = l.double()
    return l if scoring == "softmax" else l.clamp_max(0) - torch.log1p(torch.exp(-l.abs()))


def _ratios(l, ids, scoring):
    """Chosen scores over their sum, from their logarithms."""
    s = _log_scores(l, scoring).gather(1, ids)
    z = torch.exp(s - s.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def _case(scoring, far, seed, T=40, E=64, K=6):
    """Logits whose chosen experts (by a bias that outweighs every score) lie `far` below the row's maximum (softmax) or
    below zero (sigmoid)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=g, device="cuda") * 2
    chosen = torch.randperm(E, generator=g, device="cuda")[:K]
    if scoring == "softmax":
        l[:, 0] = 8.0
        chosen = chosen[chosen != 0]
    l[:, chosen] -= far
    bias = torch.zeros(E, device="cuda")
    bias[chosen] = 4.0 + torch.arange(chosen.numel(), device="cuda") / 4
    return l, bias, chosen.numel(), g


def _tol(l, ids):
    """Relative: an exponent is off by a rounding of its argument, exp by two steps, sum and quotient by a few."""
    c = l.double().gather(1, ids)
    return 2 * 2 * ref.U32 * (float((c.amax(1) - c.amin(1)).max()) + 16)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("far", [0.0, 60.0, 86.0, 95.0, 102.0, 104.0, 110.0, 700.0, 5000.0, 1e30])
def test_weights(scoring, dtype, far):
    l, bias, K, _ = _case(scoring, far, 3)
    l = l.to(dtype)
    T, E = l.shape
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring=scoring, scale=2.5)
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.full((T, K), math.nan, device="cuda")
    moe.select(d, l, ids, w, bias=bias)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    assert set(ids.flatten().tolist()) == set(torch.nonzero(bias).flatten().tolist())
    want = 2.5 * _ratios(l, ids.long(), scoring)
    assert torch.all((w.double() - want).abs() <= _tol(l, ids.long()) * want + 1e-37)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("far", [0.0, 86.0, 95.0, 104.0, 700.0, 5000.0])
@pytest.mark.parametrize("with_scores", [False, True])
def test_gradient(scoring, dtype, far, with_scores):
    """d_logits_e = scale n_e (d_w_e - sum_j d_w_j n_j) (1 - s_e with sigmoid), plus the scores' own part."""
    l, bias, K, g = _case(scoring, far, 4)
    l = l.to(dtype)
    T, E = l.shape
    ids = torch.nonzero(bias).flatten().expand(T, K).contiguous()
    dw = torch.randn((T, K), generator=g, device="cuda")
    ds = torch.randn((T, E), generator=g, device="cuda") if with_scores else None
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring=scoring, scale=1.5)
    out = torch.full((T, E), math.nan, dtype=dtype, device="cuda")
    moe.select_backward(d, l, ids.to(torch.int32), dw, out, d_scores=ds)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    n, v, s = _ratios(l, ids, scoring), 1.5 * dw.double(), ref.scores(l, scoring)
    part = n * (v - (v * n).sum(1, keepdim=True))
    mag = n * (v.abs() + (v.abs() * n).sum(1, keepdim=True))
    want, size = (torch.zeros_like(s).scatter_add_(1, ids, a) for a in (part, mag))
    if scoring == "sigmoid":
        want = want * (1 - s)
    if with_scores:
        e = ds.double()
        dot = (e * s).sum(1, keepdim=True) if scoring == "softmax" else s * e
        want, size = want + s * (e - dot), size + s * (e.abs() + dot.abs())
    if scoring == "softmax":  # sum_j s_j ds_j over the weights' part is 0, and in f32 a rounding of its terms
        size = size + s * mag.sum(1, keepdim=True)
    # factors: a ratio (as for the weights), a score (an exponent up to the row's reach), sums over K and E in f32
    reach = float((l.double().amax(1) - l.double().amin(1)).clamp_max(110).max())
    tol = (2 * _tol(l, ids) + (4 * (reach + 16) + 64) * ref.U32) * size
    if dtype == torch.bfloat16:
        tol = tol + ref.U16 * want.abs()
    assert torch.all((out.double() - want).abs() <= tol + 1e-37), float(((out.double() - want).abs() - tol).max())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_and_single(scoring):
    """Only masked experts chosen: weights and gradient 0.  One eligible expert, however far: weight 1."""
    T, E, K = 6, 16, 3
    l = torch.full((T, E), -math.inf, device="cuda")
    for t, v in enumerate((-1e4, -120.0, 0.0, 90.0)):
        l[t, 5] = v
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring=scoring)
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.select(d, l, ids, w)
    dl = torch.full((T, E), math.nan, device="cuda")
    moe.select_backward(d, l, ids, torch.randn((T, K), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"), dl)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    assert torch.equal(w[:4, 0], torch.ones(4, device="cuda")) and torch.all(ids[:4, 0] == 5)
    assert torch.all(w[:4, 1:] == 0) and torch.all(w[4:] == 0)
    assert torch.all(dl == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("at", [0.0, 8.0, 14.0, 20.0, 40.0, 80.0])
def test_gradient_of_saturated_scores(dtype, renorm, at):
    """Sigmoid scores next to 1: the factor 1 - s = 1 / (1 + e^l) keeps its relative precision."""
    T, E, K = 50, 48, 4
    g = torch.Generator(device="cuda").manual_seed(7)
    l = (torch.randn((T, E), generator=g, device="cuda") + at).to(dtype)
    dw = torch.randn((T, K), generator=g, device="cuda")
    ds = torch.randn((T, E), generator=g, device="cuda")
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring="sigmoid", renormalize=renorm)
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.select(d, l, ids, w)
    out = torch.full((T, E), math.nan, dtype=dtype, device="cuda")
    moe.select_backward(d, l, ids, dw, out, d_scores=ds)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    ids, x = ids.long(), l.double()
    s, rest = 1 / (1 + torch.exp(-x)), 1 / (1 + torch.exp(x))
    v, size = dw.double(), dw.double().abs()
    if renorm:
        n = s.gather(1, ids) / s.gather(1, ids).sum(1, keepdim=True)
        v, size = n * (v - (v * n).sum(1, keepdim=True)), n * (size + (size * n).sum(1, keepdim=True))
    else:
        v, size = v * s.gather(1, ids), size * s.gather(1, ids)
    want = (torch.zeros_like(s).scatter_add_(1, ids, v) + s * ds.double()) * rest
    size = (torch.zeros_like(s).scatter_add_(1, ids, size) + s * ds.double().abs()) * rest
    # two scores or ratios, exponents of at most `at` + 6 each (a rounding of the argument, exp by two steps), short sums
    tol = 2 * (2 * (at + 6 + 16) + K + 8) * ref.U32 * size
    if dtype == torch.bfloat16:
        tol = tol + ref.U16 * want.abs()
    assert torch.all((out.double() - want).abs() <= tol + 1e-37), float(((out.double() - want).abs() / (tol + 1e-37)).max())
