"""The sum over a token's experts of 8-bit floats: bf16 outputs are rounded once, from the sum of rows that are held more
exactly than bf16 (the rows that the experts leave for the combine)."""
import math

import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref
from tests.test_gpu_fp8 import _experts, _fp8_weights, _gen, _ok

pytestmark = pytest.mark.gpu
F16 = 2.0 ** -11  # half a step of f16, relative: torch.finfo(torch.float16).eps / 2


def _sum(x, ids, tw, sg, t, act):
    """The weighted sum in 64 bits before the output's rounding, and how far an evaluation may be off it: the experts'
    own bounds, and f32 products and additions."""
    T, K = ids.shape
    H = x.shape[1]
    q, s = ref.quantize(x.double(), "e4m3", False)
    X = q * ref.spread(s, T, H, 1)
    out, tol, mag = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(3))
    for e in torch.unique(ids).tolist():
        for k in range(K):
            rows = torch.nonzero(ids[:, k] == e).flatten()
            if rows.numel():
                y, b = ref.ffn(X[rows], *[ref.dequantize_weights(t[n][e], t[n + "_scale"][e]) for n in ("gate", "up", "down")], act)
                w = tw[rows, k, None].double()
                out[rows] += w * y
                tol[rows] += w.abs() * b
                mag[rows] += w.abs() * y.abs()
    if sg is not None:
        y, b = ref.ffn(X, *[ref.dequantize_weights(t["sh_" + n], t["sh_" + n + "_scale"]) for n in ("gate", "up", "down")], act)
        g = sg.double()[:, None]
        out += g * y
        tol += g.abs() * b
        mag += (g * y).abs()
    return out, tol + (K + 2) * ref.U32 * mag


@pytest.mark.parametrize("T,H,E,I,K,Is", [(1, 64, 16, 64, 8, 0), (1, 96, 8, 32, 8, 64), (9, 64, 16, 64, 8, 32),
                                          (70, 96, 16, 64, 8, 0), (150, 1056, 64, 32, 2, 0)])
def test_one_rounding(T, H, E, I, K, Is):
    g = _gen(T + H + K)
    t = _fp8_weights(E, H, I, Is, T + I)
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", shared_I=Is, has_shared_gate=Is > 0)
    seen = 0
    for _ in range(max(1, 64 // T)):  # (a code of h that may go either way leaves nothing to judge in its token)
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
        tw = torch.randn((T, K), generator=g, device="cuda")
        sg = torch.rand(T, generator=g, device="cuda") if Is else None
        out = _experts(d, x, t, ids, tw, sg)
        _ok()
        want, tol = _sum(x, ids, tw, sg, t, "silu")
        # half a step of bf16 next to `want`: its binade's step is 2^(e - 7) for 2^e <= |want| < 2^(e + 1)
        half = torch.exp2(torch.frexp(want).exponent.double() - 1 - 8)
        judged = tol < half / 2
        seen += int(judged.sum())
        err = (out.double() - want).abs()
        # the rounding of a value that is `tol` off: half a step of its own binade, which may be the next one
        bound = torch.exp2(torch.frexp(want.abs() + tol).exponent.double() - 1 - 8) + tol
        assert torch.all(err[judged] <= bound[judged]), float((err / bound)[judged].max())
    assert seen > 20


@pytest.mark.parametrize("T,H,E,I,K,Is,slot", [
    (1, 512, 16, 256, 8, 0, 0.0), (16, 1024, 16, 64, 8, 64, 0.0), (300, 64, 64, 96, 6, 32, 0.0), (300, 512, 64, 64, 8, 0, F16),
    (900, 160, 64, 64, 8, 64, F16), (700, 1056, 40, 256, 20, 0, F16)])
def test_bf16_layer_is_the_rounded_f32_layer(T, H, E, I, K, Is, slot):
    """The same inputs in an f32 layer take the same codes and products: the bf16 output is that one's, rounded once, and
    before it at most `slot` off for each slot row."""
    g = _gen(T + H)
    t = _fp8_weights(E, H, I, Is, T + I)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.randn((T, K), generator=g, device="cuda")
    sg = torch.rand(T, generator=g, device="cuda") if Is else None
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", shared_I=Is, has_shared_gate=Is > 0)
    d32 = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8", act_dtype="f32", shared_I=Is, has_shared_gate=Is > 0)
    out = _experts(d, x, t, ids, tw, sg)
    exact = _experts(d32, x.float(), t, ids, tw, sg)
    _ok()
    if slot == 0.0:
        assert torch.equal(out, exact.to(torch.bfloat16))
        return
    counts, offs = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp, pp = (torch.empty(T * K, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.permute(d32, ids, counts, offs, sp, pp)
    y = torch.full((T * K, H), float("nan"), device="cuda")
    ws = torch.empty(moe.workspace_bytes(d32), dtype=torch.uint8, device="cuda")
    moe.expert_ffn(d32, x.float(), moe.Weights(**t), offs, sp, torch.ones_like(tw), y, ws)
    _ok()
    mag = (y.view(T, K, H).double().abs() * tw.double().abs()[..., None]).sum(1)
    off = slot * mag + (K + 2) * 2 * ref.U32 * (mag + exact.double().abs())  # slot rows; two f32 sums of K + 1 terms
    half = torch.exp2(torch.frexp(exact.double().abs() + off).exponent.double() - 1 - 8)  # half a step of bf16
    err = (out.double() - exact.double()).abs()
    assert torch.all(err <= half + off), float((err / (half + off)).max())
    # where no border between two bf16 numbers lies within `off`, the two round alike: elsewhere the share off / step, at most
    share = float((off / half / 2).clamp_max(1).sum())
    assert int((out != exact.to(torch.bfloat16)).sum()) <= share + 4 * math.sqrt(share)


@pytest.mark.parametrize("T,H,E,I,K", [(40, 64, 4, 32, 2), (900, 160, 64, 64, 8)])  # few rows a group, many
def test_rows_of_any_size(T, H, E, I, K):
    """Slot values near the ends of f32's range: finite sums stay finite, infinite and NaN rows stay in their token."""
    g = _gen(5)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    t = _fp8_weights(E, H, I, 0, 6)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.to(torch.int32)
    tw = torch.rand((T, K), generator=g, device="cuda")
    d = moe.Desc(T=T, H=H, E=E, I=I, top_k=K, w_dtype="fp8")
    base = _experts(d, x, t, ids, tw)
    for power in (-90, 60, 110):  # the down projection's scales times a power of two: the same output times that power
        f = 2.0 ** power
        out = _experts(d, x, {**t, "down_scale": t["down_scale"] * f}, ids, tw)
        _ok()
        assert torch.equal(out.double() / f, base.double())
    for bad in (math.inf, math.nan):
        s = t["down_scale"].clone()
        s[2] = bad
        out = _experts(d, x, {**t, "down_scale": s}, ids, tw)
        _ok()
        hit = (ids == 2).any(1)
        assert not torch.isfinite(out[hit].float()).any() and torch.equal(out[~hit], base[~hit])
