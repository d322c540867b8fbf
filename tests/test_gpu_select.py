"""moe_select and moe_select_backward against their 64-bit definition."""
import math

import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from tests import _fp8ref as ref

pytestmark = pytest.mark.gpu


def _logits(T, E, dtype, pad, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, E + pad), generator=g, device="cuda") * 2).to(dtype)[:, :E], g


def _run(l, K, bias=None, scores=False, **kw):
    T, E = l.shape
    d = moe.SelectDesc(T=T, E=E, top_k=K, **kw)
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    s = torch.full((T, E), float("nan"), device="cuda") if scores else None
    moe.select(d, l, ids, w, bias=bias, scores=s)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK
    return ids, w, s


def _check(l, K, bias=None, **kw):
    """ids equal to the 64-bit selection; weights and scores within an f32 evaluation: the score's exponent is off by
    a rounding of its argument and two steps of exp, a sum over E <= 256 terms by 8 steps in pairs."""
    ids, w, s = _run(l, K, bias=bias, scores=True, **kw)
    rid, rw, rs = ref.select(l, K, kw.get("scoring", "softmax"), bias, kw.get("n_groups", 1), kw.get("topk_groups", 1),
                             kw.get("group_score", "max"), kw.get("renormalize", True), kw.get("scale", 1.0))
    assert torch.equal(ids.long(), rid)
    finite = l.float()[torch.isfinite(l.float())]
    reach = float(finite.max() - finite.min()) if finite.numel() else 0.0
    tol = 2 * ref.U32 * (reach + 16)
    assert torch.all((w.double() - rw).abs() <= 2 * tol * rw.abs() + 1e-37)
    assert torch.all((s.double() - rs).abs() <= tol * rs.abs() + 1e-37)
    return ids, w, s


@pytest.mark.parametrize("T,E,K,dtype,pad", [
    (1, 128, 8, torch.float32, 0), (1, 1, 1, torch.float32, 0), (3, 7, 7, torch.float32, 5),
    (65, 33, 4, torch.bfloat16, 1), (257, 256, 32, torch.float32, 0), (130, 60, 6, torch.bfloat16, 0)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_plain(T, E, K, dtype, pad, scoring, biased):
    l, g = _logits(T, E, dtype, pad, T + E)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if biased else None
    _check(l, K, bias, scoring=scoring)
    _check(l, K, bias, scoring=scoring, renormalize=False, scale=2.5)


@pytest.mark.parametrize("T,E,K,groups,kept", [(97, 256, 8, 8, 4), (40, 60, 3, 15, 5), (33, 24, 24, 4, 4),
                                               (50, 32, 4, 32, 7), (21, 96, 6, 2, 1)])
@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(T, E, K, groups, kept, score, scoring, biased):
    l, g = _logits(T, E, torch.float32, 0, 3 * T + groups)
    bias = torch.randn(E, generator=g, device="cuda") * 0.2 if biased else None
    _check(l, K, bias, scoring=scoring, n_groups=groups, topk_groups=kept, group_score=score, scale=1.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_ties_take_the_lower_expert(scoring, groups, kept):
    T, E, K = 64, 64, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    l = torch.randint(0, 3, (T, E), generator=g, device="cuda").float()
    l[0] = 0
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() / 4
    for b in (None, bias, torch.zeros(E, device="cuda")):
        for score in ("max", "top2"):
            _check(l, K, b, scoring=scoring, n_groups=groups, topk_groups=kept, group_score=score)


def test_border_below_f32():
    """Scores that f32 cannot tell apart: the larger one in 64 bits is chosen, whatever its index."""
    E, T = 64, 512
    g = torch.Generator(device="cuda").manual_seed(9)
    base = torch.randn(T, 1, generator=g, device="cuda").abs() + 9.0  # sigmoid within 1e-4 of 1: steps of 2^-24 hide l
    l = base + torch.randint(0, 4, (T, E), generator=g, device="cuda") * 2.0 ** -18
    bias = torch.full((E,), 0.25, device="cuda")
    _check(l, 6, bias, scoring="sigmoid")
    _check(l, 6, bias, scoring="sigmoid", n_groups=8, topk_groups=3, group_score="top2")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept,score", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
def test_masked_experts(scoring, biased, groups, kept, score):
    """-inf logits: score 0, chosen last; a row of them alone has weights 0 and ids in range."""
    T, E, K = 70, 32, 6
    l, g = _logits(T, E, torch.float32, 0, 11)
    l = l.clone()
    l[torch.rand((T, E), generator=g, device="cuda") < 0.7] = -math.inf
    l[3] = -math.inf
    l[4] = -math.inf
    l[4, 17] = 0.5
    bias = torch.randn(E, generator=g, device="cuda") - 1.0 if biased else None
    ids, w, s = _check(l, K, bias, scoring=scoring, n_groups=groups, topk_groups=kept, group_score=score)
    assert torch.all(w[3] == 0) and torch.all(s[3] == 0)
    assert ids[4, 0] == 17 and w[4, 0] == 1 and torch.all(w[4, 1:] == 0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_nan_and_inf_keep_ids_in_range(scoring):
    T, E, K = 40, 40, 5
    l, g = _logits(T, E, torch.float32, 0, 13)
    l = l.clone()
    l[5, 3] = math.nan
    l[6] = math.nan
    l[7, 2] = math.inf
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    for b in (None, bias):
        ids, w, _ = _run(l, K, bias=b, scoring=scoring)
        assert int(ids.min()) >= 0 and int(ids.max()) < E
        assert all(len(set(r)) == K for r in ids.tolist())
        keep = [t for t in range(T) if t not in (5, 6, 7)]
        rid, rw, _ = ref.select(l[keep], K, scoring, b)
        assert torch.equal(ids[keep].long(), rid)
        assert torch.isfinite(w[keep]).all()


@pytest.mark.parametrize("T,E,K,dtype,pad", [(1, 128, 8, torch.float32, 0), (37, 160, 6, torch.bfloat16, 32),
                                             (200, 256, 32, torch.float32, 1), (5, 3, 1, torch.float32, 0)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_scores", [True, False])
def test_backward(T, E, K, dtype, pad, scoring, renorm, with_scores):
    l, g = _logits(T, E, dtype, pad, 17 + T)
    ids = ref.select(l, K, scoring)[0]
    dw = torch.randn((T, K), generator=g, device="cuda")
    ds = torch.randn((T, E), generator=g, device="cuda") if with_scores else None
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring=scoring, renormalize=renorm, scale=1.5)
    out = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    moe.select_backward(d, l, ids.to(torch.int32), dw, out, d_scores=ds)
    again = torch.empty_like(out)
    moe.select_backward(d, l, ids.to(torch.int32), dw, again, d_scores=ds)
    torch.cuda.synchronize()
    assert moe.last_device_status() == moe.MOE_OK and torch.equal(out, again)
    want, mag = ref.select_backward(l, ids, dw, ds, scoring, renorm, 1.5)
    reach = float(l.float().max() - l.float().min())
    # every term is a product of at most four factors, each an f32 score off by 2 (reach + 16) half steps, and the
    # sums over K <= 32 and E <= 256 add 32 half steps
    tol = (4 * 2 * (reach + 16) + 64) * ref.U32 * mag
    if dtype == torch.bfloat16:
        tol = tol + ref.U16 * want.abs()
    assert torch.all((out.double() - want).abs() <= tol + 1e-37)


def test_backward_is_the_derivative():
    """The formula against central differences of the 64-bit weights and scores, the selection held."""
    torch.manual_seed(3)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            l = torch.randn(4, 12, dtype=torch.float64)
            ids = ref.select(l, 3, scoring)[0]
            dw, ds = torch.randn(4, 3).double(), torch.randn(4, 12).double()

            def loss(x):
                s = ref.scores(x, scoring)
                w = s.gather(1, ids)
                if renorm:
                    w = w / w.sum(1, keepdim=True)
                return ((1.5 * w * dw).sum() + (s * ds).sum()).item()

            want, _ = ref.select_backward(l, ids, dw, ds, scoring, renorm, 1.5)
            eps = 1e-5
            for t in range(4):
                for e in range(12):
                    up, dn = l.clone(), l.clone()
                    up[t, e] += eps
                    dn[t, e] -= eps
                    assert abs((loss(up) - loss(dn)) / (2 * eps) - want[t, e].item()) < 1e-8


def test_backward_bad_and_repeated_ids():
    T, E, K = 6, 16, 4
    l, g = _logits(T, E, torch.float32, 0, 23)
    ids = torch.tensor([[0, 1, 2, 3]] * T, device="cuda", dtype=torch.int32)
    ids[2] = torch.tensor([5, 5, 5, 9])
    dw = torch.randn((T, K), generator=g, device="cuda")
    d = moe.SelectDesc(T=T, E=E, top_k=K, renormalize=False)
    out = torch.empty((T, E), device="cuda")
    moe.select_backward(d, l, ids, dw, out)
    assert moe.last_device_status() == moe.MOE_OK
    want, mag = ref.select_backward(l, ids.long(), dw, None, "softmax", False, 1.0)
    assert torch.all((out.double() - want).abs() <= 600 * ref.U32 * mag)
    bad = ids.clone()
    bad[1, 0], bad[3, 2] = -1, E
    moe.select_backward(d, l, bad, dw, out)
    assert moe.last_device_status() == moe.MOE_ERR_DEVICE_INDEX
    dz = dw.clone()
    dz[1, 0], dz[3, 2] = 0, 0
    want, mag = ref.select_backward(l, bad.clamp(0, E - 1).long(), dz, None, "softmax", False, 1.0)
    assert torch.all((out.double() - want).abs() <= 600 * ref.U32 * mag)


def test_empty_batch_and_other_stream():
    d = moe.SelectDesc(T=0, E=16, top_k=2)
    e = torch.empty
    moe.select(d, e((0, 16), device="cuda"), e((0, 2), dtype=torch.int32, device="cuda"), e((0, 2), device="cuda"))
    l, _ = _logits(300, 64, torch.float32, 0, 29)
    a = _run(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = _run(l, 8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_far_rows():
    """Row offsets past 2^31 elements."""
    T, E, ld = 5, 32, (1 << 29) + 8
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    buf = torch.empty(4 * ld + E + 8, dtype=torch.bfloat16, device="cuda")
    l = buf.as_strided((T, E), (ld, 1))
    l.copy_(torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    _check(l, 4)


def test_forward_and_backward_in_a_graph():
    T, E, K = 70, 48, 4
    d = moe.SelectDesc(T=T, E=E, top_k=K, scoring="sigmoid", renormalize=True)
    l, dw = torch.randn((T, E), device="cuda"), torch.randn((T, K), device="cuda")
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    dl = torch.empty((T, E), device="cuda")

    def run():
        moe.select(d, l, ids, w)
        moe.select_backward(d, l, ids, dw, dl)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        g = torch.Generator(device="cuda").manual_seed(i)
        l.copy_(torch.randn((T, E), generator=g, device="cuda"))
        dw.copy_(torch.randn((T, K), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (ids, w, dl)]
        run()
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, dl)))
    assert moe.last_device_status() == moe.MOE_OK


@pytest.mark.parametrize("T,E,K,dtype,pad,groups,kept", [
    (4096, 256, 20, torch.float32, 0, 1, 1), (2048, 256, 32, torch.bfloat16, 0, 8, 3), (513, 256, 8, torch.bfloat16, 8, 4, 2),
    (300, 255, 12, torch.float32, 0, 15, 4), (300, 224, 7, torch.float32, 3, 7, 4), (64, 96, 32, torch.float32, 0, 16, 9)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_many_candidates(T, E, K, dtype, pad, groups, kept, scoring, biased):
    """More experts in question than a warp has lanes, rows that are and are not 16-byte aligned, groups of lanes and of
    odd sizes, and enough tokens that some of their keys are too near to each other for f32."""
    l, g = _logits(T, E, dtype, pad, T + 5 * E)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if biased else None
    _check(l, K, bias, scoring=scoring, n_groups=groups, topk_groups=kept, group_score="top2")
    _check(l, K, bias, scoring=scoring, n_groups=groups, topk_groups=kept, renormalize=False)


def test_bias_extremes():
    """Biases that outweigh the scores, that differ by less than f32 resolves beside them, and a logit's own copies."""
    T, E, K = 50, 64, 6
    l, g = _logits(T, E, torch.float32, 0, 21)
    l = l.clone()
    l[:, 1::2] = l[:, ::2]
    for bias in (torch.randn(E, generator=g, device="cuda") * 1e4,
                 1024.0 + torch.randint(0, 3, (E,), generator=g, device="cuda").float() * 2.0 ** -13,
                 torch.zeros(E, device="cuda")):
        for scoring in ("softmax", "sigmoid"):
            _check(l, K, bias, scoring=scoring)
            _check(l, K, bias, scoring=scoring, n_groups=8, topk_groups=4, group_score="top2")
