"""Argument checks of the selection and 8-bit-float calls, on the host (no device work)."""
import copy
import ctypes

import pytest
import torch

import mixture_experts_ffn_07_b200 as moe
from mixture_experts_ffn_07_b200 import _lib

INV, UNS, WS, OK = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE, _lib.MOE_OK
A, B, C, D, E_ = (i << 28 for i in range(1, 6))  # disjoint fake addresses, never dereferenced


def _sel(**kw):
    v = dict(T=4, E=16, top_k=2, scoring=0, n_groups=1, topk_groups=1, group_score=0, renormalize=1,
             logits_dtype=_lib.MOE_F32, scale=1.0)
    v.update(kw)
    return ctypes.byref(_lib.MoeSelectDesc(*[v[n] for n, _ in _lib.MoeSelectDesc._fields_]))


BAD_DESCS = [dict(T=-1), dict(T=(1 << 20) + 1), dict(E=0), dict(E=257), dict(top_k=0), dict(top_k=17), dict(E=64, top_k=33),
             dict(scoring=2), dict(n_groups=-1), dict(n_groups=33, E=66), dict(n_groups=3), dict(n_groups=4, topk_groups=0),
             dict(n_groups=4, topk_groups=5), dict(n_groups=8, topk_groups=1, top_k=3), dict(group_score=2),
             dict(renormalize=2), dict(logits_dtype=2)]


@pytest.mark.parametrize("bad", BAD_DESCS)
def test_select_descriptors(bad):
    L = _lib.lib()
    assert L.moe_select(_sel(**bad), A, 256, None, B, C, None, None) == INV
    assert L.moe_select_backward(_sel(**bad), A, 256, B, C, None, D, None) == INV


def test_select_pointers():
    L = _lib.lib()
    assert L.moe_select(None, A, 16, None, B, C, None, None) == INV
    assert L.moe_select(_sel(), None, 16, None, B, C, None, None) == INV
    assert L.moe_select(_sel(), A + 2, 16, None, B, C, None, None) == INV      # not aligned for f32
    assert L.moe_select(_sel(), A, 15, None, B, C, None, None) == INV          # rows overlap
    assert L.moe_select(_sel(), A, 16, None, None, C, None, None) == INV
    assert L.moe_select(_sel(), A, 16, None, B, None, None, None) == INV
    assert L.moe_select(_sel(), A, 16, None, A + 64, C, None, None) == INV     # ids over logits
    assert L.moe_select(_sel(), A, 16, None, B, B + 8, None, None) == INV      # w over ids
    assert L.moe_select(_sel(), A, 16, None, B, C, A, None) == INV             # scores over logits
    assert L.moe_select_backward(_sel(), A, 16, B, C, None, A, None) == INV
    assert L.moe_select_backward(_sel(), A, 16, B, C, D, D + 4, None) == INV
    assert L.moe_select_backward(_sel(), A, 16, None, C, None, D, None) == INV
    assert L.moe_select(_sel(T=0), None, 0, None, None, None, None, None) == OK
    assert L.moe_select_backward(_sel(T=0), None, 0, None, None, None, None, None) == OK


def test_quantize_arguments():
    L = _lib.lib()
    q = L.moe_fp8_quantize
    f32, e4 = _lib.MOE_F32, _lib.MOE_E4M3
    assert q(A, f32, 4, 33, 64, e4, 0, B, C, None) == INV          # C not a multiple of 32
    assert q(A, f32, -1, 64, 64, e4, 0, B, C, None) == INV
    assert q(A, 2, 4, 64, 64, e4, 0, B, C, None) == INV            # type of x
    assert q(A, f32, 4, 64, 64, f32, 0, B, C, None) == INV         # format
    assert q(A, f32, 4, 64, 64, e4, 2, B, C, None) == INV
    assert q(A, f32, 4, 64, 63, e4, 0, B, C, None) == INV          # stride
    assert q(A, f32, 4, 64, 66, e4, 0, B, C, None) == INV          # rows not 16-byte aligned
    assert q(A + 4, f32, 4, 64, 64, e4, 0, B, C, None) == INV
    assert q(A, f32, 4, 64, 64, e4, 0, B + 8, C, None) == INV
    assert q(A, f32, 4, 64, 64, e4, 0, B, C + 2, None) == INV
    assert q(A, f32, 4, 64, 64, e4, 0, A + 512, C, None) == INV    # codes over x
    assert q(A, f32, 4, 64, 64, e4, 0, B, B + 16, None) == INV     # scales over codes
    assert q(None, f32, 0, 64, 64, e4, 0, None, None, None) == OK
    w = L.moe_fp8_quantize_weights
    assert w(A, f32, 2, 64, 48, e4, 0, B, C, None) == INV
    assert w(A, f32, 70000, 64, 64, e4, 0, B, C, None) == INV
    assert w(A, f32, 2, 64, 64, 3, 0, B, C, None) == INV
    assert w(A, f32, 2, 64, 64, e4, 0, A, C, None) == INV
    assert w(None, f32, 0, 64, 64, e4, 0, None, None, None) == OK


def test_gemm_arguments():
    L = _lib.lib()
    e4, e5, f32 = _lib.MOE_E4M3, _lib.MOE_E5M2, _lib.MOE_F32

    def g(M=8, N=64, K=64, G=1, a=A, sa=B, af=e4, b=C, sb=D, bf=e5, off=None, out=E_, od=f32):
        return L.moe_fp8_gemm(M, N, K, G, a, sa, af, b, sb, bf, off, out, od, None)

    for bad in (dict(M=-1), dict(M=(1 << 25) + 1), dict(N=48), dict(N=0), dict(K=16), dict(K=80), dict(G=0),
                dict(G=257, off=A), dict(G=2), dict(af=f32), dict(bf=2), dict(od=2), dict(a=None), dict(sa=None),
                dict(b=None), dict(sb=None), dict(out=None), dict(a=A + 8), dict(b=C + 4), dict(out=E_ + 4),
                dict(sa=B + 2), dict(sb=D + 1), dict(out=A), dict(out=C + 16), dict(out=B)):
        assert g(**bad) == INV, bad
    assert g(M=0, a=None, out=None) == OK


def test_experts_arguments():
    L = _lib.lib()
    w = _lib.MoeWeights(gate=A, up=A, down=A, gate_scale=B, up_scale=B, down_scale=B)

    def call(d, w=w, x=C, ids=D, tw=D + 4096, sg=None, out=E_, ws=6 << 28, n=1 << 40):
        return L.moe_experts(ctypes.byref(d), x, ctypes.byref(w), ids, tw, sg, out, ws, n, None)

    def desc(**kw):
        return moe.Desc(**{**dict(T=4, H=256, E=8, I=128, top_k=2, w_dtype="fp8"), **kw}).c()

    assert call(desc(H=272)) == UNS
    assert call(desc(E=300)) == INV
    assert call(desc(), w=_lib.MoeWeights(gate=A, up=A, down=A)) == INV                       # no scales
    assert call(desc(), w=_lib.MoeWeights(gate=A, up=A, down=A, gate_scale=B + 2, up_scale=B, down_scale=B)) == INV
    assert call(desc(), x=None) == INV
    assert call(desc(), ids=None) == INV
    assert call(desc(), tw=None) == INV
    assert call(desc(), out=C) == INV
    assert call(desc(), out=C + 256) == INV
    assert call(desc(), n=64) == WS
    assert call(desc(), ws=None) == WS
    assert call(desc(shared_I=64)) == INV                                                     # no shared weights
    sh = _lib.MoeWeights(gate=A, up=A, down=A, gate_scale=B, up_scale=B, down_scale=B, sh_gate=A, sh_up=A, sh_down=A,
                         sh_gate_scale=B, sh_up_scale=B, sh_down_scale=B)
    assert call(desc(shared_I=64, has_shared_gate=True), w=sh) == INV                         # no gate values
    assert call(desc(T=0), x=None, ids=None, tw=None, out=None, ws=None, n=0) == OK
    # rows beyond the streaming path's limit are no matter for 8-bit weights
    assert call(desc(H=32768), n=64) == WS


def test_workspace_follows_the_format():
    d = dict(T=512, H=2048, E=64, I=1024, top_k=8)
    n = moe.workspace_bytes(moe.Desc(w_dtype="fp8", **d))
    P = 512 * 8
    assert n >= P * 2048 * 2 + P * 2048 + P * 1024 + 512 * 2048
    assert n < moe.workspace_bytes(moe.Desc(**d))
    assert moe.workspace_bytes(moe.Desc(w_dtype="fp8", act_dtype="f32", **d)) > n


def test_tensor_checks():
    """The binding refuses what the C call cannot see: types, shapes, strides, devices."""
    f = torch.zeros
    d = moe.SelectDesc(T=4, E=8, top_k=2)
    with pytest.raises(ValueError):
        moe.select(d, f(4, 8), f(4, 2, dtype=torch.int32), f(4, 2))           # not on a GPU
    with pytest.raises(ValueError):
        moe.select(d, f(4, 8, dtype=torch.float16), f(4, 2, dtype=torch.int32), f(4, 2))
    with pytest.raises(ValueError):
        moe.select(d, f(4, 9), f(4, 2, dtype=torch.int32), f(4, 2))
    with pytest.raises(ValueError):
        moe.fp8_quantize(f(4, 64), f(4, 64), f(1, 4))
    with pytest.raises(ValueError):
        moe.fp8_gemm(f(4, 64), f(1, 4), f(64, 64), f(1, 1), f(4, 64))
    with pytest.raises(ValueError):
        moe.experts(moe.Desc(T=4, H=64, E=4, I=64, top_k=2, w_dtype="fp8"), f(4, 64), moe.Weights(), None, None, None, None)


def test_select_desc_follows_its_fields():
    """The struct handed to the library is made again after a field is set, and copies have their own."""
    d = moe.SelectDesc(T=4, E=8, top_k=2)
    assert d.ref(0) is d.ref(0) and d.ref(0)._obj.E == 8 and d.ref(1)._obj.logits_dtype == 1
    other = copy.deepcopy(d)
    assert other == d
    d.E, d.scoring = 16, "sigmoid"
    assert d.ref(0)._obj.E == 16 and d.ref(0)._obj.scoring == d.c(0).scoring and other.ref(0)._obj.E == 8


def test_every_pointer_is_aligned_and_apart():
    L = _lib.lib()
    e4, f32 = _lib.MOE_E4M3, _lib.MOE_F32
    assert L.moe_select(_sel(), A, 16, B + 1, C, D, None, None) == INV         # bias
    assert L.moe_select(_sel(), A, 16, C + 16, C, D, None, None) == INV        # bias over ids
    assert L.moe_select(_sel(), A, 16, None, C + 2, D, None, None) == INV
    assert L.moe_select(_sel(), A, 16, None, C, D + 2, None, None) == INV
    assert L.moe_select(_sel(), A, 16, None, C, D, B + 2, None) == INV
    assert L.moe_select_backward(_sel(), A, 16, B + 2, C, None, D, None) == INV
    assert L.moe_select_backward(_sel(), A, 16, B, C + 2, None, D, None) == INV
    assert L.moe_select_backward(_sel(), A, 16, B, C, E_ + 2, D, None) == INV
    F = 7 << 28
    assert L.moe_fp8_gemm(4, 64, 64, 2, A, B, e4, C, D, e4, F + 2, E_, f32, None) == INV
    assert L.moe_fp8_gemm(4, 64, 64, 2, A, B, e4, C, D, e4, E_ + 16, E_, f32, None) == INV  # offsets inside the output
