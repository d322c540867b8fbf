"""MoE FFN layer for NVIDIA B200 -- Python binding of libmoe.so (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (any object with ``data_ptr()``);
streams default to torch's current stream.  PyTorch provides device memory and
streams; it computes nothing here.

    desc = Desc(T=512, H=2048, E=64, I=1024, top_k=8)
    w = Weights(router=..., gate=..., up=..., down=...)
    ws = torch.empty(workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    layer(desc, x, w, out, ws)
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import _lib
from ._lib import (MOE_ACT_GELU_TANH, MOE_ACT_SILU, MOE_BF16, MOE_ERR_CUDA, MOE_ERR_DEVICE_INDEX,  # noqa: F401
                   MOE_E4M3, MOE_E5M2, MOE_ERR_INVALID_ARG, MOE_ERR_TIMEOUT, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_F32, MOE_FP8, MOE_OK,
                   MOE_Q4_K, MOE_Q4_K_Q6_K, MOE_Q8_0, MoeError, check, status_string)

DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "q8_0": MOE_Q8_0, "q4_k": MOE_Q4_K, "q4_k_q6_k": MOE_Q4_K_Q6_K,
          "fp8": MOE_FP8}
ACTS = {"silu": MOE_ACT_SILU, "gelu_tanh": MOE_ACT_GELU_TANH}
GATINGS = {"softmax": 0, "sigmoid": 1}  # moe_gating
GROUP_SCORES = {"max": 0, "top2": 1}  # moe_group_score


@dataclass
class Desc:
    T: int
    H: int
    E: int
    I: int
    top_k: int
    act: str = "silu"
    renormalize: bool = True
    act_dtype: str = "bf16"
    w_dtype: str = "bf16"
    router_dtype: str = "bf16"
    has_router_bias: bool = False
    shared_I: int = 0
    has_shared_gate: bool = False
    gating: str = "softmax"
    n_groups: int = 0
    topk_groups: int = 0

    def c(self) -> _lib.MoeDesc:
        return _lib.MoeDesc(self.T, self.H, self.E, self.I, self.top_k, ACTS[self.act], int(self.renormalize),
                            DTYPES[self.act_dtype], DTYPES[self.w_dtype], DTYPES[self.router_dtype],
                            int(self.has_router_bias), self.shared_I, int(self.has_shared_gate),
                            GATINGS[self.gating], self.n_groups, self.topk_groups)

    @property
    def P(self) -> int:
        return self.T * self.top_k


@dataclass
class SelectDesc:
    """moe_select_desc: how `select` chooses and weights the experts of T tokens from logits [T, E]."""
    T: int
    E: int
    top_k: int
    scoring: str = "softmax"
    n_groups: int = 1
    topk_groups: int = 1
    group_score: str = "max"
    renormalize: bool = True
    scale: float = 1.0

    def __setattr__(self, name, value):
        self.__dict__.pop("_refs", None)
        self.__dict__[name] = value

    def __getstate__(self):
        return {n: v for n, v in self.__dict__.items() if n != "_refs"}

    def c(self, logits_dtype: int) -> _lib.MoeSelectDesc:
        return _lib.MoeSelectDesc(self.T, self.E, self.top_k, GATINGS[self.scoring], self.n_groups, self.topk_groups,
                                  GROUP_SCORES[self.group_score], int(self.renormalize), logits_dtype, self.scale)

    def ref(self, logits_dtype: int):
        """The C struct by reference, made once until a field is set (small calls take a few microseconds in all)."""
        refs = self.__dict__.setdefault("_refs", {})
        if logits_dtype not in refs:
            refs[logits_dtype] = ctypes.byref(self.c(logits_dtype))
        return refs[logits_dtype]


@dataclass
class Weights:
    """Device tensors, out x in.  For Q8_0 the projections are int8 and *_scale hold fp16 block scales; for fp8
    they are float8_e4m3fn and *_scale hold one f32 scale per 128 x 128 block."""
    router: object = None
    router_bias: object = None
    gate: object = None
    up: object = None
    down: object = None
    sh_gate: object = None
    sh_up: object = None
    sh_down: object = None
    sh_gate_w: object = None
    gate_scale: object = None
    up_scale: object = None
    down_scale: object = None
    sh_gate_scale: object = None
    sh_up_scale: object = None
    sh_down_scale: object = None

    def c(self) -> _lib.MoeWeights:
        return _lib.MoeWeights(*[None if t is None else t.data_ptr() for t in (
            self.router, self.router_bias, self.gate, self.up, self.down, self.sh_gate, self.sh_up, self.sh_down,
            self.sh_gate_w, self.gate_scale, self.up_scale, self.down_scale, self.sh_gate_scale, self.sh_up_scale,
            self.sh_down_scale)])


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def version() -> str:
    return _lib.lib().moe_version().decode()


def workspace_bytes(desc: Desc) -> int:
    d = desc.c()
    return _lib.lib().moe_workspace_bytes(ctypes.byref(d))


def workspace_regions(desc: Desc) -> dict:
    """moe_workspace_regions: byte offsets of the routing results moe_layer leaves in the workspace."""
    d, r = desc.c(), _lib.MoeWsRegions()
    check(_lib.lib().moe_workspace_regions(ctypes.byref(d), ctypes.byref(r)), "moe_workspace_regions")
    return {n: getattr(r, n) for n, _ in _lib.MoeWsRegions._fields_}


def route(desc, x, w, logits, topk_ids, topk_w, shared_gate=None, ws=None, stream=None):
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_route(ctypes.byref(d), _ptr(x), ctypes.byref(cw), _ptr(logits), _ptr(topk_ids),
                               _ptr(topk_w), _ptr(shared_gate), _ptr(ws), _nbytes(ws), _stream(stream)), "moe_route")


def permute(desc, topk_ids, counts, offsets, sorted_pairs, pair_pos, stream=None):
    d = desc.c()
    check(_lib.lib().moe_permute(ctypes.byref(d), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(sorted_pairs),
                                 _ptr(pair_pos), _stream(stream)), "moe_permute")


def expert_ffn(desc, x, w, offsets, sorted_pairs, topk_w, y_slots, ws, stream=None):
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_expert_ffn(ctypes.byref(d), _ptr(x), ctypes.byref(cw), _ptr(offsets), _ptr(sorted_pairs),
                                    _ptr(topk_w), _ptr(y_slots), _ptr(ws), _nbytes(ws), _stream(stream)),
          "moe_expert_ffn")


def combine(desc, y_slots, x, w, shared_gate, out, ws=None, stream=None):
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_combine(ctypes.byref(d), _ptr(y_slots), _ptr(x), ctypes.byref(cw), _ptr(shared_gate),
                                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)), "moe_combine")


def layer(desc, x, w, out, ws, stream=None):
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_layer(ctypes.byref(d), _ptr(x), ctypes.byref(cw), _ptr(out), _ptr(ws), _nbytes(ws),
                               _stream(stream)), "moe_layer")


def layer_noalloc(desc, x, w, out, stream=None):
    """moe_layer with the library's static 32 MiB device scratch: for callers that cannot allocate.

    Calls that may overlap on the GPU share that scratch and race; the first call on a device
    looks up its address and should come before any stream capture."""
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_layer_noalloc(ctypes.byref(d), _ptr(x), ctypes.byref(cw), _ptr(out), _stream(stream)),
          "moe_layer_noalloc")


def layer_host(desc, x_host, w, out_host, x_dev, out_dev, ws, stream=None):
    """moe_layer with host x/out (pinned torch CPU tensors); copies are enqueued on `stream`."""
    d, cw = desc.c(), w.c()
    check(_lib.lib().moe_layer_host(ctypes.byref(d), _ptr(x_host), ctypes.byref(cw), _ptr(out_host), _ptr(x_dev),
                                    _ptr(out_dev), _ptr(ws), _nbytes(ws), _stream(stream)), "moe_layer_host")


def q8_0_split(blocks, rows, cols, q, scales, stream=None):
    check(_lib.lib().moe_q8_0_split(_ptr(blocks), rows, cols, _ptr(q), _ptr(scales), _stream(stream)),
          "moe_q8_0_split")


def combine_backward(y, w, d_out, d_y, d_w, stream=None):
    """moe_combine_backward: y [T,K,H] (unweighted expert outputs), w [T,K], d_out [T,H] -> d_y, d_w (all f32)."""
    T, K, H = y.shape
    check(_lib.lib().moe_combine_backward(T, K, H, _ptr(y), _ptr(w), _ptr(d_out), _ptr(d_y), _ptr(d_w),
                                          _stream(stream)), "moe_combine_backward")


def act_up_backward(act, gate_up, d_h, d_gate_up, stream=None):
    """moe_act_up_backward: gate_up [P,2I] ([gate | up]), d_h [P,I] -> d_gate_up [P,2I] (all f32)."""
    P, I = d_h.shape
    check(_lib.lib().moe_act_up_backward(P, I, ACTS[act] if isinstance(act, str) else act, _ptr(gate_up), _ptr(d_h),
                                         _ptr(d_gate_up), _stream(stream)), "moe_act_up_backward")


def q6_k_split(blocks, rows, cols, q, scales, stream=None):
    """moe_q6_k_split: GGML Q6_K blocks -> 16-byte aligned quant and scale planes."""
    check(_lib.lib().moe_q6_k_split(_ptr(blocks), rows, cols, _ptr(q), _ptr(scales), _stream(stream)),
          "moe_q6_k_split")


def q6_k_srow_bytes(cols: int) -> int:
    """Bytes of one scale row of the Q6_K split form (include/moe.h)."""
    return (cols // 256 * 18 + 15) // 16 * 16


class _Types:
    """moe_dtype of each torch dtype that an argument of the calls below may have (made at the first call, so that
    importing the package does not import torch)."""
    i32 = f32 = act = bf16 = fp8 = e4m3 = torch = current_device = raw_stream = None

    @classmethod
    def ready(cls):
        if cls.i32 is None:
            import torch
            cls.torch = torch
            cls.current_device = torch._C._cuda_getDevice
            # the raw handle: building a torch.cuda.Stream to read it from takes as long as the launch
            cls.raw_stream = torch._C._cuda_getCurrentRawStream
            cls.i32 = {torch.int32: 0}
            cls.f32 = {torch.float32: MOE_F32}
            cls.act = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
            cls.bf16 = {torch.bfloat16: MOE_BF16}
            cls.e4m3 = {torch.float8_e4m3fn: MOE_E4M3}
            cls.fp8 = {torch.float8_e4m3fn: MOE_E4M3, torch.float8_e5m2: MOE_E5M2}
        return cls


def _arg(name, t, types, shape, device=None, dense=True):
    """Checks a tensor argument and returns the code of its type.  `device`: the index it has to be on."""
    code = types.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: {t.dtype}, expected one of {list(types)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    dev = t.get_device()
    if dev < 0 or (device is not None and dev != device):
        raise ValueError(f"{name} is on {t.device}" + ("" if device is None else f", not on cuda:{device}"))
    return code


def _row_stride(name, t, cols):
    """Elements between the rows of a tensor [rows, cols] whose rows are dense."""
    if t.is_contiguous():
        return cols or 1
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row are not consecutive")
    return t.stride(0) if t.shape[0] > 1 else cols


def _call(device, stream, name, fn, *args):
    """One library call with `device` current, on `stream` (default: that device's current stream)."""
    raw = _Types.raw_stream(device) if stream is None else _stream(stream)
    if _Types.current_device() == device:
        code = fn(*args, raw)
    else:
        with _Types.torch.cuda.device(device):
            code = fn(*args, raw)
    if code != MOE_OK:
        raise MoeError(code, name)


def select(desc, logits, ids, w, bias=None, scores=None, stream=None):
    """moe_select: logits [T,E] (f32 or bf16, rows may be padded) -> ids [T,K] int32, w [T,K] f32
    (, scores [T,E] f32).  bias [E] f32 moves the choice, not the weights."""
    ty = _Types.ready()
    T, E, K = desc.T, desc.E, desc.top_k
    code = _arg("logits", logits, ty.act, (T, E), dense=False)
    ld, dev = _row_stride("logits", logits, E), logits.get_device()
    _arg("ids", ids, ty.i32, (T, K), dev)
    _arg("w", w, ty.f32, (T, K), dev)
    if bias is not None:
        _arg("bias", bias, ty.f32, (E,), dev)
    if scores is not None:
        _arg("scores", scores, ty.f32, (T, E), dev)
    _call(dev, stream, "moe_select", _lib.lib().moe_select, desc.ref(code), logits.data_ptr(), ld, _ptr(bias),
          ids.data_ptr(), w.data_ptr(), _ptr(scores))


def select_backward(desc, logits, ids, d_w, d_logits, d_scores=None, stream=None):
    """moe_select_backward: d_w [T,K] f32 (, d_scores [T,E] f32) -> d_logits [T,E] of the logits' type."""
    ty = _Types.ready()
    T, E, K = desc.T, desc.E, desc.top_k
    code = _arg("logits", logits, ty.act, (T, E), dense=False)
    ld, dev = _row_stride("logits", logits, E), logits.get_device()
    _arg("ids", ids, ty.i32, (T, K), dev)
    _arg("d_w", d_w, ty.f32, (T, K), dev)
    if d_scores is not None:
        _arg("d_scores", d_scores, ty.f32, (T, E), dev)
    if _arg("d_logits", d_logits, ty.act, (T, E), dev) != code:
        raise ValueError(f"d_logits: {d_logits.dtype}, expected {logits.dtype}")
    _call(dev, stream, "moe_select_backward", _lib.lib().moe_select_backward, desc.ref(code), logits.data_ptr(),
          ld, ids.data_ptr(), d_w.data_ptr(), _ptr(d_scores), d_logits.data_ptr())


def fp8_quantize(x, q, scales, pow2=False, stream=None):
    """moe_fp8_quantize: x [R,C] (f32 or bf16, rows may be padded) -> q [R,C] (float8_e4m3fn or float8_e5m2),
    scales [ceil(C/128), R] f32."""
    ty = _Types.ready()
    R, C = x.shape
    code = _arg("x", x, ty.act, (R, C), dense=False)
    ld, dev = _row_stride("x", x, C), x.get_device()
    fmt = _arg("q", q, ty.fp8, (R, C), dev)
    _arg("scales", scales, ty.f32, ((C + 127) // 128, R), dev)
    _call(dev, stream, "moe_fp8_quantize", _lib.lib().moe_fp8_quantize, x.data_ptr(), code, R, C, ld, fmt, int(pow2),
          q.data_ptr(), scales.data_ptr())


def fp8_quantize_weights(w, q, scales, pow2=False, stream=None):
    """moe_fp8_quantize_weights: w [G,N,K] or [N,K] (f32 or bf16) -> q of the same shape (float8_e4m3fn or
    float8_e5m2), scales [G, ceil(N/128), ceil(K/128)] (or without G) f32."""
    ty = _Types.ready()
    *G, N, K = w.shape
    if len(G) > 1:
        raise ValueError("w: [G, N, K] or [N, K] expected")
    code = _arg("w", w, ty.act, w.shape)
    dev = w.get_device()
    fmt = _arg("q", q, ty.fp8, w.shape, dev)
    _arg("scales", scales, ty.f32, (*G, (N + 127) // 128, (K + 127) // 128), dev)
    _call(dev, stream, "moe_fp8_quantize_weights", _lib.lib().moe_fp8_quantize_weights, w.data_ptr(), code,
          G[0] if G else 1, N, K, fmt, int(pow2), q.data_ptr(), scales.data_ptr())


def fp8_gemm(a, a_scales, b, b_scales, out, offsets=None, stream=None):
    """moe_fp8_gemm: a [M,K] with a_scales [ceil(K/128), M], b [G,N,K] or [N,K] with b_scales
    [G, ceil(N/128), ceil(K/128)] (or without G) -> out [M,N] (f32 or bf16); offsets [G+1] int32 groups the rows."""
    ty = _Types.ready()
    M, K = a.shape
    shape = b.shape
    if len(shape) not in (2, 3):
        raise ValueError("b: [G, N, K] or [N, K] expected")
    N, kb, dev = shape[-2], (K + 127) // 128, a.get_device()
    stack = len(shape) == 3
    g = shape[0] if stack else 1
    af = _arg("a", a, ty.fp8, (M, K))
    bf = _arg("b", b, ty.fp8, (g, N, K) if stack else (N, K), dev)
    _arg("a_scales", a_scales, ty.f32, (kb, M), dev)
    _arg("b_scales", b_scales, ty.f32, (g, (N + 127) // 128, kb) if stack else ((N + 127) // 128, kb), dev)
    od = _arg("out", out, ty.act, (M, N), dev)
    if offsets is not None:
        _arg("offsets", offsets, ty.i32, (g + 1,), dev)
    _call(dev, stream, "moe_fp8_gemm", _lib.lib().moe_fp8_gemm, M, N, K, g, a.data_ptr(), a_scales.data_ptr(), af,
          b.data_ptr(), b_scales.data_ptr(), bf, _ptr(offsets), out.data_ptr(), od)


def _fp8_weights(ty, dev, E, H, I, gate, gate_scale, up, up_scale, down, down_scale):
    """Checks stacks of E experts (None: one matrix each) and their scales."""
    h, i = (H + 127) // 128, (I + 127) // 128
    wide, tall, a, b = (I, H), (H, I), (i, h), (h, i)
    if E is not None:
        wide, tall, a, b = (E, *wide), (E, *tall), (E, *a), (E, *b)
    for t in (gate, gate_scale, up, up_scale, down, down_scale):
        if t is None:
            raise ValueError("fp8 weights: gate, up and down with their scales are needed")
    _arg("gate", gate, ty.e4m3, wide, dev)
    _arg("up", up, ty.e4m3, wide, dev)
    _arg("down", down, ty.e4m3, tall, dev)
    _arg("gate_scale", gate_scale, ty.f32, a, dev)
    _arg("up_scale", up_scale, ty.f32, a, dev)
    _arg("down_scale", down_scale, ty.f32, b, dev)


def experts(desc, x, w, topk_ids, topk_w, out, ws, shared_gate=None, stream=None):
    """moe_experts: the layer on a given routing (topk_ids [T,K] int32, topk_w [T,K] f32): permutation, experts,
    shared expert, combine."""
    ty = _Types.ready()
    act = ty.f32 if desc.act_dtype == "f32" else ty.bf16
    T, H, K = desc.T, desc.H, desc.top_k
    _arg("x", x, act, (T, H))
    dev = x.get_device()
    _arg("out", out, act, (T, H), dev)
    _arg("topk_ids", topk_ids, ty.i32, (T, K), dev)
    _arg("topk_w", topk_w, ty.f32, (T, K), dev)
    if shared_gate is not None:
        _arg("shared_gate", shared_gate, ty.f32, (T,), dev)
    if ws is not None and ws.get_device() != dev:
        raise ValueError(f"ws is on {ws.device}, not on cuda:{dev}")
    if desc.w_dtype == "fp8":
        _fp8_weights(ty, dev, desc.E, H, desc.I, w.gate, w.gate_scale, w.up, w.up_scale, w.down, w.down_scale)
        if desc.shared_I > 0:
            _fp8_weights(ty, dev, None, H, desc.shared_I, w.sh_gate, w.sh_gate_scale, w.sh_up, w.sh_up_scale, w.sh_down,
                         w.sh_down_scale)
    _call(dev, stream, "moe_experts", _lib.lib().moe_experts, ctypes.byref(desc.c()), x.data_ptr(), ctypes.byref(w.c()),
          topk_ids.data_ptr(), topk_w.data_ptr(), _ptr(shared_gate), out.data_ptr(), _ptr(ws), _nbytes(ws))


def last_device_status(stream=None) -> int:
    return _lib.lib().moe_last_device_status(_stream(stream))


def launch_count() -> int:
    return _lib.lib().moe_launch_count()


def trace_enable(on: bool) -> None:
    _lib.lib().moe_trace_enable(int(on))


def trace_read(max_records: int = 4096):
    names = (ctypes.c_char_p * max_records)()
    ms = (ctypes.c_float * max_records)()
    n = _lib.lib().moe_trace_read(names, ms, max_records)
    return [(names[i].decode(), ms[i]) for i in range(min(n, max_records))]


def debug_set_wait_limit(cycles: int) -> None:
    _lib.lib().moe_debug_set_wait_limit(cycles)


def debug_set_skip_stage(enable: bool) -> None:
    _lib.lib().moe_debug_set_skip_stage(int(enable))


def debug_set_barrier_delay(cycles: int) -> None:
    """moe_debug_set_barrier_delay: CTA 0 of the cooperative kernels arrives late at its first grid barrier."""
    _lib.lib().moe_debug_set_barrier_delay(cycles)


def set_fused_front(enable: bool) -> None:
    """moe_set_fused_front: selection + permutation + row gather of the tensor-core
    path as one cooperative kernel (True, default) or three launches (False)."""
    _lib.lib().moe_set_fused_front(int(enable))


def set_pair_gemm(enable: bool) -> None:
    """moe_set_pair_gemm: full 256-row tiles of compute-bound expert GEMMs on CTA pairs
    (tcgen05.mma.cta_group::2, True, default) or every row on single CTAs (False)."""
    _lib.lib().moe_set_pair_gemm(int(enable))


def set_decode_stream(enable: bool) -> None:
    """moe_set_decode_stream: gate/up and down of the cooperative decode kernel for f32 / bf16 / Q8_0 weights
    as one TMA-fed stream of work items (True, default) or two phases with a grid barrier (False)."""
    _lib.lib().moe_set_decode_stream(int(enable))


def set_tma_gather(enable: bool) -> None:
    """moe_set_tma_gather: the routed gate/up GEMM gathers its x rows with the copy engine (True) or
    reads a copy of them in expert order (False, default); size workspaces after changing it."""
    _lib.lib().moe_set_tma_gather(int(enable))


def set_tensor_min_tokens(tokens: int) -> None:
    """moe_set_tensor_min_tokens: bf16 layers of at least `tokens` tokens take the tensor-core path
    (default 16); size workspaces after changing it."""
    _lib.lib().moe_set_tensor_min_tokens(int(tokens))


def set_fused_decode(enable: bool) -> None:
    """moe_set_fused_decode: one cooperative kernel (True, default) or step-by-step
    launches (False) for 1..64 tokens on the weight-streaming path."""
    _lib.lib().moe_set_fused_decode(int(enable))


def _nbytes(t) -> int:
    if t is None:
        return 0
    return t.numel() * t.element_size()
