"""Cases of the routing and 8-bit-float expert operators: expert selection with a balance bias (forward and backward),
block-scaled e4m3 / e5m2 quantisation, the block-scaled matrix product, and the expert FFN on a given routing.

``run`` computes a case in plain torch operations, or (``own``) with the calls a user makes of
mixture_experts_ffn_07_b200.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -100  # the smallest block maximum that a scale follows


def listed():
    return [
        # the router of one decoded token: softmax scores over 128 experts, eight kept; nothing but latency
        dict(name="select_t1", op="select", T=1, E=128, K=8, scoring="softmax", bias=False, groups=1, kept=1,
             group_score="max", renorm=True, scale=1.0, logits="f32", pad=0, scores=False),
        # the router of a long prompt: sigmoid scores, a balance bias that moves the choice only, 4 of 8 groups scored
        # by their two best experts
        dict(name="select_t8192", op="select", T=8192, E=256, K=8, scoring="sigmoid", bias=True, groups=8, kept=4,
             group_score="top2", renorm=True, scale=2.5, logits="f32", pad=0, scores=False),
        # the router's gradient in a training step on an odd batch: bf16 logits in padded rows, and the gradient of a
        # balance loss on all scores
        dict(name="select_bwd_t4095", op="select_backward", T=4095, E=160, K=6, scoring="softmax", renorm=True,
             scale=1.0, logits="bf16", pad=32, d_scores=True),
        # activations of a decode batch, f32, scales rounded up to powers of two; a row is 22 blocks
        dict(name="quantize_t16", op="quantize", R=16, C=2816, x="f32", fmt="e4m3", pow2=True),
        # activations of a long prompt in front of the experts' products
        dict(name="quantize_t8192", op="quantize", R=8192, C=7168, x="bf16", fmt="e4m3", pow2=False),
        # one projection for a decode batch: streams the weights
        dict(name="product_m16", op="product", M=16, G=1, N=2048, K=7168, a="e4m3", b="e4m3", out="f32", used=16),
        # ragged groups, some empty, rows left over behind the last group, sizes that end inside a block of 128
        dict(name="product_ragged", op="product", M=3001, G=64, N=1056, K=2080, a="e4m3", b="e4m3", out="bf16",
             used=2990),
        # one projection over a long prompt: the tensor cores' rate
        dict(name="product_m8192", op="product", M=8192, G=1, N=7168, K=2048, a="e5m2", b="e4m3", out="bf16",
             used=8192),
        # the experts of one decoded token
        dict(name="experts_t1", op="experts", T=1, H=2048, E=128, I=768, K=8, act="silu", shared=0, skew=0.5),
        # a decode batch; the hidden rows end inside a block of 128
        dict(name="experts_t16", op="experts", T=16, H=2816, E=128, I=704, K=8, act="gelu_tanh", shared=0, skew=0.5),
        # a prompt through many small experts beside a gated shared one
        dict(name="experts_t4096", op="experts", T=4096, H=2048, E=256, I=512, K=8, act="silu", shared=512, skew=0.5),
        # a long prompt through large experts, unevenly loaded
        dict(name="experts_t8192", op="experts", T=8192, H=7168, E=256, I=2048, K=8, act="silu", shared=0, skew=0.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))))


def _log32(rng, lo, hi):
    return 32 * _log(rng, lo // 32, hi // 32)


def draw(rng):
    op = rng.choice(["select", "select_backward", "quantize", "product", "experts"])
    if op in ("select", "select_backward"):
        E = rng.randint(8, 256)
        K = rng.randint(1, min(12, E // 4 + 1))
        c = dict(op=op, T=_log(rng, 1, 8192), E=E, K=K, scoring=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), logits=rng.choice(["f32", "bf16"]),
                 pad=rng.choice([0, 1, 32]))
        if op == "select_backward":
            return dict(c, d_scores=rng.random() < 0.5)
        fit = [(g, k) for g in (2, 3, 4, 8, 16) if E % g == 0 for k in range(1, g + 1) if k * (E // g) >= K]
        groups, kept = rng.choice(fit) if fit and rng.random() < 0.6 else (1, 1)
        return dict(c, bias=rng.random() < 0.6, groups=groups, kept=kept, group_score=rng.choice(["max", "top2"]),
                    scores=rng.random() < 0.3)
    if op == "quantize":
        return dict(op=op, R=_log(rng, 1, 8192), C=_log32(rng, 32, 7168), x=rng.choice(["f32", "bf16"]),
                    fmt=rng.choice(["e4m3", "e5m2"]), pow2=rng.random() < 0.5)
    if op == "product":
        M, N, K = _log(rng, 1, 8192), _log32(rng, 32, 7168), _log32(rng, 32, 7168)
        G = min(_log(rng, 1, 256), max(1, (1 << 30) // (N * K)))
        return dict(op=op, M=M, G=G, N=N, K=K, a=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    b=rng.choice(["e4m3", "e4m3", "e5m2"]), out=rng.choice(["f32", "bf16"]),
                    used=M if rng.random() < 0.5 else rng.randint(max(1, M - 20), M))
    E = rng.choice([4, 8, 32, 60, 128])
    return dict(op=op, T=_log(rng, 1, 4096), H=_log32(rng, 256, 4096), E=E, I=_log32(rng, 64, 2048),
                K=rng.randint(1, min(8, E // 2)), act=rng.choice(["silu", "gelu_tanh"]),
                shared=rng.choice([0, 0, 320]), skew=rng.choice([0.0, 0.5, 1.0]))


# ------------------------------------------------------------------------------------------------ inputs
def _code_weights(g, G, N, K, fan, fmt):
    """G weight matrices [N, K] ~ N(0, 1/sqrt(fan)) as codes with one f32 scale for each 128 x 128 block."""
    dt, top = FP8[fmt]
    nb, kb = -(-N // 128), -(-K // 128)
    q = torch.empty((G, N, K), dtype=dt, device=DEV)
    s = torch.empty((G, nb, kb), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (N * K))
    for i in range(0, G, step):
        n = min(step, G - i)
        w = torch.randn((n, N, K), generator=g, device=DEV) / math.sqrt(fan)
        w = F.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(n, nb, 128, kb, 128)
        a = w.abs().amax((2, 4)) / top
        s[i:i + n] = a
        q[i:i + n] = (w / a[:, :, None, :, None]).view(n, nb * 128, kb * 128)[:, :N, :K].to(dt)
    return q, s


def _code_rows(g, R, C, fmt):
    """R activation rows ~ N(0, 1) as codes with one scale for each 128 values, scales [ceil(C/128), R]."""
    dt, top = FP8[fmt]
    x = F.pad(torch.randn((R, C), generator=g, device=DEV), (0, -C % 128)).view(R, -1, 128)
    a = x.abs().amax(2).clamp_min(1e-6) / top
    return (x / a[..., None]).view(R, -1)[:, :C].to(dt).contiguous(), a.t().contiguous()


def _logits(c, g):
    l = torch.randn((c["T"], c["E"] + c["pad"]), generator=g, device=DEV) * 1.5
    return l.to(TYPES[c["logits"]])[:, :c["E"]]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] == "select":
        T, E, K = c["T"], c["E"], c["K"]
        c["l"] = _logits(c, g)
        c["b"] = torch.randn(E, generator=g, device=DEV) * 0.1 if c["bias"] else None
        c["ids"] = torch.empty((T, K), dtype=torch.int32, device=DEV)
        c["w"] = torch.empty((T, K), device=DEV)
        c["s"] = torch.empty((T, E), device=DEV) if c["scores"] else None
    elif c["op"] == "select_backward":
        T, E, K = c["T"], c["E"], c["K"]
        c["l"] = _logits(c, g)
        c["ids"] = c["l"].float().topk(K, 1).indices.to(torch.int32)
        c["dw"] = torch.randn((T, K), generator=g, device=DEV)
        c["ds"] = torch.randn((T, E), generator=g, device=DEV) / E if c["d_scores"] else None
        c["dl"] = torch.empty((T, E), dtype=TYPES[c["logits"]], device=DEV)
    elif c["op"] == "quantize":
        R, C = c["R"], c["C"]
        x = torch.randn((R, C), generator=g, device=DEV) * torch.rand((R, 1), generator=g, device=DEV) * 4
        c["src"] = x.to(TYPES[c["x"]])
        c["q"] = torch.empty((R, C), dtype=FP8[c["fmt"]][0], device=DEV)
        c["sc"] = torch.empty((-(-C // 128), R), device=DEV)
    elif c["op"] == "product":
        M, G, N, K = c["M"], c["G"], c["N"], c["K"]
        c["qa"], c["sa"] = _code_rows(g, M, K, c["a"])
        c["qb"], c["sb"] = _code_weights(g, G, N, K, K, c["b"])
        c["off"] = None
        if G > 1 or c["used"] < M:
            cuts = torch.sort(torch.randint(0, c["used"] + 1, (G - 1,), generator=g, device=DEV)).values
            ends = torch.tensor([c["used"]], device=DEV)
            c["off"] = torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)
        c["y"] = torch.zeros((M, N), dtype=TYPES[c["out"]], device=DEV)
    else:
        T, H, E, I, K, S = c["T"], c["H"], c["E"], c["I"], c["K"], c["shared"]
        c["xs"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        load = torch.randn(E, generator=g, device=DEV) * c["skew"]
        score = torch.randn((T, E), generator=g, device=DEV) + load
        top = score.topk(K, 1)
        c["ids"], c["w"] = top.indices.to(torch.int32), torch.softmax(top.values, 1)
        for n, (G, N, D) in dict(gate=(E, I, H), up=(E, I, H), down=(E, H, I)).items():
            c[n], c[n + "_s"] = _code_weights(g, G, N, D, D, "e4m3")
        if S:
            for n, (N, D) in dict(sh_gate=(S, H), sh_up=(S, H), sh_down=(H, S)).items():
                q, s = _code_weights(g, 1, N, D, D, "e4m3")
                c[n], c[n + "_s"] = q[0], s[0]
            c["sg"] = torch.sigmoid(torch.randn(T, generator=g, device=DEV))
        c["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return c


# ------------------------------------------------------------------------------------------------ plain form
def _scores(l, scoring):
    return torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)


def _best(key, k):
    """Indices of the k largest of each row, the lower index first among equal ones."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def _select(c):
    T, E, K, n = c["T"], c["E"], c["K"], c["groups"]
    l = c["l"].double()  # scores next to a border decide in 64 bits
    s = _scores(l, c["scoring"])
    biased = s if c["b"] is None else s + c["b"].double()
    key = l if c["b"] is None else biased
    if n > 1:
        by = biased if c["group_score"] == "top2" else key
        best = by.view(T, n, E // n).topk(min(2, E // n) if c["group_score"] == "top2" else 1, 2).values.sum(2)
        keep = torch.zeros((T, n), dtype=torch.bool, device=DEV).scatter_(1, _best(best, c["kept"]), True)
        key = key.masked_fill(~keep.repeat_interleave(E // n, 1), -math.inf)
    ids = _best(key, K)
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = {"ids": ids.to(torch.int32), "w": (w * c["scale"]).float()}
    return dict(out, scores=s.float()) if c["scores"] else out


def _select_backward(c):
    s = _scores(c["l"].float(), c["scoring"])
    ids = c["ids"].long()
    dw = c["dw"] * c["scale"]
    if c["renorm"]:
        chosen = s.gather(1, ids)
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(s).scatter_(1, ids, dw)
    if c["ds"] is not None:
        ds = ds + c["ds"]
    d = s * (ds - (ds * s).sum(1, keepdim=True)) if c["scoring"] == "softmax" else ds * s * (1 - s)
    return d.to(c["l"].dtype)


def _code(x, fmt, pow2):
    """Rows [.., C] in f32 -> codes, and the scales [.., ceil(C/128)] of their blocks of 128."""
    dt, top = FP8[fmt]
    C = x.shape[-1]
    v = F.pad(x, (0, -C % 128)).unflatten(-1, (-1, 128))
    a = v.abs().amax(-1).clamp_min(TINY)
    top = torch.full_like(a, top)  # by a tensor: a quotient with a plain number is a product with its rounded inverse
    if pow2:
        m, e = torch.frexp(a / top)
        e = torch.where(m == 0.5, e - 1, e).to(torch.int32)
        scale, inv = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    else:
        scale, inv = a / top, top / a
    return (v * inv[..., None]).flatten(-2)[..., :C].to(dt), scale


def _rows(q, s):
    """Values of coded rows: q [R, C], s [R, ceil(C/128)]."""
    return q.float() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def _matrix(q, s):
    """Values of coded weights: q [.., N, K], s [.., ceil(N/128), ceil(K/128)]."""
    return q.float() * s.repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :q.shape[-2], :q.shape[-1]]


def _product(c):
    a = _rows(c["qa"], c["sa"].t())
    out = torch.zeros_like(c["y"])
    if c["off"] is None:
        return torch.matmul(a, _matrix(c["qb"][0], c["sb"][0]).t()).to(out.dtype)
    off = c["off"].tolist()
    for g in range(c["G"]):
        if off[g + 1] > off[g]:
            out[off[g]:off[g + 1]] = torch.matmul(a[off[g]:off[g + 1]], _matrix(c["qb"][g], c["sb"][g]).t())
    return out


def _act(c, v):
    return F.silu(v) if c["act"] == "silu" else F.gelu(v, approximate="tanh")


def _ffn(c, x, gate, up, down):
    h = _act(c, torch.matmul(x, gate.mT)) * torch.matmul(x, up.mT)
    return torch.matmul(_rows(*_code(h, "e4m3", False)), down.mT)


def _experts(c):
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    x = _rows(*_code(c["xs"].float(), "e4m3", False))
    names = ("gate", "up", "down")
    if T * K <= E:  # few pairs: one batched product over the experts they name
        e = c["ids"].long().view(-1)
        y = _ffn(c, x.repeat_interleave(K, 0)[:, None], *[_matrix(c[n][e], c[n + "_s"][e]) for n in names])
        out = (y.view(T, K, H) * c["w"][..., None]).sum(1)
    else:
        flat = c["ids"].view(-1).long()
        order = torch.sort(flat, stable=True).indices
        count = torch.bincount(flat, minlength=E).tolist()
        y = torch.empty((T * K, H), device=DEV)
        at = 0
        for e in range(E):
            rows = order[at:at + count[e]]
            at += count[e]
            if count[e]:
                y[rows] = _ffn(c, x[rows // K], *[_matrix(c[n][e], c[n + "_s"][e]) for n in names])
        out = (y.view(T, K, H) * c["w"][..., None]).sum(1)
    if c["shared"]:
        out = out + c["sg"][:, None] * _ffn(c, x, *[_matrix(c["sh_" + n], c["sh_" + n + "_s"]) for n in names])
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ one pass
def _own(c):
    import mixture_experts_ffn_07_b200 as moe

    if c["op"] in ("select", "select_backward"):
        d = c.get("desc")
        if d is None:
            d = c["desc"] = moe.SelectDesc(T=c["T"], E=c["E"], top_k=c["K"], scoring=c["scoring"],
                                           n_groups=c.get("groups", 1), topk_groups=c.get("kept", 1),
                                           group_score=c.get("group_score", "max"), renormalize=c["renorm"],
                                           scale=c["scale"])
        if c["op"] == "select_backward":
            moe.select_backward(d, c["l"], c["ids"], c["dw"], c["dl"], d_scores=c["ds"])
            return c["dl"]
        moe.select(d, c["l"], c["ids"], c["w"], bias=c["b"], scores=c["s"])
        out = {"ids": c["ids"], "w": c["w"]}
        return dict(out, scores=c["s"]) if c["scores"] else out
    if c["op"] == "quantize":
        moe.fp8_quantize(c["src"], c["q"], c["sc"], pow2=c["pow2"])
        return {"q": c["q"], "scale": c["sc"]}
    if c["op"] == "product":
        moe.fp8_gemm(c["qa"], c["sa"], c["qb"], c["sb"], c["y"], offsets=c["off"])
        return c["y"]
    if "desc" not in c:
        c["desc"] = moe.Desc(T=c["T"], H=c["H"], E=c["E"], I=c["I"], top_k=c["K"], act=c["act"], w_dtype="fp8",
                             shared_I=c["shared"], has_shared_gate=c["shared"] > 0)
        c["weights"] = moe.Weights(**{n: c[n] for n in ("gate", "up", "down")},
                                   **{n + "_scale": c[n + "_s"] for n in ("gate", "up", "down")},
                                   **{n: c.get(n) for n in ("sh_gate", "sh_up", "sh_down")},
                                   **{n + "_scale": c.get(n + "_s") for n in ("sh_gate", "sh_up", "sh_down")})
        c["ws"] = torch.empty(moe.workspace_bytes(c["desc"]), dtype=torch.uint8, device=DEV)
    moe.experts(c["desc"], c["xs"], c["weights"], c["ids"], c["w"], c["y"], c["ws"], shared_gate=c.get("sg"))
    return c["y"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "select":
        return _select(state)
    if state["op"] == "select_backward":
        return _select_backward(state)
    if state["op"] == "quantize":
        q, s = _code(state["src"].float(), state["fmt"], state["pow2"])
        return {"q": q, "scale": s.t().contiguous()}
    if state["op"] == "product":
        return _product(state)
    return _experts(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] in ("select", "select_backward"):
        T, E, K, lb = c["T"], c["E"], c["K"], 4 if c["logits"] == "f32" else 2
        if c["op"] == "select":
            more = (4 * E if c["bias"] else 0) + (4 * T * E if c["scores"] else 0)
        else:
            more = lb * T * E + (4 * T * E if c["d_scores"] else 0)
        return {"bytes": lb * T * E + 8 * T * K + more, "flops": 10 * T * E}
    if c["op"] == "quantize":
        n = c["R"] * c["C"]
        return {"bytes": n * (5 if c["x"] == "f32" else 3) + 4 * c["R"] * -(-c["C"] // 128), "flops": 3 * n}
    if c["op"] == "product":
        M, G, N, K, u = c["M"], c["G"], c["N"], c["K"], c["used"]
        touched = G if G == 1 else min(G, G * (1 - (1 - 1 / G) ** u))  # groups that hold a row, about
        kb = -(-K // 128)
        return {"bytes": u * (K + 4 * kb) + touched * (N * K + 4 * kb * -(-N // 128)) + u * N * (4 if c["out"] == "f32" else 2),
                "flops": 2 * u * N * K}
    T, H, E, I, K, S = c["T"], c["H"], c["E"], c["I"], c["K"], c["shared"]
    touched = E * (1 - (1 - K / E) ** T)  # experts that some token names, about
    return {"bytes": touched * 3 * I * H * (1 + 4 / 16384) + 3 * S * H + 4 * T * H + 8 * T * K,
            "flops": 6 * T * H * (K * I + S)}


# ------------------------------------------------------------------------------------------------ 64 bits
def _round8(v, fmt):
    """v in f64 to the nearest value of the 8-bit format, half to even."""
    man, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(e.clamp_min(low) - man)
    return torch.round(v / step) * step


def _values64(x, fmt, pow2):
    """The values that rows of f64 numbers stand for once coded, the same rows before their scales, and the scales."""
    top = FP8[fmt][1]
    parts, codes, scales = [], [], []
    for lo in range(0, x.shape[1], 128):
        v = x[:, lo:lo + 128].float().double()
        a = torch.clamp(torch.amax(torch.abs(v), 1, keepdim=True), min=TINY)
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(a / top)))
            s = torch.where(s / 2 >= a / top, s / 2, torch.where(s < a / top, s * 2, s))
            inv = 1 / s
        else:  # the scale and its inverse are 32-bit numbers, and so is the product
            s, inv = (a / top).float().double(), (top / a).float().double()
        q = _round8((v * inv).float().double(), fmt)
        parts.append(q * s)
        codes.append(q)
        scales.append(s)
    return torch.cat(parts, 1), torch.cat(codes, 1), torch.cat(scales, 1)


def _weights64(q, s):
    N, K = q.shape
    rows = torch.arange(N, device=DEV) // 128
    cols = torch.arange(K, device=DEV) // 128
    return q.to(torch.float64) * s.double()[rows][:, cols]


def _ffn64(act, x, gate, up, down):
    g, u = x @ gate.T, x @ up.T
    if act == "silu":
        a = g / (1 + torch.exp(-g))
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return _values64(a * u, "e4m3", False)[0] @ down.T


def _score64(l, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    z = torch.exp(l - torch.amax(l, 1, keepdim=True))
    return z / torch.sum(z, 1, keepdim=True)


def _select64(c):
    T, E, n = c["T"], c["E"], c["groups"]
    l = c["l"].to(torch.float64)
    s = _score64(l, c["scoring"])
    with_bias = s + (c["b"].to(torch.float64) if c["b"] is not None else 0)
    key = with_bias if c["b"] is not None else l
    lowest = torch.full_like(key, -math.inf)
    if n > 1:
        rank = torch.sort((with_bias if c["group_score"] == "top2" else key).reshape(T, n, -1), 2).values
        top = rank[..., -1] + (rank[..., -2] if c["group_score"] == "top2" and E // n > 1 else 0)
        worse = (top[:, None, :] > top[:, :, None]).sum(2)  # groups that score more
        key = torch.where((worse < c["kept"])[:, torch.arange(E, device=DEV) // (E // n)], key, lowest)
    ids = torch.argsort(-key, dim=1, stable=True)[:, :c["K"]]
    w = torch.take_along_dim(s, ids, 1) * c["scale"]
    if c["renorm"]:
        w = w * c["scale"] / torch.sum(w, 1, keepdim=True)
    out = {"ids": None, "w": w}
    return dict(out, scores=s) if c["scores"] else out


def _select_backward64(c):
    l = c["l"].to(torch.float64)
    s = _score64(l, c["scoring"])
    ids = c["ids"].to(torch.int64)
    mask = torch.zeros_like(s)
    mask[torch.arange(c["T"], device=DEV)[:, None], ids] = 1
    gw = torch.zeros_like(s)
    gw[torch.arange(c["T"], device=DEV)[:, None], ids] = c["dw"].to(torch.float64) * c["scale"]
    total = (s * mask).sum(1, keepdim=True) if c["renorm"] else torch.ones_like(s[:, :1])
    mean = (gw * s).sum(1, keepdim=True) / total if c["renorm"] else 0
    gs = mask * (gw - mean) / total + (c["ds"].to(torch.float64) if c["ds"] is not None else 0)
    if c["scoring"] == "sigmoid":
        return gs * (s - s * s)
    return gs * s - s * (gs * s).sum(1, keepdim=True)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "select":
        return _select64(c)
    if c["op"] == "select_backward":
        return _select_backward64(c)
    if c["op"] == "quantize":
        _, q, s = _values64(c["src"].to(torch.float64), c["fmt"], c["pow2"])
        return {"q": q, "scale": s.T}
    if c["op"] == "product":
        cols = torch.arange(c["K"], device=DEV) // 128
        a = c["qa"].to(torch.float64) * c["sa"].double().T[:, cols]
        off = [0, c["M"]] if c["off"] is None else [int(v) for v in c["off"].cpu()]
        y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=DEV)
        for g in range(c["G"]):
            y[off[g]:off[g + 1]] = a[off[g]:off[g + 1]] @ _weights64(c["qb"][g], c["sb"][g]).T
        return y
    x = _values64(c["xs"].to(torch.float64), "e4m3", False)[0]
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    names = ("gate", "up", "down")
    for e in torch.unique(c["ids"]).tolist():
        t, k = torch.nonzero(c["ids"] == e, as_tuple=True)
        y[t] += c["w"].to(torch.float64)[t, k, None] * _ffn64(
            c["act"], x[t], *[_weights64(c[n][e], c[n + "_s"][e]) for n in names])
    if c["shared"]:
        y += c["sg"].to(torch.float64)[:, None] * _ffn64(
            c["act"], x, *[_weights64(c["sh_" + n], c["sh_" + n + "_s"]) for n in names])
    return y
