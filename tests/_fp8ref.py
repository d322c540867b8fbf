"""Plain 64-bit references of the selection and of the block-scaled 8-bit operators, with the error bounds their
32-bit evaluation has to keep (all torch float64, on whatever device the inputs are)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24   # half a step of f32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}


# ------------------------------------------------------------------------------------------------ selection
def scores(l, scoring):
    l = l.double()
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    z = torch.exp(l - torch.where(torch.isneginf(m), torch.zeros_like(m), m))
    total = z.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(z), z / total)


def select(l, K, scoring, bias=None, n_groups=1, topk_groups=1, group_score="max", renormalize=True, scale=1.0):
    """ids [T,K], w [T,K], scores [T,E] by plain loops over rows."""
    s = scores(l, scoring)
    T, E = s.shape
    masked = torch.isneginf(l.double())
    biased = s + (bias.double() if bias is not None else 0)
    key = torch.where(masked, torch.full_like(s, -math.inf), biased if bias is not None else l.double())
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    by = torch.where(masked | torch.isnan(biased), torch.full_like(s, -math.inf), biased) if group_score == "top2" else key
    ids = torch.empty((T, K), dtype=torch.int64)
    gs = E // max(n_groups, 1)
    key_l, by_l = key.tolist(), by.tolist()
    for t in range(T):
        experts = range(E)
        if n_groups > 1:
            def of(g):
                v = sorted(by_l[t][g * gs:(g + 1) * gs], reverse=True)
                return v[0] + v[1] if group_score == "top2" and gs > 1 and v[1] > -math.inf else v[0]
            best = sorted(range(n_groups), key=lambda g: (-of(g), g))[:topk_groups]
            experts = [e for e in range(E) if e // gs in best]
        ids[t] = torch.tensor(sorted(experts, key=lambda e: (-key_l[t][e], e))[:K])
    ids = ids.to(l.device)
    w = s.gather(1, ids)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return ids, w * scale, s


def select_backward(l, ids, d_w, d_scores, scoring, renormalize, scale):
    """d_logits and the sum of the absolute values of the terms it is made of."""
    s = scores(l, scoring)
    dw = d_w.double() * scale
    mag = dw.abs()
    if renormalize:
        c = s.gather(1, ids)
        total = c.sum(1, keepdim=True)
        mag = (mag + (mag * c).sum(1, keepdim=True) / total) / total
        dw = (dw - (dw * c).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_add_(1, ids, dw)
    am = torch.zeros_like(s).scatter_add_(1, ids, mag)
    if d_scores is not None:
        ds, am = ds + d_scores.double(), am + d_scores.double().abs()
    if scoring == "softmax":
        return s * (ds - (ds * s).sum(1, keepdim=True)), s * (am + (am * s).sum(1, keepdim=True))
    return ds * s * (1 - s), am * s


# ------------------------------------------------------------------------------------------------ 8-bit floats
def round8(v, fmt):
    """v (f64) to the format's nearest value, half to even."""
    _, top, man, low = FP8[fmt]
    e = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(e.clamp_min(low) - man)
    return torch.round(v / step) * step


def step8(v, fmt):
    """The largest spacing of the format's values next to v."""
    _, top, man, low = FP8[fmt]
    e = torch.frexp(v).exponent.double() - 1
    return torch.exp2(e.clamp_min(low) - man)


def block_max(x, rows):
    """max |x| of each block of 128 columns (and `rows` rows), [ceil(R/rows), ceil(C/128)]."""
    R, C = x.shape
    p = torch.nn.functional.pad(x.abs(), (0, -C % 128, 0, -R % rows))
    return p.view(-1, rows, p.shape[1] // 128, 128).amax((1, 3))


def scale_of(a, fmt, pow2):
    """(scale, inv) as f64 holding the f32 numbers of the definition."""
    top = FP8[fmt][1]
    a = a.double().clamp_min(2.0 ** -100)
    if pow2:
        m, e = torch.frexp(a / top)
        s = torch.exp2((e - (m == 0.5).to(e.dtype)).double())
        return s, 1 / s
    return (a / top).float().double(), (top / a).float().double()


def spread(s, R, C, rows):
    return s.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :C]


def quantize(x, fmt, pow2, rows=1):
    """Codes' values and scales [ceil(R/rows), ceil(C/128)] of a 2-D tensor."""
    R, C = x.shape
    s, inv = scale_of(block_max(x.double(), rows), fmt, pow2)
    return round8((x.double() * spread(inv, R, C, rows)).float().double(), fmt), s


def dequantize_rows(q, scales):
    """q [R,C] codes, scales [ceil(C/128), R]."""
    return q.float().double() * spread(scales.t().double(), q.shape[0], q.shape[1], 1)


def dequantize_weights(q, s):
    return q.float().double() * spread(s.double(), q.shape[0], q.shape[1], 128)


def sum_bound(K):
    """Relative to the sum of the terms' absolute values: 128 f32 additions inside a block (each off by at most a
    step), one scaling with a rounded scale product, and one addition per block."""
    return (128 + (K + 127) // 128 + 4) * 2 * U32


def ffn(x, gate, up, down, act):
    """One expert on dequantised rows x [n,H] and weights (f64): y, and the bound of an evaluation that takes f32
    sums, codes act(g) * u to e4m3 with a scale per 128 and multiplies in f32.  An element of h whose 64-bit value
    lies nearer to a border between two codes than its f32 evaluation may be off can take either code: the bound
    holds a whole step for it."""
    H, I = x.shape[1], gate.shape[0]
    g, u = x @ gate.T, x @ up.T
    eg, eu = sum_bound(H) * (x.abs() @ gate.abs().T), sum_bound(H) * (x.abs() @ up.abs().T)
    if act == "silu":
        a = g / (1 + torch.exp(-g))
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    h = a * u
    # |act'| <= 1.13 for both; 2^-18 relative for exp or tanh in f32 of arguments below 40, plus the absolute error
    # of 1 + tanh near -1 in units of g
    eh = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + 2.0 ** -18 * h.abs() + 2.0 ** -22 * (g * u).abs()
    n = h.shape[0]
    amax = block_max(h, 1)
    s, inv = scale_of(amax, "e4m3", False)
    es = spread(block_max(eh, 1) / amax.clamp_min(2.0 ** -100), n, I, 1) + 4 * U32  # relative error of the scale
    S, V = spread(s, n, I, 1), spread(inv, n, I, 1)
    v = h * V
    q = round8(v, "e4m3")
    ev = eh * V + v.abs() * es
    st = step8(v.abs() + ev, "e4m3")
    border = (v - q).abs()
    sure = border + ev < step8((v.abs() - ev).clamp_min(0), "e4m3") / 2
    hq = q * S
    eq = torch.where(sure, torch.zeros_like(v), st * S) + (hq.abs() + st * S) * es
    y = hq @ down.T
    return y, eq @ down.abs().T + sum_bound(I) * (hq.abs() @ down.abs().T)
