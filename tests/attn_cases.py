"""Plain implementations in binary64 of the attention sublayer's operators (FP8 linear with a scale per block of
128, query/key norm with rotation, cross attention) and the error bounds of the kernels, shared by the tests.  Torch
on whatever device the inputs are; no code of the package.

Bounds, from the roundings the operators document (u = 2^-24, half a binary32 step; h = 2^-8, half a bf16 step):
  * FP8: a block's product sums 128 exact products in 4 instructions of 32, each aligned to its largest term and
    truncated: at most 33 terms times 2u each; then one fused multiply-add per block and the bias:
    |dy| <= h |y| + (4 * 33 * 2 + 2 KB + 3) u sum |terms|.
  * norm and rotation: the mean of squares carries (dim + 3) u, its root half of that, rsqrt 2 steps, three products
    and the rotation's sum: |dy| <= h |y| + (dim / 2 + 12) u (|a cos| + |c sin|).
  * attention: a score carries (dim + 2) u sum |q k| (truncated: twice that) and the exponent two more roundings of
    its argument, the exponential 46 u (2.7e-6, the polynomial's largest relative error on its interval; 2 u where the
    special-function unit computes it), the sum over keys n u, p rounded to bf16 (h) in the numerator only:
    |do| <= h |o| + (h + 2 e) sum p |v| / sum p,  e = 2 (dim + 4) u max(scale sum |q k|) + (n + 50) u."""
import math

import torch

U = 2.0 ** -24
H = 2.0 ** -8


# ------------------------------------------------------------------------------------------------- FP8
def scale_of(amax):
    """fl32(max(amax, 2^-100) / 448): the rounded quotient (torch on CUDA multiplies by 1/448 for a Python number)."""
    a = amax.clamp_min(2.0 ** -100)
    return a / torch.full_like(a, 448.0)


def e4m3(v):
    """E4M3 value (binary64) nearest to v (any float), ties to even, clamped to 448."""
    v = v.double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def fp8_quantize(x):
    """(values of the codes [M,K] in binary64, scales f32 [M, KB]) of a bf16 or f32 tensor."""
    m, k = x.shape
    kb = -(-k // 128)
    p = torch.zeros(m, kb * 128, device=x.device)
    p[:, :k] = x.float()
    p = p.view(m, kb, 128)
    s = scale_of(p.abs().amax(2))
    prod = p * (1.0 / s)[:, :, None]  # binary32, as defined
    return e4m3(prod).view(m, kb * 128)[:, :k], s


def fp8_weight(w):
    """(values of the codes [N,K] in binary64, scales f32 [NB, KB])."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.zeros(nb * 128, kb * 128, device=w.device)
    p[:n, :k] = w.float()
    p = p.view(nb, 128, kb, 128)
    s = scale_of(p.abs().amax((1, 3)))
    return e4m3(p * (1.0 / s)[:, None, :, None]).reshape(nb * 128, kb * 128)[:n, :k], s


def fp8_linear(qx, sx, qw, sw, bias):
    """(y, bound) in binary64 from codes' values and scales."""
    m, k = qx.shape
    n = qw.shape[0]
    kb = sx.shape[1]
    ex = sx.double().repeat_interleave(128, 1)[:, :k]
    ew = sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    xs, ws = qx * ex, qw * ew
    y = xs @ ws.t()
    total = xs.abs() @ ws.abs().t()
    if bias is not None:
        y = y + bias.double()
        total = total + bias.double().abs()
    bound = H * y.abs() + (4 * 33 * 2 + 2 * kb + 3) * U * total
    # where the terms' magnitudes sum past binary32's (and bf16's) largest number, 3.39e38, the binary32 sum may
    # overflow on the way whatever its end: such an element has no bound
    return y, torch.where(total < 3.38e38, bound, math.inf)


# ------------------------------------------------------------------------------------------------- norm, rotation
def rope_table(rows, rot, device, theta=10000.0):
    pos = torch.arange(rows, dtype=torch.float64, device=device)
    freq = theta ** (-torch.arange(rot // 2, dtype=torch.float64, device=device) * 2 / rot)
    a = pos[:, None] * freq[None, :]
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def norm_rope(x, weight, eps, table, positions, pairs):
    """(y, bound) in binary64, x [B,S,H,D]."""
    b, s, _, d = x.shape
    y = x.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    spread = y.abs()
    if table is not None:
        rot = 2 * table.shape[1]
        at = positions.long() if positions is not None else torch.arange(s, device=x.device).expand(b, s)
        t = table.double()[at][:, :, None]
        cos, sin = t[..., 0], t[..., 1]
        i = torch.arange(0, rot, 2, device=x.device) if pairs == "interleaved" else torch.arange(rot // 2, device=x.device)
        j = i + (1 if pairs == "interleaved" else rot // 2)
        out, sp = y.clone(), spread.clone()
        out[..., i] = y[..., i] * cos - y[..., j] * sin
        out[..., j] = y[..., i] * sin + y[..., j] * cos
        sp[..., i] = (y[..., i] * cos).abs() + (y[..., j] * sin).abs()
        sp[..., j] = (y[..., i] * sin).abs() + (y[..., j] * cos).abs()
        y, spread = out, sp
    return y, H * y.abs() + (d / 2 + 12) * U * spread


# ------------------------------------------------------------------------------------------------- attention
def attention(q, k, v, kv_len, kv_mask, scale):
    """(o, bound) in binary64; one sample and head at a time."""
    b, sq, hq, d = q.shape
    sk, hk = k.shape[1], k.shape[2]
    o = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for i in range(b):
        keep = torch.arange(sk, device=q.device)
        if kv_len is not None:
            keep = keep[:max(0, min(sk, int(kv_len[i])))]
        if kv_mask is not None:
            keep = keep[kv_mask[i, :sk][keep] != 0]
        if keep.numel() == 0:
            continue
        for h in range(hq):
            qq, kk, vv = q[i, :, h].double(), k[i, keep, h // (hq // hk)].double(), v[i, keep, h // (hq // hk)].double()
            p = torch.softmax(scale * (qq @ kk.t()), -1)
            mag = scale * (qq.abs() @ kk.abs().t()).amax(-1, keepdim=True)
            e = 2 * (d + 4) * U * mag + (keep.numel() + 50) * U
            oo = p @ vv
            o[i, :, h] = oo
            bound[i, :, h] = H * oo.abs() + (H + 2 * e) * (p @ vv.abs())
    return o, bound


def bf16(g, *shape, device="cuda", scale=1.0):
    return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)


def generator(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def check(got, ref, bound):
    """Every element that has a bound within it; no NaN or infinity."""
    has = torch.isfinite(bound)
    g, ref, bound = got.double()[has], ref[has], bound[has]
    assert torch.isfinite(g).all()
    over = (g - ref).abs() - bound
    assert over.max() <= 0, (float(over.max()), int(over.argmax()), tuple(got.shape))
    return float((g - ref).norm() / ref.norm().clamp_min(1e-30))


def inv_sqrt(d):
    return 1.0 / math.sqrt(d)
