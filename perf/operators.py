"""The attention sublayer's operators of a diffusion transformer, as cases that can be timed and compared:

  fp8_linear       y = x W^T + b in 8-bit floating point (E4M3) with one binary32 scale for each block of 128
                   (activations: 1 x 128 along K, taken from each input; weights: 128 x 128, fixed),
  qk_norm_rope     RMS norm of the queries and keys of each head and the position rotation, in one pass,
  cross_attention  softmax(scale q k^T) v of one sequence over another's states, with per-sample key lengths or
                   key masks, and query heads that share key/value heads.

With `own` false, `run` computes them from elementary torch operations in 32 bits; with `own` true, it makes the
framework's calls.  `exact` computes the definition in 64 bits."""
import math

import torch

own = False

FP8_MAX = 448.0  # largest E4M3 value
BLOCK = 128
AMAX_MIN = 2.0 ** -100  # blocks whose largest value is below this use this (scale and its reciprocal stay normal)


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # adaLN modulation vector of a classifier-free-guidance pair, 6 x width outputs: one weight stream
        dict(name="fp8_modulation_2", op="fp8_linear", m=2, k=3072, n=18432, bias=True),
        # a short prompt's states through a projection whose width ends inside a block of 128
        dict(name="fp8_prompt_77", op="fp8_linear", m=77, k=1168, n=2312, bias=True),
        # fused QKV projection at 512 x 512 image tokens
        dict(name="fp8_qkv_1024", op="fp8_linear", m=1024, k=3072, n=9216, bias=True),
        # MLP pair at 1024 x 1024: 4096 image + 512 text tokens
        dict(name="fp8_up_4608", op="fp8_linear", m=4608, k=3072, n=12288, bias=True),
        dict(name="fp8_down_4608", op="fp8_linear", m=4608, k=12288, n=3072, bias=False),
        # one token of one sample: latency
        dict(name="qk_token", op="qk_norm_rope", b=1, s=1, hq=24, hk=24, d=128, rot=128, pairs="interleaved",
             positions=True),
        # odd sizes, shared key heads, half-split pairs on a part of the head
        dict(name="qk_odd_333", op="qk_norm_rope", b=3, s=333, hq=16, hk=4, d=72, rot=48, pairs="halves",
             positions=True),
        # a block's fused QKV output at batch 2, 1024 x 1024
        dict(name="qk_block_9216", op="qk_norm_rope", b=2, s=4608, hq=24, hk=24, d=128, rot=128,
             pairs="interleaved", positions=False),
        # one query token over long states, three query heads to a key head: the cache is read once
        dict(name="attn_token_4096", op="cross_attention", b=2, sq=1, sk=4096, hq=24, hk=8, d=128, keys="all"),
        # padded prompts with a key mask, heads of 72
        dict(name="attn_masked_300", op="cross_attention", b=8, sq=1000, sk=300, hq=16, hk=16, d=72, keys="mask"),
        # image tokens over prompts of unequal length
        dict(name="attn_prompt_512", op="cross_attention", b=2, sq=4096, sk=512, hq=24, hk=24, d=128, keys="len"),
        # image tokens over image and prompt together: the largest
        dict(name="attn_joint_4608", op="cross_attention", b=1, sq=4096, sk=4608, hq=24, hk=24, d=128, keys="all"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("fp8_linear", "qk_norm_rope", "cross_attention"))
    if op == "fp8_linear":
        m, k, n = _spread(rng, 1, 4608), _spread(rng, 256, 12288, 16), _spread(rng, 256, 12288, 8)
        while m * k * n > 4608 * 3072 * 12288:
            m = (m + 1) // 2
        return dict(op=op, m=m, k=k, n=n, bias=rng.random() < 0.7)
    d = rng.choice((40, 64, 72, 80, 96, 112, 128, 128))
    hk = rng.choice((2, 4, 8, 12, 16, 24))
    share = rng.choice((1, 1, 1, 2, 3, 4))
    hq = hk * (share if hk * share <= 24 else 1)
    b = rng.choice((1, 1, 2, 3, 4))
    if op == "qk_norm_rope":
        s = max(1, _spread(rng, 1, 4608) * 2 // b) if b > 2 else _spread(rng, 1, 4608)
        rot = rng.choice((d, d, d // 16 * 8, 0))
        return dict(op=op, b=b, s=s, hq=hq, hk=hk, d=d, rot=rot, pairs=rng.choice(("interleaved", "halves")),
                    positions=rng.random() < 0.5)
    sq = rng.choice((1, _spread(rng, 1, 64), _spread(rng, 16, 4096), _spread(rng, 64, 4096)))
    sk = _spread(rng, 1, 4608)
    while b * hq * sq * sk * d > 24 * 4096 * 4608 * 128:
        sq = (sq + 1) // 2
    return dict(op=op, b=b, sq=sq, sk=sk, hq=hq, hk=hk, d=d, keys=rng.choice(("all", "len", "mask")))


# ------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weight_codes(w):
    """E4M3 codes [N, K] and scales [ceil(N/128), ceil(K/128)] of a weight, as a checkpoint holds them."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = torch.zeros(nb * BLOCK, kb * BLOCK, device=w.device)
    p[:n, :k] = w
    p = p.view(nb, BLOCK, kb, BLOCK)
    s = p.abs().amax(dim=(1, 3)).clamp_min(AMAX_MIN) / FP8_MAX
    q = (p * (1.0 / s)[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    st = dict(case=case)
    if case["op"] == "fp8_linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = _randn(g, m, k)
        x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 200)]] *= 50.0  # outlier channels
        st["x"] = x.to(torch.bfloat16)
        st["wq"], st["ws"] = _weight_codes(_randn(g, n, k) * 0.02)
        st["bias"] = (_randn(g, n) * 0.01).to(torch.bfloat16) if case["bias"] else None
        if own:
            import diffusion_transformer_w4a4_b200 as svdq

            bias = None if st["bias"] is None else st["bias"].view(torch.int16).cpu().numpy().view("uint16")
            st["layer"] = svdq.Fp8Linear(st["wq"].view(torch.uint8).cpu().numpy(), st["ws"].cpu().numpy(), bias)
    elif case["op"] == "qk_norm_rope":
        b, s, hq, hk, d, rot = (case[f] for f in ("b", "s", "hq", "hk", "d", "rot"))
        qkv = _randn(g, b, s, hq + 2 * hk, d).to(torch.bfloat16)  # a fused projection's output
        st["q"], st["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        st["wq"] = (1.0 + 0.1 * _randn(g, d)).to(torch.bfloat16)
        st["wk"] = (1.0 + 0.1 * _randn(g, d)).to(torch.bfloat16)
        st["table"] = st["pos"] = None
        if rot:
            rows = 8192 if case["positions"] else s
            pos = torch.arange(rows, device="cuda", dtype=torch.float64)
            freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
            ang = pos[:, None] * freq[None, :]
            st["table"] = torch.stack((ang.cos(), ang.sin()), dim=-1).float().contiguous()
            if case["positions"]:
                st["pos"] = torch.randint(0, rows, (b, s), generator=g, device="cuda", dtype=torch.int32)
    else:
        b, sq, sk, hq, hk, d = (case[f] for f in ("b", "sq", "sk", "hq", "hk", "d"))
        st["q"] = _randn(g, b, sq, hq, d).to(torch.bfloat16)
        kv = _randn(g, b, sk, 2, hk, d).to(torch.bfloat16)  # a fused key/value projection's output
        st["k"], st["v"] = kv[:, :, 0], kv[:, :, 1]
        st["len"] = st["mask"] = None
        if case["keys"] == "len":
            st["len"] = torch.randint(max(1, sk // 8), sk + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        elif case["keys"] == "mask":
            st["mask"] = (torch.rand(b, sk, generator=g, device="cuda") < 0.8).to(torch.uint8)
    return st


# ------------------------------------------------------------------------------------------------- plain forms
def _blocks(x, kb):
    m, k = x.shape
    return torch.nn.functional.pad(x, (0, kb * BLOCK - k)).view(m, kb, BLOCK)


def _plain_fp8(st):
    m, k = st["x"].shape
    kb = -(-k // BLOCK)
    p = _blocks(st["x"].float(), kb)
    top = p.abs().amax(dim=2, keepdim=True).clamp_min(AMAX_MIN)
    s = top / torch.full_like(top, FP8_MAX)  # the rounded quotient (a Python number would be multiplied as 1/448)
    codes = (p * (1.0 / s)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    x = (codes.float() * s).view(m, kb * BLOCK)[:, :k]
    ws = st["ws"].repeat_interleave(BLOCK, 0)[:st["wq"].shape[0]].repeat_interleave(BLOCK, 1)[:, :k]
    y = x @ (st["wq"].float() * ws).t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(torch.bfloat16)


def _rotate(x, table, pos, rot, pairs):
    b, s, h, d = x.shape
    t = table[pos.long()] if pos is not None else table[:s].unsqueeze(0).expand(b, -1, -1, -1)
    cos, sin = t[..., 0].unsqueeze(2), t[..., 1].unsqueeze(2)
    r, rest = x[..., :rot], x[..., rot:]
    if pairs == "interleaved":
        a, c = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - c * sin, a * sin + c * cos), dim=-1).flatten(-2)
    else:
        a, c = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - c * sin, a * sin + c * cos), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _norm_rope(x, w, st, f):
    x = x.to(f)
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * w.to(f)
    rot = st["case"]["rot"]
    return _rotate(x, st["table"].to(f), st["pos"], rot, st["case"]["pairs"]) if rot else x


def _plain_qk(st):
    return [_norm_rope(st["q"], st["wq"], st, torch.float32).to(torch.bfloat16),
            _norm_rope(st["k"], st["wk"], st, torch.float32).to(torch.bfloat16)]


def _plain_attn(st):
    q, k, v = st["q"], st["k"], st["v"]
    b, sq, hq, d = q.shape
    sk, hk = k.shape[1], k.shape[2]
    qf = q.float().transpose(1, 2).reshape(b, hk, hq // hk * sq, d)  # the query heads of a key head together
    s = qf @ k.float().permute(0, 2, 3, 1) / math.sqrt(d)
    if st["len"] is not None or st["mask"] is not None:
        keep = st["mask"] != 0 if st["mask"] is not None else \
            torch.arange(sk, device=q.device)[None, :] < st["len"][:, None]
        s = torch.where(keep[:, None, None, :], s, -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(dim=-1, keepdim=True)
    o = (p @ v.float().transpose(1, 2)) / torch.where(total > 0, total, 1.0)  # a row without keys: zeros
    return o.to(torch.bfloat16).view(b, hq, sq, d).transpose(1, 2).contiguous()


def run(state):
    op = state["case"]["op"]
    if own:
        import diffusion_transformer_w4a4_b200 as svdq

        if op == "fp8_linear":
            return state["layer"].forward(state["x"])
        if op == "qk_norm_rope":
            return list(svdq.svdq_qk_norm_rope(state["q"], state["k"], state["wq"], state["wk"], eps=1e-6,
                                               rope=state["table"], positions=state["pos"],
                                               pairs=state["case"]["pairs"]))
        return svdq.svdq_cross_attn(state["q"], state["k"], state["v"], kv_len=state["len"], kv_mask=state["mask"])
    return {"fp8_linear": _plain_fp8, "qk_norm_rope": _plain_qk, "cross_attention": _plain_attn}[op](state)


# ------------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "fp8_linear":
        m, k, n = case["m"], case["k"], case["n"]
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        return dict(bytes=2 * m * k + n * k + 4 * nb * kb + (2 * n if case["bias"] else 0) + 2 * m * n,
                    flops=2 * m * n * k)
    if case["op"] == "qk_norm_rope":
        b, s, d, rot = case["b"], case["s"], case["d"], case["rot"]
        elems = b * s * (case["hq"] + case["hk"]) * d
        table = 4 * rot * (min(8192, b * s) if case["positions"] else s) + (4 * b * s if case["positions"] else 0)
        return dict(bytes=4 * elems + 4 * d + (table if rot else 0), flops=7 * elems)
    b, sq, sk, hq, hk, d = (case[f] for f in ("b", "sq", "sk", "hq", "hk", "d"))
    share = 9 / 16 if case["keys"] == "len" else 0.8 if case["keys"] == "mask" else 1.0  # keys that count, mean
    keep = 4 * b if case["keys"] == "len" else b * sk if case["keys"] == "mask" else 0
    return dict(bytes=4 * b * sq * hq * d + 4 * b * sk * share * hk * d + keep, flops=4 * b * hq * sq * sk * share * d)


# ------------------------------------------------------------------------------------------------- definitions
def exact(case, seed):
    """The definition in binary64.  What an E4M3 code is rounded from is defined in binary32: the input times the
    reciprocal of its block's scale (a quotient of two bf16 values often lies on a border of two codes)."""
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "fp8_linear":
        m, k, n = case["m"], case["k"], case["n"]
        acc = torch.zeros(m, n, dtype=f, device="cuda")
        for j in range(-(-k // BLOCK)):
            xb = st["x"][:, j * BLOCK:(j + 1) * BLOCK].to(f)
            wb = st["wq"][:, j * BLOCK:(j + 1) * BLOCK].to(f)
            sx = (xb.abs().max(dim=1).values.clamp_min(AMAX_MIN) / FP8_MAX).float().to(f)
            q = (xb.float() * (1.0 / sx.float())[:, None]).to(f)
            # E4M3: 3 fraction bits down to the exponent -6, steps of 2^-9 below; ties to even
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
            q = (torch.round(q / step) * step).clamp(-FP8_MAX, FP8_MAX)
            sw = st["ws"][:, j].to(f)[torch.arange(n, device="cuda") // BLOCK]
            acc += (q * sx[:, None]) @ (wb * sw[:, None]).t()
        return acc if st["bias"] is None else acc + st["bias"].to(f)
    if case["op"] == "qk_norm_rope":
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            y = x.to(f)
            y = w.to(f) * y / torch.sqrt(y.square().sum(dim=-1, keepdim=True) / case["d"] + 1e-6)
            rot = case["rot"]
            if rot:
                at = st["pos"].long() if st["pos"] is not None else \
                    torch.arange(case["s"], device="cuda").expand(case["b"], -1)
                turn = torch.view_as_complex(st["table"].to(f))[at][:, :, None, :]
                first = torch.arange(0, rot, 2, device="cuda") if case["pairs"] == "interleaved" else \
                    torch.arange(rot // 2, device="cuda")
                second = first + (1 if case["pairs"] == "interleaved" else rot // 2)
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return out
    b, sq, hq, d = st["q"].shape
    hk = case["hk"]
    out = torch.zeros(b, sq, hq, d, dtype=f, device="cuda")
    for i in range(b):
        at = torch.arange(case["sk"], device="cuda")
        if st["len"] is not None:
            at = at[:int(st["len"][i])]
        if st["mask"] is not None:
            at = at[st["mask"][i] != 0]
        if not at.numel():
            continue
        for h in range(hq):
            kh, vh = st["k"][i, at, h * hk // hq].to(f), st["v"][i, at, h * hk // hq].to(f)
            out[i, :, h] = torch.softmax(st["q"][i, :, h].to(f) @ kh.t() * d ** -0.5, dim=-1) @ vh
    return out
