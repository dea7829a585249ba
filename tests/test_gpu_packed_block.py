"""A packed block, loaded and run: each step of it against binary64 on what the step before gave, with rotation table and
slices made here, the layers' arrays read from the file, and the norm weights that were packed; the whole against the
dense block."""
import numpy as np
import pytest

import attn_cases as ac

pytestmark = pytest.mark.gpu

TOKENS, WIDTH, HEADS = 100, 768, 6
DIM = WIDTH // HEADS
PREFIX = "transformer_blocks.0."
# Four-bit weights and activations are off by about a tenth each (half of E2M1's steps, on average), an unrelated result
# by the square root of 2 or more: what is wired wrongly shows at this distance, what is rounded does not.
FAR = 0.5


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200 import build

    build.build()
    assert torch.cuda.is_available()
    assert svdq.svdq_device_check(0) == svdq.SVDQ_OK, "needs an sm_100a device"
    torch.cuda.set_device(0)
    svdq.attn_status()


class _Spy:
    """A layer that keeps what goes in and comes out."""

    def __init__(self, layer):
        self.layer, self.K, self.N, self.device = layer, layer.K, layer.N, layer.device

    def forward(self, x):
        self.x = x.clone()
        self.y = self.layer.forward(x)
        return self.y


def _norms(g):
    import torch

    w = [(ac.bf16(g, DIM) * 0.3 + 1).to(torch.bfloat16) for _ in range(2)]
    return w, [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in w]


def _dense(spec, x):
    import torch

    f = lambda b: torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).cuda().double()
    return x.double() @ f(spec.W).t() + f(spec.bias)


def _check_layer(spec, arrays, kind, x, y):
    """y of a layer for x: within the bound of the packed arrays (FP8), or near the dense one (W4A4)."""
    import torch

    x, y = x.reshape(-1, x.shape[-1]), y.reshape(-1, y.shape[-1])
    want = _dense(spec, x)
    assert float((y.double() - want).norm() / want.norm()) < FAR
    if kind == "fp8":
        qw = torch.from_numpy(arrays["wcodes"]).view(torch.float8_e4m3fn).double().cuda()
        sw = torch.from_numpy(arrays["wscales"]).cuda()
        b = torch.from_numpy(arrays["bias"].view(np.int16)).view(torch.bfloat16).cuda()
        ac.check(y, *ac.fp8_linear(*ac.fp8_quantize(x), qw, sw, b))


def _check_attention(block, weights, x, table, at=None, **kw):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    spy_in, spy_out = _Spy(block.attention.to_qkv), _Spy(block.attention.to_out)
    block.attention.to_qkv, block.attention.to_out = spy_in, spy_out
    try:
        y = block(x, **kw)
    finally:
        block.attention.to_qkv, block.attention.to_out = spy_in.layer, spy_out.layer
    b, s = x.shape[:2]
    fresh = spy_in.layer.forward(x).view(b, s, 3, HEADS, DIM)  # (the class normalises what the spy kept in place)
    q, k, v = fresh[:, :, 0], fresh[:, :, 1], fresh[:, :, 2]
    qn, kn = svdq.svdq_qk_norm_rope(q, k, *weights, rope=table, positions=at)
    ac.check(qn, *ac.norm_rope(q, weights[0], 1e-6, table, at, "interleaved"))
    ac.check(kn, *ac.norm_rope(k, weights[1], 1e-6, table, at, "interleaved"))
    ac.check(spy_out.x.view(b, s, HEADS, DIM), *ac.attention(qn, kn, v, None, None, ac.inv_sqrt(DIM)))
    return y, fresh, spy_out


@pytest.mark.parametrize("kind", ["svdq", "fp8"])
@pytest.mark.parametrize("weighted", [False, True])
def test_step_by_step(tmp_path, kind, weighted):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200 import compress

    weights, bits = _norms(ac.generator(7))
    norms = dict(q_norm=bits[0], k_norm=bits[1]) if weighted else {}
    weights = weights if weighted else [None, None]
    layers, inputs = compress.synthetic_flux_block(tokens=TOKENS, seed=2, width=WIDTH, heads=HEADS, **norms)
    path = str(tmp_path / "block.svdq")
    compress.compress(layers, inputs, path, rules=compress.FP8_ATTENTION_RULES if kind == "fp8" else compress.DEFAULT_RULES,
                      attention=dict(heads=HEADS, theta=10000.0, **norms))
    block = compress.load_block(path, "cuda:0")
    arrays = compress.read_packed(path)[1]
    spec = {s.name.removeprefix(PREFIX): s for s in layers}
    x = torch.from_numpy(inputs[PREFIX + "attn.to_qkv"].view(np.int16)).view(torch.bfloat16).cuda()[None]
    table = ac.rope_table(TOKENS, DIM, "cuda")
    y, qkv, spy_out = _check_attention(block, weights, x, table)
    _check_layer(spec["attn.to_qkv"], arrays[PREFIX + "attn.to_qkv"], kind, x, qkv.reshape(TOKENS, -1))
    _check_layer(spec["attn.to_out.0"], arrays[PREFIX + "attn.to_out.0"], kind, spy_out.x, spy_out.y)
    up = _dense(spec["ff.net.0.proj"], spy_out.y.view(TOKENS, -1))
    down = _dense(spec["ff.net.2"], torch.nn.functional.gelu(up))
    assert float((y[0].double() - down).norm() / down.norm()) < FAR
    rel = compress.run_packed_block(path, layers, inputs)
    print(kind, weighted, "relative error against the dense block", rel)
    assert rel < FAR
    if weighted:  # not the block without the weights, nor with the two exchanged
        for other in ({}, dict(q_norm=bits[1], k_norm=bits[0])):
            compress.pack(str(tmp_path / "o.svdq"), *_repack(path, layers, kind), layers,
                          dict(heads=HEADS, theta=10000.0, **other))
            assert not torch.equal(compress.load_block(str(tmp_path / "o.svdq"), "cuda:0")(x), y)
    assert int(svdq.attn_status().item()) == 0


def _repack(path, layers, kind):
    from diffusion_transformer_w4a4_b200 import compress

    rules = compress.FP8_ATTENTION_RULES if kind == "fp8" else compress.DEFAULT_RULES
    return compress.scan(layers, rules), compress.read_packed(path)[1]


def test_rotation_by_the_callers_table(tmp_path):
    """A table of two axes' angles side by side, and positions in it, for a batch of two."""
    import torch

    from diffusion_transformer_w4a4_b200 import compress

    weights, bits = _norms(ac.generator(8))
    layers, inputs = compress.synthetic_flux_block(tokens=TOKENS, seed=2, width=WIDTH, heads=HEADS)
    path = str(tmp_path / "block.svdq")
    compress.compress(layers, inputs, path, rules=compress.FP8_ATTENTION_RULES,
                      attention=dict(heads=HEADS, theta=10000.0, q_norm=bits[0], k_norm=bits[1]))
    block = compress.load_block(path, "cuda:0")
    g = ac.generator(9)
    x = ac.bf16(g, 2, TOKENS, WIDTH)
    rows = torch.arange(TOKENS, device="cuda")
    one = ac.rope_table(10, DIM // 2, "cuda")
    table = torch.cat((one[rows // 10], one[rows % 10]), 1).contiguous()  # 10 x 10 patches
    _check_attention(block, weights, x, table, rope=table)
    pos = torch.randint(0, TOKENS, (2, TOKENS), generator=g, device="cuda", dtype=torch.int32)
    _check_attention(block, weights, x, table, pos, rope=table, positions=pos)
    with pytest.raises(ValueError, match="rope table"):
        block(x, positions=pos)
    with pytest.raises(ValueError):
        block(x, rope=table.double())
