"""The attention sublayers as they are used: projections, head norms with rotation, attention and output projection in
one run, each step against binary64 on what the step before produced (bounds derived in attn_cases); the classes
against the same calls made one by one, on a side stream, captured and replayed; a packed block with FP8 attention
projections through the compression tool."""
import numpy as np
import pytest

import attn_cases as ac

pytestmark = pytest.mark.gpu


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


def _fp8(g, K, N):
    """(layer, plain(x) -> (y, bound)) of a random FP8 layer."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    w, b = ac.bf16(g, N, K, scale=0.03), ac.bf16(g, N, scale=0.1)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    codes, scales = svdq.svdq_fp8_prepare(bits(w))
    qw = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().cuda()
    sw = torch.from_numpy(scales).cuda()
    return svdq.Fp8Linear(codes, scales, bits(b), device="cuda:0"), \
        lambda x: ac.fp8_linear(*ac.fp8_quantize(x.reshape(-1, K)), qw, sw, b)


@pytest.mark.parametrize("b,s,sk,width,ctx,heads,kv_heads,dim", [
    (2, 200, 77, 384, 272, 6, 6, 64), (1, 1, 300, 256, 144, 8, 2, 40), (3, 700, 130, 512, 512, 12, 12, 72)])
def test_cross_attention_step_by_step(b, s, sk, width, ctx, heads, kv_heads, dim):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200.attention import CrossAttention, rope_table

    g = ac.generator(s)
    to_q, plain_q = _fp8(g, width, heads * dim)
    to_kv, plain_kv = _fp8(g, ctx, 2 * kv_heads * dim)
    to_out, plain_out = _fp8(g, heads * dim, width)
    wq, wk = ac.bf16(g, dim) + 1, ac.bf16(g, dim) + 1
    x, states = ac.bf16(g, b, s, width), ac.bf16(g, b, sk, ctx)
    table = rope_table(s, dim, device="cuda:0")
    kv_len = torch.tensor([sk, 0, sk // 2][:b], dtype=torch.int32, device="cuda")
    mod = CrossAttention(to_q, to_kv, to_out, heads, kv_heads, wq, wk)
    # the calls one by one, each checked on its own input
    kv = to_kv(states)
    ac.check(kv, *plain_kv(states))
    kv = kv.view(b, sk, 2, kv_heads, dim)
    k, v = kv[:, :, 0], kv[:, :, 1]
    kn = svdq.svdq_qk_norm_rope(k, None, wk)
    ac.check(kn, *ac.norm_rope(k, wk, 1e-6, None, None, "interleaved"))
    q = to_q(x)
    ac.check(q, *plain_q(x))
    q = q.view(b, s, heads, dim)
    qn = svdq.svdq_qk_norm_rope(q, None, wq, rope=table)
    ac.check(qn, *ac.norm_rope(q, wq, 1e-6, table, None, "interleaved"))
    o = svdq.svdq_cross_attn(qn, kn, v, kv_len=kv_len)
    ac.check(o, *ac.attention(qn, kn, v, kv_len, None, ac.inv_sqrt(dim)))
    y = to_out(o.view(b, s, -1))
    ac.check(y, *plain_out(o))
    # the same through the class: eager, on a side stream, and captured with the keys and values kept
    y = y.view(b, s, width)
    keys_values = mod.encode(states)
    assert torch.equal(mod(x, keys_values, rope=table, kv_len=kv_len), y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mod(x, keys_values, rope=table, kv_len=kv_len, stream=side)
    side.synchronize()
    assert torch.equal(got, y)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mod(xs, keys_values, rope=table, kv_len=kv_len)
    xs.copy_(x.flip(1))
    want = mod(xs, keys_values, rope=table, kv_len=kv_len).clone()
    for src, ref in ((x, y), (x.flip(1), want)):
        xs.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert int(svdq.attn_status().item()) == 0
    assert to_q.status(b * s) == to_kv.status(b * sk) == to_out.status(b * s) == 0


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
def test_self_attention_matches_its_calls(pairs):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200.attention import SelfAttention, rope_table

    g = ac.generator(3)
    b, s, heads, dim, width = 2, 150, 4, 128, 512
    to_qkv, _ = _fp8(g, width, 3 * heads * dim)
    to_out, _ = _fp8(g, heads * dim, width)
    mod = SelfAttention(to_qkv, to_out, heads, pairs=pairs)
    x, table = ac.bf16(g, b, s, width), rope_table(s, dim, device="cuda:0")
    mask = torch.rand(b, s, generator=g, device="cuda") < 0.7
    got = mod(x, rope=table, kv_mask=mask)
    q, k, v = to_qkv(x).view(b, s, 3, heads, dim).unbind(2)
    q, k = svdq.svdq_qk_norm_rope(q, k, rope=table, pairs=pairs)
    o = svdq.svdq_cross_attn(q, k, v, kv_mask=mask)
    assert torch.equal(got, to_out(o.reshape(b, s, -1)).view(b, s, width))


@pytest.mark.parametrize("rules", ["svdq", "fp8"])
def test_packed_block_runs(tmp_path, rules):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200 import compress

    layers, inputs = compress.synthetic_flux_block(tokens=100, seed=2, width=768, heads=6)
    path = str(tmp_path / "block.svdq")
    compress.compress(layers, inputs, path, rules=compress.FP8_ATTENTION_RULES if rules == "fp8" else compress.DEFAULT_RULES,
                      attention=dict(heads=6, theta=10000.0))
    block = compress.load_block(path, "cuda:0")
    assert isinstance(block.attention.to_qkv, svdq.Fp8Linear if rules == "fp8" else svdq.SvdqLinear)
    x = torch.from_numpy(inputs[layers[1].name].view(np.int16)).view(torch.bfloat16).cuda()[None]
    y = block(x)
    h = block.attention(x, rope=block._table(100))
    m = torch.empty(100, 768, dtype=torch.bfloat16, device="cuda")
    svdq.svdq_mlp_forward(block.up.handle, block.down.handle, h, 100, m, block.up.workspace(100),
                          block.down.workspace(100))
    assert torch.equal(y[0], m)
    rel = compress.run_packed_block(path, layers, inputs)
    print(rules, "relative error against the dense block", rel)
    assert np.isfinite(rel)


def test_refusals():
    import torch

    from diffusion_transformer_w4a4_b200.attention import CrossAttention, SelfAttention

    g = ac.generator(5)
    to_qkv, _ = _fp8(g, 128, 3 * 4 * 32)
    to_q, _ = _fp8(g, 128, 4 * 32)
    to_kv, _ = _fp8(g, 64, 2 * 2 * 32)
    to_out, _ = _fp8(g, 4 * 32, 128)
    for bad in (lambda: SelfAttention(to_qkv, to_out, 5), lambda: SelfAttention(to_qkv, to_kv, 4),
                lambda: SelfAttention(to_qkv, to_out, 0), lambda: CrossAttention(to_q, to_kv, to_out, 4, 4),
                lambda: CrossAttention(to_q, to_kv, to_out, 4, 3), lambda: CrossAttention(to_q, to_kv, to_kv, 4, 2)):
        with pytest.raises(ValueError):
            bad()
    mod = CrossAttention(to_q, to_kv, to_out, 4, 2)
    kv = mod.encode(ac.bf16(g, 1, 9, 64))
    for bad in (lambda: mod(ac.bf16(g, 3, 128), kv), lambda: mod(ac.bf16(g, 1, 3, 64), kv),
                lambda: mod(ac.bf16(g, 2, 3, 128), kv), lambda: mod.encode(ac.bf16(g, 1, 9, 128))):
        with pytest.raises(ValueError):
            bad()
    assert mod(ac.bf16(g, 1, 0, 128), kv).shape == (1, 0, 128)
    assert torch.isfinite(mod(ac.bf16(g, 1, 3, 128), kv)).all()


def test_block_table_streams_and_capture(tmp_path):
    """The rotation table of a larger token count: complete before any stream may read it, never made in a capture."""
    import torch

    from diffusion_transformer_w4a4_b200 import compress

    layers, inputs = compress.synthetic_flux_block(tokens=100, seed=2, width=768, heads=6)
    path = str(tmp_path / "block.svdq")
    compress.compress(layers, inputs, path, rules=compress.FP8_ATTENTION_RULES, attention=dict(heads=6, theta=10000.0))
    block = compress.load_block(path, "cuda:0")
    x = torch.from_numpy(inputs[layers[1].name].view(np.int16)).view(torch.bfloat16).cuda()[None]
    short = x[:, :40].contiguous()
    y_short = block(short)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = block(x, stream=side)  # a longer table, on another stream
    again = block(x)
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    assert torch.equal(y_short, block(short))  # the longer table's first rows are the shorter one's
    longer = torch.cat((x, x), 1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(graph):
            block(longer)
    torch.cuda.synchronize()
    want = block(longer)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out.copy_(block(longer))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_many_calls_at_once():
    """Every kind of launch (persistent, clusters, few tokens) on four streams at once: the bits of one call alone."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(41)
    calls = []
    for M, K, N in ((3, 2048, 1024), (50, 2048, 768), (100, 4096, 512), (700, 512, 2048)):
        lin, _ = _fp8(g, K, N)
        x = ac.bf16(g, M, K)
        calls.append(lambda lin=lin, x=x: lin(x))
    for b, sq, sk, hq, hk, d in ((2, 1, 2000, 8, 4, 128), (1, 300, 4100, 6, 2, 128), (1, 100, 3000, 4, 4, 64),
                                 (2, 1500, 200, 16, 16, 64)):
        q, k, v = ac.bf16(g, b, sq, hq, d), ac.bf16(g, b, sk, hk, d), ac.bf16(g, b, sk, hk, d)
        calls.append(lambda q=q, k=k, v=v: svdq.svdq_cross_attn(q, k, v))
    q, k = ac.bf16(g, 2, 900, 5, 64), ac.bf16(g, 2, 900, 3, 64)
    calls.append(lambda: torch.cat(svdq.svdq_qk_norm_rope(q, k), 2))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(8):
        for i, c in enumerate(calls):  # a call always on one stream: a layer's workspace serves one call at a time
            with torch.cuda.stream(streams[i % 4]):
                got.append((i, c()))
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, want[i]), i
    assert int(svdq.attn_status().item()) == 0
