"""svdq_qk_norm_rope against its definition in binary64 (bounds derived in attn_cases): head sizes, pairs, partial
rotation, positions, strides, in place, absent parts, positions outside the table, streams and graph replay."""
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


def _weights(g, d):
    return ac.bf16(g, d) * 0.2 + 1, ac.bf16(g, d)


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 8), (32, 32), (40, 40), (40, 24), (64, 64), (64, 16), (72, 72), (80, 40),
                                   (96, 96), (112, 56), (128, 128), (128, 64), (136, 136), (200, 104), (256, 256),
                                   (128, 0)])
def test_heads_and_pairs(d, rot, pairs):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(d + rot)
    b, s, hq, hk = 2, 37, 6, 2
    q, k = ac.bf16(g, b, s, hq, d), ac.bf16(g, b, s, hk, d, scale=30.0)
    wq, wk = _weights(g, d)
    table = ac.rope_table(s + 5, rot, "cuda") if rot else None
    oq, ok = svdq.svdq_qk_norm_rope(q, k, wq, wk, eps=1e-5, rope=table, pairs=pairs)
    for got, x, w in ((oq, q, wq), (ok, k, wk)):
        ac.check(got, *ac.norm_rope(x, w, 1e-5, table, None, pairs))
    assert int(svdq.attn_status().item()) == 0
    assert torch.isfinite(oq).all()


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("d,rot", [(8, 8), (40, 24), (64, 64), (128, 128), (256, 128)])
@pytest.mark.parametrize("b,s,hq,hk", [(2, 148, 3, 1), (1, 297, 5, 2), (3, 592, 1, 1), (1, 1777, 17, 4), (2, 1000, 33, 3)])
def test_threads_to_a_token(b, s, hq, hk, d, rot, pairs):
    """Few tokens, some and many, with few heads and many: four warps to a token, two and one."""
    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(s + d)
    qkv = ac.bf16(g, b, s, hq + hk, d)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:]
    wq, wk = _weights(g, d)
    table = ac.rope_table(s, rot, "cuda")
    oq, ok = svdq.svdq_qk_norm_rope(q, k, wq, wk, rope=table, pairs=pairs)
    ac.check(oq, *ac.norm_rope(q, wq, 1e-6, table, None, pairs))
    ac.check(ok, *ac.norm_rope(k, wk, 1e-6, table, None, pairs))


@pytest.mark.parametrize("b,s,hq,hk", [(1, 1, 1, 1), (1, 1, 24, 24), (3, 333, 16, 4), (2, 1025, 40, 1), (1, 5, 100, 3)])
def test_fused_views_positions_in_place(b, s, hq, hk):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    d = 128
    g = ac.generator(s)
    qkv = ac.bf16(g, b, s, hq + 2 * hk, d)
    before = qkv.clone()
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    wq, wk = _weights(g, d)
    table = ac.rope_table(70000, d, "cuda")
    pos = torch.randint(0, 70000, (b, s), generator=g, device="cuda", dtype=torch.int32)
    oq, ok = svdq.svdq_qk_norm_rope(q, k, wq, wk, rope=table, positions=pos)
    ac.check(oq, *ac.norm_rope(q, wq, 1e-6, table, pos, "interleaved"))
    ac.check(ok, *ac.norm_rope(k, wk, 1e-6, table, pos, "interleaved"))
    assert torch.equal(qkv, before)
    svdq.svdq_qk_norm_rope(q, k, wq, wk, rope=table, positions=pos, out_q=q, out_k=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(qkv[:, :, hq + hk:], before[:, :, hq + hk:])  # the values stay


def test_heads_first_layout_broadcast_input_and_guard():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(5)
    d, table = 64, ac.rope_table(50, 64, "cuda")
    x = ac.bf16(g, 2, 8, 50, d)  # [B, H, S, D]
    buf = torch.full((2, 8, 50, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[..., 8:8 + d].transpose(1, 2)
    svdq.svdq_qk_norm_rope(x.transpose(1, 2), rope=table, out_q=out)
    ac.check(out, *ac.norm_rope(x.transpose(1, 2), None, 1e-6, table, None, "interleaved"))
    assert (buf[..., :8] == 7).all() and (buf[..., 8 + d:] == 7).all()
    one = ac.bf16(g, 1, 50, 1, d)
    wide = one.expand(3, 50, 5, d)
    got = svdq.svdq_qk_norm_rope(wide, rope=table)
    ac.check(got, *ac.norm_rope(wide, None, 1e-6, table, None, "interleaved"))


def test_zero_rows_large_values_and_nan():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(6)
    x = ac.bf16(g, 1, 8, 4, 128)
    x[0, 1, 2] = 0
    x[0, 2] *= 1e15
    x[0, 3] *= 1e-15
    x[0, 4, 1, 5] = float("nan")
    y = svdq.svdq_qk_norm_rope(x, eps=1e-6)
    assert not y[0, 1, 2].any()
    assert torch.isnan(y[0, 4, 1]).all()
    ref, bound = ac.norm_rope(x, None, 1e-6, None, None, "interleaved")
    keep = torch.ones(8, 4, dtype=torch.bool, device="cuda")
    keep[4, 1] = False
    ac.check(y[0][keep], ref[0][keep], bound[0][keep])


def test_position_outside_the_table_is_reported():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(7)
    q, k = ac.bf16(g, 1, 6, 3, 64), ac.bf16(g, 1, 6, 1, 64)
    table = ac.rope_table(10, 64, "cuda")
    pos = torch.tensor([[0, 10, 9, -1, 3, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    oq, ok = svdq.svdq_qk_norm_rope(q, k, rope=table, positions=pos, status=status)
    assert int(status.item()) == svdq.SVDQ_ERR_INVALID_ARG
    bad = torch.tensor([False, True, False, True, False, True], device="cuda")
    for got, x in ((oq, q), (ok, k)):
        assert torch.isnan(got[0, bad]).all()
        fine = pos.clamp(0, 9)
        ref, bound = ac.norm_rope(x, None, 1e-6, table, fine, "interleaved")
        ac.check(got[0, ~bad], ref[0, ~bad], bound[0, ~bad])


def test_stream_graph_and_empty():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(8)
    table = ac.rope_table(64, 128, "cuda")
    xs = [ac.bf16(g, 2, 64, 8, 128) for _ in range(2)]
    want = [svdq.svdq_qk_norm_rope(x, rope=table) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.empty_like(want[0])
    svdq.svdq_qk_norm_rope(xs[0], rope=table, out_q=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svdq.svdq_qk_norm_rope(x, rope=table, out_q=y)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    assert svdq.svdq_qk_norm_rope(x[:, :0], rope=table).shape == (2, 0, 8, 128)


def test_refusals():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(9)
    q = ac.bf16(g, 2, 10, 4, 64)
    table = ac.rope_table(10, 64, "cuda")
    pos = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    w = ac.bf16(g, 64)
    for kw in (dict(rope=table[:, :, :1]), dict(rope=table.double()), dict(rope=table.cpu()), dict(positions=pos),
               dict(rope=table, positions=pos.long()), dict(rope=table, positions=pos[:, :5]), dict(q_weight=w[:32]),
               dict(q_weight=w.float()), dict(out_q=q.float()), dict(out_q=q[:, :5]), dict(k=q[..., :32]),
               dict(k=q.cpu()), dict(rope=table, k=q[:, :5], positions=pos)):
        with pytest.raises(ValueError):
            svdq.svdq_qk_norm_rope(q, **kw)
    with pytest.raises(ValueError):
        svdq.svdq_qk_norm_rope(q.transpose(2, 3))
    for x, kw in ((q, dict(rope=table[:5])), (q[..., :60], {}), (q, dict(eps=-1.0))):
        with pytest.raises(svdq.SvdqError) as e:
            svdq.svdq_qk_norm_rope(x, **kw)
        assert e.value.status == svdq.SVDQ_ERR_INVALID_ARG
