"""svdq_cross_attn against its definition in binary64 (bounds derived in attn_cases): head sizes and groups, query and
key counts from one to several tiles, both ways of spreading the work, key lengths and masks (none left, NaN behind
them), strides, broadcast, streams, graph replay, wait limit and refusals."""
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


def _run(b, sq, sk, hq, hk, d, kv_len=None, kv_mask=None, scale=None, seed=0, spread=1.0):
    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(seed + b + sq + sk + hq + d)
    q, k, v = ac.bf16(g, b, sq, hq, d, scale=spread), ac.bf16(g, b, sk, hk, d), ac.bf16(g, b, sk, hk, d)
    o = svdq.svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=kv_mask, scale=scale)
    assert int(svdq.attn_status().item()) == 0
    rel = ac.check(o, *ac.attention(q, k, v, kv_len, kv_mask, scale or ac.inv_sqrt(d)))
    print(b, sq, sk, hq, hk, d, rel)
    return q, k, v, o


@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 80, 96, 112, 120, 128])
@pytest.mark.parametrize("sq,sk", [(1, 1), (5, 130), (130, 257), (300, 77)])
def test_head_sizes(d, sq, sk):
    _run(2, sq, sk, 3, 3, d)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (3, 1), (6, 2), (24, 8), (5, 1), (12, 1), (40, 2), (130, 1), (256, 2)])
@pytest.mark.parametrize("sq", [1, 3, 200])
def test_shared_key_heads(hq, hk, sq):
    _run(1, sq, 200, hq, hk, 64)


@pytest.mark.parametrize("hq,hk", [(6, 3), (9, 3), (16, 4), (20, 4), (48, 4), (32, 2), (96, 3), (66, 2), (260, 2)])
@pytest.mark.parametrize("d", [40, 128])
def test_shared_key_heads_many_rows(hq, hk, d):
    """Pairs of tiles (256 rows of tokens and heads to each of the 148 SMs at least) whose rows mix tokens and heads:
    groups that divide a warp's 32 rows, and groups that do not."""
    _run(2, -(-150 * 256 // (2 * hq)) + 5, 130, hq, hk, d)


@pytest.mark.parametrize("sk", [1, 2, 127, 128, 129, 255, 256, 257, 384, 511, 513, 640, 1000, 1536, 2049, 4100])
@pytest.mark.parametrize("sq", [1, 100])
def test_key_counts_few_rows(sq, sk):
    _run(1, sq, sk, 2, 1, 128)  # split over streams and CTAs


@pytest.mark.parametrize("sk", [1, 100, 128, 129, 256, 300, 385, 512, 700, 1100])
@pytest.mark.parametrize("d", [64, 128])
def test_key_counts_many_rows(sk, d):
    _run(2, 1200, sk, 16, 16, d)  # pairs of query tiles, several items to a CTA


@pytest.mark.parametrize("sq", [127, 128, 129, 255, 256, 257, 383, 385])
def test_query_counts_many_rows(sq):
    _run(5, sq, 200, 32, 32, 64)


@pytest.mark.parametrize("b,sq,sk,hq,hk,d", [(1, 500, 4600, 24, 24, 128), (2, 300, 4100, 9, 3, 72), (1, 257, 1500, 12, 12, 128),
                                             (1, 200, 9000, 4, 2, 64), (1, 1000, 2050, 16, 16, 128)])
def test_pairs_over_split_keys(b, sq, sk, hq, hk, d):
    """Too few pairs of tiles for the SMs and many keys: the keys go over a cluster; some of its CTAs have none."""
    import torch

    _run(b, sq, sk, hq, hk, d)
    g = ac.generator(24)
    mask = torch.rand(b, sk, generator=g, device="cuda") < 0.6
    mask[:, 128:1000] = False
    _run(b, sq, sk, hq, hk, d, kv_mask=mask)
    for n in (0, 1, 129, sk // 2):
        kv_len = torch.full((b,), n, dtype=torch.int32, device="cuda")
        kv_len[0] = min(n, 200)
        o = _run(b, sq, sk, hq, hk, d, kv_len=kv_len)[3]
        if n == 0:
            assert not o.any()


def test_long_keys_split():
    _run(1, 1, 40000, 8, 1, 64)
    _run(2, 2, 20001, 2, 2, 128)


@pytest.mark.parametrize("shape", [(3, 10, 300, 4, 2, 64), (3, 700, 300, 24, 24, 64), (3, 1, 1500, 6, 2, 128),
                                   (3, 500, 300, 40, 20, 128)])
def test_key_lengths(shape):
    import torch

    for lens in ([300, 1, 129], [0, 128, 256], [-5, 10 ** 6, 0]):
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q, k, v, o = _run(*shape, kv_len=kv_len)
        for i, n in enumerate(lens):
            if n <= 0:
                assert not o[i].any()


@pytest.mark.parametrize("shape", [(4, 10, 300, 4, 2, 64), (4, 600, 300, 24, 24, 72), (4, 1, 1500, 6, 2, 128),
                                   (4, 300, 515, 40, 20, 128)])
def test_key_masks(shape):
    import torch

    b, _, sk = shape[:3]
    g = ac.generator(3)
    mask = (torch.rand(b, sk, generator=g, device="cuda") < 0.5).to(torch.uint8)
    mask[0] = 0  # nothing left
    mask[1, :-1] = 0  # only the last key
    mask[2, 128:256] = 0  # a whole tile
    mask[3] *= 255  # any nonzero byte counts
    q, k, v, o = _run(*shape, kv_mask=mask)
    assert not o[0].any()
    kv_len = torch.tensor([sk, sk, 200, 100], dtype=torch.int32, device="cuda")
    q, k, v, o = _run(*shape, kv_mask=mask, kv_len=kv_len)
    import diffusion_transformer_w4a4_b200 as svdq

    again = svdq.svdq_cross_attn(q, k, v, kv_mask=mask.bool(), kv_len=kv_len)
    assert torch.equal(o, again)


@pytest.mark.parametrize("sq,hq,hk", [(4, 4, 2), (700, 24, 24)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
def test_masked_keys_have_no_influence(sq, hq, hk, d, bad):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(11)
    b, sk = 3, 400
    q, k, v = ac.bf16(g, b, sq, hq, d), ac.bf16(g, b, sk, hk, d), ac.bf16(g, b, sk, hk, d)
    mask = (torch.rand(b, sk, generator=g, device="cuda") < 0.7)
    mask[1] = False
    kv_len = torch.tensor([400, 333, 130], dtype=torch.int32, device="cuda")
    want = svdq.svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=mask)
    gone = ~mask | (torch.arange(sk, device="cuda")[None] >= kv_len[:, None])
    k, v = k.clone(), v.clone()
    k[gone], v[gone] = bad, bad
    assert torch.equal(want, svdq.svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=mask))
    # by length alone
    k[torch.arange(sk, device="cuda")[None] < kv_len[:, None]] = 0.5
    v[torch.arange(sk, device="cuda")[None] < kv_len[:, None]] = 0.25
    o = svdq.svdq_cross_attn(q, k, v, kv_len=kv_len)
    assert (o == 0.25).all()


@pytest.mark.parametrize("sq,h,d", [(300, 4, 128), (100, 3, 128), (100, 3, 64), (2, 4, 72), (300, 6, 40)])
def test_masked_keys_have_no_influence_on_split_keys(sq, h, d):
    """The same where clusters split the keys: NaN and infinities behind a length, and behind masks, of whole tiles too."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(25)
    b, sk = 2, 3000
    q, k, v = ac.bf16(g, b, sq, h, d), ac.bf16(g, b, sk, h, d), ac.bf16(g, b, sk, h, d)
    mask = torch.rand(b, sk, generator=g, device="cuda") < 0.7
    mask[:, 256:1100] = False
    kv_len = torch.tensor([2900, 1301], dtype=torch.int32, device="cuda")
    want = svdq.svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=mask)
    ac.check(want, *ac.attention(q, k, v, kv_len, mask, ac.inv_sqrt(d)))
    by_len = svdq.svdq_cross_attn(q, k, v, kv_len=kv_len)
    past = torch.arange(sk, device="cuda")[None] >= kv_len[:, None]
    for bad in (float("nan"), float("inf"), -3.0e38):
        kk, vv = k.clone(), v.clone()
        kk[past], vv[past] = bad, bad
        assert torch.equal(by_len, svdq.svdq_cross_attn(q, kk, vv, kv_len=kv_len))
        kk[~mask], vv[~mask] = bad, bad
        assert torch.equal(want, svdq.svdq_cross_attn(q, kk, vv, kv_len=kv_len, kv_mask=mask))


def test_nan_in_a_counting_key_shows():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(12)
    q, k, v = (ac.bf16(g, 2, n, 4, 64) for n in (20, 300, 300))
    k[0, 7, 1, 3] = float("nan")
    o = svdq.svdq_cross_attn(q, k, v)
    assert torch.isnan(o[0, :, 1]).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(o[0, :, [0, 2, 3]]).all()


@pytest.mark.parametrize("sq,h", [(3, 4), (100, 2), (600, 24)])
@pytest.mark.parametrize("masked", [False, True])
def test_scores_of_minus_infinity(sq, h, masked):
    """Keys with a score of -inf have no share, however large their values; a row of nothing else gives 0."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    sk, d = 400, 64
    q = torch.full((2, sq, h, d), 3.0e38, dtype=torch.bfloat16, device="cuda")
    k = torch.full((2, sk, h, d), -3.0e38, dtype=torch.bfloat16, device="cuda")
    v = torch.full((2, sk, h, d), 3.0e38, dtype=torch.bfloat16, device="cuda")
    on = torch.rand(sk, generator=ac.generator(21), device="cuda") < 0.5
    k[1, on], v[1, on] = 0.0, 1.0  # scores of 0 and values of 1 among them
    o = svdq.svdq_cross_attn(q, k, v, kv_mask=torch.ones(2, sk, dtype=torch.uint8, device="cuda") if masked else None)
    assert not o[0].any()
    assert (o[1] == 1).all()


@pytest.mark.parametrize("sq,h", [(3, 4), (100, 2), (600, 24)])
def test_scores_past_binary32(sq, h):
    """A score, or scale times a score, past binary32: NaN in its rows, and nothing else."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(22)
    q, k, v = (ac.bf16(g, 2, n, h, 64) for n in (sq, 300, 300))
    big = q.abs()
    big[1], pos = 0.0, k.abs()
    o = svdq.svdq_cross_attn(big, pos, v, scale=3e37)
    assert torch.isnan(o[0]).all()
    ac.check(o[1:], *ac.attention(big[1:], pos[1:], v[1:], None, None, 3e37))
    k[0, 250], q[:, :, 0] = 3.0e38, 3.0e38  # the first head's rows reach +inf
    o = svdq.svdq_cross_attn(q, k, v)
    assert torch.isnan(o[0, :, 0]).all()
    assert torch.isfinite(o[1, :, 1:]).all()


@pytest.mark.parametrize("sq", [3, 600])
def test_sharp_and_growing_scores(sq):
    """Scores far apart, and rising from tile to tile, so that the running maximum moves often."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    _run(1, sq, 700, 24, 24, 64, spread=30.0)
    _run(1, sq, 700, 24, 24, 128, scale=3.0)
    _run(1, sq, 700, 24, 24, 64, scale=1e-6)
    g = ac.generator(13)
    q, k, v = ac.bf16(g, 1, sq, 24, 64).abs(), ac.bf16(g, 1, 900, 24, 64).abs(), ac.bf16(g, 1, 900, 24, 64)
    ramp = torch.linspace(0.1, 20, 900, device="cuda")[None, :, None, None]
    for kk in (k * ramp, k * ramp.flip(1), -k * ramp):
        kk = kk.to(torch.bfloat16)
        o = svdq.svdq_cross_attn(q, kk, v)
        ac.check(o, *ac.attention(q, kk, v, None, None, 0.125))


@pytest.mark.parametrize("sq,hq,hk", [(9, 6, 2), (530, 24, 24)])
def test_strides_and_broadcast(sq, hq, hk):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(14)
    b, sk, d = 2, 200, 64
    q = ac.bf16(g, b, hq, sq, d).transpose(1, 2)  # heads first
    kv = ac.bf16(g, b, sk, 2, hk, d)  # fused projection
    k, v = kv[:, :, 0], kv[:, :, 1]
    buf = torch.full((b, hq, sq, d + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[..., 8:8 + d].transpose(1, 2)
    svdq.svdq_cross_attn(q, k, v, out=out)
    ac.check(out, *ac.attention(q, k, v, None, None, 0.125))
    assert (buf[..., :8] == 3).all() and (buf[..., 8 + d:] == 3).all()
    one_k, one_v = ac.bf16(g, 1, sk, 1, d).expand(b, sk, hk, d), ac.bf16(g, 1, sk, hk, d).expand(b, sk, hk, d)
    mask = (torch.rand(1, sk, generator=g, device="cuda") < 0.5).expand(b, sk)
    ac.check(svdq.svdq_cross_attn(q, one_k, one_v, kv_mask=mask), *ac.attention(q, one_k, one_v, None, mask, 0.125))
    one_q = ac.bf16(g, b, sq, 1, d).expand(b, sq, hq, d)
    ac.check(svdq.svdq_cross_attn(one_q, k, v), *ac.attention(one_q, k, v, None, None, 0.125))


def test_no_keys_and_no_queries():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    for sq, h in ((4, 2), (700, 48)):
        q = torch.full((2, sq, h, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        kv = torch.empty(2, 0, h, 64, dtype=torch.bfloat16, device="cuda")
        assert not svdq.svdq_cross_attn(q, kv, kv).any()
        assert svdq.svdq_cross_attn(q[:, :0], q, q).shape == (2, 0, h, 64)


@pytest.mark.parametrize("sq,hq", [(2, 4), (600, 40)])
def test_equal_bits_streams_and_graphs(sq, hq):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(15)
    q, k, v = ac.bf16(g, 2, sq, hq, 128), ac.bf16(g, 2, 1100, hq, 128), ac.bf16(g, 2, 1100, hq, 128)
    q2 = ac.bf16(g, 2, sq, hq, 128)
    want, want2 = svdq.svdq_cross_attn(q, k, v), svdq.svdq_cross_attn(q2, k, v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]  # two calls at once
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs += [svdq.svdq_cross_attn(q, k, v) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)
    o = torch.empty_like(want)
    qq = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svdq.svdq_cross_attn(qq, k, v, out=o)
    for src, ref in ((q2, want2), (q, want)):
        qq.copy_(src)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref)


@pytest.mark.parametrize("b,sq,sk,hq,hk,d", [(2, 900, 300, 24, 8, 72), (1, 3, 1030, 6, 2, 64), (2, 100, 700, 3, 1, 64),
                                             (2, 700, 400, 40, 8, 128)])
def test_equal_bits_whatever_ran_before(b, sq, sk, hq, hk, d):
    """Groups of heads that leave rows of a tile unused: what an earlier call left in shared memory changes nothing."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(23)
    q, k, v = ac.bf16(g, b, sq, hq, d), ac.bf16(g, b, sk, hk, d), ac.bf16(g, b, sk, hk, d)
    want = svdq.svdq_cross_attn(q, k, v)
    for spread in (0.0, 1.0, 30.0, 1e4, 1e20):
        other = ac.bf16(g, 8, 1000, 24, 128, scale=spread)
        svdq.svdq_cross_attn(other, other, other)  # every SM's shared memory
        assert torch.equal(want, svdq.svdq_cross_attn(q, k, v))


@pytest.mark.parametrize("sq,hq,sk", [(2, 4, 3000), (600, 40, 600)])
def test_wait_limit_reports_and_recovers(sq, hq, sk):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(16)
    q, k, v = ac.bf16(g, 1, sq, hq, 64), ac.bf16(g, 1, sk, hq, 64), ac.bf16(g, 1, sk, hq, 64)
    want = svdq.svdq_cross_attn(q, k, v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        svdq.svdq_set_wait_limit(1)
        svdq.svdq_cross_attn(q, k, v, status=status)
        torch.cuda.synchronize()
    finally:
        svdq.svdq_set_wait_limit(0)
    assert int(status.item()) == svdq.SVDQ_ERR_TIMEOUT
    assert torch.equal(want, svdq.svdq_cross_attn(q, k, v))
    assert int(svdq.attn_status().item()) == 0


def test_refusals():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(17)
    q, k = ac.bf16(g, 2, 4, 4, 64), ac.bf16(g, 2, 9, 2, 64)
    ln = torch.ones(2, dtype=torch.int32, device="cuda")
    m = torch.ones(2, 9, dtype=torch.uint8, device="cuda")
    for args, kw in (((q.half(), k, k), {}), ((q[0], k, k), {}), ((q, k.cpu(), k), {}), ((q, k, k[:, :5]), {}),
                     ((q, k[:1], k[:1]), {}), ((q, k[..., :32], k[..., :32]), {}), ((q.transpose(2, 3), k, k), {}),
                     ((q, k, k), dict(kv_len=ln.long())), ((q, k, k), dict(kv_len=ln[:1])),
                     ((q, k, k), dict(kv_len=ln.cpu())), ((q, k, k), dict(kv_mask=m[:, :5])),
                     ((q, k, k), dict(kv_mask=m.float())), ((q, k, k), dict(kv_mask=m.t().contiguous().t())),
                     ((q, k, k), dict(out=q[:1])), ((q, k, k), dict(out=q.float())),
                     ((q, k, k), dict(status=ln.long()))):
        with pytest.raises(ValueError):
            svdq.svdq_cross_attn(*args, **kw)
    wide = ac.bf16(g, 2, 4, 4, 136)
    for args, kw in (((q[:, :, :3], k, k), {}), ((wide, wide, wide), {}), ((q, k, k), dict(scale=0.0)),
                     ((q, k, k), dict(scale=-1.0)), ((q[..., :60], k[..., :60], k[..., :60]), {}),
                     ((q[..., 4:], k[..., 4:], k[..., 4:]), {}),
                     ((q, k, k), dict(out=q[:, :1].expand(2, 4, 4, 64)))):
        with pytest.raises(svdq.SvdqError) as e:
            svdq.svdq_cross_attn(*args, **kw)
        assert e.value.status == svdq.SVDQ_ERR_INVALID_ARG
