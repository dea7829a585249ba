"""GPU parity of the FP8 layer (one scale for each block of 128) through the C ABI: activation codes and scales equal
to the definition's, bf16 Y within the bound derived in attn_cases; shapes with short last blocks, few and many
rows, every tile width; NaN and infinities; guard bands; wait limit; graph replay."""
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


def _bits(t):
    import torch

    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _layer(K, N, seed, bias=True):
    """(layer, codes' values, scales, bias): block ranges of W spread over several powers of ten."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(seed)
    w = ac.bf16(g, N, K, scale=0.02)
    w = (w.float() * torch.exp2(torch.randint(-6, 6, (N, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    b = ac.bf16(g, N, scale=0.1) if bias else None
    codes, scales = svdq.svdq_fp8_prepare(_bits(w))
    lin = svdq.Fp8Linear(codes, scales, None if b is None else _bits(b), device="cuda:0")
    qw = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().cuda()
    return lin, qw, torch.from_numpy(scales).cuda(), b


def _x(g, M, K):
    import torch

    x = ac.bf16(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 50
    return x


def _check(lin, x, y, qw, sw, b):
    import torch

    M = x.shape[0]
    assert lin.status(M) == 0
    qx, sx = ac.fp8_quantize(x)
    got = lin.read_act(M)
    np.testing.assert_array_equal(got["scales"], sx.cpu().numpy())
    codes = torch.from_numpy(got["codes"]).view(torch.float8_e4m3fn).double().cuda()
    assert torch.equal(codes, qx)
    ref, bound = ac.fp8_linear(qx, sx, qw, sw, b)
    return ac.check(y, ref, bound)


@pytest.mark.parametrize("M,K,N", [
    (1, 16, 8), (1, 128, 128), (2, 144, 136), (3, 3072, 64), (7, 1168, 2312), (16, 2048, 1024), (17, 4096, 264),
    (33, 256, 3072), (64, 400, 520), (65, 1536, 776), (77, 1168, 2312), (127, 128, 1000), (128, 512, 128),
    (129, 640, 4616), (300, 1152, 4608), (513, 2048, 1032), (1000, 272, 9216), (2100, 512, 2568),
    # few tokens: every token tile, clusters of each size, and inputs past what a cluster's table of scales holds
    (1, 12288, 3072), (15, 640, 136), (18, 6144, 1536), (32, 384, 9224), (48, 8208, 520), (64, 12288, 256),
    (33, 100096, 8), (5, 32768, 24)])
def test_parity(M, K, N):
    lin, qw, sw, b = _layer(K, N, M + K + N, bias=N % 16 == 0)
    x = _x(ac.generator(M), M, K)
    print(M, K, N, _check(lin, x, lin.forward(x), qw, sw, b))


@pytest.mark.parametrize("M", [1, 16, 31, 33, 64, 65, 128, 130, 300, 700])
@pytest.mark.parametrize("K,N", [(144, 72), (528, 328), (1040, 1000), (1552, 136), (2064, 3080), (4112, 520), (9744, 264)])
def test_every_split(M, K, N):
    """Tokens, inputs and outputs for which the inputs go over clusters of every size, tiles of every width."""
    lin, qw, sw, b = _layer(K, N, K + N)
    x = _x(ac.generator(M), M, K)
    y = lin.forward(x)
    _check(lin, x, y, qw, sw, b)
    assert (lin.forward(x) == y).all()


@pytest.mark.parametrize("K,N", [(3072, 12288), (12288, 3072)])
def test_mlp_shapes(K, N):
    lin, qw, sw, b = _layer(K, N, K)
    x = _x(ac.generator(1), 4608, K)
    print(K, N, _check(lin, x, lin.forward(x), qw, sw, b))


def test_zero_and_tiny_rows_and_no_tokens():
    import torch

    lin, qw, sw, b = _layer(512, 384, 5)
    x = torch.zeros(70, 512, dtype=torch.bfloat16, device="cuda")
    x[3, 5] = 1e-38
    x[4, 130:260] = 3e38
    y = lin.forward(x)
    assert torch.equal(y[:3], b.expand(3, -1)) and torch.equal(y[5:], b.expand(65, -1))
    _check(lin, x, y, qw, sw, b)
    assert lin.forward(x[:0]).shape == (0, 384)


def test_nan_and_infinity_stay_in_their_token():
    import torch

    lin, qw, sw, b = _layer(768, 256, 6)
    x = _x(ac.generator(2), 200, 768)
    clean = lin.forward(x).clone()
    x[7, 300] = float("nan")
    x[150, 0] = float("inf")
    y = lin.forward(x)
    assert lin.status(200) == 0
    bad = torch.zeros(200, dtype=torch.bool, device="cuda")
    bad[7] = bad[150] = True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("M,K,N", [(5, 400, 136), (130, 272, 264), (300, 512, 520)])
def test_writes_stay_inside(M, K, N):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    lin, qw, sw, b = _layer(K, N, 9)
    x = _x(ac.generator(3), M, K)
    want = lin.forward(x)
    pad, nb = 4096, lin.workspace_size(M)
    wbuf = torch.full((nb + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    ybuf = torch.full((2 * M * N + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    y = ybuf[pad:pad + 2 * M * N].view(torch.bfloat16).view(M, N)
    svdq.svdq_fp8_forward(lin.handle, x, M, y, wbuf[pad:pad + nb])
    assert torch.equal(y, want)
    for buf, n in ((wbuf, nb), (ybuf, 2 * M * N)):
        assert (buf[:pad] == 0xA5).all() and (buf[pad + n:] == 0xA5).all()


def test_equal_calls_give_equal_bits_on_a_side_stream():
    import torch

    lin, *_ = _layer(2048, 1024, 11)
    for M in (3, 40, 700):
        x = _x(ac.generator(M), M, 2048)
        want = lin.forward(x)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            again = [lin.forward(x) for _ in range(3)]
        s.synchronize()
        assert all(torch.equal(want, a) for a in again)
        explicit = lin.forward(x, out=torch.empty_like(want), stream=s)
        s.synchronize()
        assert torch.equal(want, explicit)


@pytest.mark.parametrize("M", [2, 300])
def test_graph_replay(M):
    import torch

    lin, *_ = _layer(768, 400, 13)
    xs = [_x(ac.generator(k), M, 768) for k in (1, 2)]
    want = [lin.forward(x).clone() for x in xs]
    x, y = xs[0].clone(), torch.empty_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out=y)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])


@pytest.mark.parametrize("M", [4, 512])
def test_wait_limit_reports_and_recovers(M):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    lin, qw, sw, b = _layer(2048, 1536, 17)
    x = _x(ac.generator(4), M, 2048)
    try:
        svdq.svdq_set_wait_limit(1)
        lin.forward(x)
        torch.cuda.synchronize()
        st = lin.status(M)
    finally:
        svdq.svdq_set_wait_limit(0)
    assert st == svdq.SVDQ_ERR_TIMEOUT
    _check(lin, x, lin.forward(x), qw, sw, b)


@pytest.mark.parametrize("M,K,N", [(100, 4096, 512), (400, 6144, 1536), (2, 4096, 512)])
def test_wait_limit_of_a_cluster(M, K, N):
    """A wait that runs out in one CTA of a cluster: reported, the others leave too, and the next call is right."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    lin, qw, sw, b = _layer(K, N, 31)
    x = _x(ac.generator(9), M, K)
    _check(lin, x, lin.forward(x), qw, sw, b)
    try:
        svdq.svdq_set_wait_limit(1)
        lin.forward(x)
        torch.cuda.synchronize()
        st = lin.status(M)
    finally:
        svdq.svdq_set_wait_limit(0)
    assert st == svdq.SVDQ_ERR_TIMEOUT
    _check(lin, x, lin.forward(x), qw, sw, b)


def test_refusals():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    lin, *_ = _layer(256, 128, 19)
    x = _x(ac.generator(5), 8, 256)
    ws = lin.workspace(8)
    y = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
    raw = torch.empty(4096, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: svdq.svdq_fp8_forward(lin.handle, x, 8, y, ws[:-1]),
                 lambda: svdq.svdq_fp8_forward(lin.handle, x, -1, y, ws),
                 lambda: svdq.svdq_fp8_forward(lin.handle, x, (1 << 30) + 1, y, ws),  # more tokens than counted
                 lambda: svdq.svdq_fp8_workspace_size(lin.handle, (1 << 30) + 1),
                 lambda: svdq.svdq_fp8_forward(lin.handle, raw[1:], 8, y, ws),
                 lambda: svdq.svdq_fp8_forward(lin.handle, x, 8, raw[1:], ws),
                 lambda: svdq.svdq_fp8_forward(lin.handle, x, 8, None, ws),
                 lambda: svdq.svdq_fp8_forward(lin.handle, None, 8, y, ws)):
        with pytest.raises(svdq.SvdqError) as e:
            call()
        assert e.value.status == svdq.SVDQ_ERR_INVALID_ARG
    with pytest.raises(svdq.SvdqError):
        svdq.svdq_fp8_layer_create(torch.empty(1 << 20, dtype=torch.uint8).pin_memory(), 1 << 20, 128, 256)
    for bad in (x.float(), x[:, :128], x.t().contiguous().t()):
        with pytest.raises(ValueError):
            lin.forward(bad)
    for out in (y[:4], y.float(), y.t().contiguous().t()):
        with pytest.raises(ValueError):
            lin.forward(x, out=out)
