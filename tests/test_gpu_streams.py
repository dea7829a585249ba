"""Memory that a layer allocates for a call on another stream than the current one: it is that stream's, so work that is
still pending on the current stream never shares it, and a dropped layer's memory waits for every stream that used it."""
import numpy as np
import pytest

import attn_cases as ac

pytestmark = pytest.mark.gpu

CYCLES = 200_000_000  # about a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200 import build

    build.build()
    assert torch.cuda.is_available()
    assert svdq.svdq_device_check(0) == svdq.SVDQ_OK, "needs an sm_100a device"
    torch.cuda.set_device(0)


def _fp8(K, N, seed):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    w = ac.bf16(ac.generator(seed), N, K, scale=0.05)
    return svdq.Fp8Linear(*svdq.svdq_fp8_prepare(w.view(torch.int16).cpu().numpy().view(np.uint16)), device="cuda:0")


def _on_side(torch, side, M, K):
    """Inputs that live on `side`, complete there."""
    with torch.cuda.stream(side):
        x = ac.bf16(ac.generator(M), M, K)
    torch.cuda.synchronize()
    return x


def _pending_fill(torch, sizes):
    """Freed blocks of the current stream that it has yet to write; their addresses."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(CYCLES)
    for b in blocks:
        b.fill_(0xA5)
    return [b.data_ptr() for b in blocks]


@pytest.mark.parametrize("raw", [False, True])
def test_first_call_on_a_side_stream_keeps_its_workspace(raw):
    import torch

    M, K, N = 700, 2048, 1024
    want_codes, want_scales = ac.fp8_quantize(_on_side(torch, torch.cuda.Stream(), M, K))
    lin, side = _fp8(K, N, 1), torch.cuda.Stream()
    x = _on_side(torch, side, M, K)
    torch.cuda.empty_cache()
    freed = _pending_fill(torch, [lin.workspace_size(M), 2 * M * N])
    y = lin.forward(x, stream=side.cuda_stream if raw else side)  # its first call with M tokens
    torch.cuda.synchronize()  # the fill has run by now
    assert lin.workspace(M).data_ptr() not in freed and y.data_ptr() not in freed
    act = lin.read_act(M)
    assert torch.equal(torch.from_numpy(act["codes"]).view(torch.float8_e4m3fn).double().cuda(), want_codes)
    np.testing.assert_array_equal(act["scales"], want_scales.cpu().numpy())
    assert lin.status(M) == 0 and torch.equal(y, lin.forward(x))


@pytest.mark.parametrize("explicit", [False, True])
def test_dropped_layer_waits_for_the_other_stream(explicit):
    """A layer and its workspace, memory of the current stream, used on another one and dropped while that still works:
    neither is handed out."""
    import torch

    M, K, N = 700, 2048, 1024
    lin, side = _fp8(K, N, 2), torch.cuda.Stream()
    x = _on_side(torch, side, M, K)
    want = lin.forward(x)
    out = torch.empty_like(want)
    used = [(t.data_ptr(), t.numel()) for t in (lin.workspace(M), lin.blob)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
        if not explicit:
            lin.forward(x, out=out)
    if explicit:
        lin.forward(x, out=out, stream=side)
    del lin
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in used]
    for t in again:
        assert all(t.data_ptr() + t.numel() <= at or t.data_ptr() >= at + n for at, n in used)
        t.fill_(0xFF)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_destroyed_raw_stream_before_the_layer():
    """A raw handle's stream destroyed before the layer is dropped: nothing is recorded on it."""
    import ctypes

    import torch

    M, K, N = 300, 512, 256
    rt = ctypes.CDLL("libcudart.so.12")
    lin = _fp8(K, N, 3)
    x = ac.bf16(ac.generator(M), M, K)
    want = lin.forward(x)
    torch.cuda.synchronize()
    handle = ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(handle)) == 0
    got = lin.forward(x, stream=handle.value)
    torch.cuda.synchronize()
    equal = torch.equal(got, want)
    del got, lin  # (what the call allocated goes back before its stream does)
    torch.cuda.synchronize()
    assert rt.cudaStreamDestroy(handle) == 0
    assert equal


def _older_layer(kind, N, K):
    import numpy as np

    import diffusion_transformer_w4a4_b200 as svdq

    g = np.random.default_rng(5)
    bits = lambda a: (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    W, X = bits(g.standard_normal((N, K)) * 0.05), bits(g.standard_normal((64, K)))
    if kind == "awq":
        return svdq.AwqLinear(svdq.svdq_awq_prepare(W, None, X), device="cuda:0")
    if kind == "w8a8":
        return svdq.W8A8Linear(*svdq.svdq_w8a8_prepare(W), device="cuda:0")
    amax = np.abs((X.astype(np.uint32) << 16).view(np.float32)).max(0)
    return svdq.SvdqLinear(svdq.svdq_prepare(W, None, amax, 0.5, 32, kind), device="cuda:0")


@pytest.mark.parametrize("kind", ["nvfp4", "int4", "w8a8", "awq"])
def test_first_call_on_a_side_stream_of_the_other_layers(kind):
    """Workspace, its initialisation and output on the given stream: right at once, whatever the current one has yet to do."""
    import torch

    M, K, N = 300, 512, 384
    lin, side = _older_layer(kind, N, K), torch.cuda.Stream()
    x = _on_side(torch, side, M, K)
    torch.cuda.empty_cache()
    sizes = [2 * M * N] if kind == "awq" else [2 * M * N, 1 << 20]
    freed = _pending_fill(torch, sizes)
    y = lin.forward(x, stream=side)
    side.synchronize()
    first = y.cpu()  # (on the current stream, behind the fill)
    assert y.data_ptr() not in freed
    if kind != "awq":
        assert lin.workspace(M).data_ptr() not in freed
    torch.cuda.synchronize()
    assert torch.equal(first, lin.forward(x).cpu())
    assert (lin.status() if kind == "awq" else lin.status(M)) == 0


@pytest.mark.parametrize("first", ["side", "current"])
def test_calls_of_one_object_on_two_streams_are_in_order(first):
    """An attention sublayer's second call, on another stream, comes after the first, which shares its workspaces."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200.attention import SelfAttention

    svdq.attn_status()
    mod = SelfAttention(_fp8(256, 3 * 4 * 64, 11), _fp8(4 * 64, 256, 12), 4)
    g = ac.generator(13)
    xs = [ac.bf16(g, 2, 150, 256) for _ in range(2)]
    want = [mod(x) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.current_stream()]
    if first == "current":
        streams.reverse()
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        torch.cuda._sleep(CYCLES)
        one = mod(xs[0])
    with torch.cuda.stream(streams[1]):
        two = mod(xs[1])
    streams[1].synchronize()
    assert streams[0].query()
    assert torch.equal(one, want[0]) and torch.equal(two, want[1])


def test_call_after_a_raw_handle_that_is_gone():
    import ctypes

    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200.attention import SelfAttention

    svdq.attn_status()
    rt = ctypes.CDLL("libcudart.so.12")
    mod = SelfAttention(_fp8(256, 3 * 4 * 64, 11), _fp8(4 * 64, 256, 12), 4)
    x = ac.bf16(ac.generator(14), 1, 100, 256)
    want = mod(x)
    torch.cuda.synchronize()
    handle = ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(handle)) == 0
    got = mod(x, stream=handle.value)
    torch.cuda.synchronize()
    equal = torch.equal(got, want)
    del got
    assert rt.cudaStreamDestroy(handle) == 0
    assert equal and torch.equal(mod(x), want)


@pytest.mark.parametrize("kind", ["nvfp4", "w8a8", "awq", "fp8", "attention", "norm", "attn"])
def test_handle_0_is_the_default_stream(kind):
    """A raw handle of the default stream, which is 0: the work comes after what that stream has yet to do."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq
    from diffusion_transformer_w4a4_b200.attention import SelfAttention

    svdq.attn_status()
    assert torch.cuda.current_stream().cuda_stream == 0
    g = ac.generator(21)
    shape = (300, 512)
    if kind in ("norm", "attn"):
        shape = (2, 100, 4, 64)
        call = (lambda x, **kw: svdq.svdq_qk_norm_rope(x, **kw)) if kind == "norm" else \
            (lambda x, **kw: svdq.svdq_cross_attn(x, x, x, **kw))
    elif kind == "attention":
        shape = (2, 150, 256)
        call = SelfAttention(_fp8(256, 3 * 4 * 64, 11), _fp8(4 * 64, 256, 12), 4)
    else:
        call = (_fp8(512, 384, 22) if kind == "fp8" else _older_layer(kind, 384, 512)).forward
    src = ac.bf16(g, *shape)
    want = call(src)
    torch.cuda.synchronize()
    if kind in ("nvfp4", "w8a8", "awq"):
        call = _older_layer(kind, 384, 512).forward  # without a workspace
        torch.cuda.synchronize()
    x = torch.zeros_like(src)
    torch.cuda._sleep(CYCLES)
    x.copy_(src)
    got = call(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
