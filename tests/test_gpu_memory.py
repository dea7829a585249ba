"""Memory that the attention sublayer's objects keep between calls: bounded by the largest call, whatever the number of
token counts, and not taken from a captured graph."""
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


def _fp8(K, N, seed=1):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    w = ac.bf16(ac.generator(seed), N, K, scale=0.05)
    return svdq.Fp8Linear(*svdq.svdq_fp8_prepare(w.view(torch.int16).cpu().numpy().view(np.uint16)), device="cuda:0")


@pytest.mark.parametrize("counts", [range(1, 1000, 3), range(999, 0, -3)])
def test_token_counts_share_a_workspace(counts):
    import torch

    lin = _fp8(2048, 64)
    x = ac.bf16(ac.generator(2), 1000, 2048)
    want = lin.forward(x[:counts[0]]).clone()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for m in counts:
        lin.forward(x[:m])
    torch.cuda.synchronize()
    # a buffer is at most half as large again as what made it necessary, and three times the last bounds the sum of buffers
    # that each are half as large again as the one before: 1.5 (1 + 2/3 + 4/9 + ...) = 4.5
    assert torch.cuda.memory_allocated() - before <= 4.5 * lin.workspace_size(1000) + (1 << 20)
    assert torch.equal(lin.forward(x[:counts[0]]), want)


def test_status_and_codes_of_any_token_count():
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    lin = _fp8(400, 136)
    assert lin.status(5) == 0  # before any call
    x = ac.bf16(ac.generator(3), 300, 400)
    for m in (300, 1, 64, 299, 17):
        lin.forward(x[:m])
        act = lin.read_act(m)
        codes, scales = ac.fp8_quantize(x[:m])
        assert torch.equal(torch.from_numpy(act["codes"]).view(torch.float8_e4m3fn).double().cuda(), codes)
        np.testing.assert_array_equal(act["scales"], scales.cpu().numpy())
        assert lin.status(m) == lin.status(300) == 0
    try:
        svdq.svdq_set_wait_limit(1)
        lin.forward(x[:200])
        torch.cuda.synchronize()
    finally:
        svdq.svdq_set_wait_limit(0)
    assert lin.status(200) == lin.status(1) == svdq.SVDQ_ERR_TIMEOUT
    lin.forward(x[:1])
    assert lin.status(1) == 0


def test_captured_graphs_keep_their_workspace():
    """Graphs of several token counts, each captured before a larger one made a new workspace, replayed afterwards."""
    import torch

    lin = _fp8(768, 264)
    xs = [ac.bf16(ac.generator(m), m, 768) for m in (3, 40, 500, 1100)]
    graphs, ys = [], []
    for x in xs:
        lin.forward(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(lin.forward(x))
        graphs.append(g)
    want = [lin.forward(x) for x in xs]
    fill = [torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(32)]  # what was freed is used
    for g, y in zip(graphs, ys):
        y.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want)) and len(fill) == 32


def test_block_tables_grow_by_halves(tmp_path):
    import torch

    from diffusion_transformer_w4a4_b200 import compress
    from diffusion_transformer_w4a4_b200.attention import rope_table

    layers, inputs = compress.synthetic_flux_block(tokens=40, seed=2, width=768, heads=6)
    path = str(tmp_path / "block.svdq")
    compress.compress(layers, inputs, path, rules=compress.FP8_ATTENTION_RULES, attention=dict(heads=6, theta=10000.0))
    block = compress.load_block(path, "cuda:0")
    for tokens in range(10, 400, 7):
        table = block._table(tokens)
        assert table.shape[0] >= tokens
        assert torch.equal(table, rope_table(table.shape[0], 128))
    assert sum(t.shape[0] for t in block._ropes) <= 3 * block._ropes[-1].shape[0] <= 3 * 1.5 * 400
