"""The ends of the numbers' range in the attention sublayer's operators: head norms whose squares leave binary32, and FP8
scales whose product does."""
import numpy as np
import pytest

import attn_cases as ac

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133  # a step of the smallest bf16 (and of what passes through binary32 on the way to it)


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


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("d,rot", [(8, 8), (72, 48), (128, 128), (256, 0)])
@pytest.mark.parametrize("s", [3, 400, 2000])  # four warps to a token, two and one
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-38])
def test_norm_of_squares_outside_binary32(s, eps, d, rot, pairs):
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(s + d)
    x = ac.bf16(g, 1, s, 9, d)
    w = ac.bf16(g, d) + 1
    table = ac.rope_table(s, rot, "cuda") if rot else None
    plain = svdq.svdq_qk_norm_rope(x, None, w, eps=eps, rope=table, pairs=pairs)
    odd = x.double()
    odd[:, :, 1] *= 1e37                                      # every square past binary32
    odd[:, ::2, 2, 3] = 3.3e38                                # one element
    odd[:, :, 3] = 0.0
    odd[:, :, 3, d - 1] = -2.0 ** 64                          # the least whose square is
    odd[:, :, 4] *= 2.0 ** -60                                # squares that underflow, with eps and without
    odd[:, :, 5] *= 2.0 ** -128
    odd[:, :, 6] = 2.0 ** -133                                # the smallest bf16
    odd[:, :, 7] *= 1e19                                      # the sum, not the squares
    odd = odd.to(torch.bfloat16)
    got = svdq.svdq_qk_norm_rope(odd, None, w, eps=eps, rope=table, pairs=pairs)
    ref, bound = ac.norm_rope(odd, w, float(np.float32(eps)), table, None, pairs)
    ac.check(got, ref, bound + TINY)
    assert torch.equal(got[:, :, [0, 8]], plain[:, :, [0, 8]])  # the heads beside them
    assert int(svdq.attn_status().item()) == 0


def test_norm_of_infinities_and_zero_rows():
    """As the formula has it: 0 where another element is infinite, NaN there, and NaN for zeros over no eps."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    x = ac.bf16(ac.generator(1), 1, 5, 4, 64)
    x[0, 1, 2, 7] = float("-inf")
    x[0, 2, 3, 0] = float("nan")
    x[0, 3, 1] = 0
    y = svdq.svdq_qk_norm_rope(x, eps=0.0)
    hit = torch.arange(64, device="cuda") == 7
    assert torch.isnan(y[0, 1, 2][hit]).all() and not y[0, 1, 2][~hit].any()
    assert torch.isnan(y[0, 2, 3]).all() and torch.isnan(y[0, 3, 1]).all()
    assert not svdq.svdq_qk_norm_rope(x, eps=1e-30)[0, 3, 1].any()
    keep = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[2, 3] = keep[3, 1] = False
    ref, bound = ac.norm_rope(x, None, 0.0, None, None, "interleaved")
    ac.check(y[0][keep], ref[0][keep], bound[0][keep])


# every kernel of the product: few tokens (16, 32, 64; alone and in clusters), tiles of 64, 128 and 256 columns (alone and
# in clusters)
@pytest.mark.parametrize("M,K,N", [(5, 640, 136), (2, 4096, 512), (24, 400, 264), (30, 2048, 768), (60, 2048, 512),
                                   (100, 4096, 512), (300, 9728, 264), (129, 640, 4616), (300, 400, 520), (700, 512, 2048),
                                   (1100, 1168, 2312), (2100, 512, 2568)])
def test_fp8_scales_whose_product_leaves_binary32(M, K, N):
    """Tokens of 2^60 and more in one block over a weight scale of 2^70: the product of the scales is infinite, the block's
    sum is 0 or 2^-18, and so the output is an ordinary number or one of about 2^112."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    g = ac.generator(M + K)
    qw, sw = ac.fp8_weight(ac.bf16(g, N, K, scale=0.02))
    rows = torch.arange(N, device="cuda") % 3 == 0
    at = 256 if K > 256 else 0  # the block
    qw[:, at:at + 128] = 0
    qw[rows, at + 1] = 2.0 ** -9  # the smallest code
    sw[:, at // 128] = 2.0 ** 70
    codes = qw.float().to(torch.float8_e4m3fn).view(torch.uint8).cpu().numpy()
    lin = svdq.Fp8Linear(codes, sw.cpu().numpy(), device="cuda:0")
    x = ac.bf16(g, M, K)
    x[:, at:at + 128] = 0
    plain = lin.forward(x).clone()
    big = torch.arange(M, device="cuda") % 2 == 0
    x[big, at] = 448 * 2.0 ** 60         # times a code of 0
    x[big, at + 1] = 2.0 ** 60 * 2.0 ** -9  # the smallest code, times the smallest or 0
    qx, sx = ac.fp8_quantize(x)
    assert not torch.isfinite((sx[big][:, at // 128, None] * sw[:, at // 128])).any()
    y = lin.forward(x)
    assert lin.status(M) == 0
    ref, bound = ac.fp8_linear(qx, sx, qw, sw, None)
    assert torch.isfinite(bound).all() and ref[0, 0].abs() > 2.0 ** 111
    ac.check(y, ref, bound)
    assert torch.equal(y[~big], plain[~big])


def test_fp8_infinite_inputs_over_large_scales():
    """An infinite input gives NaN over any weight scale, 0 and the largest among them."""
    import torch

    import diffusion_transformer_w4a4_b200 as svdq

    N, K = 264, 512
    g = ac.generator(3)
    qw, sw = ac.fp8_weight(ac.bf16(g, N, K, scale=0.02))
    sw[1] = 3.4e38
    sw[2] = 0.0
    lin = svdq.Fp8Linear(qw.float().to(torch.float8_e4m3fn).view(torch.uint8).cpu().numpy(), sw.cpu().numpy(),
                         device="cuda:0")
    for M in (3, 70, 300):
        x = ac.bf16(g, M, K)
        x[1, 5] = float("inf")
        y = lin.forward(x)
        assert torch.isnan(y[1]).all() and not y[0, 256:].any() and torch.isfinite(y[0, :128]).all()
