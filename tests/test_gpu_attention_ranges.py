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
