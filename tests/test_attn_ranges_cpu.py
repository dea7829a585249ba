"""The packed FP8 blob says whether a weight scale is so large that its product with an activation's may leave binary32."""
import numpy as np
import pytest

import diffusion_transformer_w4a4_b200 as svdq


@pytest.fixture(scope="module", autouse=True)
def _built():
    from diffusion_transformer_w4a4_b200 import build

    build.build()


@pytest.mark.parametrize("N,K", [(8, 16), (136, 272), (256, 1024)])
def test_pack_marks_scales_above_448(N, K):
    codes = np.zeros((N, K), np.uint8)
    scales = np.ones((-(-N // 128), -(-K // 128)), np.float32)
    size = svdq.svdq_fp8_packed_size(N, K)
    mark = lambda s: int(svdq.svdq_fp8_pack(codes, s)[-1024:-1020].view(np.int32)[0])
    assert svdq.svdq_fp8_pack(codes, scales).size == size
    assert mark(scales) == 0 and mark(scales * 448) == 0
    for at in (0, scales.size - 1):
        big = scales.copy()
        big.flat[at] = np.nextafter(np.float32(448), np.float32(449))
        assert mark(big) == 1


def test_largest_activation_scale_times_448_is_finite():
    """The largest bf16 over 448 is the largest scale of a finite input: up to a weight scale of 448 the product is finite."""
    top = np.float32(2.0 ** 128 - 2.0 ** 120)
    with np.errstate(over="raise"):
        assert np.isfinite(np.float32(top / np.float32(448)) * np.float32(448))
