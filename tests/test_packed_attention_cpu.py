"""The packed file holds a block's head norms: their weights come back bit by bit, and calibration uses them."""
import numpy as np
import torch

import attn_cases as ac
import oracle
import workloads as wl
from diffusion_transformer_w4a4_b200 import compress


def _bits(rng, n):
    return wl.f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(n)).astype(np.float32))


def test_norm_weights_in_the_packed_file(tmp_path):
    rng = np.random.default_rng(0)
    wq, wk = _bits(rng, 128), _bits(rng, 128)
    layers, inputs = compress.synthetic_flux_block(tokens=32, seed=1, width=256, heads=2, q_norm=wq, k_norm=wk)
    path = str(tmp_path / "b.svdq")
    plans, canon = compress.compress(layers, inputs, path, rank=16, rules=compress.FP8_ATTENTION_RULES,
                                     attention=dict(heads=2, theta=500.0, eps=1e-5, q_norm=wq, k_norm=wk))
    header, back = compress.read_packed(path)
    a = header["attention"]
    assert (a["heads"], a["theta"], a["eps"]) == (2, 500.0, 1e-5)
    np.testing.assert_array_equal(a["q_norm"], wq)
    np.testing.assert_array_equal(a["k_norm"], wk)
    for p in plans:  # and the layers' arrays as before
        for f, v in back[p.name].items():
            if isinstance(v, np.ndarray):
                np.testing.assert_array_equal(v, canon[p.name][f])
    compress.pack(path, plans, canon, layers, dict(heads=2, theta=500.0, q_norm=None, k_norm=wk))
    a = compress.read_packed(path)[0]["attention"]
    assert "q_norm" not in a and np.array_equal(a["k_norm"], wk)


def test_dense_attention_with_norm_weights():
    rng = np.random.default_rng(1)
    S, heads, dim = 29, 2, 16
    wq, wk = _bits(rng, dim), _bits(rng, dim)
    bits = wl.f32_to_bf16_bits(rng.standard_normal((S, 3 * heads * dim)).astype(np.float32))
    out = compress.dense_attention(bits, heads, q_norm=wq, k_norm=wk)
    as_bf16 = lambda b: torch.from_numpy(b.view(np.int16)).view(torch.bfloat16)
    t = as_bf16(bits).view(1, S, 3, heads, dim)
    table = ac.rope_table(S, dim, "cpu")
    q, _ = ac.norm_rope(t[:, :, 0], as_bf16(wq), 1e-6, table, None, "interleaved")
    k, _ = ac.norm_rope(t[:, :, 1], as_bf16(wk), 1e-6, table, None, "interleaved")
    o, _ = ac.attention(q.to(torch.bfloat16), k.to(torch.bfloat16), t[:, :, 2], None, None, dim ** -0.5)
    got = torch.from_numpy(oracle.bf16_to_f32(out)).double().view(S, heads, dim)
    # half a bf16 step of the output, and what q's and k's roundings (the table here is in binary32, there in binary64:
    # 2^-8 of a value at most, where one falls the other way) move a softmax of scores below 4
    assert ((got - o[0]).abs() <= 2.0 ** -8 * o[0].abs() + 2.0 ** -6 * t[:, :, 2].double().abs().amax()).all()
    assert not np.array_equal(out, compress.dense_attention(bits, heads))
