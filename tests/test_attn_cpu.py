"""Checks of the FP8 layer, the query/key norm and the cross attention that need no GPU: the FP8 host preparation
against the definition in binary64, the packed layout, sizes, and every refusal that is decided on the host before
a device is looked at."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import attn_cases as ac
import diffusion_transformer_w4a4_b200 as svdq
import oracle
import workloads as wl


@pytest.fixture(scope="module")
def lib():
    from diffusion_transformer_w4a4_b200 import build

    build.build()
    return svdq.lib()


def _e4m3_value(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).double()


# ------------------------------------------------------------------------------------------------- FP8 host half
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (136, 272), (264, 1168), (520, 400)])
def test_fp8_prepare_matches_the_definition(lib, N, K):
    rng = np.random.default_rng(N + K)
    w = (rng.standard_normal((N, K)) * 10.0 ** rng.integers(-3, 3, (N, 1))).astype(np.float32)
    W = wl.f32_to_bf16_bits(w)
    codes, scales = svdq.svdq_fp8_prepare(W)
    q, s = ac.fp8_weight(torch.from_numpy(wl.bf16_bits_to_f32(W).copy()))
    np.testing.assert_array_equal(scales, s.numpy())
    np.testing.assert_array_equal(_e4m3_value(codes).numpy(), q.numpy())


def test_fp8_prepare_zero_tiny_and_largest_blocks(lib):
    w = np.zeros((128, 384), np.float32)
    w[:, 128:256] = 2.0 ** -126
    w[3, 300] = 3.0e38
    codes, scales = svdq.svdq_fp8_prepare(wl.f32_to_bf16_bits(w))
    assert np.isfinite(scales).all() and (scales > 0).all()
    assert not codes[:, :256].any()  # far below the floor of 2^-100
    assert codes[3, 300] == 0x7E and codes[:, 256:].astype(bool).sum() == 1
    bad = wl.f32_to_bf16_bits(w)
    bad[5, 5] = 0x7F80  # infinity
    with pytest.raises(svdq.SvdqError) as e:
        svdq.svdq_fp8_prepare(bad)
    assert e.value.status == svdq.SVDQ_ERR_NUMERIC


def test_fp8_pack_layout_and_refusals(lib):
    N, K = 136, 272
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 0x7F, (N, K)).astype(np.uint8)
    scales = rng.uniform(0.0, 2.0, (2, 3)).astype(np.float32)
    bias = oracle.f32_to_bf16(rng.standard_normal(N).astype(np.float32))
    blob = svdq.svdq_fp8_pack(codes, scales, bias)
    assert blob.size == svdq.svdq_fp8_packed_size(N, K) and blob.size % 1024 == 0
    assert np.array_equal(blob[:4 * N].view(np.float32), oracle.bf16_to_f32(bias))
    assert np.array_equal(blob[1024:1024 + 32].view(np.float32).reshape(2, 4), np.pad(scales, ((0, 0), (0, 1))))
    assert np.array_equal(blob[2048:2048 + N * K].reshape(N, K), codes)
    assert not svdq.svdq_fp8_pack(codes, scales)[:4 * N].any()  # no bias: zeros
    nan_code = codes.copy()
    nan_code[1, 2] = 0xFF
    for c, s in ((nan_code, scales), (codes, -scales), (codes, np.full_like(scales, np.inf))):
        with pytest.raises(svdq.SvdqError) as e:
            svdq.svdq_fp8_pack(c, s, bias)
        assert e.value.status == svdq.SVDQ_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        svdq.svdq_fp8_pack(codes, scales[:1], bias)
    with pytest.raises(ValueError):
        svdq.svdq_fp8_pack(codes, scales, bias[:-1])


@pytest.mark.parametrize("N,K", [(4, 128), (12, 128), (128, 8), (128, 24), (0, 16), ((1 << 24) + 8, 16),
                                 (8, (1 << 20) + 16)])
def test_fp8_shapes_refused(lib, N, K):
    with pytest.raises(svdq.SvdqError) as e:
        svdq.svdq_fp8_packed_size(N, K)
    assert e.value.status == svdq.SVDQ_ERR_INVALID_ARG


def test_fp8_null_arguments_refused(lib):
    n = ctypes.c_size_t()
    one = (ctypes.c_uint8 * 4096)()
    h = ctypes.c_void_p()
    assert lib.svdq_fp8_prepare(None, 128, 128, one, one) == 1
    assert lib.svdq_fp8_packed_size(128, 128, None) == 1
    assert lib.svdq_fp8_pack(128, 128, None, one, None, one, 1 << 20) == 1
    assert lib.svdq_fp8_pack(8, 16, one, one, None, one, 16) == 1  # blob too small
    assert lib.svdq_fp8_layer_create(None, 1 << 20, 128, 128, ctypes.byref(h)) == 1
    assert lib.svdq_fp8_layer_create(ctypes.c_void_p(256), 16, 128, 128, ctypes.byref(h)) == 1  # blob too small
    assert lib.svdq_fp8_layer_create(ctypes.c_void_p(256), 1 << 20, 128, 128, None) == 1
    assert lib.svdq_fp8_workspace_size(None, 1, ctypes.byref(n)) == 1
    for f in (lib.svdq_fp8_quantize_act, lib.svdq_fp8_forward):
        args = [None, one, 1, one, 4096, None] if f is lib.svdq_fp8_quantize_act else [None, one, 1, one, one, 4096, None]
        assert f(*args) == 1
    assert lib.svdq_fp8_gemm(None, 1, one, one, 4096, None) == 1
    lib.svdq_fp8_layer_destroy(None)


# ------------------------------------------------------------------------------------------------- norm and rotation
def _rope_bytes(**kw):
    d = dict(x=256, xs=(1024, 1024, 128), y=4096, ys=(1024, 1024, 128), batch=1, tokens=1, heads=2, weight=0, rope=0,
             rows=0, pos=0)
    d.update(kw)
    return struct.pack("P3qP3q3qPPqP", d["x"], *d["xs"], d["y"], *d["ys"], d["batch"], d["tokens"], d["heads"],
                       d["weight"], d["rope"], d["rows"], d["pos"])


def _rope_call(lib, a, k=None, dim=64, rot=0, pairs=0, eps=1e-6, status=None):
    return lib.svdq_qk_norm_rope(a, k, dim, rot, pairs, eps, status, None)


@pytest.mark.parametrize("kw,call", [
    (None, {}), ({}, dict(dim=0)), ({}, dict(dim=12)), ({}, dict(dim=264)), ({}, dict(rot=72)), ({}, dict(rot=12)),
    ({}, dict(rot=-8)), ({}, dict(pairs=2)), ({}, dict(eps=-1.0)), ({}, dict(eps=float("nan"))),
    ({}, dict(eps=float("inf"))), ({}, dict(status=ctypes.c_void_p(2))), (dict(x=0), {}), (dict(x=8), {}),
    (dict(y=0), {}), (dict(y=20), {}), (dict(batch=-1), {}), (dict(tokens=-1), {}), (dict(heads=-1), {}),
    (dict(batch=1 << 31), {}), (dict(batch=1 << 16, tokens=1 << 16), {}), (dict(xs=(1024, 1024, 12)), {}),
    (dict(xs=(1024, 1024, -128)), {}), (dict(xs=(1024, 1024, 56)), {}), (dict(ys=(1024, 1024, 0)), {}),
    (dict(tokens=2, ys=(1024, 128, 128)), {}), (dict(tokens=2, ys=(1024, 64, 64)), {}),
    (dict(tokens=3, batch=2, ys=(2048, 1024, 128)), {}),
    (dict(tokens=2, xs=(1024, 0, 128)), {}), (dict(batch=2, ys=(0, 1024, 128)), {}), (dict(weight=8), {}),
    (dict(rope=8, rows=4), dict(rot=64)), (dict(rope=256, rows=0), dict(rot=64)),
    (dict(rope=256, rows=1, tokens=2), dict(rot=64)), (dict(rope=256, rows=4, pos=2), dict(rot=64)),
])
def test_norm_rope_refusals(lib, kw, call):
    a = None if kw is None else _rope_bytes(**kw)
    assert _rope_call(lib, a, **call) == svdq.SVDQ_ERR_INVALID_ARG
    if kw is not None:  # as the keys' side too
        good = _rope_bytes()
        assert _rope_call(lib, good, a, **call) == svdq.SVDQ_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
def test_output_strides_in_any_order(lib):
    """Views whose elements are all different pass the checks (and stop at the missing device)."""
    word = ctypes.c_int32()
    for kw in (dict(os=(4096, 64, 256)), dict(os=(64, 128, 512), batch=2), dict(os=(0, 256, 64)), dict(os=(4096, 512, 128)),
               dict(batch=2, os=(1984, 512, 64))):  # 64 + 3 * 64 + 3 * 512 = 1792
        assert lib.svdq_cross_attn(_attn_bytes(**kw), ctypes.byref(word), None) == svdq.SVDQ_ERR_UNSUPPORTED_DEVICE
    for kw in (dict(tokens=2, ys=(1024, 64, 128)), dict(tokens=2, ys=(0, 128, 64)),
               dict(tokens=2, x=4096, xs=(0, 128, 64), ys=(0, 128, 64))):
        assert _rope_call(lib, _rope_bytes(**kw)) == svdq.SVDQ_ERR_UNSUPPORTED_DEVICE


def test_norm_rope_empty_is_a_no_op(lib):
    for kw in (dict(batch=0, x=0, y=0), dict(tokens=0, x=0, y=0), dict(heads=0, x=0, y=0)):
        assert _rope_call(lib, _rope_bytes(**kw)) == svdq.SVDQ_OK


# ------------------------------------------------------------------------------------------------- attention
def _attn_bytes(**kw):
    d = dict(q=256, k=512, v=1024, o=2048, s=(4096, 512, 64), batch=1, sq=4, sk=4, hq=4, hk=2, dim=64, kv_len=0,
             mask=0, mask_ld=0, scale=0.125, qs=None, ks=None, vs=None, os=None)
    d.update(kw)
    st = [d[f] or d["s"] for f in ("qs", "ks", "vs", "os")]
    return struct.pack("P3qP3qP3qP3q6qPPqf4x", d["q"], *st[0], d["k"], *st[1], d["v"], *st[2], d["o"], *st[3],
                       d["batch"], d["sq"], d["sk"], d["hq"], d["hk"], d["dim"], d["kv_len"], d["mask"], d["mask_ld"],
                       d["scale"])


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(q=8), dict(k=0), dict(v=24), dict(o=0), dict(o=4), dict(batch=-1), dict(sq=-1), dict(sk=-1),
    dict(batch=1 << 31), dict(sq=1 << 31), dict(sk=1 << 31), dict(hq=0), dict(hk=0), dict(hq=5), dict(hq=8192, hk=1),
    dict(dim=0), dict(dim=4), dict(dim=60), dict(dim=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=3e38), dict(qs=(4096, 512, 60)), dict(ks=(4096, 512, 56)), dict(ks=(4096, 0, 64)),
    dict(qs=(4096, 0, 64)), dict(vs=(4096, -512, 64)), dict(os=(4096, 512, 0)), dict(batch=2, os=(0, 512, 64)),
    dict(batch=2, mask=64, mask_ld=-4), dict(kv_len=2), dict(os=(4096, 64, 64)), dict(os=(4096, 192, 64)),
    dict(os=(4096, 64, 128)), dict(batch=2, os=(1784, 512, 64)), dict(o=256), dict(o=512), dict(o=1024),
])
def test_attention_refusals(lib, kw):
    word = ctypes.c_int32()
    assert lib.svdq_cross_attn(_attn_bytes(**kw), ctypes.byref(word), None) == svdq.SVDQ_ERR_INVALID_ARG


def test_attention_needs_a_status_word(lib):
    assert lib.svdq_cross_attn(_attn_bytes(), None, None) == svdq.SVDQ_ERR_INVALID_ARG
    assert lib.svdq_cross_attn(_attn_bytes(), ctypes.c_void_p(2), None) == svdq.SVDQ_ERR_INVALID_ARG
    assert lib.svdq_cross_attn(None, ctypes.c_void_p(256), None) == svdq.SVDQ_ERR_INVALID_ARG


def test_attention_without_queries_is_a_no_op(lib):
    for kw in (dict(batch=0, q=0, k=0, v=0, o=0), dict(sq=0, q=0, o=0)):
        assert lib.svdq_cross_attn(_attn_bytes(**kw), ctypes.c_void_p(256), None) == svdq.SVDQ_OK


def test_python_refusals():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        svdq.svdq_cross_attn(q, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        svdq.svdq_qk_norm_rope(q)
    with pytest.raises(ValueError, match="CUDA device"):
        svdq.attn_status("cpu")


# ------------------------------------------------------------------------------------------------- compression tool
def test_fp8_layers_in_the_packed_file(tmp_path):
    from diffusion_transformer_w4a4_b200 import compress

    layers, inputs = compress.synthetic_flux_block(tokens=32, seed=1, width=256, heads=2)
    path = str(tmp_path / "b.svdq")
    plans, canon = compress.compress(layers, inputs, path, rank=16, rules=compress.FP8_ATTENTION_RULES,
                                     attention=dict(heads=2, theta=10000.0))
    kinds = {p.name.split("transformer_blocks.0.")[1]: p.kind for p in plans}
    assert kinds == {"norm1.linear": compress.AWQ, "attn.to_qkv": compress.FP8, "attn.to_out.0": compress.FP8,
                     "ff.net.0.proj": compress.SVDQ, "ff.net.2": compress.SVDQ}
    header, back = compress.read_packed(path)
    assert header["attention"] == dict(heads=2, theta=10000.0)
    for p in plans:
        for f, a in back[p.name].items():
            if isinstance(a, np.ndarray):
                np.testing.assert_array_equal(a, canon[p.name][f])
    name = "transformer_blocks.0.attn.to_qkv"
    assert back[name]["wcodes"].dtype == np.uint8 and back[name]["wscales"].shape == (6, 2)
    # without the rules and heads the tool does what it did
    plain, _ = compress.synthetic_flux_block(tokens=32, seed=1, width=256)
    assert all(np.array_equal(a.W, b.W) for a, b in zip(layers, plain))
    assert all(p.kind != compress.FP8 for p in compress.scan(plain))
    bad = [compress.LinearSpec("attn.to_q", np.zeros((12, 24), np.uint16))]
    assert compress.scan(bad, compress.FP8_ATTENTION_RULES)[0].kind == compress.KEEP


def test_dense_attention_of_the_synthetic_block():
    from diffusion_transformer_w4a4_b200 import compress

    rng = np.random.default_rng(0)
    S, heads, dim = 37, 3, 16
    bits = wl.f32_to_bf16_bits(rng.standard_normal((S, 3 * heads * dim)).astype(np.float32))
    out = compress.dense_attention(bits, heads)
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).view(1, S, 3, heads, dim)
    table = ac.rope_table(S, dim, "cpu")
    q, _ = ac.norm_rope(t[:, :, 0], None, 1e-6, table, None, "interleaved")
    k, _ = ac.norm_rope(t[:, :, 1], None, 1e-6, table, None, "interleaved")
    o, _ = ac.attention(q.to(torch.bfloat16), k.to(torch.bfloat16), t[:, :, 2], None, None, dim ** -0.5)
    got = torch.from_numpy(oracle.bf16_to_f32(out)).double().view(S, heads, dim)
    # a table in binary32 against one in binary64 may round a q or k the other way (2^-8 of it at most)
    assert ((got - o[0]).abs() <= 2.0 ** -8 * o[0].abs() + 2.0 ** -6 * t[:, :, 2].double().abs().amax()).all()
