"""The bounds-checked debug variant of the attention sublayer's operators: run in a child process with
SVDQ_LIBRARY=debug, every variant of the FP8 layer, the head norm and the attention at ragged shapes reports no bounds
error (status 0) and gives outputs bit-identical to the release library's."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import os, sys, numpy as np, torch
sys.path.insert(0, ROOT); sys.path.insert(0, os.path.join(ROOT, "tests"))
import attn_cases as ac
import diffusion_transformer_w4a4_b200 as svdq
torch.cuda.set_device(0)
out = {"debug": svdq.svdq_debug_build()}
bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
g = ac.generator(1)
for K, N in ((400, 136), (1168, 264), (272, 2056)):
    w, b = ac.bf16(g, N, K, scale=0.05), ac.bf16(g, N)
    lin = svdq.Fp8Linear(*svdq.svdq_fp8_prepare(bits(w)), bits(b), device="cuda:0")
    for M in (1, 5, 17, 33, 64, 65, 300, 1100):
        out[f"fp8_{K}_{N}_{M}"] = bits(lin(ac.bf16(g, M, K)))
        out[f"fp8_{K}_{N}_{M}_status"] = lin.status(M)
for d, rot in ((8, 8), (40, 24), (64, 64), (128, 128), (136, 64), (256, 256)):
    table = ac.rope_table(50, rot, "cuda")
    pos = torch.randint(0, 50, (3, 9), generator=g, device="cuda", dtype=torch.int32)
    x = ac.bf16(g, 3, 9, 11, d)
    for pairs in ("interleaved", "halves"):
        q, k = svdq.svdq_qk_norm_rope(x[:, :, :7], x[:, :, 7:], ac.bf16(g, d), None, rope=table, positions=pos,
                                      pairs=pairs)
        out[f"norm_{d}_{pairs}_q"], out[f"norm_{d}_{pairs}_k"] = bits(q), bits(k)
for b, sq, sk, hq, hk, d in ((2, 1, 300, 6, 2, 64), (1, 3, 1030, 4, 2, 128), (2, 100, 700, 2, 1, 72),
                             (2, 300, 129, 3, 3, 40), (3, 700, 300, 24, 24, 64), (2, 900, 300, 24, 8, 72),
                             (2, 900, 300, 40, 20, 128), (2, 500, 3000, 12, 4, 128), (1, 2100, 77, 24, 6, 120), (2, 2000, 77, 40, 1, 64)):
    q, kv = ac.bf16(g, b, sq, hq, d), ac.bf16(g, b, sk, 2, hk, d)
    mask = (torch.rand(b, sk, generator=g, device="cuda") < 0.8)
    lens = torch.randint(1, sk + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    for name, kw in (("all", {}), ("masked", dict(kv_mask=mask, kv_len=lens))):
        out[f"attn_{b}_{sq}_{sk}_{hq}_{hk}_{d}_{name}"] = bits(svdq.svdq_cross_attn(q, kv[:, :, 0], kv[:, :, 1], **kw))
out["attn_status"] = int(svdq.attn_status().item())
np.savez(sys.argv[1], **out)
'''


def _run(tmp_path, variant):
    path = str(tmp_path / f"{variant}.npz")
    env = dict(os.environ, SVDQ_LIBRARY=variant)
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT)), path], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    return dict(np.load(path))


def test_debug_variant_matches_release(tmp_path):
    from diffusion_transformer_w4a4_b200 import build

    build.build()
    build.build(debug=True)
    rel = _run(tmp_path, "release")
    dbg = _run(tmp_path, "debug")
    assert int(rel["debug"]) == 0 and int(dbg["debug"]) == 1
    assert rel.keys() == dbg.keys() and len(rel) > 70
    for k in rel:
        if k.endswith("status"):
            assert int(dbg[k]) == 0 and int(rel[k]) == 0, (k, int(dbg[k]), int(rel[k]))
        elif k != "debug":
            np.testing.assert_array_equal(dbg[k], rel[k], err_msg=k)
