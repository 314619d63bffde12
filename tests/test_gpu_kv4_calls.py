"""Calls of the decode over the 4-bit cache that the documentation allows: without a workspace, with a row of NaN among rows
that see different slots."""

import pytest

from test_gpu_kv4 import TORCH, fa, i32, make_cache  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_without_a_workspace(fa):  # noqa: F811
    B, H, hkv, d, cap = 3, 8, 2, 128, 2048
    cache, _, _ = make_cache(B, hkv, cap, d, 90)
    q = torch.randn(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
    lens = i32([2000, 7, 900])
    w = torch.zeros(B, hkv, cap, device="cuda")
    ref, ref_l = fa.attention_decode_kv4(q, cache, lens, weights_out=w)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        for weights in (False, True):
            o, lse, w2 = torch.zeros_like(ref), torch.zeros_like(ref_l), torch.zeros_like(w)
            torch.cuda.synchronize()
            fa.fa_decode_kv4(q, cache, lens, o, lse, d ** -0.5, weights_out=w2 if weights else None, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(o, ref) and torch.equal(lse, ref_l) and (not weights or torch.equal(w2, w))
    # no query rows: no workspace, nothing to do
    fa.fa_decode_kv4(q[:, :, :0], cache, lens, ref[:, :, :0], ref_l[:, :, :0], d ** -0.5)
