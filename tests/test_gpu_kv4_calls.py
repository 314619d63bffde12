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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [90, 1500])  # one CTA has the head, several have
def test_weights_of_slots_that_a_row_of_nan_does_not_see(fa, d, n):  # noqa: F811
    # causal, four new rows: a NaN in the first one's query is in the weights of the slots that it sees, and not in those of
    # the three behind it
    cap, nq = 1536, 4
    cache, _, _ = make_cache(2, 1, cap, d, 91)
    g = torch.Generator().manual_seed(92)
    q = torch.randn(2, 2, nq, d, generator=g).bfloat16().cuda()
    w = [torch.zeros(2, 1, cap, device="cuda") for _ in range(2)]
    fa.attention_decode_kv4(q, cache, i32([n, n]), causal=True, weights_out=w[0])
    q[0, 1, 0, 3] = float("nan")
    fa.attention_decode_kv4(q, cache, i32([n, n]), causal=True, weights_out=w[1])
    fa.fa_check_device_error()
    assert torch.isnan(w[1][0, 0, :n - 3]).all()
    # each result is within 2 ds + 2^-18 of the formula, relative, with ds = (d / 16 + 8) 2^-21 |q| . |k| scale below 2^-10
    # (|q| . |k| scale < 85), and within 9 roundings of its sum
    a, b = (x[0, 0, n - 3:n] for x in w)
    assert ((a - b).abs() <= 2 * (2.0 ** -9 + 2.0 ** -18 + 9 * 2.0 ** -24) * a).all(), (a, b)
    assert torch.equal(w[0][1], w[1][1])
