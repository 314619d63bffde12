"""Norm and rotation over layouts that are allowed and rare: single heads, heads of one tensor, in place, padded batches with positions,
broadcast inputs: the same bits as over tensors of their own."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


@pytest.mark.parametrize("B,N,H,Hkv", [(2, 50, 4, 1), (2, 50, 1, 3), (3, 50, 1, 1), (1, 50, 4, 1), (3, 1, 4, 1), (1, 1, 1, 1)])
@pytest.mark.parametrize("d", [64, 72])
def test_heads_of_one_tensor(fa, B, N, H, Hkv, d):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g).half().cuda()  # noqa: E731
    x, wq, wk, table = r(B, N, H + Hkv, d), r(d), r(d), fa.rope_table(N, d)
    q, k = x[:, :, :H], x[:, :, H:]
    want = fa.qk_norm_rope(q, k, wq, wk, table)
    y = torch.full((B, H + Hkv, N, d), 7.0, dtype=torch.float16, device="cuda")
    fa.fa_qk_norm_rope(q, k, wq, wk, table, y[:, :H].transpose(1, 2), y[:, H:].transpose(1, 2))
    assert torch.equal(y[:, :H], want[0]) and torch.equal(y[:, H:], want[1])
    dy = r(B, H + Hkv, N, d)
    grads = fa.qk_norm_rope_backward(dy[:, :H], dy[:, H:], q, k, wq, wk, table)
    dwq, dwk = torch.empty_like(wq), torch.empty_like(wk)
    dq, dk = dy[:, :H].transpose(1, 2), dy[:, H:].transpose(1, 2)
    fa.fa_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, table, dq, dk, dwq, dwk)  # over the gradients that it reads
    assert all(torch.equal(a, b) for a, b in zip(grads, (dq, dk, dwq, dwk)))
    fa.fa_check_device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_padded_batch_with_positions_of_its_own(fa, dtype, interleaved):
    """Each sequence the same as packed rows at its positions; the weights' gradients are the sums over all of them."""
    B, N, H, Hkv, d = 3, 37, 4, 2, 96
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    x, wq, wk, table = r(B, N, H + Hkv, d), r(d).float(), r(d).float(), fa.rope_table(500, 64)
    pos = torch.randint(0, 500, (B, N), generator=g, dtype=torch.int32).cuda()
    kw = {"interleaved": interleaved}
    qo, ko = fa.qk_norm_rope(x[:, :, :H], x[:, :, H:], wq, wk, table, pos, **kw)
    dqo, dko = r(B, H, N, d), r(B, Hkv, N, d)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dqo, dko, x[:, :, :H], x[:, :, H:], wq, wk, table, pos, **kw)
    sums = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for b in range(B):
        q1, k1 = fa.qk_norm_rope(x[b, :, :H], x[b, :, H:], wq, wk, table, pos[b], **kw)
        assert torch.equal(qo[b].transpose(0, 1), q1) and torch.equal(ko[b].transpose(0, 1), k1)
        g1 = fa.qk_norm_rope_backward(dqo[b].transpose(0, 1), dko[b].transpose(0, 1), x[b, :, :H], x[b, :, H:], wq, wk, table, pos[b],
                                      **kw)
        assert torch.equal(dq[b], g1[0]) and torch.equal(dk[b], g1[1])
        for s, t in zip(sums, g1[2:]):
            s += t.double()
    # sums of up to 444 fp32 terms in another order: 2^-24 for each of them, relative to the terms, which are 4 on average at most
    for s, t in zip(sums, (dwq, dwk)):
        assert ((t.double() - s).abs() <= B * N * H * 2.0 ** -24 * B * N * H * 4).all()
    fa.fa_check_device_error()


def test_inputs_that_are_broadcast(fa):
    """Steps of 0 between batches, tokens or heads of what is read."""
    B, N, H, Hkv, d = 3, 20, 4, 4, 64
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k = r(1, N, H, d).expand(B, N, H, d), r(B, N, 1, d).expand(B, N, Hkv, d)
    dqo, dko = r(1, 1, 1, d).expand(B, H, N, d), r(B, 1, N, d).expand(B, Hkv, N, d)
    w, table = r(d), fa.rope_table(N, d)
    real = [t.contiguous() for t in (dqo, dko, q, k)]
    assert all(torch.equal(a, b) for a, b in zip(fa.qk_norm_rope(q, k, w, w, table), fa.qk_norm_rope(*real[2:], w, w, table)))
    got, want = (fa.qk_norm_rope_backward(*t, w, w, table) for t in ((dqo, dko, q, k), real))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    fa.fa_check_device_error()
