"""Norm and rotation with a single query or key head, into heads of one tensor and in place: the same bits as into tensors of their own."""

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
