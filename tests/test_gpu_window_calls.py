"""Calls with windows and sinks that are allowed and rare: the largest arguments, other streams, long items."""

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


def make(B, H, Hkv, N, d, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g).to(dtype).cuda() for h in (H, Hkv, Hkv, H)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [301, 2 ** 31 - 200, 2 ** 31 - 1])
def test_a_masked_window_past_every_length_hides_nothing(fa, causal, window):
    """(A window of N rows, by the same kernels, is the reference: nothing is hidden, and no sum changes its order.)"""
    q, k, v, do = make(1, 4, 2, 300, 64, 1)
    o, lse = fa.attention_forward(q, k, v, causal=causal, window=300)
    o2, lse2 = fa.attention_forward(q, k, v, causal=causal, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    grads = fa.attention_backward(q, k, v, o, do, lse, causal=causal, window=300)
    grads2 = fa.attention_backward(q, k, v, o, do, lse, causal=causal, window=window)
    assert torch.equal(grads[1], grads2[1]) and torch.equal(grads[2], grads2[2])
    # (dQ's sums come in no fixed order, in 32 bits: a unit in the last place now and then)
    assert ((grads[0].double() - grads2[0].double()).abs() <= 2.0 ** -7 * grads[0].double().abs() + 1e-5).all()
    fa.fa_check_device_error()
