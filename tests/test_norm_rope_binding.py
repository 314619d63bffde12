"""What the binding refuses of norm and rotation calls before it looks for a GPU (CPU tensors; nothing is launched)."""

import pytest

torch = pytest.importorskip("torch")

from exact_tiled_attention_07_gb300 import binding as fa  # noqa: E402


@pytest.mark.parametrize("which", [0, 1])
def test_a_weight_gradient_without_its_own_weight_has_the_other_weights_dtype(which):
    """The library writes both in one dtype: d floats into a 16-bit tensor would end behind it."""
    q, k, t = torch.zeros(4, 2, 64).half(), torch.zeros(4, 1, 64).half(), torch.zeros(8, 64)
    weights, grads = [None, None], [torch.zeros(64), torch.zeros(64)]
    weights[which], grads[1 - which] = torch.ones(64), torch.zeros(64).half()
    with pytest.raises(ValueError, match="weights' dtype"):
        fa.fa_qk_norm_rope_bwd(q, k, q, k, *weights, t, q, k, *grads)
    grads[1 - which] = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):  # nothing else is wrong with it
        fa.fa_qk_norm_rope_bwd(q, k, q, k, *weights, t, q, k, *grads)


def test_more_rows_than_a_c_int_counts_are_refused():
    """(ctypes takes the low 32 bits: 2^32 + 5 tokens would be 5.)"""
    many = torch.zeros(1).expand(2 ** 32 + 5, 1, 8)
    with pytest.raises(ValueError, match="too many rows"):
        fa.qk_norm_rope(many, many, None, None, None)
    with pytest.raises(ValueError, match="too many rows"):
        fa.qk_norm_rope_backward(many, many, many, many, None, None, None, out=(many, many))


@pytest.mark.parametrize("B,N,H,Hkv", [(2, 10, 4, 1), (2, 10, 1, 3), (2, 10, 1, 1), (1, 10, 4, 1), (3, 1, 4, 1), (1, 1, 1, 1)])
def test_results_may_be_heads_of_one_tensor_with_one_head_each_too(B, N, H, Hkv, monkeypatch):
    """Qo = y[:, :H], Ko = y[:, H:] of y [B, H + Hkv, N, d]: a one-head tensor's stride between heads is open, and says nothing against
    it. (Without a GPU the call ends behind the checks, with an error of CUDA's; with one it runs.)"""
    from exact_tiled_attention_07_gb300 import build

    build.build()
    if torch.cuda.is_available():
        pytest.skip("where there is a GPU, a call that is not refused would run on these pointers")
    monkeypatch.setattr(fa, "_ready", lambda *ts, strided=(): None)
    monkeypatch.setattr(fa, "_current", lambda stream: 0)
    d = 64
    x, y = torch.zeros(B, N, H + Hkv, d).half(), torch.zeros(B, H + Hkv, N, d).half()
    q, k = x[:, :, :H], x[:, :, H:]
    qo, ko = y[:, :H].transpose(1, 2), y[:, H:].transpose(1, 2)
    with pytest.raises(fa.FAError) as e:
        fa.fa_qk_norm_rope(q, k, None, None, None, qo, ko)
    assert e.value.status == 3, str(e.value)
    # one row too close is refused as before
    if B * N * (H + Hkv) > 2:
        flat = torch.zeros(B * (H + Hkv) * N * d).half()
        near = flat[:y.numel()].view(y.shape)
        low = near[:, H:].as_strided(near[:, H:].shape, near.stride(), (H * N - 1) * d).transpose(1, 2)
        with pytest.raises(fa.FAError) as e:
            fa.fa_qk_norm_rope(q, k, None, None, None, near[:, :H].transpose(1, 2), low)
        assert e.value.status == 1
