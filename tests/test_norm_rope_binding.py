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
