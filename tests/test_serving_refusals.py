"""Arguments that the serving calls refuse before anything is launched (no GPU: the pointers are not followed)."""

import ctypes

import pytest

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding.load_library()


def message(lib):
    return lib.fa_last_error_message().decode()


P = [0x10000000 * (i + 1) for i in range(12)]  # 256 MB apart
BF16 = 0


def append(lib, capacity=128, T=3, strides=(256, 128) * 2):
    return lib.fa_kv4_append(*P[:5], None, 1, T, 2, capacity, 128, *strides, BF16, None)


def test_the_dtype_code(lib):
    import torch

    from exact_tiled_attention_07_gb300 import binding

    assert binding.DTYPE_CODES[torch.bfloat16] == BF16


# slots are counted in 32 bits, up to some thousand behind the last one
@pytest.mark.parametrize("capacity", [2 ** 31 - 64, 2 ** 31 - 1024])
def test_capacity_near_the_end_of_32_bits(lib, capacity):
    assert append(lib, capacity) == INVALID and "too large" in message(lib)
    assert lib.fa_kv4_read(*P[:5], 1, 3, 2, capacity, 128, 256, 128, 256, 128, BF16, None) == INVALID
    for weights in (0, 1):
        assert lib.fa_decode_kv4_workspace_size(1, 1, 1, 1, capacity, 64, weights) == 0
    assert lib.fa_decode_kv4(*P[:5], None, None, 1, 1, 1, 1, capacity, 64, 0.1, 0, BF16, P[6], 1 << 62, None) == INVALID
    assert "too large" in message(lib)
    for caps in ((capacity, 128), (128, capacity)):
        assert lib.fa_kv4_evict(*P[:3], 64, 3, *P[3:7], 1, 1, *caps, 64, None) == INVALID and "too large" in message(lib)
    # a capacity of 2^31 - 8192 is one
    assert lib.fa_decode_kv4_workspace_size(1, 1, 1, 1, 2 ** 31 - 8192, 64, 1) > 4 * (2 ** 31 - 8192)
