"""Arguments that the serving calls refuse before anything is launched (no GPU: the pointers are not followed)."""

import pytest

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("where there is a GPU, a call that is not refused would run on these pointers")
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


# cache of 1 x 2 heads of 128 slots: 2 x 2 x 72 x 64 bytes; out_cache of 64 slots: half of that
@pytest.mark.parametrize("which,at", [
    ("out_cache", ("cache", 16)), ("out_cache", ("cache", 2 * 2 * 72 * 64 - 16)), ("out_cache", ("cache", -16)),
    ("out_weights", ("weights", 4)), ("out_weights", ("weights", -4)), ("out_weights", ("cache", 64)),
    ("kept", ("weights", 0)), ("kept", ("lens", 0)), ("kept", ("out_cache", 2 * 72 * 64 - 4)), ("out_lens", ("kept", 8)),
    ("out_weights", ("lens", -4)), ("out_lens", ("lens", 4)), ("out_lens", ("cache", 0)), ("kept", ("out_weights", 0))])
def test_evict_refuses_overlaps(lib, which, at):
    names = ("cache", "weights", "lens", "out_cache", "out_weights", "out_lens", "kept")
    ptr = dict(zip(names, P))
    ptr[which] = ptr[at[0]] + at[1]

    def call(B=2):
        return lib.fa_kv4_evict(ptr["cache"], ptr["weights"], ptr["lens"], 32, 3, ptr["out_cache"], ptr["out_weights"],
                                ptr["out_lens"], ptr["kept"], B, 2, 128, 64, 64, None)

    assert call() == INVALID and "another" in message(lib), message(lib)


# (token stride, head stride) of 3 rows of 2 heads, d = 128, where two output rows share elements
@pytest.mark.parametrize("ts,hs", [(128, 128), (128, 256), (192, 320), (256, 256), (312, 192)])
def test_output_rows_over_one_another(lib, ts, hs):
    good = (256, 128)
    for k, v in (((ts, hs), good), (good, (ts, hs))):
        assert lib.fa_kv4_read(*P[:5], 1, 3, 2, 128, 128, *k, *v, BF16, None) == INVALID and "output" in message(lib)
    assert lib.fa_fwd_varlen(*P[:6], 1, 3, 2, 2, 128, *good, *good, *good, ts, hs, 0.1, 1, BF16, None) == INVALID
    assert "output" in message(lib)


# rows that lie apart pass this check (the call then ends at its number of rows)
@pytest.mark.parametrize("ts,hs", [(256, 128), (1024, 128), (1024, 512), (384, 256)])
def test_output_rows_apart(lib, ts, hs):
    T = 2 ** 31 - 1
    assert lib.fa_kv4_read(*P[:5], 1, T, 2, 128, 128, ts, hs, ts, hs, BF16, None) == INVALID
    assert "too many" in message(lib)


def test_weights_need_query_rows(lib):
    # weights_out = weights_in + nothing is a copy that the call does not make; in place there is nothing to do
    for H, nq in ((0, 1), (4, 0)):
        decode = lambda w_in, w_out, B=1: lib.fa_decode_kv4(  # noqa: E731
            *P[:5], w_in, w_out, B, H, 2, nq, 128, 64, 0.1, 0, BF16, P[7], 1 << 30, None)
        assert decode(P[5], P[6]) == INVALID and "query rows" in message(lib)
        assert decode(None, P[6]) == INVALID
        assert decode(P[6], P[6]) == 0 and decode(None, None) == 0 and decode(P[5], P[6], B=0) == 0


def test_weights_partly_over_one_another(lib):
    for at in (4, -4, 4 * 127):
        assert lib.fa_decode_kv4(*P[:5], P[6] + at, P[6], 1, 4, 1, 1, 128, 64, 0.1, 0, BF16, P[7], 1 << 30, None) == INVALID
        assert "weights_in" in message(lib)
