"""How far values that are not finite reach, as the header states it."""

import math

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


def randn(seed, *shape, dtype=torch.float16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("G", [1, 4, 40, 130])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_a_value_that_is_not_finite_stays_in_its_column_of_the_rows_that_see_it(fa, d, G, value):
    B, Hkv, C, P = 3, 2, 700, 300
    q, k, v = randn(1, B, G * Hkv, 1, d), randn(2, B, Hkv, C, d), randn(3, B, Hkv, C, d)
    kp, vp = randn(4, Hkv, P, d), randn(5, Hkv, P, d)
    lens = torch.tensor([700, 257, 90], dtype=torch.int32, device="cuda")

    def reached(o, lse, o2, lse2, where):
        hit = torch.zeros(B, Hkv, G, d, dtype=torch.bool, device="cuda")
        hit[where] = True
        hit = hit.view(o.shape)
        assert not o2[hit].isfinite().any() and torch.equal(o2[~hit], o[~hit]) and torch.equal(lse, lse2)

    clean = fa.attention_decode_window(q, k, v, lens, 200, 4)
    for slot in (2, 56, 57, 120, 256):  # of sequence 1: a sink, the last hidden one, the window's first, middle and last
        v2 = v.clone()
        v2[1, 1, slot, 5] = value
        seen = slot < 4 or slot >= 57
        got = fa.attention_decode_window(q, k, v2, lens, 200, 4)
        reached(*clean, *got, (1, 1, slice(None), 5) if seen else (slice(0, 0),))
    clean = fa.attention_decode_prefix(q, kp, vp, k, v, lens)
    for slot in (0, 130, 299):
        vp2 = vp.clone()
        vp2[0, slot, 7] = value
        reached(*clean, *fa.attention_decode_prefix(q, kp, vp2, k, v, lens), (slice(None), 0, slice(None), 7))
    fa.fa_check_device_error()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sinks", [1, 4, 16, 17, 33, 100, 128, 131, 200])
def test_window_a_value_behind_the_sinks_stays_with_the_queries_whose_window_is_near(fa, d, sinks):
    """Hidden values in the sinks' own tiles: the queries of a block of 256 that see sinks alone of those tiles do not get them."""
    N, window, H, Hkv = 1000, 100, 4, 2
    q, k, v = randn(1, 2, H, N, d), randn(2, 2, Hkv, N, d), randn(3, 2, Hkv, N, d)
    clean = fa.attention_forward(q, k, v, causal=True, window=window, sinks=sinks)
    cu = torch.tensor([0, 7, 7 + N, 7 + N + 60], dtype=torch.int32, device="cuda")
    pack = lambda t: torch.cat((t[0, :, :7], t[1], t[0, :, :60]), 1).transpose(0, 1)  # noqa: E731
    packed = fa.attention_forward_varlen(pack(q), pack(k), pack(v), cu, causal=True, window=window, sinks=sinks)
    last = sinks // 128 * 128 + 128  # behind the tile of the first row that is no sink
    first = (last + window - 1 + 255) // 256 * 256  # of the blocks whose windows lie behind those
    for rows in (slice(sinks, last), slice(sinks, sinks + 1)):
        for value in (math.nan, math.inf):
            v2 = v.clone()
            v2[:, :, rows] = value
            o, lse = fa.attention_forward(q, k, v2, causal=True, window=window, sinks=sinks)
            assert torch.equal(lse, clean[1])
            assert torch.equal(o[:, :, first:], clean[0][:, :, first:])
            assert not o[:, :, sinks:sinks + window].isfinite().any()
            o, lse = fa.attention_forward_varlen(pack(q), pack(k), pack(v2), cu, causal=True, window=window, sinks=sinks)
            assert torch.equal(lse, packed[1]) and torch.equal(o[7 + first:7 + N], packed[0][7 + first:7 + N])
    fa.fa_check_device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_rows_whose_squares_pass_32_bits(fa, dtype):
    x = randn(1, 5, 3, 64, dtype=dtype)
    x[2, 1] *= 1e30
    k = x[:, :1].contiguous()
    w, table = torch.ones(64, device="cuda"), fa.rope_table(5, 64)
    y, _ = fa.qk_norm_rope(x, k, w, w, table)
    clean = x.clone()
    clean[2, 1] = 1.0
    want, _ = fa.qk_norm_rope(clean, k, w, w, table)
    assert (y[2, 1] == 0).all()
    want[2, 1] = 0
    assert torch.equal(y, want)
