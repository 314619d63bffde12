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
