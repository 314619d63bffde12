"""The fp64 statement of the 4-bit cache: pins of the format by hand, its error bound, the decode against
a plain softmax and eviction by hand; and the binding's refusals, which come before the library is called."""

import numpy as np
import pytest

from oracle import kv4 as KV

torch = pytest.importorskip("torch")

from exact_tiled_attention_07_gb300 import binding as fa  # noqa: E402


def test_format_by_hand():
    x = np.arange(64, dtype=np.float32) / 63 * 15 - 8  # -8 .. 7: step 1, middle 0
    codes, step, middle = KV.quantize_rows(x[None])
    assert step[0, 0] == 1 and middle[0, 0] == 0
    assert np.array_equal(codes[0], np.rint(x) + 8)
    const = np.full((1, 64), 3.0, np.float32)
    codes, step, middle = KV.quantize_rows(const)
    assert (codes == 8).all() and step[0, 0] == 0 and middle[0, 0] == 3
    bad = const.copy()
    bad[0, 5] = 40000.0
    _, step, middle = KV.quantize_rows(bad)
    assert np.isnan(step[0, 0]) and np.isnan(middle[0, 0])


@pytest.mark.parametrize("scale,offset", [(1.0, 0.0), (1e-3, 0.0), (1.0, 300.0), (3000.0, 0.0), (1e-7, 0.0)])
def test_error_bound(scale, offset):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((200, 128)) * scale + offset).astype(np.float32)
    codes, step, middle = KV.quantize_rows(x)
    err = np.abs(KV.dequantize_rows(codes, step, middle) - x).reshape(200, 2, 64).max(-1)
    s, m = step.astype(np.float64), np.abs(middle.astype(np.float64))
    # a middle's rounding moves the ends of the range by half a step of fp16 (2^-11 of it; 2^-25 below
    # the normal numbers); x itself carries fp32 roundings of the two sums
    assert (err <= np.maximum(s / 2, m * 2.0 ** -11 + 2.0 ** -25) + 2.0 ** -22 * np.abs(x).max()).all()


def test_blocks_round_trip():
    rng = np.random.default_rng(4)
    k, v = (KV.quantize_rows(rng.standard_normal((2, 128, 64)).astype(np.float32)) for _ in range(2))
    blocks = KV.pack_blocks(k, v)
    assert blocks.shape == (2, 2, 72 * 64)
    for a, b in zip(KV.unpack_blocks(blocks), (k, v)):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_decode_by_hand():
    q = np.ones((1, 1, 2, 64))
    k = np.zeros((1, 1, 64, 64))
    v = np.arange(64.0)[None, None, :, None] * np.ones(64)
    o, L, w, _ = KV.decode64(q, k, v, [3], 0.1, True)
    assert np.allclose(o[0, 0, :, 0], [0.5, 1.0]) and np.allclose(L[0, 0], np.log([2, 3]))
    assert np.allclose(w[0, 0, :4], [0.5 + 1 / 3, 0.5 + 1 / 3, 1 / 3, 0])


def test_eviction_by_hand():
    w = np.array([1, 5, 5, np.nan, 0, 2, 9, 9], np.float32)
    assert KV.evict(w, 8, 4, 2).tolist() == [1, 3, 6, 7]
    assert KV.evict(w, 8, 5, 2).tolist() == [1, 2, 3, 6, 7]
    assert KV.evict(w, 3, 4, 2).tolist() == [0, 1, 2]
    assert KV.evict(np.zeros(8, np.float32), 8, 3, 0).tolist() == [0, 1, 2]


def test_refusals_before_the_library():
    cache = fa.kv4_cache(2, 2, 100, 64, device="cpu")
    assert tuple(cache.shape) == (2, 2, 2, 72 * 64)
    with pytest.raises(ValueError, match="supports d"):
        fa.kv4_cache(1, 1, 64, 96, device="cpu")
    rows, lens = torch.zeros(5, 2, 64), torch.zeros(2, dtype=torch.int32)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    q, L = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 1)
    w = torch.zeros(2, 2, 128)
    for call in (lambda: fa.fa_kv4_append(rows, rows, cu, lens, cache), lambda: fa.fa_kv4_read(cache, cu, lens, rows, rows),
                 lambda: fa.fa_decode_kv4(q, cache, lens, q, L, 0.1),
                 lambda: fa.fa_fwd_varlen(rows, rows, rows, rows, torch.zeros(2, 5), cu, 0.1, True),
                 lambda: fa.fa_kv4_evict(cache, w, lens, 8, 2, cache, w, lens, torch.zeros(32, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    with pytest.raises(ValueError, match="last dimension"):
        fa.fa_kv4_append(torch.zeros(5, 2, 128)[..., ::2], rows, cu, lens, cache)
    with pytest.raises(ValueError, match="packed"):
        fa.fa_kv4_append(rows[0], rows, cu, lens, cache)
    with pytest.raises(ValueError, match="4-bit cache is"):
        fa.fa_decode_kv4(q, cache.float(), lens, q, L, 0.1)


def test_packed_strides():
    t = torch.zeros(7, 10, 64)
    assert fa._packed(t[:, 2:5], "K") == (7, 3, 64, 640, 64)
    assert fa._packed(t.transpose(0, 1)[:1, :3], "K") == (1, 3, 64, 192, 640)  # one row: its own stride is free
    assert fa._packed(t[:, :1], "K")[3:] == (640, 64)
