"""Rows of no sequence are not read by fa_kv4_append: the debug build checks every row that it loads (an index check that
records an error and skips the load; all rows are backed by memory here)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    release = build.build()
    binding.load_library(build.build(debug=True))
    try:
        yield binding
    finally:
        binding.load_library(release)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu,lens", [([0, 3, 7], [3, 64]), ([5, 9, 9], [4, 0]), ([30, 30, 64], [1, 34])])
def test_rows_of_no_sequence_are_not_read(fa, cu, lens, dtype):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.randn(64, 2, 128, device="cuda").to(dtype)
    cache = fa.kv4_cache(2, 2, 64, 128)
    fa.fa_kv4_append(k, -k, i32(cu), i32(lens), cache)
    fa.fa_check_device_error()
    rk, rv = fa.kv4_read(cache, i32(cu), i32(lens), 64, dtype=dtype)
    fa.fa_check_device_error()
    own = slice(cu[0], cu[-1])
    # steps of a group of 64 normal numbers are below (4.5 + 4.5) / 15
    assert (rk[own].float() - k[own].float()).abs().max() < 0.35 and (rv[own].float() + k[own].float()).abs().max() < 0.35
