"""The FA_DEBUG build runs the windowed, packed and cache kernels with its index checks: no false alarm, the same bits as the
release build.  (Loaded in place of the release build for this module, which is put back afterwards.)"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def calls(fa, d):
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, do = r(2, 4, 700, d), r(2, 2, 700, d), r(2, 2, 700, d), r(2, 4, 700, d)
    kw = {"causal": True, "window": 150, "sinks": 5}
    o, lse = fa.attention_forward(q, k, v, **kw)
    out = [o, lse, *fa.attention_backward(q, k, v, o, do, lse, **kw)[1:]]
    cu = torch.tensor([0, 300, 301, 600], dtype=torch.int32, device="cuda")
    out += fa.attention_forward_varlen(*(t[0, :, :600].transpose(0, 1) for t in (q, k, v)), cu, **kw)
    lens = torch.tensor([700, 3], dtype=torch.int32, device="cuda")
    q1 = r(2, 4, 2, d)
    out += fa.attention_decode_window(q1, k, v, lens, 150, 5)
    out += fa.attention_decode_prefix(q1, k[0], v[0], k, v, lens)
    fa.fa_check_device_error()
    return out


def test_debug_build_agrees_with_the_release_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    release = build.build()
    want = {d: calls(binding, d) for d in (64, 128, 256)}
    binding.load_library(build.build(debug=True))
    try:
        assert binding.fa_debug_build()
        for d, w in want.items():
            assert all(torch.equal(a, b) for a, b in zip(w, calls(binding, d)))
    finally:
        binding.load_library(release)
