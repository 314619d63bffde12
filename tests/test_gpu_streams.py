"""Calls on a stream that is not the current one take no memory that work queued on the current stream still uses.

A block of each of a call's sizes is freed while kernels that read it, and then write it, wait on the current stream behind a pause (a
kernel that counts clocks). The call on the other stream is done long before them: what they read has to be what was
there, and what they write must not reach the call's results.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PAUSE = 200_000_000  # clocks: about 0.1 s


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def randn(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def qkv(B=2, H=8, Hkv=4, N=1000, d=128, seed=0):
    return randn(seed, B, H, N, d), randn(seed + 1, B, Hkv, N, d), randn(seed + 2, B, Hkv, N, d)


def forward(fa, **kw):
    q, k, v = qkv()
    return lambda s: fa.attention_forward(q, k, v, causal=True, stream=s, **kw), 0


def backward(fa, **kw):
    q, k, v = qkv()
    do = randn(9, *q.shape)
    o, lse = fa.attention_forward(q, k, v, causal=True, **kw)
    # (dK and dV: dQ's sums come in no fixed order)
    return lambda s: fa.attention_backward(q, k, v, o, do, lse, causal=True, stream=s, **kw)[1:], fa.fa_bwd_workspace_size(*q.shape)


def varlen(fa, **kw):
    x = randn(3, 2000, 16, 128)
    cu = torch.tensor([0, 700, 2000], dtype=torch.int32, device="cuda")
    return lambda s: fa.attention_forward_varlen(x[:, :8], x[:, 8:12], x[:, 12:], cu, causal=True, stream=s, **kw), 0


def caches(C=4000):
    B, H, Hkv, d = 4, 16, 4, 128
    lens = torch.tensor([C, 3000, 1, 777], dtype=torch.int32, device="cuda")
    return randn(4, B, H, 1, d), randn(5, B, Hkv, C, d), randn(6, B, Hkv, C, d), lens


def decode(fa):
    q, k, v, _ = caches()
    size = fa.fa_decode_workspace_size(4, 16, 4, 1, 4000, 128)
    return lambda s: fa.attention_decode(q, k, v, stream=s), size


def decode_window(fa):
    q, k, v, lens = caches()
    size = fa.fa_decode_window_workspace_size(4, 16, 4, 1, 4000, 128)
    return lambda s: fa.attention_decode_window(q, k, v, lens, 3000, 4, stream=s), size


def decode_prefix(fa):
    q, k, v, lens = caches()
    kp, vp = randn(7, 4, 5000, 128), randn(8, 4, 5000, 128)
    size = fa.fa_decode_prefix_workspace_size(4, 16, 4, 1, 5000, 4000, 128)
    return lambda s: fa.attention_decode_prefix(q, kp, vp, k, v, lens, stream=s), size


def decode_window_into(fa):
    q, k, v, lens = caches()
    o, lse = torch.empty_like(q), torch.empty(4, 16, 1, device="cuda")

    def call(s):
        fa.fa_decode_window(q, k, v, lens, o, lse, 0.1, 3000, 4, stream=s)
        return o, lse

    return call, fa.fa_decode_window_workspace_size(4, 16, 4, 1, 4000, 128)


def norm(fa):
    x = randn(3, 3, 700, 12, 128)
    w, table = torch.rand(128, device="cuda"), fa.rope_table(700, 128)
    return lambda s: fa.qk_norm_rope(x[:, :, :8], x[:, :, 8:], w, w, table, stream=s), 0


def norm_backward(fa):
    x = randn(3, 3, 700, 12, 128)
    w, table = torch.rand(128, device="cuda"), fa.rope_table(700, 128)
    dq, dk = randn(4, 3, 8, 700, 128), randn(5, 3, 4, 700, 128)
    call = lambda s: fa.qk_norm_rope_backward(dq, dk, x[:, :, :8], x[:, :, 8:], w, w, table, stream=s)  # noqa: E731
    return call, fa.fa_qk_norm_rope_bwd_workspace_size(128)


def kv4(fa, read):
    cache = fa.kv4_cache(4, 4, 1024, 128)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 500, 1300, 1301, 2000], [500, 800, 1, 699]))
    fa.fa_kv4_append(randn(1, 2000, 4, 128), randn(2, 2000, 4, 128), cu, lens, cache)
    if read:
        return lambda s: fa.kv4_read(cache, cu, lens, 2000, stream=s), 0
    q = randn(3, 4, 16, 1, 128)
    return lambda s: fa.attention_decode_kv4(q, cache, lens, stream=s), fa.fa_decode_kv4_workspace_size(4, 16, 4, 1, 1024, 128)


def fp8(fa, quantize):
    q, k, v = qkv()
    if quantize:
        return lambda s: fa.quantize_fp8(q, stream=s), 0
    (q8, qs), (k8, ks), (v8, vs) = (fa.quantize_fp8(x) for x in (q, k, v))
    return lambda s: fa.attention_forward_fp8(q8, k8, v8, qs, ks, vs, causal=True, stream=s), 0


CALLS = {
    "forward": forward, "forward_window": lambda fa: forward(fa, window=300), "forward_sinks": lambda fa: forward(fa, window=300, sinks=4),
    "backward": backward, "backward_window": lambda fa: backward(fa, window=300),
    "backward_sinks": lambda fa: backward(fa, window=300, sinks=4), "varlen": varlen,
    "varlen_sinks": lambda fa: varlen(fa, window=300, sinks=4), "decode": decode, "decode_window": decode_window,
    "decode_window_into": decode_window_into, "decode_prefix": decode_prefix, "norm": norm, "norm_backward": norm_backward,
    "kv4_read": lambda fa: kv4(fa, True), "decode_kv4": lambda fa: kv4(fa, False), "quantize_fp8": lambda fa: fp8(fa, True),
    "forward_fp8": lambda fa: fp8(fa, False),
}


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", list(CALLS))
def test_freed_blocks_with_work_queued_are_left_alone(fa, name, raw):
    call, scratch = CALLS[name](fa)
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + ([scratch] if scratch else [])
    side = torch.cuda.Stream()
    call(side)  # (what a first call sets up)
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    read = [b.clone() for b in blocks]
    for b in blocks:
        b.fill_(5)
    del blocks, b
    got = call(side.cuda_stream if raw else side)
    side.synchronize()
    assert all(torch.equal(r, torch.full_like(r, 3)) for r in read)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    fa.fa_check_device_error()


def test_results_of_another_stream_may_be_read_later(fa):
    """A result that is dropped while the current stream still has reads of it queued: the other stream's next call does not get its
    memory."""
    q, k, v = qkv()
    want = fa.attention_forward(q, k, v, causal=True, window=300, sinks=4)[0]
    side = torch.cuda.Stream()
    o, _ = fa.attention_forward(q, k, v, causal=True, window=300, sinks=4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    later = o.clone()
    del o, _
    for i in range(3):
        fa.attention_forward(q * 2, k, v, causal=True, window=300, sinks=4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(later, want)


@pytest.mark.parametrize("name", ["forward_sinks", "backward_sinks", "decode_window", "norm_backward", "decode_kv4"])
def test_a_stream_that_joins_a_capture(fa, name):
    """Results and workspaces of a call on another stream inside a capture belong to the graph."""
    call, _ = CALLS[name](fa)
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = call(side)
        call(side)  # (results that are dropped inside the capture)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in first:
            t.fill_(0)
        others = [torch.full_like(t, 7) for t in first for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, want))
        assert all((t == 7).all() for t in others)
    fa.fa_check_device_error()


def test_the_default_stream_by_its_handle(fa):
    q, k, v = qkv()
    want = fa.attention_forward(q, k, v, causal=True, window=300, sinks=4)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = fa.attention_forward(q, k, v, causal=True, window=300, sinks=4, stream=0)
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        got = [t.clone() for t in got]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
