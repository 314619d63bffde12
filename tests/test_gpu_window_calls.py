"""Calls with windows and sinks that are allowed and rare: the largest arguments, other streams, long items."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_window import run  # noqa: E402


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def make(B, H, Hkv, N, d, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g).to(dtype).cuda() for h in (H, Hkv, Hkv, H)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [301, 2 ** 31 - 200, 2 ** 31 - 1])
def test_a_masked_window_past_every_length_hides_nothing(fa, causal, window):
    """(A window of N rows, by the same kernels, is the reference: nothing is hidden, and no sum changes its order.)"""
    q, k, v, do = make(1, 4, 2, 300, 64, 1)
    o, lse = fa.attention_forward(q, k, v, causal=causal, window=300)
    o2, lse2 = fa.attention_forward(q, k, v, causal=causal, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    grads = fa.attention_backward(q, k, v, o, do, lse, causal=causal, window=300)
    grads2 = fa.attention_backward(q, k, v, o, do, lse, causal=causal, window=window)
    assert torch.equal(grads[1], grads2[1]) and torch.equal(grads[2], grads2[2])
    # (dQ's sums come in no fixed order, in 32 bits: a unit in the last place now and then)
    assert ((grads[0].double() - grads2[0].double()).abs() <= 2.0 ** -7 * grads[0].double().abs() + 1e-5).all()
    fa.fa_check_device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N,window,sinks", [(257, 300, 0), (1000, 300, 5), (640, 33, 0), (300, 40, 300)])
def test_first_queries_of_a_sequence_see_few_keys(fa, dtype, d, N, window, sinks):
    """dQ of a sequence's first 64 queries under a longer window, by the bound of queries whose D does not come from the rounded O:
    dS = p (dP - D) off by (e + 2 ds) |dS| + p (2 ds sum p |dP| + 2 the error of dP), e the rounding of dS to 16 bits and ds that of
    a score, (d / 16 + 8) 2^-23 |q| |k| scale + 2^-20; dQ rounded once more."""
    B, H, Hkv, rows = 6, 8, 4, 64
    q, k, v, do = make(B, H, Hkv, N, d, N + d, dtype)
    scale, e = d ** -0.5, torch.finfo(dtype).eps / 2
    o, lse = fa.attention_forward(q, k, v, causal=True, window=window, sinks=sinks)
    dq = fa.attention_backward(q, k, v, o, do, lse, causal=True, window=window, sinks=sinks)[0]
    fa.fa_check_device_error()
    i, j = torch.arange(rows, device="cuda")[:, None], torch.arange(rows, device="cuda")
    hidden = (j > i) | ((i - j >= window) & (j >= sinks))
    q1, do1, got = (x[:, :, :rows].double() for x in (q, do, dq))
    k1, v1 = (x[:, :, :rows].double().repeat_interleave(H // Hkv, 1) for x in (k, v))
    ds = (d / 16 + 8) * 2.0 ** -23 * scale * float(q1.norm(dim=-1).max() * k1.norm(dim=-1).max()) + 2.0 ** -20
    p = torch.softmax((q1 @ k1.transpose(-1, -2) * scale).masked_fill(hidden, float("-inf")), -1)
    dp = do1 @ v1.transpose(-1, -2)
    g = p * (dp - (p * dp).sum(-1, keepdim=True))
    dp_tol = (d / 16 + 8) * 2.0 ** -23 * do1.norm(dim=-1, keepdim=True) * v1.norm(dim=-1).max()
    g_tol = (e + 2 * ds) * g.abs() + p * (2 * ds * (p * dp.abs()).sum(-1, keepdim=True) + 2 * dp_tol)
    want = scale * (g @ k1)
    worst = ((got - want).abs() / (e * want.abs() + scale * (g_tol @ k1.abs()) + 2.0 ** -24)).max()
    assert worst <= 1, float(worst)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv,N,window,sinks", [(8, 1, 4097, 256, 4), (16, 2, 2500, 700, 300), (12, 1, 3001, 1, 1)])
def test_many_query_heads_over_a_long_sequence(fa, d, H, Hkv, N, window, sinks):
    """The key tiles with sinks meet all later queries of all heads of their group: thousands of steps of one block in the backward."""
    run(fa, 1, H, Hkv, N, d, "bf16", window, sinks)


@pytest.mark.parametrize("window", [1, 8, 32, 300])
def test_backward_in_graphs_that_share_a_workspace_and_on_streams_of_their_own(fa, window):
    """D's launch and the preprocess beside it: replayed, in turn with another call over the same workspace, and side by side with
    calls over others. dV and dK do not depend on the run, dQ's sums (in no fixed order, in 32 bits) on a unit in the last place."""
    shapes = [(2, 4, 2, 700, 128), (1, 8, 8, 1500, 64)]
    calls = []
    ws = torch.empty(max(fa.fa_bwd_workspace_size(B, H, N, d) for B, H, _, N, d in shapes), dtype=torch.uint8, device="cuda")
    for i, (B, H, Hkv, N, d) in enumerate(shapes):
        q, k, v, do = make(B, H, Hkv, N, d, i)
        o, lse = fa.attention_forward(q, k, v, causal=True, window=window, sinks=0)
        kw = {"causal": True, "window": window, "sinks": 0}
        calls.append(lambda a=(q, k, v, o, do, lse), kw=kw, **more: fa.attention_backward(*a, **kw, **more))
    want = [call() for call in calls]

    def same(got, ref):
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
        assert ((got[0].double() - ref[0].double()).abs() <= 2.0 ** -7 * ref[0].double().abs() + 1e-5).all()

    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(workspace=ws))
        graphs.append(graph)
    ws.fill_(255)
    for _ in range(3):
        for i in (0, 1):
            graphs[i].replay()
            same(calls[1 - i](workspace=ws), want[1 - i])
            same(outs[i], want[i])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [[call(stream=s) for s in streams] for _ in range(4) for call in calls]
    torch.cuda.synchronize()
    for n, outs in enumerate(many):
        for got in outs:
            same(got, want[n % 2])
    fa.fa_check_device_error()
