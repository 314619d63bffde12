"""Causal attention with a sliding window and sinks (forward, gradients, packed prompts) vs its definition in 64 bits.

Tolerances (e = EPS, half a step of the 16-bit type, relative).  Scores are fp32 sums of d products, L and the exponentials fp32:
together ds = (d / 16 + 8) 2^-23 |q| |k| scale + 2^-20 of a score, so a probability is off by (2 ds) p before it is rounded (e p).
O: |O| e + e sum p |v| + 2 ds max |v|.  Gradients: dV sums rounded p times dO; dS = p (dP - D) takes p unrounded and is rounded itself, and D = sum
dO O takes the rounded O, so D is off by dD = sum |dO| |dO's O error|; dS by (e + 2 ds) |dS| + p (dD + (d / 16 + 8) 2^-23 |dO| |v|);
dQ and dK sum dS times k and q; each is rounded once at the end (e).
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def visible(n, window, sinks):
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")
    return (j <= i) & ((i - j < window) | (j < sinks))


def reference(q, k, v, window, sinks, scale, do=None):
    """(value, tolerance) of O, L and, with dO, dQ, dK, dV of one head group: q, do [g, n, d], k, v [n, d]."""
    e = EPS["bf16" if q.dtype == torch.bfloat16 else "fp16"]
    q, k, v = q.double(), k.double(), v.double()
    n, d = k.shape
    ds = (d / 16 + 8) * 2.0 ** -23 * scale * float(q.norm(dim=-1).max() * k.norm(dim=-1).max()) + 2.0 ** -20
    s = (q @ k.T * scale).masked_fill(~visible(n, window, sinks), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    o = p @ v
    o_tol = e * (o.abs() + p @ v.abs()) + (2 * ds + 2.0 ** -20) * v.abs().max()
    out = {"o": (o, o_tol), "lse": (lse, ds + 2.0 ** -20 * (8 + lse.abs()))}
    if do is None:
        return out
    do = do.double()
    dp = do @ v.T
    big = (do * o).sum(-1, keepdim=True)
    g = p * (dp - big)
    big_tol = (do.abs() * o_tol).sum(-1, keepdim=True)
    dp_tol = (d / 16 + 8) * 2.0 ** -23 * do.norm(dim=-1, keepdim=True) * v.norm(dim=-1).max()
    g_tol = (e + 2 * ds) * g.abs() + p * (big_tol + dp_tol)
    dq, dk, dv = scale * (g @ k), scale * (g.transpose(-1, -2) @ q).sum(0), (p.transpose(-1, -2) @ do).sum(0)
    out["dq"] = dq, e * dq.abs() + scale * (g_tol @ k.abs()) + 2.0 ** -24
    out["dk"] = dk, e * dk.abs() + scale * (g_tol.transpose(-1, -2) @ q.abs()).sum(0) + 2.0 ** -24
    out["dv"] = dv, e * dv.abs() + (e + 2 * ds) * (p.transpose(-1, -2) @ do.abs()).sum(0) + 2.0 ** -24
    return out


def close(got, ref):
    value, tol = ref
    assert got.isfinite().all()
    worst = ((got.double() - value).abs() / tol).max()
    assert worst <= 1, float(worst)


def make(B, H, Hkv, N, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g).to(TORCH[dtype]).cuda() for h in (H, Hkv, Hkv, H)]


def run(fa, B, H, Hkv, N, d, dtype, window, sinks, seed=0, backward=True):
    q, k, v, do = make(B, H, Hkv, N, d, dtype, seed + N + window)
    scale = d ** -0.5
    o, lse = torch.full_like(q, 7.0), torch.full((B, H, N), 9.0, device="cuda")
    fa.fa_fwd_window(q, k, v, o, lse, scale, window, sinks)
    grads = None
    if backward:
        grads = [torch.full_like(t, 5.0) for t in (q, k, v)]
        ws = torch.full((fa.fa_bwd_workspace_size(B, H, N, d),), 255, dtype=torch.uint8, device="cuda")
        fa.fa_bwd_window(q, k, v, o, do, lse, *grads, ws, scale, window, sinks)
    fa.fa_check_device_error()
    G = H // Hkv
    for b in range(B):
        for h in range(Hkv):
            mine = slice(h * G, (h + 1) * G)
            ref = reference(q[b, mine], k[b, h], v[b, h], window, sinks, scale, do[b, mine] if backward else None)
            close(o[b, mine], ref["o"])
            close(lse[b, mine], ref["lse"])
            if backward:
                close(grads[0][b, mine], ref["dq"])
                close(grads[1][b, h], ref["dk"])
                close(grads[2][b, h], ref["dv"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (100, 4), (128, 128), (129, 130), (300, 5), (257, 300), (2000, 4)])
def test_windows_and_sinks_around_the_tiles(fa, dtype, d, window, sinks):
    run(fa, 1, 2, 2, 700, d, dtype, window, sinks)


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 255, 256, 257, 511, 1025])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(fa, N, d):
    run(fa, 1, 2, 1, N, d, "bf16", 50, 3)
    run(fa, 1, 2, 1, N, d, "fp16", N, N + 7)


@pytest.mark.parametrize("H,Hkv", [(3, 1), (8, 2), (7, 7), (16, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_heads(fa, H, Hkv, d):
    run(fa, 2, H, Hkv, 400, d, "bf16", 150, 9)


def test_more_items_than_one_wave(fa):
    run(fa, 3, 8, 4, 3001, 64, "fp16", 700, 200)
    run(fa, 2, 16, 16, 1500, 128, "bf16", 333, 17)


def test_largest_arguments(fa):
    top = 2 ** 31 - 1
    run(fa, 1, 2, 1, 300, 64, "fp16", top, top)
    run(fa, 1, 2, 1, 300, 128, "bf16", 10, top)
    run(fa, 1, 2, 1, 300, 256, "bf16", top, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_same_as_causal_and_as_the_masked_window(fa, d):
    q, k, v, do = make(2, 4, 2, 900, d, "bf16", 5)
    o, lse = fa.attention_forward(q, k, v, causal=True)
    for window, sinks in ((900, 1), (40, 900)):  # everything is visible
        o2, lse2 = fa.attention_forward(q, k, v, causal=True, window=window, sinks=sinks)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o, lse = fa.attention_forward(q, k, v, causal=True, window=200)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    fa.fa_fwd_window(q, k, v, o2, lse2, d ** -0.5, 200, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ref = fa.attention_backward(q, k, v, o, do, lse, causal=True, window=200)
    got = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(fa.fa_bwd_workspace_size(2, 4, 900, d), dtype=torch.uint8, device="cuda")
    fa.fa_bwd_window(q, k, v, o, do, lse, *got, ws, d ** -0.5, 200, 0)
    assert torch.equal(ref[2], got[2])  # (dK: the masked kernel's dS takes the rounded probabilities)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_tiles_are_not_read(fa, d):
    q, k, v, do = make(1, 2, 1, 1000, d, "bf16", 6)
    o, lse = fa.attention_forward(q, k, v, causal=True, window=100, sinks=4)
    for t, x in ((k, math.nan), (v, math.inf), (v, math.nan)):
        t2 = t.clone()
        t2[:, :, 200:300] = x
        o2, lse2 = fa.attention_forward(q, t2 if t is k else k, t2 if t is v else v, causal=True, window=100, sinks=4)
        for rows in (slice(0, 128), slice(512, 1000)):
            assert torch.equal(o[:, :, rows], o2[:, :, rows]) and torch.equal(lse[:, :, rows], lse2[:, :, rows])


def test_gradients_against_differences(fa):
    """Along one direction, by the forward's own O in 64 bits: the definition's gradient and the kernel's agree with differences
    of the definition (h^2 of the third derivative, below 1e-6 here; the kernel's part is bounded above)."""
    q, k, v, do = make(1, 2, 1, 200, 64, "fp16", 7)
    window, sinks, scale = 30, 3, 0.125
    f = lambda k_: float((reference(q[0], k_, v[0, 0], window, sinks, scale)["o"][0] * do[0].double()).sum())  # noqa: E731
    ref = reference(q[0], k[0, 0], v[0, 0], window, sinks, scale, do[0])
    o, lse = fa.attention_forward(q, k, v, causal=True, scale=scale, window=window, sinks=sinks)
    dk = fa.attention_backward(q, k, v, o, do, lse, causal=True, scale=scale, window=window, sinks=sinks)[1]
    e = torch.zeros(200, 64, dtype=torch.float64, device="cuda")
    e[1], e[77] = 1.0, -0.5
    h = 1e-4
    diff = (f(k[0, 0].double() + h * e) - f(k[0, 0].double() - h * e)) / (2 * h)
    assert abs(diff - float((ref["dk"][0] * e).sum())) < 1e-5
    assert abs(diff - float((dk[0, 0].double() * e).sum())) <= float((ref["dk"][1] * e.abs()).sum()) + 1e-5


# ------------------------------------------------------------------------------------------------ packed prompts


def packed(T, H, Hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(TORCH[dtype]).cuda()
    return qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]


def cu_of(lens, first=0):
    return torch.tensor(np.concatenate(([first], first + np.cumsum(lens))), dtype=torch.int32, device="cuda")


def check_packed(q, k, v, o, lse, lens, first, window, sinks):
    G, at = q.shape[1] // k.shape[1], first
    for n in lens:
        for h in range(k.shape[1] if n else 0):
            rows, heads = slice(at, at + n), slice(h * G, (h + 1) * G)
            ref = reference(q[rows, heads].transpose(0, 1), k[rows, h], v[rows, h], window, sinks, q.shape[2] ** -0.5)
            close(o[rows, heads].transpose(0, 1), ref["o"])
            close(lse[heads, rows], ref["lse"])
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (128, 129), (300, 0), (5000, 7)])
def test_packed_prompts(fa, dtype, d, window, sinks):
    lens, first, behind = [1, 0, 127, 128, 129, 700, 257, 2, 500], 40, 60
    T = first + sum(lens) + behind
    q, k, v = packed(T, 4, 2, d, dtype, 3)
    o, lse = torch.full((T, 4, d), 7.0, dtype=TORCH[dtype], device="cuda"), torch.full((4, T), 9.0, device="cuda")
    fa.fa_fwd_varlen_window(q, k, v, o, lse, cu_of(lens, first), d ** -0.5, window, sinks)
    fa.fa_check_device_error()
    check_packed(q, k, v, o, lse, lens, first, window, sinks)
    end = first + sum(lens)
    assert (o[:first] == 7).all() and (o[end:] == 7).all() and (lse[:, :first] == 9).all() and (lse[:, end:] == 9).all()


def test_packed_prompts_of_many_waves_and_sequences_apart(fa):
    lens = [3000, 1, 777, 2050, 130, 64]
    q, k, v = (t.clone() for t in packed(sum(lens), 8, 2, 128, "bf16", 4))
    o, lse = fa.attention_forward_varlen(q, k, v, cu_of(lens), causal=True, window=512, sinks=4)
    check_packed(q, k, v, o, lse, lens, 0, 512, 4)
    bad = slice(3001, 3778)
    q[bad], k[bad], v[bad] = math.nan, math.inf, math.nan
    o2, lse2 = fa.attention_forward_varlen(q, k, v, cu_of(lens), causal=True, window=512, sinks=4)
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])


def test_captured_and_replayed_and_on_other_streams(fa):
    q, k, v, do = make(2, 8, 4, 2000, 128, "bf16", 8)
    kw = {"causal": True, "window": 300, "sinks": 6}
    o, lse = fa.attention_forward(q, k, v, **kw)
    grads = fa.attention_backward(q, k, v, o, do, lse, **kw)
    qp, kp, vp = packed(3000, 8, 4, 128, "bf16", 9)
    cu = cu_of([1000, 1500, 500])
    op, lp = fa.attention_forward_varlen(qp, kp, vp, cu, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = fa.attention_forward(q, k, v, **kw)
        grads2 = fa.attention_backward(q, k, v, o2, do, lse2, **kw)
        op2, lp2 = fa.attention_forward_varlen(qp, kp, vp, cu, **kw)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(op, op2) and torch.equal(lp, lp2)
        assert torch.equal(grads[1], grads2[1]) and torch.equal(grads[2], grads2[2])
        # (dQ's sums come in no fixed order, in 32 bits: a unit in the last place now and then)
        assert ((grads[0].double() - grads2[0].double()).abs() <= 2.0 ** -7 * grads[0].double().abs() + 1e-5).all()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [fa.attention_forward(q, k, v, **kw, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in outs)
    fa.fa_check_device_error()


def test_refusals(fa):
    q, k, v, do = make(1, 2, 1, 64, 64, "bf16", 1)
    with pytest.raises(ValueError, match="sinks go with"):
        fa.attention_forward(q, k, v, causal=False, window=10, sinks=2)
    with pytest.raises(ValueError, match="sinks go with"):
        fa.attention_forward(q, k, v, causal=True, sinks=2)
    with pytest.raises(fa.FAError, match="tensor-core kernels"):
        fa.attention_forward(q.float(), k.float(), v.float(), causal=True, window=10, sinks=2)
    empty = [t[:, :, :0].contiguous() for t in (q, k, v)]
    assert fa.attention_forward(*empty, causal=True, window=10, sinks=2)[0].shape == (1, 2, 0, 64)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N,window,sinks", [(700, 1, 0), (700, 2, 0), (701, 4, 1), (700, 20, 12), (257, 1, 31), (130, 1000, 3), (256, 100, 90),
                                            (1, 5, 0), (17, 3, 2)])
def test_few_keys_in_sight(fa, dtype, d, N, window, sinks):
    """dS = p (dP - D) where D does not come from the rounded O: dD = (2 ds) sum p |dP| + the error of dP."""
    B, H, Hkv = 2, 4, 2
    q, k, v, do = make(B, H, Hkv, N, d, dtype, N + window)
    scale, e, G = d ** -0.5, EPS[dtype], H // Hkv
    o, lse = fa.attention_forward(q, k, v, causal=True, window=window, sinks=sinks)
    grads = fa.attention_backward(q, k, v, o, do, lse, causal=True, window=window, sinks=sinks)
    fa.fa_check_device_error()
    for b in range(B):
        for h in range(Hkv):
            mine = slice(h * G, (h + 1) * G)
            q1, k1, v1, do1 = (x.double() for x in (q[b, mine], k[b, h], v[b, h], do[b, mine]))
            ds = (d / 16 + 8) * 2.0 ** -23 * scale * float(q1.norm(dim=-1).max() * k1.norm(dim=-1).max()) + 2.0 ** -20
            p = torch.softmax((q1 @ k1.T * scale).masked_fill(~visible(N, window, sinks), -math.inf), -1)
            dp = do1 @ v1.T
            g = p * (dp - (p * dp).sum(-1, keepdim=True))
            dp_tol = (d / 16 + 8) * 2.0 ** -23 * do1.norm(dim=-1, keepdim=True) * v1.norm(dim=-1).max()
            g_tol = (e + 2 * ds) * g.abs() + p * (2 * ds * (p * dp.abs()).sum(-1, keepdim=True) + 2 * dp_tol)
            dq, dk = scale * (g @ k1), scale * (g.transpose(-1, -2) @ q1).sum(0)
            close(grads[0][b, mine], (dq, e * dq.abs() + scale * (g_tol @ k1.abs()) + 2.0 ** -24))
            close(grads[1][b, h], (dk, e * dk.abs() + scale * (g_tol.transpose(-1, -2) @ q1.abs()).sum(0) + 2.0 ** -24))


def test_values_outside_a_small_window_do_not_reach_d(fa):
    """D sums visible keys alone: a hidden value that is not finite leaves the gradients of the 256-query blocks
    that do not see its tile of 128 keys, here all but the second.  (A query
    here meets two tiles at most, whose shares of dQ add up to the same bits in either order.)"""
    q, k, v, do = make(1, 2, 2, 600, 64, "bf16", 3)
    o, lse = fa.attention_forward(q, k, v, causal=True, window=8, sinks=0)
    want = fa.attention_backward(q, k, v, o, do, lse, causal=True, window=8, sinks=0)
    v2 = v.clone()
    v2[:, :, 300] = math.nan
    got = fa.attention_backward(q, k, v2, o, do, lse, causal=True, window=8, sinks=0)
    assert torch.equal(got[0][:, :, :256], want[0][:, :, :256]) and torch.equal(got[0][:, :, 512:], want[0][:, :, 512:])
    assert got[0][:, :, 300:308].isnan().all()


def test_sinks_given_as_0_are_a_window_alone(fa):
    q, k, v, do = make(1, 4, 2, 500, 64, "fp16", 5)
    o, lse = torch.empty_like(q), torch.empty(1, 4, 500, device="cuda")
    fa.fa_fwd_window(q, k, v, o, lse, 0.125, 70, 0)
    a = fa.attention_forward(q, k, v, causal=True, window=70, sinks=0)
    assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    assert all(torch.equal(x, y) for x, y in zip(fa.attention_forward(q, k, v, window=70, sinks=0), fa.attention_forward(q, k, v, window=70)))
