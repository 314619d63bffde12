"""The operators around attention as a model uses them together: a training step (norms and rotation, attention with a window and
sinks, all gradients) and a generation loop (packed prompts, then one token at a time), each against the definition in 64 bits.

Tolerances (e: half a step of the type, relative): what each operator rounds is an input of the next one, so a result's error is that of
the last operator on the rounded inputs that it really got, which the tests read back, and not of the whole chain.
"""

import math

import numpy as np
import pytest

from oracle.norm_rope import norm_rope64, norm_rope64_backward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def attend(q, k, v, see, scale):
    """One head in 64 bits: q [n, d] over k, v [m, d] where see [n, m]; (O, sum p |v|)."""
    s = (q.double() @ k.double().T * scale).masked_fill(~see, -math.inf)
    p = torch.softmax(s, -1)
    return p @ v.double(), p @ v.double().abs()


def band(n, window, sinks):
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")
    return (j <= i) & ((i - j < window) | (j < sinks))


def test_training_step(fa):
    B, N, H, Hkv, d, window, sinks, e = 2, 300, 4, 2, 64, 100, 4, 2.0 ** -11
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, N, H + 2 * Hkv, d, generator=g).half().cuda()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:].transpose(1, 2).contiguous()
    wq, wk = (torch.rand(d, generator=g).cuda() + 0.5 for _ in range(2))
    table = fa.rope_table(N, d)
    kw = {"causal": True, "window": window, "sinks": sinks}
    qr, kr = fa.qk_norm_rope(q, k, wq, wk, table)
    o, lse = fa.attention_forward(qr, kr, v, **kw)
    do = torch.randn(o.shape, generator=g).half().cuda()
    dqr, dkr, dv = fa.attention_backward(qr, kr, v, o, do, lse, **kw)
    dqkv = torch.empty_like(qkv)
    dqkv[:, :, H + Hkv:] = dv.transpose(1, 2)
    _, _, dwq, dwk = fa.qk_norm_rope_backward(dqr, dkr, q, k, wq, wk, table, out=(dqkv[:, :, :H], dqkv[:, :, H:H + Hkv]))
    fa.fa_check_device_error()
    cos, sin = (np.tile(f64(t), (B, 1)) for t in table.split(d // 2, -1))
    rows = lambda t: f64(t).reshape(-1, *t.shape[-2:])  # noqa: E731
    for x, w, y, dy, dx, dw in ((q, wq, qr, dqr, dqkv[:, :, :H], dwq), (k, wk, kr, dkr, dqkv[:, :, H:H + Hkv], dwk)):
        ry = norm_rope64(rows(x), f64(w), cos, sin, 1e-6, False)
        assert (np.abs(rows(y.transpose(1, 2)) - ry) <= (e + 2.0 ** -18) * np.abs(ry) + 2.0 ** -18).all()
        rdx, rdw = norm_rope64_backward(rows(dy.transpose(1, 2)), rows(x), f64(w), cos, sin, 1e-6, False)
        assert (np.abs(rows(dx) - rdx) <= e * np.abs(rdx) + 2.0 ** -17 * np.abs(rdx).max()).all()
        assert (np.abs(f64(dw) - rdw) <= 2.0 ** -16 * np.abs(rdw).max()).all()
    see = band(N, window, sinks)
    for b in range(B):
        for h in range(H):
            ro, mag = attend(qr[b, h], kr[b, h // 2], v[b, h // 2], see, d ** -0.5)
            assert ((o[b, h].double() - ro).abs() <= e * (ro.abs() + mag) + 2.0 ** -14).all()
    # the whole chain's gradient of the projection along one direction, against differences of the chain in 64 bits

    def loss(x):
        xs = x.cpu().numpy()
        qq = norm_rope64(xs[:, :, :H].reshape(-1, H, d), f64(wq), cos, sin, 1e-6, False).reshape(B, N, H, d)
        kk = norm_rope64(xs[:, :, H:H + Hkv].reshape(-1, Hkv, d), f64(wk), cos, sin, 1e-6, False).reshape(B, N, Hkv, d)
        qq, kk, vv = (torch.from_numpy(t).cuda() for t in (qq, kk, np.ascontiguousarray(xs[:, :, H + Hkv:])))
        return sum(float((attend(qq[b, :, h], kk[b, :, h // 2], vv[b, :, h // 2], see, d ** -0.5)[0] * do[b, h].double()).sum())
                   for b in range(B) for h in range(H))

    step = torch.zeros_like(qkv, dtype=torch.float64)
    step[0, 3], step[1, 120] = 1.0, -0.5
    step[..., ::2] *= -1
    eps = 1e-4
    diff = (loss(qkv.double() + eps * step) - loss(qkv.double() - eps * step)) / (2 * eps)
    # three operators in a row round their gradients (e each, relative to the rows' magnitudes): 4 e of the sum of magnitudes
    assert abs(diff - float((dqkv.double() * step).sum())) <= 4 * e * float((dqkv.double() * step).abs().sum()) + 1e-3


def test_generation_loop(fa):
    H, Hkv, d, C, window, sinks, e = 8, 2, 128, 300, 64, 3, 2.0 ** -8
    prompts, steps = [70, 1, 200], 6
    B, T = len(prompts), sum(prompts)
    g = torch.Generator().manual_seed(2)
    weights = [(torch.rand(d, generator=g) + 0.5).bfloat16().cuda() for _ in range(2)]
    table = fa.rope_table(C, d)
    cache = [torch.full((B, Hkv, C, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(prompts))), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompts]).cuda()
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k = fa.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], *weights, table, pos)
    o, _ = fa.attention_forward_varlen(q, k, qkv[:, H + Hkv:], cu, causal=True, window=window, sinks=sinks)
    at = 0
    for b, n in enumerate(prompts):
        cache[0][b, :, :n], cache[1][b, :, :n] = k[at:at + n].transpose(0, 1), qkv[at:at + n, H + Hkv:].transpose(0, 1)
        for h in range(H):
            ro, mag = attend(q[at:at + n, h], k[at:at + n, h // 4], qkv[at:at + n, H + Hkv + h // 4], band(n, window, sinks), d ** -0.5)
            assert ((o[at:at + n, h].double() - ro).abs() <= e * (ro.abs() + mag) + 2.0 ** -12).all()
        at += n
    # one token of each sequence: a captured step, replayed
    x = torch.empty(B, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    each = torch.arange(B, device="cuda")

    def step():
        q1, k1 = fa.qk_norm_rope(x[:, :H], x[:, H:H + Hkv], *weights, table, lens)
        cache[0][each, :, lens.long()], cache[1][each, :, lens.long()] = k1, x[:, H + Hkv:]
        lens.add_(1)
        q1 = q1.unsqueeze(2)
        return q1, fa.attention_decode_window(q1, *cache, lens, window, sinks)[0]

    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (*cache, lens)]
    x.copy_(torch.randn(x.shape, generator=g))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q1, o1 = step()
    for t, s in zip((*cache, lens), saved):
        t.copy_(s)
    for i in range(steps):
        x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        for b, n in enumerate(prompts):
            n += i + 1
            see = band(n, window, sinks)[-1:]
            for h in range(H):
                ro, mag = attend(q1[b, h], cache[0][b, h // 4, :n], cache[1][b, h // 4, :n], see, d ** -0.5)
                assert ((o1[b, h].double() - ro).abs() <= e * (ro.abs() + mag) + 2.0 ** -12).all()
    assert lens.tolist() == [n + steps for n in prompts]
    fa.fa_check_device_error()


def test_shared_prefix_is_the_same_as_a_cache_that_holds_it(fa):
    """Decoding behind a shared prefix and over caches that begin with it: within both calls' own rounding."""
    B, H, Hkv, d, P, C, e = 5, 8, 2, 128, 200, 300, 2.0 ** -8
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, kp, vp, k, v = r(B, H, 1, d), r(Hkv, P, d), r(Hkv, P, d), r(B, Hkv, C, d), r(B, Hkv, C, d)
    lens = torch.tensor([1, 40, 77, 99, 0], dtype=torch.int32, device="cuda")
    o, lse = fa.attention_decode_prefix(q, kp, vp, k, v, lens)
    whole = [torch.cat((x.expand(B, Hkv, P, d), y), 2).contiguous() for x, y in ((kp, k), (vp, v))]
    o2, lse2 = fa.attention_decode_window(q, *whole, lens + P)
    # each rounds its weights and its result once: e (|O| + sum p |v|) of both, with sum p |v| below the largest |v| of 300 (4)
    assert ((o.double() - o2.double()).abs() <= 2 * e * (o.double().abs() + 4.0)).all()
    assert ((lse - lse2).abs() <= 1e-5 * (1 + lse.abs())).all()
