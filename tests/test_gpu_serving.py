"""The serving operators together, as a generation loop uses them: packed prompts through the forward, their
keys and values into the 4-bit cache, tokens decoded one by one with their attention weights added up, the
cache thinned out by those weights, and decoding over what is left."""

import numpy as np
import pytest

import oracle
from oracle import kv4 as KV
from oracle.gqa import expand_kv

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


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Mirror:
    """What the cache holds, per sequence and key/value head, in fp64."""

    def __init__(self, B, hkv, d):
        self.k = [[np.zeros((0, d)) for _ in range(hkv)] for _ in range(B)]
        self.v = [[np.zeros((0, d)) for _ in range(hkv)] for _ in range(B)]
        self.w = [[np.zeros(0) for _ in range(hkv)] for _ in range(B)]

    def append(self, b, k, v):  # [n, hkv, d]
        for h in range(k.shape[1]):
            for store, x in ((self.k, k), (self.v, v)):
                store[b][h] = np.concatenate((store[b][h], KV.dequantize_rows(*KV.quantize_rows(x[:, h]))))
            self.w[b][h] = np.concatenate((self.w[b][h], np.zeros(len(k))))

    def decode(self, b, q, scale):  # q [H, d]; O [H, d], L [H]; weights added
        H, hkv = q.shape[0], len(self.k[b])
        o, L = np.zeros(q.shape), np.zeros(H)
        for i in range(H):
            h = i * hkv // H
            s = scale * (self.k[b][h] @ q[i])
            m = s.max()
            p = np.exp(s - m)
            L[i] = m + np.log(p.sum())
            p /= p.sum()
            o[i] = p @ self.v[b][h]
            self.w[b][h] += p
        return o, L


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_prompt_cache_decode_evict(fa, dtype, d):
    B, H, hkv, cap, keep, recent = 4, 8, 2, 320, 96, 32
    prompts = [70, 1, 200, 129]
    T, scale = sum(prompts), d ** -0.5
    g = torch.Generator().manual_seed(5)

    def tokens(n):
        qkv = torch.randn(n, H + 2 * hkv, d, generator=g).to(TORCH[dtype]).cuda()
        return qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]

    q, k, v = tokens(T)
    cu, lens = i32(np.concatenate(([0], np.cumsum(prompts)))), i32(prompts)
    cache, weights = fa.kv4_cache(B, hkv, cap, d), torch.full((B, hkv, cap), 5.0, device="cuda")
    o, lse = fa.attention_forward_varlen(q, k, v, cu, causal=True)
    fa.fa_kv4_append(k, v, cu, lens, cache, weights)
    mirror, at = Mirror(B, hkv, d), 0
    for b, n in enumerate(prompts):
        x = [f64(t[at:at + n]).swapaxes(0, 1)[None] for t in (q, k, v)]
        ro, rl = oracle.attn_fwd64(x[0], expand_kv(x[1], H), expand_kv(x[2], H), scale, True)
        vmax = np.abs(x[2]).max()
        assert np.abs(f64(o[at:at + n]).swapaxes(0, 1) - ro[0]).max() <= EPS[dtype] * 2 * vmax + 1e-4
        assert np.abs(f64(lse[:, at:at + n]) - rl[0]).max() <= 1e-4
        mirror.append(b, f64(k[at:at + n]).astype(np.float32), f64(v[at:at + n]).astype(np.float32))
        at += n

    steps = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for step in range(8):
        q, k, v = tokens(B)
        lens += 1
        fa.fa_kv4_append(k, v, steps, lens, cache, weights)
        o, lse = fa.attention_decode_kv4(q.contiguous().view(B, H, 1, d), cache, lens, causal=True, scale=scale,
                                         weights_in=weights, weights_out=weights)
        fa.fa_check_device_error()
        for b in range(B):
            mirror.append(b, f64(k[b:b + 1]).astype(np.float32), f64(v[b:b + 1]).astype(np.float32))
            ro, rl = mirror.decode(b, f64(q[b]), scale)
            vmax = max(np.abs(x).max() for x in mirror.v[b])
            assert np.abs(f64(lse[b, :, 0]) - rl).max() <= 1e-4
            # P and its product with the step in fp16 (2^-11), O in its own type
            assert np.abs(f64(o[b, :, 0]) - ro).max() <= vmax * (2.0 ** -11 + EPS[dtype] + 1e-4)
            n = int(lens[b])
            for h in range(hkv):
                # every step adds at most 1e-4 relative (scores, log-sum-exp) to what it adds
                got = f64(weights[b, h, :n])
                assert np.abs(got - mirror.w[b][h]).max() <= 1e-4 * (step + 1)
                mirror.w[b][h] = got  # the kernel's own, so that near ties are decided alike below
        if step == 4:
            out, w2 = fa.kv4_cache(B, hkv, 128, d), torch.zeros(B, hkv, 128, device="cuda")
            kept = torch.zeros(B, hkv, keep, dtype=torch.int32, device="cuda")
            n2 = torch.empty_like(lens)
            fa.fa_kv4_evict(cache, weights, lens, keep, recent, out, w2, n2, kept)
            fa.fa_check_device_error()
            assert n2.tolist() == [min(int(n), keep) for n in lens]
            for b in range(B):
                for h in range(hkv):
                    src = KV.evict(mirror.w[b][h].astype(np.float32), int(lens[b]), keep, recent)
                    assert kept[b, h, :len(src)].tolist() == src.tolist()
                    mirror.k[b][h], mirror.v[b][h] = mirror.k[b][h][src], mirror.v[b][h][src]
                    mirror.w[b][h] = mirror.w[b][h][src]
            cache, weights, lens = out, w2, n2
    # what is read back is what the mirror holds
    total = int(lens.sum())
    rk, rv = fa.kv4_read(cache, i32(np.concatenate(([0], np.cumsum(lens.tolist())))), lens, total, dtype=torch.float32)
    at = 0
    for b in range(B):
        n = int(lens[b])
        for h in range(hkv):
            assert np.abs(f64(rk[at:at + n, h]) - mirror.k[b][h]).max() <= 2.0 ** -22 * np.abs(mirror.k[b][h]).max()
            assert np.abs(f64(rv[at:at + n, h]) - mirror.v[b][h]).max() <= 2.0 ** -22 * np.abs(mirror.v[b][h]).max()
        at += n


def test_a_captured_step_serves_a_growing_cache(fa):
    """One graph of append + decode + the lengths' count, replayed while the cache grows past block borders."""
    B, H, hkv, d, cap = 2, 4, 2, 64, 256
    g = torch.Generator().manual_seed(6)
    cache, w = fa.kv4_cache(B, hkv, cap, d), torch.zeros(B, hkv, cap, device="cuda")
    lens, steps = i32([60, 0]), torch.arange(B + 1, dtype=torch.int32, device="cuda")
    first = torch.randn(60, hkv, d, generator=g).to(torch.bfloat16).cuda()
    fa.fa_kv4_append(first, first, i32([0, 60, 60]), lens, cache)
    q = torch.zeros(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros(B, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, hkv, d, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
    ws = torch.empty(fa.fa_decode_kv4_workspace_size(B, H, hkv, 1, cap, d, True), dtype=torch.uint8, device="cuda")
    twin_cache, twin_w, twin_lens = cache.clone(), w.clone(), lens.clone()

    def step(cache, w, lens, o, lse):
        lens.add_(1)
        fa.fa_kv4_append(k, v, steps, lens, cache, w)
        fa.fa_decode_kv4(q, cache, lens, o, lse, d ** -0.5, True, w, w, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, w, lens, o, lse)
    for _ in range(10):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        graph.replay()
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        step(twin_cache, twin_w, twin_lens, o2, lse2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fa.fa_check_device_error()
    assert lens.tolist() == [70, 10] and torch.equal(cache, twin_cache) and torch.equal(w, twin_w)
