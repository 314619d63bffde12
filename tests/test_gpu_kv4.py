"""The 4-bit key/value cache on the GPU against the fp64 oracle: rows in and out bit for bit, decode over it
with its attention weights, eviction, and the four used together."""

import numpy as np
import pytest

from oracle import kv4 as KV

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step, relative


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def cu_of(rows):
    return i32(np.concatenate(([0], np.cumsum(rows))))


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def rows_of(t):
    return t.detach().float().cpu().numpy()


def same_bytes(a, b):
    return np.ascontiguousarray(a).tobytes() == np.ascontiguousarray(b).tobytes()


def random_rows(T, hkv, d, dtype, seed, special=True):
    """Rows as a model makes them, and (special) groups with the values that go wrong."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g) * torch.exp(torch.randn(T, hkv, 1, generator=g) * 2)
    if special and T >= 12:
        x[0] = 0.0
        x[1] = -0.0
        x[2] = 3.0
        x[3, 0, :64] = float("nan")
        x[4, 0, 7] = float("inf")
        x[5, 0, 63] = -32768.0
        x[6, 0, 1] = 40000.0
        x[7] = x[7] * 1e-7
        x[8] = x[8] * 1e-30
        x[9] = x[9] + 1000.0
        x[10, 0, :64] = torch.arange(64) / 4.0  # many exact halves
        x[11, 0, ::2] = 32768.0
    return x.to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_and_read_bits(fa, dtype, d):
    hkv, rows, before, cap = 3, [13, 0, 1, 70], [0, 5, 63, 60], 192
    T = sum(rows)
    kv = torch.cat([random_rows(T, hkv, d, dtype, 1), random_rows(T, hkv, d, dtype, 2)], 1).cuda()
    k, v = kv[:, :hkv], kv[:, hkv:]  # slices of one projection: token stride 2 hkv d
    lens = i32(np.add(rows, before))
    cache = torch.full((len(rows), hkv, cap // 64, 72 * d), 0xA5, dtype=torch.uint8, device="cuda")
    weights = torch.full((len(rows), hkv, cap), 7.0, device="cuda")
    fa.fa_kv4_append(k, v, cu_of(rows), lens, cache, weights)
    fa.fa_check_device_error()
    want = np.full(cache.shape, 0xA5, np.uint8)
    (kc, ks, km), (vc, vs, vm) = KV.unpack_blocks(want)
    w_want = np.full((len(rows), hkv, cap), 7.0)
    at = 0
    val = []
    for x, (c, s, m) in ((k, (kc, ks, km)), (v, (vc, vs, vm))):
        qc, qs, qm = KV.quantize_rows(rows_of(x))
        val.append(KV.dequantize_rows(qc, qs, qm))
        at = 0
        for b, n in enumerate(rows):
            sl = slice(before[b], before[b] + n)
            c[b, :, sl] = qc[at:at + n].swapaxes(0, 1)
            s[b, :, sl], m[b, :, sl] = qs[at:at + n].swapaxes(0, 1), qm[at:at + n].swapaxes(0, 1)
            w_want[b, :, sl] = 0
            at += n
    got = KV.unpack_blocks(cache.cpu().numpy())
    for (c, s, m), (gc, gs, gm) in zip(((kc, ks, km), (vc, vs, vm)), got):
        assert np.array_equal(c, gc)
        for a, b in ((s, gs), (m, gm)):  # bit for bit; a NaN is a NaN
            same = a.view(np.uint16) == b.view(np.uint16)
            assert (same | (np.isnan(a) & np.isnan(b))).all()
    assert np.array_equal(w_want, f64(weights))
    for out in ("bf16", "fp16", "fp32"):
        rk, rv = fa.kv4_read(cache, cu_of(rows), lens, T, dtype=TORCH[out])
        for x, y in zip(val, (rk, rv)):
            want_t = torch.from_numpy(x.astype(np.float32)).to(TORCH[out])
            assert torch.equal(torch.nan_to_num(want_t, nan=123.0), torch.nan_to_num(y.cpu(), nan=123.0))


def test_rows_outside_the_lists_and_the_cache(fa):
    d, hkv, cap = 64, 2, 64
    k = random_rows(20, hkv, d, "bf16", 3, special=False).cuda()
    cache = fa.kv4_cache(2, hkv, cap, d)
    # rows 0-2 and 15-19 belong to no sequence
    cu, lens = i32([3, 9, 15]), i32([6, 64])
    fa.fa_kv4_append(k, k, cu, lens, cache)
    fa.fa_check_device_error()
    back = torch.full_like(k, 9.0)
    fa.fa_kv4_read(cache, cu, lens, back, back.clone())
    assert (back[:3] == 9).all() and (back[15:] == 9).all() and not (back[3:15] == 9).all()
    # six rows end at slot 4: two of them would lie before the cache; six at slot 70: behind it
    for bad in (i32([4, 64]), i32([6, 70]), i32([-5, 64])):
        untouched = cache.clone()
        fa.fa_kv4_append(k, k, cu, bad, cache)
        with pytest.raises(fa.FAError, match="device check"):
            fa.fa_check_device_error()
        fa.fa_check_device_error()  # cleared
        cache.copy_(untouched)


def test_refusals(fa):
    d = 128
    cache, lens = fa.kv4_cache(2, 2, 128, d), i32([1, 2])
    q = torch.zeros(2, 4, 1, d, dtype=torch.bfloat16, device="cuda")
    L = torch.zeros(2, 4, 1, device="cuda")
    ws = torch.empty(fa.fa_decode_kv4_workspace_size(2, 4, 2, 1, 128, d), dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, 2, 128, device="cuda")
    with pytest.raises(fa.FAError, match="workspace"):
        fa.fa_decode_kv4(q, cache, lens, q.clone(), L, 0.1, workspace=ws[:-16])
    with pytest.raises(fa.FAError, match="weights_in without"):
        fa.fa_decode_kv4(q, cache, lens, q.clone(), L, 0.1, weights_in=w, workspace=ws)
    with pytest.raises(fa.FAError, match="scale"):
        fa.fa_decode_kv4(q, cache, lens, q.clone(), L, -1.0, workspace=ws)
    with pytest.raises(fa.FAError, match="bf16 or fp16"):
        fa.fa_decode_kv4(q.float(), cache, lens, q.float(), L, 0.1, workspace=ws)
    with pytest.raises(fa.FAError, match="multiple of Hkv"):
        fa.attention_decode_kv4(torch.zeros(2, 3, 1, d, dtype=torch.bfloat16, device="cuda"), cache, lens)
    out, kept, n2 = fa.kv4_cache(2, 2, 64, d), torch.zeros(2, 2, 32, dtype=torch.int32, device="cuda"), i32([0, 0])
    w2 = torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(fa.FAError, match="keep"):
        fa.fa_kv4_evict(cache, w, lens, 65, 0, out, w2, n2, torch.zeros(2, 2, 65, dtype=torch.int32, device="cuda"))
    with pytest.raises(fa.FAError, match="recent"):
        fa.fa_kv4_evict(cache, w, lens, 32, 33, out, w2, n2, kept)
    with pytest.raises(fa.FAError, match="another cache"):
        fa.fa_kv4_evict(cache, w, lens, 32, 3, cache, w, n2, kept)
    k = torch.zeros(3, 1, d, dtype=torch.bfloat16, device="cuda").expand(3, 2, d)
    fa.fa_kv4_append(k, k, i32([0, 1, 3]), lens, cache)  # one head for all: fine to read, not to write
    with pytest.raises(fa.FAError, match="output stride"):
        fa.fa_kv4_read(cache, i32([0, 1, 3]), lens, k, k)
    with pytest.raises(fa.FAError, match="16 bytes"):
        odd = torch.zeros(3, 2, 132, dtype=torch.bfloat16, device="cuda")[..., :128]
        fa.fa_kv4_append(odd, odd, i32([0, 1, 3]), lens, cache)


def make_cache(B, hkv, cap, d, seed, garbage=None, lens=None):
    """A cache tensor and the fp64 keys and values that it holds; with `garbage`, slots behind lens hold
    bytes of that value (0xFF: NaN parameters)."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, hkv, cap, d), dtype=np.float32) + 2 * rng.standard_normal(d).astype(np.float32)
    v = rng.standard_normal((B, hkv, cap, d), dtype=np.float32)
    qk, qv = KV.quantize_rows(k), KV.quantize_rows(v)
    blocks = KV.pack_blocks(qk, qv)
    if garbage is not None:
        parts = KV.unpack_blocks(blocks)
        for c, s, m in parts:
            for b, n in enumerate(lens):
                c[b, :, n:] = garbage & 15
                s[b, :, n:], m[b, :, n:] = np.nan, np.inf
        blocks = KV.pack_blocks(*parts)
    return torch.from_numpy(blocks).cuda(), KV.dequantize_rows(*qk), KV.dequantize_rows(*qv)


def check_decode(fa, B, H, hkv, nq, lens, d, dtype, causal, cap, seed, weights=False, sharp=1.0):
    cache, k, v = make_cache(B, hkv, cap, d, seed, 0xFF, lens)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, H, nq, d, generator=g) * sharp).to(TORCH[dtype])
    scale = d ** -0.5
    args = {}
    if weights:
        w_in = torch.rand(B, hkv, cap, generator=g).cuda()
        w_out = torch.full((B, hkv, cap), -3.0, device="cuda")
        args = dict(weights_in=w_in, weights_out=w_out)
    o, lse = fa.attention_decode_kv4(q.cuda(), cache, i32(lens), causal=causal, scale=scale, **args)
    fa.fa_check_device_error()
    ro, rl, rw, mag = KV.decode64(f64(q), k, v, lens, scale, causal)
    go, gl = f64(o), f64(lse)
    # scores: fp32 sums of products; every one of the d / 16 matrix steps and the group sums rounds (or
    # truncates) the running value, at most |q| . |k| (the codes' and the middles' parts apart: 4 times it), by 2^-23
    ds = (d / 16 + 8) * 4 * 2.0 ** -23 * mag + 2.0 ** -21
    seen = np.isfinite(rl)
    assert np.array_equal(seen, np.isfinite(gl)) and (gl[~seen] == -np.inf).all()
    # L: |dL| <= max |dS|; exponent argument and logarithm in fp32 (|x| < 2^8: 2^-15 would be far off)
    tol_l = ds + 2.0 ** -21 * (8 + np.abs(np.where(seen, rl, 0)))
    assert (np.abs(gl[seen] - rl[seen]) <= tol_l[seen]).all(), np.abs(gl[seen] - rl[seen]).max()
    # O: probabilities and values rounded to fp16 (2^-11 each), scores' error twice (numerator and
    # sum), the smallest probabilities' absolute rounding (2^-33 of the largest, per slot), O's own type
    vmax = max(np.abs(v[b, :, :n]).max() for b, n in enumerate(lens) if n)
    tol_o = vmax * (2 * 2.0 ** -11 + 2 * (ds + 2.0 ** -20) + max(lens) * 2.0 ** -33)[..., None] + EPS[dtype] * np.abs(ro)
    assert (np.abs(go - ro) <= tol_o).all(), np.abs(go - ro).max()
    assert (go[~seen] == 0).all()
    if weights:
        gw = f64(w_out)
        for b, n in enumerate(lens):
            want = f64(w_in)[b, :, :n] + rw[b, :, :n]
            rows = (H // hkv) * nq
            # each probability's relative error is that of its score plus that of L; the sum rounds per row
            tol = rw[b, :, :n] * (2 * ds[b].max() + 2.0 ** -18) + (rows + 1) * 2.0 ** -24 * want
            assert (np.abs(gw[b, :, :n] - want) <= tol + 1e-12).all()
            assert (gw[b, :, n:] == -3.0).all()
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_lengths(fa, dtype, d, weights):
    check_decode(fa, 8, 8, 2, 1, [0, 1, 63, 64, 65, 127, 500, 1000], d, dtype, False, 1024, 10 + d, weights)


@pytest.mark.parametrize("H,hkv,nq", [(1, 1, 1), (8, 8, 1), (7, 1, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (6, 2, 5),
                                      (8, 1, 4), (4, 2, 20)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_rows_and_groups(fa, H, hkv, nq, d):
    # 1 .. 40 rows on a key/value head: one and two groups of eight, several row groups
    check_decode(fa, 3, H, hkv, nq, [3, 130, 321], d, "bf16", True, 384, 40 + H + nq, weights=True)
    check_decode(fa, 3, H, hkv, nq, [3, 130, 321], d, "fp16", False, 384, 41 + H + nq)


def test_decode_many_short_and_one_long(fa):
    lens = [1] * 40 + [3000] + [2, 0, 70] * 10
    check_decode(fa, len(lens), 2, 1, 1, lens, 128, "bf16", False, 3008, 50, weights=True)


def test_decode_one_head_over_every_cta(fa):
    check_decode(fa, 1, 4, 1, 1, [20001], 128, "bf16", False, 20032, 51, weights=True)
    check_decode(fa, 1, 4, 1, 2, [10000], 256, "fp16", True, 10048, 52)


def test_decode_sharp_scores(fa):
    # scores of some hundreds: one key takes nearly all the weight
    check_decode(fa, 2, 4, 2, 1, [700, 1500], 128, "bf16", False, 1536, 53, weights=True, sharp=8.0)


def test_decode_of_nan_rows(fa):
    d, cap = 64, 128
    cache, k, v = make_cache(2, 1, cap, d, 60)
    bad = torch.zeros(1, 1, d, dtype=torch.float32, device="cuda")
    bad[0, 0, 3] = float("nan")
    fa.fa_kv4_append(bad, bad, i32([0, 1, 1]), i32([11, 0]), cache)  # slot 10 of sequence 0
    q = torch.randn(2, 2, 1, d, dtype=torch.float16, device="cuda")
    o, lse = fa.attention_decode_kv4(q, cache, i32([20, 20]))
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()  # its row sees the NaN
    assert torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()
    o, lse = fa.attention_decode_kv4(q, cache, i32([10, 20]))  # behind the sequence: not seen
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_nan_in_a_slot_that_a_row_does_not_see(fa, d, dtype):
    # causal, four new rows: a NaN in the third newest slot reaches the two rows behind it and itself only
    cap, n, nq = 128, 90, 4
    for weights in (False, True):
        cache, _, held_v = make_cache(2, 1, cap, d, 62)
        cache_max = np.abs(held_v).max()
        g = torch.Generator().manual_seed(63)
        q = torch.randn(2, 4, nq, d, generator=g).to(TORCH[dtype]).cuda()
        args = dict(weights_out=torch.zeros(2, 1, cap, device="cuda")) if weights else {}
        ref, ref_l = fa.attention_decode_kv4(q, cache, i32([n, n]), causal=True, **args)
        # a row that does not see it: both results are within O's tolerance of the formula (check_decode; the
        # scores' part, 2 (d / 16 + 9) 2^-21 |q| . |k| scale for |q| . |k| scale < 64, is below 2^-9)
        tol = 2 * (cache_max * (2 * 2.0 ** -11 + 2.0 ** -9) + EPS[dtype] * ref[0, :, 0].abs().max().item())
        for bad_k in (False, True):
            k = torch.randn(1, 1, d, generator=g).cuda()
            v = k.clone()
            (k if bad_k else v)[0, 0, 5] = float("nan")
            c = cache.clone()
            fa.fa_kv4_append(k, v, i32([0, 1, 1]), i32([n - 2, 0]), c)  # slot n - 3 of sequence 0
            o, lse = fa.attention_decode_kv4(q, c, i32([n, n]), causal=True, **args)
            assert torch.equal(o[1], ref[1]) and torch.equal(lse[1], ref_l[1])
            assert ((o[0, :, 0].float() - ref[0, :, 0].float()).abs() <= tol).all()  # (false for NaN)
            assert ((lse[0, :, 0] - ref_l[0, :, 0]).abs() <= 2.0 ** -9).all()
            assert torch.isnan(o[0, :, 1:, :64]).all()  # the group of 64 channels that holds it
            assert torch.isnan(lse[0, :, 1:]).all() == bad_k


def test_decode_length_outside_the_cache(fa):
    d, cap = 64, 128
    cache, _, _ = make_cache(3, 1, cap, d, 61)
    q = torch.randn(3, 2, 1, d, dtype=torch.float16, device="cuda")
    o, lse = fa.attention_decode_kv4(q, cache, i32([500, -4, 128]))
    with pytest.raises(fa.FAError, match="device check"):
        fa.fa_check_device_error()
    ref, ref_l = fa.attention_decode_kv4(q, cache, i32([128, 0, 128]))
    fa.fa_check_device_error()
    assert torch.equal(o, ref) and torch.equal(lse, ref_l)


def test_decode_repeats_bit_for_bit_and_in_graphs(fa):
    B, H, hkv, d, cap = 3, 8, 2, 128, 2048
    cache, _, _ = make_cache(B, hkv, cap, d, 62)
    q = torch.randn(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
    lens = i32([2000, 7, 900])
    w = torch.zeros(B, hkv, cap, device="cuda")
    ref, ref_l = fa.attention_decode_kv4(q, cache, lens, weights_out=w)
    o, lse, w2 = torch.empty_like(ref), torch.empty_like(ref_l), torch.zeros_like(w)
    ws = torch.empty(fa.fa_decode_kv4_workspace_size(B, H, hkv, 1, cap, d, True), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        fa.fa_decode_kv4(q, cache, lens, o, lse, d ** -0.5, weights_out=w2, workspace=ws)
        assert torch.equal(o, ref) and torch.equal(lse, ref_l) and torch.equal(w2, w)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        fa.fa_decode_kv4(q, cache, lens, o, lse, d ** -0.5, weights_out=w2, workspace=ws)
    o.zero_()
    graph.replay()
    assert torch.equal(o, ref)
    lens.copy_(i32([1, 2048, 0]))  # the graph reads the lengths
    graph.replay()
    ref, ref_l = fa.attention_decode_kv4(q, cache, lens)
    assert torch.equal(o, ref) and torch.equal(lse, ref_l)
    # accumulated in place: twice the weights
    lens.copy_(i32([2000, 7, 900]))
    acc = torch.zeros_like(w)
    for _ in range(2):
        fa.fa_decode_kv4(q, cache, lens, o, lse, d ** -0.5, weights_in=acc, weights_out=acc, workspace=ws)
    assert torch.equal(acc, w + w)


def test_decode_on_two_streams(fa):
    B, H, hkv, d, cap = 2, 8, 2, 128, 4096
    cache, _, _ = make_cache(B, hkv, cap, d, 63)
    q = torch.randn(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
    a, b = i32([4000, 3]), i32([77, 4096])
    refs = [fa.attention_decode_kv4(q, cache, n) for n in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for i, n in enumerate((a, b)):
            outs[i].append(fa.attention_decode_kv4(q, cache, n, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in outs[i]:
            assert torch.equal(o, refs[i][0]) and torch.equal(lse, refs[i][1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (64, 0), (100, 100), (130, 17), (500, 64)])
def test_evict(fa, d, keep, recent):
    B, hkv, cap, out_cap = 5, 2, 1088, 576
    lens = [0, 1, keep, 700, 1088]
    lens[2] = min(keep, cap)
    cache, _, _ = make_cache(B, hkv, cap, d, 70)
    g = torch.Generator().manual_seed(keep)
    w = torch.round(torch.exp(torch.randn(B, hkv, cap, generator=g)) * 4) / 4  # many ties
    w[3, 0, 5], w[3, 0, 9], w[3, 0, 11] = float("nan"), float("inf"), -1.0
    w[4, 1] = 0.0
    w[4, 1, ::3] = -0.0
    out = torch.full((B, hkv, out_cap // 64, 72 * d), 0x5A, dtype=torch.uint8, device="cuda")
    w2 = torch.full((B, hkv, out_cap), -7.0, device="cuda")
    n2 = i32([9] * B)
    kept = torch.full((B, hkv, keep), 99, dtype=torch.int32, device="cuda")
    fa.fa_kv4_evict(cache, w.cuda(), i32(lens), keep, recent, out, w2, n2, kept)
    fa.fa_check_device_error()
    assert n2.tolist() == [min(n, keep) for n in lens]
    src = KV.unpack_blocks(cache.cpu().numpy())
    dst = KV.unpack_blocks(out.cpu().numpy())
    fill = KV.unpack_blocks(np.full(out.shape, 0x5A, np.uint8))
    for b in range(B):
        for h in range(hkv):
            want = KV.evict(w[b, h].numpy(), lens[b], keep, recent)
            n = len(want)
            assert kept[b, h].tolist() == want.tolist() + [-1] * (keep - n)
            assert np.array_equal(w2[b, h, :n].cpu().numpy(), w[b, h].numpy()[want], equal_nan=True)
            assert (w2[b, h, n:] == -7).all()
            for s, t, f in zip(src, dst, fill):
                for x, y, z in zip(s, t, f):
                    assert same_bytes(x[b, h][want], y[b, h][:n])
                    assert same_bytes(z[b, h][n:], y[b, h][n:])


@pytest.mark.parametrize("B,hkv,cap,keep", [(40, 2, 20032, 3000), (1, 1, 140032, 20000)])
def test_evict_more_slots_than_a_block_holds(fa, B, hkv, cap, keep):
    d, recent = 64, 100
    cache = torch.randint(0, 256, (B, hkv, cap // 64, 72 * d), dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 5000, (B, hkv, cap), device="cuda").float()  # ties
    lens = [cap - 7 * b for b in range(B)]
    out, w2 = fa.kv4_cache(B, hkv, keep, d), torch.zeros(B, hkv, (keep + 63) // 64 * 64, device="cuda")
    kept = torch.zeros(B, hkv, keep, dtype=torch.int32, device="cuda")
    n2 = i32([0] * B)
    fa.fa_kv4_evict(cache, w, i32(lens), keep, recent, out, w2, n2, kept)
    fa.fa_check_device_error()
    for b in range(0, B, 13):
        for h in range(hkv):
            want = KV.evict(w[b, h].cpu().numpy(), lens[b], keep, recent)
            assert kept[b, h].tolist() == want.tolist()
            assert np.array_equal(w2[b, h, :keep].cpu().numpy(), w[b, h].cpu().numpy()[want])


def test_evict_long_and_in_place_lengths(fa):
    B, hkv, cap, d, keep, recent = 1, 2, 40000 // 64 * 64, 64, 5000, 300
    cache = torch.randint(0, 256, (B, hkv, cap // 64, 72 * d), dtype=torch.uint8, device="cuda")
    w = torch.rand(B, hkv, cap, device="cuda")
    lens = i32([cap - 3])
    out, w2 = fa.kv4_cache(B, hkv, keep, d), torch.zeros(B, hkv, (keep + 63) // 64 * 64, device="cuda")
    kept = torch.zeros(B, hkv, keep, dtype=torch.int32, device="cuda")
    fa.fa_kv4_evict(cache, w, lens, keep, recent, out, w2, lens, kept)
    assert lens.tolist() == [keep]
    for h in range(hkv):
        assert kept[0, h].tolist() == KV.evict(w[0, h].cpu().numpy(), cap - 3, keep, recent).tolist()
