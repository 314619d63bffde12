"""Decode over 16-bit caches of different lengths, with a window and sinks or behind a shared prefix, vs its definition in 64 bits.

Tolerances (e = EPS, half a step of the 16-bit type, relative): scores are fp32 sums of d products, statistics and exponentials
fp32: ds = (d / 16 + 8) 2^-23 |q| |k| scale + 2^-20 of a score; the joining of segments adds a few fp32 roundings of O, l and m (2^-20).
O: e |O| + e sum p |v| + (2 ds + 2^-20) max |v|; L: ds + 2^-20 (8 + |L|).
"""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def make(lens, H, Hkv, Nq, d, dtype, C, P=None, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * d + H + C)
    B, dt = len(lens), TORCH[dtype]
    r = lambda *s: torch.randn(s, generator=g).to(dt).cuda()  # noqa: E731
    q, k, v = r(B, H, Nq, d), r(B, Hkv, C, d), r(B, Hkv, C, d)
    k[..., 3] *= 4.0  # rows of clearly different weight
    for b, n in enumerate(lens):  # what lies behind a sequence is not to be looked at
        k[b, :, max(0, n):] = math.nan
        v[b, :, max(0, n):] = math.nan
    prefix = (r(Hkv, P, d), r(Hkv, P, d)) if P is not None else None
    return q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), prefix


def check(q, k, v, lens, o, lse, scale, window=0, sinks=0, prefix=None):
    B, H, Nq, d = q.shape
    Hkv = k.shape[1]
    G, e = H // Hkv, EPS[q.dtype]
    assert o.isfinite().all()
    for b, n in enumerate(lens.tolist()):
        n = max(0, min(n, k.shape[2]))
        i = n - Nq + torch.arange(Nq, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        see = j <= i
        if window:
            see = see & ((i - j < window) | (j < sinks))
        for h in range(Hkv):
            ks, vs = k[b, h, :n].double(), v[b, h, :n].double()
            dark = ~see
            if prefix is not None:
                ks, vs = torch.cat((prefix[0][h].double(), ks)), torch.cat((prefix[1][h].double(), vs))
                dark = torch.cat((torch.zeros(Nq, prefix[0].shape[1], dtype=torch.bool, device="cuda"), dark), 1)
            mine = slice(h * G, (h + 1) * G)
            got, gl = o[b, mine].double(), lse[b, mine].double()
            if ks.shape[0] == 0:
                assert (got == 0).all() and (gl == -math.inf).all()
                continue
            qs = q[b, mine].double()
            s = (qs @ ks.T * scale).masked_fill(dark, -math.inf)
            rl = torch.logsumexp(s, -1)
            none = rl == -math.inf
            p = torch.exp(s - rl.masked_fill(none, 0.0)[..., None])
            ro = p @ vs
            ds = (d / 16 + 8) * 2.0 ** -23 * scale * float(qs.norm(dim=-1).max() * ks.norm(dim=-1).max()) + 2.0 ** -20
            tol = e * (ro.abs() + p @ vs.abs()) + (2 * ds + 2.0 ** -20) * vs.abs().max()
            assert ((got - ro).abs() <= tol).all(), float(((got - ro).abs() / tol).max())
            assert ((gl == -math.inf) == none).all()
            assert ((gl - rl).abs()[~none] <= (ds + 2.0 ** -20 * (8 + rl.abs()))[~none]).all()


def run(fa, lens, H, Hkv, Nq, d, dtype, C, window=0, sinks=0, P=None, seed=0):
    q, k, v, ln, prefix = make(lens, H, Hkv, Nq, d, dtype, C, P, seed)
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 9.0, device="cuda")
    B = len(lens)
    if prefix is None:
        ws = torch.full((fa.fa_decode_window_workspace_size(B, H, Hkv, Nq, C, d),), 255, dtype=torch.uint8, device="cuda")
        fa.fa_decode_window(q, k, v, ln, o, lse, d ** -0.5, window, sinks, ws)
    else:
        ws = torch.full((fa.fa_decode_prefix_workspace_size(B, H, Hkv, Nq, P, C, d),), 255, dtype=torch.uint8, device="cuda")
        fa.fa_decode_prefix(q, *prefix, k, v, ln, o, lse, d ** -0.5, ws)
    fa.fa_check_device_error()
    check(q, k, v, ln, o, lse, d ** -0.5, window, sinks, prefix)


def test_one_sequence_one_head(fa):
    for n in (1, 2, 15, 16, 17, 127, 128, 129, 300):
        run(fa, [n], 1, 1, 1, 128, "bf16", 300)
    run(fa, [0], 1, 1, 1, 64, "fp16", 1)
    run(fa, [1], 1, 1, 1, 64, "fp16", 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,C", [([5], 5), ([700, 0, 1, 64, 129], 700), ([3000, 2, 1999], 4001)])
def test_lengths(fa, dtype, d, lens, C):
    run(fa, lens, 8, 2, 1, d, dtype, C)


@pytest.mark.parametrize("H,Hkv,Nq", [(1, 1, 1), (8, 8, 2), (8, 2, 4), (7, 1, 5), (16, 1, 4), (12, 2, 7), (8, 1, 16), (24, 2, 8),
                                      (32, 1, 9)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_a_head(fa, H, Hkv, Nq, d):
    """One copy of the rows and several, and more than one tile of them; sequences shorter than their new rows."""
    run(fa, [260, 3, 1000, 0], H, Hkv, Nq, d, "bf16", 1000)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [1, 3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (100, 4), (128, 128), (129, 200), (300, 0), (1000, 7), (4000, 4)])
def test_windows_and_sinks(fa, d, Nq, window, sinks):
    run(fa, [1500, 1, 2, 128, 129, 130, 333, 0, 1024], 4, 2, Nq, d, "bf16", 1500, window, sinks)


def test_largest_window_and_sinks(fa):
    top = 2 ** 31 - 1
    for window, sinks in ((top, top), (top, 0), (5, top), (1, top)):
        run(fa, [300, 7], 4, 2, 2, 128, "fp16", 300, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("P", [0, 1, 127, 128, 1000])
def test_prefixes(fa, dtype, d, P):
    run(fa, [30, 0, 1, 200, 77], 8, 2, 1, d, dtype, 256, P=P)


@pytest.mark.parametrize("B,H,Hkv,Nq", [(1, 1, 1, 1), (3, 4, 4, 1), (9, 8, 1, 1), (17, 7, 1, 3), (40, 8, 2, 1), (65, 2, 1, 1), (33, 8, 2, 4)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_a_prefix(fa, B, H, Hkv, Nq, d):
    """From one row to several tiles of rows of all sequences."""
    run(fa, [(37 * i) % 150 for i in range(B)], H, Hkv, Nq, d, "bf16", 150, P=700)


def test_more_segments_than_blocks_and_long_runs(fa):
    run(fa, [10 + i % 50 for i in range(300)], 4, 4, 1, 64, "fp16", 64)
    run(fa, [20000, 100, 30000, 1], 8, 2, 1, 128, "bf16", 30000)
    run(fa, [9000, 8000], 16, 8, 1, 128, "fp16", 9001, window=6000, sinks=3)
    run(fa, [5000] * 8, 32, 4, 1, 128, "bf16", 5000, P=9000)


def test_agrees_with_decode_of_one_length(fa):
    q, k, v, lens, _ = make([512] * 3, 8, 2, 1, 128, "bf16", 512)
    o, lse = fa.attention_decode_window(q, k, v, lens)
    ro, rl = fa.attention_decode(q, k, v)
    # Each rounds its weights p to bf16 against a maximum of its own, so an element is off by e sum p |v| whatever its size: with
    # 512 keys of |v| around 0.8 that is up to 2^-8 0.8 = 2^-8.3, 2^-7.3 between the two, where elements are 2^-4.  So
    # not their difference relative to the element is bounded, but each one's distance from the definition, as above.
    check(q, k, v, lens, o, lse, 128 ** -0.5)
    check(q, k, v, lens, ro, rl, 128 ** -0.5)


def test_lengths_outside_the_cache_are_clamped_and_recorded(fa):
    q, k, v, _, prefix = make([64, 64, 64], 4, 2, 1, 64, "fp16", 64, P=100)
    for bad in ([65, -1, 64], [2 ** 31 - 1, -2 ** 31, 3]):
        lens = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda n: fa.attention_decode_window(q, k, v, n), lambda n: fa.attention_decode_window(q, k, v, n, 10, 3),
                     lambda n: fa.attention_decode_prefix(q, *prefix, k, v, n)):
            got = call(lens)
            with pytest.raises(fa.FAError, match="device check"):
                fa.fa_check_device_error()
            want = call(lens.clamp(0, 64))
            fa.fa_check_device_error()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_is_hidden_from_all_rows_is_not_looked_at(fa):
    q, k, v, lens, _ = make([1000, 700], 8, 2, 1, 128, "bf16", 1100)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate([1000, 700]):
        k2[b, :, 4:n - 200], v2[b, :, 4:n - 200] = math.nan, math.inf
    a, b = (fa.attention_decode_window(q, *x, lens, 200, 4) for x in ((k, v), (k2, v2)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0].isfinite().all()


def test_scores_far_apart_and_infinite_keys(fa):
    q, k, v, lens, _ = make([400, 300], 4, 2, 1, 64, "fp16", 400)
    k[0, 0, 200] = q[0, 0, 0] * 30  # one key takes all the weight late in the sequence
    o, lse = fa.attention_decode_window(q, k, v, lens)
    check(q, k, v, lens, o, lse, 0.125)
    k[1, 1, 17] = math.nan  # a row's own head only
    o2, _ = fa.attention_decode_window(q, k, v, lens)
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[1, :2], o[1, :2]) and o2[1, 2:].isnan().all()
    k[1, 1, :300] = math.nan
    assert fa.attention_decode_window(q, k, v, lens)[0][1, 2:].isnan().all()


def test_results_do_not_depend_on_the_run(fa):
    q, k, v, lens, prefix = make([3000, 17, 900], 8, 2, 2, 128, "bf16", 3000, P=5000)
    for call in (lambda: fa.attention_decode_window(q, k, v, lens, 2000, 4), lambda: fa.attention_decode_prefix(q, *prefix, k, v, lens)):
        a = call()
        for _ in range(5):
            b = call()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_graph_for_growing_lengths_and_two_streams(fa):
    q, k, v, lens, prefix = make([2000] * 3, 8, 2, 1, 128, "bf16", 2000, P=300)
    lens.copy_(torch.tensor([1, 500, 1990]))
    graph = torch.cuda.CUDAGraph()
    fa.attention_decode_window(q, k, v, lens, 700, 4)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = fa.attention_decode_window(q, k, v, lens, 700, 4)
        b = fa.attention_decode_prefix(q, *prefix, k, v, lens)
        lens += 1
    for step in range(4):
        graph.replay()
        seen = lens - 1
        check(q, k, v, seen, *a, 128 ** -0.5, 700, 4)
        check(q, k, v, seen, *b, 128 ** -0.5, prefix=prefix)
    want = fa.attention_decode_prefix(q, *prefix, k, v, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [fa.attention_decode_prefix(q, *prefix, k, v, lens, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in outs)
    fa.fa_check_device_error()


def test_tiles_that_are_met(fa):
    q, k, v, lens, prefix = make([10000, 200], 4, 2, 1, 128, "bf16", 10000, P=1000)
    fa.fa_tile_counter(reset=True)
    fa.attention_decode_window(q, k, v, lens, 1024, 4)
    assert fa.fa_tile_counter(reset=True) == 2 * (1 + 8) + 2 * 2  # sinks and window; the short one whole
    fa.attention_decode_prefix(q, *prefix, k, v, lens)
    assert fa.fa_tile_counter(reset=True) == 2 * 8 + 2 * 79 + 2 * 2


def test_refusals(fa):
    q, k, v, lens, prefix = make([64], 4, 2, 1, 64, "fp16", 64, P=10)
    with pytest.raises(ValueError, match="int32"):
        fa.attention_decode_window(q, k, v, lens.long())
    with pytest.raises(ValueError, match="dtype"):
        fa.attention_decode_window(q, k.float(), v.float(), lens)
    with pytest.raises(ValueError, match="prefix"):
        fa.attention_decode_prefix(q, prefix[0][:1], prefix[1][:1], k, v, lens)
    with pytest.raises(ValueError, match="contiguous"):
        fa.attention_decode_window(q, k.transpose(2, 3).contiguous().transpose(2, 3), v, lens)
    with pytest.raises(fa.FAError, match="sinks"):
        fa.attention_decode_window(q, k, v, lens, 0, 4)
    empty = fa.attention_decode_window(q[:, :, :0].contiguous(), k, v, lens)
    assert empty[0].shape == (1, 4, 0, 64)


@pytest.mark.parametrize("P", [None, 300])
def test_more_sequences_than_the_second_launch_looks_through(fa, P):
    """600 sequences, several rows a block of the second launch, 38 tiles of rows behind the prefix."""
    run(fa, [(i * 37) % 70 for i in range(600)], 16, 2, 1, 64, "fp16", 70, P=P)


def test_prefix_in_pieces(fa):
    """Several tiles of rows: the prefix is cut into pieces as long as a run, here of 26 tiles and of one."""
    run(fa, [50] * 64, 32, 8, 1, 128, "bf16", 50, P=32768)
    run(fa, [0] * 130, 8, 4, 2, 64, "fp16", 64, P=1300)
    run(fa, [1, 2000] * 40, 8, 2, 1, 256, "bf16", 2000, P=777)


def test_rows_longer_than_their_sequence_under_the_largest_window(fa):
    run(fa, [1, 2, 0, 5], 2, 1, 9, 128, "bf16", 8, 2 ** 31 - 1, 2 ** 31 - 1)


def test_another_workspace_and_outputs_keep_their_neighbours(fa):
    q, k, v, lens, prefix = make([300, 7], 4, 2, 1, 128, "bf16", 300, P=200)
    B, H, Nq, d = q.shape
    n = fa.fa_decode_prefix_workspace_size(B, H, 2, Nq, 200, 300, d)
    ws = torch.full((n + 512,), 3, dtype=torch.uint8, device="cuda")
    o = torch.full((B + 2, H, Nq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B + 2, H, Nq), 9.0, device="cuda")
    fa.fa_decode_prefix(q, *prefix, k, v, lens, o[1:3], lse[1:3], d ** -0.5, ws[256:256 + n])
    check(q, k, v, lens, o[1:3], lse[1:3], d ** -0.5, prefix=prefix)
    assert (o[0] == 7).all() and (o[3] == 7).all() and (lse[0] == 9).all() and (lse[3] == 9).all()
    assert (ws[:256] == 3).all() and (ws[256 + n:] == 3).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 32])
def test_rows_that_see_nothing_are_zero_whatever_the_values_are(fa, d, H):
    """Rows in front of the sequence's first token, with values that are not finite in slots that later rows see."""
    q, k, v, lens, _ = make([3, 9], H, 2, 9, d, "bf16", 16)
    v[0, :, 1], v[0, :, 2] = math.inf, math.nan
    o, lse = fa.attention_decode_window(q, k, v, lens)
    assert (o[0, :, :6] == 0).all() and (lse[0, :, :6] == -math.inf).all() and lse[0, :, 6:].isfinite().all()
    check(q[1:], k[1:], v[1:], lens[1:], o[1:], lse[1:], d ** -0.5)
