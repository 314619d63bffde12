"""Arguments that the norm, window and prefix calls refuse before anything is launched (no GPU: the pointers are not followed)."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("where there is a GPU, a call that is not refused would run on these pointers")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding.load_library()


def message(lib):
    return lib.fa_last_error_message().decode()


P = [0x10000000 * (i + 1) for i in range(16)]  # 256 MB apart
SIZES = {"B": 2, "N": 10, "H": 4, "Hkv": 2, "d": 64, "rotary": 64, "adjacent": 0, "table_len": 100, "eps": 1e-6,
         "dtype": BF16, "wdtype": FP32}


def strides(B, N, H, Hkv, d, packed=None):
    """(batch, token, head) of contiguous [B][N][heads][d] tensors: queries, keys, queries, keys ..."""
    return [(N * h * d, h * d, d) for h in (H, Hkv)]


def norm(lib, ptrs=None, st=None, n=4, **kw):
    a = dict(SIZES, **kw)
    st = st or strides(a["B"], a["N"], a["H"], a["Hkv"], a["d"]) * (n // 2)
    flat = (ctypes.c_int64 * (3 * n))(*[x for t in st for x in t])
    tail = (a["B"], a["N"], a["H"], a["Hkv"], a["d"], a["rotary"], a["adjacent"], a["table_len"], a["eps"], a["dtype"],
            a["wdtype"], None)
    if n == 4:
        q, k, qo, ko, wq, wk, table, pos = ptrs or P[:8]
        return lib.fa_qk_norm_rope(q, k, wq, wk, table, pos, qo, ko, flat, *tail)
    dqo, dko, q, k, dq, dk, wq, wk, table, pos, dwq, dwk, ws = ptrs or P[:13]
    return lib.fa_qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, table, pos, dq, dk, dwq, dwk, ws, a.get("bytes", 1 << 40), flat, *tail)


@pytest.mark.parametrize("n", [4, 6])
@pytest.mark.parametrize("change,status,text", [
    ({"dtype": 5}, UNSUPPORTED, "dtype"), ({"wdtype": FP16}, UNSUPPORTED, "weights"), ({"B": -1}, INVALID, "negative"),
    ({"H": -1}, INVALID, "negative"), ({"d": 60, "rotary": 0}, UNSUPPORTED, "multiple of 8"),
    ({"d": 264, "rotary": 0}, UNSUPPORTED, "multiple of 8"), ({"d": 0, "rotary": 0}, UNSUPPORTED, "multiple of 8"),
    ({"rotary": 4}, INVALID, "rotary"), ({"rotary": 72}, INVALID, "rotary"), ({"rotary": -8}, INVALID, "rotary"),
    ({"eps": float("nan")}, INVALID, "eps"), ({"eps": -1e-6}, INVALID, "eps"), ({"eps": float("inf")}, INVALID, "eps"),
    ({"B": 1 << 20, "N": 1 << 10}, INVALID, "too many"), ({"table_len": 0}, INVALID, "table")])
def test_norm_sizes(lib, n, change, status, text):
    assert norm(lib, n=n, **change) == status and text in message(lib)


@pytest.mark.parametrize("n", [4, 6])
def test_norm_pointers_and_strides(lib, n):
    count = {4: 8, 6: 13}[n]
    for i in range(n):  # rows: null, not aligned
        for bad, text in ((None, "null"), (P[i] + 8, "aligned")):
            assert norm(lib, [bad if j == i else P[j] for j in range(count)], n=n) == INVALID and text in message(lib)
    for i in (n, n + 1):  # weights may be null, not off their elements
        assert norm(lib, [P[j] + (2 if j == i else 0) for j in range(count)], n=n) == INVALID and "aligned" in message(lib)
    assert norm(lib, [None if j == n + 2 else P[j] for j in range(count)], n=n) == INVALID and "null" in message(lib)
    assert norm(lib, [P[j] + (2 if j == n + 3 else 0) for j in range(count)], n=n) == INVALID and "4-byte" in message(lib)
    # no positions: the table has to reach N
    assert norm(lib, [None if j == n + 3 else P[j] for j in range(count)], n=n, table_len=9) == INVALID
    assert "table_len" in message(lib)
    good = strides(2, 10, 4, 2, 64) * (n // 2)
    for i in range(n):
        for dim in range(3):
            for bad, text in ((-64, "negative"), (good[i][dim] + 4, "16 bytes"), (1 << 40, "too large")):
                st = [list(t) for t in good]
                st[i][dim] = bad
                assert norm(lib, st=st, n=n) == INVALID and text in message(lib)
    for i in (n - 2, n - 1):  # rows of outputs over one another
        for dim, bad in ((0, 64), (1, 64), (2, 0), (2, 32), (0, good[i][0] - 64), (1, 0)):
            st = [list(t) for t in good]
            st[i][dim] = bad
            assert norm(lib, st=st, n=n) == INVALID and "overlap" in message(lib)
    assert lib.fa_qk_norm_rope(*P[:8], None, 1, 1, 1, 1, 64, 64, 0, 100, 1e-6, BF16, FP32, None) == INVALID
    assert "strides" in message(lib)


def test_norm_overlaps(lib):
    size = 2 * 10 * 4 * 64 * 2  # bytes of Q
    for which, at in ((2, P[0] + 16), (2, P[0] - size + 16), (2, P[1]), (3, P[0]), (3, P[2] + size - 16), (3, P[2])):
        ptrs = P[:8]
        ptrs[which] = at
        assert norm(lib, ptrs) == INVALID and "overlaps" in message(lib)
    # side by side inside a token of one buffer, but one row too close, or with other strides
    fused = [(10 * 512, 512, 64)] * 4
    at = lambda heads: P[8] + heads * 128  # noqa: E731
    assert norm(lib, [*P[:2], at(0), at(3), *P[4:8]], fused) == INVALID and "overlaps" in message(lib)
    assert norm(lib, [*P[:2], at(0), at(7), *P[4:8]], fused) == INVALID and "overlaps" in message(lib)
    other = [fused[0], fused[0], fused[0], (10 * 512, 1024, 64)]
    assert norm(lib, [*P[:2], at(0), at(4), *P[4:8]], other) == INVALID
    # in place with other strides than the input's
    assert norm(lib, [P[0], P[1], P[0], P[3], *P[4:8]], [(2560, 256, 64), (1280, 128, 64), (256, 512, 64), (1280, 128, 64)]) \
        == INVALID
    # the keys' result over the queries
    assert norm(lib, [P[0], P[1], P[2], P[0], *P[4:8]]) == INVALID and "overlaps" in message(lib)
    # backward: a weight's gradient twice, a workspace that is too small or none
    ptrs = P[:13]
    ptrs[11] = ptrs[10]
    assert norm(lib, ptrs, n=6) == INVALID and "dwq" in message(lib)
    ptrs[11] = ptrs[10] + 64 * 4 - 16
    assert norm(lib, ptrs, n=6) == INVALID and "dwq" in message(lib)
    # heads of one tensor [B][heads][N][d]: not one head too close
    outer = [(10 * 64 * 8, 64, 640)] * 2
    assert norm(lib, [*P[:2], P[8], P[8] + 3 * 640 * 2, *P[4:8]], strides(2, 10, 4, 2, 64) + outer) == INVALID
    assert norm(lib, P[:12] + [None], n=6) == INVALID and "null" in message(lib)
    need = lib.fa_qk_norm_rope_bwd_workspace_size(64)
    assert need > 0 and lib.fa_qk_norm_rope_bwd_workspace_size(60) == 0 and lib.fa_qk_norm_rope_bwd_workspace_size(512) == 0


def test_norm_without_rows_is_nothing(lib):
    none = [None] * 8
    for change in ({"B": 0}, {"N": 0}, {"H": 0, "Hkv": 0}):
        assert norm(lib, none, **change) == OK
        assert norm(lib, [None] * 13, n=6, **change) == OK


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    from exact_tiled_attention_07_gb300 import binding as fa

    q, k, w, t = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64), torch.ones(64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(q, k, w, w, t)
    with pytest.raises(ValueError, match="batch, tokens"):
        fa.fa_qk_norm_rope(q, k[:3], w, w, t, q, k[:3])
    with pytest.raises(ValueError, match="contiguous"):
        fa.fa_qk_norm_rope(q, k, w, w, t, torch.zeros(4, 64, 2).transpose(1, 2), k)
    with pytest.raises(ValueError, match="heads"):
        fa.fa_qk_norm_rope(q, k, w, w, t, q, q)
    with pytest.raises(ValueError, match="without weights"):
        fa.fa_qk_norm_rope_bwd(q, k, q, k, None, None, t, q, k, w, w)


# ------------------------------------------------------------------------------------------------ window with sinks


def fwd_window(lib, window=10, sinks=2, d=64, dtype=BF16, H=4, Hkv=2, scale=0.125, ptrs=P[:5], N=100):
    return lib.fa_fwd_window(*ptrs, 1, H, Hkv, N, d, scale, window, sinks, dtype, None)


def bwd_window(lib, window=10, sinks=2, d=64, dtype=BF16, H=4, Hkv=2, scale=0.125, ptrs=P[:10], N=100, size=1 << 40):
    return lib.fa_bwd_window(*ptrs, size, 1, H, Hkv, N, d, scale, window, sinks, dtype, None)


def varlen_window(lib, window=10, sinks=2, d=64, dtype=BF16, H=4, Hkv=2, scale=0.125, ptrs=P[:6], T=100, strides=(256, 64) * 4):
    return lib.fa_fwd_varlen_window(*ptrs, 3, T, H, Hkv, d, *strides, scale, window, sinks, dtype, None)


@pytest.mark.parametrize("call,n", [(fwd_window, 5), (bwd_window, 10), (varlen_window, 6)])
def test_window_arguments(lib, call, n):
    for bad in ({"window": 0}, {"window": -1}):
        assert call(lib, **bad) == INVALID and "window" in message(lib)
    assert call(lib, sinks=-1) == INVALID and "sinks" in message(lib)
    assert call(lib, H=3) == INVALID and "multiple of Hkv" in message(lib)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == INVALID and "scale" in message(lib)
    assert call(lib, dtype=FP32) == UNSUPPORTED and call(lib, d=96) == UNSUPPORTED and call(lib, d=512) == UNSUPPORTED
    for i in range(n):
        assert call(lib, ptrs=[None if j == i else P[j] for j in range(n)]) == INVALID and "null" in message(lib)
        assert call(lib, ptrs=[P[j] + (2 if j == i else 0) for j in range(n)]) == INVALID and "aligned" in message(lib)
    assert bwd_window(lib, size=1000) == INVALID and "workspace" in message(lib)
    assert varlen_window(lib, strides=(256, 64) * 3 + (64, 64)) == INVALID and "overlap" in message(lib)
    assert fwd_window(lib, N=0, ptrs=[None] * 5) == OK and bwd_window(lib, N=0, ptrs=[None] * 10) == OK
    assert varlen_window(lib, T=0, ptrs=[None] * 6) == OK


def test_binding_keeps_sinks_to_causal_windows():
    from exact_tiled_attention_07_gb300 import binding as fa

    assert not fa._sinks_allowed(False, 0, 0) and fa._sinks_allowed(True, 5, 1)
    for causal, window, mask in ((False, 5, None), (True, 0, None), (True, 5, object())):
        with pytest.raises(ValueError, match="sinks go with"):
            fa._sinks_allowed(causal, window, 3, mask)


# ------------------------------------------------------------------------------------------------ decode over caches


def decode_window(lib, B=2, H=4, Hkv=2, Nq=1, C=100, d=64, scale=0.125, window=10, sinks=2, dtype=BF16, ptrs=P[:6], ws=P[6],
                  size=1 << 50):
    return lib.fa_decode_window(*ptrs, B, H, Hkv, Nq, C, d, scale, window, sinks, dtype, ws, size, None)


def decode_prefix(lib, B=2, H=4, Hkv=2, Nq=1, C=100, d=64, scale=0.125, dtype=BF16, ptrs=P[:8], ws=P[8], size=1 << 50, Pn=50):
    return lib.fa_decode_prefix(*ptrs, B, H, Hkv, Nq, Pn, C, d, scale, dtype, ws, size, None)


@pytest.mark.parametrize("call,n,words", [(decode_window, 6, (3, 5)), (decode_prefix, 8, (5, 7))])
def test_decode_arguments(lib, call, n, words):
    for bad in ({"B": -1}, {"H": -2}, {"Nq": -1}):
        assert call(lib, **bad) == INVALID and "negative" in message(lib)
    assert call(lib, C=0) == INVALID and "capacity" in message(lib)
    assert call(lib, H=3) == INVALID and call(lib, Hkv=0) == INVALID
    assert call(lib, d=96) == UNSUPPORTED and call(lib, dtype=FP32) == UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == INVALID and "scale" in message(lib)
    for big in ({"C": 2 ** 31 - 100}, {"B": 2 ** 20, "Nq": 2 ** 10}, {"B": 2 ** 28, "Hkv": 4, "Nq": 1}):
        assert call(lib, **big) == INVALID and "too large" in message(lib)
    for i in range(n):
        assert call(lib, ptrs=[None if j == i else P[j] for j in range(n)]) == INVALID and "null" in message(lib)
        off = 2 if i in words else 8
        assert call(lib, ptrs=[P[j] + (off if j == i else 0) for j in range(n)]) == INVALID and "aligned" in message(lib)
    assert call(lib, ws=None) == INVALID and "null" in message(lib)
    assert call(lib, size=100) == INVALID and "workspace" in message(lib)
    for nothing in ({"B": 0}, {"H": 0}, {"Nq": 0}):
        assert call(lib, ptrs=[None] * n, ws=None, size=0, **nothing) == OK
    assert lib.fa_decode_window_workspace_size(2, 4, 2, 1, 100, 64) > 0
    assert lib.fa_decode_prefix_workspace_size(2, 4, 2, 1, 50, 100, 64) > lib.fa_decode_window_workspace_size(2, 4, 2, 1, 100, 64)
    assert lib.fa_decode_window_workspace_size(2, 3, 2, 1, 100, 64) == 0


def test_decode_window_and_prefix_sizes(lib):
    assert decode_window(lib, window=-1) == INVALID and "window" in message(lib)
    assert decode_window(lib, sinks=-1) == INVALID and "sinks" in message(lib)
    assert decode_window(lib, window=0, sinks=1) == INVALID and "sinks" in message(lib)
    assert decode_prefix(lib, Pn=-1) == INVALID and "negative" in message(lib)
    assert decode_prefix(lib, Pn=2 ** 31 - 1) == INVALID and "too large" in message(lib)
