"""The serving calls with lengths and offsets outside their range: the error is recorded, what lies inside the range is done,
and nothing outside it is written."""

import numpy as np
import pytest

from oracle import kv4 as KV
from test_gpu_kv4 import cu_of, fa, i32, make_cache, random_rows, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def reported(fa):  # noqa: F811
    with pytest.raises(fa.FAError, match="device check"):
        fa.fa_check_device_error()
    fa.fa_check_device_error()  # cleared


# rows 3-8 of sequence 0, 9-14 of sequence 1 end at lens[b]; a slot outside [0, 64) is none
@pytest.mark.parametrize("lens", [[4, 64], [6, 70], [-5, 64], [0, 200], [67, 3]])
@pytest.mark.parametrize("d", [64, 256])
def test_append_and_read_outside_the_cache(fa, lens, d):  # noqa: F811
    hkv, cap = 2, 64
    cu = [3, 9, 15]
    k, v = (random_rows(20, hkv, d, "bf16", s, special=False).cuda() for s in (3, 4))
    # two sequences between two more, which stay as they are
    cache = torch.full((4, hkv, cap // 64, 72 * d), 0xA5, dtype=torch.uint8, device="cuda")
    weights = torch.full((4, hkv, cap), 7.0, device="cuda")
    fa.fa_kv4_append(k, v, i32(cu), i32(lens), cache[1:3], weights[1:3])
    reported(fa)
    want = np.full(cache.shape, 0xA5, np.uint8)
    w_want = np.full(weights.shape, 7.0)
    parts = KV.unpack_blocks(want)
    rows = [(b, r, lens[b] - cu[b + 1] + r) for b in range(2) for r in range(cu[b], cu[b + 1])]
    rows = [(b, r, slot) for b, r, slot in rows if 0 <= slot < cap]
    held = []
    for x, (c, s, m) in zip((k, v), parts):
        qc, qs, qm = KV.quantize_rows(rows_of(x))
        held.append(KV.dequantize_rows(qc, qs, qm))
        for b, r, slot in rows:
            c[1 + b, :, slot], s[1 + b, :, slot], m[1 + b, :, slot] = qc[r], qs[r], qm[r]
            w_want[1 + b, :, slot] = 0
    assert np.array_equal(KV.pack_blocks(*parts), cache.cpu().numpy())
    assert np.array_equal(w_want, weights.cpu().numpy())
    # read: rows whose slots are none are left as they were
    rk, rv = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    fa.fa_kv4_read(cache[1:3], i32(cu), i32(lens), rk, rv)
    reported(fa)
    for x, h in ((rk, held[0]), (rv, held[1])):
        want_x = torch.full(k.shape, 9.0, dtype=torch.bfloat16)
        for _, r, _ in rows:
            want_x[r] = torch.from_numpy(h[r].astype(np.float32)).bfloat16()
        assert torch.equal(want_x, x.cpu())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("keep,cap", [(100, 1088), (3000, 20032)])
def test_evict_lengths_outside_the_cache(fa, d, keep, cap):  # noqa: F811
    hkv, out_cap = 2, (keep + 63) // 64 * 64 + 64
    cache = torch.randint(0, 256, (4, hkv, cap // 64, 72 * d), dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 50, (4, hkv, cap), device="cuda").float()
    got = []
    for lens in ([-4, cap + 100, keep + 7, 2 ** 31 - 1], [0, cap, keep + 7, cap]):
        # outputs between guards
        out = torch.full((6, hkv, out_cap // 64, 72 * d), 0x5A, dtype=torch.uint8, device="cuda")
        w2 = torch.full((6, hkv, out_cap), -7.0, device="cuda")
        n2, kept = i32([99] * 6), torch.full((6, hkv, keep), 99, dtype=torch.int32, device="cuda")
        fa.fa_kv4_evict(cache, w, i32(lens), keep, 11, out[1:5], w2[1:5], n2[1:5], kept[1:5])
        if lens[0] < 0:
            reported(fa)
        fa.fa_check_device_error()
        got.append((out, w2, n2, kept))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    out, w2, n2, kept = got[0]
    assert n2.tolist() == [99, 0, keep, keep, keep, 99]
    for end in (0, 5):
        assert (out[end] == 0x5A).all() and (w2[end] == -7).all() and (kept[end] == 99).all()
    assert (w2[1:5, :, keep:] == -7).all() and (out[1] == 0x5A).all() and (kept[1] == -1).all()


@pytest.mark.parametrize("lens", [[500, -4, 128, 2 ** 31 - 1], [-2 ** 31, 129, 1, 0]])
@pytest.mark.parametrize("d", [64, 256])
def test_decode_lengths_outside_the_cache(fa, lens, d):  # noqa: F811
    cap, B = 128, 4
    cache, _, _ = make_cache(B, 1, cap, d, 61)
    q = torch.randn(B, 2, 2, d, dtype=torch.float16, device="cuda")
    got = []
    for n in (lens, [min(max(x, 0), cap) for x in lens]):
        o, lse = torch.full((B + 2, 2, 2, d), 5.0, dtype=torch.float16, device="cuda"), torch.full((B + 2, 2, 2), 5.0, device="cuda")
        w = torch.full((B + 2, 1, cap), -3.0, device="cuda")
        ws = torch.empty(fa.fa_decode_kv4_workspace_size(B, 2, 1, 2, cap, d, True), dtype=torch.uint8, device="cuda")
        fa.fa_decode_kv4(q, cache, i32(n), o[1:-1], lse[1:-1], d ** -0.5, causal=True, weights_out=w[1:-1], workspace=ws)
        if n is lens:
            reported(fa)
        fa.fa_check_device_error()
        got.append((o, lse, w))
    for a, b, guard in zip(*got, (5, 5, -3)):
        assert torch.equal(a, b) and (a[0] == guard).all() and (a[-1] == guard).all()


# offsets and the sequences that are left of them: clamped to [0, T], empty where they decrease
@pytest.mark.parametrize("cu,left", [([0, 5000], [(0, 256)]), ([300, 200, 100], []), ([-50, 100, 2 ** 31 - 1], [(0, 100), (100, 256)]),
                                     ([-7, -3, 60, 60, 40], [(0, 60)])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_packed_offsets_outside_the_rows(fa, cu, left, d):  # noqa: F811
    T, H = 256, 2
    g = torch.Generator().manual_seed(13)
    # rows in front of and behind the T that the call is given
    q, k, v = (torch.randn(T + 400, h, d, generator=g).bfloat16().cuda()[200:200 + T] for h in (H, 1, 1))
    o = torch.full((T + 400, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    flat = torch.full((H * T + 400,), 9.0, device="cuda")
    lse = flat[200:200 + H * T].view(H, T)
    fa.fa_fwd_varlen(q, k, v, o[200:200 + T], lse, i32(cu), d ** -0.5, True)
    reported(fa)
    assert (o[:200] == 7).all() and (o[200 + T:] == 7).all() and (flat[:200] == 9).all() and (flat[200 + H * T:] == 9).all()
    seen = torch.zeros(T, dtype=torch.bool, device="cuda")
    for first, end in left:
        ro, rl = fa.attention_forward_varlen(q[first:end], k[first:end], v[first:end], cu_of([end - first]), causal=True)
        assert torch.equal(o[200 + first:200 + end], ro) and torch.equal(lse[:, first:end], rl)
        seen[first:end] = True
    assert (o[200:200 + T][~seen] == 7).all() and (lse[:, ~seen] == 9).all()
