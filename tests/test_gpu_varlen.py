"""Packed sequences of different lengths through the C ABI vs the fp64 oracle, one sequence at a time."""

import numpy as np
import pytest

import oracle
from oracle.gqa import expand_kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step, relative


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def cu_of(lens, first=0):
    return torch.tensor(np.concatenate(([first], first + np.cumsum(lens))), dtype=torch.int32, device="cuda")


def inputs(T, H, hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * hkv, d, generator=g).to(TORCH[dtype]).cuda()
    return qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]  # slices of one projection


def check(q, k, v, o, lse, lens, first, causal, dtype, scale):
    """Tolerances: P and O are each rounded to the 16-bit type (half a step, relative to the row's largest
    |V|), scores are fp32 sums of d products (d / 16 steps, each 2^-23 of the largest partial sum)."""
    H, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    at = first
    for n in lens:
        if n == 0:
            continue
        x = [f64(t[at:at + n]).swapaxes(0, 1)[None] for t in (q, k, v)]
        ro, rl = oracle.attn_fwd64(x[0], expand_kv(x[1], H), expand_kv(x[2], H), scale, causal)
        mag = scale * np.linalg.norm(x[0], axis=-1).max() * np.linalg.norm(x[1], axis=-1).max()
        ds = (d / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -20
        go, gl = f64(o[at:at + n]).swapaxes(0, 1)[None], f64(lse[:, at:at + n])[None]
        vmax = np.abs(x[2]).max()
        assert np.abs(gl - rl).max() <= ds + 2.0 ** -20 * (8 + np.abs(rl).max())
        assert (np.abs(go - ro) <= EPS[dtype] * (vmax + np.abs(ro)) + 2 * (ds + 2.0 ** -20) * vmax).all()
        at += n


def run(fa, lens, H, hkv, d, dtype, causal, seed, first=0, behind=0):
    T = first + sum(lens) + behind
    q, k, v = inputs(T, H, hkv, d, dtype, seed)
    o = torch.full((T, H, d), 7.0, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((H, T), 9.0, device="cuda")
    scale = d ** -0.5
    fa.fa_fwd_varlen(q, k, v, o, lse, cu_of(lens, first), scale, causal)
    fa.fa_check_device_error()
    check(q, k, v, o, lse, lens, first, causal, dtype, scale)
    end = first + sum(lens)  # rows of no sequence: as they were
    assert (o[:first] == 7).all() and (o[end:] == 7).all() and (lse[:, :first] == 9).all() and (lse[:, end:] == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_around_the_tiles(fa, dtype, d, causal):
    run(fa, [1, 0, 127, 128, 129, 255, 256, 257, 2, 500, 64], 4, 2, d, dtype, causal, 1)


@pytest.mark.parametrize("H,hkv", [(1, 1), (3, 1), (8, 8), (8, 1)])
def test_heads(fa, H, hkv):
    run(fa, [300, 5, 700], H, hkv, 128, "bf16", True, 2)
    run(fa, [300, 5, 700], H, hkv, 64, "fp16", False, 3)


def test_one_token_and_one_sequence(fa):
    run(fa, [1], 4, 4, 128, "bf16", True, 4)
    run(fa, [1500], 4, 2, 128, "bf16", True, 5)
    run(fa, [0, 0, 1, 0], 2, 1, 64, "fp16", True, 6)


def test_many_short_sequences(fa):
    rng = np.random.default_rng(7)
    run(fa, rng.integers(0, 40, 300).tolist(), 4, 2, 64, "bf16", True, 7)


def test_rows_of_no_sequence(fa):
    for d in (64, 128, 256):
        run(fa, [100, 30, 200], 2, 1, d, "bf16", True, 8, first=70, behind=300)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_sequences_do_not_reach_each_other(fa, d, causal):
    lens = [130, 77, 300, 1, 200]
    T = sum(lens)
    q, k, v = (t.clone() for t in inputs(T, 4, 2, d, "bf16", 9))
    o, lse = fa.attention_forward_varlen(q, k, v, cu_of(lens), causal=causal)
    bad = slice(130, 207)
    for t, x in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        t[bad] = x
    o2, lse2 = fa.attention_forward_varlen(q, k, v, cu_of(lens), causal=causal)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])
    assert torch.isnan(o2[bad]).all()


def test_same_as_the_unpacked_forward(fa):
    # equal lengths: bit for bit the forward over a batch
    B, n, H, hkv, d = 3, 384, 4, 2, 128
    q, k, v = inputs(B * n, H, hkv, d, "bf16", 10)
    o, lse = fa.attention_forward_varlen(q, k, v, cu_of([n] * B), causal=True)
    un = lambda t: t.unflatten(0, (B, n)).transpose(1, 2).contiguous()  # noqa: E731
    ro, rl = fa.attention_forward(un(q), un(k), un(v), causal=True)
    assert torch.equal(un(o), ro) and torch.equal(lse.view(H, B, n).transpose(0, 1), rl)


def test_output_strides_and_transposed_layout(fa):
    lens, H, d = [200, 131], 4, 128
    T = sum(lens)
    q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in inputs(T, H, H, d, "fp16", 11))  # head-major
    wide = torch.full((T, H, 2 * d), 5.0, dtype=torch.float16, device="cuda")
    o, lse = wide[..., :d], torch.empty(H, T, device="cuda")
    fa.fa_fwd_varlen(q, k, v, o, lse, cu_of(lens), d ** -0.5, True)
    check(q, k, v, o, lse, lens, 0, True, "fp16", d ** -0.5)
    assert (wide[..., d:] == 5).all()


def test_graph_with_other_lengths_and_two_streams(fa):
    T, H, hkv, d = 1000, 8, 2, 128
    q, k, v = inputs(T, H, hkv, d, "bf16", 12)
    cu = cu_of([1000, 0, 0, 0])
    o, lse = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(H, T, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_varlen(q, k, v, o, lse, cu, d ** -0.5, True)
    for lens in ([1000, 0, 0, 0], [1, 500, 130, 369], [250] * 4):
        cu.copy_(cu_of(lens))
        graph.replay()
        check(q, k, v, o, lse, lens, 0, True, "bf16", d ** -0.5)
    refs = [fa.attention_forward_varlen(q, k, v, cu_of(n), causal=True) for n in ([400, 600], [1, 999])]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    cus = [cu_of([400, 600]), cu_of([1, 999])]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            outs[i].append(fa.attention_forward_varlen(q, k, v, cus[i], causal=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in outs[i]:
            assert torch.equal(a, refs[i][0]) and torch.equal(b, refs[i][1])


def test_bad_offsets_are_reported(fa):
    # offsets outside [0, T] or decreasing are clamped in the kernel, so nothing outside the tensors is touched
    T, d = 256, 64
    q, k, v = inputs(T, 2, 1, d, "bf16", 13)
    for cu in ([0, 5000], [-50, 100, 90, 256], [300, 200, 100]):
        fa.attention_forward_varlen(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), causal=True)
        with pytest.raises(fa.FAError, match="device check"):
            fa.fa_check_device_error()


def test_refusals(fa):
    q, k, v = inputs(64, 4, 2, 64, "bf16", 14)
    cu = cu_of([64])
    with pytest.raises(fa.FAError, match="bf16 or fp16"):
        fa.attention_forward_varlen(q.float(), k.float(), v.float(), cu)
    with pytest.raises(fa.FAError, match="supports d"):
        fa.attention_forward_varlen(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), cu)
    with pytest.raises(fa.FAError, match="stride"):
        fa.attention_forward_varlen(q, k[:, :1].expand(64, 2, 64), v, cu)
    with pytest.raises(ValueError, match="multiple of Hkv"):
        fa.attention_forward_varlen(q[:, :3], k, v, cu)
    with pytest.raises(ValueError, match="int32"):
        fa.attention_forward_varlen(q, k, v, cu.long())
    empty, lse = fa.attention_forward_varlen(q[:0], k[:0], v[:0], cu_of([0]))
    assert empty.shape[0] == 0 and lse.shape == (4, 0)
