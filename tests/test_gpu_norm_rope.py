"""Norms of query and key heads with the rotation by position, and its gradients, vs the fp64 oracle.

Tolerances, from what the kernels round: results once to their type (half a step: EPS, relative); before that everything is in
32 bits (u = 2^-24 a rounding).  The sum of squares has d <= 256 positive terms added in at most 8 + 5 steps (13 u), mean, eps,
square root and product with x and w 5 more, halved by the root where they come before it: y = x r w is off by at most
16 u |y|; the rotation adds two roundings of products and one of their sum: |y_a|, |y_b| of a pair weigh in fully, 20 u (|y_a| + |y_b|)
in all.  dx = r (g - xh m) with m = mean(g xh): g is a rotated row times w (4 u of |u| w), m a sum of d products, whose
error is 16 u of mean |g xh|; 32 u r (|g|' + |xh| mean|g|'|xh|) with |g|' from the magnitudes of both channels of a pair.  dw: sums
of n terms in three levels of at most n' = n / groups + groups + blocks steps; (64 + n / 1000) u of the sum of the
terms' magnitudes covers what the tests' sizes make of them.
"""

import numpy as np
import pytest

from oracle.norm_rope import norm_rope64, norm_rope64_backward, rotation

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
U = 2.0 ** -24
E = 1e-5  # eps of the norm


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_07_gb300 import binding, build

    build.build()
    return binding


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype, v):
    """Half a step of the type at |v|, with its smallest spacing."""
    tiny = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}[dtype]
    return EPS[dtype] * np.abs(v) + tiny


def spread(v, cos, sin, interleaved):
    """|v| of a row with both channels of a pair counted in each (v [T, heads, d])."""
    out = np.empty_like(v)
    for t in range(v.shape[0]):
        R = (rotation(cos[t], sin[t], v.shape[-1], interleaved) != 0).astype(float)
        np.fill_diagonal(R, 1.0)
        pairs = np.minimum(R + R.T, 1.0)
        out[t] = np.abs(v[t]) @ pairs
    return out


class Case:
    def __init__(self, fa, T, H, Hkv, d, rotary, dtype, wdtype, interleaved, seed, length=300, positions=True, packed=True,
                 B=1):
        g = torch.Generator().manual_seed(seed)
        self.interleaved, self.dtype, self.wdtype = interleaved, dtype, wdtype
        shape = (T, H + 2 * Hkv, d) if packed else (B, T, H + 2 * Hkv, d)
        scale = 4.0 ** torch.randint(-2, 3, (*shape[:-1], 1), generator=g)
        self.qkv = (torch.randn(shape, generator=g) * scale).to(TORCH[dtype]).cuda()
        self.q, self.k = self.qkv[..., :H, :], self.qkv[..., H:H + Hkv, :]
        self.wq, self.wk = ((1 + 0.5 * torch.randn(d, generator=g)).to(TORCH[wdtype]).cuda() for _ in range(2))
        self.table = fa.rope_table(length, rotary) if rotary else None
        self.pos = torch.randint(0, length, (B * T,), generator=g, dtype=torch.int32).cuda() if positions else None
        at = self.pos.cpu().numpy() if positions else np.tile(np.arange(T), B)
        tab = f64(self.table) if rotary else np.zeros((length, 0))
        self.cos, self.sin = tab[at, :rotary // 2], tab[at, rotary // 2:]

    def rows(self, t):
        return f64(t).reshape(-1, *t.shape[-2:])

    def check_forward(self, qo, ko):
        for x, w, y in ((self.q, self.wq, qo), (self.k, self.wk, ko)):
            xs, ws = self.rows(x), f64(w)
            want = norm_rope64(xs, ws, self.cos, self.sin, E, self.interleaved)
            plain = xs * ws / np.sqrt((xs * xs).mean(-1, keepdims=True) + E)
            tol = half_step(self.dtype, want) + 20 * U * (1 + EPS[self.dtype]) * spread(plain, self.cos, self.sin,
                                                                                        self.interleaved)
            assert (np.abs(self.rows(y) - want) <= tol).all()

    def check_backward(self, dqo, dko, dq, dk, dwq, dwk):
        for x, w, dy, dx, dw in ((self.q, self.wq, dqo, dq, dwq), (self.k, self.wk, dko, dk, dwk)):
            xs, ws, dys = self.rows(x), f64(w), self.rows(dy)
            want, wantw = norm_rope64_backward(dys, xs, ws, self.cos, self.sin, E, self.interleaved)
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + E)
            xh = np.abs(xs * r)
            gm = spread(dys, self.cos, self.sin, self.interleaved)
            m = (gm * np.abs(ws) * xh).mean(-1, keepdims=True)
            tol = half_step(self.dtype, want) + 32 * U * r * (gm * np.abs(ws) + xh * m)
            assert (np.abs(self.rows(dx) - want) <= tol).all()
            n = xs.shape[0] * xs.shape[1]
            tolw = half_step(self.wdtype, wantw) + (64 + n / 1000) * U * (gm * xh).sum((0, 1))
            assert (np.abs(f64(dw) - wantw) <= tolw).all()


SHAPES = [  # T, H, Hkv, d, rotary, interleaved
    (1, 1, 1, 64, 64, False), (5, 3, 1, 128, 128, False), (33, 4, 4, 256, 256, True), (17, 7, 7, 64, 32, True),
    (40, 12, 4, 128, 64, False), (9, 5, 2, 96, 96, False), (8, 2, 1, 80, 16, True), (3, 1, 8, 8, 8, False),
    (21, 9, 1, 16, 8, True), (6, 2, 2, 248, 240, False), (257, 8, 2, 128, 128, True), (12, 4, 2, 64, 0, False)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("bf16", "fp32")])
@pytest.mark.parametrize("T,H,Hkv,d,rotary,interleaved", SHAPES)
def test_packed_rows_and_their_gradients(fa, T, H, Hkv, d, rotary, interleaved, dtype, wdtype):
    c = Case(fa, T, H, Hkv, d, rotary, dtype, wdtype, interleaved, 1000 * T + d + rotary)
    args = (c.q, c.k, c.wq, c.wk, c.table, c.pos, E, interleaved)
    qo, ko = fa.qk_norm_rope(*args)
    c.check_forward(qo, ko)
    g = torch.Generator().manual_seed(T)
    dqo, dko = (torch.randn(t.shape, generator=g).to(t.dtype).cuda() for t in (qo, ko))
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dqo, dko, *args)
    fa.fa_check_device_error()
    c.check_backward(dqo, dko, dq, dk, dwq, dwk)


@pytest.mark.parametrize("B,N,H,Hkv,d,dtype", [(2, 50, 4, 2, 128, "bf16"), (3, 7, 2, 2, 64, "fp16"), (1, 1, 1, 1, 256, "fp32")])
def test_padded_batches_go_to_the_layout_of_attention(fa, B, N, H, Hkv, d, dtype):
    c = Case(fa, N, H, Hkv, d, d, dtype, "fp32", False, 5 + N, positions=False, packed=False, B=B)
    args = (c.q, c.k, c.wq, c.wk, c.table)
    qo, ko = fa.qk_norm_rope(*args, eps=E)
    assert qo.shape == (B, H, N, d) and ko.shape == (B, Hkv, N, d) and qo.is_contiguous() and ko.is_contiguous()
    c.check_forward(qo.transpose(1, 2), ko.transpose(1, 2))
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    dqkv = torch.full_like(c.qkv, 7.0)
    out = (dqkv[..., :H, :], dqkv[..., H:H + Hkv, :])  # a fused gradient
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dqo, dko, *args, eps=E, out=out)
    fa.fa_check_device_error()
    c.check_backward(dqo.transpose(1, 2), dko.transpose(1, 2), dq, dk, dwq, dwk)
    assert (dqkv[..., H + Hkv:, :] == 7.0).all()


def test_many_rows_and_the_sum_of_their_weights_gradients(fa):
    c = Case(fa, 4001, 8, 2, 64, 64, "fp16", "fp32", False, 77)
    args = (c.q, c.k, c.wq, c.wk, c.table, c.pos, E, False)
    g = torch.Generator().manual_seed(3)
    dqo, dko = (torch.randn(t.shape, generator=g).half().cuda() for t in (c.q, c.k))
    got = fa.qk_norm_rope_backward(dqo, dko, *args)
    c.check_backward(dqo, dko, *got)
    again = fa.qk_norm_rope_backward(dqo, dko, *args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # whatever the timing


def test_gradients_against_differences(fa):
    c = Case(fa, 6, 2, 1, 64, 64, "fp32", "fp32", False, 21)
    f = lambda q, w: sum(float((f64(y) * f64(dy)).sum()) for y, dy in zip(  # noqa: E731
        fa.qk_norm_rope(q, c.k, w, c.wk, c.table, c.pos, E), (dqo, dko)))
    g = torch.Generator().manual_seed(4)
    dqo, dko = (torch.randn(t.shape, generator=g).cuda() for t in (c.q, c.k))
    dq, _, dwq, _ = fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, c.wq, c.wk, c.table, c.pos, E)
    # along a direction of one row (a step of h moves y by h |dx| within 32 bits' rounding of the sum of |y dy|, about
    # 500 terms of size 1: 500 u / h) and along one of the weights; the second difference's h^2 is below both
    for h in (2.0 ** -9,):
        e = torch.zeros_like(c.q)
        e[3, 1] = torch.randn(64, generator=g).cuda() * c.q[3, 1].abs().mean()
        got = (f(c.q + h * e, c.wq) - f(c.q - h * e, c.wq)) / (2 * h)
        assert abs(got - float((f64(dq) * f64(e)).sum())) <= 500 * 2 * U / h + 64 * h * h * 16
        ew = torch.randn(64, generator=g).cuda()
        got = (f(c.q, c.wq + h * ew) - f(c.q, c.wq - h * ew)) / (2 * h)
        assert abs(got - float((f64(dwq) * f64(ew)).sum())) <= 500 * 8 * U / h + 64 * h * h * 16


def test_no_weights_no_keys_no_rotation_no_tokens(fa):
    c = Case(fa, 10, 3, 2, 128, 128, "bf16", "fp32", False, 8)
    ones = torch.ones(128, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(fa.qk_norm_rope(c.q, c.k, None, None, c.table, c.pos, E),
                                                 fa.qk_norm_rope(c.q, c.k, ones, ones, c.table, c.pos, E)))
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(c.q, c.k, c.q, c.k, None, None, c.table, c.pos, E)
    assert dwq is None and dwk is None and dq.isfinite().all() and dk.isfinite().all()
    none = c.k[:, :0]
    qo, ko = fa.qk_norm_rope(c.q, none, c.wq, None, c.table, c.pos, E)
    assert ko.shape == (10, 0, 128) and torch.equal(qo, fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, c.pos, E)[0])
    assert torch.equal(fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, None, None, E)[0],
                       fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, torch.zeros_like(c.pos), E)[0])
    q0, k0 = c.q[:0], c.k[:0]
    got = fa.qk_norm_rope_backward(q0, k0, q0, k0, c.wq, c.wk, c.table, c.pos[:0], E)
    assert got[0].shape == q0.shape and (got[2] == 0).all() and (got[3] == 0).all()
    # keys without heads: their weights' gradient is 0
    assert (fa.qk_norm_rope_backward(c.q, none, c.q, none, c.wq, c.wk, c.table, c.pos, E)[3] == 0).all()
    fa.fa_check_device_error()


def test_zero_rows_and_rows_that_are_not_finite(fa):
    c = Case(fa, 8, 2, 2, 128, 128, "bf16", "fp32", False, 9)
    c.qkv[2, 1] = 0.0
    c.qkv[5, 0, 17] = float("nan")
    c.qkv[6, 3, 3] = float("inf")
    qo, ko = fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, c.pos, E)
    assert (qo[2, 1] == 0).all() and qo[5, 0].isnan().all()
    bad_q, bad_k = torch.zeros(8, 2, dtype=torch.bool), torch.zeros(8, 2, dtype=torch.bool)
    bad_q[5, 0] = bad_k[6, 1] = True
    assert (qo.isfinite().all(-1).cpu() == ~bad_q).all() and (ko.isfinite().all(-1).cpu() == ~bad_k).all()
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(torch.ones_like(qo), torch.ones_like(ko), c.q, c.k, c.wq, c.wk, c.table, c.pos, E)
    assert dq[2, 1].isfinite().all() and (dq.isfinite().all(-1).cpu() == ~bad_q).all()
    assert dwq.isnan().any() and dwk.isnan().any()


def test_positions_outside_the_table_are_clamped_and_recorded(fa):
    c = Case(fa, 4, 2, 1, 64, 64, "fp16", "fp32", False, 10, length=100)
    pos = torch.tensor([-1, 99, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    qo, _ = fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, pos, E)
    with pytest.raises(fa.FAError, match="device check"):
        fa.fa_check_device_error()
    want, _ = fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, pos.clamp(0, 99), E)
    fa.fa_check_device_error()
    assert torch.equal(qo, want)


def test_in_place_and_into_one_buffer(fa):
    c = Case(fa, 30, 4, 2, 128, 128, "bf16", "bf16", False, 12)
    qo, ko = fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, c.pos, E)
    both = torch.full((30, 6, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, both[:, 2:], both[:, :2], c.pos, E)
    assert torch.equal(both[:, 2:], qo) and torch.equal(both[:, :2], ko)
    v = c.qkv[:, 6:].clone()
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    want = fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, c.wq, c.wk, c.table, c.pos, E)
    got = fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, c.wq, c.wk, c.table, c.pos, E, out=(dqo, dko))
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(dqo, want[0])
    fa.fa_qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, c.q, c.k, c.pos, E)
    assert torch.equal(c.q, qo) and torch.equal(c.k, ko) and torch.equal(c.qkv[:, 6:], v)


def test_results_are_heads_of_one_tensor(fa):
    c = Case(fa, 20, 4, 2, 64, 64, "bf16", "bf16", False, 13, positions=False, packed=False, B=3)
    qo, ko = fa.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, eps=E)
    both = torch.full((3, 8, 20, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_qk_norm_rope(c.q, c.k, c.wq, c.wk, c.table, both[:, 1:5].transpose(1, 2), both[:, 6:].transpose(1, 2), eps=E)
    assert torch.equal(both[:, 1:5], qo) and torch.equal(both[:, 6:], ko)
    assert (both[:, 0] == 3.0).all() and (both[:, 5] == 3.0).all()


def test_another_stream_and_a_replayed_graph(fa):
    c = Case(fa, 64, 4, 2, 128, 128, "bf16", "fp32", True, 14)
    args = (c.wq, c.wk, c.table, c.pos, E, True)
    want = fa.qk_norm_rope(c.q, c.k, *args)
    dqo, dko = torch.randn_like(want[0]), torch.randn_like(want[1])
    wantb = fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fa.qk_norm_rope(c.q, c.k, *args, stream=side)
    gotb = fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, *args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wantb), (*got, *gotb)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (*fa.qk_norm_rope(c.q, c.k, *args), *fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, *args))
    c.qkv.copy_(c.qkv.flip(0))
    for _ in range(2):
        graph.replay()
    new = (*fa.qk_norm_rope(c.q, c.k, *args), *fa.qk_norm_rope_backward(dqo, dko, c.q, c.k, *args))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, new)) and not torch.equal(out[0], want[0])


def test_more_blocks_than_one_wave_and_guards(fa):
    """Large strides, rows between others' rows: nothing else is written."""
    T, H, d = 3000, 3, 64
    g = torch.Generator().manual_seed(2)
    buf = torch.randn(T, 8, d, generator=g).to(torch.float16).cuda()
    out = torch.full((2, T, 8, d), 5.0, dtype=torch.float16, device="cuda")
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    table = fa.rope_table(T, d)
    fa.fa_qk_norm_rope(buf[:, 1:1 + H], buf[:, 5:7], w, w, table, out[0, :, 2:2 + H], out[1, :, ::4], None, E)
    want = fa.qk_norm_rope(buf[:, 1:1 + H], buf[:, 5:7], w, w, table, None, E)
    assert torch.equal(out[0, :, 2:5], want[0]) and torch.equal(out[1, :, ::4], want[1])
    out[0, :, 2:5] = 5.0
    out[1, :, ::4] = 5.0
    assert (out == 5.0).all()
