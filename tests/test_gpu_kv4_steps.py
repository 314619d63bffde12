"""Decode over the 4-bit cache whose values have steps of very different sizes: a row's O keeps the precision of the values
that the row looks at, whatever steps other slots or other rows' slots have."""

import pytest

from test_gpu_kv4 import EPS, TORCH, fa, i32  # noqa: F401
from test_gpu_kv4_long_runs import values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HEADS, SLOTS = 608, 1024  # 16 blocks a CTA and more


def make(mode, d, rows, dtype):
    """q [1, HEADS rows, 1, d] and a cache [1, HEADS, 16, 72 d].  Queries are near 1 in every channel, so a key's middle
    moves its score; keys' steps give scores a deviation of about 1."""
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    G = d // 64
    q = 1 + 0.3 * torch.randn(1, HEADS * rows, 1, d, generator=g, device="cuda")
    codes = torch.randint(0, 256, (HEADS, SLOTS // 64, 64 * d), generator=g, dtype=torch.uint8, device="cuda")
    ks = (0.2 + 0.1 * rand(HEADS, SLOTS, G)) * d ** -0.5 * 8
    km = ks / 2  # the codes' mean is 7.5
    vs, vm = 0.001 * (1 + rand(HEADS, SLOTS, G)), 0.002 * rand(HEADS, SLOTS, G)
    up = 1 / d ** 0.5  # a middle that raises the score by 1 (of q k / sqrt d with q near 1)
    slot = torch.arange(SLOTS, device="cuda")
    big = slot % 32 == 5
    if mode == "slot":  # large values that nobody looks at, and one key some 7 (10 log2 units) in front
        vs[:, big] = 4096.0
        km[:, big] -= 60 * up
        km[:, 600] += 7 * up
    elif mode == "late":  # large values that the first blocks' queries look at until a key 25 in front comes
        vs[:, big & (slot < 300)] = 4096.0
        km[:, slot >= 320] += 25 * up
        ks[:, slot >= 320] *= 0.2
    elif mode == "channels":  # all large, of the last 64 channels
        vs[..., -1] *= 2.0 ** 21
    elif mode == "nan":
        vs[:, 40, -1], vm[:, 40, -1] = float("nan"), float("nan")
    elif mode == "rows":  # the slots that half of the rows look at are large
        vs[:, big] = 4096.0
        km[:, big] -= 40 * up
        q[:, ::2] = -q[:, ::2]
    par = lambda s, m: torch.stack((s, m), -1).half().view(torch.uint8).view(HEADS, SLOTS // 64, 4 * d)  # noqa: E731
    cache = torch.cat((codes, par(ks, km), par(vs, vm)), -1)[None]
    return q.to(TORCH[dtype]), cache.contiguous()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows", [4, 16])
@pytest.mark.parametrize("mode,d", [(m, d) for m in ("slot", "late", "channels", "nan", "rows") for d in (64, 128, 256)
                                    if d > 64 or m not in ("channels", "nan")])  # (d = 64 is one group of channels)
def test_steps_of_different_sizes(fa, mode, d, rows, dtype):  # noqa: F811
    q, cache = make(mode, d, rows, dtype)
    scale = d ** -0.5
    o, lse = fa.attention_decode_kv4(q, cache, i32([SLOTS]), scale=scale)
    fa.fa_check_device_error()
    for h in (0, 301, HEADS - 1):
        k, v = values(cache[0, h], 0), values(cache[0, h], 1).view(SLOTS, -1, 64)
        x = q[0, h * rows:(h + 1) * rows, 0].double()
        s = x @ k.T * scale
        p = torch.softmax(s, -1)
        # the row's largest product of a probability and a step (a NaN is none)
        par = cache[0, h, :, 68 * d:].contiguous().view(torch.float16).double().view(SLOTS, -1, 2)
        most = torch.stack([(p * par[:, gr, 0].nan_to_num(0.0)).amax(-1) for gr in range(d // 64)]).amax(0)
        got = o[0, h * rows:(h + 1) * rows, 0].double().view(rows, -1, 64)
        mag = (x.abs() @ k.abs().T).max().item() * scale
        ds = (d / 16 + 8) * 4 * 2.0 ** -23 * mag + 2.0 ** -20
        assert (lse[0, h * rows:(h + 1) * rows, 0].double() - torch.logsumexp(s, -1)).abs().max() <= ds + 2.0 ** -16
        for gr in range(d // 64):
            step, middle = par[:, gr, 0], par[:, gr, 1]
            if step.isnan().any():
                assert got[:, gr].isnan().all()
                continue
            ref = p @ v[:, gr]
            # sizes of what is added up: probabilities times steps, and times all that a value can be
            y = p * step
            size = (y * 8 + p * middle.abs()).sum(-1)
            # Probabilities times steps are rounded to fp16, for fp16 queries the rounding errors too (2^-11 of 2^-11), but
            # to no less than 2^-33 of the row's largest; a code - 8 is at most 8 from 0.  Scores' errors
            # count twice (numerator and sum); each of SLOTS / 16 matrix steps (two each for fp16 queries) cuts less than
            # 2^-23 off sums of codes up to 15, twice `size` at the most; corr's sums are rounded SLOTS times.
            r = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
            tol = 8 * (r * y.sum(-1) + SLOTS * 2.0 ** -33 * most) + size * (
                2 * ds + 2 * SLOTS / 16 * 2.0 ** -23 * 2 + SLOTS * 2.0 ** -24)
            tol = tol[:, None] + EPS[dtype] * ref.abs() + (2.0 ** -25 if dtype == "fp16" else 0)  # fp16's subnormal O
            err = (got[:, gr] - ref).abs()
            worst = (err / tol).max().item()
            assert worst <= 1, (h, gr, worst, (err / ref.abs().mean()).max().item())
