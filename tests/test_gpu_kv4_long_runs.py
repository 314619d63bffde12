"""Decode over the 4-bit cache where a CTA takes hundreds of blocks of one head: the error of O against fp64, relative to
O's own size.

A value is middle + step (code - 8) with codes all over 0 .. 15, so O is what is left of sums that are hundreds of times
larger when the weights are flat; the products' fp32 sums are truncated at each matrix step, always
downwards, and this is where that shows."""

import pytest

from test_gpu_kv4 import EPS, TORCH, fa, i32  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# tokens that a warp adds up before it takes the codes' offset off the sums
FOLD = 128


def cache_of(B, hkv, cap, d, seed):
    """Random codes; steps about 1/4, middles that make the values' mean 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = cap // 64
    cache = torch.randint(0, 256, (B, hkv, nb, 72 * d), generator=g, dtype=torch.uint8, device="cuda")
    step = torch.rand(B, hkv, nb, 8 * d // 4, generator=g, device="cuda") * 0.1 + 0.2  # one for every 64 channels of a row
    cache[..., 64 * d:] = torch.stack((step, step / 2), -1).half().view(torch.uint8).flatten(-2)
    return cache


def values(blocks, which):
    """fp64 [cap, d] keys (0) or values (1) of one head's blocks [cap / 64, 72 d]."""
    d = blocks.shape[-1] // 72
    by = blocks[:, which * 32 * d:(which + 1) * 32 * d].reshape(-1, d // 2)
    code = torch.stack((by & 15, by >> 4), -1).flatten(-2).double().unflatten(-1, (-1, 64))
    par = blocks[:, (64 + 4 * which) * d:(68 + 4 * which) * d].contiguous().view(torch.float16).double().view(-1, d // 64, 2)
    return (par[..., 1:] + par[..., :1] * (code - 8)).flatten(-2)


# 4 rows a head in one row tile (608 CTAs; 304 at d = 256), 16 in two (304): 200 to 400 blocks a CTA
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,H,hkv,cap,d", [(8, 240, 15, 65536, 64), (30, 32, 8, 32768, 128), (15, 16, 4, 65536, 256)])
def test_decode_error_relative_to_what_is_left(fa, B, H, hkv, cap, d, dtype):  # noqa: F811
    cache = cache_of(B, hkv, cap, d, 5)
    rows = H // hkv
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(B, H, 1, d, generator=g, device="cuda").to(TORCH[dtype])
    scale = 0.8 / d ** 0.5  # keys' deviation is 0.25 x 4.6: scores of deviation 0.9
    o, lse = fa.attention_decode_kv4(q, cache, i32([cap] * B), scale=scale)
    fa.fa_check_device_error()
    off = total = bias = 0.0
    n, mag = 0, 0.0
    for b, h in ((0, 0), (1, hkv - 1), (B // 2, hkv // 2), (B - 1, hkv - 1)):
        k, v = values(cache[b, h], 0), values(cache[b, h], 1)
        x = q[b, h * rows:(h + 1) * rows, 0].double()
        s = x @ k.T * scale
        mag = max(mag, (x.abs() @ k.abs().T).max().item() * scale)
        ref = torch.softmax(s, -1) @ v
        e = o[b, h * rows:(h + 1) * rows, 0].double() - ref
        off, total, bias, n = off + (e ** 2).sum().item(), total + (ref ** 2).sum().item(), bias + e.sum().item(), n + e.numel()
        dl = (lse[b, h * rows:(h + 1) * rows, 0].double() - torch.logsumexp(s, -1)).abs().max().item()
        assert dl <= 2.0 ** -12, dl
    rms = (total / n) ** 0.5
    # Matrix steps of 16 tokens (twice for fp16 queries, whose probabilities' rounding errors are a second operand),
    # each off by less than 2^-23 of the sum that it adds to, downwards: with weights w of mean 1 that sum grows to
    # 7.5 FOLD before the offset of 8 comes off, 7.5 FOLD / 2 on average.  O is what cap tokens leave of it:
    # deviation 4.6 of a code, sqrt(cap) w's root mean square (1.5 for scores of deviation 0.9: e^(0.9^2 / 2)).
    # What is left of O in the sum, 4.6 sqrt(cap / warps) at the most, has either sign and adds less.
    times = 2 if dtype == "fp16" else 1
    cut = cap / 16 * times * 2.0 ** -23 * 7.5 * FOLD / 2 / (4.6 * cap ** 0.5 * 1.5)
    # The scores' errors, as elsewhere (2^-23 of |q| . |k| for each of d / 16 matrix steps and the group sums, 4 |q| . |k|
    # at the most), and bf16 queries' probabilities times steps, rounded to fp16, fall on every token apart: relative to
    # what is left they count as they are
    ds = (d / 16 + 8) * 4 * 2.0 ** -23 * mag
    apart = ds + (0 if dtype == "fp16" else 2.0 ** -11)
    print(f"{dtype} d={d}: rms {(off / n) ** 0.5 / rms:.2e} (bound {cut + apart + EPS[dtype]:.2e}), "
          f"mean {bias / n / rms:.2e} (bound {cut + 6 * (apart + EPS[dtype]) / n ** 0.5:.2e})")
    assert (off / n) ** 0.5 <= (cut + apart + EPS[dtype]) * rms
    # the errors that fall on tokens and on outputs one by one have no sign: their mean over n outputs is within six
    # deviations of 0
    assert abs(bias / n) <= (cut + 6 * (apart + EPS[dtype]) / n ** 0.5) * rms
