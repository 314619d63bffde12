"""fp16 queries over the 4-bit cache: what rounding the probabilities times the steps to fp16 loses comes back through a
second matrix product, so O is off by its own rounding, its scores' errors and nothing else."""

import numpy as np
import pytest

from oracle import kv4 as KV
from test_gpu_kv4 import EPS, f64, fa, i32, make_cache  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("nq", [1, 6])  # 2 and 12 rows a head: one and two row tiles
@pytest.mark.parametrize("d", [64, 128, 256])
def test_no_rounding_but_its_own(fa, d, nq):  # noqa: F811
    # a few slots, so that the products' rounding errors do not average out, and short queries, so that the scores' stay small
    lens, cap = [1, 2, 3, 7, 40], 64
    cache, k, v = make_cache(len(lens), 2, cap, d, 80 + d)
    g = torch.Generator().manual_seed(81)
    q = (torch.randn(len(lens), 4, nq, d, generator=g) * 0.02).half()
    scale = d ** -0.5
    o, lse = fa.attention_decode_kv4(q.cuda(), cache, i32(lens), scale=scale)
    fa.fa_check_device_error()
    ro, rl, _, mag = KV.decode64(f64(q), k, v, lens, scale, False)
    ds = (d / 16 + 8) * 4 * 2.0 ** -23 * mag + 2.0 ** -20  # as for every decode: scores and exponentials in fp32
    # Numerator and sum carry the scores' errors.  Sums of codes up to 15 steps (up to 4 times the largest value) are cut by
    # 2^-23 in at most 3 matrix steps of 16 slots and the second operand's 3; a product of a probability and a step is off
    # by 2^-22; the offset's and middles' sums are rounded for every slot.
    vmax = np.abs(v).max()
    tol = (vmax * (2 * ds + 4 * (6 * 2.0 ** -23 + 2.0 ** -22) + max(lens) * 2.0 ** -24))[..., None] + EPS["fp16"] * np.abs(
        ro) + 2.0 ** -25
    worst = (np.abs(f64(o) - ro) / tol).max()
    print(f"d={d}: {worst:.2f} of the bound; a rounding of the products by 2^-11 would be up to "
          f"{(vmax * 2.0 ** -11 / tol).max():.0f} of it")
    assert worst <= 1
