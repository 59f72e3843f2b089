"""What the update's accuracy tests rest on, from its arithmetic emulated on the CPU: their bounds
hold for it, and not for it with products left out."""
import math

import pytest
import torch
from ortho_arithmetic import emulate, momentum, off, plain

# A bf16 result of up to 128 rows, relative in the Frobenius norm: rounding it is 1.7e-3 (2^-9 of
# a value's binade: 2^-9 sqrt(E[1 / m^2]) = 1.4e-3 to 2.0e-3 by the mantissas m, 1.66e-3 where they
# are spread out), X X^T and A A of leading terms 0.3e-3 to 1.0e-3 beside it.  Leading terms in P X
# add 1.2e-3 to 2.1e-3.
BF16_128 = 2.2e-3


def noise(M, N, gen):
    return torch.randn(M, N, generator=gen)


@pytest.mark.parametrize("make,rows,cols", [(momentum, 64, 512), (momentum, 96, 520),
                                            (momentum, 128, 768), (noise, 64, 512),
                                            (noise, 128, 512)])
def test_bf16_up_to_128_rows(make, rows, cols):
    G = make(rows, cols, torch.Generator().manual_seed(rows + cols))
    ref = plain(G)
    assert 1.5e-3 < off(ref.bfloat16(), ref) < 1.8e-3
    assert off(emulate(G, False, True), ref) < BF16_128 < off(emulate(G, False, False), ref)


def rank_one_bound(m):
    """What an fp32 result of m rows is off by where every other singular value is zero: noise
    beside the one direction grows by a = 3.45 a step.  In the mean square, relative to X:
    rounding X to two terms, 2^-22 / 3 (two roundings of 2^-11 / sqrt(3)), at the start and after
    each step but the last: 3.45 + ... + 3.45^5 = 688 of it remain.  The sums of P X, |P| <= 2.8
    times a chain of n instructions of 16 products (32 at most, then added up rounded to nearest),
    each truncated by a part, evenly spread, of 2^-23 at most of what has come together: n / 36
    in the square, and 0.07 n / 2 for what the mean of it, half a last bit, differs by from one
    mantissa to another; 1 + ... + 3.45^4 = 199 of it remain.  (The error of A reaches the noise
    along the one direction alone, 1 / sqrt(m) of it.)  Times 1.5, for X's norm of up to 1.2."""
    x = 688 * 2.0 ** -22 / 3
    n = min((m + 15) // 16, 32)
    p = 199 * 2.8 * 2.0 ** -23 * math.sqrt(n / 36 + (0.07 * n / 2) ** 2)
    return 1.5 * math.hypot(x, p)


@pytest.mark.parametrize("rows,cols", [(64, 512), (128, 512), (256, 512), (512, 520)])
def test_rank_one(rows, cols):
    gen = torch.Generator().manual_seed(rows)
    G = torch.randn(rows, 1, generator=gen) @ torch.randn(1, cols, generator=gen)
    ref = plain(G)
    assert off(emulate(G, True, True), ref) < rank_one_bound(rows)
    assert off(emulate(G, True, True, both=False), ref) > 1.3 * rank_one_bound(rows)
