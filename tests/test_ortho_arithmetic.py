"""What the update's accuracy tests rest on, from its arithmetic emulated on the CPU: their bounds
hold for it, and not for it with products left out."""
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
