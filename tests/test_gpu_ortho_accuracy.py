"""The orthogonalised update's accuracy by the way that a matrix goes (its bounds:
test_ortho_arithmetic.py)."""
import pytest
import torch
from ortho_arithmetic import momentum, off, plain
from test_ortho_arithmetic import BF16_128, rank_one_bound

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def noise(M, N, gen, device="cuda"):
    return torch.randn(M, N, generator=gen, device=device)


def stack(make, batch, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(batch + rows + cols)
    return torch.stack([make(rows, cols, gen, "cuda") for _ in range(batch)])


def run(G, out_dtype):
    out = torch.full(G.shape, 7.0, dtype=out_dtype, device="cuda")
    p = m.ortho(G.shape[1], G.shape[2], G.shape[0], dtype=G.dtype, out_dtype=out_dtype)
    ws = m.mlp_orthogonalize(p, G, out)
    assert m.mlp_device_status(ws) == 0
    return out


def worst(got, G):
    return max(off(a, plain(g)) for a, g in zip(got, G))


@pytest.mark.parametrize("make", [momentum, noise])
# (one launch; more columns than it takes, just above them too; stacks too large for it)
@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 2048), (1, 128, 2048), (1, 128, 2056),
                                             (1, 64, 4096), (1, 120, 8192), (1, 4104, 104),
                                             (15, 128, 1024), (16, 128, 2048), (20, 2048, 128),
                                             (40, 64, 1024), (61, 72, 264)])
def test_bf16_up_to_128_rows(make, batch, rows, cols):
    G = stack(make, batch, rows, cols)
    e = worst(run(G, BF), G)
    assert e < BF16_128, e


@pytest.mark.parametrize("policy", [1, 2])
@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 512), (3, 128, 1032), (200, 72, 136)])
def test_bf16_up_to_128_rows_by_tile_policy(batch, rows, cols, policy):
    G = stack(momentum, batch, rows, cols)
    want = run(G, BF)
    m.mlp_set_tile_policy(policy)
    try:
        got = run(G, BF)
        again = run(G, BF)
    finally:
        m.mlp_set_tile_policy(0)
    assert torch.equal(got, again)
    assert worst(got, G) < BF16_128 and worst(want, G) < BF16_128


def test_without_the_linear_term():
    # b = 0: P = c A A has nothing to add, and its second term is stored over A all the same
    G = stack(momentum, 3, 96, 4096)
    out = torch.empty(G.shape, dtype=F32, device="cuda")
    coeffs = (1.5, 0.0, -0.3)
    got = {}
    for t in (BF, F32):
        out = torch.empty(G.shape, dtype=t, device="cuda")
        m.mlp_orthogonalize(m.ortho(96, 4096, 3, coeffs=coeffs, dtype=F32, out_dtype=t), G, out)
        got[t] = out.double()
    for g, a, c in zip(G, got[BF], got[F32]):
        a0, _, c0 = coeffs
        X = g.double() / (g.double().norm() + 1e-7)
        for _ in range(5):
            A = X @ X.t()
            X = a0 * X + c0 * (A @ A) @ X
        assert off(a, X) < BF16_128 and off(c, X) < 1e-4


@pytest.mark.parametrize("rows,cols", [(64, 512), (96, 1024), (1024, 96), (128, 4096), (136, 4152),
                                       (256, 2048), (512, 512), (512, 1408), (1408, 512),
                                       (1408, 2048), (2048, 4872)])
def test_fp32_of_rank_one(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    G = (rn(1, rows, 1) @ rn(1, 1, cols)).float()
    e = worst(run(G, F32), G)
    assert e < rank_one_bound(min(rows, cols)), e


# An fp32 result of 129 to 512 rows.  Emulated on the CPU with sums truncated to 24 bits twice an
# instruction (every 8 products), chunks of one and two k-blocks (64 of K) leave 1.0e-6 to 1.4e-6 at
# 136 x 512 to 512 x 512; twice that.  (Chunks of four and eight: measured up to 7.6e-6.)
FP32_512 = 2.8e-6


@pytest.mark.parametrize("make", [momentum, noise])
@pytest.mark.parametrize("batch,rows,cols", [(1, 136, 1024), (1, 136, 4152), (1, 256, 512),
                                             (1, 256, 14336), (1, 2048, 256), (1, 304, 1000),
                                             (1, 320, 6000), (4, 512, 1408), (1, 512, 8192),
                                             (20, 264, 264)])
def test_fp32_of_129_to_512_rows(make, batch, rows, cols):
    G = stack(make, batch, rows, cols)
    e = worst(run(G, F32), G)
    assert e < FP32_512, e


# One launch, momenta: sums of two instructions leave 0.7e-6 to 0.8e-6 by the same emulation; two and
# a half times that, for the sums over the CTAs and what an instruction truncates inside.  (Sums of
# eight instructions: measured 1.9e-6 at 64 x 1024, 2.7e-6 to 3.6e-6 from 96 x 1024.)
FP32_ONE_LAUNCH = 2.0e-6


@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 64), (1, 64, 1024), (1, 96, 1024),
                                             (1, 1024, 128), (1, 128, 512), (10, 128, 768)])
def test_fp32_in_one_launch(batch, rows, cols):
    G = stack(momentum, batch, rows, cols)
    e = worst(run(G, F32), G)
    assert e < FP32_ONE_LAUNCH, e


# A bf16 result of more than 128 rows: leading terms in P X.  Emulated, 2.0e-3 to 2.6e-3 for momenta
# and noise of 136 x 1024 to 512 x 512, of which rounding is 1.7e-3; a quarter more, for what single
# matrices differ by.
BF16_ABOVE = 3.3e-3


@pytest.mark.parametrize("make", [momentum, noise])
@pytest.mark.parametrize("batch,rows,cols", [(1, 136, 1024), (1, 136, 4152), (1, 256, 2048),
                                             (1, 512, 512), (4, 1032, 520), (1, 1408, 2048),
                                             (2, 2056, 1536)])
def test_bf16_above_128_rows(make, batch, rows, cols):
    G = stack(make, batch, rows, cols)
    e = worst(run(G, BF), G)
    assert e < BF16_ABOVE, e
