"""The linear layer (and the experts' widths) at the ends of their sizes: more row tiles than a grid's y or z
holds, and more blocks of few rows than SMs (two of them share an SM)."""
import ctypes

import pytest
import torch

import activated_mlp_gemms_gb300 as m
from test_gpu_linear import check

BF = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("M", [16, 48, 160, 200])
def test_more_blocks_than_sms(M):
    check(M, 20488, 264, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("back", [False, True])
def test_more_row_tiles_than_a_grid_dimension(back):
    """16.8 million rows of 896 values to 8 (and dx, from 1408 features to 8): 65537 row
    tiles.  The rows repeat a table's; every result is its table row's."""
    M, K, N = 65536 * 256 + 44, 1408 if back else 896, 8
    gen = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randn((509, K), generator=gen, device="cuda").to(BF)
    at = torch.arange(M, device="cuda") % 509
    x = table[at]
    out = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
    if back:  # dx = dz W, W [896, 8]
        W = (torch.randn((K, N), generator=gen, device="cuda") / 30).to(BF)
        m.mlp_linear_bwd(m.linear(M, K, N), x, None, W, dx=out)
        want = table.double() @ W.double()
    else:
        W = (torch.randn((N, K), generator=gen, device="cuda") / 30).to(BF)
        m.mlp_linear_fwd(m.linear(M, N, K), x, W, None, None, out)
        want = table.double() @ W.double().t()
    # one rounding to bf16, and an fp32 sum of K products
    mag = table.double().abs() @ W.double().abs().reshape(K, N) if back else \
        table.double().abs() @ W.double().abs().t()
    tol = (2.0 ** -8 * want.abs() + K * 2.0 ** -24 * mag).float()
    want = want.float()
    for r in range(0, M, 1 << 22):
        part = slice(r, min(M, r + (1 << 22)))
        assert ((out[part].float() - want[at[part]]).abs() <= tol[at[part]]).all()


def test_sizes_whose_tiles_pass_32_bits_are_refused():
    for kw in (dict(M=0x7fffffff, N=8, K=8), dict(M=1, N=0x7ffffff8, K=8),
               dict(M=1, N=8, K=0x7ffffff8)):
        p = m.linear(**kw)
        assert m.mlp_linear_workspace_size(p) == 0
        assert m.lib().mlp_linear_fwd(ctypes.byref(p), 0x10000, 0x10000, None, None, 0x20000, None,
                                      0x30000, 1 << 40, None) == -3
    for kw in (dict(H=0x7ffffff8, I=8), dict(H=8, I=0x7ffffff8)):
        p = m.moe(1, 1, 1, **kw)
        assert m.mlp_moe_workspace_size(p, m.MODE_FWD) == 0
        assert (m.lib().mlp_moe_rows(ctypes.byref(p)) == 0) == (kw["H"] > 8)


@pytest.mark.gpu
def test_row_strides_past_32_bits_are_refused():
    x = torch.zeros((1 << 32) + 64, dtype=BF, device="cuda").as_strided((2, 64), (1 << 32, 1))
    W, out = torch.zeros((8, 64), dtype=BF, device="cuda"), torch.zeros((2, 8), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="stride"):
        m.mlp_linear_fwd(m.linear(2, 8, 64), x, W, None, None, out)
    with pytest.raises(ValueError, match="stride"):
        m.mlp_linear_bwd(m.linear(2, 8, 64), out, x, W, dW=torch.empty_like(W))
