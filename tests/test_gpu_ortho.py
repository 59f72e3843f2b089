"""The orthogonalised update against its formula in 64 bits.

Tolerances, relative in the Frobenius norm.  X carries 22 bits, and with the leading fp16 terms
a product's operands are off by 2^-11 at most, 2^-11 / sqrt(3) in the mean square; a step has
three such products (X X^T, A A, P X) with factors that the polynomial bounds, and what they
add to singular values near one is contracted by the next.  Emulated in 64 bits over spectra
from flat to rank one the result is off by 4.1e-3 (8 x 8) down to 1.3e-3 (1024 x 1024; the bound
here is 4.5e-3), and a bf16 result rounds by 2^-8 / sqrt(3) = 2.3e-3 beside it; with both terms
the emulation is off by 2.9e-5 at most, the fp32 sums over K add sqrt(K) 2^-24 a product,
stretched by at most 3.45^4 (the bound here is 1e-4)."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 4.5e-3 + 2.3e-3, F32: 1e-4}


def plain(G, steps=5, coeffs=m.MUON_COEFFS, eps=1e-7, scale=1.0):
    a, b, c = coeffs
    X = G.double()
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.transpose(-2, -1)
    for _ in range(steps):
        A = X @ X.transpose(-2, -1)
        X = a * X + (b * A + c * A @ A) @ X
    return scale * (X.transpose(-2, -1) if tall else X)


def run(G, out_dtype=BF, **kw):
    shape = G.shape if G.dim() == 3 else (1,) + G.shape
    p = m.ortho(shape[1], shape[2], shape[0], dtype=G.dtype, out_dtype=out_dtype, **kw)
    out = torch.full(G.shape, 7.0, dtype=out_dtype, device="cuda")
    ws = m.mlp_orthogonalize(p, G, out)
    assert m.mlp_device_status(ws) == 0
    return out


def off(got, ref):
    d = (got.double() - ref).flatten(-2).norm(dim=-1) / ref.flatten(-2).norm(dim=-1)
    return float(d.max())


def check(G, out_dtype=BF, more=0.0, **kw):
    got = run(G, out_dtype, **kw)
    e = off(got, plain(G, **kw))
    assert e <= TOL[out_dtype] + more, e
    return got


def rank_one(m_, n_):
    """What fp32 sums cost where every other singular value is zero: the tensor cores truncate
    the accumulator once an instruction (16 of K), by 2^-23 of it at most, so A is off by n / 16
    2^-23 of itself, A A by twice that and m / 16 2^-23, P X by m / 16 2^-23 and P's own error;
    with |b|, c and |P| <= 2.8 of the first step, all of it stretched by 3.45 four times.
    (The formula in fp32 on CUDA cores is off by 1.9e-4 at 512 x 1408, measured; the library
    by 1.2e-4.)"""
    first = (4.775 + 2 * 2.0315) * n_ + (2.0315 + 2.8) * m_
    return 3.45 ** 4 * first / 16 * 2.0 ** -23


def make(*shape, dtype=F32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return (1e-3 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


SIZES = [(8, 8), (8, 1000), (1000, 8), (64, 64), (72, 136), (128, 128), (136, 128), (264, 248),
         (256, 2048), (2048, 256), (520, 520), (352, 256), (1032, 1024), (776, 2056), (1408, 2048),
         (2048, 1408), (1536, 1536), (2304, 2320),
         (64, 4104), (264, 8200), (8200, 136), (128, 2048), (2048, 120), (120, 1032), (24, 264),
         (1024, 128), (16, 520), (8, 2048)]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, dtype, out_dtype):
    check(make(rows, cols, dtype=dtype), out_dtype)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("batch,rows,cols", [(3, 8, 8), (5, 136, 264), (8, 352, 256),
                                             (16, 256, 352), (2, 1408, 1024), (4, 1032, 520),
                                             (30, 64, 1024), (41, 2048, 40)])
def test_stacks(batch, rows, cols, out_dtype):
    G = make(batch, rows, cols)
    G *= torch.logspace(-3, 3, batch, device="cuda")[:, None, None]  # each by its own norm
    check(G, out_dtype)
    # a matrix does not depend on its neighbours: to the bit where the sums over K are not shared
    # out (how they are goes by the number of tiles in the stack)
    m.mlp_set_tile_policy(1)
    try:
        assert torch.equal(run(G, out_dtype)[-1], run(G[-1].contiguous(), out_dtype))
    finally:
        m.mlp_set_tile_policy(0)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("tile_policy", [1, 2])
@pytest.mark.parametrize("rows,cols", [(8, 264), (520, 776), (1032, 520), (1536, 2048)])
def test_tile_policies(rows, cols, tile_policy, out_dtype):
    m.mlp_set_tile_policy(tile_policy)
    try:
        check(make(rows, cols), out_dtype)
        check(make(3, rows, cols), out_dtype)
    finally:
        m.mlp_set_tile_policy(0)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(512, 512), (512, 1408), (1408, 512), (128, 512),
                                       (1024, 96)])
def test_spectra(rows, cols, out_dtype):
    """Singular values down to 1e-4 of the largest, and a few strong directions over noise (what
    momenta look like): in bf16 terms alone these are off by 5-30 %."""
    m_, n_ = min(rows, cols), max(rows, cols)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    U, V = torch.linalg.qr(rn(m_, m_))[0], torch.linalg.qr(rn(n_, m_))[0]
    log = (U * torch.logspace(0, -4, m_, device="cuda", dtype=torch.float64)) @ V.t()
    low = rn(m_, 8) @ rn(8, n_) + 1e-2 * rn(m_, n_)
    one = rn(m_, 1) @ rn(1, n_)
    for G, more in ((log, 0.0), (low, 0.0), (one, rank_one(m_, n_))):
        G = (G if rows <= cols else G.t()).float().contiguous()
        check(G, out_dtype, more if out_dtype == F32 else 0.0)


def test_steps_coefficients_and_scale():
    G = make(200, 304)
    for kw in (dict(steps=1), dict(steps=2), dict(steps=9), dict(coeffs=(1.5, -0.5, 0.0), steps=12),
               dict(coeffs=(2.0, -1.5, 0.5), steps=7), dict(scale=0.2), dict(scale=-3.0, steps=4),
               dict(eps=0.5)):
        check(G, F32, **kw)
        check(G, BF, **kw)


def test_a_converged_iteration_is_orthogonal():
    # X (3 X - X^3) / 2 converges to the orthogonal factor itself
    G = make(192, 320)
    out = run(G, F32, coeffs=(1.5, -0.5, 0.0), steps=32).double()
    eye = torch.eye(192, dtype=torch.float64, device="cuda")
    assert (out @ out.t() - eye).abs().max() < 1e-5
    U, _, Vt = torch.linalg.svd(G.double(), full_matrices=False)
    assert off(out, U @ Vt) < 1e-4


@pytest.mark.parametrize("size", [1e-15, 1e-6, 1.0, 1e4, 1e15])
def test_magnitudes(size):
    # the result does not depend on G's size but through eps
    G = make(136, 264) * 1e3 * size
    check(G, F32, eps=0.0)
    check(G, BF, eps=1e-7)


def test_zero_and_nan():
    G = make(3, 136, 136)
    G[1] = 0
    clean = run(G, F32)
    assert not clean[1].any()
    G[2, 5, 7] = float("nan")
    got = run(G, F32)
    assert torch.equal(got[:2], clean[:2]) and got[2].isnan().all()
    G[2, 5, 7] = float("inf")
    assert run(G, F32)[2].isnan().any()


def test_uneven_rows():
    # an embedding's update: most rows are hardly ever touched
    G = make(520, 512)
    G[::3] *= 1e-5
    G[1::3] = 0
    ref = plain(G)
    got = run(G, F32)
    assert off(got, ref) < TOL[F32] and not got[1::3].any()
    assert off(run(G, BF), ref) < TOL[BF]


def test_in_place_and_guarded():
    for dtype in (BF, F32):
        G = make(2, 264, 136, dtype=dtype)
        want = run(G, dtype)
        p = m.ortho(264, 136, 2, dtype=dtype, out_dtype=dtype)
        room = torch.full((2 * 264 * 136 + 64,), 3.0, dtype=dtype, device="cuda")
        H = room[32:-32].view(2, 264, 136)
        H.copy_(G)
        m.mlp_orthogonalize(p, H, H)
        assert torch.equal(H, want)
        assert (room[:32] == 3).all() and (room[-32:] == 3).all()
    # the workspace is not written past its end
    p = m.ortho(264, 136, 2)
    n = m.mlp_ortho_workspace_size(p)
    ws = torch.full((n + 512,), 9, dtype=torch.uint8, device="cuda")
    m.mlp_orthogonalize(p, make(2, 264, 136, dtype=BF), torch.empty(2, 264, 136, dtype=BF,
                                                                    device="cuda"), ws=ws[:n])
    assert (ws[n:] == 9).all()


def test_same_bits_graphs_and_streams():
    G = make(4, 352, 256)
    p = m.ortho(352, 256, 4, dtype=F32, out_dtype=BF)
    ws = m.alloc_ortho_workspace(p)
    want, out = run(G), torch.empty(4, 352, 256, dtype=BF, device="cuda")
    m.mlp_orthogonalize(p, G, out, ws=ws)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mlp_orthogonalize(p, G, out, ws=ws)
    for s in (1, 2):
        G.copy_(make(4, 352, 256, seed=s))
        out.zero_()
        graph.replay()
        got = out.clone()
        assert torch.equal(got, run(G))
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    m.mlp_orthogonalize(p, G, out, stream=side)
    side.synchronize()
    assert torch.equal(out, got)


def test_refusals():
    G = make(64, 64)
    p = m.ortho(64, 64)
    o = torch.empty(64, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):  # not bf16
        m.mlp_orthogonalize(p, G, o)
    with pytest.raises(ValueError):
        m.mlp_orthogonalize(p, o[:32], o)
    with pytest.raises(ValueError):
        m.mlp_orthogonalize(p, o.t()[:, :], o.t()[:, ::2])
    with pytest.raises(m.MlpError):
        q = m.ortho(60, 64)
        m.mlp_orthogonalize(q, o[:60], o[:60].clone())
    with pytest.raises(m.MlpError):
        m.mlp_orthogonalize(p, o, o.clone(), ws=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_bounded_waits():
    """Without loads every wait runs out: the status says so and the next call works."""
    for size, policy in ((520, 0), (520, 1), (520, 2), (104, 0)):
        # (0: K shared by clusters; the whole call on one)
        G = make(size, size)
        want = run(G)
        p = m.ortho(size, size, dtype=F32)
        out = torch.empty(size, size, dtype=BF, device="cuda")
        m.mlp_set_tile_policy(policy)
        m.mlp_set_wait_timeout_ms(20)
        m.mlp_debug_set_flags(m.DEBUG_NO_WORK)
        try:
            ws = m.mlp_orthogonalize(p, G, out, ws=m.alloc_ortho_workspace(p))
            assert m.mlp_device_status(ws) == -6
        finally:
            m.mlp_debug_set_flags(0)
            m.mlp_set_wait_timeout_ms(0)
            m.mlp_set_tile_policy(0)
        assert torch.equal(run(G), want)


@pytest.mark.parametrize("batch,rows,cols,out_dtype", [
    (1, 1536, 8200, BF), (1, 8200, 1288, BF), (1, 2048, 4872, F32), (1, 1544, 2568, F32),
    (3, 1000, 4104, F32), (2, 1032, 14336, BF)])
def test_long_rows_shared_by_pairs(batch, rows, cols, out_dtype):
    """X X^T of few large tiles over a long K (two CTA pairs a tile), odd halves of it too."""
    G = make(batch, rows, cols, dtype=BF if out_dtype == BF else F32)
    got = check(G, out_dtype)
    assert torch.equal(got, run(G, out_dtype))


def test_bounded_waits_of_pairs():
    G = make(1536, 8192, dtype=BF)
    want = run(G)
    out = torch.empty_like(want)
    m.mlp_set_wait_timeout_ms(20)
    m.mlp_debug_set_flags(m.DEBUG_NO_WORK)
    try:
        p = m.ortho(1536, 8192)
        ws = m.mlp_orthogonalize(p, G, out, ws=m.alloc_ortho_workspace(p))
        assert m.mlp_device_status(ws) == -6
    finally:
        m.mlp_debug_set_flags(0)
        m.mlp_set_wait_timeout_ms(0)
    assert torch.equal(run(G), want)
