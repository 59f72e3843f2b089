"""The sort of slots by expert, the dispatch, the combine and their gradients
against a plain fp64 implementation.

Tolerances: the sorted layout and the copied rows are exact.  A bf16 output is
an fp32 sum rounded once: the unit roundoff of bf16's 8-bit significand (2^-8 of
the value) plus the fp32 summation error, at most (terms) * 2^-24 of the sum
of magnitudes.  dweights
in fp32 sums H products in some order: H * 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def plain_plan(ids, E):
    """(offsets, counts, pos, src) by walking the slots expert by expert."""
    T, k = ids.shape
    n = T * k
    rows = (n + min(E, n) * 15) // 16 * 16
    offsets, counts = [0], []
    pos, src = np.full((T, k), -1, np.int32), np.full(rows, -1, np.int32)
    at = 0
    for e in range(E):
        slots = np.flatnonzero(ids.reshape(-1) == e)
        src[at:at + len(slots)] = slots
        pos.reshape(-1)[slots] = at + np.arange(len(slots))
        counts.append(len(slots))
        at += (len(slots) + 15) // 16 * 16
        offsets.append(at)
    return np.array(offsets), np.array(counts), pos, src


def make_ids(kind, T, E, k, rng):
    if kind == "random":
        return rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one":  # every slot to the last expert
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":  # every slot dropped
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)  # dropped slots, and whole tokens
    ids[rng.random((T, k)) < 0.3] = -1
    ids[rng.random(T) < 0.2] = E + 5
    return ids


SHAPES = [(1, 1, 1, 8), (1, 64, 8, 256), (3, 5, 2, 24), (17, 64, 8, 1032), (129, 8, 2, 2048),
          (700, 7, 3, 512), (2049, 60, 4, 64), (4099, 1024, 8, 16), (20000, 3, 8, 8)]


@pytest.mark.parametrize("kind", ["random", "one", "none", "dropped"])
@pytest.mark.parametrize("T,E,k,H", SHAPES)
def test_plan(T, E, k, H, kind):
    ids = make_ids(kind, T, E, k, np.random.default_rng(T + E))
    p = m.moe(T, E, k, H)
    plan = m.alloc_moe_plan(p)
    plan.fill_(-7)
    m.mlp_moe_sort(p, torch.from_numpy(ids).cuda(), plan)
    got = {n: v.cpu().numpy() for n, v in m.moe_plan_views(p, plan).items()}
    offsets, counts, pos, src = plain_plan(ids, E)
    assert np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["counts"], counts)
    assert np.array_equal(got["pos"], pos)
    assert np.array_equal(got["src"], src)


def near(got, ref, mag, terms):
    """|got - ref| within the unit roundoff of got's type plus an fp32 sum's error."""
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = step * ref.abs() + terms * 2.0 ** -24 * mag + 1e-38
    assert ((got.double().cpu() - ref).abs() <= tol * 1.001).all()


@pytest.mark.parametrize("wdt", [torch.float32, BF])
@pytest.mark.parametrize("kind", ["random", "one", "none", "dropped"])
@pytest.mark.parametrize("T,E,k,H", SHAPES[:7])
def test_rows_there_and_back(T, E, k, H, kind, wdt):
    rng = np.random.default_rng(T * 7 + E)
    gen = torch.Generator().manual_seed(T + H)
    ids = make_ids(kind, T, E, k, rng)
    _, _, pos, src = plain_plan(ids, E)
    pos, src = torch.from_numpy(pos).long(), torch.from_numpy(src).long()
    rows = len(src)
    rn = lambda *s: torch.randn(s, generator=gen).to(BF)  # noqa: E731
    x, r, dout, y, dxs = rn(T, H), rn(T, H), rn(T, H), rn(rows, H), rn(rows, H)
    w = torch.rand((T, k), generator=gen).to(wdt)
    y[src < 0] = float("inf")  # never read
    p = m.moe(T, E, k, H, weights_dtype=wdt)
    assert m.mlp_moe_rows(p) == rows
    plan = m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, torch.from_numpy(ids).cuda(), plan)
    nan = lambda *s, dt=BF: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731

    xs = nan(rows, H)
    m.mlp_moe_dispatch(p, plan, x.cuda(), xs)
    want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k], torch.zeros(1, dtype=BF))
    assert torch.equal(xs.cpu(), want)

    have = (pos >= 0).double()[..., None]
    picked = torch.where(have > 0, y.double()[pos.clamp(min=0)], 0.0)
    wd = w.double()[..., None]
    for res in (None, r):
        out = nan(T, H)
        m.mlp_moe_combine(p, plan, y.cuda(), w.cuda(), None if res is None else res.cuda(), out)
        base = torch.zeros(T, H, dtype=torch.float64) if res is None else res.double()
        near(out, base + (wd * picked).sum(1), base.abs() + (wd * picked).abs().sum(1), 2 * k + 1)
    same = r.cuda()
    m.mlp_moe_combine(p, plan, y.cuda(), w.cuda(), same, same)  # in place over the residual
    assert torch.equal(same, out)

    dx = nan(T, H)
    m.mlp_moe_dispatch_bwd(p, plan, dxs.cuda(), dx)
    back = dxs.double()[pos.clamp(min=0)] * have
    near(dx, back.sum(1), back.abs().sum(1), k)

    dy, dw = nan(rows, H), nan(T, k, dt=wdt)
    m.mlp_moe_combine_bwd(p, plan, dout.cuda(), y.cuda(), w.cuda(), dy, dw)
    ref = torch.where((src >= 0)[:, None],
                      w.double().reshape(-1)[src.clamp(min=0)][:, None]
                      * dout.double()[src.clamp(min=0) // k], 0.0)
    near(dy, ref, ref.abs(), 2)
    terms = dout.double()[:, None] * picked
    near(dw, terms.sum(2), terms.abs().sum(2), H + 8)
    # each alone gives the same bits
    dy2, dw2 = nan(rows, H), nan(T, k, dt=wdt)
    m.mlp_moe_combine_bwd(p, plan, dout.cuda(), None, w.cuda(), dy2, None)
    m.mlp_moe_combine_bwd(p, plan, dout.cuda(), y.cuda(), None, None, dw2)
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


def test_weights_gradient_against_differences():
    """The combine is linear in the weights: a step of one weight changes
    <dout, out> by that step times its gradient."""
    T, E, k, H = 9, 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    ids = torch.randint(0, E, (T, k), generator=gen, dtype=torch.int32).cuda()
    p = m.moe(T, E, k, H)
    plan = m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, ids, plan)
    rows = m.mlp_moe_rows(p)
    # small integers: every product and sum below is exact in bf16 or fp32
    y = torch.randint(-3, 4, (rows, H), generator=gen).to(BF).cuda()
    dout = torch.randint(-2, 3, (T, H), generator=gen).to(BF).cuda()
    w = torch.randint(0, 4, (T, k), generator=gen).float().cuda()
    dw = torch.empty_like(w)
    m.mlp_moe_combine_bwd(p, plan, dout, y, w, None, dw)

    def loss(weights):
        out = torch.empty((T, H), dtype=BF, device="cuda")
        m.mlp_moe_combine(p, plan, y, weights, None, out)
        return (out.double() * dout.double()).sum()

    for t in range(T):
        for j in range(k):
            step = w.clone()
            step[t, j] += 1
            assert (loss(step) - loss(w)).item() == dw[t, j].item()


def test_bf16_weights_at_an_odd_address():
    # rows of an odd number of bf16 weights: the same bits as from an aligned copy
    T, E, k, H, I = 7, 4, 3, 64, 128
    gen = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=gen).to(BF).cuda()  # noqa: E731
    p = m.moe(T, E, k, H, I, weights_dtype=BF)
    w = rn(T + 1, k)[1:]
    assert w.data_ptr() % 4 == 2 and w.is_contiguous()
    ids = torch.randint(0, E, (T, k), generator=gen, dtype=torch.int32).cuda()
    rows, plan = m.mlp_moe_rows(p), m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, ids, plan)
    x, y, dout = rn(T, H), rn(rows, H), rn(T, H)
    Wg, Wu, Wd = rn(E, I, H), rn(E, I, H), rn(E, H, I)
    res = []
    for v, dw in ((w, torch.zeros(T + 1, k, dtype=BF, device="cuda")[1:]),
                  (w.clone(), torch.zeros(T, k, dtype=BF, device="cuda"))):
        out, lay, dy = torch.empty_like(x), torch.empty_like(x), torch.empty_like(y)
        m.mlp_moe_combine(p, plan, y, v, None, out)
        m.mlp_moe_combine_bwd(p, plan, dout, y, v, dy, dw)
        m.mlp_moe_fwd_infer(p, x, ids, v, Wg, Wu, Wd, None, lay)
        res.append((out, dy, dw, lay))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_another_stream_and_repeat():
    """On a side stream the calls order with the work there, and give the same bits again."""
    T, E, k, H = 4099, 16, 4, 512
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, device="cuda")
    p = m.moe(T, E, k, H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(s):
        for _ in range(2):
            x = torch.zeros(T, H, device="cuda")
            x = (x + torch.arange(H, device="cuda")).to(BF)
            plan = m.alloc_moe_plan(p)
            xs = torch.empty((m.mlp_moe_rows(p), H), dtype=BF, device="cuda")
            out = torch.empty((T, H), dtype=BF, device="cuda")
            m.mlp_moe_sort(p, ids, plan)
            m.mlp_moe_dispatch(p, plan, x, xs)
            m.mlp_moe_combine(p, plan, xs, w, None, out)
            outs.append((plan, out))
    s.synchronize()
    assert torch.equal(outs[0][1], outs[1][1])
    for a, b in zip(m.moe_plan_views(p, outs[0][0]).values(),
                    m.moe_plan_views(p, outs[1][0]).values()):
        assert torch.equal(a, b)
    ref = (x.double() * w.double().sum(1, keepdim=True))
    assert ((outs[0][1].double() - ref).abs() <= 2.0 ** -8 * ref.abs()).all()
