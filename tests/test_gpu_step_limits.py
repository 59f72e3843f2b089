"""The router, the layer norm and the orthogonalised update where their sizes pass 32 bits, on
threads of their own, captured with their gradients, and with results changed in place.

A row's results (a matrix's) do not depend on the rows beside it, so that the last ones of a
large call are those of a small call on them alone."""
import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TAIL = 40


def test_router_past_32_bits():
    E, k = 1024, 4
    T = (1 << 31) // E + 1000  # the last rows begin past 2^31 values
    x = torch.randn(TAIL, E, device="cuda").to(BF).repeat(T // TAIL + 1, 1)[:T].contiguous()
    p = m.router(T, E, k, logits_dtype=BF)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    bal = torch.empty(E + 1, device="cuda")
    m.mlp_moe_router_fwd(p, x, None, ids, w, counts, bal)
    dw = torch.randn(TAIL, k, device="cuda").repeat(T // TAIL + 1, 1)[:T].contiguous()
    dl = torch.ones(1, device="cuda")
    dx = torch.empty_like(x)
    m.mlp_moe_router_bwd(p, x, None, ids, bal, dw, dl, dx)
    assert int(counts.sum()) == T * k
    q = m.router(TAIL, E, k, logits_dtype=BF)
    ids2, w2, dx2 = torch.empty_like(ids[:TAIL]), torch.empty_like(w[:TAIL]), torch.empty_like(x[:TAIL])
    for rows in (slice(0, TAIL), slice(T - TAIL, T)):
        m.mlp_moe_router_fwd(q, x[rows], None, ids2, w2)
        m.mlp_moe_router_bwd(q, x[rows], None, ids2, bal, dw[rows], dl, dx2)
        assert torch.equal(ids[rows], ids2) and torch.equal(w[rows], w2)
        assert torch.equal(dx[rows], dx2)


def test_layer_norm_past_32_bits():
    H = 8200
    M = (1 << 31) // H + 1000
    x = torch.randn(TAIL, H, device="cuda").to(BF).repeat(M // TAIL + 1, 1)[:M].contiguous()
    w, b = torch.randn(2, H, device="cuda").to(BF)
    p, q = m.layernorm(M, H), m.layernorm(TAIL, H)
    y, h = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(2, M, device="cuda")
    m.mlp_layernorm_fwd(p, x, x, w, b, y, h, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    m.mlp_layernorm_bwd(p, x, h, w, mean, rstd, y, dx, dw, db)
    assert dw.isfinite().all() and db.isfinite().all()
    y2, h2, dx2 = (torch.empty_like(x[:TAIL]) for _ in range(3))
    mean2, rstd2 = torch.empty(2, TAIL, device="cuda")
    for rows in (slice(0, TAIL), slice(M - TAIL, M)):
        xr = x[rows]
        m.mlp_layernorm_fwd(q, xr, xr, w, b, y2, h2, mean2, rstd2)
        m.mlp_layernorm_bwd(q, xr, h2, w, mean2, rstd2, y2, dx2)
        assert torch.equal(y[rows], y2) and torch.equal(h[rows], h2)
        assert torch.equal(mean[rows], mean2) and torch.equal(rstd[rows], rstd2)
        assert torch.equal(dx[rows], dx2)


def test_pitches_past_32_bits():
    pitch, rows = 1 << 21, 1030  # the last rows begin past 2^31 values
    wide = torch.empty(rows, pitch, dtype=BF, device="cuda")
    x = wide[:, 64:320]
    x.copy_(torch.randn(rows, 256, device="cuda"))
    y, y2 = (torch.empty(rows, 256, dtype=BF, device="cuda") for _ in range(2))
    m.mlp_layernorm_fwd(m.layernorm(rows, 256), x, None, None, None, y)
    m.mlp_layernorm_fwd(m.layernorm(rows, 256), x.contiguous(), None, None, None, y2)
    assert torch.equal(y, y2)
    p = m.router(rows, 256, 4, logits_dtype=BF)
    out = [(torch.empty(rows, 4, dtype=torch.int32, device="cuda"),
            torch.empty(rows, 4, device="cuda")) for _ in range(2)]
    dense, dw = x.contiguous(), torch.randn(rows, 4, device="cuda")
    for t, (ids, w) in zip((x, dense), out):
        m.mlp_moe_router_fwd(p, t, None, ids, w)
        m.mlp_moe_router_bwd(p, t, None, ids, None, dw, None, t)  # over the logits
    assert all(torch.equal(a, b) for a, b in zip(*out)) and torch.equal(x, dense)


def test_ortho_past_32_bits():
    m_, n_ = 520, 4096
    batch = (1 << 31) // (m_ * n_) + 4  # the last matrices begin past 2^31 values
    G = torch.randn(4, m_, n_, device="cuda").to(BF).repeat(batch // 4 + 1, 1, 1)[:batch]
    G = G.contiguous()
    out = torch.empty_like(G)
    m.mlp_orthogonalize(m.ortho(m_, n_, batch, steps=2), G, out)
    want = torch.empty_like(G[:4])
    m.mlp_orthogonalize(m.ortho(m_, n_, 4, steps=2), G[:4], want)
    for b in (0, 3, batch - 4, batch - 1):
        # (few matrices share K among CTAs: another order of the same sums)
        d = (out[b].double() - want[b % 4].double()).norm() / want[b % 4].double().norm()
        assert float(d) < 4.5e-3 + 2 * 2.3e-3, b
    assert torch.equal(out[batch - 8:batch - 4], out[batch - 4:])


def test_threads_with_streams_of_their_own():
    """Two host threads run all of the calls at once, without a workspace of theirs."""
    jobs, errors = [], []
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        jobs.append(dict(l=rn(5000, 60), x=rn(900, 1032).to(BF), dy=rn(900, 1032).to(BF),
                         G=rn(3, 264, 520).to(BF), s=rn(64, 512).to(BF)))

    def work(j):
        x = j["x"].detach().requires_grad_(True)
        w = torch.ones(1032, dtype=BF, device="cuda", requires_grad=True)
        l = j["l"].detach().requires_grad_(True)
        ids, wt, counts, loss = m.router_func(l, 4)
        y = m.layer_norm_func(x, w)
        res = [ids, wt, counts, loss, y, *torch.autograd.grad([wt.square().sum() + loss], [l]),
               *torch.autograd.grad(y, [x, w], j["dy"])]
        for G in (j["G"], j["s"]):
            o = torch.empty_like(G)
            m.mlp_orthogonalize(m.ortho(*G.shape[-2:], G.shape[0] if G.dim() == 3 else 1), G, o)
            res.append(o)
        return [r.detach() for r in res]

    want = [work(j) for j in jobs]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                got = [work(jobs[i]) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
            for g in got:
                assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
        except BaseException as e:  # noqa: BLE001  (for the main thread)
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_gradients_in_a_graph():
    """Forward and gradients captured together (no eager graph of the leaves is alive)."""
    l = torch.randn(3000, 64, device="cuda").requires_grad_(True)
    x = torch.randn(800, 2048, device="cuda").to(BF).requires_grad_(True)
    r = torch.randn(800, 2048, device="cuda").to(BF).requires_grad_(True)
    w = torch.randn(2048, device="cuda").requires_grad_(True)

    def step():
        ids, wt, counts, loss = m.router_func(l, 6)
        y, h = m.layer_norm_func(x, w, None, r)
        gl, = torch.autograd.grad(wt.square().sum() + 2 * loss, [l])
        gs = torch.autograd.grad([y, h], [x, r, w], [h.detach(), y.detach()])
        return [t.detach() for t in (ids, wt, counts, loss, y, gl, *gs)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        with torch.no_grad():
            for t in (l, x, r, w):
                t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_results_changed_in_place():
    """The loss and the weights are the caller's: to scale, or to add another layer's to."""
    x = torch.randn(40, 16, device="cuda").requires_grad_(True)
    _, w, _, loss = m.router_func(x, 3)
    want, = torch.autograd.grad(2 * (w * 3).square().sum() + 5 * loss, [x])
    _, w, _, loss = m.router_func(x, 3)
    loss *= 5
    w *= 3
    loss += 2 * w.square().sum()
    got, = torch.autograd.grad(loss, [x])
    assert torch.equal(got, want)


FIRST_CALLS = """
import torch, activated_mlp_gemms_gb300 as m
torch.manual_seed(0)
l, x = torch.randn(3000, 60, device="cuda"), torch.randn(700, 2048, device="cuda").bfloat16()
Gs = [torch.randn(*s, device="cuda") for s in ((64, 512), (520, 264), (1536, 4096), (2, 1032, 1024))]
def calls():
    r = list(m.router_func(l, 4)) + [m.layer_norm_func(x)]
    for G in Gs:
        for t in (torch.bfloat16, torch.float32):
            o = torch.empty_like(G, dtype=t)
            p = m.ortho(*G.shape[-2:], G.shape[0] if G.dim() == 3 else 1, dtype=G.dtype, out_dtype=t)
            m.mlp_orthogonalize(p, G, o)
            r.append(o)
    return r
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, calls()))
print("same")
"""


def test_first_calls_of_a_process_captured():
    """What is set up once (attributes, occupancies) may be set up while a graph is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True,
                       timeout=300, cwd=Path(__file__).resolve().parent.parent)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
