"""The workspaces that the Python calls allocate by themselves, on other streams and
from several host threads."""
import gc
import threading

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def layer(seed, T=300, E=8, k=2, H=256, inner=512):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)  # noqa: E731
    p = m.moe(T, E, k, H, inner)
    x, Ws = rn(T, H), (rn(E, inner, H) / 16, rn(E, inner, H) / 16, rn(E, H, inner) / 23)
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, -1)[1].int()
    w = torch.rand(T, k, generator=gen, device="cuda")
    n = m.mlp_moe_workspace_size(p, m.MODE_INFER)
    return n, lambda out, **kw: m.mlp_moe_fwd_infer(p, x, ids, w, *Ws, None, out, **kw), x


def dense(seed, M=300, H=256, inner=512):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)  # noqa: E731
    p = m.problem(M, H, inner, "swiglu", 1.0, 1.0)
    x, Ws = rn(M, H), (rn(inner, H) / 16, rn(inner, H) / 16, rn(H, inner) / 23)
    n = m.mlp_workspace_size(p, m.MODE_INFER)
    return n, lambda out, **kw: m.mlp_fwd_infer(p, x, *Ws, out, **kw), x


@pytest.mark.parametrize("make", [layer, dense])
def test_memory_that_the_current_stream_still_reads(make):
    # temporaries of the call's size are freed on the current stream, where a copy of
    # them still waits: the call on another stream must get other memory
    n, call, x = make(5)
    want, got = torch.empty_like(x), torch.zeros_like(x)
    call(want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    other = torch.cuda.Stream()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    kept = [t.clone() for t in held]
    del held
    call(got, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((t == 7).all()) for t in kept)


def small(seed):
    """A linear forward and backward whose workspaces are small enough to be kept."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: (torch.randn(s, generator=gen, device="cuda") / 8).to(BF)  # noqa: E731
    M, N, K = 40 + seed, 264, 136
    p, x, W, b, dout = m.linear(M, N, K, "silu"), rn(M, K), rn(N, K), rn(N), rn(M, N)

    def run():
        out, pre = torch.empty_like(dout), torch.empty_like(dout)
        dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty_like(b)
        m.mlp_linear_fwd(p, x, W, b, None, out, pre)
        m.mlp_linear_bwd(p, dout, x, W, pre, dx, dW, db)
        return out, dx, dW, db

    return run


def test_threads_and_streams_do_not_share():
    jobs = [small(i) for i in range(4)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(4)

    def work(i):
        try:
            streams = [torch.cuda.Stream(), torch.cuda.Stream()]
            start.wait()
            for n in range(200):
                with torch.cuda.stream(streams[n & 1]):
                    got = jobs[i]()
                if n % 20 == 0:
                    torch.cuda.synchronize()
                    bad.extend((i, n, k) for k, (a, b) in enumerate(zip(got, want[i]))
                               if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001 (shown below)
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_a_thread_s_workspaces_go_with_it():
    small(0)()
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            small(1)()

    for _ in range(8):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    gc.collect()
    assert torch.cuda.memory_allocated() <= before
