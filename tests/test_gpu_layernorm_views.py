"""layer_norm_func on tensors that are dense but begin off a multiple of 16 bytes: slices of flat
buffers, and gradients that autograd hands on as such.  The results are those of copies at
aligned addresses, to the bit."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
M, H = 40, 520


def off_by_one(t):
    """t's values, dense, one element into a buffer."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = flat[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def grads(x, w, b, r, dy, dh, move):
    """y (and h), and the gradients, with the operands named in `move` off by one."""
    at = lambda t, name: off_by_one(t) if name in move else t  # noqa: E731
    leaves = [at(t, n).requires_grad_(True) for t, n in ((x, "x"), (w, "w"), (b, "b"))]
    rr = None if r is None else at(r, "r").requires_grad_(True)
    out = m.layer_norm_func(leaves[0], leaves[1], leaves[2], rr)
    outs = [out] if r is None else list(out)
    g = torch.autograd.grad(outs, leaves + ([] if r is None else [rr]),
                            [at(dy, "dy")] + ([] if r is None else [at(dh, "dh")]))
    return [o.detach() for o in outs] + list(g)


@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("residual", [True, False])
def test_operands_off_an_aligned_address(t, wt, residual):
    gen = torch.Generator(device="cuda").manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy = rn(M, H).to(t), rn(M, H).to(t)
    r, dh = (rn(M, H).to(t), rn(M, H).to(t)) if residual else (None, None)
    w, b = rn(H).to(wt), rn(H).to(wt)
    want = grads(x, w, b, r, dy, dh, ())
    names = ["x", "w", "b", "dy"] + (["r", "dh"] if residual else [])
    for move in [(n,) for n in names] + [tuple(names)]:
        got = grads(x.clone(), w.clone(), b.clone(), None if r is None else r.clone(), dy, dh, move)
        assert len(got) == len(want)
        for a, c in zip(got, want):
            assert torch.equal(a, c), move


def test_gradients_of_flattened_parts():
    # the backward of a cat of flattened tensors hands each a slice of one buffer
    x = torch.randn(M, H, device="cuda").to(BF).requires_grad_(True)
    dy = torch.randn(1 + M * H, device="cuda").to(BF)
    y = m.layer_norm_func(x)
    odd = torch.zeros(1, dtype=BF, device="cuda", requires_grad=True)
    got, = torch.autograd.grad(torch.cat([odd, y.reshape(-1)]), x, dy)
    want, = torch.autograd.grad(m.layer_norm_func(x), x, dy[1:].view(M, H).clone())
    assert torch.equal(got, want)


def test_fused_accumulation_of_a_weight_in_a_flat_buffer():
    x = torch.randn(M, H, device="cuda").to(BF)
    dy = torch.randn(M, H, device="cuda").to(BF)
    w0 = torch.randn(H, device="cuda")
    res = []
    for w in (w0.clone(), off_by_one(w0)):
        w.requires_grad_(True)
        w.main_grad = torch.ones(H, device="cuda")
        m.layer_norm_func(x, w, fuse_grad_accum=True).backward(dy)
        res.append(w.main_grad)
    assert torch.equal(*res) and (res[0] != 1).any()


def test_strided_weights_and_rows():
    x = torch.randn(M, 2 * H, device="cuda").to(BF)
    w = torch.randn(2 * H, device="cuda")
    want = m.layer_norm_func(x[:, ::2].contiguous(), w[::2].contiguous())
    assert torch.equal(m.layer_norm_func(x[:, ::2], w[::2]), want)
