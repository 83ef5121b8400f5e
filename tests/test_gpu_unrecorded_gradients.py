"""Calls that record no gradient refuse tensors that ask for one, instead of returning results that have lost it; under
no_grad they run, and so do tensors that carry no tangent inside a forward-mode context."""

import pytest
import torch
from torch.autograd import forward_ad

import nvfp4_block_scaled_mm_b200 as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32
T, K, E, H = 20, 2, 4, 256


def setup(dtype=BF):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).to(DEV)
    return x, ids, torch.rand(T, K, generator=g).to(DEV)


def calls():
    """(name of the argument that may ask for a gradient, that tensor, the call)"""
    x, ids, w = setup()
    one = torch.ones(H, dtype=BF, device=DEV)
    q, s = L.fp8_quantize(x)
    b, bs = L.fp8_quantize(torch.ones(H, H, dtype=BF, device=DEV), block_rows=128)
    bias, out, res, norm = one.clone(), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    s2 = torch.zeros(T, 2, device=DEV)
    p = L.moe_permute(x, ids, E)
    rows, rows2, gx, back = p.rows.clone(), p.rows.clone(), torch.zeros_like(x), torch.zeros_like(x)
    c = x.clone()
    yield "x", x, lambda: L.fp8_quantize(x)
    yield "scales", s2, lambda: L.fp8_quantize(c, scales=s2)
    for name, t in (("x", x), ("weight", one), ("residual", res), ("norm_out", norm)):
        yield name, t, lambda: L.add_rmsnorm_fp8_quantize(x, one, res, norm_out=norm)
    for name, t in (("a_scale", s), ("b_scale", bs), ("bias", bias), ("out", out)):
        yield name, t, lambda: L.mm_fp8(q, b, s, bs, bias=bias, out=out)
    yield "out", rows, lambda: L.moe_permute(c, ids, E, out=rows)
    yield "out", gx, lambda: L.moe_permute_backward(rows2, p.expanded_idx_to_permuted_idx, out=gx)
    yield "out", back, lambda: L.moe_unpermute(rows2, p, w, out=back)
    yield "grad_rows", rows2, lambda: L.moe_permute_backward(rows2, p.expanded_idx_to_permuted_idx)
    yield "grad_out", x, lambda: L.moe_unpermute_backward(x, rows, *p[2:], p.m_indptr, w)
    yield "grad_rows", rows, lambda: L.moe_unpermute_backward(c, rows2, *p[2:], p.m_indptr, w, grad_rows=rows)


def test_tensors_that_require_gradients_are_refused():
    for name, t, call in calls():
        call()
        t.requires_grad_()
        before = t.detach().clone()
        with pytest.raises(ValueError, match=f"{name} requires one"):
            call()
        assert torch.equal(t, before)
        with torch.no_grad():
            call()
        t.requires_grad_(False)
    L.nvfp4lora_device_status()


def test_tensors_that_carry_tangents_are_refused():
    x, ids, w = setup(FP)
    p = L.moe_permute(x, ids, E)
    one = torch.ones(H, device=DEV)
    q, s = L.fp8_quantize(x)
    b, bs = L.fp8_quantize(torch.ones(H, H, device=DEV), block_rows=128)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t.clone(), torch.ones_like(t))

        xd, rd, wd = dual(x), dual(p.rows), dual(w)
        for call in (lambda: L.moe_permute(xd, ids, E), lambda: L.moe_unpermute(rd, p, w), lambda: L.moe_unpermute(p.rows, p, wd),
                     lambda: L.moe_unpermute(rd, p.expanded_idx_to_permuted_idx),
                     lambda: L.moe_permute_backward(rd, p.expanded_idx_to_permuted_idx),
                     lambda: L.moe_unpermute_backward(xd, p.rows, *p[2:], p.m_indptr, w),
                     lambda: L.moe_unpermute_backward(x, rd, *p[2:], p.m_indptr, w), lambda: L.fp8_quantize(xd),
                     lambda: L.add_rmsnorm_fp8_quantize(xd, one), lambda: L.add_rmsnorm_fp8_quantize(x, dual(one)),
                     lambda: L.mm_fp8(q, b, dual(s), bs)):
            with pytest.raises(ValueError, match="tangent"):
                call()
        # nothing that carries one
        got = L.moe_unpermute(L.moe_permute(x, ids, E).rows, p, w)
        codes = L.moe_permute(q.view(torch.uint8), ids, E)
        L.mm_fp8(q, b, s, bs)
    assert torch.equal(got, L.moe_unpermute(p.rows, p, w))
    assert torch.equal(codes.m_indptr, p.m_indptr)


def test_recorded_calls_still_record():
    """The sort and its way back, also where a second derivative's graph is asked for: its use is refused by autograd."""
    x, ids, w = setup(FP)
    x.requires_grad_()
    p = L.moe_permute(x, ids, E)
    out = L.moe_unpermute(p.rows, p, w)
    (gx,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    assert torch.allclose(gx, w.sum(1, keepdim=True).expand(T, H), rtol=1e-6)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
