"""Buffers that calls write by address count the write in their version counters, as in-place operations of torch do:
autograd refuses a saved tensor that a later call has overwritten, where it would otherwise form wrong gradients."""

import pytest
import torch

import nvfp4_block_scaled_mm_b200 as L
from gpu_util import Dev
from workloads import make_grouped_problem, make_problem

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
T, K, E, H = 40, 2, 4, 256


def routed(seed=1, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32).to(DEV)
    return torch.randn(T, H, generator=g).to(dtype).to(DEV), ids, torch.rand(T, K, generator=g).to(DEV)


def writers():
    """(name, buffers written, call) of every call that takes a buffer to write."""
    x, ids, w = routed()
    p = L.moe_permute(x, ids, E)
    rows = torch.zeros_like(p.rows)
    f8, one = torch.zeros(T, H, dtype=torch.float8_e4m3fn, device=DEV), torch.ones(H, dtype=BF, device=DEV)
    s = torch.zeros(T, 2, device=DEV)
    q, qs = L.fp8_quantize(x)
    wq, ws = L.fp8_quantize(torch.ones(H, H, dtype=BF, device=DEV), block_rows=128)

    def new():
        return torch.zeros_like(x)

    out, res, norm, gx, mm = new(), new(), new(), new(), new()
    grads = torch.zeros_like(rows)
    yield "moe_permute", [rows], lambda: L.moe_permute(x, ids, E, out=rows)
    yield "moe_unpermute", [out], lambda: L.moe_unpermute(p.rows, p, w, out=out)
    yield "moe_permute_backward", [gx], lambda: L.moe_permute_backward(p.rows, p.expanded_idx_to_permuted_idx, out=gx)
    yield "moe_unpermute_backward", [grads], lambda: L.moe_unpermute_backward(x, p.rows, *p[2:], p.m_indptr, w, grad_rows=grads)
    yield "fp8_quantize", [f8, s], lambda: L.fp8_quantize(x, q=f8, scales=s)
    yield "add_rmsnorm_fp8_quantize", [res, norm, f8, s], lambda: L.add_rmsnorm_fp8_quantize(x, one, res, norm_out=norm, q=f8, scales=s)
    yield "mm_fp8", [mm], lambda: L.mm_fp8(q, wq, qs, ws, out=mm)
    d = Dev(make_problem(16, 256, 256, 8, seed=3, alpha=2.0 ** -9, lora_scale=1.5, bias=False))
    d_out = d.new_out()
    yield "mm_nvfp4_lora", [d_out], lambda: L.mm_nvfp4_lora(d.a, d.b, d.a_sf, d.b_sf, d.alpha, out=d_out)
    adapter = L.prepare_nvfp4_lora_adapter(d.lora_b, d.lora_scale, d.alpha)
    yield "mm_nvfp4_lora, prepared", [d_out], lambda: L.mm_nvfp4_lora(d.a, d.b, d.a_sf, d.b_sf, d.alpha, d.d, lora_adapter=adapter, out=d_out)
    gp = make_grouped_problem([128, 256], 256, 256, 8, seed=4)
    t = [getattr(gp, k).to(DEV) for k in ("a", "b", "a_sf", "b_sf", "m_indptr", "alpha")]
    g_out = torch.zeros(gp.rows, gp.N, dtype=BF, device=DEV)
    yield "grouped_mm_nvfp4_lora", [g_out], lambda: L.grouped_mm_nvfp4_lora(*t, out=g_out)
    banks = [torch.zeros(8 * H, dtype=BF, device=DEV) for _ in range(E)]
    ptr = L.fill_w_ptr(banks)
    delta, lids = new(), torch.zeros(T, dtype=torch.int32, device=DEV)
    yield "bgmv_moe_gemm2_lora_delta", [delta], lambda: L.bgmv_moe_gemm2_lora_delta(
        p.rows, p.expanded_idx_to_permuted_idx, ptr, 0, ptr, 0, ids.clamp(min=0), w, lids, 8, H, out=delta)
    codes, sf = torch.zeros(T, H // 2, dtype=torch.uint8, device=DEV), torch.zeros(128 * H // 16, dtype=torch.uint8, device=DEV)
    yield "fp4_quantize", [codes, sf], lambda: L.fp4_quantize(x, torch.ones(1, device=DEV), codes=codes, scales=sf)


def test_every_written_buffer_counts_the_write():
    for name, buffers, call in writers():
        before = [b._version for b in buffers]
        call()
        for b, v in zip(buffers, before):
            assert b._version > v, name
    L.nvfp4lora_device_status()


def test_a_refused_call_counts_nothing():
    x, ids, w = routed()
    p = L.moe_permute(x, ids, E)
    before = x._version, p.rows._version
    with pytest.raises(ValueError, match="overlap"):
        L.moe_unpermute(p.rows, p, w, out=p.rows[:T])
    with pytest.raises(ValueError, match="eps"):
        L.add_rmsnorm_fp8_quantize(x, torch.ones(H, dtype=BF, device=DEV), x, eps=-1.0)
    assert (x._version, p.rows._version) == before


@pytest.mark.parametrize("overwrite", ["permute", "residual", "norm_out", "product"])
def test_backward_refuses_rows_that_a_call_has_overwritten(overwrite):
    x, ids, w = routed()
    w.requires_grad_()
    p = L.moe_permute(x, ids, E)
    y = p.rows.clone()
    out = L.moe_unpermute(y, p, w)
    one = torch.ones(H, dtype=BF, device=DEV)
    if overwrite == "permute":
        L.moe_permute(x * 3, ids, E, out=y)
    elif overwrite == "residual":
        L.add_rmsnorm_fp8_quantize(torch.ones_like(y), one, y)
    elif overwrite == "norm_out":
        L.add_rmsnorm_fp8_quantize(torch.ones_like(y), one, norm_out=y)
    else:
        q, s = L.fp8_quantize(y.new_ones(y.shape[0], 128))
        b, bs = L.fp8_quantize(y.new_ones(H, 128), block_rows=128)
        L.mm_fp8(q, b, s, bs, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    assert w.grad is None


def test_inference_tensors_and_capture_still_run():
    x, ids, w = routed()
    with torch.inference_mode():
        p = L.moe_permute(x, ids, E)
        res = torch.zeros(T, H, dtype=BF, device=DEV)
        L.add_rmsnorm_fp8_quantize(x, torch.ones(H, dtype=BF, device=DEV), res)
        assert torch.equal(res, x)
    out = torch.zeros_like(x)
    p = L.moe_permute(x, ids, E)
    L.moe_unpermute(p.rows, p, w, out=out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_unpermute(p.rows, p, w, out=out)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)
