"""Each one-to-one forwarder of the routed-token and 8-bit entry points against the call above it."""

import pytest
import torch

import nvfp4_block_scaled_mm_b200 as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("side", [False, True])
def test_routed_tokens(T, side):
    k, E, H = 2, 6, 96
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).to(DEV)
    x, w = torch.randn(T, H, generator=g).to(BF).to(DEV), torch.rand(T, k, generator=g).to(DEV)
    cap = L.moe_capacity(T, k, E, 8)
    start = torch.full((cap, H), 3.0, dtype=BF, device=DEV)
    want = L.moe_permute(x, ids, E, align=8, zero_padding=False, out=start.clone())
    out = L.moe_unpermute(want.rows, want, w)
    gx = L.moe_permute_backward(want.rows, want.expanded_idx_to_permuted_idx)
    gy, gw = L.moe_unpermute_backward(x, want.rows, *want[2:], want.m_indptr, w, grad_rows=start.clone())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    rows, got, got_gx, got_gy = start.clone(), torch.zeros_like(x), torch.zeros_like(x), start.clone()
    tables = [torch.empty_like(t) for t in want[1:]]
    work, got_gw = torch.empty(64 * E, dtype=torch.int32, device=DEV), torch.zeros_like(w)
    torch.cuda.synchronize()
    L.nvfp4lora_moe_permute(x, T, 2 * H, ids, k, E, 8, False, rows, cap, *tables, work, 4 * work.numel(), stream=stream)
    L.nvfp4lora_moe_unpermute(rows, cap, H, 0, tables[1], w, T, k, got, stream=stream)
    L.nvfp4lora_moe_permute_backward(rows, cap, H, 0, tables[1], T, k, got_gx, stream=stream)
    L.nvfp4lora_moe_unpermute_backward(x, rows, cap, H, 0, tables[1], tables[2], tables[0], E, w, T, k, got_gy, got_gw, stream=stream)
    torch.cuda.synchronize()
    for a, b in zip((rows, *tables, got, got_gx, got_gy, got_gw), (*want, out, gx, gy, gw)):
        assert torch.equal(a, b)
    L.nvfp4lora_device_status()


@pytest.mark.parametrize("side", [False, True])
def test_8_bit_calls(side):
    M, N, K = 20, 200, 272
    x, one, bias = torch.randn(M, K, device=DEV).to(BF), torch.ones(K, dtype=BF, device=DEV), torch.randn(N, device=DEV).to(BF)
    weight = torch.randn(N, K, device=DEV)
    res = torch.randn(M, K, device=DEV).to(BF)
    want_res, want_norm = res.clone(), torch.empty_like(x)
    wb, wbs = L.fp8_quantize(weight, block_rows=128)
    wq, ws = L.add_rmsnorm_fp8_quantize(x, one, want_res, eps=1e-3, norm_out=want_norm)
    want = L.mm_fp8(wq, wb, ws, wbs, bias=bias, out_dtype=FP)
    stream = torch.cuda.Stream() if side else None
    b, bs, q, s = torch.empty_like(wb), torch.empty_like(wbs), torch.empty_like(wq), torch.empty_like(ws)
    norm, out = torch.empty_like(x), torch.empty(M, N, device=DEV)
    torch.cuda.synchronize()
    L.nvfp4lora_fp8_quantize(weight, N, K, 2, 128, b, bs, *bs.stride(), stream=stream)
    L.nvfp4lora_rmsnorm_fp8_quantize(x, res, one, M, K, 0, 1e-3, norm, q, s, *s.stride(), stream=stream)
    L.nvfp4lora_mm_fp8(q, b, s, *s.stride(), bs, bias, out, 2, M, N, K, stream=stream)
    torch.cuda.synchronize()
    for got, ref in ((b.view(torch.uint8), wb.view(torch.uint8)), (bs, wbs), (q.view(torch.uint8), wq.view(torch.uint8)), (s, ws),
                     (res, want_res), (norm, want_norm), (out, want)):
        assert torch.equal(got, ref)
    L.nvfp4lora_device_status()


def test_gradient_of_the_weights_in_their_place():
    """grad_weights may be topk_weights itself: every slot's weight is read before its gradient is written."""
    for T, k, H in ((50, 16, 96), (700, 7, 2056)):
        E, g = 6, torch.Generator().manual_seed(T)
        ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).to(DEV)
        x, w = torch.randn(T, H, generator=g).to(BF).to(DEV), torch.rand(T, k, generator=g).to(DEV)
        p = L.moe_permute(x, ids, E)
        zeros = torch.zeros_like(p.rows)
        gy, gw = L.moe_unpermute_backward(x, p.rows, *p[2:], p.m_indptr, w, grad_rows=zeros.clone())
        L.nvfp4lora_moe_unpermute_backward(x, p.rows, p.rows.shape[0], H, 0, *p[2:], p.m_indptr, E, w, T, k, zeros, w)
        assert torch.equal(zeros, gy) and torch.equal(w, gw)
    L.nvfp4lora_device_status()
