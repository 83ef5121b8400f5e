"""The device's error word: a time-out is never replaced by the report of a bad table entry, whichever comes first."""

import pytest
import torch

import nvfp4_block_scaled_mm_b200 as L
from workloads import make_grouped_problem

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


def bad_entries():
    """(name, call): each leaves out a bad entry and reports it."""
    x = torch.ones(8, 64, dtype=BF, device=DEV)
    ids = torch.full((8, 2), 4, dtype=torch.int32, device=DEV)
    many = torch.full((5000, 1), 4, dtype=torch.int32, device=DEV)
    idx = torch.full((8, 2), 16, dtype=torch.int32, device=DEV)
    inv, indptr = torch.zeros(16, dtype=torch.int32, device=DEV), torch.tensor([0, 16], dtype=torch.int32, device=DEV)
    w, rows = torch.ones(8, 2, device=DEV), torch.ones(16, 64, dtype=BF, device=DEV)
    p = make_grouped_problem([128, 256], 256, 256, 8, seed=4)
    t = {k: getattr(p, k).to(DEV) for k in ("a", "b", "a_sf", "b_sf", "m_indptr", "alpha")}
    t["m_indptr"][1] = 100
    ptr = L.fill_w_ptr([torch.zeros(8 * 64, dtype=BF, device=DEV) for _ in range(4)])
    yield "permute", lambda: L.moe_permute(x, ids, 4)
    yield "permute, counted", lambda: L.moe_permute(torch.ones(5000, 8, device=DEV), many, 4)
    yield "unpermute", lambda: L.moe_unpermute(rows, idx)
    yield "unpermute gradient", lambda: L.moe_unpermute_backward(x, rows, idx, inv, indptr, w)
    yield "grouped", lambda: L.grouped_mm_nvfp4_lora(**t)
    yield "LoRA delta", lambda: L.bgmv_moe_gemm2_lora_delta(rows, idx, ptr, 0, ptr, 0, ids, w, torch.zeros(8, dtype=torch.int32, device=DEV), 8, 64)


def test_a_timeout_outranks_bad_entries():
    for name, call in bad_entries():
        call()
        with pytest.raises(ValueError):
            L.nvfp4lora_device_status()
        for first in (True, False):
            if not first:
                call()
            L.nvfp4lora_selftest_wait_timeout(1_000_000)          # 1 ms
            if first:
                call()
            with pytest.raises(L.DeviceTimeoutError):
                L.nvfp4lora_device_status()
            L.nvfp4lora_device_status()                           # the word is cleared


def test_the_first_bad_entry_is_reported():
    calls = dict(bad_entries())
    calls["unpermute"]()
    calls["LoRA delta"]()
    with pytest.raises(ValueError, match="routed tokens"):
        L.nvfp4lora_device_status()
    calls["LoRA delta"]()
    calls["permute"]()
    with pytest.raises(ValueError, match="LoRA delta"):
        L.nvfp4lora_device_status()
    L.nvfp4lora_device_status()
