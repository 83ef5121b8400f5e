"""The one-to-one forwarders of the routed-token and 8-bit entry points: as many arguments as the C function takes, in its
order, on the tensors' device and that device's current stream, or on the stream given and its device."""

import contextlib

import pytest
import torch

import nvfp4_block_scaled_mm_b200 as L

CALLS = {
    "moe_permute": "x num_tokens row_bytes topk_ids top_k num_experts align zero_padding rows padded_rows m_indptr "
                   "expanded_idx_to_permuted_idx permuted_idx_to_expanded_idx workspace workspace_bytes",
    "moe_unpermute": "y padded_rows H dtype expanded_idx_to_permuted_idx topk_weights num_tokens top_k out",
    "moe_permute_backward": "grad_rows padded_rows H dtype expanded_idx_to_permuted_idx num_tokens top_k grad_x",
    "moe_unpermute_backward": "grad_out y padded_rows H dtype expanded_idx_to_permuted_idx permuted_idx_to_expanded_idx m_indptr "
                              "num_experts topk_weights num_tokens top_k grad_rows grad_weights",
    "fp8_quantize": "x rows H dtype block_rows q scales scale_stride_row scale_stride_group",
    "rmsnorm_fp8_quantize": "x residual weight rows H dtype eps norm_out q scales scale_stride_row scale_stride_group",
    "mm_fp8": "a b a_scale a_scale_stride_m a_scale_stride_k b_scale bias out out_dtype M N K",
}
NUMBERS = {"num_tokens", "row_bytes", "top_k", "num_experts", "align", "zero_padding", "padded_rows", "workspace_bytes", "H", "dtype",
           "block_rows", "scale_stride_row", "scale_stride_group", "eps", "a_scale_stride_m", "a_scale_stride_k", "out_dtype",
           "M", "N", "K"}


class FakeLib:
    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        return lambda *args: self.seen.append((name, args)) or 0


def arguments(name):
    """Each argument by its name: numbers that all differ, a tensor for every pointer."""
    number = NUMBERS if name == "moe_permute" else NUMBERS | {"rows"}
    return {k: 1 if k == "zero_padding" else 100 + i if k in number else torch.zeros(3) for i, k in enumerate(CALLS[name].split())}


def plain(v):
    return v.data_ptr() if isinstance(v, torch.Tensor) else v


@pytest.mark.parametrize("name", CALLS)
def test_forwarders_pass_every_argument_on_the_right_device(name, monkeypatch):
    from nvfp4_block_scaled_mm_b200.build import build
    build(quiet=True)
    types = getattr(L._load(), "nvfp4lora_" + name).argtypes
    args = arguments(name)
    assert len(types) == len(args) + 1
    lib, entered = FakeLib(), []
    monkeypatch.setattr(L, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered.append(d) or contextlib.nullcontext())
    monkeypatch.setattr(L, "_raw_stream", lambda index: 5000 + index)
    f = getattr(L, "nvfp4lora_" + name)

    class On(torch.Tensor):                        # a host tensor that says it is on another GPU
        device = torch.device("cuda", 1)

    away = {k: v.as_subclass(On) if isinstance(v, torch.Tensor) else v for k, v in args.items()}
    f(**away)
    f(**args, stream=type("S", (), {"device": torch.device("cuda", 3), "cuda_stream": 9000})())
    assert lib.seen[0] == ("nvfp4lora_" + name, (*map(plain, args.values()), 5001))
    assert lib.seen[1] == ("nvfp4lora_" + name, (*map(plain, args.values()), 9000))
    assert [torch.device("cuda", d) if isinstance(d, int) else d for d in entered] == [torch.device("cuda", 1), torch.device("cuda", 3)]
