"""CPU checks of the routed-token, norm, quantizer and 8-bit product calls: the oracle against torch's
own conversions and hand-made tables, and every rule that the host refuses before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import routed_fp8 as R

P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_mm_b200.build import build
    lib = ctypes.CDLL(build(quiet=True))
    lib.nvfp4lora_last_error.restype = ctypes.c_char_p
    lib.nvfp4lora_moe_permute.argtypes = [P, I64, I64, P, I64, I64, I64, I32, P, I64, P, P, P, P, I64, P]
    lib.nvfp4lora_moe_unpermute.argtypes = [P, I64, I64, I32, P, P, I64, I64, P, P]
    lib.nvfp4lora_moe_permute_backward.argtypes = [P, I64, I64, I32, P, I64, I64, P, P]
    lib.nvfp4lora_moe_unpermute_backward.argtypes = [P, P, I64, I64, I32, P, P, P, I64, P, I64, I64, P, P, P]
    lib.nvfp4lora_fp8_quantize.argtypes = [P, I64, I64, I32, I64, P, P, I64, I64, P]
    lib.nvfp4lora_rmsnorm_fp8_quantize.argtypes = [P, P, P, I64, I64, I32, F32, P, P, P, I64, I64, P]
    lib.nvfp4lora_mm_fp8.argtypes = [P, P, P, I64, I64, P, P, P, I32, I64, I64, I64, P]
    return lib


def refused(lib, f, ok, bad):
    args = dict(ok)
    for k in bad:
        assert k in args, k
    args.update(bad)
    st = f(*args.values(), None)
    assert st == 1, (bad, st)
    return lib.nvfp4lora_last_error().decode()


PERMUTE = dict(x=0x10000, T=100, row_bytes=64, ids=0x20000, k=4, E=8, align=128, zero=1, rows=0x30000, cap=1408,
               indptr=0x40000, idx=0x50000, inv=0x60000, ws=None, ws_bytes=0)


@pytest.mark.parametrize("bad,word", [
    (dict(T=-1), "num_tokens"), (dict(k=0), "top_k"), (dict(k=17), "top_k"), (dict(E=0), "num_experts"),
    (dict(E=1025), "num_experts"), (dict(align=0), "align"), (dict(align=4097), "align"), (dict(row_bytes=0), "row_bytes"),
    (dict(cap=1279), "padded_rows"), (dict(indptr=None), "m_indptr"), (dict(indptr=0x40002), "m_indptr"),
    (dict(x=None), "non-null"), (dict(ids=None), "non-null"), (dict(rows=None), "non-null"), (dict(idx=None), "non-null"),
    (dict(inv=None), "non-null"), (dict(ids=0x20001), "4-byte aligned"),
    (dict(T=5000, cap=1 << 20), "workspace"), (dict(T=5000, cap=1 << 20, ws=0x70000, ws_bytes=64 * 8 * 4 - 1), "workspace"),
    (dict(T=1 << 29), "too large"), (dict(cap=1 << 31), "padded_rows"),
    (dict(rows=0x10000), "overlap"), (dict(rows=0x118C0), "overlap"), (dict(x=0x45FFF), "overlap"),
])
def test_permute_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_moe_permute, PERMUTE, bad)


UNPERMUTE = dict(y=0x10000, rows=512, H=64, dtype=0, idx=0x20000, w=0x30000, T=100, k=4, out=0x40000)


@pytest.mark.parametrize("bad,word", [
    (dict(T=-1), "num_tokens"), (dict(k=0), "top_k"), (dict(k=17), "top_k"), (dict(H=0), "H = 0"), (dict(dtype=3), "dtype"),
    (dict(dtype=-1), "dtype"), (dict(y=None), "non-null"), (dict(idx=None), "non-null"), (dict(out=None), "non-null"),
    (dict(y=0x10001), "aligned"), (dict(dtype=2, out=0x40002), "aligned"), (dict(w=0x30002), "aligned"), (dict(rows=-1), "padded_rows"),
    (dict(out=0x10000), "overlap"), (dict(out=0x1FFFE), "overlap"), (dict(y=0x431FE), "overlap"),
])
def test_unpermute_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_moe_unpermute, UNPERMUTE, bad)
    if "w" not in bad:
        ok = {k: v for k, v in UNPERMUTE.items() if k != "w"}
        assert word in refused(lib, lib.nvfp4lora_moe_permute_backward, ok, bad)


BACKWARD = dict(g=0x10000, y=0x18000, rows=512, H=64, dtype=0, idx=0x20000, inv=0x28000, indptr=0x30000, E=4, w=0x38000,
                T=100, k=4, gy=0x40000, gw=0x48000)


@pytest.mark.parametrize("bad,word", [
    (dict(k=17), "top_k"), (dict(H=0), "H = 0"), (dict(dtype=7), "dtype"), (dict(E=0), "num_experts"), (dict(gw=None), "go together"),
    (dict(w=None), "go together"), (dict(indptr=None), "m_indptr"), (dict(g=None), "non-null"), (dict(y=None), "non-null"),
    (dict(inv=None), "non-null"), (dict(gy=None), "non-null"), (dict(gy=0x40001), "aligned"), (dict(rows=0), "padded_rows"),
    (dict(g=0x40000), "overlap"), (dict(g=0x4FFFE), "overlap"), (dict(y=0x40010), "overlap"),
])
def test_unpermute_backward_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_moe_unpermute_backward, BACKWARD, bad)


QUANT = dict(x=0x10000, rows=10, H=300, dtype=0, block_rows=1, q=0x20000, scales=0x30000, sr=1, sg=10)


@pytest.mark.parametrize("bad,word", [
    (dict(rows=0), "rows >= 1"), (dict(H=0), "H >= 1"), (dict(H=1 << 21), "2^20"), (dict(dtype=5), "dtype"),
    (dict(block_rows=64), "block_rows"), (dict(x=None), "non-null"), (dict(q=None), "non-null"), (dict(scales=None), "non-null"),
    (dict(scales=0x30002), "aligned"), (dict(dtype=2, x=0x10002), "aligned"), (dict(sg=9), "overlap"), (dict(sr=0, sg=0), "overlap"),
    (dict(sr=-1), "overlap"), (dict(sr=2, sg=1), "overlap"),
])
def test_quantize_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_fp8_quantize, QUANT, bad)


NORM = dict(x=0x10000, res=0x18000, weight=0x20000, rows=10, H=300, dtype=0, eps=1e-6, norm=None, q=0x28000, scales=0x30000,
            sr=3, sg=1)


@pytest.mark.parametrize("bad,word", [
    (dict(weight=None), "weight"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(res=0x18001), "aligned"),
    (dict(norm=0x19001), "aligned"), (dict(rows=0), "rows >= 1"), (dict(sr=2), "overlap"),
    (dict(norm=0x18000), "must not overlap"), (dict(norm=0x10010), "must not overlap"), (dict(res=0x10010), "must not overlap"),
])
def test_norm_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_rmsnorm_fp8_quantize, NORM, bad)


MM = dict(a=0x10000, b=0x20000, sa=0x30000, sm=1, sk=16, sb=0x40000, bias=None, out=0x50000, dtype=0, M=16, N=256, K=256)


@pytest.mark.parametrize("bad,word", [
    (dict(M=0), "M >= 1"), (dict(N=0), "N >= 1"), (dict(K=0), "multiple of 16"), (dict(K=24), "multiple of 16"),
    (dict(M=1 << 31), "2^30"), (dict(K=1 << 21), "2^20"), (dict(dtype=3), "out_dtype"), (dict(a=None), "non-null"),
    (dict(sb=None), "non-null"), (dict(out=None), "non-null"), (dict(a=0x10008), "16-byte aligned"), (dict(b=0x20001), "16-byte aligned"),
    (dict(sa=0x30002), "4-byte aligned"), (dict(out=0x50001), "aligned"), (dict(bias=0x60001), "aligned"), (dict(sk=-1), "negative"),
])
def test_mm_rules(lib, bad, word):
    assert word in refused(lib, lib.nvfp4lora_mm_fp8, MM, bad)


def test_binding_refuses_tensors_of_the_host():
    import nvfp4_block_scaled_mm_b200 as L
    x, ids = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    f8 = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    s = torch.ones(4, 1)
    for call in (lambda: L.moe_permute(x, ids, 4), lambda: L.moe_unpermute(x, ids), lambda: L.moe_permute_backward(x, ids),
                 lambda: L.moe_unpermute_backward(x, x, ids, ids, ids), lambda: L.fp8_quantize(x),
                 lambda: L.add_rmsnorm_fp8_quantize(x, x[0]), lambda: L.mm_fp8(f8, f8, s, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_capacity_holds_the_worst_routing():
    import nvfp4_block_scaled_mm_b200 as L
    for T, k, E, align in ((1, 1, 1, 128), (5, 2, 4, 128), (64, 2, 8, 128), (7, 3, 5, 8), (0, 2, 4, 128), (3, 16, 2, 1)):
        cap = L.moe_capacity(T, k, E, align)
        assert cap == R.moe_capacity(T, k, E, align)
        n = T * k
        # as many experts as possible with one row past a multiple of the alignment
        ids = np.minimum(np.arange(n), E - 1).reshape(T, k) if n else np.zeros((0, k), dtype=np.int64)
        assert R.moe_tables(ids, E, align, cap)[0][-1] <= cap


def test_oracle_tables_by_hand():
    ids = np.array([[1, 0], [-1, 1], [1, 1]])
    indptr, idx, inv = R.moe_tables(ids, 3, 2, 8)
    assert indptr.tolist() == [0, 2, 6, 6]
    assert idx.tolist() == [[2, 0], [-1, 3], [4, 5]]
    assert inv.tolist() == [1, -1, 0, 3, 4, 5, -1, -1]


def test_oracle_e4m3_is_torch_s():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(R.E4M3)) and np.array_equal(v[~np.isnan(v)], R.E4M3[~np.isnan(v)])
    x = torch.cat([torch.randn(20000) * s for s in (1e-3, 1.0, 100.0)]).clamp(-448, 448)
    x = torch.cat([x, torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 448.0, -448.0])])
    assert np.array_equal(R.e4m3_encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_norm_gradient_free_identities():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 40))
    h, y = R.add_rmsnorm(x, x, np.ones(40), 0.0)
    assert np.allclose(h, 2 * x) and np.allclose((y * y).mean(axis=1), 1.0)


# bf16 x: 10 x 300 in [0x10000, 0x11770); q: [0x20000, 0x20BB8); scales (r, g) at r + 10 g: [0x30000, 0x30078)
@pytest.mark.parametrize("bad", [
    dict(q=0x10000), dict(q=0x1176F), dict(q=0x10000 - 2999), dict(x=0x20BB6), dict(scales=0x10000), dict(scales=0x1176C),
    dict(scales=0x10000 - 116), dict(scales=0x20BB4), dict(scales=0x20000 - 116),
    dict(scales=0x10000 - 400, sr=100, sg=1), dict(scales=0x20000 - 3612, sr=401, sg=200), dict(block_rows=128, scales=0x1176C, sr=3, sg=1),
])
def test_quantize_refuses_overlapping_buffers(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_fp8_quantize, QUANT, bad)


def passes_the_host(f, ok, change):
    """The call's own rules hold: without a GPU the next step finds no device."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can be launched")
    return f(*{**ok, **change}.values(), None) != 1


@pytest.mark.parametrize("ok", [
    dict(), dict(q=0x11770), dict(q=0x10000 - 3000), dict(scales=0x11770), dict(scales=0x10000 - 120), dict(scales=0x20BB8),
    # scales (r, g) at r + 4000 g, a column of 40 bytes every 16000: x in the gap after the first, q after the second
    dict(scales=0x10000 - 40, sg=4000, q=0x10000 + 16000), dict(scales=0x10000 - 0x100, sg=4000),
    # scales two elements apart, a row of 20 bytes every 4000 (or 20000)
    dict(scales=0x20000 - 20, sr=1000, sg=2), dict(scales=0x10000 - 20, sr=5000, sg=2),
])
def test_quantize_takes_buffers_side_by_side(lib, ok):
    assert passes_the_host(lib.nvfp4lora_fp8_quantize, QUANT, ok)


def test_overlap_of_strided_scales_by_brute_force(lib):
    """Exact for matrices, transposes and their slices: against the sets of bytes."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can be launched")
    rng = np.random.default_rng(5)
    seen = [0, 0]
    for _ in range(4000):
        rows, groups = int(rng.integers(1, 5)), int(rng.integers(1, 4))
        H = 128 * (groups - 1) + 1
        inner, outer = (rows, groups) if rng.random() < 0.5 else (groups, rows)
        si = int(rng.integers(1, 4))
        so = (inner - 1) * si + 1 + int(rng.integers(0, 400))
        sr, sg = (si, so) if inner == rows else (so, si)
        base, q = 0x100000, 0x100000 + 4 * int(rng.integers(-400, 1200))
        x = 0x900000
        bytes_s = {base + 4 * (r * sr + g * sg) + b for r in range(rows) for g in range(groups) for b in range(4)}
        bytes_q = range(q, q + rows * H)
        want = any(b in bytes_s for b in bytes_q)
        args = dict(x=x, rows=rows, H=H, dtype=0, block_rows=1, q=q, scales=base, sr=sr, sg=sg)
        assert (lib.nvfp4lora_fp8_quantize(*args.values(), None) == 1) == want, args
        seen[want] += 1
    assert min(seen) > 300


# bf16 rows of 10 x 300 (0x1770 bytes): x 0x10000, residual 0x18000, norm_out 0x38000, q (0xBB8 bytes) 0x28000;
# weight (0x258 bytes) 0x20000; scales (0x78 bytes) 0x30000
NORMED = dict(NORM, norm=0x38000)


@pytest.mark.parametrize("bad", [
    dict(q=0x10000), dict(q=0x1176F), dict(q=0x18000 - 2999), dict(q=0x3976F), dict(q=0x20257), dict(q=0x20000 - 2999),
    dict(weight=0x18000 + 0x176E), dict(weight=0x38000 - 0x256), dict(weight=0x28000), dict(scales=0x1176C), dict(scales=0x18000 - 116),
    dict(scales=0x38000), dict(scales=0x20254), dict(scales=0x28BB4), dict(x=0x28BB6), dict(x=0x18000, q=0x18000),
    dict(x=0x38000, q=0x3976F), dict(x=0x18000, norm=0x18000),
])
def test_norm_refuses_overlapping_buffers(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_rmsnorm_fp8_quantize, NORMED, bad)


@pytest.mark.parametrize("ok", [
    dict(), dict(x=0x18000), dict(x=0x38000), dict(res=None, x=0x38000), dict(norm=None, x=0x18000), dict(weight=0x10000 + 600),
    dict(q=0x11770, scales=0x10000 - 120, weight=0x19770), dict(res=None, norm=None), dict(q=0x10000 - 3000, norm=0x19770),
])
def test_norm_takes_buffers_side_by_side(lib, ok):
    assert passes_the_host(lib.nvfp4lora_rmsnorm_fp8_quantize, NORMED, ok)


# a 16 x 256 in [0x10000, 0x11000), b 256 x 256 in [0x20000, 0x30000), a_scale (m, kb) at m + 16 kb in [0x30000, 0x30080),
# b_scale 2 x 2 in [0x40000, 0x40010), out bf16 16 x 256 (0x2000 bytes) at 0x50000, bias (0x200 bytes) at 0x60000
PRODUCT = dict(MM, bias=0x60000)


@pytest.mark.parametrize("bad", [
    dict(out=0x10000), dict(out=0x10FFE), dict(out=0x10000 - 0x1FFE), dict(out=0x2FFFE), dict(out=0x3007E), dict(out=0x30000 - 0x1FFE),
    dict(out=0x4000E), dict(out=0x40000 - 0x1FFE), dict(out=0x601FE), dict(bias=0x51FFE), dict(dtype=2, bias=0x53FFE),
    dict(sa=0x50000 - 0x100, sm=64, sk=1), dict(sa=0x51FFC, sm=0, sk=0), dict(sa=0x50000 - 120, sm=2, sk=1),
])
def test_mm_refuses_overlapping_buffers(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_mm_fp8, PRODUCT, bad)


@pytest.mark.parametrize("ok", [
    dict(), dict(a=0x20000), dict(out=0x11000), dict(out=0x10000 - 0x2000), dict(out=0x30080), dict(out=0x30000 + 0x10010),
    dict(bias=0x52000), dict(bias=None), dict(sa=0x52000, sm=0, sk=0), dict(sa=0x50000 - 4, sm=0, sk=0),
    dict(sa=0x50000 - 64, sk=4000), dict(sa=0x50000 - 8, sm=3000, sk=1),
])
def test_mm_takes_buffers_side_by_side(lib, ok):
    assert passes_the_host(lib.nvfp4lora_mm_fp8, PRODUCT, ok)


# 5000 tokens, 4 slots, 8 experts, 1 byte per row: x 0x100000 (0x1388 bytes), ids 0x110000 (0x13880), rows 0x140000 (0x10000),
# m_indptr 0x160000 (0x24), idx 0x170000 (0x13880), inv 0x1A0000 (0x40000), workspace 0x200000 (0x800)
ROUTED = dict(x=0x100000, T=5000, row_bytes=1, ids=0x110000, k=4, E=8, align=128, zero=1, rows=0x140000, cap=0x10000,
              indptr=0x160000, idx=0x170000, inv=0x1A0000, ws=0x200000, ws_bytes=0x800)
# bf16 rows of 64: grad_out 0x100000 (0x3200), y 0x110000 (0x10000), idx 0x130000 (0x640), inv 0x140000 (0x800),
# m_indptr 0x150000 (0x14), weights 0x160000 (0x640), grad_rows 0x170000 (0x10000), grad_weights 0x190000 (0x640)
GRADS = dict(g=0x100000, y=0x110000, rows=512, H=64, dtype=0, idx=0x130000, inv=0x140000, indptr=0x150000, E=4, w=0x160000,
             T=100, k=4, gy=0x170000, gw=0x190000)


@pytest.mark.parametrize("bad", [
    dict(rows=0x101387), dict(rows=0x110000), dict(indptr=0x101384), dict(indptr=0x14FFFC), dict(idx=0x11387C), dict(idx=0x160020),
    dict(inv=0x100000), dict(inv=0x18387C), dict(inv=0x14FFFC), dict(ws=0x12387C), dict(ws=0x1DFFFC), dict(ws=0x160000), dict(x=0x200000),
    dict(ids=0x1DFFFC), dict(ids=0x2007FC),
])
def test_permute_refuses_overlapping_tables(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_moe_permute, ROUTED, bad)


@pytest.mark.parametrize("bad", [
    dict(idx=0x40000), dict(idx=0x431FC), dict(w=0x431FC), dict(out=0x30000 + 0x63E), dict(out=0x20000 - 0x31FE),
])
def test_unpermute_refuses_overlapping_tables(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_moe_unpermute, UNPERMUTE, bad)


@pytest.mark.parametrize("bad", [
    dict(idx=0x17FFFC), dict(inv=0x170000), dict(indptr=0x17FFFC), dict(w=0x170000), dict(gw=0x17FFFC), dict(gw=0x130000),
    dict(gw=0x1407FC), dict(gw=0x150010), dict(gw=0x160004), dict(gw=0x1031FC), dict(gw=0x11FFFC), dict(y=0x170000, gw=0x17FFFC),
    dict(gw=None, w=None, indptr=0x170000),
])
def test_unpermute_backward_refuses_overlapping_tables(lib, bad):
    assert "must not overlap" in refused(lib, lib.nvfp4lora_moe_unpermute_backward, GRADS, bad)


def test_routed_calls_take_buffers_side_by_side(lib):
    for f, base, oks in (
            (lib.nvfp4lora_moe_permute, ROUTED, (dict(), dict(x=0x110000), dict(indptr=0x150000), dict(ws=0x1E0000), dict(rows=0x123880),
                                                dict(T=100, ws=0x160000, ws_bytes=0x800))),       # a workspace that is not used
            (lib.nvfp4lora_moe_unpermute, UNPERMUTE, (dict(), dict(w=None), dict(idx=0x43200), dict(w=0x20000))),
            (lib.nvfp4lora_moe_unpermute_backward, GRADS, (dict(), dict(y=0x170000), dict(gw=None, w=None), dict(gw=None, w=None, y=0x170010),
                                                           dict(gw=0x150014), dict(gw=0x160000), dict(gw=0x180000), dict(y=0x180000)))):
        for ok in oks:
            assert passes_the_host(f, base, ok), (ok, lib.nvfp4lora_last_error())
