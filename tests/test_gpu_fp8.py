"""8-bit quantizers, norm and product against the 64-bit references: codes and scales of the quantizer
bit for bit, the norm within its fp32 sums, the product within its rounding and exactly on whole
numbers; odd sizes, strides, one row to many, every kernel of the product, capture and streams."""

import numpy as np
import pytest
import torch

from oracle import routed_fp8 as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
F8 = torch.float8_e4m3fn


def randn(*shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def codes(q):
    return q.detach().cpu().view(torch.uint8).numpy()


QUANT = [(1, 1, BF), (1, 128, BF), (3, 130, HF), (5, 136, FP), (130, 256, BF), (17, 1000, BF), (257, 264, HF), (129, 127, FP),
         (33, 8192, FP), (600, 384, BF)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("T,H,dt", QUANT)
def test_quantizer_bit_for_bit(T, H, dt, block_rows):
    import nvfp4_block_scaled_mm_b200 as L
    x = randn(T, H, dtype=dt, seed=T + H, std=3.0)
    x[0, 0] = 0.0
    if T > 2 and H > 128:
        x[2, :128] = 0.0                            # a group of zeros
    q, s = L.fp8_quantize(x.to(DEV), block_rows=block_rows)
    wq, ws = R.fp8_quantize(x.float().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(codes(q), wq)


def test_quantizer_extremes():
    import nvfp4_block_scaled_mm_b200 as L
    x = torch.zeros(6, 128)
    x[0, :2] = torch.tensor([3e38, -1.0])
    x[1, :2] = torch.tensor([1e-38, -1e-40])        # below the smallest scale
    x[2, 5] = 2.0 ** -100
    x[3, 7] = -0.0
    x[4, :] = torch.linspace(-448, 448, 128)
    x[5, 3], x[5, 4] = float("nan"), 2.0
    q, s = L.fp8_quantize(x.to(DEV))
    wq, ws = R.fp8_quantize(x[:5].numpy())
    assert np.array_equal(s.cpu().numpy()[:5], ws) and np.array_equal(codes(q)[:5], wq)
    last = q[5].float().cpu()
    assert torch.isnan(last[3]) and last[4] == 448 and float(s[5, 0]) == np.float32(2) / np.float32(448)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("H", [256, 254])            # packed maxima of aligned rows, and elements
@pytest.mark.parametrize("dt", [BF, HF])
def test_quantizer_extremes_of_16_bit_types(dt, H, block_rows):
    import nvfp4_block_scaled_mm_b200 as L
    info = torch.finfo(dt)
    sub = 2.0 ** (-133 if dt == BF else -24)         # the smallest subnormal
    n = 5
    x = torch.zeros(n * 128, H, dtype=dt)
    b = [x[i * 128:(i + 1) * 128] for i in range(n)]  # a block of rows for each value
    b[0][:, 1::2] = -sub
    b[1][:, ::3] = info.max
    b[2][:, 5] = -info.tiny
    b[3][:] = randn(128, H, dtype=dt, seed=9)
    b[3][7, :9] = float("nan")                       # in both halves of a pair, and beside the rows around it
    b[3][7, 20] = -0.0
    b[4][:] = float("nan")
    q, s = L.fp8_quantize(x.to(DEV), block_rows=block_rows)
    bad = torch.isnan(x)
    wq, ws = R.fp8_quantize(torch.where(bad, torch.zeros_like(x), x).float().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert torch.equal(torch.isnan(q.float().cpu()), bad)
    assert np.array_equal(codes(q)[~bad.numpy()], wq[~bad.numpy()])


def test_quantizer_strided_outputs_and_misaligned_input():
    import nvfp4_block_scaled_mm_b200 as L
    x = randn(50, 512, dtype=BF, seed=1).to(DEV)
    q, s = L.fp8_quantize(x)
    assert s.stride() == (1, 50)
    rows = torch.zeros(50, 4, device=DEV)
    q2, s2 = L.fp8_quantize(x, scales=rows)
    assert torch.equal(s2, s) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    wide = torch.full((50, 9), -1.0, device=DEV)
    L.fp8_quantize(x, scales=wide[:, :4])
    assert torch.equal(wide[:, :4], s) and torch.all(wide[:, 4:] == -1)
    shifted = torch.empty(50 * 512 + 1, dtype=BF, device=DEV)[1:].view(50, 512).copy_(x)
    for rows_per in (1, 128):
        a, b = L.fp8_quantize(shifted, block_rows=rows_per), L.fp8_quantize(x, block_rows=rows_per)
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


NORM = [(1, 8, BF), (2, 128, BF), (16, 4096, BF), (7, 1000, HF), (3, 5, FP), (9, 131, BF), (4, 8192, FP), (5, 16384, BF),
        (3, 16392, HF), (300, 264, BF), (2, 6144, HF), (11, 2056, FP),
        # many rows: a warp per row, and one, two and four chunks per warp, aligned and not
        (1201, 200, BF), (1203, 205, HF), (1200, 512, FP), (1205, 500, BF), (1190, 1000, BF), (1187, 1001, FP),
        (1184, 3000, HF), (1185, 4095, BF), (1186, 4104, BF), (1184, 8200, HF), (1184, 8199, BF)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H,dt", NORM)
def test_norm_against_the_formula(T, H, dt, residual):
    import nvfp4_block_scaled_mm_b200 as L
    x, w = randn(T, H, dtype=dt, seed=1), (1 + 0.2 * randn(H, dtype=FP, seed=2)).to(dt)
    r = randn(T, H, dtype=dt, seed=3, std=2.0) if residual else None
    rd = None if r is None else r.to(DEV)
    y = torch.empty(T, H, dtype=dt, device=DEV)
    q, s = L.add_rmsnorm_fp8_quantize(x.to(DEV), w.to(DEV), rd, eps=1e-5, norm_out=y)
    if residual:                                     # the fp32 sum of two values, rounded once: bit for bit
        assert torch.equal(rd.cpu(), (x.float() + r.float()).to(dt))
    _, ref = R.add_rmsnorm(f64(x), None if r is None else f64(r), f64(w), 1e-5)
    # y in fp32: the sum of H squares is a tree of at most H / 8 / 32 + 42 additions in a row (2^-24 each,
    # halved by the square root), then a few operations
    rel = (H / 256 + 42) / 2 * 2.0 ** -24 + 12 * 2.0 ** -24
    assert np.all(np.abs(f64(y) - ref) <= (torch.finfo(dt).eps / 2 + rel) * np.abs(ref) + torch.finfo(dt).tiny)
    pad = np.zeros((T, -(-H // 128) * 128))
    pad[:, :H] = np.abs(ref)
    want = np.maximum(pad.reshape(T, -1, 128).max(2), 2.0 ** -100) / 448
    assert np.all(np.abs(f64(s) - want) <= (rel + 2 * 2.0 ** -24) * want)
    t = ref / np.repeat(want, 128, axis=1)[:, :H]    # the code's value before its rounding, |t| <= 448
    assert np.all(np.abs(f64(q.float()) - t) <= (2.0 ** -4 + 4 * rel) * np.abs(t) + 2.0 ** -10)


def test_norm_reads_and_writes_in_place():
    import nvfp4_block_scaled_mm_b200 as L
    x, w = randn(20, 1024, dtype=BF, seed=4).to(DEV), torch.ones(1024, dtype=BF, device=DEV)
    y = torch.empty_like(x)
    q, s = L.add_rmsnorm_fp8_quantize(x, w, norm_out=y)
    keep = x.clone()
    q2, s2 = L.add_rmsnorm_fp8_quantize(x, w, norm_out=x)
    assert torch.equal(x, y) and torch.equal(s, s2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    a, b = keep.clone(), keep.clone()                # the residual is x itself: h = 2 x
    L.add_rmsnorm_fp8_quantize(a, w, a)
    assert torch.equal(a, (b.float() * 2).to(BF))


def test_norm_zero_and_nan_rows():
    import nvfp4_block_scaled_mm_b200 as L
    for H in (256, 250):
        x = torch.zeros(3, H, dtype=FP, device=DEV)
        x[1, 4] = float("nan")
        x[2] = 1.0
        q, s = L.add_rmsnorm_fp8_quantize(x, torch.ones(H, device=DEV), eps=0.25)
        f = q.float()
        assert torch.all(f[0] == 0) and torch.all(torch.isnan(f[1])) and torch.all(f[2] == 448)
        assert torch.isfinite(s).all()


def product_problem(M, N, K, seed, whole=False):
    g = torch.Generator().manual_seed(seed)
    G, B = -(-K // 128), -(-N // 128)
    if whole:                                        # sums of whole numbers below 2^24: exact in fp32
        a = torch.randint(-8, 9, (M, K), generator=g).float().to(F8)
        b = torch.randint(-8, 9, (N, K), generator=g).float().to(F8)
        sa = 2.0 ** torch.randint(0, 3, (M, G), generator=g).float()
        sb = 2.0 ** torch.randint(0, 3, (B, G), generator=g).float()
    else:
        a = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(F8)
        b = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(F8)
        sa = (torch.rand(M, G, generator=g) + 0.5) * 0.01
        sb = (torch.rand(B, G, generator=g) + 0.5) * 0.0002
    return a, b, sa, sb


# few rows (split K; 16, 32, 64 and 128 token columns, several token tiles), the SM pair, ragged everything
MM = [(1, 1, 16), (1, 4096, 4096), (16, 384, 128), (17, 130, 144), (16, 1000, 2064), (33, 129, 400), (64, 300, 1024),
      (65, 257, 272), (100, 1028, 1040), (128, 512, 2048), (129, 100, 96), (200, 130, 4096), (300, 4100, 4112),
      (257, 2057, 528), (512, 4096, 512), (1000, 5001, 208), (2048, 2304, 1152), (65, 8200, 272),
      (128, 8192, 528), (200, 4096, 6160), (513, 9475, 144)]


@pytest.mark.parametrize("M,N,K", MM)
def test_product_of_whole_numbers_is_exact(M, N, K):
    import nvfp4_block_scaled_mm_b200 as L
    a, b, sa, sb = product_problem(M, N, K, M + N + K, whole=True)
    out = L.mm_fp8(a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=FP)
    L.nvfp4lora_device_status()
    ref, mag = R.mm_fp8(codes(a), codes(b), sa.numpy(), sb.numpy())
    assert mag.max() < 2 ** 24
    assert np.array_equal(f64(out), ref)


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (16, 1000, 2064), (40, 300, 4096), (100, 1028, 1040), (300, 2052, 4112),
                                   (1024, 2048, 1040)])
def test_product_against_the_formula(M, N, K, dt):
    import nvfp4_block_scaled_mm_b200 as L
    a, b, sa, sb = product_problem(M, N, K, M)
    bias = randn(N, dtype=BF, seed=9)
    for bi in (None, bias):
        out = L.mm_fp8(a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), bias=None if bi is None else bi.to(DEV), out_dtype=dt)
        ref, mag = R.mm_fp8(codes(a), codes(b), sa.numpy(), sb.numpy(), None if bi is None else f64(bi))
        # one rounding to the type, and fp32 sums of K products (at most one step of 2^-23 of the total size
        # each), K / 128 scaled additions and the bias
        tol = torch.finfo(dt).eps / 2 * np.abs(ref) + (128 + K / 128 + 4) * 2.0 ** -23 * (mag + np.abs(ref))
        assert np.all(np.abs(f64(out) - ref) <= tol)
    L.nvfp4lora_device_status()


def test_product_scale_strides_and_repeats():
    import nvfp4_block_scaled_mm_b200 as L
    for M in (5, 150, 400):
        a, b, sa, sb = [t.to(DEV) for t in product_problem(M, 520, 656, 3)]
        ref = L.mm_fp8(a, b, sa, sb, out_dtype=FP)
        for _ in range(3):
            assert torch.equal(L.mm_fp8(a, b, sa, sb, out_dtype=FP), ref)
        assert torch.equal(L.mm_fp8(a, b, sa.t().contiguous().t(), sb, out_dtype=FP), ref)
        wide = torch.full((M, 17), float("nan"), device=DEV)
        wide[:, 2:14:2] = sa
        assert torch.equal(L.mm_fp8(a, b, wide[:, 2:14:2], sb, out_dtype=FP), ref)
        one = L.mm_fp8(a, b, sa[:1, :1].expand(M, 6), sb, out_dtype=FP)
        assert torch.equal(one, L.mm_fp8(a, b, sa[:1, :1].repeat(M, 6), sb, out_dtype=FP))


def test_product_leaves_what_is_behind_its_rows():
    import nvfp4_block_scaled_mm_b200 as L
    for M, N in ((3, 136), (3, 131), (200, 264), (200, 259), (700, 1032), (700, 1031)):
        a, b, sa, sb = [t.to(DEV) for t in product_problem(M, N, 256, 3)]
        buf = torch.full((M * N + 512,), 7.0, dtype=BF, device=DEV)
        out = L.mm_fp8(a, b, sa, sb, out=buf[:M * N].view(M, N))
        assert torch.all(buf[M * N:] == 7) and torch.equal(out, L.mm_fp8(a, b, sa, sb))


def test_product_nan_stays_in_its_row_and_column():
    import nvfp4_block_scaled_mm_b200 as L
    for M in (20, 100, 500):
        a, b, sa, sb = product_problem(M, 500, 256, 5)
        a.view(torch.uint8)[7, 3] = 0x7F
        b.view(torch.uint8)[11, 200] = 0xFF
        out = L.mm_fp8(*[t.to(DEV) for t in (a, b, sa, sb)]).cpu()
        bad = torch.zeros(M, 500, dtype=torch.bool)
        bad[7], bad[:, 11] = True, True
        assert torch.equal(torch.isnan(out), bad)


def test_binding_refusals():
    import nvfp4_block_scaled_mm_b200 as L
    a, b, sa, sb = [t.to(DEV) for t in product_problem(8, 256, 256, 1)]
    x, w = randn(8, 256, dtype=BF, seed=1).to(DEV), torch.ones(256, dtype=BF, device=DEV)
    for call, word in (
            (lambda: L.mm_fp8(a.view(torch.uint8), b, sa, sb), "float8"), (lambda: L.mm_fp8(a, b[:, :128], sa, sb), "contiguous"),
            (lambda: L.mm_fp8(a, b[:, :128].contiguous(), sa, sb), "K differs"), (lambda: L.mm_fp8(a, b, sa[:7], sb), "a_scale"),
            (lambda: L.mm_fp8(a, b, sa, sb[:1]), "b_scale"), (lambda: L.mm_fp8(a, b, sa, sb.t()), "contiguous"),
            (lambda: L.mm_fp8(a, b, sa, sb, out_dtype=torch.float64), "out_dtype"), (lambda: L.mm_fp8(a, b, sa, sb, out=x[:4]), "out must"),
            (lambda: L.mm_fp8(a, b, sa, sb, bias=w[:200]), "bias"), (lambda: L.mm_fp8(a, b, sa, sb.cpu()), "CUDA"),
            (lambda: L.mm_fp8(a[:, :24].contiguous(), b[:, :24].contiguous(), sa[:, :1], sb[:, :1].contiguous()), "multiple of 16"),
            (lambda: L.mm_fp8(a[:0], b, sa[:0], sb), "M >= 1"),
            (lambda: L.fp8_quantize(x, block_rows=2), "block_rows"), (lambda: L.fp8_quantize(x.t()), "contiguous"),
            (lambda: L.fp8_quantize(x, q=a[:4]), "q must"), (lambda: L.fp8_quantize(x, scales=sa[:, :1]), "scales"),
            (lambda: L.fp8_quantize(x, scales=sa[:1].expand(8, 2)), "overlap"), (lambda: L.fp8_quantize(x[:0]), "rows >= 1"),
            (lambda: L.add_rmsnorm_fp8_quantize(x, w.float()), "bfloat16"), (lambda: L.add_rmsnorm_fp8_quantize(x, w[:128]), "weight"),
            (lambda: L.add_rmsnorm_fp8_quantize(x, w, x[:4]), "residual"), (lambda: L.add_rmsnorm_fp8_quantize(x, w, eps=-1.0), "eps"),
            (lambda: L.add_rmsnorm_fp8_quantize(x, w, norm_out=x.float()), "norm_out")):
        with pytest.raises(ValueError, match=word):
            call()


def test_captured_layer_replays_on_new_inputs_and_a_side_stream():
    """Norm, product, quantizer and product as a captured step, replayed on inputs copied in; the eager
    calls on another stream give the same bits."""
    import nvfp4_block_scaled_mm_b200 as L
    H, F = 512, 1024
    w = torch.ones(H, dtype=BF, device=DEV)
    w1, s1 = L.fp8_quantize(randn(F, H, dtype=BF, seed=1, std=0.1).to(DEV), block_rows=128)
    w2, s2 = L.fp8_quantize(randn(H, F, dtype=BF, seed=2, std=0.1).to(DEV), block_rows=128)
    for T in (4, 24, 60, 100, 300, 700):
        x = randn(T, H, dtype=BF, seed=3).to(DEV)
        res = torch.zeros_like(x)

        def step():
            q, s = L.add_rmsnorm_fp8_quantize(x, w, res)
            h = torch.relu(L.mm_fp8(q, w1, s, s1))
            return L.mm_fp8(*[t for t in (L.fp8_quantize(h)[0], w2)], L.fp8_quantize(h)[1], s2)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for seed in (5, 6):
            x.copy_(randn(T, H, dtype=BF, seed=seed))
            res.zero_()
            graph.replay()
            res.zero_()
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                want = step()
            side.synchronize()
            assert torch.equal(got, want)
            # the layer in 64 bits from the same 8-bit weights, within the 8-bit rounding of its two inputs
            xd = x.double()
            y = xd / (xd.square().mean(1, keepdim=True) + 1e-6).sqrt()
            W1 = w1.double() * s1.double().repeat_interleave(128, 0)[:F].repeat_interleave(128, 1)[:, :H]
            W2 = w2.double() * s2.double().repeat_interleave(128, 0)[:H].repeat_interleave(128, 1)[:, :F]
            ref = torch.relu(y @ W1.t()) @ W2.t()
            worst = (y.abs() @ W1.abs().t()) * 2.0 ** -4 @ W2.abs().t() + (torch.relu(y @ W1.t()) @ W2.abs().t()) * 2.0 ** -3
            assert torch.all((got.double() - ref).abs() <= worst + 2.0 ** -6)
    L.nvfp4lora_device_status()


def test_outputs_past_32_bit_offsets():
    import nvfp4_block_scaled_mm_b200 as L
    M, N, K = 70000, 65536, 16                       # 9.2 GB of bf16: offsets past 2^32 bytes and elements
    a = torch.zeros(M, K, dtype=torch.uint8, device=DEV).view(F8)
    b = torch.zeros(N, K, dtype=torch.uint8, device=DEV).view(F8)
    a.view(torch.uint8)[-3:] = 0x38                  # 1.0
    b.view(torch.uint8)[-5:] = 0x38
    sa, sb = torch.ones(M, 1, device=DEV), torch.ones(N // 128, 1, device=DEV)
    out = L.mm_fp8(a, b, sa, sb)
    assert float(out[-1, -1]) == 16.0 and float(out[-3, -5]) == 16.0 and float(out[-4, -1]) == 0.0
    assert float(out.sum(dtype=torch.float64)) == 16.0 * 15
    L.nvfp4lora_device_status()


@pytest.mark.parametrize("T", [1, 5, 1200])
@pytest.mark.parametrize("H", [4, 12, 100, 260, 1004])
def test_fp32_rows_of_four_modulo_eight(T, H):
    """Quantizer and norm of fp32 rows that are whole 16-byte units but no multiple of eight elements: within their
    row, and nothing written behind the last."""
    import nvfp4_block_scaled_mm_b200 as L
    x, r, w = randn(T, H, dtype=FP, seed=1), randn(T, H, dtype=FP, seed=2), 1 + 0.2 * randn(H, dtype=FP, seed=3)
    q_all = torch.full((T * H + 64,), 3, dtype=torch.uint8, device=DEV)
    q = q_all[:T * H].view(F8).view(T, H)
    for block_rows in (1, 128):
        _, s = L.fp8_quantize(x.to(DEV), block_rows=block_rows, q=q)
        wq, ws = R.fp8_quantize(x.numpy(), block_rows)
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(codes(q), wq) and torch.all(q_all[T * H:] == 3)
    res_all = torch.full((T * H + 64,), 7.0, device=DEV)
    out_all = res_all.clone()
    res, out = res_all[:T * H].view(T, H), out_all[:T * H].view(T, H)
    res.copy_(r)
    L.add_rmsnorm_fp8_quantize(x.to(DEV), w.to(DEV), res, eps=1e-5, norm_out=out, q=q)
    assert torch.equal(res.cpu(), x + r)
    for whole in (res_all, out_all):
        assert torch.all(whole[T * H:] == 7)
    assert torch.all(q_all[T * H:] == 3)
    _, ref = R.add_rmsnorm(f64(x), f64(r), f64(w), 1e-5)
    rel = (H / 256 + 42) / 2 * 2.0 ** -24 + 12 * 2.0 ** -24
    assert np.all(np.abs(f64(out) - ref) <= (2.0 ** -24 + rel) * np.abs(ref) + torch.finfo(FP).tiny)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("H", [512, 510])            # registers of aligned rows, and elements
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_quantizer_infinities(dt, H, block_rows):
    """An infinity makes its group's scale infinite: it becomes a NaN and the group's finite values zeros of their sign;
    a NaN stays one, and other groups are as without it."""
    import nvfp4_block_scaled_mm_b200 as L
    x = randn(256, H, dtype=dt, seed=4)
    clean = x.clone()
    x[3, 130], x[3, 140], x[3, 200] = float("inf"), float("nan"), -0.0
    x[200, 300], x[200, 301] = float("-inf"), float("inf")
    q, s = L.fp8_quantize(x.to(DEV), block_rows=block_rows)
    wq, ws = R.fp8_quantize(clean.float().numpy(), block_rows)
    got_q, got_s = codes(q), s.cpu().numpy()
    hit = np.zeros(ws.shape, dtype=bool)
    hit[3 // block_rows, 1] = hit[200 // block_rows, 2] = True
    cells = np.repeat(np.repeat(hit, block_rows, axis=0), 128, axis=1)[:256, :H]
    assert np.all(np.isposinf(got_s[hit])) and np.array_equal(got_s[~hit], ws[~hit])
    assert np.array_equal(got_q[~cells], wq[~cells])
    bad = (~torch.isfinite(x)).numpy()
    assert np.all((got_q[bad] & 0x7F) == 0x7F)
    finite = cells & ~bad
    sign = np.signbit(x.float().numpy())
    assert np.array_equal(got_q[finite], np.where(sign[finite], 0x80, 0))


@pytest.mark.parametrize("T,H", [(6, 512), (1200, 256), (6, 1000), (6, 1001), (1200, 4104), (6, 16392), (6, 16385)])
@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_norm_infinities(T, H, dt):
    """An infinity in x + residual makes the row's norm infinite: itself a NaN, the rest zeros; opposite infinities, as
    any NaN, make the whole row NaN; finite rows are not touched by it.  Scales stay finite."""
    import nvfp4_block_scaled_mm_b200 as L
    x, r, w = randn(T, H, dtype=dt, seed=1), randn(T, H, dtype=dt, seed=2), torch.ones(H, dtype=dt)
    x0, r0 = x.clone(), r.clone()
    x[1, 7] = float("inf")
    r[2, H - 1] = float("-inf")
    x[4, 3], r[4, 3] = float("inf"), float("-inf")
    out = [torch.empty(T, H, dtype=dt, device=DEV) for _ in range(2)]
    rd, rd0 = r.to(DEV), r0.to(DEV)
    q, s = L.add_rmsnorm_fp8_quantize(x.to(DEV), w.to(DEV), rd, norm_out=out[0])
    q0, s0 = L.add_rmsnorm_fp8_quantize(x0.to(DEV), w.to(DEV), rd0, norm_out=out[1])
    same = [i for i in range(T) if i not in (1, 2, 4)]
    assert torch.equal(q.view(torch.uint8)[same], q0.view(torch.uint8)[same]) and torch.equal(s[same], s0[same])
    assert torch.equal(out[0][same], out[1][same])
    assert torch.isfinite(s).all()
    for i, j in ((1, 7), (2, H - 1)):
        for got in (q[i].float(), out[0][i].float()):
            assert torch.isnan(got[j]) and torch.all(torch.cat([got[:j], got[j + 1:]]) == 0)
    assert torch.isnan(q[4].float()).all() and torch.isnan(out[0][4]).all()
    assert torch.isposinf(rd[1, 7]) and torch.isneginf(rd[2, H - 1]) and torch.isnan(rd[4, 3])


def test_norm_of_rows_whose_squares_pass_fp32():
    """Documented: the mean square is held in fp32, and a row for which it overflows gives zeros."""
    import nvfp4_block_scaled_mm_b200 as L
    x = torch.full((3, 256), 1.0, device=DEV)
    x[1] = 1e20
    x[2] = 1e18
    q, s = L.add_rmsnorm_fp8_quantize(x, torch.ones(256, device=DEV))
    assert torch.all(q[1].float() == 0) and torch.all(q[0].float() == 448) and torch.all(q[2].float() == 448)
    assert torch.isfinite(s).all()
