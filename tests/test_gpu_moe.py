"""Routed tokens sorted by expert and back, with gradients, against the 64-bit references: tables and
copied rows exactly, sums within the rounding of their type, over both counting paths, every vector
width, one token to many, inactive slots, repeated and unused experts; refusals, streams and capture."""

import numpy as np
import pytest
import torch

from oracle import routed_fp8 as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def routing(T, k, E, seed, inactive=0.1, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":                              # every slot on one expert
        ids = torch.full((T, k), E - 1, dtype=torch.int32)
    else:                                          # repeats within a token included
        ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < inactive] = -1
    return ids


def rows_of(T, H, dtype, seed):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


# (T, top_k, E, H, dtype, align, inactive share, kind)
SHAPES = [
    (1, 1, 1, 8, BF, 128, 0.0, "mixed"),
    (1, 16, 1024, 64, BF, 128, 0.2, "mixed"),
    (37, 3, 5, 65, HF, 8, 0.1, "mixed"),            # 2-byte rows
    (37, 3, 5, 66, HF, 1, 0.1, "mixed"),            # 4-byte vectors, no padding
    (50, 2, 7, 24, FP, 128, 0.1, "mixed"),
    (64, 2, 8, 4096, BF, 128, 0.0, "mixed"),        # the decode batch
    (20, 4, 16, 40, BF, 128, 1.0, "mixed"),         # no active slot
    (300, 8, 64, 136, FP, 3, 0.0, "one"),           # one expert holds all
    (512, 8, 96, 72, BF, 128, 0.05, "mixed"),       # 4096 slots: the most that each CTA counts itself
    (513, 8, 96, 72, BF, 128, 0.05, "mixed"),       # one token more: the counting kernel
    (2049, 8, 96, 2056, BF, 128, 0.05, "mixed"),
    (9001, 5, 1024, 16, HF, 16, 0.05, "mixed"),
    (30000, 1, 3, 8, BF, 128, 0.0, "mixed"),
    (4000, 8, 2, 16, BF, 128, 0.0, "one"),
    (3000, 16, 40, 520, BF, 1, 0.1, "mixed"),       # more than one batch of slots per CTA
]


@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[0]}k{s[1]}E{s[2]}H{s[3]}a{s[5]}{s[7]}")
def test_permute_tables_and_rows(shape, zero):
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H, dt, align, inactive, kind = shape
    ids, x = routing(T, k, E, T + H, inactive, kind), rows_of(T, H, dt, 5)
    cap = L.moe_capacity(T, k, E, align)
    before = torch.full((cap + 3, H), 7.0, dtype=dt, device=DEV)
    p = L.moe_permute(x.to(DEV), ids.to(DEV), E, align=align, zero_padding=zero, out=before)
    L.nvfp4lora_device_status()
    indptr, idx, inv = R.moe_tables(ids.numpy(), E, align, cap + 3)
    assert p.m_indptr.tolist() == indptr.tolist()
    assert np.array_equal(p.expanded_idx_to_permuted_idx.cpu().numpy(), idx)
    assert np.array_equal(p.permuted_idx_to_expanded_idx.cpu().numpy(), inv)
    want = torch.full((cap + 3, H), 7.0, dtype=dt)
    if zero:
        want[:int(indptr[-1])] = 0.0
    at = np.nonzero(inv >= 0)[0]
    want[at] = x[inv[at] // k]
    assert torch.equal(p.rows.cpu(), want)


@pytest.mark.parametrize("dt", [torch.uint8, torch.float8_e4m3fn, torch.int32, torch.float64])
def test_permute_copies_any_element_type(dt):
    import nvfp4_block_scaled_mm_b200 as L
    ids = routing(40, 3, 6, 1)
    x = torch.randint(0, 100, (40, 9), generator=torch.Generator().manual_seed(2)).to(dt)
    p = L.moe_permute(x.to(DEV), ids.to(DEV), 6, align=8)
    inv = p.permuted_idx_to_expanded_idx.cpu()
    at = torch.nonzero(inv >= 0).reshape(-1)
    assert torch.equal(p.rows.cpu().view(torch.uint8)[at], x[inv[at].long() // 3].view(torch.uint8))


def test_permute_of_no_tokens():
    import nvfp4_block_scaled_mm_b200 as L
    x, ids = torch.zeros(0, 16, dtype=BF, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    p = L.moe_permute(x, ids, 4)
    assert p.m_indptr.tolist() == [0, 0, 0, 0, 0] and p.rows.shape == (0, 16)
    out = torch.full((5, 16), 3.0, dtype=BF, device=DEV)
    p = L.moe_permute(x, ids, 4, out=out)
    assert torch.all(p.rows == 3) and p.permuted_idx_to_expanded_idx.tolist() == [-1] * 5
    assert L.moe_unpermute(p.rows, p).shape == (0, 16)
    gy, gw = L.moe_unpermute_backward(x, p.rows, p.expanded_idx_to_permuted_idx, p.permuted_idx_to_expanded_idx, p.m_indptr,
                                      torch.zeros(0, 2, device=DEV))
    assert gy.shape == (5, 16) and gw.shape == (0, 2)
    L.nvfp4lora_device_status()


def test_permute_misaligned_rows_and_base():
    """Rows that start off a 16-byte boundary take a narrower copy."""
    import nvfp4_block_scaled_mm_b200 as L
    ids, x = routing(33, 2, 4, 3), rows_of(33, 64, BF, 4)
    ref = L.moe_permute(x.to(DEV), ids.to(DEV), 4, align=8)
    for shift in (1, 2):
        buf = torch.empty(33 * 64 + shift, dtype=BF, device=DEV)[shift:].view(33, 64).copy_(x)
        p = L.moe_permute(buf, ids.to(DEV), 4, align=8)
        n = int(p.m_indptr[-1])
        assert torch.equal(p.rows[:n], ref.rows[:n])


@pytest.mark.parametrize("T,k", [(40, 2), (3000, 8)])
def test_expert_id_out_of_range_is_left_out_and_reported(T, k):
    import nvfp4_block_scaled_mm_b200 as L
    ids, x = routing(T, k, 6, 9, 0.0), rows_of(T, 32, BF, 1)
    ids[T // 2, 1] = 6
    p = L.moe_permute(x.to(DEV), ids.to(DEV), 6)
    with pytest.raises(ValueError, match="expert id"):
        L.nvfp4lora_device_status()
    indptr, idx, _ = R.moe_tables(ids.numpy(), 6, 128, p.rows.shape[0])
    assert p.m_indptr.tolist() == indptr.tolist()
    assert np.array_equal(p.expanded_idx_to_permuted_idx.cpu().numpy(), idx)
    L.nvfp4lora_device_status()


def sum_tolerance(ref, mag, terms, dtype):
    """One rounding to the type (half a step) on fp32 sums of `terms` products of total size `mag`
    (each product and each addition is off by at most 2^-24 of `mag`)."""
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + (2 * terms + 1) * 2.0 ** -24 * mag + torch.finfo(dtype).tiny


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[0]}k{s[1]}E{s[2]}H{s[3]}a{s[5]}{s[7]}")
def test_unpermute_and_its_gradients(shape, weighted):
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H, dt, align, inactive, kind = shape
    if T * k * H > 2 ** 21:                         # the reference walks the slots: keep the row count
        T = max(1, 2 ** 21 // (k * H))
    ids = routing(T, k, E, T + H, inactive, kind)
    cap = R.moe_capacity(T, k, E, align) + 2
    indptr, idx, inv = R.moe_tables(ids.numpy(), E, align, cap)
    y, g = rows_of(cap, H, dt, 6), rows_of(T, H, dt, 7)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(8)) if weighted else None
    y[torch.from_numpy(inv < 0)] = float("nan")     # rows of no slot are never read into a result
    d = [t if t is None else torch.as_tensor(t, dtype=torch.int32).to(DEV) for t in (idx, inv, indptr)]
    wd = None if w is None else w.to(DEV)
    out = L.moe_unpermute(y.to(DEV), d[0], wd)
    buf = torch.full((cap, H), 7.0, dtype=dt, device=DEV)
    gy, gw = L.moe_unpermute_backward(g.to(DEV), y.to(DEV), *d, wd, grad_rows=buf)
    L.nvfp4lora_device_status()
    yn, gn, wn = f64(y), f64(g), None if w is None else f64(w)
    ref = R.moe_sum(yn, idx, wn)
    mag = R.moe_sum(np.abs(yn), idx, wn)
    assert np.all(np.abs(f64(out) - ref) <= sum_tolerance(ref, mag, k, dt))
    ry, rw = R.moe_unpermute_grads(gn, yn, idx, wn, np.full((cap, H), 7.0), int(indptr[-1]), inv)
    assert np.all(np.abs(f64(gy) - ry) <= sum_tolerance(ry, np.abs(ry), 1, dt))
    if weighted:
        _, mw = R.moe_unpermute_grads(np.abs(gn), np.abs(yn), idx, wn, np.zeros((cap, H)), int(indptr[-1]), inv)
        assert np.all(np.abs(f64(gw) - rw) <= H * 2.0 ** -24 * mw)
    else:
        assert gw is None
        gx = L.moe_permute_backward(y.to(DEV), d[0])
        assert torch.equal(gx, out)


def test_index_out_of_range_is_left_out_and_reported():
    import nvfp4_block_scaled_mm_b200 as L
    y = rows_of(10, 16, FP, 1).to(DEV)
    idx = torch.tensor([[0, 10], [3, 4]], dtype=torch.int32, device=DEV)
    out = L.moe_unpermute(y, idx)
    with pytest.raises(ValueError, match="permuted index"):
        L.nvfp4lora_device_status()
    assert torch.equal(out, torch.stack([y[0], y[3] + y[4]]))
    inv = torch.full((10,), -1, dtype=torch.int32, device=DEV)
    indptr = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    w = torch.ones(2, 2, device=DEV)
    _, gw = L.moe_unpermute_backward(torch.ones(2, 16, device=DEV), y, idx, inv, indptr, w)
    with pytest.raises(ValueError, match="permuted index"):
        L.nvfp4lora_device_status()
    assert float(gw[0, 1]) == 0.0


def test_gradients_against_differences():
    """Both operators in one graph, in fp32, against central differences of the 64-bit references."""
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H = 6, 3, 4, 5
    ids = routing(T, k, E, 11, 0.15)
    g = torch.Generator().manual_seed(12)
    x = torch.randn(T, H, generator=g)
    w = torch.rand(T, k, generator=g)
    c = torch.randn(T, H, generator=g)
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    p = L.moe_permute(xd, ids.to(DEV), E, align=4)
    out = L.moe_unpermute(p.rows * p.rows, p, wd)
    (out * c.to(DEV)).sum().backward()
    _, idx, inv = R.moe_tables(ids.numpy(), E, 4, p.rows.shape[0])

    def loss(xv, wv):
        rows = np.zeros((len(inv), H))
        at = inv >= 0
        rows[at] = xv[inv[at] // k]
        return float((R.moe_sum(rows * rows, idx, wv) * c.numpy()).sum())

    xn, wn, h = x.double().numpy(), w.double().numpy(), 1e-6
    for base, grad, f in ((xn, xd.grad, lambda v: loss(v, wn)), (wn, wd.grad, lambda v: loss(xn, v))):
        for i in np.ndindex(base.shape):
            up, dn = base.copy(), base.copy()
            up[i] += h
            dn[i] -= h
            want = (f(up) - f(dn)) / (2 * h)
            assert abs(float(grad[i]) - want) <= 1e-5 * (1 + abs(want)), (i, float(grad[i]), want)


def test_no_gradient_where_none_is_asked_for():
    import nvfp4_block_scaled_mm_b200 as L
    ids, x = routing(8, 2, 4, 1).to(DEV), rows_of(8, 16, FP, 1).to(DEV)
    w = torch.rand(8, 2, device=DEV, requires_grad=True)
    p = L.moe_permute(x, ids, 4)
    assert not p.rows.requires_grad
    out = L.moe_unpermute(p.rows, p, w)
    out.sum().backward()
    assert w.grad is not None
    with torch.no_grad():
        assert not L.moe_unpermute(p.rows, p.expanded_idx_to_permuted_idx, w).requires_grad


def test_binding_refusals():
    import nvfp4_block_scaled_mm_b200 as L
    ids, x = routing(8, 2, 4, 1).to(DEV), rows_of(8, 16, BF, 1).to(DEV)
    p = L.moe_permute(x, ids, 4)
    xg = x.clone().requires_grad_()
    for call, word in (
            (lambda: L.moe_permute(x.t(), ids, 4), "contiguous"), (lambda: L.moe_permute(x[:7], ids, 4), "7 rows"),
            (lambda: L.moe_permute(x, ids.long(), 4), "int32"), (lambda: L.moe_permute(x, ids, 0), "num_experts"),
            (lambda: L.moe_permute(x, ids, 4, align=0), "align"), (lambda: L.moe_permute(x, ids, 4, out=x), "capacity"),
            (lambda: L.moe_permute(xg, ids, 4, out=p.rows), "out is not supported"),
            (lambda: L.moe_permute(x, ids.repeat(1, 9), 4), "top_k"),
            (lambda: L.moe_unpermute(xg, p.expanded_idx_to_permuted_idx), "MoePermutation"),
            (lambda: L.moe_unpermute(xg, p), "rows"),
            (lambda: L.moe_unpermute(p.rows, p, torch.rand(8, 3, device=DEV)), "topk_weights"),
            (lambda: L.moe_unpermute(p.rows, p, torch.rand(8, 2, device=DEV).to(BF)), "float32"),
            (lambda: L.moe_unpermute(p.rows.to(torch.float64), p), "float32"),
            (lambda: L.moe_unpermute_backward(x, x, *p[2:], p.m_indptr, torch.rand(8, 2, device=DEV)), "rows, H"),
            (lambda: L.moe_permute_backward(p.rows, p.permuted_idx_to_expanded_idx), "2 dimensions")):
        with pytest.raises(ValueError, match=word):
            call()


def test_capture_replay_with_new_routing_and_refusal_of_recording():
    """One captured sort, experts' work and way back serve new routings, on a side stream's capture with
    an eager graph of the same weights alive; recording a gradient inside a capture is refused."""
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H = 3000, 6, 32, 64                     # the counting kernel and its workspace too
    x, w = rows_of(T, H, FP, 1).to(DEV), torch.rand(T, k, device=DEV)
    leaf = x.clone().requires_grad_()
    p = L.moe_permute(leaf, routing(T, k, E, 1).to(DEV), E)
    alive = L.moe_unpermute(p.rows * 2.0, p, w)      # an eager graph of `leaf`, kept
    ids = routing(T, k, E, 2).to(DEV)

    def step():
        q = L.moe_permute(leaf.detach(), ids, E)
        y = q.rows * 2.0
        out = L.moe_unpermute(y, q, w)
        gy, gw = L.moe_unpermute_backward(out, y, q.expanded_idx_to_permuted_idx, q.permuted_idx_to_expanded_idx,
                                          q.m_indptr, w)
        return out, gw, L.moe_permute_backward(gy, q.expanded_idx_to_permuted_idx)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            L.moe_permute(leaf, ids, E)
        with pytest.raises(ValueError, match="captured"):
            L.moe_unpermute(p.rows, p, w)
        got = step()
    for seed in (3, 4):
        ids.copy_(routing(T, k, E, seed))
        graph.replay()
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    alive.sum().backward()
    assert torch.isfinite(leaf.grad).all()
    L.nvfp4lora_device_status()


def test_recorded_gradients_are_refused_in_a_capture(monkeypatch):
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H = 20, 2, 4, 32
    leaf, w = rows_of(T, H, FP, 1).to(DEV).requires_grad_(), torch.rand(T, k, device=DEV)
    p = L.moe_permute(leaf, routing(T, k, E, 1).to(DEV), E)
    out = L.moe_unpermute(p.rows.detach().requires_grad_(), p, w)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError, match="moe_permute_backward"):
        p.rows.sum().backward()
    with pytest.raises(ValueError, match="moe_unpermute_backward"):
        out.sum().backward()


def test_buffers_that_overlap():
    """The sort and the way back refuse to run in place; the gradient may replace y, x its own norm."""
    import nvfp4_block_scaled_mm_b200 as L
    x, ids = rows_of(40, 64, BF, 1).to(DEV), routing(40, 1, 4, 1).to(DEV)
    with pytest.raises(ValueError, match="overlap"):
        L.moe_permute(x, ids, 4, align=1, out=x)
    p = L.moe_permute(x, ids, 4, align=1)
    with pytest.raises(ValueError, match="overlap"):
        L.moe_unpermute(p.rows, p, out=p.rows)
    with pytest.raises(ValueError, match="overlap"):
        L.moe_unpermute_backward(x, None, p[2], p[3], p.m_indptr, grad_rows=x)
    with pytest.raises(ValueError, match="overlap"):
        L.add_rmsnorm_fp8_quantize(x, x[0].clone(), p.rows, norm_out=p.rows)
    for T, k, H, dt in ((300, 8, 520, BF), (50, 16, 33, HF), (70, 3, 4096, FP)):
        ids, w = routing(T, k, 8, 2).to(DEV), torch.rand(T, k, device=DEV)
        p, g = L.moe_permute(rows_of(T, H, dt, 2).to(DEV), ids, 8), rows_of(T, H, dt, 3).to(DEV)
        args = (p[2], p[3], p.m_indptr, w)
        used = int(p.m_indptr[-1])
        want = L.moe_unpermute_backward(g, p.rows, *args)
        got = L.moe_unpermute_backward(g, p.rows, *args, grad_rows=p.rows)
        assert got[0] is p.rows and torch.equal(got[0][:used], want[0][:used]) and torch.equal(got[1], want[1])
    L.nvfp4lora_device_status()


def test_side_stream_and_repeats_are_bitwise_equal():
    import nvfp4_block_scaled_mm_b200 as L
    ids, x = routing(5000, 8, 60, 3).to(DEV), rows_of(5000, 96, BF, 3).to(DEV)
    w = torch.rand(5000, 8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    runs = []
    for _ in range(2):
        with torch.cuda.stream(s):
            p = L.moe_permute(x, ids, 60)
            out = L.moe_unpermute(p.rows, p, w)
            gy, gw = L.moe_unpermute_backward(out, p.rows, *p[2:], p.m_indptr, w, grad_rows=torch.zeros_like(p.rows))
        runs.append((p.rows[:int(p.m_indptr[-1])], *p[1:], out, gy, gw))
    s.synchronize()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    """Rows whose byte offset and element offset pass 2^32."""
    import nvfp4_block_scaled_mm_b200 as L
    H, cap = 1 << 16, 66000                          # 8.6 GB of bf16 rows
    T, k, E = 40, 1, 1
    x = rows_of(T, H, BF, 1).to(DEV)
    idx = torch.arange(cap - T, cap, dtype=torch.int32, device=DEV).view(T, 1)
    inv = torch.full((cap,), -2, dtype=torch.int32, device=DEV)
    y = torch.zeros(cap, H, dtype=BF, device=DEV)
    y[cap - T:] = x
    assert torch.equal(L.moe_unpermute(y, idx), x)
    inv.fill_(0)
    gy, _ = L.moe_unpermute_backward(x * 2, None, idx, inv, torch.tensor([0, cap], dtype=torch.int32, device=DEV), grad_rows=y)
    assert torch.equal(gy[cap - T:], x * 2)
    del gy, y
    ids = torch.zeros(33000, 2, dtype=torch.int32, device=DEV)
    xs = torch.zeros(33000, H, dtype=BF, device=DEV)
    xs[-1] = x[0]
    p = L.moe_permute(xs, ids, 1, align=1)
    assert torch.equal(p.rows[-2:], x[:1].expand(2, H))
    L.nvfp4lora_device_status()


def test_sorted_rows_through_the_grouped_product():
    """Tokens sorted by expert, quantized, through the grouped NVFP4 product and back, against the same
    rows sorted on the host; the LoRA delta reads the same table."""
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H, N = 200, 2, 4, 512, 256
    ids, x = routing(T, k, E, 21, 0.05), rows_of(T, H, BF, 21)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(1))
    p = L.moe_permute(x.to(DEV), ids.to(DEV), E)
    gs = torch.tensor([40.0], device=DEV)
    a, a_sf = L.fp4_quantize(p.rows[:, :].contiguous(), gs)
    bw = rows_of(E * N, H, BF, 22).to(DEV)
    b, b_sf = L.fp4_quantize(bw, gs)
    alpha = torch.full((E,), 1 / 1600.0, device=DEV)
    y = L.grouped_mm_nvfp4_lora(a, b.view(E, N, H // 2), a_sf, b_sf, p.m_indptr, alpha)
    out = L.moe_unpermute(y, p, w.to(DEV))
    L.nvfp4lora_device_status()
    # each token's rows through the dense product of its expert
    want = torch.zeros(T, N, dtype=torch.float64)
    xa, xa_sf = L.fp4_quantize(x.to(DEV), gs)
    for e in range(E):
        be, be_sf = L.fp4_quantize(bw[e * N:(e + 1) * N].contiguous(), gs)
        ye = L.mm_nvfp4_lora(xa, be, xa_sf, be_sf, alpha[:1]).cpu().double()
        want += ((ids == e) * w).sum(1, keepdim=True).double() * ye
    size = want.abs().max().item()
    # each row is rounded to bf16 once by either product (their sums may differ in order), the total once more
    assert (out.cpu().double() - want).abs().max().item() <= 2.0 ** -7 * size + 2.0 ** -8 * size


def test_sorted_rows_into_the_lora_delta_replayed():
    """The rows and the table that one captured call writes are what the next reads, at every replay: sorted
    tokens straight into the LoRA delta, against the same calls with the device idle in between."""
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, I, H, rank = 64, 2, 8, 512, 256, 16
    a_banks = [rows_of(2 * rank, I, BF, 30 + e).to(DEV) for e in range(E)]
    b_banks = [rows_of(2 * H, rank, BF, 50 + e).to(DEV) for e in range(E)]
    wa, wb = L.fill_w_ptr(a_banks), L.fill_w_ptr(b_banks)
    x, ids = rows_of(T, I, BF, 1).to(DEV), routing(T, k, E, 1).to(DEV)
    w = torch.rand(T, k, device=DEV)
    lids = (torch.arange(T, device=DEV) % 2).int()

    def step(idle=lambda: None):
        valid = ids.clamp(min=0)
        out = torch.zeros(T, H, dtype=BF, device=DEV)
        p = L.moe_permute(x, ids, E, align=8)
        idle()
        delta = L.bgmv_moe_gemm2_lora_delta(p.rows, p.expanded_idx_to_permuted_idx, wa, rank * I, wb, H * rank, valid, w,
                                            lids, rank, H, out=out)
        idle()
        return delta, L.moe_unpermute(p.rows, p, w)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(2, 12):
        x.copy_(rows_of(T, I, BF, seed))
        ids.copy_(routing(T, k, E, seed))
        want = step(torch.cuda.synchronize)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), seed
    L.nvfp4lora_device_status()


def guarded(rows, H, dtype, fill, tail=64):
    """A [rows, H] view and the whole buffer, whose last `tail` elements no call may touch."""
    whole = torch.full((rows * H + tail,), fill, dtype=dtype, device=DEV)
    return whole[:rows * H].view(rows, H), whole


@pytest.mark.parametrize("T,k,E,align", [(1, 1, 1, 1), (1, 3, 2, 4), (37, 3, 5, 8), (300, 8, 16, 1)])
@pytest.mark.parametrize("H,dt", [(4, FP), (12, FP), (100, FP), (252, FP), (260, FP), (1004, FP), (2052, FP), (4, BF), (12, HF), (100, BF)])
def test_rows_that_end_inside_a_lanes_eight_elements(T, k, E, align, H, dt):
    """Row lengths of 4 modulo 8: the last lane of a row holds four of its eight elements.  Sums, gradients and zeros
    end with their row, in its middle and at the buffer's end, and nothing behind the last row is read into a result."""
    import nvfp4_block_scaled_mm_b200 as L
    ids = routing(T, k, E, T + H, 0.1 if T > 1 else 0.0)
    cap = R.moe_capacity(T, k, E, align)
    indptr, idx, inv = R.moe_tables(ids.numpy(), E, align, cap)
    y, g = rows_of(cap, H, dt, 6), rows_of(T, H, dt, 7)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(8))
    y[torch.from_numpy(inv < 0)] = float("nan")
    tables = [torch.as_tensor(t, dtype=torch.int32).to(DEV) for t in (idx, inv, indptr)]
    yd, _ = guarded(cap, H, dt, float("nan"))
    gd, _ = guarded(T, H, dt, float("nan"))
    yd.copy_(y)
    gd.copy_(g)
    out, out_all = guarded(T, H, dt, 7.0)
    gx, gx_all = guarded(T, H, dt, 7.0)
    gy, gy_all = guarded(cap, H, dt, 7.0)
    L.moe_unpermute(yd, tables[0], w.to(DEV), out=out)
    L.moe_permute_backward(yd, tables[0], out=gx)
    _, gw = L.moe_unpermute_backward(gd, yd, *tables, w.to(DEV), grad_rows=gy)
    L.nvfp4lora_device_status()
    for whole, n in ((out_all, T * H), (gx_all, T * H), (gy_all, cap * H)):
        assert torch.all(whole[n:] == 7)
    yn, gn, wn = f64(y), f64(g), f64(w)
    for got, wt in ((out, wn), (gx, None)):
        ref, mag = R.moe_sum(yn, idx, wt), R.moe_sum(np.abs(yn), idx, wt)
        assert np.all(np.abs(f64(got) - ref) <= sum_tolerance(ref, mag, k, dt))
    ry, rw = R.moe_unpermute_grads(gn, yn, idx, wn, np.full((cap, H), 7.0), int(indptr[-1]), inv)
    assert np.all(np.abs(f64(gy) - ry) <= sum_tolerance(ry, np.abs(ry), 1, dt))
    _, mw = R.moe_unpermute_grads(np.abs(gn), np.abs(yn), idx, wn, np.zeros((cap, H)), int(indptr[-1]), inv)
    assert np.all(np.abs(f64(gw) - rw) <= max(H, 2) * 2.0 ** -24 * mw)
    # the gradient in y's place reads the same rows that it writes
    again, gw2 = L.moe_unpermute_backward(gd, yd, *tables, w.to(DEV), grad_rows=yd)
    used = int(indptr[-1])
    assert torch.equal(again[:used], gy[:used]) and torch.equal(gw, gw2)


def test_gradients_of_fp32_rows_of_twelve_through_autograd():
    import nvfp4_block_scaled_mm_b200 as L
    T, k, E, H = 50, 2, 4, 12
    ids, x = routing(T, k, E, 3), rows_of(T, H, FP, 3)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(4))
    c = rows_of(T, H, FP, 5)
    xl, wl = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    p = L.moe_permute(xl, ids.to(DEV), E, align=4)
    (L.moe_unpermute(p.rows * p.rows, p, wl) * c.to(DEV)).sum().backward()
    # out = sum_j w_j x^2 over the active slots
    xn, cn, wn = f64(x), f64(c), f64(w) * (ids >= 0).numpy()
    gx = 2 * wn.sum(1, keepdims=True) * xn * cn
    gw = (cn * xn * xn).sum(1, keepdims=True) * (ids >= 0).numpy()
    mw = (np.abs(cn) * xn * xn).sum(1, keepdims=True) * (ids >= 0).numpy()
    # x: k terms, four roundings each and k - 1 additions (all terms of one sign); w: H terms of three roundings
    assert np.all(np.abs(f64(xl.grad) - gx) <= (4 + k) * 2.0 ** -24 * np.abs(gx))
    assert np.all(np.abs(f64(wl.grad) - gw) <= (H + 4) * 2.0 ** -24 * mw)
