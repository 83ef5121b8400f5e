"""What is measured of the routed-token, 8-bit product, norm and quantizer operators: the cases, their inputs, the
operators' plain forms in elementary torch operations, and the same results in 64 bits.

`own` selects between the plain forms and the package's calls."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = torch.float8_e4m3fn
TINY = 2.0 ** -100          # the smallest group maximum that a scale is formed from


def listed():
    return [
        # a decode batch of 64 tokens routed top-2 over a layer of 8 experts, rows for the grouped product
        dict(name="permute_decode", op="permute", T=64, k=2, E=8, H=4096, dtype="bf16", align=128, zero=True, train=False),
        # a training step's tokens sorted by expert for 128 experts, and the gradient of the tokens
        dict(name="permute_train", op="permute", T=8192, k=8, E=128, H=4096, dtype="bf16", align=128, zero=True, train=True),
        # a ragged prefill batch, an odd row length and no padding of the segments
        dict(name="permute_odd", op="permute", T=1777, k=6, E=60, H=1001, dtype="fp16", align=1, zero=True, train=False),
        # the experts' rows of a decode batch brought back with their weights
        dict(name="unpermute_decode", op="unpermute", T=64, k=2, E=8, H=4096, dtype="bf16", align=128, train=False),
        # a training step: the weighted sum, the gradients of the experts' rows and of the weights
        dict(name="unpermute_train", op="unpermute", T=4096, k=8, E=64, H=4096, dtype="bf16", align=128, train=True),
        # one decode step's norm in front of an 8-bit projection
        dict(name="norm_decode", op="norm", T=16, H=4096, dtype="bf16", residual=True, norm_out=False),
        # a prefill's norm, its rows kept in 16 bits for the router too
        dict(name="norm_prefill", op="norm", T=8192, H=8192, dtype="bf16", residual=True, norm_out=True),
        # the input of a down projection at a decode step
        dict(name="quantize_decode", op="quantize", T=16, H=14336, dtype="bf16", block_rows=1),
        # a projection's weights, once when a model is loaded
        dict(name="quantize_weight", op="quantize", T=28672, H=8192, dtype="bf16", block_rows=128),
        # a decode step's projection
        dict(name="mm_decode", op="mm", M=16, N=4096, K=4096, out="bf16", bias=False),
        # a short ragged prompt, no dimension a multiple of the tiles
        dict(name="mm_ragged", op="mm", M=300, N=4100, K=4112, out="fp16", bias=True),
        # a prefill's MLP-up projection
        dict(name="mm_prefill", op="mm", M=8192, N=28672, K=8192, out="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "norm", "quantize", "mm", "mm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("permute", "unpermute"):
        k = rng.randint(1, 10)
        E = max(k, _log(rng, 4, 256))
        H = _log(rng, 64, 8192)
        H = H if rng.random() < 0.3 else (H + 63) // 64 * 64
        T = _log(rng, 1, max(2, min(8192, 2 ** 27 // (H * k))))
        c = dict(op=op, T=T, k=k, E=E, H=H, dtype=dtype, align=rng.choice([1, 8, 128, 128]), train=rng.random() < 0.5)
        if op == "permute":
            c["zero"] = rng.random() < 0.7
        return c
    if op == "norm":
        H = _log(rng, 100, 16384)
        H = H if rng.random() < 0.25 else (H + 127) // 128 * 128
        return dict(op=op, T=_log(rng, 1, min(16384, 2 ** 26 // H)), H=H, dtype=dtype, residual=rng.random() < 0.7,
                    norm_out=rng.random() < 0.4)
    if op == "quantize":
        H = _log(rng, 100, 16384)
        H = H if rng.random() < 0.25 else (H + 127) // 128 * 128
        return dict(op=op, T=_log(rng, 1, min(30000, 2 ** 27 // H)), H=H, dtype=dtype, block_rows=rng.choice([1, 1, 128]))
    M, N, K = _log(rng, 1, 8192), _log(rng, 64, 28672), 16 * _log(rng, 8, 900)
    if rng.random() < 0.5:
        N, K = (N + 127) // 128 * 128, (K + 127) // 128 * 128
    return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), bias=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _capacity(c):
    """The rows that any routing of T tokens to k of E experts can need."""
    n, a = c["T"] * c["k"], c["align"]
    return (n + min(c["E"], n) * (a - 1)) // a * a


def _routing(c, g):
    """Distinct experts per token with some experts preferred, one slot in sixteen inactive, softmax weights."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 1 / 16, -1, ids).to(torch.int32)
    return ids, torch.softmax(top, dim=1).float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, dtype, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=c)
    if c["op"] in ("permute", "unpermute"):
        dt, R = DTYPES[c["dtype"]], _capacity(c)
        s["ids"], s["w"] = _routing(c, g)
        if c["op"] == "permute":
            s["x"] = rnd(c["T"], c["H"], dtype=dt)
            s["rows"] = torch.full((R, c["H"]), 0.5, dtype=dt, device="cuda")
            if c["train"]:
                s["grad_rows"] = rnd(R, c["H"], dtype=dt)
        else:
            s["indptr"], s["idx"], s["inv"] = _tables(s["ids"], c["E"], c["align"], R)
            s["y"] = rnd(R, c["H"], dtype=dt)
            if c["train"]:
                s["grad"] = rnd(c["T"], c["H"], dtype=dt)
                s["grad_y"] = torch.full((R, c["H"]), 0.5, dtype=dt, device="cuda")
    elif c["op"] == "norm":
        dt = DTYPES[c["dtype"]]
        s["x"] = rnd(c["T"], c["H"], dtype=dt)
        s["weight"] = (1 + 0.2 * torch.randn(c["H"], generator=g, device="cuda")).to(dt)
        s["residual"] = rnd(c["T"], c["H"], dtype=dt, std=2.0) if c["residual"] else None
        s["norm_out"] = torch.empty(c["T"], c["H"], dtype=dt, device="cuda") if c["norm_out"] else None
    elif c["op"] == "quantize":
        s["x"] = rnd(c["T"], c["H"], dtype=DTYPES[c["dtype"]], std=0.5)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        G = -(-K // 128)
        s["a"], s["b"] = rnd(M, K, dtype=FP8, std=100.0), rnd(N, K, dtype=FP8, std=100.0)
        s["a_scale"] = torch.rand(G, M, generator=g, device="cuda").add_(0.5).mul_(0.01).t()
        s["b_scale"] = torch.rand(-(-N // 128), G, generator=g, device="cuda").add_(0.5).mul_(0.0002)
        s["bias"] = rnd(N, dtype=torch.bfloat16) if c["bias"] else None
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def _tables(ids, E, align, R):
    """Segment bounds, the row of each slot and the slot of each row, by a stable sort of the expert ids."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    padded = (count[:E] + align - 1) // align * align
    indptr = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    first = torch.cat([count.new_zeros(1), count.cumsum(0)[:-1]])
    ks = key[order]
    row = torch.where(ks < E, indptr[ks] + torch.arange(n, device=ids.device) - first[ks], -1)
    idx = torch.empty(n, dtype=torch.long, device=ids.device).scatter_(0, order, row)
    inv = torch.full((R + 1,), -1, dtype=torch.long, device=ids.device).scatter_(0, torch.where(row < 0, R, row), order)[:R]
    return indptr.int(), idx.int().view(ids.shape), inv.int()


def _gather_sum(rows, idx, w):
    """sum_j w[t, j] * rows[idx[t, j]] over the active slots, in 32 bits."""
    on = (idx >= 0)
    got = rows[idx.clamp(min=0).long()].float()
    got = torch.where(on[..., None], got, 0.0)
    return (got if w is None else got * w[..., None]).sum(1)


def _quantize(y, block_rows):
    """e4m3 values and scales of 1 x 128 groups or 128 x 128 blocks of y (32 bits)."""
    T, H = y.shape
    G, B = -(-H // 128), -(-T // block_rows)
    p = torch.nn.functional.pad(y, (0, G * 128 - H, 0, B * block_rows - T)).view(B, block_rows, G, 128)
    amax = p.abs().amax(dim=(1, 3)).clamp(min=TINY)
    q = (p * (448.0 / amax)[:, None, :, None]).clamp(-448, 448).to(FP8)
    return q.view(B * block_rows, G * 128)[:T, :H].contiguous(), amax / 448.0


def _spread(scale, block, n):
    return scale.repeat_interleave(block, dim=-1)[..., :n]


def _plain(s):
    c = s["case"]
    if c["op"] == "permute":
        E, R = c["E"], _capacity(c)
        indptr, idx, inv = _tables(s["ids"], E, c["align"], R)
        got = s["x"][inv.clamp(min=0).long() // c["k"]]
        pad = torch.arange(R, device=inv.device) < indptr[E]
        fill = torch.where(pad[:, None], 0.0, s["rows"]) if c["zero"] else s["rows"]
        s["rows"].copy_(torch.where((inv >= 0)[:, None], got, fill))
        out = [s["rows"], indptr, idx, inv]
        if c["train"]:
            out.append(_gather_sum(s["grad_rows"], idx, None).to(s["x"].dtype))
        return out
    if c["op"] == "unpermute":
        out = [_gather_sum(s["y"], s["idx"], s["w"]).to(s["y"].dtype)]
        if c["train"]:
            on, idx = s["idx"] >= 0, s["idx"].clamp(min=0).long()
            grad, R, k = s["grad"].float(), s["y"].shape[0], c["k"]
            gw = torch.where(on, (s["y"][idx].float() * grad[:, None]).sum(2), 0.0)
            slot = s["inv"].clamp(min=0).long()
            gy = (grad[slot // k] * s["w"].reshape(-1)[slot][:, None]).to(s["y"].dtype)
            used = torch.arange(R, device=idx.device) < s["indptr"][c["E"]]
            keep = torch.where(used[:, None], 0.0, s["grad_y"])
            s["grad_y"].copy_(torch.where((s["inv"] >= 0)[:, None], gy, keep))
            out += [s["grad_y"], gw]
        return out
    if c["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
            s["residual"].copy_(h)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * s["weight"].float()
        out = list(_quantize(y, 1)) + ([s["residual"]] if s["residual"] is not None else [])
        if s["norm_out"] is not None:
            out.append(s["norm_out"].copy_(y))
        return out
    if c["op"] == "quantize":
        return list(_quantize(s["x"].float(), c["block_rows"]))
    M, N, K = c["M"], c["N"], c["K"]
    a = s["a"].float() * _spread(s["a_scale"], 128, K)
    b = s["b"].float() * _spread(s["b_scale"], 128, K).repeat_interleave(128, dim=0)[:N]
    out = a @ b.t()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return out.to(DTYPES[c["out"]])


def _calls(s):
    import nvfp4_block_scaled_mm_b200 as L
    c = s["case"]
    if c["op"] == "permute":
        p = L.moe_permute(s["x"], s["ids"], c["E"], align=c["align"], zero_padding=c["zero"], out=s["rows"])
        out = [p.rows, p.m_indptr, p.expanded_idx_to_permuted_idx, p.permuted_idx_to_expanded_idx]
        if c["train"]:
            out.append(L.moe_permute_backward(s["grad_rows"], p.expanded_idx_to_permuted_idx))
        return out
    if c["op"] == "unpermute":
        out = [L.moe_unpermute(s["y"], s["idx"], s["w"])]
        if c["train"]:
            out += L.moe_unpermute_backward(s["grad"], s["y"], s["idx"], s["inv"], s["indptr"], s["w"], grad_rows=s["grad_y"])
        return out
    if c["op"] == "norm":
        out = list(L.add_rmsnorm_fp8_quantize(s["x"], s["weight"], s["residual"], eps=1e-6, norm_out=s["norm_out"]))
        return out + [t for t in (s["residual"], s["norm_out"]) if t is not None]
    if c["op"] == "quantize":
        return list(L.fp8_quantize(s["x"], block_rows=c["block_rows"]))
    return L.mm_fp8(s["a"], s["b"], s["a_scale"], s["b_scale"], bias=s["bias"], out_dtype=DTYPES[c["out"]])


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ---------------------------------------------------------------------------------------------------------------
# work, and the results in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("permute", "unpermute"):
        size = 4 if c["dtype"] == "fp32" else 2
        n, row = c["T"] * c["k"], c["H"] * size
        # the expected share of active slots; padding rows are not counted
        act = n * 15 / 16
        if c["op"] == "permute":
            b = c["T"] * row + act * row + 4 * (2 * n + _capacity(c) + c["E"] + 1)
            return dict(bytes=b + ((act + c["T"]) * row + 4 * n if c["train"] else 0), flops=act * c["H"] if c["train"] else 0)
        b = act * row + c["T"] * row + 8 * n
        f = 2 * act * c["H"]
        if c["train"]:
            b += c["T"] * row + 2 * act * row + 12 * n + 4 * _capacity(c)
            f += 3 * act * c["H"]
        return dict(bytes=b, flops=f)
    if c["op"] in ("norm", "quantize"):
        size = 4 if c["dtype"] == "fp32" else 2
        n = c["T"] * c["H"]
        scales = 4 * -(-c["T"] // c.get("block_rows", 1)) * -(-c["H"] // 128)
        if c["op"] == "quantize":
            return dict(bytes=n * (size + 1) + scales, flops=3 * n)
        b = n * (size + 1 + (2 * size if c["residual"] else 0) + (size if c["norm_out"] else 0)) + scales + c["H"] * size
        return dict(bytes=b, flops=8 * n)
    M, N, K = c["M"], c["N"], c["K"]
    G = -(-K // 128)
    b = M * K + N * K + 4 * (M * G + -(-N // 128) * G) + M * N * (4 if c["out"] == "fp32" else 2) + (2 * N if c["bias"] else 0)
    return dict(bytes=b, flops=2 * M * N * K)


def _exact_tables(ids, E, align, R):
    """The tables by counting, for each slot, the earlier slots of its expert."""
    flat = ids.reshape(-1).long()
    hot = flat[:, None] == torch.arange(E, device=ids.device)
    before = hot.int().cumsum(0) - hot.int()
    total = hot.sum(0)
    seg = torch.div(total + align - 1, align, rounding_mode="floor") * align
    end = seg.cumsum(0)
    idx = (hot * (before + (end - seg))).sum(1).where(hot.any(1), torch.tensor(-1, device=ids.device))
    inv = torch.full((R,), -1, dtype=torch.long, device=ids.device)
    inv[idx[idx >= 0]] = torch.nonzero(idx >= 0).reshape(-1)
    return torch.cat([end.new_zeros(1), end]), idx.view(ids.shape), inv


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("permute", "unpermute"):
        E, R, k = c["E"], _capacity(c), c["k"]
        indptr, idx, inv = _exact_tables(s["ids"], E, c["align"], R)
        at = torch.nonzero(inv >= 0).reshape(-1)
        last = int(indptr[E])
        if c["op"] == "permute":
            rows = s["rows"].double()
            if c["zero"]:
                rows[:last] = 0
            rows[at] = s["x"].double()[inv[at] // k]
            out = [rows, None, None, None]
            if c["train"]:
                gx = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
                for j in range(k):
                    on = idx[:, j] >= 0
                    gx[on] += s["grad_rows"][idx[on, j]].double()
                out.append(gx)
            return out
        total = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        gw = torch.zeros(c["T"], k, dtype=torch.float64, device="cuda")
        for j in range(k):
            on = idx[:, j] >= 0
            got = s["y"][idx[on, j]].double()
            total[on] += got * s["w"][on, j, None].double()
            if c["train"]:
                gw[on, j] = torch.einsum("th,th->t", got, s["grad"][on].double())
        if not c["train"]:
            return [total]
        gy = s["grad_y"].double()
        gy[:last] = 0
        gy[at] = s["grad"].double()[inv[at] // k] * s["w"].double().view(-1)[inv[at], None]
        return [total, gy, gw]
    if c["op"] in ("norm", "quantize"):
        y, more = s["x"].double(), []
        if c["op"] == "norm":
            if s["residual"] is not None:
                y = y + s["residual"].double()
                more.append(y)
            rms = (torch.linalg.vector_norm(y, dim=1, keepdim=True).square() / c["H"] + 1e-6).sqrt()
            y = y / rms * s["weight"].double()
            if s["norm_out"] is not None:
                more.append(y)
        T, H = y.shape
        rows = c.get("block_rows", 1)
        amax = torch.zeros(-(-T // rows), -(-H // 128), dtype=torch.float64, device="cuda")
        where = (torch.arange(T, device="cuda")[:, None] // rows) * amax.shape[1] + torch.arange(H, device="cuda") // 128
        amax.view(-1).scatter_reduce_(0, where.reshape(-1), y.abs().reshape(-1), "amax")
        amax.clamp_(min=TINY)
        return [y * 448 / amax.view(-1)[where], amax / 448] + more
    M, N, K = c["M"], c["N"], c["K"]
    block = torch.arange(K, device="cuda") // 128
    a = s["a"].to(torch.float64).mul_(s["a_scale"].double().index_select(1, block))
    b = s["b"].to(torch.float64).mul_(s["b_scale"].double()[torch.arange(N, device="cuda") // 128][:, block])
    out = torch.mm(a, b.t())
    return out if s["bias"] is None else out + s["bias"].double()
