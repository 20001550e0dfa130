"""Performance cases of the grouped expert products and of the experts' 4-bit weights.

Five operators on rows in expert order, expert e owning rows [offsets[e], offsets[e+1]),
at the sizes of this repository's workloads (``workloads/configs.py``) and around them:

  mm        out[p] = W[e] a[a_rows[p]]                  (W: [experts][n][k])
  dgrad     da[p] = W[e]^T dy[p]
  wgrad     dW[e] = dW_add[e] + sum of dy[p] a[a_rows[p]]^T over the expert's rows
  weights4  a weight matrix into its 4-bit form and back
  gemm4     mm with 4-bit weights (down), or silu(W0 a) * (W1 a) (gate/up)

A 4-bit weight matrix holds blocks of 32 columns: with amax the block's largest
magnitude, e = max(floor(log2 amax) - 2, -126) and every weight as the nearest of
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6} 2^e (ties to the even code, larger values to 6), two codes
a byte (the even column in the low half), the scale byte e + 127.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` the inputs,
``run(state)`` one pass (the package's kernels where ``own`` is true, else plain
torch operations), ``exact(case, seed)`` the same outputs in float64, ``work(case)``
the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases

def _rows_case(op, name, T, N, K, rho, n, k, dtype, out, spread=0.5, extra=False):
    """op on the rows of T tokens with K slots each over N experts, a fraction rho of the
    slots real: [n][k] weights, dtype inputs, out outputs. spread: unevenness of the
    experts' popularity. extra: wgrad adds to an earlier gradient; gemm4 is gate/up."""
    return {"name": name, "op": op, "T": T, "N": N, "K": K, "rho": rho, "n": n, "k": k, "dtype": dtype,
            "out": out, "spread": spread, "extra": extra}


def _pack_case(name, N, n, k, dtype):
    return {"name": name, "op": "weights4", "N": N, "n": n, "k": k, "dtype": dtype}


def listed():
    return [
        # up projection of the sparsest workload's training batch, gather fused in
        _rows_case("mm", "mm_large", 16384, 64, 8, 0.25, 1536, 2048, "bf16", "bf16"),
        # a decode step of a small batch: 16 rows, about 14 experts
        _rows_case("mm", "mm_decode", 8, 64, 2, 1.0, 768, 1024, "bf16", "bf16"),
        # ragged half-precision batch, a few experts with most of the rows
        _rows_case("mm", "mm_skewed", 3001, 60, 4, 0.5, 1016, 776, "f16", "f32", 2.0),
        # data gradient of the same large batch's down projection
        _rows_case("dgrad", "dgrad_large", 16384, 64, 8, 0.25, 2048, 1536, "bf16", "bf16"),
        # small float32 experts
        _rows_case("dgrad", "dgrad_f32", 301, 16, 6, 0.5, 520, 264, "f32", "f32"),
        # weight gradient of the same large batch, float32
        _rows_case("wgrad", "wgrad_large", 16384, 64, 8, 0.25, 1536, 2048, "bf16", "f32"),
        # the second micro-batch of a float32 step: added to the first one's gradient
        _rows_case("wgrad", "wgrad_f32", 1237, 8, 2, 0.5, 128, 64, "f32", "f32", 0.5, True),
        # a layer's gate weights into the form that is served
        _pack_case("weights4_large", 64, 1536, 2048, "bf16"),
        # one small float32 expert group
        _pack_case("weights4_small", 8, 128, 64, "f32"),
        # one token's gate/up at the sparsest workload: two experts of 64
        _rows_case("gemm4", "gemm4_token", 1, 64, 8, 0.25, 1536, 2048, "bf16", "bf16", 0.5, True),
        # a decode batch's down projection, every expert touched
        _rows_case("gemm4", "gemm4_batch", 64, 64, 8, 0.5, 2048, 1536, "bf16", "f32"),
        # odd half-precision batch, experts of very unequal popularity
        _rows_case("gemm4", "gemm4_skewed", 131, 60, 4, 0.67, 1000, 544, "f16", "f16", 2.0, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "dgrad", "wgrad", "weights4", "gemm4"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    N = rng.choice([1, 8, 16, 60, 64, 128])
    if op == "weights4":
        case = _pack_case("", N, _log_int(rng, 16, 2048), 32 * _log_int(rng, 2, 64), dtype)
        largest = 64 * 1536 * 2048 // (2 if dtype == "f32" else 1)
        while case["N"] * case["n"] * case["k"] > largest:
            case["n"] = case["n"] * 2 // 3
    else:
        K = min(N, rng.choice([1, 2, 3, 4, 6, 8]))
        rho = rng.choice([0.25, 0.5, 0.67, 1.0])
        spread = rng.choice([0.0, 0.5, 2.0])
        n = 8 * _log_int(rng, 8, 256)
        if op == "gemm4":
            case = _rows_case(op, "", _log_int(rng, 1, 256), N, K, rho, n, 32 * _log_int(rng, 2, 64), dtype,
                              rng.choice(["bf16", "f16", "f32"]), spread, rng.random() < 0.5)
        else:
            case = _rows_case(op, "", _log_int(rng, 1, 16384), N, K, rho, n, 8 * _log_int(rng, 8, 256), dtype,
                              rng.choice([dtype, "f32"]), spread, op == "wgrad" and rng.random() < 0.5)
            # float32 products run at a sixteenth of the 16-bit rate
            most = 2.0 * 32768 * 1536 * 2048 / (16 if dtype == "f32" else 1)
            while work(case)["flops"] > most:
                case["T"] = case["T"] * 2 // 3
        while N * case["n"] * case["k"] > 64 * 1536 * 2048:
            case["n"] = case["n"] // 16 * 8
    del case["name"]
    return case


def _rows(case):
    return max(1, round(case["T"] * case["K"] * case["rho"]))


def work(case):
    op, N, n, k = case["op"], case["N"], case["n"], case["k"]
    b = BYTES[case["dtype"]]
    if op == "weights4":  # weights in, codes and scales out; those in, weights out
        return {"bytes": N * n * k * 2 * b + 2 * (N * n * k // 2 + N * n * (k // BLOCK)), "flops": 4 * N * n * k}
    R, T, o = _rows(case), case["T"], BYTES[case["out"]]
    touched = N * (1 - (1 - 1 / N) ** R)  # experts with rows
    flops = 2 * R * n * k
    if op == "dgrad":
        return {"bytes": int(R * n * b + touched * n * k * b + R * k * o), "flops": flops}
    tokens = min(R, T) * k * b
    if op == "wgrad":
        return {"bytes": R * n * b + tokens + N * n * k * (o + (4 if case["extra"] else 0)), "flops": flops}
    if op == "mm":
        return {"bytes": int(tokens + touched * n * k * b + R * n * o), "flops": flops}
    pair = 2 if case["extra"] else 1
    return {"bytes": int(tokens + pair * touched * n * (k // 2 + k // BLOCK) + R * n * o), "flops": pair * flops}


# -------------------------------------------------------------------------- inputs

def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(DTYPES[dtype])


def _dispatch(case, gen):
    """Slots as the layer's routing and counting sort leave them: distinct experts a token,
    a fraction rho of the slots real, rows in expert order."""
    T, N, K = case["T"], case["N"], case["K"]
    scores = torch.randn((T, N), generator=gen, device="cuda")
    scores += case["spread"] * torch.randn((N,), generator=gen, device="cuda")
    idx = scores.topk(K, dim=1).indices
    n_real = (torch.rand((T, K), generator=gen, device="cuda") < case["rho"]).sum(1, keepdim=True)
    n_real[0] = n_real[0].clamp(min=1)
    on = torch.arange(K, device="cuda") < n_real
    expert = torch.where(on, idx, N).reshape(-1)
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=N + 1)[:N]
    offsets = torch.zeros((N + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    # rows behind the last segment name no token; entries there are never followed
    a_rows = torch.where(torch.arange(T * K, device="cuda") < offsets[N], order // K, 0)
    return offsets, a_rows.to(torch.int32), int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) + 1)
    s = {"case": case}
    op, N, n, k, dt = case["op"], case["N"], case["n"], case["k"], case["dtype"]
    if op == "weights4":
        # rows of unequal scale, as trained weights have
        scale = torch.exp(0.5 * torch.randn((N, n, 1), generator=gen, device="cuda")).to(DTYPES[dt])
        s["w"] = _normal(gen, (N, n, k), dt, 0.02) * scale
        s["codes"] = torch.zeros((N, n, k // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((N, n, k // BLOCK), dtype=torch.uint8, device="cuda")
        s["out"] = torch.zeros((N, n, k), dtype=DTYPES[dt], device="cuda")
        return s
    T, cap = case["T"], case["T"] * case["K"]
    s["offsets"], s["a_rows"], s["longest"] = _dispatch(case, gen)
    out = {"dtype": DTYPES[case["out"]], "device": "cuda"}
    if op in ("mm", "wgrad", "gemm4"):
        s["a"] = _normal(gen, (T, k), dt)
    if op in ("dgrad", "wgrad"):
        s["dy"] = _normal(gen, (cap, n), dt)
    if op in ("mm", "dgrad"):
        s["w"] = _normal(gen, (N, n, k), dt, 0.02)
    if op == "gemm4":
        for i in range(2 if case["extra"] else 1):
            s["codes%d" % i] = torch.randint(0, 256, (N, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
            s["scales%d" % i] = torch.randint(118, 123, (N, n, k // BLOCK), generator=gen, device="cuda",
                                              dtype=torch.uint8)
    if op == "wgrad":
        s["dw_add"] = _normal(gen, (N, n, k), "f32") if case["extra"] else None
        s["out"] = torch.zeros((N, n, k), **out)
    else:
        s["out"] = torch.zeros((cap, k if op == "dgrad" else n), **out)
    return s


# ---------------------------------------------------------------------- plain form

def _padded(s, rows):
    """[experts][longest segment][cols] float32 of rows in expert order (zeros behind a
    segment's end); rows(p) gives the rows at positions p."""
    off = s["offsets"].long()
    pos = off[:-1, None] + torch.arange(s["longest"], device=off.device)
    live = pos < off[1:, None]
    return torch.where(live[..., None], rows(pos.clamp(max=s["a_rows"].numel() - 1)).float(), 0.0)


def _unpadded(s, y):
    """The rows of y [experts][longest segment][cols] into s["out"]; rows behind the last
    segment stay as they were."""
    off = s["offsets"].long()
    p = torch.arange(s["a_rows"].numel(), device=off.device)
    e = torch.searchsorted(off[1:], p, right=True).clamp(max=off.numel() - 2)
    at = (e * s["longest"] + p - off[e]).clamp(max=y.shape[0] * y.shape[1] - 1)
    s["out"].copy_(torch.where((p < off[-1])[:, None], y.reshape(-1, y.shape[2])[at], s["out"].float()))
    return s["out"]


def _pack(w):
    """Blocks of 32: signed values of the 4-bit grid and the exponents they are scaled by."""
    v = w.float().reshape(*w.shape[:-1], -1, BLOCK)
    _, x = torch.frexp(v.abs().amax(-1, keepdim=True))  # amax = m 2^x, m in [1/2, 1)
    e = (x - 3).clamp(min=-126)
    m = torch.ldexp(v.abs(), -e)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign(((m / step).round() * step).clamp(max=6.0), v), e


def _values(codes, scales):
    """float32 weights that codes and scale bytes stand for."""
    grid = torch.tensor(FP4 + tuple(-v for v in FP4), device=codes.device)
    nibbles = torch.stack((codes & 15, codes >> 4), -1).reshape(*scales.shape, BLOCK)
    w = torch.ldexp(grid[nibbles.int()], scales.int()[..., None] - 127)
    return w.reshape(*codes.shape[:-1], -1)


def _plain(s):
    op = s["case"]["op"]
    if op == "weights4":
        q, e = _pack(s["w"])
        s["out"].copy_(torch.ldexp(q, e).reshape(s["w"].shape))
        return s["out"]
    if op == "dgrad":
        return _unpadded(s, torch.bmm(_padded(s, lambda p: s["dy"][p]), s["w"].float()))
    a = _padded(s, lambda p: s["a"][s["a_rows"].long()[p]])
    if op == "mm":
        return _unpadded(s, torch.bmm(a, s["w"].float().transpose(1, 2)))
    if op == "gemm4":
        y = torch.bmm(a, _values(s["codes0"], s["scales0"]).transpose(1, 2))
        if s["case"]["extra"]:
            y = y * torch.sigmoid(y) * torch.bmm(a, _values(s["codes1"], s["scales1"]).transpose(1, 2))
        return _unpadded(s, y)
    dw = torch.bmm(_padded(s, lambda p: s["dy"][p]).transpose(1, 2), a)
    if s["dw_add"] is not None:
        dw = dw + s["dw_add"]
    s["out"].copy_(dw)
    return s["out"]


def _own(s):
    import token_choice_routing_amd as tcr
    op = s["case"]["op"]
    if op == "weights4":
        tcr.moe_weights4_pack(s["w"], s["codes"], s["scales"])
        tcr.moe_weights4_unpack(s["codes"], s["scales"], s["out"])
    elif op == "mm":
        tcr.moe_grouped_mm(s["a"], s["offsets"], s["w"], s["out"], a_rows=s["a_rows"])
    elif op == "dgrad":
        tcr.moe_grouped_mm_dgrad(s["dy"], s["offsets"], s["w"], s["out"])
    elif op == "wgrad":
        tcr.moe_grouped_mm_wgrad(s["dy"], s["a"], s["offsets"], s["out"], a_rows=s["a_rows"], dw_add=s["dw_add"])
    elif s["case"]["extra"]:
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, s["a"], s["offsets"], s["codes0"], s["scales0"], s["out"],
                              s["codes1"], s["scales1"], a_rows=s["a_rows"])
    else:
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, s["a"], s["offsets"], s["codes0"], s["scales0"], s["out"],
                              a_rows=s["a_rows"])
    return s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- float64 definition

def _exact_weights4(w):
    """Values of the 4-bit form, the nearest grid value chosen by comparing with the
    midpoints (a value on a midpoint goes to the even code)."""
    out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    mids = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    for c in range(0, w.shape[-1], BLOCK):
        b = w[..., c:c + BLOCK].double()
        amax = b.abs().amax(-1, keepdim=True)
        # floor(log2 amax) is the exponent field of the float64 (0 gives -1023, clamped)
        e = (((amax.contiguous().view(torch.int64) >> 52) - 1023) - 2).clamp(min=-126)
        step = ((e + 1023) << 52).view(torch.float64)
        m = b.abs() / step
        q = torch.zeros_like(m)
        for i, mid in enumerate(mids):
            above = m >= mid if i % 2 else m > mid
            q = torch.where(above, FP4[i + 1], q)
        out[..., c:c + BLOCK] = torch.sign(b) * q * step
    return out


def _exact_values(codes, scales, e):
    """Expert e's [n][k] weights in float64."""
    c = codes[e].long()
    n = c.shape[0]
    w = torch.empty((n, 2 * c.shape[1]), dtype=torch.float64, device=c.device)
    for half in range(2):
        q = (c >> (4 * half)) & 15
        man, exp = q & 1, (q >> 1) & 3
        mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (exp - 1).double())
        w[:, half::2] = torch.where(q >= 8, -mag, mag)
    step = torch.pow(2.0, scales[e].double() - 127)
    return w * step.repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weights4":
        return _exact_weights4(s["w"])
    off = s["offsets"].tolist()
    src = s["a_rows"].long()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["N"]):
        lo, hi = off[e], off[e + 1]
        if op == "wgrad":
            if s["dw_add"] is not None:
                out[e] = s["dw_add"][e].double()
            if hi > lo:
                out[e] += s["dy"][lo:hi].double().t() @ s["a"][src[lo:hi]].double()
        elif hi > lo:
            if op == "dgrad":
                out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
                continue
            a = s["a"][src[lo:hi]].double()
            if op == "mm":
                out[lo:hi] = a @ s["w"][e].double().t()
            else:
                y = a @ _exact_values(s["codes0"], s["scales0"], e).t()
                if case["extra"]:
                    y = y / (1 + torch.exp(-y)) * (a @ _exact_values(s["codes1"], s["scales1"], e).t())
                out[lo:hi] = y
    return out
