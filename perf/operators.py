"""Performance cases of the dispatch gradients and of the 8-bit activation checkpoints.

Five operators around the experts of a token-choice layer, at the sizes of this
repository's workloads (``workloads/configs.py``) and around them:

  combine           y_t = ys_t + sum_k w_tk r_tk over the token's slots, r_tk the
                    expert row of a real slot, the null source of a null slot
  combine_backward  dy_perm[p] = w_tk dy_t, dw_tk = <dy_t, r_tk>, the null source's
                    gradient, and each expert row's weight and slot
  permute_backward  dx_t = add_t + sum_k dx_perm[slot_pos_tk] over the real slots
  act8              a tensor into its 8-bit checkpoint and back
  swiglu8           a SwiGLU that keeps gate and up in 8 bits, and its backward pass

A checkpoint holds blocks of 32 columns (the last of a row may be shorter): with
amax the block's largest magnitude, e = max(floor(log2 amax) - 6, -126) and codes
q = clamp(rint(v 2^-e), -127, 127), which stand for q 2^e.

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


# --------------------------------------------------------------------------- cases

def _routing_case(op, name, T, d, N, K, rho, dtype, rows, null, extra=False):
    """op on T tokens of d columns: K slots a token over N experts, a fraction rho of
    the slots real; dtype: activations, rows: expert rows; null: what a null slot
    outputs; extra: a shared expert's output (combine) or a gradient added in
    (permute_backward)."""
    return {"name": name, "op": op, "T": T, "d": d, "N": N, "K": K, "rho": rho, "dtype": dtype,
            "rows": rows, "null": null, "extra": extra}


def _act_case(op, name, rows, live, cols, dtype, weighted=False):
    """op on live of rows rows of cols columns; weighted (swiglu8): the rows carry
    routing weights, whose gradient the backward returns."""
    return {"name": name, "op": op, "rows": rows, "live": live, "cols": cols, "dtype": dtype,
            "weighted": weighted}


def listed():
    return [
        # one decode step of a small batch, shared expert: latency
        _routing_case("combine", "combine_decode", 8, 1024, 64, 2, 1.0, "bf16", "bf16", "zero", True),
        # the training batch of the sparsest workload (8 of 64 + 192, a quarter real), shared expert
        _routing_case("combine", "combine_large", 16384, 2048, 64, 8, 0.25, "bf16", "bf16", "zero", True),
        # ragged float32 batch, half-precision experts, null slots that copy the token
        _routing_case("combine", "combine_copy_f32", 1237, 1032, 60, 6, 0.5, "f32", "f16", "copy"),
        # gradients of the same large batch
        _routing_case("combine_backward", "combine_backward_large", 16384, 2048, 64, 8, 0.25, "bf16", "bf16", "zero"),
        # constant null expert: its vector's gradient sums over all tokens
        _routing_case("combine_backward", "combine_backward_constant", 2047, 1024, 64, 4, 0.5, "bf16", "f32",
                      "constant"),
        # the last few tokens of a batch, float32, copied tokens
        _routing_case("combine_backward", "combine_backward_small", 5, 520, 16, 4, 0.5, "f32", "f32", "copy"),
        # float32 gradients, shared expert's added in, half of four slots real
        _routing_case("permute_backward", "permute_backward_large", 8192, 1024, 64, 4, 0.5, "f32", "f32", "zero",
                      True),
        # odd batch with every slot real, bf16 gradients in and out
        _routing_case("permute_backward", "permute_backward_dense", 1001, 1016, 64, 2, 1.0, "bf16", "bf16", "zero"),
        # a layer's input kept over the forward pass
        _act_case("act8", "act8_large", 16384, 16384, 2048, "bf16"),
        # a few float32 rows, the last block of each row short
        _act_case("act8", "act8_small", 13, 13, 1032, "f32"),
        # the routed experts' activations of the large batch: rows sized for more than are live
        _act_case("swiglu8", "swiglu8_large", 40960, 32768, 1536, "bf16", True),
        # one small float32 expert, ragged
        _act_case("swiglu8", "swiglu8_small", 77, 77, 776, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine", "combine_backward", "permute_backward", "act8", "swiglu8"])
    if op in ("act8", "swiglu8"):
        cols = 8 * _log_int(rng, 8, 256)
        most = 16384 * 2048 if op == "act8" else 32768 * 1536
        dtype = rng.choice(["bf16", "f16", "f32"])
        if dtype == "f32":
            most //= 2
        live = _log_int(rng, 1, min(65536, most // cols))
        rows = live + rng.choice([0, rng.randrange(1, live // 4 + 2)])
        case = _act_case(op, "", rows, live, cols, dtype, op == "swiglu8" and rng.random() < 0.5)
    else:
        T = _log_int(rng, 1, 16384)
        K = rng.choice([1, 2, 3, 4, 6, 8])
        N = rng.choice([8, 16, 60, 64, 128])
        rho = rng.choice([0.25, 0.5, 0.67, 1.0])
        dtype = rng.choice(["bf16", "f32"])
        rows = rng.choice(["bf16", "f32", "f16"])
        null = "zero" if op == "permute_backward" else rng.choice(["zero", "copy", "constant"])
        d = 8 * _log_int(rng, 8, 256)
        case = _routing_case(op, "", T, d, N, K, rho, dtype, rows, null, op != "combine_backward" and rng.random() < 0.5)
        largest = {c["op"]: work(c)["bytes"] for c in listed() if c["name"].endswith("_large")}[op]
        while work(case)["bytes"] > largest:
            case["T"] = case["T"] * 2 // 3
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op in ("act8", "swiglu8"):
        n, b = case["live"] * case["cols"], BYTES[case["dtype"]]
        kept = case["live"] * (case["cols"] + -(-case["cols"] // BLOCK))
        if op == "act8":  # tensor in, checkpoint out; checkpoint in, tensor out
            return {"bytes": 2 * n * b + 2 * kept, "flops": 4 * n}
        # g, u in, h and two checkpoints out; the checkpoints and dh in, dg, du and h out
        rows = 8 * case["live"] if case["weighted"] else 0
        return {"bytes": 7 * n * b + 4 * kept + rows, "flops": 30 * n}
    T, d, K = case["T"], case["d"], case["K"]
    R = round(T * K * case["rho"])
    e, r = BYTES[case["dtype"]], BYTES[case["rows"]]
    copied = T * d * e if case["null"] == "copy" else d * e if case["null"] == "constant" else 0
    if op == "combine":
        shared = T * d * r if case["extra"] else 0
        return {"bytes": R * d * r + T * d * e + T * K * 8 + shared + copied, "flops": 2 * R * d}
    if op == "combine_backward":
        dnull = {"zero": 0, "copy": T * d * 4, "constant": d * 4}[case["null"]]
        return {"bytes": T * d * e + 2 * R * d * r + T * K * 12 + R * 8 + copied + dnull, "flops": 3 * R * d}
    return {"bytes": R * d * r + T * d * (e + (4 if case["extra"] else 0)) + T * K * 4, "flops": R * d}


# -------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) + 1)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(DTYPES[dtype])


def _routing(case, gen):
    """Slots as the layer's routing and counting sort leave them: r_t reals first
    (binomial, mean rho K, so some tokens have none), experts of unequal popularity,
    positions in expert order, weights over the chosen entries."""
    T, N, K, rho = case["T"], case["N"], case["K"], case["rho"]
    scores = torch.randn((T, N), generator=gen, device="cuda") + 0.5 * torch.randn((N,), generator=gen, device="cuda")
    top, idx = scores.topk(K, dim=1)
    real = torch.rand((T, K), generator=gen, device="cuda") < rho
    n_real = real.sum(1, keepdim=True)
    slot = torch.arange(K, device="cuda").expand(T, K)
    on = slot < n_real
    if case["null"] == "zero":
        w = torch.where(on, torch.softmax(torch.where(on, top, float("-inf")), 1), 0.0)
    else:
        w = torch.softmax(torch.where(on, top, 0.0), 1)
    w = torch.where(on.any(1, keepdim=True) | (case["null"] != "zero"), w, 0.0).float().contiguous()
    expert = torch.where(on, idx, N).reshape(-1)
    order = torch.argsort(expert, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * K, device="cuda")
    slot_pos = torch.where(on, pos.reshape(T, K), -1).to(torch.int32).contiguous()
    return slot_pos, w


def prepare(case, seed):
    gen = _generator(seed)
    s = {"case": case}
    if case["op"] in ("act8", "swiglu8"):
        rows, cols, dt = case["rows"], case["cols"], case["dtype"]
        like = {"device": "cuda"}
        s["n_rows"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
        names = ("x",) if case["op"] == "act8" else ("g", "u", "dh")
        for n in names:
            # columns of unequal spread, as activations have
            spread = torch.exp(0.5 * torch.randn((cols,), generator=gen, device="cuda")).to(DTYPES[dt])
            s[n] = _normal(gen, (rows, cols), dt) * spread
        outs = ("out",) if case["op"] == "act8" else ("h", "dg", "du", "h8")
        for n in outs:
            s[n] = torch.zeros((rows, cols), dtype=DTYPES[dt], **like)
        for n in names[:2] if case["op"] == "swiglu8" else names:
            s[n + "_codes"] = torch.zeros((rows, cols), dtype=torch.int8, **like)
            s[n + "_scales"] = torch.zeros((rows, -(-cols // BLOCK)), dtype=torch.uint8, **like)
        if case["weighted"]:
            s["w"] = torch.rand((rows,), generator=gen, **like)
            s["dw"] = torch.zeros((rows,), **like)
        return s
    T, d, K = case["T"], case["d"], case["K"]
    cap = T * K
    s["slot_pos"], s["topk_w"] = _routing(case, gen)
    out = {"dtype": DTYPES[case["dtype"]], "device": "cuda"}
    s["null_src"] = None
    if case["null"] != "zero":
        s["null_src"] = _normal(gen, (T, d) if case["null"] == "copy" else (d,), case["dtype"])
    s["rows"] = _normal(gen, (cap, d), case["rows"])
    if case["op"] == "combine":
        s["shared"] = _normal(gen, (T, d), case["rows"]) if case["extra"] else None
        s["y"] = torch.zeros((T, d), **out)
    elif case["op"] == "combine_backward":
        s["dy"] = _normal(gen, (T, d), case["dtype"])
        s["dy_perm"] = torch.zeros((cap, d), dtype=DTYPES[case["rows"]], device="cuda")
        s["w_perm"] = torch.zeros((cap,), device="cuda")
        s["row_slot"] = torch.zeros((cap,), dtype=torch.int32, device="cuda")
        s["dtopk_w"] = torch.zeros((T, K), device="cuda")
        s["dnull"] = None
        if case["null"] != "zero":
            s["dnull"] = torch.zeros(s["null_src"].shape, device="cuda")
    else:
        s["add"] = _normal(gen, (T, d), "f32") if case["extra"] else None
        s["dx"] = torch.zeros((T, d), **out)
    if own:
        import token_choice_routing_amd as tcr
        kinds = {"zero": tcr.MOE_NULL_ZERO, "copy": tcr.MOE_NULL_COPY, "constant": tcr.MOE_NULL_CONSTANT}
        # null copies enough for any token to have none but null slots
        s["dims"] = tcr.make_dims(T, d, case["N"], K, K, 8, 0,
                                  tcr.MOE_BF16 if case["dtype"] == "bf16" else tcr.MOE_F32, kinds[case["null"]])
        if case["op"] == "combine_backward":
            need = tcr.workspace_bytes(s["dims"], tcr.MOE_WS_COMBINE_BACKWARD)
            s["ws"] = torch.empty((max(need, 256),), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------- plain form

def _blocks(v):
    """[rows][cols] -> [rows][blocks][32], zeros past the last column."""
    rows, cols = v.shape
    pad = -cols % BLOCK
    return torch.nn.functional.pad(v, (0, pad)).reshape(rows, -1, BLOCK)


def _pack(v):
    v = _blocks(v.float())
    _, k = torch.frexp(v.abs().amax(2, keepdim=True))  # amax = m 2^k, m in [1/2, 1)
    e = (k - 7).clamp(min=-126)
    return torch.ldexp(v, -e).round().clamp(-127, 127).to(torch.int8), e


def _unpack(codes, e, cols):
    return torch.ldexp(codes.float(), e).reshape(codes.shape[0], -1)[:, :cols]


def _slot_rows(s, T, K, d):
    """[T][K][d] float32 rows of the slots and which of them are real."""
    real = s["slot_pos"] >= 0
    rows = s["rows"][s["slot_pos"].clamp(min=0).long()].float()
    if s["null_src"] is None:
        rows = torch.where(real[..., None], rows, 0.0)
    else:
        rows = torch.where(real[..., None], rows, s["null_src"].float().reshape(-1, 1, d))
    return rows, real


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "act8":
        n = case["live"]
        s["out"][:n] = _unpack(*_pack(s["x"][:n]), case["cols"]).to(s["out"].dtype)
        return s["out"]
    if op == "swiglu8":
        n, F, dt = case["live"], case["cols"], s["h"].dtype
        g, u, dh = s["g"][:n], s["u"][:n], s["dh"][:n].float()
        s["h"][:n] = (g.float() * torch.sigmoid(g.float()) * u.float()).to(dt)
        z, v = _unpack(*_pack(g), F), _unpack(*_pack(u), F)
        sig = torch.sigmoid(z)
        h = z * sig * v
        if case["weighted"]:
            s["dw"][:n] = (dh * h).sum(1)
            dh = dh * s["w"][:n, None]
        s["dg"][:n] = (dh * v * sig * (1 + z * (1 - sig))).to(dt)
        s["du"][:n] = (dh * z * sig).to(dt)
        s["h8"][:n] = h.to(dt)
        out = {k: s[k] for k in ("h", "dg", "du", "h8")}
        if case["weighted"]:
            out["dw"] = s["dw"]
        return out
    T, K, d = case["T"], case["K"], case["d"]
    rows, real = _slot_rows(s, T, K, d)
    if op == "combine":
        y = (s["topk_w"][..., None] * rows).sum(1)
        if s["shared"] is not None:
            y = y + s["shared"].float()
        s["y"].copy_(y)
        return s["y"]
    if op == "permute_backward":
        dx = rows.sum(1)
        if s["add"] is not None:
            dx = dx + s["add"]
        s["dx"].copy_(dx)
        return s["dx"]
    dy, w = s["dy"].float(), s["topk_w"]
    s["dtopk_w"].copy_((rows * dy[:, None]).sum(2))
    t, k = real.nonzero(as_tuple=True)
    p = s["slot_pos"][t, k].long()
    s["dy_perm"][p] = (w[t, k][:, None] * dy[t]).to(s["dy_perm"].dtype)
    s["w_perm"][p] = w[t, k]
    s["row_slot"][p] = (t * K + k).to(torch.int32)
    out = {n: s[n] for n in ("dy_perm", "w_perm", "row_slot", "dtopk_w")}
    if s["dnull"] is not None:
        wn = torch.where(real, 0.0, w).sum(1, keepdim=True)
        if case["null"] == "copy":
            s["dnull"].copy_(wn * dy)
        else:  # a sum over every token
            s["dnull"].copy_((wn.double() * dy.double()).sum(0))
        out["dnull"] = s["dnull"]
    return out


def _own(s):
    import token_choice_routing_amd as tcr
    codes = {"bf16": tcr.MOE_BF16, "f16": tcr.MOE_F16, "f32": tcr.MOE_F32}
    case = s["case"]
    op = case["op"]
    if op == "act8":
        tcr.moe_act8_pack(s["x"], s["x_codes"], s["x_scales"], n_rows=s["n_rows"])
        tcr.moe_act8_unpack(s["x_codes"], s["x_scales"], s["out"], n_rows=s["n_rows"])
        return s["out"]
    if op == "swiglu8":
        kept = (s["g_codes"], s["g_scales"], s["u_codes"], s["u_scales"])
        tcr.moe_swiglu_keep8(s["g"], s["u"], s["h"], *kept, n_rows=s["n_rows"])
        out = {k: s[k] for k in ("h", "dg", "du", "h8")}
        if case["weighted"]:
            out["dw"] = s["dw"]
            tcr.moe_swiglu_backward8(*kept, s["dh"], s["dg"], s["du"], h=s["h8"], w_rows=s["w"], dw=s["dw"],
                                     n_rows=s["n_rows"])
        else:
            tcr.moe_swiglu_backward8(*kept, s["dh"], s["dg"], s["du"], h=s["h8"], n_rows=s["n_rows"])
        return out
    if op == "combine":
        tcr.moe_combine_rows(s["dims"], codes[case["rows"]], s["rows"], s["slot_pos"], s["topk_w"], s["shared"],
                             s["y"], null_src=s["null_src"])
        return s["y"]
    if op == "permute_backward":
        tcr.moe_permute_backward(s["dims"], codes[case["rows"]], s["rows"], s["slot_pos"], s["add"],
                                 codes[case["dtype"]], s["dx"])
        return s["dx"]
    tcr.moe_combine_backward(s["dims"], codes[case["rows"]], s["dy"], s["rows"], s["slot_pos"], s["topk_w"],
                             s["dy_perm"], s["w_perm"], s["row_slot"], s["dtopk_w"], null_src=s["null_src"],
                             dnull=s["dnull"], ws=s["ws"])
    out = {n: s[n] for n in ("dy_perm", "w_perm", "row_slot", "dtopk_w")}
    if s["dnull"] is not None:
        out["dnull"] = s["dnull"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- float64 definition

def _exact_kept(v):
    """The values a checkpoint of v stands for, block by block along the columns."""
    v = v.double()
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        amax = b.abs().max(1, keepdim=True).values
        # floor(log2 amax) is the exponent field of the float64 (0 gives -1023, clamped)
        e = (amax.contiguous().view(torch.int64) >> 52) - 1023
        step = ((e - 6).clamp(min=-126) + 1023 << 52).view(torch.float64)
        out[:, c:c + BLOCK] = torch.clamp(torch.round(b / step), -127, 127) * step
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("act8", "swiglu8"):
        n = case["live"]

        def whole(v):  # rows behind the live ones stay as they were
            o = torch.zeros((case["rows"],) + tuple(v.shape[1:]), dtype=torch.float64, device=v.device)
            o[:n] = v
            return o

        if op == "act8":
            return whole(_exact_kept(s["x"][:n]))
        g, u, dh = (s[k][:n].double() for k in ("g", "u", "dh"))
        out = {"h": whole(g / (1 + torch.exp(-g)) * u)}
        g, u = _exact_kept(g), _exact_kept(u)
        q = 1 / (1 + torch.exp(-g))
        w = s["w"][:n, None].double() if case["weighted"] else 1.0
        # d silu(z)/dz = q + z q (1 - q)
        out["dg"] = whole(w * dh * u * (q + g * q * (1 - q)))
        out["du"] = whole(w * dh * (g * q))
        out["h8"] = whole(g * q * u)
        if case["weighted"]:
            out["dw"] = whole((dh * (g * q) * u).sum(1))
        return out
    T, K, d = case["T"], case["K"], case["d"]
    pos, w = s["slot_pos"].long(), s["topk_w"].double()
    src = None if s["null_src"] is None else s["null_src"].double().expand(T, d)

    def slot(k):  # rows of slot k of every token
        on = (pos[:, k] >= 0)[:, None]
        r = s["rows"][pos[:, k].clamp(min=0)].double()
        return torch.where(on, r, torch.zeros_like(r) if src is None else src)

    if op == "combine":
        y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
        if s["shared"] is not None:
            y += s["shared"].double()
        for k in range(K):
            y += w[:, k:k + 1] * slot(k)
        return y
    if op == "permute_backward":
        dx = torch.zeros((T, d), dtype=torch.float64, device="cuda")
        if s["add"] is not None:
            dx += s["add"].double()
        for k in range(K):
            dx += slot(k)
        return dx
    dy = s["dy"].double()
    out = {"dy_perm": torch.zeros((T * K, d), dtype=torch.float64, device="cuda"),
           "w_perm": torch.zeros((T * K,), dtype=torch.float64, device="cuda"),
           "row_slot": torch.zeros((T * K,), dtype=torch.int32, device="cuda"),
           "dtopk_w": torch.zeros((T, K), dtype=torch.float64, device="cuda")}
    wn = torch.zeros((T, 1), dtype=torch.float64, device="cuda")
    for k in range(K):
        out["dtopk_w"][:, k] = (dy * slot(k)).sum(1)
        t = torch.nonzero(pos[:, k] >= 0).flatten()
        p = pos[t, k]
        out["dy_perm"][p] = w[t, k][:, None] * dy[t]
        out["w_perm"][p] = w[t, k]
        out["row_slot"][p] = (t * K + k).to(torch.int32)
        wn += torch.where(pos[:, k:k + 1] < 0, w[:, k:k + 1], 0.0)
    if case["null"] == "copy":
        out["dnull"] = wn * dy
    elif case["null"] == "constant":
        out["dnull"] = (wn * dy).sum(0)
    return out
