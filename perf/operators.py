"""Cases of the block norms, the gradient norm with clipping and the 8-bit
integer linear: their inputs, their plain form in elementary torch operations,
their definition in 64 bits, and the bytes and operations each cannot do
without.

`own` selects between the plain form (False) and the library's calls (True).
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the norms between two blocks while generating: a handful of tokens, latency only
        {"name": "norm_fwd_4x8192", "op": "norm_fwd", "M": 4, "D": 8192, "x": "bf16", "h": "bf16", "y": "bf16",
         "w": "bf16", "post": True, "pre": True, "gate_rows": 0, "alpha": 1.0, "offset": 0.0},
        # the same during training of the 70B-shaped layer: 4 sequences of 2048 tokens, a gate per sequence
        {"name": "norm_fwd_8192x8192", "op": "norm_fwd", "M": 8192, "D": 8192, "x": "bf16", "h": "bf16", "y": "bf16",
         "w": "bf16", "post": True, "pre": True, "gate_rows": 2048, "alpha": 1.0, "offset": 1.0},
        # an odd width and a ragged last group, fp32 residual stream
        {"name": "norm_fwd_1001x2051", "op": "norm_fwd", "M": 1001, "D": 2051, "x": "f32", "h": "bf16", "y": "bf16",
         "w": "f32", "post": True, "pre": True, "gate_rows": 1001, "alpha": 0.5, "offset": 0.0},
        # backward of a short sequence with frozen norms (QLoRA trains the adapters only)
        {"name": "norm_bwd_64x4096_frozen", "op": "norm_bwd", "M": 64, "D": 4096, "x": "bf16", "h": "bf16",
         "y": "f32", "w": "bf16", "post": True, "pre": True, "gate_rows": 0, "alpha": 1.0, "offset": 0.0,
         "train": False},
        # backward of the 7B-shaped MLP's tokens, all norm weights and a gate trained, dy in fp32 as the linears give it
        {"name": "norm_bwd_8192x4096", "op": "norm_bwd", "M": 8192, "D": 4096, "x": "bf16", "h": "bf16", "y": "f32",
         "w": "bf16", "post": True, "pre": True, "gate_rows": 8192, "alpha": 1.0, "offset": 0.0, "train": True},
        # clipping the adapter gradients of one linear
        {"name": "clip_1_layer_r8", "op": "clip", "layers": 1, "hidden": 512, "ffn": 1408, "r": 8, "dt": "f32",
         "max_norm": 0.1},
        # clipping all adapter gradients of a 7B-shaped model: 448 tensors, 160 M values
        {"name": "clip_32_layers_r64", "op": "clip", "layers": 32, "hidden": 4096, "ffn": 11008, "r": 64, "dt": "f32",
         "max_norm": 0.3},
        # the optimizer step of a small adapter with clipping
        {"name": "adamw_2_layers_r8", "op": "adamw", "layers": 2, "hidden": 1024, "ffn": 2731, "r": 8, "dt": "f32",
         "max_norm": 1.0},
        # the optimizer step of the 7B-shaped model's adapters with clipping
        {"name": "adamw_32_layers_r64", "op": "adamw", "layers": 32, "hidden": 4096, "ffn": 11008, "r": 64,
         "dt": "f32", "max_norm": 0.3},
        # an 8-bit linear while generating: bound by reading the weight
        {"name": "int8_8x28672x8192", "op": "int8", "M": 8, "N": 28672, "K": 8192, "x": "bf16", "y": "bf16"},
        # a ragged prompt through the 7B-shaped gate linear
        {"name": "int8_519x11008x4096", "op": "int8", "M": 519, "N": 11008, "K": 4096, "x": "bf16", "y": "f32"},
        # the 70B-shaped gate linear over 2048 tokens: bound by the tensor cores
        {"name": "int8_2048x28672x8192", "op": "int8", "M": 2048, "N": 28672, "K": 8192, "x": "bf16", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "clip", "adamw", "int8"])
    if op.startswith("norm"):
        D = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        M = _log(rng, 1, min(16384, 2 ** 25 // D))
        case = {"op": op, "M": M, "D": D, "x": rng.choice(["bf16", "f32"]), "h": rng.choice(["bf16", "bf16", "f32"]),
                "y": rng.choice(["bf16", "f32"]), "w": rng.choice(["bf16", "f32"]), "post": rng.random() < 0.7,
                "pre": rng.random() < 0.85, "gate_rows": rng.choice([0, M, _log(rng, 1, M)]),
                "alpha": rng.choice([1.0, 0.5, 1.25]), "offset": rng.choice([0.0, 1.0])}
        if op == "norm_bwd":
            case["train"] = rng.random() < 0.6
        return case
    if op in ("clip", "adamw"):
        hidden = _log(rng, 64, 8192)
        ffn = int(hidden * rng.uniform(1.3, 3.5))
        r = rng.choice([1, 3, 8, 16, 32, 64])
        per_layer = r * (11 * hidden + 3 * ffn)
        layers = _log(rng, 1, max(1, min(80, 120_000_000 // per_layer)))
        return {"op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "r": r,
                "dt": "f32" if op == "adamw" else rng.choice(["f32", "bf16"]),
                "max_norm": rng.choice([0.3, 1.0, 1e6])}
    K = 16 * _log(rng, 4, 1792)
    N = _log(rng, 1, 28672)
    M = _log(rng, 1, max(1, min(4096, 2 ** 38 // (N * K))))
    return {"op": op, "M": M, "N": N, "K": K, "x": rng.choice(["bf16", "bf16", "f32"]), "y": rng.choice(["bf16", "f32"])}


def _groups(case):
    """Rows that share one gate, and how many gates there are."""
    rows = case["gate_rows"]
    return rows, (-(-case["M"] // rows) if rows else 0)


def _adapter_sizes(case):
    """Numbers of values of the adapter gradients of `layers` decoder layers: dA and dB of seven linears."""
    r, hidden, ffn = case["r"], case["hidden"], case["ffn"]
    layer = [r * hidden, hidden * r] * 4 + [r * hidden, ffn * r] * 2 + [r * ffn, hidden * r]
    return layer * case["layers"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def normal(*shape, scale=1.0, dtype="f32"):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(DTYPES[dtype])

    if op.startswith("norm"):
        M, D = case["M"], case["D"]
        rows, G = _groups(case)
        # a residual stream has a few channels far larger than the others
        wide = torch.ones(D, device=dev)
        wide[torch.randint(0, D, (max(1, D // 512),), generator=gen, device=dev)] = 20.0
        stream = (torch.randn(M, D, generator=gen, device=dev) * wide).to(DTYPES[case["x"]])
        s["x"] = stream
        s["h"] = normal(M, D, scale=0.5, dtype=case["h"])
        centre = 1.0 - case["offset"]
        s["w_pre"] = (centre + 0.1 * torch.randn(D, generator=gen, device=dev)).to(DTYPES[case["w"]]) if case["pre"] else None
        s["w_post"] = (centre + 0.1 * torch.randn(D, generator=gen, device=dev)).to(DTYPES[case["w"]]) if case["post"] else None
        s["gate"] = normal(G, D, scale=0.7, dtype=case["w"]) if G else None
        f32 = torch.float32
        if op == "norm_fwd":
            s["x_out"] = torch.empty(M, D, dtype=DTYPES[case["x"]], device=dev)
            s["y"] = torch.empty(M, D, dtype=DTYPES[case["y"]], device=dev) if case["pre"] else None
            s["rstd_pre"] = torch.empty(M, dtype=f32, device=dev) if case["pre"] else None
            s["rstd_post"] = torch.empty(M, dtype=f32, device=dev) if case["post"] else None
        else:
            # what the forward pass left: the stream after the block, and the two factors of each row
            s["rstd_pre"] = (stream.double().square().mean(1) + 1e-6).rsqrt().float() if case["pre"] else None
            s["rstd_post"] = (s["h"].double().square().mean(1) + 1e-6).rsqrt().float() if case["post"] else None
            s["dy"] = normal(M, D, scale=1e-3, dtype=case["y"]) if case["pre"] else None
            s["dx_out"] = normal(M, D, scale=1e-3, dtype=case["x"])
            s["dx"] = torch.empty_like(s["dx_out"])
            s["dh"] = torch.empty_like(s["h"])
            s["dw_pre"] = torch.empty(D, dtype=f32, device=dev) if case["train"] and case["pre"] else None
            s["dw_post"] = torch.empty(D, dtype=f32, device=dev) if case["train"] and case["post"] else None
            s["dgate"] = torch.empty(G, D, dtype=f32, device=dev) if case["train"] and G else None
        if own:
            import bit_nf4_quantized_10_b200 as q
            s["norm"] = q.BlockNorm(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], gate_rows=rows,
                                    alpha=case["alpha"], eps=1e-6, w_offset=case["offset"])
            if op == "norm_bwd":
                s["ws"] = torch.empty(max(16, q.qlora_workspace_size(q.QL_OP_BLOCK_NORM_BWD, M, D, rows)),
                                      dtype=torch.uint8, device=dev)
        return s
    if op in ("clip", "adamw"):
        # one flat buffer, as the data-parallel bucket keeps it: each tensor starts on a 16-byte boundary
        dt = DTYPES[case["dt"]]
        align = 16 // SIZE[case["dt"]]
        sizes, at, starts = _adapter_sizes(case), 0, []
        for n in sizes:
            starts.append(at)
            at += -(-n // align) * align
        flat = torch.randn(at, generator=gen, device=dev) * 1e-3
        for o, n in zip(starts, sizes):
            if n % align:
                flat[o + n:o + -(-n // align) * align] = 0.0
        s["flat"] = flat.to(dt)
        s["grads"] = [s["flat"][o:o + n] for o, n in zip(starts, sizes)]
        if op == "adamw":
            s["p"] = normal(at, scale=0.02)
            s["m"] = normal(at, scale=1e-4)
            s["v"] = normal(at, scale=1e-3).square()
            s["p_bf16"] = torch.empty(at, dtype=torch.bfloat16, device=dev)
        s["norm_out"] = torch.empty(1, dtype=torch.float32, device=dev)
        s["coef"] = torch.empty(1, dtype=torch.float32, device=dev)
        if own:
            import bit_nf4_quantized_10_b200 as q
            s["list"] = q.TensorList([s["flat"]] if op == "adamw" else s["grads"])
            s["ws"] = torch.empty(max(16, q.qlora_workspace_size(q.QL_OP_GRAD_NORM, len(s["list"]))), dtype=torch.uint8,
                                  device=dev)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    wide = torch.ones(K, device=dev)
    wide[torch.randint(0, K, (max(1, K // 512),), generator=gen, device=dev)] = 8.0
    s["x"] = (torch.randn(M, K, generator=gen, device=dev) * wide).to(DTYPES[case["x"]])
    # the weight in 8 bits, one scale for each output channel
    w = torch.randn(N, K, generator=gen, device=dev) * 0.02
    s["w_scales"] = w.abs().amax(1) / 127.0
    s["w_codes"] = (w / s["w_scales"][:, None]).round_().clamp_(-127, 127).to(torch.int8)
    del w
    s["x_codes"] = torch.empty(M, K, dtype=torch.int8, device=dev)
    s["x_scales"] = torch.empty(M, dtype=torch.float32, device=dev)
    s["y"] = torch.empty(M, N, dtype=DTYPES[case["y"]], device=dev)
    if own:
        import bit_nf4_quantized_10_b200 as q
        s["ws"] = torch.empty(max(16, q.qlora_workspace_size(q.QL_OP_INT8_GEMM, M, N, K)), dtype=torch.uint8, device=dev)
    return s


ADAM = {"t": 10, "lr": 2e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "clip": _clip, "adamw": _adamw, "int8": _int8}[op](state)


def _run_own(s, op):
    import bit_nf4_quantized_10_b200 as q
    if op == "norm_fwd":
        q.qlora_block_norm_fwd(s["norm"], s["x"], s["h"], s["x_out"], s["y"], s["rstd_pre"], s["rstd_post"])
        return {k: s[k] for k in ("x_out", "y", "rstd_pre", "rstd_post")}
    if op == "norm_bwd":
        q.qlora_block_norm_bwd(s["norm"], s["x"], s["h"], s["rstd_pre"], s["rstd_post"], s["dx_out"], s["dy"], s["dx"],
                               s["dh"], dw_pre=s["dw_pre"], dw_post=s["dw_post"], dgate=s["dgate"], ws=s["ws"])
        return {k: s[k] for k in ("dx", "dh", "dw_pre", "dw_post", "dgate")}
    if op == "clip":
        q.qlora_grad_norm(s["list"], s["case"]["max_norm"], s["norm_out"], s["coef"], s["ws"])
        q.qlora_grad_scale(s["list"], s["coef"])
        return {"norm": s["norm_out"], "coef": s["coef"], "grads": s["flat"]}
    if op == "adamw":
        q.qlora_grad_norm(s["list"], s["case"]["max_norm"], s["norm_out"], s["coef"], s["ws"])
        q.qlora_adamw_step_clipped(s["p"], s["flat"], s["m"], s["v"], s["p"].numel(), ADAM["t"], ADAM["lr"], s["coef"],
                                   ADAM["beta1"], ADAM["beta2"], ADAM["eps"], ADAM["weight_decay"], p_bf16=s["p_bf16"])
        return {"norm": s["norm_out"], "coef": s["coef"], "p": s["p"], "m": s["m"], "v": s["v"], "p_bf16": s["p_bf16"]}
    q.int8_quantize(s["x"], s["x_codes"], s["x_scales"])
    q.int8_gemm(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["y"], ws=s["ws"])
    return {"y": s["y"], "scales": s["x_scales"]}


# ------------------------------------------------------------- the plain forms
def _gate_rows(s):
    """The gate of each token, [M, D]."""
    rows, _ = _groups(s["case"])
    index = torch.arange(s["case"]["M"], device=s["gate"].device) // rows
    return s["gate"].float()[index]


def _norm_fwd(s):
    c = s["case"]
    branch, rstd_post = s["h"].float(), None
    if c["post"]:
        rstd_post = (branch.square().mean(1) + 1e-6).rsqrt()
        branch = branch * rstd_post[:, None] * (s["w_post"].float() + c["offset"])
    if s["gate"] is not None:
        branch = branch * _gate_rows(s)
    x_out = (s["x"].float() * c["alpha"] + branch).to(s["x"].dtype)
    y, rstd_pre = None, None
    if c["pre"]:
        kept = x_out.float()          # the norm reads the stream as it is stored
        rstd_pre = (kept.square().mean(1) + 1e-6).rsqrt()
        y = (kept * rstd_pre[:, None] * (s["w_pre"].float() + c["offset"])).to(DTYPES[c["y"]])
    return {"x_out": x_out, "y": y, "rstd_pre": rstd_pre, "rstd_post": rstd_post}


def _norm_bwd(s):
    c = s["case"]
    rows, G = _groups(c)
    dr, dw_pre, dw_post, dgate = s["dx_out"].float(), None, None, None
    if c["pre"]:
        n = s["x"].float() * s["rstd_pre"][:, None]
        dy = s["dy"].float()
        if c["train"]:
            dw_pre = (dy * n).sum(0)
        dn = dy * (s["w_pre"].float() + c["offset"])
        dr = dr + s["rstd_pre"][:, None] * (dn - n * (dn * n).mean(1, keepdim=True))
    nh = s["h"].float()
    if c["post"]:
        nh = nh * s["rstd_post"][:, None]
    weight = s["w_post"].float() + c["offset"] if c["post"] else None
    gate = _gate_rows(s) if G else None
    if c["train"] and G:
        shared = dr * nh if weight is None else dr * nh * weight
        shared = torch.nn.functional.pad(shared, (0, 0, 0, G * rows - c["M"]))
        dgate = shared.reshape(G, rows, c["D"]).sum(1)
    dnh = dr if gate is None else dr * gate
    if c["post"]:
        if c["train"]:
            dw_post = (dnh * nh).sum(0)
        dnh = dnh * weight
        dnh = s["rstd_post"][:, None] * (dnh - nh * (dnh * nh).mean(1, keepdim=True))
    return {"dx": (dr * c["alpha"]).to(DTYPES[c["x"]]), "dh": dnh.to(DTYPES[c["h"]]), "dw_pre": dw_pre,
            "dw_post": dw_post, "dgate": dgate}


def _norm_and_coef(s, grads):
    total = torch.stack([g.float().square().sum() for g in grads]).sum()
    norm = total.sqrt().reshape(1)
    return norm, (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0)


def _clip(s):
    norm, coef = _norm_and_coef(s, s["grads"])
    s["flat"].copy_(s["flat"].float() * coef)
    return {"norm": norm, "coef": coef, "grads": s["flat"]}


def _adamw(s):
    a = ADAM
    norm, coef = _norm_and_coef(s, [s["flat"]])
    g = s["flat"] * coef
    s["p"].mul_(1 - a["lr"] * a["weight_decay"])
    s["m"].mul_(a["beta1"]).add_(g * (1 - a["beta1"]))
    s["v"].mul_(a["beta2"]).add_(g * g * (1 - a["beta2"]))
    root = (s["v"] / (1 - a["beta2"] ** a["t"])).sqrt() + a["eps"]
    s["p"].sub_(s["m"] / (1 - a["beta1"] ** a["t"]) / root * a["lr"])
    s["p_bf16"].copy_(s["p"])
    return {"norm": norm, "coef": coef, "p": s["p"], "m": s["m"], "v": s["v"], "p_bf16": s["p_bf16"]}


def _int8(s):
    x = s["x"].float()
    scales = x.abs().amax(1) / 127.0
    codes = torch.where(scales[:, None] > 0, x / scales[:, None], 0.0).round().clamp(-127, 127)
    product = codes @ s["w_codes"].float().t()
    y = product * (scales[:, None] * s["w_scales"][None, :])
    return {"y": y.to(DTYPES[s["case"]["y"]]), "scales": scales}


# ------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = torch.float64
    if op == "norm_fwd":
        w = lambda t: 1.0 if t is None else t.to(d) + case["offset"]  # noqa: E731
        rms = lambda t: torch.sqrt((t * t).sum(1) / case["D"] + 1e-6)  # noqa: E731
        h, rows = s["h"].to(d), _groups(case)[0]
        rp = rms(h) if case["post"] else None
        f = h * w(s["w_post"]) / rp[:, None] if case["post"] else h
        if rows:
            f = f * torch.repeat_interleave(s["gate"].to(d), rows, 0)[:case["M"]]
        f = f + case["alpha"] * s["x"].to(d)
        if not case["pre"]:
            return {"x_out": f, "y": None, "rstd_pre": None, "rstd_post": 1 / rp if case["post"] else None}
        stored = f.to(DTYPES[case["x"]]).to(d)
        rx = rms(stored)
        return {"x_out": f, "y": stored * w(s["w_pre"]) / rx[:, None], "rstd_pre": 1 / rx,
                "rstd_post": 1 / rp if case["post"] else None}
    if op == "norm_bwd":
        return _exact_norm_bwd(case, s, d)
    if op in ("clip", "adamw"):
        g = s["flat"].to(d)
        norm = torch.linalg.vector_norm(g).reshape(1)
        coef = torch.minimum(torch.ones_like(norm), case["max_norm"] / (norm + 1e-6))
        if op == "clip":
            return {"norm": norm, "coef": coef, "grads": g * coef}
        a, g = ADAM, g * coef
        m = a["beta1"] * s["m"].to(d) + (1 - a["beta1"]) * g
        v = a["beta2"] * s["v"].to(d) + (1 - a["beta2"]) * g ** 2
        step = (m / (1 - a["beta1"] ** a["t"])) / (torch.sqrt(v / (1 - a["beta2"] ** a["t"])) + a["eps"])
        p = s["p"].to(d) * (1 - a["lr"] * a["weight_decay"]) - a["lr"] * step
        return {"norm": norm, "coef": coef, "p": p, "m": m, "v": v, "p_bf16": p}
    # the scale and the quotient are 32-bit values by definition: a code is the nearest whole number to the latter
    top = s["x"].abs().amax(1).to(d)
    scales = (top / 127).float().to(d)
    quotient = (s["x"].to(d) / scales.clamp(min=1e-300)[:, None]).float().to(d)
    codes = torch.round(quotient)
    y = torch.empty(case["M"], case["N"], dtype=d, device=codes.device)
    for lo in range(0, case["N"], 4096):
        hi = min(case["N"], lo + 4096)
        y[:, lo:hi] = torch.einsum("mk,nk->mn", codes, s["w_codes"][lo:hi].to(d)) * s["w_scales"][lo:hi].to(d)
    return {"y": y * scales[:, None], "scales": scales}


def _exact_norm_bwd(case, s, d):
    """Gradients by automatic differentiation of the forward formulas in 64 bits."""
    leaf = lambda t: None if t is None else t.to(d).requires_grad_(True)  # noqa: E731
    rms = lambda t: torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    pick = lambda t, want: t.grad if want and t is not None else None  # noqa: E731
    r, w_pre = leaf(s["x"]), leaf(s["w_pre"])
    total = (r * s["dx_out"].to(d)).sum()
    if case["pre"]:
        total = total + (r / rms(r) * (w_pre + case["offset"]) * s["dy"].to(d)).sum()
    total.backward()
    dr = r.grad
    h, w_post, gate = leaf(s["h"]), leaf(s["w_post"]), leaf(s["gate"])
    f = h / rms(h) * (w_post + case["offset"]) if case["post"] else h
    if gate is not None:
        f = f * torch.repeat_interleave(gate, case["gate_rows"], 0)[:case["M"]]
    (f * dr).sum().backward()
    t = case["train"]
    return {"dx": dr * case["alpha"], "dh": h.grad, "dw_pre": pick(w_pre, t), "dw_post": pick(w_post, t),
            "dgate": pick(gate, t)}


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        M, D = case["M"], case["D"]
        _, G = _groups(case)
        vectors = (int(case["pre"]) + int(case["post"]) + G) * D * SIZE[case["w"]]
        rows = (int(case["pre"]) + int(case["post"])) * M * 4
        x, h, y = SIZE[case["x"]], SIZE[case["h"]], SIZE[case["y"]] if case["pre"] else 0
        if op == "norm_fwd":
            return {"bytes": M * D * (2 * x + h + y) + vectors + rows, "flops": 12 * M * D}
        # the stream itself is read for its norm alone; h for its norm, or for the gate's gradient
        reads = (x if case["pre"] else 0) + (h if case["post"] or (case["train"] and G) else 0) + x + y
        sums = (int(case["pre"]) + int(case["post"]) + G) * D * 4 if case["train"] else 0
        return {"bytes": M * D * (reads + x + h) + vectors + rows + sums, "flops": 24 * M * D}
    if op in ("clip", "adamw"):
        n = sum(_adapter_sizes(case))
        if op == "clip":
            # read for the norm, which every value has a part in; then scaled in place
            return {"bytes": n * SIZE[case["dt"]] * 3, "flops": 3 * n}
        return {"bytes": n * (4 + 4 * 4 + 3 * 4 + 2), "flops": 16 * n}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": M * K * SIZE[case["x"]] + N * K + 4 * (M + N) + M * N * SIZE[case["y"]], "flops": 2 * M * N * K}
