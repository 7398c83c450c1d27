"""The operators together, as a fine-tuning step and as serving use them: norms
around QLoRA MLPs, forward and backward, the adapter gradients in one bucket,
clipped, the AdamW step; then the trained MLP merged and served in 8 bits.

Every stage of a run is checked against float64 on the device's own inputs to
that stage (its stored bf16 tensors), so that the bars are those of the single
operators: a chain of fifteen stored tensors compounds the bf16 steps that fp32
accumulation flips and has no sharp bound of its own.
"""
import numpy as np
import pytest
import torch

from oracle import adamw, block_norm, int8, lora, nf4
from synthetic import inputs as S
from tests._parity import assert_fp_close, np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_10_b200 as q
    assert torch.cuda.is_available()
    return q


def _oracle_weight(W):
    packed, c, _ = nf4.quantize(W)
    e, s2, mu = nf4.double_quant(c)
    N, K = W.shape
    return nf4.dequant(packed, N * K, nf4.dq_constants(e, s2, mu)).reshape(N, K)


def _mlp(D, H, r, seed):
    c = {"Wg": S.custom_weight(H, D, 0.02, seed), "Wu": S.custom_weight(H, D, 0.02, seed + 1),
         "Wd": S.custom_weight(D, H, 0.02, seed + 2)}
    for i, (a, k) in enumerate((("g", D), ("u", D), ("d", H))):
        n = D if a == "d" else H
        c["A" + a] = S.uniform((r, k), 1 / np.sqrt(k), seed + 3 + i)
        c["B" + a] = S.normal((n, r), 0.01, seed + 6 + i, dtype=BF)
    return c


def _build(q, D, H, M, r, s, L, gate_rows, offset=0.0, train=True):
    from bit_nf4_quantized_10_b200.mlp import QLoRAMLP, QLoRAMLPStack
    cs = [_mlp(D, H, r, 100 * (i + 1)) for i in range(L)]
    mlps = []
    for c in cs:
        w = [q.quantize_weight(c[k].cuda()) for k in ("Wg", "Wu", "Wd")]
        mlps.append(QLoRAMLP(*w, *(c[k].cuda() for k in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd")), r, s, M))
    g = torch.Generator(device="cuda").manual_seed(7)
    vec = lambda n: (1 - offset + 0.1 * torch.randn(n, generator=g, device="cuda")).to(BF)  # noqa: E731
    G = -(-M // gate_rows) if gate_rows else 0
    norms = [q.BlockNorm(w_pre=vec(D), w_offset=offset)]
    for _ in range(L):
        gate = torch.randn(G, D, generator=g, device="cuda").to(BF) if G else None
        norms.append(q.BlockNorm(vec(D), vec(D), gate, gate_rows, alpha=0.9, w_offset=offset))
    return cs, mlps, norms, QLoRAMLPStack(mlps, norms, train_norms=train)


def _params(n):
    return dict(w_post=None if n.w_post is None else np64(n.w_post), gate=None if n.gate is None else np64(n.gate),
                gate_rows=n.gate_rows, alpha=n.alpha, w_offset=n.w_offset)


def _near(got, ref, scale, what, terms=64):
    """Within `terms` 2^-24 of the sum of the absolute values of the terms, and the rounding to the type (the
    bound of tests/test_gpu_block_norm.py)."""
    half = torch.finfo(got.dtype).eps / 2
    bound = terms * 2.0 ** -24 * np.broadcast_to(scale, ref.shape)
    excess = np.abs(np64(got) - ref) - (bound + half * (np.abs(ref) + bound) + 2.0 ** -133)
    assert np.all(excess <= 0), f"{what}: {np.max(excess):.3e} past the bound"


@pytest.mark.parametrize("M,gate_rows,offset", [(160, 80, 0.0), (37, 0, 1.0), (200, 200, 0.0)])
def test_stack_clip_and_step(q, M, gate_rows, offset):
    from bit_nf4_quantized_10_b200.dp import GradBucket
    D, H, r, s, L = 512, 1408, 16, 2.0, 2
    cs, mlps, norms, stack = _build(q, D, H, M, r, s, L, gate_rows, offset)
    bucket = GradBucket([sh for m in mlps for sh in m.gradient_shapes()], device="cuda")
    for i, m in enumerate(mlps):
        m.use_gradients(bucket.views[6 * i:6 * i + 6])
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(M, D, generator=g, device="cuda").to(BF)
    dx_out = (torch.randn(M, D, generator=g, device="cuda")).to(BF)
    dy_out = torch.randn(M, D, generator=g, device="cuda")
    xl, yl = stack.forward(x)
    dx = stack.backward(dx_out, dy_out).clone()
    torch.cuda.synchronize()
    assert q.qlora_get_status() == q.QL_OK and xl is stack.x[-1] and yl is stack.y[-1]

    # forward, stage by stage
    W = [[_oracle_weight(c[k]) for k in ("Wg", "Wu", "Wd")] for c in cs]
    args = lambda i, y: (y, W[i][0], cs[i]["Ag"], cs[i]["Bg"], W[i][1], cs[i]["Au"], cs[i]["Bu"], W[i][2],  # noqa: E731
                         cs[i]["Ad"], cs[i]["Bd"], s)
    for j, n in enumerate(norms):
        if j:
            f, _ = block_norm.post(np64(stack.x[j - 1]), np64(stack.h[j - 1]), **_params(n))
            kept = np.abs(n.alpha * np64(stack.x[j - 1]))
            _near(stack.x[j], f, kept + np.abs(f - n.alpha * np64(stack.x[j - 1])), f"x {j}")
        ref, rx = block_norm.pre(np64(stack.x[j]), np64(n.w_pre), w_offset=n.w_offset)
        _near(stack.y[j], ref, np.abs(np64(stack.x[j])) * rx[:, None] * (np.abs(np64(n.w_pre)) + offset), f"y {j}")
    fs = [lora.mlp_forward(*args(i, np64(stack.y[i]))) for i in range(L)]
    for i in range(L):
        assert_fp_close(np64(stack.h[i]), fs[i]["y"], f"h {i}", rel_fro=2e-3 + 2.0 ** -9, max_abs_rms=0.1)

    # backward: the same calls one by one, which the stack must equal bit for bit,
    # each against the formulas on its own inputs
    kept = [[getattr(m, name).clone() for name in m.GRADIENTS] for m in mlps]
    sums = [[None if t is None else t.clone() for t in lst] for lst in (stack.dw_pre, stack.dw_post, stack.dgate)]
    d_x, d_y = dx_out, dy_out
    for j in reversed(range(L + 1)):
        n, last = norms[j], j == 0
        o = {"dx": torch.empty_like(x), "dw_pre": torch.empty(D, device="cuda")}
        if not last:
            o["dh"], o["dw_post"] = torch.empty_like(x), torch.empty(D, device="cuda")
            if n.gate is not None:
                o["dgate"] = torch.empty(n.gate.shape, device="cuda")
        h = None if last else stack.h[j - 1]
        q.qlora_block_norm_bwd(n, stack.x[j], h, stack.rstd_pre[j], None if last else stack.rstd_post[j], d_x, d_y,
                               o["dx"], o.get("dh"), dw_pre=o["dw_pre"], dw_post=o.get("dw_post"),
                               dgate=o.get("dgate"), ws=stack.ws)
        ref = block_norm.backward(np64(stack.x[j]), None if last else np64(h), np64(d_x), np64(d_y), np64(n.w_pre),
                                  **_params(n))
        for name, t in o.items():
            terms = (64 if name in ("dx", "dh") else 64 + M) * 3 * (4 if offset else 1)
            _near(t, ref[name], ref[name + "_abs"], f"{name} of norm {j}", terms)
        for lst, name in zip(sums, ("dw_pre", "dw_post", "dgate")):
            if lst[j] is not None:
                assert torch.equal(lst[j], o[name]), f"{name} of norm {j}"
        d_x = o["dx"]
        if last:
            break
        mlps[j - 1].backward(stack.y[j - 1], o["dh"])
        d_y = mlps[j - 1].dX
        b = lora.mlp_backward(*args(j - 1, np64(stack.y[j - 1])), np64(o["dh"]), fs[j - 1])
        for name, was in zip(mlps[j - 1].GRADIENTS, kept[j - 1]):
            assert torch.equal(getattr(mlps[j - 1], name), was), name
            assert_fp_close(np64(was), b[name], f"{name} of block {j - 1}", max_abs_rms=0.1)
    assert torch.equal(d_x, dx)

    # the norm of exactly these gradients, the clipped step, bit for bit
    before = bucket.buffer.clone()
    n = bucket.buffer.numel()
    want, want_c = adamw.clip([np64(v) for v in bucket.views], 0.3)
    norm, coef = bucket.clip(0.3, scale=False)
    assert abs(norm.item() - want) <= 2.0 ** -23 * want and abs(coef.item() - want_c) <= 2.0 ** -21 * want_c
    assert torch.equal(bucket.buffer, before)
    p0 = torch.randn(n, generator=g, device="cuda") * 0.02
    p, m_, v_ = p0.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    q.qlora_adamw_step_clipped(p, bucket.buffer, m_, v_, n, 1, 1e-3, coef, weight_decay=0.01)
    bucket.clip(0.3)
    assert torch.equal(bucket.buffer, before * coef)
    p2, m2, v2 = p0.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    q.qlora_adamw_step(p2, bucket.buffer, m2, v2, n, 1, 1e-3, weight_decay=0.01)
    assert torch.equal(p, p2) and torch.equal(m_, m2) and torch.equal(v_, v2)
    P = adamw.adamw_step_fp32(p0.cpu().numpy(), bucket.buffer.cpu().numpy(), np.zeros(n, np.float32),
                              np.zeros(n, np.float32), 1, 1e-3, 0.9, 0.999, 1e-8, 0.01)[0]
    assert np.array_equal(p.cpu().numpy(), P)


def test_whole_step_in_a_graph(q):
    """Forward, backward, clip and step captured once and replayed: the bits of the eager step."""
    from bit_nf4_quantized_10_b200.dp import GradBucket
    D, H, M, r, s = 512, 1408, 96, 16, 2.0
    _, mlps, _, stack = _build(q, D, H, M, r, s, 2, 32)
    bucket = GradBucket([sh for m in mlps for sh in m.gradient_shapes()], device="cuda")
    for i, m in enumerate(mlps):
        m.use_gradients(bucket.views[6 * i:6 * i + 6])
    n = bucket.buffer.numel()
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dx_out = (torch.randn(M, D, generator=g, device="cuda").to(BF) for _ in range(2))
    p, m_, v_ = (torch.zeros(n, device="cuda") for _ in range(3))

    def step():
        stack.forward(x)
        stack.backward(dx_out, None)
        _, coef = bucket.clip(0.3, scale=False)
        q.qlora_adamw_step_clipped(p, bucket.buffer, m_, v_, n, 1, 1e-3, coef)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (p, m_, v_, stack.dx, *[d for d in stack.dgate if d is not None])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (p, m_, v_):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [p, m_, v_, stack.dx, *[d for d in stack.dgate if d is not None]]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert q.qlora_get_status() == q.QL_OK


@pytest.mark.parametrize("m", [1, 8, 33, 64])
def test_merged_mlp_served_in_8_bits(q, m):
    """Norm, 8-bit MLP, norm: the merged weights' codes exactly, every linear
    within three fp32 roundings of float64 on the device's own codes, and a
    bf16 rounding where it stores bf16."""
    from bit_nf4_quantized_10_b200.mlp import MergedInt8MLP
    D, H, r, s = 512, 1408, 16, 2.0
    cs, mlps, norms, _ = _build(q, D, H, 64, r, s, 1, 0)
    served = MergedInt8MLP(mlps[0], 64)
    for (codes, scales), k, a in zip(served.weights, ("Wg", "Wu", "Wd"), "gud"):
        W = lora.merge(_oracle_weight(cs[0][k]), np64(cs[0]["A" + a]), np64(cs[0]["B" + a]), s)
        rc, rs = int8.quantize(W.astype(np.float32))
        assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, D, generator=g, device="cuda").to(BF)
    y0, h, x1, y1 = (torch.empty(m, D, dtype=BF, device="cuda") for _ in range(4))
    q.qlora_block_norm_fwd(norms[0], x, None, None, y0)
    served.forward(y0, h)
    q.qlora_block_norm_fwd(norms[1], x, h, x1, y1)
    torch.cuda.synchronize()
    assert q.qlora_get_status() == q.QL_OK
    ry, rx = block_norm.pre(np64(x), np64(norms[0].w_pre))
    _near(y0, ry, np.abs(np64(x)) * rx[:, None] * np.abs(np64(norms[0].w_pre)), "y")
    w8 = [(c.cpu().numpy(), sc.cpu().numpy()) for c, sc in served.weights]
    lin = lambda t, w: int8.gemm(*int8.quantize(np64(t).astype(np.float32)), *w)  # noqa: E731
    for got, t, w in ((served.g[:m], y0, w8[0]), (served.u[:m], y0, w8[1]), (h, served.h[:m], w8[2])):
        ref = lin(t, w)
        _near(got, ref, np.abs(ref), "linear", 4)
    f, _ = block_norm.post(np64(x), np64(h), np64(norms[1].w_post), alpha=norms[1].alpha)
    _near(x1, f, np.abs(norms[1].alpha * np64(x)) + np.abs(f - norms[1].alpha * np64(x)), "x")
    ry, rx = block_norm.pre(np64(x1), np64(norms[1].w_pre))
    _near(y1, ry, np.abs(np64(x1)) * rx[:, None] * np.abs(np64(norms[1].w_pre)), "y1")


def test_stack_and_served_mlp_refuse(q):
    from bit_nf4_quantized_10_b200.mlp import MergedInt8MLP, QLoRAMLPStack
    _, mlps, norms, _ = _build(q, 512, 1408, 16, 8, 2.0, 1, 0)
    with pytest.raises(ValueError):
        QLoRAMLPStack(mlps, norms[:1])
    with pytest.raises(ValueError):
        QLoRAMLPStack(mlps, norms[::-1])
    served = MergedInt8MLP(mlps[0], 16)
    with pytest.raises(ValueError):
        served.forward(torch.empty(17, 512, dtype=BF, device="cuda"), torch.empty(17, 512, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        mlps[0].use_gradients([torch.empty(3, device="cuda")] * 6)
    x = torch.randn(4, 512, device="cuda").to(BF)
    with pytest.raises(ValueError):      # another stream's tensor shapes
        q.qlora_block_norm_fwd(norms[0], x, None, None, torch.empty(5, 512, device="cuda"))
    with pytest.raises(ValueError):
        q.qlora_block_norm_fwd(norms[0], x.t(), None, None, torch.empty(512, 4, device="cuda"))
    with pytest.raises(q.QLoraError):
        q.qlora_block_norm_fwd(q.BlockNorm(), x, None, None, torch.empty(4, 512, device="cuda"))
