"""Global gradient norm, clipping in place and the clipped AdamW step.

Squares are summed in float64 (relative error below 1e-12 at these sizes), so
the fp32 norm is within half a step (2^-24) and 1e-12 of the exact one; the
coefficient takes a sum and a quotient more (two roundings of 2^-24, and one of
the norm).  Given the device's coefficient, the scaled gradients and the AdamW
states are single fp32 operations and compared bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import adamw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_10_b200 as q
    assert torch.cuda.is_available()
    return q


def _tensors(sizes, dts, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dt) for n, dt in zip(sizes, dts)]


def _norm(q, tensors, max_norm, ws=None):
    lst = q.TensorList(tensors)
    norm, coef = torch.full((1,), -1.0, device="cuda"), torch.full((1,), -1.0, device="cuda")
    if ws is None:
        ws = torch.empty(q.qlora_workspace_size(q.QL_OP_GRAD_NORM, len(lst)), dtype=torch.uint8, device="cuda")
    q.qlora_grad_norm(lst, max_norm, norm, coef, ws)
    return lst, norm, coef


def _check(q, tensors, max_norm):
    before = [t.clone() for t in tensors]
    lst, norm, coef = _norm(q, tensors, max_norm)
    q.qlora_grad_scale(lst, coef)
    want, want_c = adamw.clip([b.double().cpu().numpy() for b in before], max_norm)
    assert abs(norm.item() - want) <= (2.0 ** -24 + 1e-12) * want + 2.0 ** -150
    assert abs(coef.item() - want_c) <= 4 * 2.0 ** -24 * want_c
    assert coef.item() <= 1.0
    for t, b in zip(tensors, before):
        assert torch.equal(t, (b.float() * coef).to(b.dtype))
    return norm, coef


SIZES = [[1], [3], [8], [8191], [8192], [8193], [5, 0, 1, 7, 4097], [100_000, 1, 33], [16 * 1024 + 3] * 40,
         list(range(1, 300)), [12_345] * 1023, [4099] * 1024, [130] * 1025, [64] * 2100]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_sizes(q, sizes, dt):
    _check(q, _tensors(sizes, [dt] * len(sizes)), 1e-2)
    _check(q, _tensors(sizes, [dt] * len(sizes), seed=1), 1e6)


def test_mixed_types_and_large(q):
    _check(q, _tensors([300_001, 17, 90_000, 5], [F32, BF, BF, F32]), 0.1)
    _check(q, _tensors([60_000_003, 5], [F32, BF]), 0.3)


def test_empty_lists(q):
    for tensors in ([], [torch.empty(0, device="cuda")], [torch.empty(0, device="cuda"), torch.empty(0, device="cuda")]):
        lst, norm, coef = _norm(q, tensors, 1.0)
        q.qlora_grad_scale(lst, coef)
        assert norm.item() == 0.0 and coef.item() == 1.0


@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e15, 1e25])
def test_squares_neither_vanish_nor_overflow(q, scale):
    _check(q, _tensors([70_001], [F32], scale=scale), scale)


def test_limits(q):
    t = _tensors([1000], [F32])
    _, norm, coef = _norm(q, t, float("inf"))
    assert coef.item() == 1.0
    _, norm, coef = _norm(q, t, 0.0)
    assert coef.item() == 0.0
    lst = q.TensorList(t)
    ws = torch.empty(q.qlora_workspace_size(q.QL_OP_GRAD_NORM, 1), dtype=torch.uint8, device="cuda")
    n2 = torch.empty(1, device="cuda")
    q.qlora_grad_norm(lst, 1.0, n2, None, ws)
    assert torch.equal(n2, norm)
    assert q.qlora_get_status() == q.QL_OK


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dt", [F32, BF])
def test_non_finite_gradients_are_reported(q, bad, dt):
    t = _tensors([9000, 50], [dt, dt])
    t[1][49] = bad
    _, norm, coef = _norm(q, t, 1.0)
    assert q.qlora_get_status() == q.QL_ERR_NONFINITE
    assert not np.isfinite(norm.item())
    assert coef.item() == 0.0 if abs(bad) == float("inf") else np.isnan(coef.item())
    assert q.qlora_get_status() == q.QL_OK


def test_neighbours_untouched(q):
    buf = torch.full((40_000,), 2.0, device="cuda")
    views = [buf[4:4 + 8195], buf[8208:8208 + 3], buf[16_000:16_000 + 20_001]]
    inside = torch.zeros(40_000, dtype=torch.bool, device="cuda")
    for a, n in ((4, 8195), (8208, 3), (16_000, 20_001)):
        inside[a:a + n] = True
    lst, _, coef = _norm(q, views, 1.0)
    q.qlora_grad_scale(lst, coef)
    assert bool((buf[~inside] == 2.0).all()) and bool((buf[inside] < 2.0).all())


def test_same_bits_and_two_graphs_sharing_a_workspace(q):
    """Two captured graphs of different lists use one workspace, one after the other."""
    a, b = _tensors([200_003, 77], [F32, BF], seed=3), _tensors([64] * 1100, [F32] * 1100, seed=4)
    ws = torch.empty(q.qlora_workspace_size(q.QL_OP_GRAD_NORM, 1100), dtype=torch.uint8, device="cuda")
    want = [_norm(q, t, 0.1, ws)[1].item() for t in (a, b)]
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            keep = _norm(q, t, 0.1, ws)
        graphs.append((g, keep))
    for _ in range(3):
        for (g, keep), w in zip(graphs, want):
            g.replay()
            assert keep[1].item() == w


@pytest.mark.parametrize("n", [1, 3, 4096, 131_072 + 17])
def test_clipped_adamw_bit_exact(q, n):
    rng = np.random.default_rng(n)
    p0 = (rng.standard_normal(n) * 0.02).astype(np.float32)
    p, m, v = torch.tensor(p0, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    pb = torch.empty(n, dtype=BF, device="cuda")
    P, Mr, V = p0.copy(), np.zeros(n, np.float32), np.zeros(n, np.float32)
    for t in range(1, 4):
        g0 = rng.standard_normal(n).astype(np.float32)
        g = torch.tensor(g0, device="cuda")
        _, _, coef = _norm(q, [g], 0.3)
        q.qlora_adamw_step_clipped(p, g, m, v, n, t, 1e-3, coef, 0.9, 0.999, 1e-8, 0.01, p_bf16=pb)
        c = np.float32(coef.item())
        P, Mr, V = adamw.adamw_step_fp32(P, (g0 * c).astype(np.float32), Mr, V, t, 1e-3, 0.9, 0.999, 1e-8, 0.01)
        assert np.array_equal(p.cpu().numpy(), P) and np.array_equal(m.cpu().numpy(), Mr)
        assert np.array_equal(v.cpu().numpy(), V) and torch.equal(pb, p.bfloat16())
        assert np.array_equal(g.cpu().numpy(), g0)
