"""Row-wise int8 quantization (bit for bit) and the int8 product.

The product's sum is an exact integer; the output takes three fp32 roundings
(the sum to fp32, the product of the two scales, their product), so it is within
3.01 2^-24 of the exact value, relative, plus the rounding to bf16.
"""
import numpy as np
import pytest
import torch

from oracle import int8 as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_10_b200 as q
    assert torch.cuda.is_available()
    return q


def _quantize(q, x):
    codes = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    scales = torch.full((x.shape[0],), -1.0, device="cuda")
    q.int8_quantize(x, codes, scales)
    return codes, scales


def _same(q, x):
    codes, scales = _quantize(q, x)
    want, s = O.quantize(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (200, 64), (7, 512), (33, 4096), (5, 8192), (4, 8208), (2, 28672),
                                    (2, 131056)])
def test_quantize(q, rows, K, dt):
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g, device="cuda")
    x[:, 3] *= 20
    _same(q, x.to(dt))
    assert q.qlora_get_status() == q.QL_OK


@pytest.mark.parametrize("K", [64, 16400])
def test_quantize_ties_zeros_and_tiny_rows(q, K):
    x = torch.zeros(12, K, device="cuda")
    x[1, 5] = -0.0
    for i, s in enumerate((1.0, 2.0 ** -20, 2.0 ** 90)):      # s an exact power of two: halves are ties
        x[2 + i] = (torch.arange(K, device="cuda") % 255 - 127 + 0.5).clamp(-127, 127) * s
        x[2 + i, 0] = 127 * s
    for i, top in enumerate((2.0 ** -149, 63 * 2.0 ** -149, 64 * 2.0 ** -149, 190 * 2.0 ** -149, 2.0 ** -127, 3e38)):
        x[5 + i] = torch.linspace(-1, 1, K, device="cuda") * top
        x[5 + i, 7] = top
    _same(q, x)
    _same(q, x.bfloat16())
    assert q.qlora_get_status() == q.QL_OK


def test_quantize_every_bf16_quotient_near_a_half(q):
    """Rows of every bf16 value up to the row's largest: all quotients a bf16 row can have."""
    for top in (1.0, 1.5703125, 1.9921875, 93.5, 6e-3):
        v = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
        v = v[v <= top]
        v = torch.cat([v, v.new_zeros(-v.numel() % 16)])
        _same(q, torch.stack([v, -v]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_quantize_reports_non_finite_rows(q, bad):
    x = torch.randn(4, 96, device="cuda")
    x[2, 95] = bad
    codes, scales = _quantize(q, x)
    assert q.qlora_get_status() == q.QL_ERR_NONFINITE
    assert torch.isnan(scales[2]) and not codes[2].any()
    want, s = O.quantize(x[[0, 1, 3]].cpu().numpy())
    assert np.array_equal(codes[[0, 1, 3]].cpu().numpy(), want)


def _operands(M, N, K, seed=0, extreme=False):
    g = torch.Generator(device="cuda").manual_seed(seed + M * 7 + N * 3 + K)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    b = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    if extreme:
        a.fill_(-128)
        b.fill_(-128)
        b[::2] = 127
    sa = torch.rand(M, generator=g, device="cuda") * 0.1 + 1e-3
    sb = torch.rand(N, generator=g, device="cuda") * 0.1 + 1e-3
    return a, sa, b, sb


def _product(q, a, sa, b, sb, dt, **k):
    M, N, K = a.shape[0], b.shape[0], a.shape[1]
    pad = 1000
    buf = torch.full((M * N + pad,), 3.0, dtype=dt, device="cuda")
    Y = buf[:M * N].view(M, N)
    ws = torch.full((max(16, q.qlora_workspace_size(q.QL_OP_INT8_GEMM, M, N, K)),), 0xFF, dtype=torch.uint8, device="cuda")
    q.int8_gemm(a, sa, b, sb, Y, ws=ws, **k)
    torch.cuda.synchronize()
    assert bool((buf[M * N:] == 3.0).all())
    return Y


def _check(q, M, N, K, dt=F32, extreme=False):
    a, sa, b, sb = _operands(M, N, K, extreme=extreme)
    Y = _product(q, a, sa, b, sb, dt)
    ref = (a.double() @ b.double().t()) * (sa.double()[:, None] * sb.double()[None, :])
    tol = 3.01 * 2.0 ** -24 + (torch.finfo(dt).eps / 2 * (1 + 2.0 ** -20) if dt == BF else 0.0)
    assert bool(((Y.double() - ref).abs() <= tol * ref.abs()).all()), (M, N, K)
    assert q.qlora_get_status() == q.QL_OK


@pytest.mark.parametrize("M", [1, 7, 16, 31, 32, 33, 64, 65, 255, 256, 257, 300, 519])
def test_tokens(q, M):
    for N, K in ((1000, 144), (257, 4096)):
        _check(q, M, N, K)
        _check(q, M, N, K, BF)


@pytest.mark.parametrize("N", [1, 2, 8, 31, 127, 128, 129, 255, 256, 257, 513])
def test_channels(q, N):
    _check(q, 5, N, 512)
    _check(q, 70, N, 2064, BF)


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 1024, 4112, 28672])
def test_reductions(q, K):
    _check(q, 3, 300, K)
    _check(q, 290, 520, K, BF)


@pytest.mark.parametrize("M,N,K", [(1, 19000, 1024), (8, 28672, 2048), (40, 18944, 640), (600, 8000, 512),
                                   (1024, 19200, 256), (2500, 2300, 1040), (16, 37888, 128),
                                   (1024, 19200, 2064), (2100, 9001, 2048), (601, 28600, 2192), (2049, 8193, 2304)])
def test_whole_rounds_and_shared_tiles(q, M, N, K):
    """Whole rounds of tiles, rounds and shared tiles, shared tiles alone."""
    _check(q, M, N, K)


def test_largest_sums(q):
    """128^2 131056 is the largest sum that int32 must hold."""
    _check(q, 3, 5, 131056, extreme=True)
    _check(q, 300, 40, 131056)


def test_oracle_agrees(q):
    a, sa, b, sb = _operands(9, 17, 256)
    ref = O.gemm(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy())
    Y = _product(q, a, sa, b, sb, F32)
    assert np.all(np.abs(Y.double().cpu().numpy() - ref) <= 3.01 * 2.0 ** -24 * np.abs(ref))


def test_nan_and_zero_scales(q):
    a, sa, b, sb = _operands(6, 40, 64)
    sa[2], sa[4] = float("nan"), 0.0
    Y = _product(q, a, sa, b, sb, F32)
    assert bool(torch.isnan(Y[2]).all()) and not Y[4].any() and bool(torch.isfinite(Y[[0, 1, 3, 5]]).all())


def test_no_tokens(q):
    a, sa, b, sb = _operands(1, 40, 64)
    q.int8_gemm(a[:0], sa[:0], b, sb, torch.empty(0, 40, device="cuda"))


def test_two_streams_and_captured_graphs(q):
    """Two products at once on two streams, each with its workspace, and one graph replayed on new codes."""
    shapes = [(40, 18944, 1024), (8, 28672, 1024)]
    ops = [_operands(*s) for s in shapes]
    want = [_product(q, *o, F32) for o in ops]
    streams = [torch.cuda.Stream() for _ in shapes]
    wss = [torch.empty(q.qlora_workspace_size(q.QL_OP_INT8_GEMM, *s), dtype=torch.uint8, device="cuda") for s in shapes]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for o, y, w, st in zip(ops, outs, wss, streams):
            q.int8_gemm(*o, y, ws=w, stream=st)
    torch.cuda.synchronize()
    for y, w in zip(outs, want):
        assert torch.equal(y, w)
    (a, sa, b, sb), y = ops[0], outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.int8_gemm(a, sa, b, sb, y, ws=wss[0])
    a2 = _operands(*shapes[0], seed=5)
    for dst, src in zip((a, sa, b, sb), a2):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, _product(q, *a2, F32))


def test_quantized_linear_close_to_the_float_one(q):
    """Both roundings together: each factor is off by at most half a code, so a
    sum of K products by at most K (s_a/2 |b| + s_b/2 |a| + s_a s_b / 4)."""
    M, N, K = 50, 300, 1024
    x, w = torch.randn(M, K, device="cuda").bfloat16(), (torch.randn(N, K, device="cuda") * 0.02).bfloat16()
    (a, sa), (b, sb) = _quantize(q, x), _quantize(q, w)
    Y = _product(q, a, sa, b, sb, F32).double()
    ref = x.double() @ w.double().t()
    sa, sb = sa.double()[:, None], sb.double()[None, :]
    bound = (sa / 2 * w.double().abs().sum(1)[None] + sb / 2 * x.double().abs().sum(1)[:, None] + K * sa * sb / 4) * 1.001
    assert bool(((Y - ref).abs() <= bound).all())
