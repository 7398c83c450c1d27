"""Refusals of the block norms, the gradient norm and the int8 linear, without
a GPU: every call fails its checks before anything is launched."""
import ctypes

import pytest
import torch

FAKE = 1 << 20      # aligned, never dereferenced
S0 = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    import bit_nf4_quantized_10_b200._lib as L
    return L


def _norm(lib, w_pre=FAKE, w_post=FAKE, gate=None, w_dt=1, eps=1e-6, gate_rows=0):
    return ctypes.byref(lib.ql_block_norm(w_pre, w_post, gate, w_dt, 0.0, 1.0, eps, gate_rows))


def test_block_norm_forward(lib):
    f = lambda n=None, x=FAKE, xt=1, h=FAKE, ht=1, M=4, D=64, xo=FAKE, y=FAKE, yt=1, rp=FAKE, ro=FAKE: (  # noqa: E731
        lib.LIB.qlora_block_norm_fwd(_norm(lib) if n is None else n, x, xt, h, ht, M, D, xo, y, yt, rp, ro, S0))
    bad = lib.QL_ERR_INVALID_ARG
    assert lib.LIB.qlora_block_norm_fwd(None, FAKE, 1, FAKE, 1, 4, 64, FAKE, FAKE, 1, FAKE, FAKE, S0) == bad
    assert f(x=None) == bad and f(x=FAKE + 8) == bad and f(h=FAKE + 2) == bad
    assert f(xt=7) == bad and f(ht=-1) == bad and f(yt=2) == bad
    assert f(M=-1) == bad and f(D=0) == bad
    assert f(xo=None, y=None) == bad and f(y=FAKE + 4) == bad and f(xo=FAKE + 4) == bad and f(rp=FAKE + 4) == bad
    assert f(n=_norm(lib, w_pre=None)) == bad
    assert f(n=_norm(lib, w_dt=5)) == bad and f(n=_norm(lib, eps=-1.0)) == bad and f(n=_norm(lib, eps=float("nan"))) == bad
    assert f(n=_norm(lib, gate=FAKE, gate_rows=0)) == bad and f(n=_norm(lib, gate=FAKE + 4, gate_rows=1)) == bad
    assert f(n=_norm(lib, w_post=FAKE + 8)) == bad
    assert f(D=16385) == lib.QL_ERR_UNSUPPORTED and f(M=1 << 31) == lib.QL_ERR_UNSUPPORTED
    assert f(M=0) == lib.QL_OK


def test_block_norm_backward(lib):
    def f(n=None, xo=FAKE, xt=1, h=FAKE, ht=1, rp=FAKE, ro=FAKE, dxo=FAKE, dy=FAKE, yt=0, M=4, D=64, dx=FAKE, dh=FAKE,
          wp=None, wo=None, dg=None, ws=None, wb=0):
        return lib.LIB.qlora_block_norm_bwd(_norm(lib) if n is None else n, xo, xt, h, ht, rp, ro, dxo, dy, yt, M, D, dx,
                                            dh, wp, wo, dg, ws, wb, S0)
    bad, gated = lib.QL_ERR_INVALID_ARG, _norm(lib, gate=FAKE, gate_rows=2)
    assert f(dx=None, dh=None) == bad and f(dxo=None, dy=None) == bad
    assert f(xo=None) == bad and f(rp=None) == bad and f(ro=None) == bad and f(h=None) == bad
    assert f(n=_norm(lib, w_pre=None)) == bad
    assert f(dy=None, wp=FAKE) == bad                                   # dw_pre needs dy
    assert f(wo=FAKE, n=_norm(lib, w_post=None)) == bad and f(dg=FAKE) == bad
    assert f(n=gated, dg=FAKE, h=None) == bad
    assert f(yt=9) == bad and f(xt=3) == bad and f(ht=3) == bad
    assert f(dx=FAKE + 8) == bad and f(dh=FAKE + 8) == bad and f(dxo=FAKE + 8) == bad and f(wp=FAKE + 8) == bad
    assert f(wp=FAKE, ws=FAKE, wb=16) == lib.QL_ERR_WORKSPACE
    need = lib.qlora_workspace_size(lib.QL_OP_BLOCK_NORM_BWD, 4, 64, 0)
    assert f(wp=FAKE, ws=FAKE + 4, wb=need) == bad and f(wp=FAKE, ws=None, wb=need) == bad
    assert f(D=16392) == lib.QL_ERR_UNSUPPORTED and f(M=1 << 31) == lib.QL_ERR_UNSUPPORTED


def test_block_norm_workspace_holds_the_parts(lib):
    """[blocks, D] twice and, for gates of several chunks, [chunks, D], each a multiple of 256 bytes."""
    f = lambda M, D, g: lib.qlora_workspace_size(lib.QL_OP_BLOCK_NORM_BWD, M, D, g)  # noqa: E731
    for M, D in ((1, 1), (10, 100), (5000, 4096), (8192, 16384)):
        plain = f(M, D, 0)
        assert plain % 512 == 0 and 2 * D * 4 <= plain <= 2 * (min(M, 8 * 160) * D * 4 + 256)
        assert f(M, D, 1) <= plain          # a gate per token: its gradient needs no parts
        assert f(M, D, M) >= plain
    assert f(0, 64, 0) == 0 and f(8, 16385, 0) == 0


def _list(lib, n=1, data=FAKE, numel=10, dt=0):
    d, s, t = (ctypes.c_void_p * n)(*[data] * n), (ctypes.c_int64 * n)(*[numel] * n), (ctypes.c_int32 * n)(*[dt] * n)
    c = ctypes
    return lib.ql_tensor_list(c.cast(d, c.POINTER(c.c_void_p)), c.cast(s, c.POINTER(c.c_int64)),
                              c.cast(t, c.POINTER(c.c_int32)), n), (d, s, t)


def test_grad_norm(lib):
    L, bad = lib.LIB, lib.QL_ERR_INVALID_ARG
    l, keep = _list(lib)
    r = ctypes.byref
    need = lib.qlora_workspace_size(lib.QL_OP_GRAD_NORM, 1)
    assert need > 0 and lib.qlora_workspace_size(lib.QL_OP_GRAD_NORM, 0) == need
    assert lib.qlora_workspace_size(lib.QL_OP_GRAD_NORM, 1024) == need
    assert lib.qlora_workspace_size(lib.QL_OP_GRAD_NORM, 1025) == 2 * need
    assert L.qlora_grad_norm(None, 1.0, FAKE, FAKE, FAKE, need, S0) == bad
    assert L.qlora_grad_norm(r(l), -1.0, FAKE, FAKE, FAKE, need, S0) == bad
    assert L.qlora_grad_norm(r(l), float("nan"), FAKE, FAKE, FAKE, need, S0) == bad
    assert L.qlora_grad_norm(r(l), 1.0, FAKE + 2, FAKE, FAKE, need, S0) == bad
    assert L.qlora_grad_norm(r(l), 1.0, FAKE, FAKE + 1, FAKE, need, S0) == bad
    assert L.qlora_grad_norm(r(l), 1.0, FAKE, FAKE, None, need, S0) == bad
    assert L.qlora_grad_norm(r(l), 1.0, FAKE, FAKE, FAKE, need - 1, S0) == lib.QL_ERR_WORKSPACE
    for kw in ({"data": None}, {"data": FAKE + 4}, {"numel": -1}, {"dt": 2}):
        b, keep_b = _list(lib, **kw)
        assert L.qlora_grad_norm(r(b), 1.0, FAKE, FAKE, FAKE, need, S0) == bad
        assert L.qlora_grad_scale(r(b), FAKE, S0) == bad
    b, keep_b = _list(lib, numel=1 << 43)
    assert L.qlora_grad_norm(r(b), 1.0, FAKE, FAKE, FAKE, need, S0) == lib.QL_ERR_UNSUPPORTED
    assert L.qlora_grad_scale(r(l), None, S0) == bad and L.qlora_grad_scale(None, FAKE, S0) == bad
    assert L.qlora_grad_scale(r(lib.ql_tensor_list(None, None, None, 1)), FAKE, S0) == bad
    assert L.qlora_grad_scale(r(lib.ql_tensor_list(None, None, None, -1)), FAKE, S0) == bad
    assert L.qlora_grad_scale(r(lib.ql_tensor_list(None, None, None, 0)), FAKE, S0) == lib.QL_OK
    step = lambda n=16, t=1, coef=FAKE, g=FAKE: L.qlora_adamw_step_clipped(  # noqa: E731
        FAKE, g, FAKE, FAKE, None, n, t, 1e-3, 0.9, 0.999, 1e-8, 0.0, coef, S0)
    assert step(n=0) == bad and step(t=0) == bad and step(coef=None) == bad and step(coef=FAKE + 2) == bad
    assert step(g=None) == bad


def test_int8(lib):
    L, bad, no = lib.LIB, lib.QL_ERR_INVALID_ARG, lib.QL_ERR_UNSUPPORTED
    f = lambda x=FAKE, dt=1, rows=4, K=64, c=FAKE, s=FAKE: L.int8_quantize(x, dt, rows, K, c, s, S0)  # noqa: E731
    assert f(x=None) == bad and f(x=FAKE + 2) == bad and f(dt=4) == bad and f(rows=0) == bad and f(K=0) == bad
    assert f(c=FAKE + 8) == bad and f(s=None) == bad
    assert f(K=24) == no and f(K=131072) == no and f(rows=1 << 31) == no
    g = lambda a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, M=8, N=64, K=64, Y=FAKE, dt=0, ws=FAKE, wb=1 << 30: (  # noqa: E731
        L.int8_gemm(a, sa, b, sb, M, N, K, Y, dt, ws, wb, S0))
    assert g(M=-1) == bad and g(N=0) == bad and g(K=0) == bad and g(dt=3) == bad
    assert g(a=None) == bad and g(sa=FAKE + 4) == bad and g(b=FAKE + 1) == bad and g(sb=None) == bad and g(Y=FAKE + 8) == bad
    assert g(K=40) == no and g(K=131072) == no and g(M=1 << 31) == no and g(N=1 << 31) == no
    assert g(M=(1 << 31) - 1, N=(1 << 31) - 1) == no
    assert g(M=0) == lib.QL_OK
    need = lib.qlora_workspace_size(lib.QL_OP_INT8_GEMM, 33, 1024, 28672)      # split along K
    assert need > 0 and lib.qlora_workspace_size(lib.QL_OP_INT8_GEMM, 8, 28672, 8192) == 0
    assert g(M=33, N=1024, K=28672, wb=need - 1) == lib.QL_ERR_WORKSPACE
    assert g(M=33, N=1024, K=28672, ws=FAKE + 4, wb=need) == bad


def test_binding_refuses_what_the_library_cannot_see(lib):
    """Tensors on the CPU, of another shape or type, or not contiguous (device -1 is the CPU's)."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.TensorList([x])
    with pytest.raises(TypeError):
        lib.BlockNorm(w_pre=torch.zeros(4), w_post=torch.zeros(4, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        lib.BlockNorm(w_pre=torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError):
        lib.BlockNorm(gate=torch.zeros(4, 4))
    with pytest.raises(ValueError):
        lib._buf(x, "x", (4, 64), 0)
    with pytest.raises(ValueError):
        lib._buf(x, "x", (4, 63), -1)
    with pytest.raises(TypeError):
        lib._buf(x, "x", (4, 64), -1, torch.float32)
    with pytest.raises(ValueError):
        lib._buf(x.t(), "x", (64, 4), -1)
    with pytest.raises(TypeError):
        lib._dt_of(torch.zeros(2, dtype=torch.float16))
    assert lib._buf(None, "x", (4, 4), 0) is None and lib._buf(x, "x", (4, 64), -1) == x.data_ptr()
