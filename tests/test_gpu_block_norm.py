"""The norms around a block, forward and backward, against float64
(oracle/block_norm.py).

Bounds.  u = 2^-24 is half an ulp of fp32 relative to the value.  A thread adds
at most 32 values of a row in sequence and a tree of at most 10 levels joins the
threads, so a sum over a row is off by at most 42 u of the sum of absolute
values; the factor rstd by half of that plus 4 u for the quotient, the sum with
eps, the root and the reciprocal.  An output takes at most 10 further fp32
operations.  So every output is within 64 u of the sum of the absolute values
of its terms, plus the rounding to its type (half a step, 2^-8 relative for
bf16).  Sums over M tokens add at most M values in sequence on top.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_10_b200 as q
    assert torch.cuda.is_available()
    return q


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, ref, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -133 if got.dtype == BF else 2.0 ** -149      # half a subnormal step
    g = _f64(got)
    assert np.all(np.isfinite(g)), what
    excess = np.abs(g - ref) - (bound + half * (np.abs(ref) + bound) + tiny)
    assert np.all(excess <= 0), f"{what}: off by {np.max(excess):.3e} more than the bound allows"


class Case:
    def __init__(self, q, M, D, xt=BF, ht=BF, yt=BF, wt=BF, post=True, gate_rows=0, alpha=1.0, offset=0.0, seed=0,
                 h=True, eps=1e-6):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + M * 31 + D)
        r = lambda *s, k=1.0: torch.randn(*s, generator=g, device="cuda") * k  # noqa: E731
        self.M, self.D, self.yt, self.eps = M, D, yt, eps
        self.x = r(M, D).to(xt)
        if D > 8:
            self.x[:, D // 3] *= 30
        self.h = r(M, D, k=0.5).to(ht) if h else None
        self.w_pre = (1 - offset + 0.2 * r(D)).to(wt)
        self.w_post = (1 - offset + 0.2 * r(D)).to(wt) if post else None
        G = -(-M // gate_rows) if gate_rows else 0
        self.gate = r(G, D).to(wt) if G else None
        self.gate_rows, self.alpha, self.offset = gate_rows, alpha, offset
        self.norm = q.BlockNorm(self.w_pre, self.w_post, self.gate, gate_rows, alpha=alpha, eps=eps, w_offset=offset)
        self.rstd_pre, self.rstd_post = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        self.x_out = torch.empty_like(self.x)
        self.y = torch.empty(M, D, dtype=yt, device="cuda")
        self.dx_out, self.dy = r(M, D).to(xt), r(M, D).to(yt)

    def forward(self, q, **k):
        q.qlora_block_norm_fwd(self.norm, self.x, self.h, self.x_out, self.y, self.rstd_pre, self.rstd_post, **k)

    def check_forward(self, what=""):
        p = dict(w_post=_f64(self.w_post), gate=_f64(self.gate), gate_rows=self.gate_rows, alpha=self.alpha,
                 eps=self.eps, w_offset=self.offset)
        x, h = _f64(self.x), _f64(self.h)
        if h is None:
            f, rp, mag = self.alpha * x, None, np.abs(self.alpha * x)
        else:
            f, rp = O.post(x, h, **p)
            mag = np.abs(self.alpha * x) + np.abs(f - self.alpha * x)
        _close(self.x_out, f, 64 * U * mag, what + " x_out")
        if rp is not None:
            _close(self.rstd_post, rp, 64 * U * rp, what + " rstd_post")
        y, rx = O.pre(_f64(self.x_out), _f64(self.w_pre), eps=self.eps, w_offset=self.offset)
        w_abs = np.abs(_f64(self.w_pre)) + abs(self.offset)       # the weight's own sum with the offset
        _close(self.y, y, 64 * U * np.abs(_f64(self.x_out)) * rx[:, None] * w_abs, what + " y")
        _close(self.rstd_pre, rx, 64 * U * rx, what + " rstd_pre")

    def backward(self, q, sums=True, dx_out=True, dy=True, **k):
        G = self.gate.shape[0] if self.gate is not None else 0
        dev = dict(device="cuda")
        o = {"dx": torch.empty_like(self.x), "dh": torch.empty_like(self.h) if self.h is not None else None}
        o["dw_pre"] = torch.full((self.D,), float("nan"), **dev) if sums and dy else None
        o["dw_post"] = torch.full((self.D,), float("nan"), **dev) if sums and self.w_post is not None and self.h is not None else None
        o["dgate"] = torch.full((G, self.D), float("nan"), **dev) if sums and G and self.h is not None else None
        ws = torch.empty(max(16, q.qlora_workspace_size(q.QL_OP_BLOCK_NORM_BWD, self.M, self.D, self.gate_rows)),
                         dtype=torch.uint8, device="cuda")
        q.qlora_block_norm_bwd(self.norm, self.x_out, self.h, self.rstd_pre, self.rstd_post,
                               self.dx_out if dx_out else None, self.dy if dy else None, o["dx"], o["dh"],
                               dw_pre=o["dw_pre"], dw_post=o["dw_post"], dgate=o["dgate"], ws=ws, **k)
        return o

    def check_backward(self, o, dx_out=True, dy=True, what=""):
        ref = O.backward(_f64(self.x_out), _f64(self.h), _f64(self.dx_out) if dx_out else None,
                         _f64(self.dy) if dy else None, _f64(self.w_pre), _f64(self.w_post), _f64(self.gate),
                         self.gate_rows, self.alpha, self.eps, self.offset)
        # a weight stored around zero: its sum with the offset is off by u of the larger term
        spread = 1.0 if self.offset == 0 else 4.0
        for name, t in o.items():
            if t is not None:
                terms = 64 if name in ("dx", "dh") else 64 + self.M
                # dh and the sums build on dr, which carries an error of its own
                terms *= 1 if name == "dx" else 3
                _close(t, ref[name], spread * terms * U * ref[name + "_abs"], f"{what} {name}")


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 9), (9, 64), (33, 1000), (17, 1001), (64, 1024), (9, 1032), (40, 2051),
          (300, 4096), (7, 4100), (5, 8192), (3, 8205), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("M,D", SHAPES)
def test_shapes(q, M, D):
    c = Case(q, M, D, gate_rows=max(1, M // 2))
    c.forward(q)
    c.check_forward()
    c.check_backward(c.backward(q))


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("ht", [BF, F32])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32])
def test_types(q, xt, ht, yt, wt):
    for M, D in ((13, 520), (11, 515), (6, 1544), (5, 1541), (3, 8200), (3, 4099)):
        c = Case(q, M, D, xt, ht, yt, wt, gate_rows=4, alpha=0.5, offset=1.0)
        c.forward(q)
        c.check_forward(f"{M}x{D}")
        c.check_backward(c.backward(q), what=f"{M}x{D}")


@pytest.mark.parametrize("gate_rows", [0, 1, 2, 3, 7, 299, 300, 1000])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("D", [1032, 1035])
def test_gates(q, gate_rows, post, D):
    """One gate per token, per few tokens with a ragged last group, one for all, none."""
    c = Case(q, 300, D, post=post, gate_rows=gate_rows)
    c.forward(q)
    c.check_forward()
    c.check_backward(c.backward(q))


def test_many_rows(q):
    """More rows than the blocks take at once, in several chunks per gate."""
    for D, M in ((264, 5000), (1032, 1700), (1029, 1700), (4104, 700), (4101, 700), (8191, 300)):
        for gate_rows in (0, 1, 3, 333, M):
            c = Case(q, M, D, gate_rows=gate_rows, yt=F32 if D % 2 else BF)
            c.forward(q)
            c.check_forward(f"{M}x{D}/{gate_rows}")
            c.check_backward(c.backward(q), what=f"{M}x{D}/{gate_rows}")
            c.check_backward(c.backward(q, sums=False, dx_out=False), dx_out=False, what=f"{M}x{D}/{gate_rows} frozen")


@pytest.mark.parametrize("D", [96, 99, 2048, 2049])
@pytest.mark.parametrize("M", [21, 300])
def test_parts_left_out(q, M, D):
    c = Case(q, M, D, gate_rows=6)
    c.forward(q)
    for dx_out, dy in ((True, False), (False, True)):
        c.check_backward(c.backward(q, dx_out=dx_out, dy=dy), dx_out, dy)
    frozen, trained = c.backward(q, sums=False), c.backward(q)
    c.check_backward(frozen)
    for name in ("dx", "dh"):
        assert torch.equal(frozen[name], trained[name])
    # the norm in front of the first block: no block output
    n = Case(q, M, D, h=False, post=False)
    n.forward(q)
    n.check_forward()
    n.check_backward(n.backward(q))
    # sums alone, and the stream's gradient alone
    o = {"dw_pre": torch.empty(D, device="cuda"), "dw_post": torch.empty(D, device="cuda"),
         "dgate": torch.empty(c.gate.shape, device="cuda")}
    ws = torch.empty(q.qlora_workspace_size(q.QL_OP_BLOCK_NORM_BWD, M, D, 6), dtype=torch.uint8, device="cuda")
    q.qlora_block_norm_bwd(c.norm, c.x_out, c.h, c.rstd_pre, c.rstd_post, c.dx_out, c.dy, None, None, ws=ws, **o)
    for name in o:
        assert torch.equal(o[name], trained[name]), name
    dx = torch.empty_like(c.x)
    q.qlora_block_norm_bwd(c.norm, c.x_out, None, c.rstd_pre, None, c.dx_out, c.dy, dx, None)
    assert torch.equal(dx, trained["dx"])
    # after the last block: the stream alone
    x_only = torch.empty_like(c.x)
    q.qlora_block_norm_fwd(c.norm, c.x, c.h, x_only, None)
    assert torch.equal(x_only, c.x_out)
    # the norm's output alone
    y_only = torch.empty_like(c.y)
    q.qlora_block_norm_fwd(c.norm, c.x, c.h, None, y_only)
    assert torch.equal(y_only, c.y)


def test_plain_residual_passes_gradients_through(q):
    """No norm and no gate: dh is dx_out, bit for bit, and h is not needed."""
    c = Case(q, 9, 515, post=False)
    dx, dh = torch.empty_like(c.x), torch.empty_like(c.h)
    q.qlora_block_norm_bwd(q.BlockNorm(), None, None, None, None, c.dx_out, None, dx, dh)
    assert torch.equal(dx, c.dx_out) and torch.equal(dh, c.dx_out)


@pytest.mark.parametrize("D", [1024, 1027, 4100])
def test_in_place_and_neighbours_untouched(q, D):
    """x_out may be x and dx may be dx_out; what lies behind the last row stays as it was."""
    M = 6
    c = Case(q, M, D, gate_rows=M)
    c.forward(q)
    o = c.backward(q)
    pad = 4096
    def guarded(t):
        buf = torch.full((M * D + pad,), 7.0, dtype=t.dtype, device="cuda")
        buf[:M * D] = t.reshape(-1)
        return buf, buf[:M * D].view(M, D)
    xb, x = guarded(c.x)
    yb, y = guarded(torch.zeros_like(c.y))
    q.qlora_block_norm_fwd(c.norm, x, c.h, x, y)
    assert torch.equal(x, c.x_out) and torch.equal(y, c.y)
    gb, g = guarded(c.dx_out)
    hb, dh = guarded(torch.zeros_like(c.h))
    q.qlora_block_norm_bwd(c.norm, c.x_out, c.h, c.rstd_pre, c.rstd_post, g, c.dy, g, dh)
    assert torch.equal(g, o["dx"]) and torch.equal(dh, o["dh"])
    for b in (xb, yb, gb, hb):
        assert bool((b[M * D:] == 7.0).all())


def test_a_gate_for_more_rows_than_there_are(q):
    """gate_rows far past M (and past 32 bits) is one gate for all."""
    c = Case(q, 30, 264, gate_rows=30)
    c.forward(q)
    want = c.x_out.clone()
    c.norm = q.BlockNorm(c.w_pre, c.w_post, c.gate, 2 ** 62)
    c.forward(q)
    assert torch.equal(c.x_out, want)
    assert torch.equal(c.backward(q)["dgate"], Case.backward(c, q)["dgate"])


def test_no_gradient_at_all_is_refused(q):
    c = Case(q, 3, 64)
    with pytest.raises(ValueError):
        q.qlora_block_norm_bwd(c.norm, c.x_out, c.h, c.rstd_pre, c.rstd_post, None, None, c.x, None)


@pytest.mark.parametrize("D", [1024, 1025])
def test_no_tokens(q, D):
    c = Case(q, 2, D)
    e = lambda t: t[:0]  # noqa: E731
    q.qlora_block_norm_fwd(c.norm, e(c.x), e(c.h), e(c.x_out), e(c.y), e(c.rstd_pre), e(c.rstd_post))
    dw = torch.ones(D, device="cuda")
    q.qlora_block_norm_bwd(c.norm, e(c.x), e(c.h), e(c.rstd_pre), e(c.rstd_post), e(c.dx_out), e(c.dy), e(c.x_out),
                           e(c.h), dw_pre=dw)
    assert not dw.any()


def test_rows_of_zeros_and_non_finite_rows(q):
    """A zero row has rstd eps^-1/2 and output 0; a row with a NaN or an infinity spoils itself alone."""
    c = Case(q, 6, 520, gate_rows=6)
    c.x[1], c.h[1] = 0, 0
    c.x[3, 5] = float("nan")
    c.h[4, 519] = float("inf")
    c.forward(q)
    assert not c.y[1].any() and not c.x_out[1].any()
    assert abs(c.rstd_post[1].item() - 1e3) < 1e-3 and abs(c.rstd_pre[1].item() - 1e3) < 1e-3
    good = [0, 1, 2, 5]
    assert bool(torch.isfinite(c.y[good].float()).all()) and bool(torch.isnan(c.y[3].float()).all())
    assert bool(torch.isnan(c.y[4].float()).any())


def test_same_bits_every_time_and_on_another_stream(q):
    c = Case(q, 1500, 1032, gate_rows=500)
    c.forward(q)
    first = c.backward(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = c.backward(q, stream=s)
        s.synchronize()
        for name, t in first.items():
            assert torch.equal(t, again[name]), name


def test_captured_forward_and_backward(q):
    """One graph replayed on new values in the same buffers."""
    c = Case(q, 70, 1032, gate_rows=35)
    outs = {"dx": torch.empty_like(c.x), "dh": torch.empty_like(c.h), "dw_pre": torch.empty(1032, device="cuda"),
            "dw_post": torch.empty(1032, device="cuda"), "dgate": torch.empty(2, 1032, device="cuda")}
    ws = torch.empty(q.qlora_workspace_size(q.QL_OP_BLOCK_NORM_BWD, 70, 1032, 35), dtype=torch.uint8, device="cuda")

    def step():
        c.forward(q)
        q.qlora_block_norm_bwd(c.norm, c.x_out, c.h, c.rstd_pre, c.rstd_post, c.dx_out, c.dy, outs["dx"], outs["dh"],
                               outs["dw_pre"], outs["dw_post"], outs["dgate"], ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6):
        d = Case(q, 70, 1032, gate_rows=35, seed=seed)
        for name in ("x", "h", "dx_out", "dy", "w_pre", "w_post", "gate"):
            getattr(c, name).copy_(getattr(d, name))
        graph.replay()
        torch.cuda.synchronize()
        c.check_forward()
        c.check_backward(outs)


def test_gradients_equal_differences_of_the_device_forward(q):
    """Directional differences of the fp32 forward itself.  The forward's values
    are off by about 64 u = 4e-6 and the step is 1e-2, so a difference of sums of
    2000 terms of order 1 is good to 2000^(1/2) 4e-6 / 1e-2 = 2e-2 in absolute
    terms; the curvature adds (1e-2)^2 of the directional derivative."""
    c = Case(q, 10, 200, F32, F32, F32, F32, gate_rows=4)
    c.forward(q)
    o = c.backward(q)
    dev = lambda t: torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))  # noqa: E731

    def value():
        c.forward(q)
        return float((c.x_out.double() * c.dx_out.double()).sum() + (c.y.double() * c.dy.double()).sum())
    for name, arg in (("dx", c.x), ("dh", c.h), ("dw_pre", c.w_pre), ("dw_post", c.w_post), ("dgate", c.gate)):
        direction, keep = dev(arg), arg.clone()
        want = float((o[name].double() * direction.double()).sum())
        arg.copy_(keep + 1e-2 * direction)
        up = value()
        arg.copy_(keep - 1e-2 * direction)
        got = (up - value()) / 2e-2
        arg.copy_(keep)
        assert abs(got - want) <= 2e-2 + 2e-3 * abs(want) + 1e-3 * float(o[name].double().norm()), (name, got, want)
