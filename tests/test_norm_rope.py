"""norm_rope, norm_rope_backward and norm_rope_kv_append: refusals on the host
(no GPU needed), then values against plain 64-bit formulas at the layouts,
widths, strides, types and indices where they can go wrong.

Tolerances: r takes a sum of up to 512 squares, at most 64 of them one after
another in FP32, then 5 joins, a root of 2 units and two products: below 2^-18
of every normed value; a turn adds two roundings.  The result is rounded once
(half a step of the type), on top of at most 2^-18 of the pair's magnitudes."""
import math

import pytest
import torch

from kv_insert_gb300 import _build
from kv_insert_gb300 import qkv_front as qf

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
LAYOUTS = ("interleaved", "half")
ROUND = 2.0 ** -18

X, O, POS, CS, W, G, WS, DW, SL, CACHE, K, V = ((i + 1) << 40 for i in range(12))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qf.load()


@pytest.fixture(scope="module")
def dev(lib):
    qf.status()
    return torch.device("cuda:0")


# ---- host refusals -----------------------------------------------------------

def norm_call(lib, **kw):
    a = dict(x=X, xt=512, xh=64, w=W, wd=0, pos=POS, cs=CS, rows=128, o=O, ot=512, oh=64, T=4, H=8, D=64, rot=64,
             lay=0, eps=1e-6, dt=0)
    a.update(kw)
    code = lib.norm_rope(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.norm_rope_unsupported(*a.values())) > 5
    return code


def test_norm_rope_refusals(lib):
    assert norm_call(lib, T=-1) == 1 and norm_call(lib, T=(1 << 24) + 1) == 1
    for kw in (dict(dt=3), dict(H=0), dict(D=514), dict(rot=63), dict(rot=66), dict(lay=2), dict(oh=32), dict(wd=1),
               dict(wd=3), dict(dt=1, wd=0)):
        assert norm_call(lib, **kw) == 10, kw
    for eps in (-1e-6, 1.5, math.nan, math.inf):
        assert norm_call(lib, eps=eps) == 9
    assert norm_call(lib, x=0) == 3 and norm_call(lib, w=W + 1) == 4 and norm_call(lib, w=W + 2, wd=2) == 4
    assert norm_call(lib, w=O + 64) == 9 and norm_call(lib, o=X + 64) == 9
    assert norm_call(lib, T=0, x=0) == 0
    if not torch.cuda.is_available():
        assert norm_call(lib) in (5, 6) and norm_call(lib, w=0) in (5, 6) and norm_call(lib, o=X) in (5, 6)
        assert norm_call(lib, wd=2) in (5, 6) and norm_call(lib, eps=0.0) in (5, 6)


def back_call(lib, **kw):
    a = dict(g=G, gt=512, gh=64, x=X, xt=512, xh=64, w=W, wd=0, pos=POS, cs=CS, rows=128, dx=O, dt_=512, dh=64, dw=DW,
             dwd=2, T=4, H=8, D=64, rot=64, lay=0, eps=1e-6, dt=0, ws=WS, n=1 << 30)
    a.update(kw)
    code = lib.norm_rope_backward(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.norm_rope_backward_unsupported(*a.values())) > 5
    return code


def test_norm_rope_backward_refusals(lib):
    assert back_call(lib, T=-1) == 1
    for kw in (dict(dt=3), dict(xt=-8), dict(xh=(1 << 36) + 1), dict(dwd=1), dict(rot=0), dict(dh=32)):
        assert back_call(lib, **kw) == 10, kw
    assert back_call(lib, w=0) == 9                                  # a gradient of no weight
    for name in ("g", "x", "dx", "ws", "pos"):
        assert back_call(lib, **{name: 0}) == 3, name
    assert back_call(lib, x=X + 1) == 4 and back_call(lib, ws=WS + 128) == 4 and back_call(lib, dw=DW + 2) == 4
    assert back_call(lib, dx=X) == 9 and back_call(lib, dx=X + 64) == 9 and back_call(lib, dw=X) == 9
    assert back_call(lib, ws=X - 4096) == 9 and back_call(lib, dw=W) == 9 and back_call(lib, dw=G) == 9
    assert back_call(lib, T=0, dw=0, x=0) == 0
    if not torch.cuda.is_available():
        assert back_call(lib) in (5, 6) and back_call(lib, dx=G) in (5, 6)
        assert back_call(lib, w=0, dw=0, ws=0, n=0) in (5, 6) and back_call(lib, xh=0, xt=64) in (5, 6)


def append_call(lib, **kw):
    a = dict(q=X, qt=512, qh=64, k=K, kt=128, kh=64, v=V, vt=128, vh=64, qw=W, kw=W + 4096, wd=0, pos=POS, sl=SL, cs=CS,
             rows=128, o=O, ot=512, oh=64, c=CACHE, pages=8, T=4, H=8, nkv=2, D=64, rot=64, lay=0, eps=1e-6, dt=0)
    a.update(kw)
    code = lib.norm_rope_kv_append(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.norm_rope_kv_append_unsupported(*a.values())) > 5
    return code


def test_norm_rope_kv_append_refusals(lib):
    assert append_call(lib, T=-1) == 1 and append_call(lib, dt=2) == 10 and append_call(lib, wd=1) == 10
    assert append_call(lib, eps=2.0) == 9 and append_call(lib, qw=CACHE) == 9 and append_call(lib, kw=O) == 9
    assert append_call(lib, kw=W + 1) == 4 and append_call(lib, k=0) == 3
    assert append_call(lib, T=0, k=0) == 0
    if not torch.cuda.is_available():
        assert append_call(lib) in (5, 6) and append_call(lib, qw=0, kw=0) in (5, 6)
        assert append_call(lib, H=0, q=0, o=0) in (5, 6)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 3, 64, dtype=BF), torch.zeros(64, dtype=BF)
    pos, cs = torch.zeros(2, dtype=torch.int64), torch.zeros(8, 64)
    assert "CUDA" in qf.norm_rope_unsupported(x, w, pos, cs, x)
    assert "CUDA" in qf.norm_rope_backward_unsupported(x, x, w, pos, cs, x)
    with pytest.raises(ValueError):
        qf.norm_rope(x, w, pos, cs, out=x)


# ---- values ------------------------------------------------------------------

def table(rows, rot, dev="cuda"):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def pairs_of(rot, layout):
    i = torch.arange(rot // 2, device="cuda")
    return (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)


def turn(x, rows, layout, sign=1.0):
    """x (64 bits) turned, and the magnitudes that the turn adds up."""
    rot = rows.shape[1]
    a, b = pairs_of(rot, layout)
    c, s = rows[:, None, :rot // 2].double(), sign * rows[:, None, rot // 2:].double()
    y, m = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    m[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    m[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, m


def normed(x, w, eps):
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def close(got, ref, mags, dtype, factor=ROUND):
    tol = torch.finfo(dtype).eps / 2 * ref.abs() + factor * mags + 2.0 ** -25
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got.double() - ref).abs() / tol).max())}"


def inputs(T, H, D, rot, dtype, rows=300, seed=0, wdtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, device="cuda") * torch.exp(torch.randn(T, H, 1, generator=g, device="cuda"))
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wdtype or dtype)
    pos = torch.randint(0, rows, (T,), generator=g, device="cuda")
    grad = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    return x.to(dtype), w, pos, table(rows, rot), grad


SHAPES = [(1, 1, 64, 64), (8, 64, 64, 64), (33, 5, 128, 128), (37, 9, 80, 32), (5, 3, 96, 96), (301, 7, 128, 64),
          (7, 2, 256, 256), (6, 3, 512, 512), (9, 4, 512, 16), (3, 2, 8, 8), (11, 3, 128, 82), (13, 1, 130, 130),
          (4, 3, 2, 2), (10, 17, 64, 2), (5, 6, 100, 36), (65, 33, 24, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("T,H,D,rot", SHAPES)
def test_norm_rope_values(dev, T, H, D, rot, dtype, layout):
    x, w, pos, cs, _ = inputs(T, H, D, rot, dtype, wdtype=FL if T % 2 else None)
    ref, mags = turn(normed(x, w, 1e-6), cs[pos], layout)
    close(qf.norm_rope(x, w, pos, cs, layout=layout), ref, mags, dtype)
    ref, mags = turn(normed(x, None, 1e-2), cs[pos], layout)
    close(qf.norm_rope(x, None, pos, cs, eps=1e-2, layout=layout), ref, mags, dtype)
    y = x.clone()
    assert qf.norm_rope(y, w, pos, cs, out=y, layout=layout) is y     # in place
    assert torch.equal(y, qf.norm_rope(x, w, pos, cs, layout=layout))
    assert qf.status() == 0


def check_grads(dx, dw, grad, x, w, pos, cs, layout, eps, dtype):
    g, gm = turn(grad.double(), cs[pos], layout, -1.0)
    X = x.double()
    ms = X.square().mean(-1, keepdim=True) + eps
    r = ms.rsqrt()
    W = torch.ones(x.shape[2], device="cuda", dtype=torch.float64) if w is None else w.double()
    ref = r * g * W - X * r ** 3 * (g * W * X).mean(-1, keepdim=True)
    # as for the norm, twice (r and r^3), and a second sum of D products
    mags = r * gm * W.abs() + X.abs() * r ** 3 * (gm * W.abs() * X.abs()).mean(-1, keepdim=True)
    close(dx, ref, mags, dtype, 4 * ROUND)
    if w is None:
        assert dw is None
        return
    # at most 512 partial sums one after another, in FP32
    close(dw, (g * X * r).sum((0, 1)), (gm * X.abs() * r).sum((0, 1)), dw.dtype, 512 * 2.0 ** -24 + 4 * ROUND)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("T,H,D,rot", SHAPES + [(4099, 25, 80, 32)])
def test_norm_rope_backward_values(dev, T, H, D, rot, dtype, layout):
    x, w, pos, cs, grad = inputs(T, H, D, rot, dtype, wdtype=FL if T % 2 else None)
    dx, dw = qf.norm_rope_backward(grad, x, w, pos, cs, layout=layout)
    assert dw.dtype == FL
    check_grads(dx, dw, grad, x, w, pos, cs, layout, 1e-6, dtype)
    again = qf.norm_rope_backward(grad, x, w, pos, cs, layout=layout)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])     # bit for bit
    narrow = torch.empty(D, dtype=dtype, device="cuda")
    qf.norm_rope_backward(grad, x, w, pos, cs, layout=layout, grad_weight=narrow)
    assert torch.equal(narrow, dw.to(dtype))
    g = grad.clone()
    dx2, none = qf.norm_rope_backward(g, x, None, pos, cs, layout=layout, grad_x=g)   # in place, no weight
    assert none is None and dx2 is g
    check_grads(g, None, grad, x, None, pos, cs, layout, 1e-6, dtype)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradients_against_differences(dev, layout):
    """fp32: directional derivatives of a smooth loss by central differences of
    the 64-bit formula (step 1e-4: the truncation is below 1e-6 of the value)."""
    x, w, pos, cs, grad = inputs(5, 3, 32, 16, FL, seed=3)
    x.requires_grad_(), w.requires_grad_()
    y = qf.norm_rope(x, w, pos, cs, layout=layout)
    dx, dw = torch.autograd.grad((y * grad).sum(), (x, w))
    g = torch.Generator(device="cuda").manual_seed(9)

    def loss(X, W):
        return float((turn(normed(X, W, 1e-6), cs[pos], layout)[0] * grad.double()).sum())
    for _ in range(4):
        ex = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64) * x.detach().abs().mean()
        ew = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        X, W, h = x.detach().double(), w.detach().double(), 1e-4
        num = (loss(X + h * ex, W) - loss(X - h * ex, W)) / (2 * h)
        assert abs(num - float((dx.double() * ex).sum())) < 1e-4 * float((dx.double() * ex).abs().sum())
        num = (loss(X, W + h * ew) - loss(X, W - h * ew)) / (2 * h)
        assert abs(num - float((dw.double() * ew).sum())) < 1e-4 * float((dw.double() * ew).abs().sum())


@pytest.mark.gpu
def test_autograd_graph(dev):
    x, w, pos, cs, grad = inputs(33, 4, 64, 64, BF)
    x.requires_grad_(), w.requires_grad_()
    y = qf.norm_rope(x, w, pos, cs, layout="half")
    y.backward(grad)
    dx, dw = qf.norm_rope_backward(grad, x.detach(), w.detach(), pos, cs, layout="half")
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw.to(BF))
    # only the weight, only x, no weight; a gradient that is one value expanded
    for a, b in ((x.detach(), w), (x, w.detach()), (x, None)):
        for t in (x, w):
            t.grad = None
        qf.norm_rope(a, b, pos, cs, layout="half").sum().backward()
        one = torch.ones_like(grad)
        dx, dw = qf.norm_rope_backward(one, x.detach(), None if b is None else w.detach(), pos, cs, layout="half")
        assert (x.grad is None) == (a is not x) and (w.grad is None) == (b is not w)
        assert x.grad is None or torch.equal(x.grad, dx)
        assert w.grad is None or torch.equal(w.grad, dw.to(BF))
    # a shared weight (q and k of one layer): its gradients add up
    w.grad = None
    (qf.norm_rope(x, w, pos, cs) * grad).sum().backward(retain_graph=False)
    once = w.grad.clone()
    w.grad = None
    ((qf.norm_rope(x, w, pos, cs) + qf.norm_rope(x, w, pos, cs)) * grad).sum().backward()
    assert torch.equal(w.grad, 2 * once)
    with pytest.raises(RuntimeError):   # no graph of the gradient
        (d,) = torch.autograd.grad(qf.norm_rope(x, w, pos, cs).float().square().sum(), x, create_graph=True)
        d.sum().backward()
    with pytest.raises(ValueError, match="out"):
        qf.norm_rope(x, w, pos, cs, out=torch.empty_like(x))
    with pytest.raises(ValueError, match="cos_sin"):
        qf.norm_rope(x, w, pos, cs.clone().requires_grad_())
    with torch.no_grad():
        assert not qf.norm_rope(x, w, pos, cs, out=torch.empty_like(x)).requires_grad
    y = qf.norm_rope(x, w, pos, cs)
    with torch.no_grad():
        x.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


@pytest.mark.gpu
def test_capture(dev):
    """Captured calls repeat on new contents; what belongs to an autograd graph is refused under capture."""
    x, w, pos, cs, grad = inputs(17, 5, 128, 128, BF)
    out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(128, device="cuda")
    ws = torch.empty(qf.norm_rope_backward_workspace_bytes(17, 5, 128), dtype=torch.uint8, device="cuda")

    def step():
        qf.norm_rope(x, w, pos, cs, out=out)
        qf.norm_rope_backward(grad, x, w, pos, cs, grad_x=dx, grad_weight=dw, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.mul_(-0.5), grad.mul_(3), pos.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, qf.norm_rope(x, w, pos, cs))
    ref = qf.norm_rope_backward(grad, x, w, pos, cs)
    assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    w.requires_grad_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        refused = torch.cuda.CUDAGraph()
        refused.capture_begin()
        try:
            with pytest.raises(ValueError, match="capture"):
                qf.norm_rope(x, w, pos, cs)
            qf.norm_rope(x, w.detach(), pos, cs, out=out)
        finally:
            refused.capture_end()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FL])
def test_strides_and_alignment(dev, dtype, layout):
    """Packed rows, transposed heads, a broadcast gradient, rows off the 16-byte grid: the same bits or values."""
    T, H, D = 19, 6, 64
    x, w, pos, cs, grad = inputs(T, H, D, 64, dtype)
    want = qf.norm_rope(x, w, pos, cs, layout=layout)
    want_dx, want_dw = qf.norm_rope_backward(grad, x, w, pos, cs, layout=layout)
    packed = torch.zeros(T, H + 5, D, dtype=dtype, device="cuda")
    packed[:, 2:2 + H] = x
    swapped = x.transpose(0, 1).contiguous().transpose(0, 1)
    for v in (packed[:, 2:2 + H], swapped):
        out = torch.empty(H, T, D, dtype=dtype, device="cuda").transpose(0, 1)
        assert torch.equal(qf.norm_rope(v, w, pos, cs, out=out, layout=layout), want)
        dx, dw = qf.norm_rope_backward(grad, v, w, pos, cs, layout=layout, grad_x=out)
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
    buf = torch.zeros(T * H * D + 1, dtype=dtype, device="cuda")[1:].view(T, H, D)
    buf.copy_(x)
    ref, mags = turn(normed(x, w, 1e-6), cs[pos], layout)
    close(qf.norm_rope(buf, w, pos, cs, layout=layout), ref, mags, dtype)
    odd_w = torch.zeros(D + 1, dtype=dtype, device="cuda")[1:]
    odd_w.copy_(w)
    close(qf.norm_rope(x, odd_w, pos, cs, layout=layout), ref, mags, dtype)
    dx, dw = qf.norm_rope_backward(grad, buf, odd_w, pos, cs, layout=layout)
    check_grads(dx, dw, grad, x, w, pos, cs, layout, 1e-6, dtype)
    one = grad[:, :1].expand(T, H, D)
    dx, dw = qf.norm_rope_backward(one, x, w, pos, cs, layout=layout)
    check_grads(dx, dw, one, x, w, pos, cs, layout, 1e-6, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 130])
def test_bad_positions(dev, D):
    """Tokens off the table: outputs kept, or zeros in new ones; nothing in the weight's gradient; flagged."""
    x, w, pos, cs, grad = inputs(9, 3, D, D, BF)
    good = torch.tensor([0, 2, 3, 5, 6, 7], device="cuda")
    bad = torch.tensor([1, 4, 8], device="cuda")
    pos[bad] = torch.tensor([300, -1, 1 << 40], device="cuda")
    want = qf.norm_rope(x[good], w, pos[good], cs)
    dxg, dwg = qf.norm_rope_backward(grad[good], x[good], w, pos[good], cs)
    assert qf.status() == 0
    out = torch.full_like(x, 7.0)
    qf.norm_rope(x, w, pos, cs, out=out)
    assert qf.status() == 2
    assert torch.equal(out[good], want) and (out[bad] == 7).all()
    y = qf.norm_rope(x, w, pos, cs)
    assert torch.equal(y[good], want) and (y[bad] == 0).all()
    x[bad] = math.nan
    dx, dw = qf.norm_rope_backward(grad, x, w, pos, cs)
    assert torch.equal(dx[good], dxg) and (dx[bad] == 0).all() and torch.isfinite(dw).all()
    torch.testing.assert_close(dw, dwg, rtol=1e-4, atol=1e-4 * float(dwg.abs().max()))   # (other groups of rows)
    dx = torch.full_like(x, 7.0)
    qf.norm_rope_backward(grad, x, w, pos, cs, grad_x=dx)
    assert torch.equal(dx[good], dxg) and (dx[bad] == 7).all()
    assert qf.status() == 2


@pytest.mark.gpu
def test_odd_values(dev):
    """Zeros, infinities and NaN stay in their head; no tokens at all."""
    x, w, pos, cs, grad = inputs(5, 4, 64, 32, BF)
    want = qf.norm_rope(x, w, pos, cs)
    x[1, 2] = 0.0
    x[3, 1, 5] = math.inf
    x[4, 0, 60] = math.nan
    y = qf.norm_rope(x, w, pos, cs)
    same = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    same[1, 2] = same[3, 1] = same[4, 0] = False
    assert torch.equal(y[same], want[same]) and (y[1, 2] == 0).all() and y[4, 0].isnan().all()
    assert y[3, 1].isnan().any()
    for tiny in (1e-30, 1e18):   # squares far below eps, and near the end of FP32
        z = torch.full((1, 1, 64), tiny, device="cuda")
        got = qf.norm_rope(z, None, pos[:1], cs)
        ref, mags = turn(normed(z, None, 1e-6), cs[pos[:1]], "interleaved")
        close(got, ref, mags, FL)
    assert qf.norm_rope(x[:0], w, pos[:0], cs).shape == (0, 4, 64)
    dx, dw = qf.norm_rope_backward(grad[:0], x[:0], w, pos[:0], cs)
    assert dx.shape == (0, 4, 64) and (dw == 0).all()
    assert qf.status() == 0


@pytest.mark.gpu
def test_streams(dev):
    """Calls on a stream of their own, behind the kernels that make their inputs."""
    side = torch.cuda.Stream()
    x, w, pos, cs, grad = inputs(400, 16, 128, 128, BF)
    want = qf.norm_rope(2 * x, w, pos, cs)
    want_dx, want_dw = qf.norm_rope_backward(grad, 2 * x, w, pos, cs)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            y = 2 * x
            got = qf.norm_rope(y, w, pos, cs)
        dx, dw = qf.norm_rope_backward(grad, y, w, pos, cs, stream=side)
        raw = qf.norm_rope(y, w, pos, cs, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(dx, want_dx) and torch.equal(dw, want_dw) and torch.equal(raw, want)


@pytest.mark.gpu
def test_large_calls(dev):
    """More rows than one pass of the grid, strides that pass 2^31 elements."""
    T, H, D = 20011, 9, 128
    x, w, pos, cs, grad = inputs(T, H, D, 128, BF)
    y = qf.norm_rope(x, w, pos, cs, layout="half")
    dx, dw = qf.norm_rope_backward(grad, x, w, pos, cs, layout="half")
    at = torch.tensor([0, 1, 777, T - 2, T - 1], device="cuda")
    ref, mags = turn(normed(x[at], w, 1e-6), cs[pos[at]], "half")
    close(y[at], ref, mags, BF)
    check_grads(dx, dw, grad, x, w, pos, cs, "half", 1e-6, BF)
    base = torch.empty((1 << 31) + 4096, dtype=BF, device="cuda")
    far = torch.as_strided(base, (2, 3, 128), (1 << 31, 128, 1))
    far.copy_(x[:2, :3])
    assert torch.equal(qf.norm_rope(far, w, pos[:2], cs, layout="half"), y[:2, :3])
    qf.norm_rope(x[:2, :3], w, pos[:2], cs, out=far, layout="half")
    assert torch.equal(far, y[:2, :3])


@pytest.mark.gpu
@pytest.mark.parametrize("T,nkv,group,D,rot,layout,dtype", [
    (1, 1, 1, 64, 64, "interleaved", BF), (33, 8, 4, 128, 128, "half", BF), (70, 3, 5, 128, 64, "half", HF),
    (17, 2, 7, 80, 78, "interleaved", HF), (9, 16, 1, 96, 36, "half", BF), (300, 1, 8, 256, 256, "half", BF)])
def test_append(dev, T, nkv, group, D, rot, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    hq, rows = nkv * group, 300
    row = torch.randn(T, (hq + 2 * nkv) * D, generator=g, device="cuda").to(dtype)
    q, k, v = (row[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, hq), (hq, hq + nkv), (hq + nkv, hq + 2 * nkv)))
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2))
    pos, cs = torch.randint(0, rows, (T,), generator=g, device="cuda"), table(rows, rot)
    pages = -(-T // 16) + 3
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:T]
    cache = torch.randn(pages, nkv, 16, 2 * D, generator=g, device="cuda").to(dtype)
    old = cache.clone()
    if T > 4:
        slots[1], slots[2], pos[3] = -5, pages * 16, rows
    out = qf.norm_rope_kv_append(q, k, v, qw, kw, pos, slots, cs, cache, layout=layout)
    assert qf.status() == (3 if T > 4 else 0)
    fine = torch.ones(T, dtype=torch.bool, device="cuda")
    if T > 4:
        fine[3] = False
        assert (out[3] == 0).all()
    ref, mags = turn(normed(q[fine], qw, 1e-6), cs[pos[fine]], layout)
    close(out[fine], ref, mags, dtype)
    if T > 4:
        fine[1] = fine[2] = False
    at = slots[fine]
    flat = cache.permute(0, 2, 1, 3).reshape(-1, nkv, 2 * D)
    ref, mags = turn(normed(k[fine], kw, 1e-6), cs[pos[fine]], layout)
    close(flat[at][..., :D], ref, mags, dtype)
    assert torch.equal(flat[at][..., D:], v[fine])
    rest = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(flat[rest], old.permute(0, 2, 1, 3).reshape(-1, nkv, 2 * D)[rest])
    # without weights, append only, fp32 weights, q in place
    c2, c3 = old.clone(), old.clone()
    qf.norm_rope_kv_append(None, k, v, None, kw.float(), pos, slots, cs, c2, layout=layout)
    assert torch.equal(c2, cache)
    q2 = qf.norm_rope_kv_append(q, k, v, None, kw, pos, slots, cs, c3, q_out=q, layout=layout)
    assert torch.equal(c3, cache) and q2 is q
    qf.status()


@pytest.mark.gpu
def test_same_numbers_with_and_without_the_cache(dev):
    """norm_rope of q, and rope's cache, from the fused call."""
    T, nkv, hq, D = 50, 4, 12, 64
    x, w, pos, cs, _ = inputs(T, hq, D, 64, BF)
    k, _, _, _, v = inputs(T, nkv, D, 64, BF, seed=5)
    cache = torch.zeros(8, nkv, 16, 2 * D, dtype=BF, device="cuda")
    slots = torch.arange(T, device="cuda")
    q = qf.norm_rope_kv_append(x, k, v, w, w, pos, slots, cs, cache)
    assert torch.equal(q, qf.norm_rope(x, w, pos, cs))
    flat = cache.permute(0, 2, 1, 3).reshape(-1, nkv, 2 * D)[:T]
    assert torch.equal(flat[..., :D], qf.norm_rope(k, w, pos, cs)) and torch.equal(flat[..., D:], v)
    assert "dtype" in qf.norm_rope_kv_append_unsupported(x, k, v, w, w.float(), pos, slots, cs, cache)
    assert qf.norm_rope_kv_append_unsupported(x, k, v, w, w, pos, slots, cs, cache) is None
    assert qf.norm_rope_unsupported(x, w, pos, cs, x) is None
    assert "weight" in qf.norm_rope_unsupported(x, w.double(), pos, cs, x)
    assert "workspace" in qf.norm_rope_backward_unsupported(x, x, w, pos, cs, torch.empty_like(x), w.clone(),
                                                            torch.empty(256, dtype=torch.uint8, device="cuda"))


def check_scaled(dx, grad, x, w, pos, cs, layout, eps):
    """As check_grads, without an absolute term: the gradient may be of any size."""
    g, gm = turn(grad.double(), cs[pos], layout, -1.0)
    X, W = x.double(), w.double()
    r = (X.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = X * r
    ref = r * (g * W - n * (g * W * n).mean(-1, keepdim=True))
    mags = r * (gm * W.abs() + n.abs() * (gm * W.abs() * n.abs()).mean(-1, keepdim=True))
    tol = torch.finfo(dx.dtype).eps / 2 * ref.abs() + 4 * ROUND * mags
    assert dx.isfinite().all()
    assert ((dx.double() - ref).abs() <= tol).all(), float(((dx.double() - ref).abs() / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("size,eps", [(1e-18, 0.0), (1e-15, 0.0), (1e-15, 1e-30), (1e-13, 0.0), (1.0, 0.0), (1e13, 1e-6),
                                      (1e16, 1e-6), (1e17, 1e-6)])
def test_gradients_at_the_ends_of_the_range(dev, size, eps, dtype, layout):
    """r^3 alone leaves FP32 long before the gradient does (r is 1e18 to 1e-17 here; the squares stay in range):
    chunks of a head, half pairs through shared memory, rows off the 16-byte grid."""
    for T, H, D, rot in ((7, 3, 64, 64), (6, 5, 24, 12), (5, 2, 130, 82)):
        x, w, pos, cs, grad = inputs(T, H, D, rot, FL)
        x = (size * x / x.square().mean(-1, keepdim=True).sqrt()).to(dtype)
        w, grad = w.to(dtype), grad.to(dtype)
        dx, dw = qf.norm_rope_backward(grad, x, w, pos, cs, eps=eps, layout=layout)
        check_scaled(dx, grad, x, w, pos, cs, layout, eps)
        g, gm = turn(grad.double(), cs[pos], layout, -1.0)
        n = x.double() * (x.double().square().mean(-1, keepdim=True) + eps).rsqrt()
        close(dw, (g * n).sum((0, 1)), (gm * n.abs()).sum((0, 1)), FL, 512 * 2.0 ** -24 + 4 * ROUND)


@pytest.mark.gpu
def test_no_weight_gradient(dev, monkeypatch):
    """grad_weight=False: none is formed (nor by a graph whose weight needs none), and x's gradient is the same."""
    x, w, pos, cs, grad = inputs(33, 4, 64, 64, BF)
    dx, dw = qf.norm_rope_backward(grad, x, w, pos, cs)
    seen, run = [], qf._run
    monkeypatch.setattr(qf, "_run", lambda name, index, args, stream: (seen.append((name, args)), run(name, index, args, stream)))
    got, none = qf.norm_rope_backward(grad, x, w, pos, cs, grad_weight=False)
    assert none is None and torch.equal(got, dx)
    x.requires_grad_()
    qf.norm_rope(x, w, pos, cs).backward(grad)
    assert torch.equal(x.grad, dx)
    backs = [args for name, args in seen if name == "norm_rope_backward"]
    assert len(backs) == 2 and all(a[14] == 0 and a[23] == 0 and a[24] == 0 for a in backs)   # dw, workspace, its bytes


@pytest.mark.gpu
def test_written_tensors_that_a_graph_holds(dev):
    """A graph saves x and the weight; a call that overwrites them is seen by its backward pass, as torch's own
    in-place operations are."""
    def graph():
        x, w, pos, cs, grad = inputs(6, 4, 64, 64, BF)
        x.requires_grad_()
        return qf.norm_rope(x, w, pos, cs), x.detach(), w, pos, cs, grad
    cache = torch.zeros(4, 4, 16, 128, dtype=BF, device="cuda")
    slots, starts = torch.arange(6, device="cuda"), torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(qf.chunk_attn_workspace_bytes(6, 1, 4, 4, 64, 1), qf.prefix_attn_workspace_bytes(1, 6, 4, 4, 64, 0, 1)),
                     dtype=torch.uint8, device="cuda")
    for write in (lambda x, w, p, c, g: qf.norm_rope(x, w, p, c, out=x),
                  lambda x, w, p, c, g: qf.rope(x, p, c, out=x),
                  lambda x, w, p, c, g: qf.norm_rope_backward(g, g.clone(), w, p, c, grad_x=x),
                  lambda x, w, p, c, g: qf.norm_rope_backward(g, x, w.clone(), p, c, grad_weight=w),
                  lambda x, w, p, c, g: qf.rope_kv_append(g, g, g, p, slots, c, cache, q_out=x),
                  lambda x, w, p, c, g: qf.norm_rope_kv_append(g, g, g, w, w, p, slots, c, cache, q_out=x),
                  lambda x, w, p, c, g: qf.chunk_attn(g, cache, starts, table, starts[1:], ws, out=x),
                  lambda x, w, p, c, g: qf.prefix_attn(g, cache, None, None, table, starts[1:], ws, q_len=6, out=x)):
        y, x, w, pos, cs, grad = graph()
        write(x, w, pos, cs, grad)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward(grad)
    y, x, w, pos, cs, grad = graph()   # reading them is no change
    qf.norm_rope(x, w, pos, cs)
    y.backward(grad)
    with torch.inference_mode():
        z = torch.zeros_like(grad)
        qf.norm_rope(grad, w, pos, cs, out=z)


def test_forward_mode_is_refused():
    """A tangent would be dropped without a word."""
    x, pos, cs = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int64), torch.zeros(8, 64)
    w = torch.ones(64)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        wd = torch.autograd.forward_ad.make_dual(w, torch.ones_like(w))
        for call in (lambda: qf.norm_rope(dual, w, pos, cs), lambda: qf.norm_rope(x, wd, pos, cs),
                     lambda: qf.norm_rope(dual, None, pos, cs, out=x), lambda: qf.rope(dual, pos, cs),
                     lambda: qf.rope_backward(dual, pos, cs)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        with pytest.raises(ValueError, match="CUDA"):   # no tangent: the other checks
            qf.norm_rope(x, w, pos, cs, out=x)
