"""rope_table, rope / rope_backward and rope_kv_append: refusals on the host
(no GPU needed), then values against plain 64-bit formulas at the layouts,
widths, strides, types and indices where they can go wrong."""
import decimal
import math

import pytest
import torch

from kv_insert_gb300 import _build
from kv_insert_gb300 import qkv_front as qf

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
LAYOUTS = ("interleaved", "half")

# fake, 16-byte aligned addresses: the checks below fail before anything is read
X, O, POS, SL, CS, CACHE, K, V = ((i + 1) << 40 for i in range(8))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qf.load()


@pytest.fixture(scope="module")
def dev(lib):
    qf.status()
    return torch.device("cuda:0")


# ---- host refusals -----------------------------------------------------------

def test_rope_table_refusals(lib):
    ok = dict(t=X, first=0, rows=16, rot=64, base=1e4, sc=0, f=1.0, L=0, slow=1.0, fast=32.0, mag=1.0)

    def call(**kw):
        return lib.rope_table(*dict(ok, **kw).values(), None)
    for rot in (0, 1, 63, 514, -2):
        assert call(rot=rot) == 10
    assert call(rows=-1) == 7 and call(rows=(1 << 32) + 1) == 7 and call(first=-1) == 7
    assert call(base=1.0) == 9 and call(base=math.nan) == 9 and call(sc=4) == 9 and call(sc=-1) == 9
    assert call(sc=1, f=0.5) == 9 and call(sc=1, f=math.inf) == 9 and call(sc=2, rot=2, f=2.0) == 9
    assert call(sc=3, f=2.0) == 9 and call(sc=3, f=2.0, L=8, slow=4.0, fast=4.0) == 9
    assert call(mag=0.0) == 9 and call(mag=math.nan) == 9
    assert call(t=0) == 3 and call(t=X + 4) == 4
    assert call(rows=0, t=0) == 0
    why = lib.rope_table_unsupported(*dict(ok, rot=63).values())
    assert b"rot_dim" in why
    if not torch.cuda.is_available():
        assert call() in (5, 6)


def rope_call(lib, **kw):
    a = dict(x=X, xt=512, xh=64, pos=POS, cs=CS, rows=128, o=O, ot=512, oh=64, T=4, H=8, D=64, rot=64,
             lay=0, inv=0, dt=0)
    a.update(kw)
    code = lib.rope(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.rope_unsupported(*a.values())) > 5
    return code


def test_rope_refusals(lib):
    assert rope_call(lib, T=-1) == 1 and rope_call(lib, T=(1 << 24) + 1) == 1
    for kw in (dict(dt=3), dict(dt=-1), dict(H=0), dict(H=4097), dict(D=0), dict(D=514), dict(rot=63),
               dict(rot=66), dict(rot=0), dict(lay=2), dict(xt=-1), dict(oh=(1 << 36) + 1),
               dict(ot=0), dict(oh=32), dict(ot=448)):   # the last three: out's heads overlap
        assert rope_call(lib, **kw) == 10, kw
    assert rope_call(lib, inv=2) == 9 and rope_call(lib, rows=0) == 7
    assert rope_call(lib, x=0) == 3 and rope_call(lib, o=0) == 3 and rope_call(lib, pos=0) == 3
    assert rope_call(lib, x=X + 1) == 4 and rope_call(lib, x=X + 2, dt=2) == 4
    assert rope_call(lib, cs=CS + 4) == 4 and rope_call(lib, pos=POS + 4) == 4
    assert rope_call(lib, o=X + 64) == 9                       # shifted onto x
    assert rope_call(lib, o=X, ot=1024) == 9                   # x with other strides
    assert rope_call(lib, o=POS - 16) == 9 and rope_call(lib, o=CS + 64) == 9
    assert rope_call(lib, T=0, x=0) == 0
    if not torch.cuda.is_available():   # taken: they reach the device query
        assert rope_call(lib) in (5, 6)
        assert rope_call(lib, o=X) in (5, 6)                   # in place
        assert rope_call(lib, o=X + 1024, xt=1024, ot=1024) in (5, 6)   # other columns of one buffer
        assert rope_call(lib, x=X + 2, xt=513, xh=64) in (5, 6)         # element alignment is enough
        assert rope_call(lib, xt=0, xh=0) in (5, 6)            # a broadcast input
        assert rope_call(lib, T=1, ot=0, H=1, oh=0) in (5, 6)  # strides of a single row do not matter
    assert rope_call(lib, o=X + 1000, xt=1024, ot=1024) == 9   # 12 columns into x's


def append_call(lib, **kw):
    a = dict(q=X, qt=512, qh=64, k=K, kt=128, kh=64, v=V, vt=128, vh=64, pos=POS, sl=SL, cs=CS, rows=128,
             o=O, ot=512, oh=64, c=CACHE, pages=8, T=4, H=8, nkv=2, D=64, rot=64, lay=0, dt=0)
    a.update(kw)
    code = lib.rope_kv_append(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.rope_kv_append_unsupported(*a.values())) > 5
    return code


def test_rope_kv_append_refusals(lib):
    assert append_call(lib, T=-1) == 1
    for kw in (dict(dt=2), dict(H=-1), dict(nkv=0), dict(nkv=1025), dict(D=60), dict(D=520), dict(rot=65),
               dict(rot=66), dict(lay=-1), dict(kt=-8), dict(ot=100)):
        assert append_call(lib, **kw) == 10, kw
    assert append_call(lib, rows=0) == 7 and append_call(lib, pages=0) == 7
    for name in ("q", "k", "v", "pos", "sl", "cs", "o", "c"):
        assert append_call(lib, **{name: 0}) == 3, name
    assert append_call(lib, k=K + 1) == 4 and append_call(lib, c=CACHE + 8) == 4 and append_call(lib, sl=SL + 4) == 4
    for name in ("q", "k", "v", "pos", "sl", "cs", "o"):
        assert append_call(lib, **{name: CACHE + 4096}) == 9, name
    assert append_call(lib, o=X + 64) == 9 and append_call(lib, k=O) == 9 and append_call(lib, cs=O) == 9
    assert append_call(lib, T=0, k=0) == 0
    if not torch.cuda.is_available():
        assert append_call(lib) in (5, 6)
        assert append_call(lib, H=0, q=0, o=0) in (5, 6)       # append only
        # q, k and v in one packed buffer, q rotated in place
        packed = dict(q=X, qt=768, k=X + 1024, kt=768, v=X + 1280, vt=768, o=X, ot=768)
        assert append_call(lib, **packed) in (5, 6)
        assert append_call(lib, **dict(packed, k=X + 1022)) == 9   # k starts inside the last q head


def test_table_on_the_host_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        qf.rope_table(8, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        qf.rope_table(8, 64, out=torch.zeros(8, 64))


@pytest.mark.gpu
def test_reasons_for_new_outputs_and_missing_tensors(dev):
    """The reason functions take what the calls take: an output left to the call,
    a tensor that is missing."""
    q, k, v, pos, slots, cs, cache = append_inputs(5, 2, 3, 64, 64, BF, 3)
    assert qf.rope_kv_append_unsupported(q, k, v, pos, slots, cs, cache) is None
    assert qf.rope_kv_append_unsupported(None, k, v, pos, slots, cs, cache) is None
    assert "slots" in qf.rope_kv_append_unsupported(q, k, v, pos, slots[:4], cs, cache)
    assert "positions" in qf.rope_kv_append_unsupported(q, k, v, None, slots, cs, cache)
    assert "q" in qf.rope_kv_append_unsupported(q.cpu(), k, v, pos, slots, cs, cache)
    out, pages = torch.empty_like(q), torch.zeros(2, dtype=torch.int32, device=dev)
    lens = torch.zeros(5, dtype=torch.int32, device=dev)
    ws = torch.empty(qf.prefix_attn_workspace_bytes(5, 1, 6, 2, 64, 2, 0), dtype=torch.uint8, device=dev)
    assert qf.prefix_attn_unsupported(q, cache, pages, lens[:1], None, lens, ws, out) is None
    for change, name in ((dict(prefix_len=None), "prefix_len"), (dict(context_lens=None), "context_lens"),
                         (dict(workspace=None), "workspace"), (dict(out=None), "out")):
        a = dict(dict(prefix_len=lens[:1], context_lens=lens, workspace=ws, out=out), **change)
        assert name in qf.prefix_attn_unsupported(q, cache, pages, a["prefix_len"], None, a["context_lens"],
                                                  a["workspace"], a["out"])
    with pytest.raises(ValueError, match="prefix_len"):
        qf.prefix_attn(q, cache, pages, None, None, lens, ws)


def test_zero_skipped_flag(lib):
    """The flag goes with every type an operator takes, and makes no other type of one."""
    z = qf.DTYPE_ZERO_SKIPPED
    for call, types in ((rope_call, (0, 1, 2)), (append_call, (0, 1))):
        for dt in range(-1, 6):
            for flag in (z, 2 * z, 3 * z):
                code = call(lib, dt=dt + flag, T=0)
                assert code == (0 if dt in types and flag == z else 10), (dt, flag, code)


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        qf.rope(x, torch.zeros(4, dtype=torch.int64), torch.zeros(8, 64), out=x)
    with pytest.raises(ValueError, match="CUDA"):
        qf.rope_kv_append(None, x, x, torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64),
                          torch.zeros(8, 64), torch.zeros(1, 2, 16, 128, dtype=BF))
    with pytest.raises(ValueError, match="scaling"):
        qf.rope_table(8, 64, scaling="stretch")
    with pytest.raises(ValueError):
        qf.rope_table(8, 1 << 33)


# ---- values ------------------------------------------------------------------

def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, slow=1.0, fast=32.0):
    f = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        v = b ** (-2.0 * i / rot)
        if scaling == "linear":
            v /= factor
        if scaling == "ramp":
            g = min(1.0, max(0.0, (original * v / (2 * math.pi) - slow) / (fast - slow)))
            v = (1 - g) * v / factor + g * v
        f.append(v)
    return torch.tensor(f, dtype=torch.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,rot,first,kw", [
    (1, 2, 0, {}), (7, 64, 0, {}), (300, 64, 0, {}), (1000, 128, (1 << 20) - 5, {}),
    (513, 48, 77, dict(scaling="linear", factor=4.0)),
    (257, 96, 4000, dict(scaling="base", factor=8.0, base=500000.0)),
    (129, 128, 131000, dict(scaling="ramp", factor=16.0, original_len=8192)),
    (65, 512, 3, dict(scaling="ramp", factor=2.0, original_len=100, slow=0.0, fast=4.0, magnitude=0.5)),
    (2, 30, 0, {}), (70000, 6, 12345, {}),
])
def test_rope_table(dev, rows, rot, first, kw):
    got = qf.rope_table(rows, rot, first_position=first, device=dev, **kw).cpu().double()
    named = dict(kw)
    mag = named.pop("magnitude", 0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "ramp" else 1.0)
    named["original"] = named.pop("original_len", 0)
    ang = (first + torch.arange(rows, dtype=torch.float64))[:, None] * frequencies(rot, **named)
    ref = torch.cat([ang.cos(), ang.sin()], 1) * mag
    # the angle in half turns is rounded to fp32 (2^-24 of up to pi radians),
    # sincospif is good to 1 ulp (2^-23 at most), one product and mag round
    # (2^-24 each), the 64-bit angle itself is good to 1e-9 here
    tol = mag * (math.pi * 2.0 ** -24 + 2.0 ** -23 + 2 * 2.0 ** -24 + 1e-9)
    assert (got - ref).abs().max() <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, (1 << 24) + 3, (1 << 31) - 1, (1 << 36) + 77, 1 << 40])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0)])
def test_rope_table_at_far_positions(dev, first, scaling, factor):
    """Against angles to 60 digits.  The fixed-point product loses nothing, so
    what a position multiplies is the error of the frequency as a double: a
    power (1 ulp, 2^-52), one or two divisions and the constant of a turn
    (2^-53 each), and the 64-bit rate's 2^-64 turns."""
    rows, rot, base = 3, 32, 10000.0
    got = qf.rope_table(rows, rot, base=base, scaling=scaling, factor=factor, first_position=first, device=dev).cpu().double()
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        turn = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        for i in range(rot // 2):
            f = (decimal.Decimal(base).ln() * decimal.Decimal(-2 * i) / rot).exp() / decimal.Decimal(factor)
            for r in range(rows):
                p = first + r
                angle = 2 * math.pi * float((p * f / turn) % 1)
                tol = math.pi * 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -24 + p * float(f) * 2.0 ** -50 + 2 * math.pi * p * 2.0 ** -64
                assert abs(float(got[r, i]) - math.cos(angle)) <= tol and \
                    abs(float(got[r, rot // 2 + i]) - math.sin(angle)) <= tol, (p, i)


@pytest.mark.gpu
def test_rope_table_out_and_zero_rows(dev):
    out = torch.full((4, 64), 7.0, device=dev)
    assert qf.rope_table(4, 64, out=out) is out
    assert torch.equal(out[0], torch.cat([torch.ones(32), torch.zeros(32)]).to(dev))
    assert qf.rope_table(0, 64, device=dev).shape == (0, 64)
    with pytest.raises(ValueError):
        qf.rope_table(5, 64, out=out)


def turned(x, row, layout, back):
    """The rotation of x [T, H, D] in 64 bits, and the bound on what FP32
    products and sums may lose of it: 2^-23 (|a| + |b|) for table entries up
    to 1 (a product and a fused sum, each off by 2^-24 of a term)."""
    x, row = x.double(), row.double()
    half = row.shape[1] // 2
    c, s = row[:, None, :half], row[:, None, half:] * (-1 if back else 1)
    y, slack = x.clone(), torch.zeros_like(x)
    a = slice(0, 2 * half, 2) if layout == "interleaved" else slice(0, half)
    b = slice(1, 2 * half, 2) if layout == "interleaved" else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    slack[..., a] = slack[..., b] = 2.0 ** -23 * (x[..., a].abs() + x[..., b].abs())
    return y, slack


def close(got, ref, slack, dtype):
    """Within the FP32 bound and one rounding to dtype: half a step, 2^-25 at
    least for fp16's subnormals."""
    least = 2.0 ** -25 if dtype == HF else 0.0
    tol = slack + torch.finfo(dtype).eps / 2 * (ref.abs() + slack) + least
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {(got.double() - ref).abs().max():.3g}"


def inputs(T, H, D, rot, dtype, rows=509, seed=0, dev="cuda:0"):
    g = torch.Generator().manual_seed(1000 * T + H + seed)
    x = torch.randn(T, H, D, generator=g).to(dtype).to(dev)
    pos = torch.randint(0, rows, (T,), generator=g).to(dev)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * frequencies(rot)
    return x, pos, torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)


SHAPES = [  # T, heads, head_dim, rot_dim
    (1, 1, 2, 2), (1, 1, 64, 64), (3, 72, 64, 64), (5, 9, 80, 32), (2, 4, 128, 64), (7, 3, 96, 96),
    (4, 5, 7, 6), (3, 2, 33, 20), (6, 5, 128, 82), (2, 3, 256, 256), (3, 1, 512, 510), (130, 2, 64, 48),
    (1000, 3, 128, 128), (33, 40, 72, 24), (4, 4096, 4, 2), (2500, 1, 16, 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope_values(dev, shape, layout, dtype):
    x, pos, cs = inputs(*shape, dtype)
    for back, f in ((False, qf.rope), (True, qf.rope_backward)):
        out = f(x, pos, cs, layout=layout)
        ref, slack = turned(x, cs[pos], layout, back)
        close(out, ref, slack, dtype)
        assert torch.equal(out[..., shape[3]:], x[..., shape[3]:])
        kept = x.clone()
        assert f(kept, pos, cs, out=kept, layout=layout) is kept      # in place: the same bits
        assert torch.equal(kept, out)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rope_backward_is_the_gradient(dev, layout):
    """Against central differences of the 64-bit formula: with a linear map
    they are exact up to rounding, so the bound is the kernel's own."""
    x, pos, cs = inputs(3, 2, 12, 8, FL)
    gout = torch.randn(3, 2, 12, generator=torch.Generator().manual_seed(5)).to(dev)
    grad = qf.rope_backward(gout, pos, cs, layout=layout)
    base = x.double()
    diff = torch.zeros_like(base)
    for k in range(base.numel()):
        e = torch.zeros(base.numel(), dtype=torch.float64, device=dev)
        e[k] = 0.5
        up, _ = turned(base + e.view_as(base), cs[pos], layout, False)
        lo, _ = turned(base - e.view_as(base), cs[pos], layout, False)
        diff.view(-1)[k] = ((up - lo) * gout.double()).sum()
    _, slack = turned(gout, cs[pos], layout, True)
    close(grad, diff, slack + 1e-12, FL)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FL])
def test_rope_in_an_autograd_graph(dev, layout, dtype):
    """The result belongs to x's graph: its gradient is rope_backward's, through
    views, expanded gradients, a broadcast x and a graph of the gradient."""
    x, pos, cs = inputs(6, 3, 40, 24, dtype)
    g = torch.randn(6, 3, 40, generator=torch.Generator().manual_seed(6)).to(dtype).to(dev)
    leaf = x.clone().requires_grad_()
    y = qf.rope(leaf, pos, cs, layout=layout)
    assert y.requires_grad and torch.equal(y, qf.rope(x, pos, cs, layout=layout))
    y.backward(g)
    assert torch.equal(leaf.grad, qf.rope_backward(g, pos, cs, layout=layout))
    leaf.grad = None
    qf.rope(leaf, pos, cs, layout=layout).sum().backward()            # a gradient with strides of 0
    assert torch.equal(leaf.grad, qf.rope_backward(torch.ones_like(x), pos, cs, layout=layout))
    leaf.grad = None
    qf.rope(leaf, pos, cs, layout=layout).backward(g.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(leaf.grad, qf.rope_backward(g, pos, cs, layout=layout))
    packed = torch.randn(6, 5 * 40, generator=torch.Generator().manual_seed(7)).to(dtype).to(dev).requires_grad_()
    qf.rope(packed[:, 40:160].view(6, 3, 40), pos, cs, layout=layout).backward(g)
    assert torch.equal(packed.grad[:, 40:160].reshape(6, 3, 40), qf.rope_backward(g, pos, cs, layout=layout))
    assert torch.all(packed.grad[:, :40] == 0) and torch.all(packed.grad[:, 160:] == 0)
    one = x[:, :1].detach().clone().requires_grad_()
    qf.rope(one.expand(6, 3, 40), pos, cs, layout=layout).backward(g)   # one head shared by three
    ref, slack = turned(g, cs[pos], layout, True)
    # three gradients, each within its bound of the formula, and two sums of them
    tol = (slack + torch.finfo(dtype).eps / 2 * (ref.abs() + slack)).sum(1) + torch.finfo(dtype).eps * 1.01 * ref.abs().sum(1)
    assert ((one.grad[:, 0].double() - ref.sum(1)).abs() <= tol).all()
    pos[2] = -1                                                       # a skipped token takes no part
    leaf.grad = None
    qf.rope(leaf, pos, cs, layout=layout).backward(g)
    assert torch.all(leaf.grad[2] == 0) and torch.equal(leaf.grad[3], qf.rope_backward(g[3:4], pos[3:4], cs, layout=layout)[0])
    assert qf.status() == qf.STATUS_BAD_POSITION
    pos[2] = 5
    if dtype == FL:
        w = torch.randn_like(x, requires_grad=True)
        y = qf.rope(leaf, pos, cs, layout=layout)
        grad, = torch.autograd.grad(y, leaf, w, create_graph=True)
        grad.backward(g)                                              # linear in w: turned forth again
        assert torch.equal(w.grad, qf.rope(g, pos, cs, layout=layout))
    table = cs.clone()
    y = qf.rope(leaf, pos, table, layout=layout)
    qf.rope_table(cs.shape[0], cs.shape[1], first_position=9, out=table)   # the graph's table is gone
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    leaf.grad = None
    y = qf.rope(leaf, pos, cs, layout=layout, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.backward(g)
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad, qf.rope_backward(g, pos, cs, layout=layout))


@pytest.mark.gpu
def test_rope_refuses_a_lost_gradient(dev):
    """Where the result cannot belong to the graph, no gradient is lost in
    silence; without gradients asked for, the same calls run."""
    x, pos, cs = inputs(4, 2, 64, 64, BF)
    leaf = x.clone().requires_grad_()
    out = torch.empty_like(x)
    for f in (qf.rope, qf.rope_backward):
        with pytest.raises(ValueError, match="no_grad"):
            f(leaf, pos, cs, out=out)
        with pytest.raises(ValueError, match="cos_sin"):
            f(x, pos, cs.clone().requires_grad_())
        with torch.no_grad():
            ref = f(x, pos, cs)
            assert f(leaf, pos, cs, out=out) is out and torch.equal(out, ref)
            assert not f(leaf, pos, cs).requires_grad
    keep = qf.rope(leaf, pos, cs)                                      # a graph of the leaf that lives on
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            qf.rope(leaf, pos, cs)
        with torch.no_grad():
            y = qf.rope(leaf, pos, cs)
            dx = qf.rope_backward(y, pos, cs)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, keep) and torch.equal(dx, qf.rope_backward(keep.detach(), pos, cs))
    keep.backward(x)
    assert torch.equal(leaf.grad, qf.rope_backward(x, pos, cs)) and qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FL])
def test_rope_strided_views(dev, layout, dtype):
    """q and k columns of packed rows in place, a transposed [heads, tokens]
    buffer, a misaligned start, a broadcast input."""
    T, H, D, rot = 37, 6, 64, 48
    row, pos, cs = inputs(T, 1, 10 * D + 3, rot, dtype)
    row = row.view(T, -1)
    before = row.clone()
    q = row[:, D:D + H * D].view(T, H, D)
    ref, slack = turned(q.clone(), cs[pos], layout, False)
    qf.rope(q, pos, cs, out=q, layout=layout)
    close(q, ref, slack, dtype)
    assert torch.equal(row[:, :D], before[:, :D]) and torch.equal(row[:, D + H * D:], before[:, D + H * D:])

    x = before[:, 3:3 + H * D].view(T, H, D)            # rows start off the 16-byte grid
    out = torch.full((H, T, D + 1), 9.0, dtype=dtype, device=dev)
    qf.rope(x, pos, cs, out=out[:, :, :D].transpose(0, 1), layout=layout)
    ref, slack = turned(x, cs[pos], layout, False)
    close(out[:, :, :D].transpose(0, 1), ref, slack, dtype)
    assert torch.all(out[:, :, D] == 9.0)

    one = before[:1, :D].view(1, 1, D).expand(T, H, D)
    ref, slack = turned(one, cs[pos], layout, False)
    close(qf.rope(one, pos, cs, layout=layout), ref, slack, dtype)
    with pytest.raises(qf.QkvFrontError):
        qf.rope(x, pos, cs, out=one, layout=layout)     # an output with one address twice
    with pytest.raises(ValueError, match="contiguous"):
        qf.rope(before[:, :H * D].view(T, H, D)[..., ::2], pos, cs)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rope_special_values_stay_in_their_pairs(dev, layout):
    """Infinities and NaN reach their own pair only; columns behind rot_dim
    are copied bit for bit."""
    x, pos, cs = inputs(5, 3, 64, 40, BF)
    pos[:] = torch.arange(5, device=dev)
    clean = qf.rope(x, pos, cs, layout=layout)
    x[1, 0, 7], x[2, 1, 8], x[3, 2, 60] = math.inf, math.nan, math.nan
    out = qf.rope(x, pos, cs, layout=layout)
    touched = torch.zeros_like(x, dtype=torch.bool)
    other = {7: 6, 8: 9} if layout == "interleaved" else {7: 27, 8: 28}
    touched[1, 0, [7, other[7]]] = touched[2, 1, [8, other[8]]] = True
    touched[3, 2, 60] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert not torch.isfinite(out[touched].float()).any()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D,rot,dtype,layout", [
    (1 << 24, 1, 8, 8, BF, "half"), (1 << 24, 1, 6, 2, HF, "interleaved"), (1 << 24, 3, 16, 10, BF, "half"),
    (1 << 24, 1, 512, 16, FL, "half"), (4099, 4096, 128, 128, BF, "interleaved"),
], ids=str)
def test_rope_largest_calls(dev, T, H, D, rot, dtype, layout):
    """As many tokens and heads as a call takes, up to more than 2^30 threads
    and offsets past 2^32 bytes: the first, the last and some rows in between,
    in place."""
    g = torch.Generator().manual_seed(T + H)
    ang = torch.arange(97, dtype=torch.float64)[:, None] * frequencies(rot)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)
    pattern = torch.randn(101, H, D, generator=g).to(dtype).to(dev)         # token t holds row t % 101
    x = torch.empty(T, H, D, dtype=dtype, device=dev)
    whole = T // 101 * 101
    x[:whole].view(-1, 101, H, D).copy_(pattern.expand(whole // 101, 101, H, D))
    x[whole:] = pattern[:T - whole]
    pos = torch.arange(T, device=dev) % 97
    qf.rope(x, pos, cs, out=x, layout=layout)
    assert qf.status() == 0
    some = torch.cat([torch.arange(200), torch.randint(0, T, (2000,), generator=g), torch.arange(T - 200, T)]).unique().to(dev)
    for t in some.split(64):
        close(x[t], *turned(pattern[t % 101], cs[pos[t]], layout, False), dtype)


@pytest.mark.gpu
def test_rope_bad_positions_and_zero_tokens(dev):
    x, pos, cs = inputs(6, 2, 64, 64, BF)
    good = qf.rope(x, pos, cs)
    pos[1], pos[4] = -1, cs.shape[0]
    out = torch.full_like(x, 3.0)
    qf.rope(x, pos, cs, out=out)
    assert qf.status() == qf.STATUS_BAD_POSITION and qf.status() == 0
    keep = torch.tensor([0, 2, 3, 5], device=dev)
    assert torch.equal(out[keep], good[keep]) and torch.all(out[[1, 4]] == 3.0)
    assert qf.rope(x[:0], pos[:0], cs).shape == (0, 2, 64)
    assert qf.rope_unsupported(x, pos, cs, out) is None
    assert "overlap" in qf.rope_unsupported(x[1:], pos[1:], cs, x[:-1])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("shape", [(40, 9, 64, 64), (40, 2, 96, 96), (33, 17, 128, 82), (20, 5, 33, 20), (70, 1, 256, 250)], ids=str)
def test_skipped_tokens_of_a_new_output_are_zero(dev, shape, dtype, layout):
    """An output that the call makes holds nothing before: where memory is used
    again, a token with a bad position must not show what lay there."""
    x, pos, cs = inputs(*shape, dtype)
    good = qf.rope(x, pos, cs, layout=layout), qf.rope_backward(x, pos, cs, layout=layout)
    pos[3], pos[7], pos[-1] = -1, cs.shape[0], 1 << 40
    keep = torch.ones(shape[0], dtype=torch.bool, device=dev)
    keep[[3, 7, -1]] = False
    for f, ref in zip((qf.rope, qf.rope_backward), good):
        torch.full_like(x, 3.0)                                    # its memory is the next output's
        out = f(x, pos, cs, layout=layout)
        assert torch.equal(out[keep], ref[keep]) and torch.all(out[~keep] == 0)
        assert qf.status() == qf.STATUS_BAD_POSITION
    if dtype == BF and shape[2] % 8 == 0:
        nkv, D = 1, shape[2]
        cache = torch.zeros(8, nkv, 16, 2 * D, dtype=dtype, device=dev)
        slots = torch.arange(shape[0], device=dev)
        torch.full_like(x, 3.0)
        out = qf.rope_kv_append(x, x[:, :1], x[:, :1], pos, slots, cs, cache, layout=layout)
        assert torch.equal(out[keep], good[0][keep]) and torch.all(out[~keep] == 0)
        rows = cache.permute(0, 2, 1, 3).reshape(128, 2 * D)
        assert torch.all(rows[:shape[0]][~keep] == 0) and torch.equal(rows[:shape[0], D:][keep], x[keep, 0])
        assert qf.status() == qf.STATUS_BAD_POSITION


def append_inputs(T, nkv, G, D, rot, dtype, pages, seed=0):
    x, pos, cs = inputs(T, nkv * (G + 2), D, rot, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + T)
    slots = torch.randperm(pages * 16, generator=g)[:T].to("cuda:0")
    cache = torch.randn(pages, nkv, 16, 2 * D, generator=g).to(dtype).to("cuda:0")
    h = nkv * G
    return x[:, :h], x[:, h:h + nkv], x[:, h + nkv:], pos, slots, cs, cache


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,nkv,G,D,rot", [
    (1, 1, 1, 8, 2), (1, 1, 8, 64, 64), (8, 8, 8, 64, 64), (37, 2, 5, 128, 64), (16, 3, 1, 96, 82),
    (5, 4, 0, 64, 64), (300, 1, 7, 80, 32), (1031, 2, 4, 128, 128), (3, 40, 2, 256, 250), (2, 1, 3, 512, 512),
])
def test_rope_kv_append(dev, T, nkv, G, D, rot, layout, dtype):
    pages = (T + 15) // 16 + 3
    q, k, v, pos, slots, cs, cache = append_inputs(T, nkv, G, D, rot, dtype, pages)
    before = cache.clone()
    out = qf.rope_kv_append(q if G else None, k, v, pos, slots, cs, cache, layout=layout)
    assert qf.status() == 0
    if G:
        assert torch.equal(out, qf.rope(q, pos, cs, layout=layout))
        close(out, *turned(q, cs[pos], layout, False), dtype)
    else:
        assert out is None
    rows = cache[slots // 16, :, slots % 16]                       # [T, nkv, 2 D]
    close(rows[..., :D], *turned(k, cs[pos], layout, False), dtype)
    assert torch.equal(rows[..., :D], qf.rope(k, pos, cs, layout=layout))
    assert torch.equal(rows[..., D:], v)
    cache[slots // 16, :, slots % 16] = before[slots // 16, :, slots % 16]
    assert torch.equal(cache, before)                              # nothing else was written


@pytest.mark.gpu
def test_rope_kv_append_index_rules_and_in_place(dev):
    """Padding tokens, a slot past the cache, bad positions; q in place in the
    packed rows it came in, whose other columns stay."""
    T, nkv, G, D = 40, 2, 3, 64
    q, k, v, pos, slots, cs, _ = append_inputs(T, nkv, G, D, D, BF, 8)
    packed = torch.cat([q, k, v], 1).reshape(T, -1).contiguous()
    parent = torch.zeros(16, nkv, 16, 2 * D, dtype=BF, device=dev)
    cache = parent[:8]
    good = qf.rope_kv_append(q, k, v, pos, slots, cs, cache.clone())
    slots[3], slots[7], pos[11], pos[12] = -1, 8 * 16, -5, cs.shape[0]
    view = packed[:, :G * nkv * D].view(T, G * nkv, D)
    kk = packed[:, G * nkv * D:(G + 1) * nkv * D].view(T, nkv, D)
    vv = packed[:, (G + 1) * nkv * D:].view(T, nkv, D)
    assert qf.rope_kv_append(view, kk, vv, pos, slots, cs, cache, q_out=view) is view
    assert qf.status() == qf.STATUS_BAD_SLOT | qf.STATUS_BAD_POSITION
    keep = torch.ones(T, dtype=torch.bool, device=dev)
    keep[[11, 12]] = False
    assert torch.equal(view[keep], good[keep]) and torch.equal(view[~keep], q[~keep])
    assert torch.equal(kk, k) and torch.equal(vv, v)
    assert torch.all(parent[8:] == 0)
    keep[[3, 7]] = False
    used = torch.zeros(8 * 16, dtype=torch.bool, device=dev)
    used[slots[keep]] = True
    rows = cache.permute(0, 2, 1, 3).reshape(8 * 16, -1)
    assert torch.all(rows[~used] == 0) and torch.equal(rows[slots[keep]].view(-1, nkv, 2 * D)[..., D:], v[keep])


@pytest.mark.gpu
def test_rope_kv_append_far_slot(dev):
    """A slot whose element offset passes 2^32."""
    nkv, D = 8, 128
    pages = (1 << 32) // (nkv * 16 * 2 * D) + 8
    cache = torch.empty(pages, nkv, 16, 2 * D, dtype=BF, device=dev)
    cache[-1].zero_()
    cache[0].zero_()
    q, k, v, pos, _, cs, _ = append_inputs(2, nkv, 1, D, D, BF, 1)
    slots = torch.tensor([pages * 16 - 3, 5], device=dev)
    qf.rope_kv_append(None, k, v, pos, slots, cs, cache)
    assert qf.status() == 0
    assert torch.equal(cache[-1, :, 13, D:], v[0]) and torch.equal(cache[0, :, 5, D:], v[1])
    assert torch.equal(cache[-1, :, 13, :D], qf.rope(k, pos, cs)[0])
    assert torch.all(cache[-1, :, :13] == 0) and torch.all(cache[0, :, 6:] == 0)


@pytest.mark.gpu
def test_streams_and_graphs(dev):
    """Calls on a side stream and captured calls give the direct call's bits,
    replays follow the inputs' new contents."""
    T, nkv, G, D = 50, 2, 4, 64
    q, k, v, pos, slots, cs, cache = append_inputs(T, nkv, G, D, 32, HF, 6)
    table = qf.rope_table(cs.shape[0], 32, device=dev)
    ref = qf.rope_kv_append(q, k, v, pos, slots, table, cache, layout="half")
    ref_cache = cache.clone()
    cache.zero_()
    cache[:] = ref_cache
    cache[slots // 16, :, slots % 16] = 0
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    t2 = qf.rope_table(cs.shape[0], 32, device=dev, stream=s)
    out = qf.rope_kv_append(q, k, v, pos, slots, t2, cache, layout="half", stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(cache, ref_cache)
    g = torch.cuda.CUDAGraph()
    qq, q_out = q.clone(), torch.zeros_like(ref)
    with torch.cuda.graph(g):
        qf.rope_table(cs.shape[0], 32, out=t2)
        qf.rope_kv_append(qq, k, v, pos, slots, t2, cache, q_out=q_out, layout="half")
        back = qf.rope_backward(q_out, pos, t2, layout="half")
    cache.zero_()
    qq.copy_(q.flip(0))
    t2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, qf.rope(q.flip(0), pos, table, layout="half"))
    assert torch.equal(back, qf.rope_backward(q_out, pos, table, layout="half"))
    assert torch.equal(cache[slots // 16, :, slots % 16], ref_cache[slots // 16, :, slots % 16])
    assert qf.status() == 0
