"""chunk_attn and key_weights: refusals on the host (no GPU needed), values
against a plain 64-bit softmax at the lengths, head layouts and contents where
they can go wrong, and the serving chain around them.

Tolerances: a score is a sum of D products in FP32, off by at most D 2^-24 of
the sum of their magnitudes (es); a weight exp(s - m) by 2 es and 2^-21, and it
is rounded to the type (half a step); the output is rounded once more.  The sums
over L keys add blocks of at most 64 or 128 values, one after another: at most
64 + L / 64 additions follow one another, 2^-24 each."""
import math
import random

import pytest
import torch

from kv_insert_gb300 import _build
from kv_insert_gb300 import qkv_front as qf

BF, HF = torch.bfloat16, torch.float16
PAGE = 16

Q, C, ST, BT, CL, O, LSE, WS, WT, OW = ((i + 1) << 42 for i in range(10))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qf.load()


@pytest.fixture(scope="module")
def dev(lib):
    qf.status()
    return torch.device("cuda:0")


# ---- host refusals -----------------------------------------------------------

def chunk_call(lib, **kw):
    a = dict(q=Q, qt=512, qh=64, c=C, pages=64, st=ST, bt=BT, mb=4, cl=CL, T=9, R=3, H=8, nkv=2, D=64, sc=0.125, dt=0,
             o=O, lse=LSE, ws=WS, n=1 << 40)
    a.update(kw)
    code = lib.chunk_attn(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.chunk_attn_unsupported(*a.values())) > 5
    return code


def weights_call(lib, **kw):
    a = dict(q=Q, qt=512, qh=64, c=C, pages=64, lse=LSE, st=ST, bt=BT, mb=4, cl=CL, T=9, R=3, H=8, nkv=2, D=64, win=0,
             dec=1.0, sc=0.125, dt=0, w=WT, o=OW, ws=WS, n=1 << 40)
    a.update(kw)
    code = lib.key_weights(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.key_weights_unsupported(*a.values())) > 5
    return code


@pytest.mark.parametrize("call", [chunk_call, weights_call])
def test_shared_refusals(lib, call):
    assert call(lib, R=-1) == 1 and call(lib, R=65536) == 1 and call(lib, T=-1) == 1 and call(lib, T=(1 << 24) + 1) == 1
    for kw in (dict(D=32), dict(D=96), dict(nkv=0), dict(nkv=65, H=65), dict(H=0), dict(H=9), dict(H=130),
               dict(dt=2), dict(qt=-8), dict(qt=516), dict(qh=60)):
        assert call(lib, **kw) == 10, kw
    assert call(lib, mb=0) == 7 and call(lib, mb=(1 << 20) + 1) == 7 and call(lib, pages=0) == 7
    assert call(lib, pages=1 << 31) == 7 and call(lib, T=1 << 24, H=128) == 7
    for sc in (0.0, -1.0, math.nan, math.inf):
        assert call(lib, sc=sc) == 9
    for name in ("q", "c", "st", "bt", "cl", "o", "ws"):
        assert call(lib, **{name: 0}) == 3, name
    assert call(lib, q=Q + 8) == 4 and call(lib, bt=BT + 2) == 4 and call(lib, ws=WS + 128) == 4 and call(lib, lse=LSE + 2) == 4
    assert call(lib, o=Q) == 9 and call(lib, o=C + 4096) == 9 and call(lib, ws=Q) == 9 and call(lib, ws=BT) == 9
    assert call(lib, o=CL) == 9 and call(lib, o=ST) == 9 and call(lib, o=LSE) == 9
    if not torch.cuda.is_available():
        assert call(lib) in (5, 6)


def test_own_refusals(lib):
    assert chunk_call(lib, o=O + 8) == 4 and chunk_call(lib, R=0, T=0, q=0) == 0 and chunk_call(lib, T=0, q=0, o=0) == 0
    assert weights_call(lib, win=-1) == 9 and weights_call(lib, R=0) == 0
    for dec in (-0.5, 1.5, math.nan):
        assert weights_call(lib, dec=dec) == 9
    assert weights_call(lib, w=0) == 3 and weights_call(lib, lse=0) == 3 and weights_call(lib, w=OW + 64) == 9
    assert weights_call(lib, w=WS) == 9
    assert weights_call(lib, qt=0) == 10 and weights_call(lib, qh=0) == 10   # (a copy's strides are above 0)
    if not torch.cuda.is_available():
        assert chunk_call(lib, lse=0) in (5, 6)
        assert weights_call(lib, w=OW) in (5, 6) and weights_call(lib, w=0, dec=0.0) in (5, 6)


# ---- inputs and the formula --------------------------------------------------

class Batch:
    """Requests of (new tokens, keys); every slot that no key uses holds NaN."""

    def __init__(self, lens, nkv, group, D, dtype, seed=0, scale=None, spread=1.0, extra=0, mb=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nkv, self.group, self.D, self.dtype = lens, nkv, group, D, dtype
        self.scale = D ** -0.5 if scale is None else scale
        T, R = sum(max(n, 0) for n, _ in lens) + extra, len(lens)
        self.q = (spread * torch.randn(T, nkv * group, D, generator=g, device="cuda")).to(dtype)
        counts = [-(-max(L, 0) // PAGE) for _, L in lens]
        self.mb = max([1] + counts) if mb is None else mb
        pages = torch.randperm(sum(counts) + 3, generator=g, device="cuda")[:sum(counts)].to(torch.int32)
        self.cache = torch.full((sum(counts) + 3, nkv, PAGE, 2 * D), math.nan, dtype=dtype, device="cuda")
        self.table = torch.full((R, self.mb), -7, dtype=torch.int32, device="cuda")
        at = 0
        for r, ((_, L), n) in enumerate(zip(lens, counts)):
            self.table[r, :n] = pages[at:at + n]
            at += n
            j = torch.arange(max(L, 0), device="cuda")
            kv = torch.randn(len(j), nkv, 2 * D, generator=g, device="cuda").to(dtype)
            self.cache[self.table[r].long()[j // PAGE], :, j % PAGE] = kv
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.context = torch.tensor([L for _, L in lens], dtype=torch.int32, device="cuda")
        self.lse = torch.full((T, nkv * group), 3.0, device="cuda")
        self.ws = torch.full((self.bytes(qf.chunk_attn_workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
        self.wws = torch.full((self.bytes(qf.key_weights_workspace_bytes),), 255, dtype=torch.uint8, device="cuda")

    def bytes(self, f):
        T, H, D = self.q.shape
        return f(T, len(self.lens), H, self.nkv, D, self.mb)

    def attn(self, **kw):
        return qf.chunk_attn(self.q, self.cache, self.starts, self.table, self.context, self.ws, scale=self.scale, **kw)

    def weights(self, w, **kw):
        return qf.key_weights(self.q, self.cache, self.lse, self.starts, self.table, self.context, w, self.wws,
                              scale=self.scale, **kw)

    def keys(self, r):
        L = max(self.lens[r][1], 0)
        j = torch.arange(L, device="cuda")
        kv = self.cache[self.table[r].long()[j // PAGE], :, j % PAGE].double()   # [L, nkv, 2 D]
        return kv.permute(1, 0, 2)

    def rows(self, r):
        return slice(int(self.starts[r]), int(self.starts[r + 1]))

    def scores(self, r):
        """Scores [nkv, group, n, L] with -infinity for unseen keys, and how far FP32 may be off them."""
        n, L = self.lens[r]
        k = self.keys(r)[..., :self.D]
        q = self.q[self.rows(r)].double().view(n, self.nkv, self.group, self.D).permute(1, 2, 0, 3)
        s = torch.einsum("ghnd,gld->ghnl", q, k) * self.scale
        es = torch.einsum("ghnd,gld->ghnl", q.abs(), k.abs()) * self.scale * self.D * 2.0 ** -24
        seen = torch.arange(L, device="cuda") <= torch.arange(L - n, L, device="cuda")[:, None]
        return s.masked_fill(~seen, -math.inf), es.masked_fill(~seen, 0.0)

    def check_attn(self, out, lse, only=None):
        half = torch.finfo(self.dtype).eps / 2
        for r, (n, L) in enumerate(self.lens):
            if n <= 0 or L < 0 or (only is not None and r not in only):
                continue
            s, es = self.scores(r)
            v = self.keys(r)[..., self.D:]
            z = torch.logsumexp(s, -1, keepdim=True) if L else s.new_full((*s.shape[:3], 1), -math.inf)
            w = torch.where(z == -math.inf, 0.0, torch.exp(s - torch.where(z == -math.inf, 0.0, z)))
            # (a V that is not finite counts where it is seen only)
            ref, mag = torch.einsum("ghnl,gld->ghnd", w, v), torch.einsum("ghnl,gld->ghnd", w, v.abs())
            err = es.amax(-1, keepdim=True) if L else s.new_zeros(*s.shape[:3], 1)

            def flat(t):
                return t.permute(2, 0, 1, 3).reshape(n, self.nkv * self.group, -1)
            got, ref, mag, err, z = out[self.rows(r)].double(), flat(ref), flat(mag), flat(err), flat(z)[..., 0]
            sums = (64 + L / 64) * 2.0 ** -24
            tol = half * ref.abs() + (half + 2 * err + 2.0 ** -20 + 2 * sums) * mag + 2.0 ** -24
            bad = (got - ref).abs() > tol
            assert got.isfinite().all() and not bad.any(), (r, n, L, int(bad.sum()), float(((got - ref).abs() / tol).max()))
            if lse is None:
                continue
            got = lse[self.rows(r)].double()
            dead = z == -math.inf
            assert (got[dead] == -math.inf).all()
            off = (got - z)[~dead].abs() - err[..., 0][~dead] - 2.0 ** -20 * (1 + z[~dead].abs()) - sums
            assert not (off > 0).any(), (r, n, L, float(off.max()))


HEADS = [(1, 1, 64), (2, 8, 64), (8, 4, 128), (3, 5, 128), (1, 7, 64), (2, 64, 64), (1, 33, 128)]
LENS = {
    "one": [(1, 1)], "decode": [(1, L) for L in (1, 2, 15, 16, 17, 127, 128, 129, 300)],
    "prefill": [(200, 200)], "chunk": [(129, 700)], "mixed": [(1, 300), (77, 77), (1, 1), (130, 515), (0, 40), (2, 33)],
    "empty": [(5, 3), (4, 0), (0, 0), (3, 3), (1, 0), (260, 100)], "edges": [(16, 16), (17, 129), (128, 256), (31, 128)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("nkv,group,D", HEADS)
@pytest.mark.parametrize("lens", LENS)
def test_values(dev, lens, nkv, group, D, dtype):
    b = Batch(LENS[lens], nkv, group, D, dtype, seed=len(lens))
    out = b.attn(lse=b.lse)
    assert qf.status() == 0
    b.check_attn(out, b.lse)
    lse = b.lse.clone()
    assert torch.equal(b.attn(out=torch.zeros_like(out), lse=b.lse), out) and torch.equal(b.lse, lse)   # bit for bit
    assert torch.equal(b.attn(), out)
    check_weights(b)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,nkv,group,D", [
    ([(2050, 2050)], 1, 4, 128), ([(1, 20000)], 2, 8, 64), ([(3, 9001), (1, 33), (700, 5000)], 2, 4, 128),
    ([(1, L) for L in range(1, 400, 3)], 1, 8, 64), ([(7, 3000 + r) for r in range(40)], 1, 3, 128),
    ([(1500, 1500), (1, 700), (90, 8000), (400, 401)], 1, 8, 64), ([(513, 513)] * 5, 2, 2, 64)])
def test_longer_values(dev, lens, nkv, group, D):
    b = Batch(lens, nkv, group, D, BF, seed=5)
    out = b.attn(lse=b.lse)
    assert qf.status() == 0
    b.check_attn(out, b.lse)
    check_weights(b, windows=(0, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_drawn_batches(dev, seed):
    rng = random.Random(seed)
    for _ in range(6):
        nkv, group, D = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128])
        lens = []
        for _ in range(rng.randint(1, 12)):
            n = rng.choice([0, 1, 1, 1, rng.randint(2, 300)])
            lens.append((n, max(0, n + rng.choice([0, 0, -1, rng.randint(0, 2000)]))))
        b = Batch(lens, nkv, group, D, rng.choice([BF, HF]), seed=seed, extra=rng.choice([0, 0, 5]))
        out = b.attn(lse=b.lse)
        assert qf.status() == 0
        b.check_attn(out, b.lse)
        check_weights(b, windows=(0, rng.randint(1, 50)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("spread,scale", [(8.0, None), (0.0, None), (30.0, 1.0), (1.0, 1e-4)])
def test_scores_of_other_sizes(dev, dtype, spread, scale):
    b = Batch([(40, 400), (1, 700)], 2, 4, 64, dtype, spread=spread, scale=scale)
    out = b.attn(lse=b.lse)
    b.check_attn(out, b.lse)


@pytest.mark.gpu
def test_growing_scores(dev):
    """Every block's scores exceed the last one's, and the reverse: the running maximum follows, or stays."""
    for sign in (1, -1):
        for D in (64, 128):
            b = Batch([(64, 1500), (1, 900)], 1, 4, D, BF)
            b.q[:] = 0
            b.q[..., 0] = 4.0
            for r, (_, L) in enumerate(b.lens):
                j = torch.arange(L, device="cuda")
                ramp = (j if sign > 0 else L - j).float() / 2
                b.cache[b.table[r].long()[j // PAGE], :, j % PAGE, 0] = ramp.to(BF)[:, None]
            b.check_attn(b.attn(lse=b.lse), b.lse)


@pytest.mark.gpu
def test_fp16_weights_far_below_a_dominant_one(dev):
    """One early key takes most of the weight, thousands behind it make the output: none of them is lost."""
    for D in (64, 128):
        b = Batch([(3, 6000)], 1, 4, D, HF)
        b.q[:] = 0
        b.q[..., 0] = 1.0
        j = torch.arange(6000, device="cuda")
        at = b.table[0].long()[j // PAGE], slice(None), j % PAGE
        b.cache[at[0], :, at[2], 0] = 0.0
        b.cache[at[0][0], :, 0, 0] = 15.0 * math.log(2.0) / b.scale
        b.cache[at[0][0], :, 0, D:] = 0.0
        b.cache[at[0][1:], :, at[2][1:], D:] = 1.0
        b.check_attn(b.attn(lse=b.lse), b.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("D,group", [(64, 8), (128, 4), (128, 1), (64, 64)])
def test_values_that_later_tokens_alone_see(dev, D, group):
    """Infinity and NaN in K or V of a new token reach its own and later rows, no earlier ones."""
    for n, L, cut in ((70, 70, 33), (70, 400, 35), (300, 333, 150), (2, 2, 1), (200, 200, 128)):
        for part, value in (("v", math.inf), ("v", math.nan), ("k", math.nan), ("k", math.inf), ("v", -math.inf)):
            b = Batch([(n, L), (1, 50)], 2, group, D, BF, seed=n)
            want = b.attn(lse=b.lse).clone()
            lse = b.lse.clone()
            j = L - n + cut
            col = slice(D, 2 * D) if part == "v" else slice(0, D)
            b.cache[int(b.table[0, j // PAGE]), :, j % PAGE, col] = value
            out = b.attn(lse=b.lse)
            keep = torch.arange(n + 1, device="cuda")
            keep = keep[(keep < cut) | (keep >= n)]
            assert torch.equal(out[keep], want[keep]) and torch.equal(b.lse[keep], lse[keep]), (n, L, part, value)
            after = out[cut:n]
            if part == "v":
                assert torch.equal(b.lse, lse)
                assert (after.isnan() if math.isnan(value) else after == value).all(), (n, L, part, value)
            elif math.isnan(value):
                assert after.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,group", [(64, 8), (128, 4), (128, 1), (64, 64)])
def test_infinite_keys(dev, D, group):
    """A column of K is infinite: the rows whose score it makes -infinity leave that key out, those whose score it
    makes infinite are NaN, and neither reaches a neighbour."""
    class Without(Batch):
        def scores(self, r):
            cache, self.cache = self.cache, self.clean
            s, es = super().scores(r)
            self.cache = cache
            if r == 0:
                s[..., self.key], es[..., self.key] = -math.inf, 0.0
            return s, es

    for n, L, key in ((70, 70, 33), (70, 400, 365), (300, 700, 20), (2, 2000, 1500), (1, 5000, 4999)):
        b = Without([(n, L), (1, 50)], 2, group, D, BF, seed=n)
        b.q[..., 0] = -b.q[..., 0].abs().clamp_min(0.25)
        clean = b.attn(lse=b.lse).clone()
        b.clean, b.key = b.cache.clone(), key
        b.cache[int(b.table[0, key // PAGE]), :, key % PAGE, 0] = math.inf
        none = b.attn(lse=b.lse).clone()
        b.check_attn(none, b.lse)
        lse = b.lse.clone()
        up = torch.rand(b.q.shape[:2], device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) < 0.5
        up[n:] = False
        b.q[..., 0] = torch.where(up, -b.q[..., 0], b.q[..., 0])
        out = b.attn(lse=b.lse)
        assert torch.equal(out[~up], none[~up]) and torch.equal(b.lse[~up], lse[~up])
        sees = L - n + torch.arange(n + 1, device="cuda") >= key
        sees[n:] = False
        assert out[up & sees[:, None]].isnan().all() and out[up & ~sees[:, None]].isfinite().all()
        assert torch.equal(out[n:], clean[n:])


@pytest.mark.gpu
def test_rows_of_no_request(dev):
    """Padding requests, rows behind the last and before the first: left alone, or zeros in a new output."""
    b = Batch([(5, 40), (3, 20), (6, 90)], 2, 4, 64, BF, extra=9)
    want = b.attn(lse=b.lse).clone()
    assert (want[14:] == 0).all() and (b.lse[14:] == 3).all()
    b.context[1] = -(1 << 31)
    out = torch.full_like(b.q, 7.0)
    b.lse.fill_(3.0)
    b.attn(out=out, lse=b.lse)
    assert torch.equal(out[:5], want[:5]) and torch.equal(out[8:14], want[8:14])
    assert (out[5:8] == 7).all() and (out[14:] == 7).all() and (b.lse[5:8] == 3).all() and (b.lse[14:] == 3).all()
    assert (b.attn()[5:8] == 0).all() and qf.status() == 0
    b.starts += 4
    out.fill_(7.0)
    b.attn(out=out)
    assert (out[:4] == 7).all() and (out[18:] == 7).all() and (out[9:12] == 7).all()
    w = torch.full((3, 2, b.mb * PAGE), 2.0, device="cuda")
    b.weights(w, decay=0.0)
    assert (w[1] == 2).all() and (w[0, :, 40:] == 2).all() and not (w[0, :, :40] == 2).any()
    assert qf.status() == 0
    none = Batch([], 2, 4, 64, BF, extra=3, mb=2)
    assert (none.attn() == 0).all()
    out = torch.full_like(none.q, 7.0)
    none.attn(out=out)
    assert (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,group", [(64, 8), (128, 3)])
def test_bad_requests(dev, D, group):
    """Lengths beyond the table, starts that decrease or leave the rows, pages outside the cache: flagged, that
    request alone skipped."""
    def batch():
        return Batch([(4, 300), (150, 400), (1, 200), (3, 50)], 2, group, D, BF)
    b = batch()
    want = b.attn(lse=b.lse).clone()
    w0 = b.weights(torch.zeros(4, 2, b.mb * PAGE, device="cuda"))
    assert qf.status() == 0

    def check(b, bad):
        out = torch.full_like(b.q, 7.0)
        lse = torch.full_like(b.lse, 3.0)
        b.attn(out=out, lse=lse)
        assert qf.status() == 8
        w = torch.full_like(w0, 2.0)
        b.weights(w, decay=0.0)
        assert qf.status() == 8
        for r in range(4):
            rows = b0.rows(r)
            if r in bad:
                assert (out[rows] == 7).all() and (lse[rows] == 3).all()
            else:
                assert torch.equal(out[rows], want[rows])
                L = b0.lens[r][1]
                assert torch.equal(w[r, :, :L], w0[r, :, :L]) and (w[r, :, L:] == 2).all()
    b0 = batch()
    for r, value in ((0, b.mb * PAGE + 1), (2, (1 << 31) - 1)):
        b = batch()
        b.lse.copy_(lse_of(b0))
        b.context[r] = value
        check(b, {r})
    for r, j, page in ((0, 0, -1), (1, 0, 1 << 30), (2, 200 // PAGE, len(b.cache)), (3, 2, -(1 << 31))):
        b = batch()
        b.lse.copy_(lse_of(b0))
        b.table[r, j] = page
        check(b, {r})
    b = batch()
    b.lse.copy_(lse_of(b0))
    b.starts[4] = b.q.shape[0] + 1
    check(b, {3})
    b = batch()
    b.lse.copy_(lse_of(b0))
    b.starts[0] = -1
    check(b, {0})
    b = batch()
    b.starts[1:3] = torch.tensor([154, 4], dtype=torch.int32)   # request 1 decreases; its neighbours overlap
    b.attn()
    assert qf.status() == 8


def lse_of(b):
    lse = torch.empty_like(b.lse)
    b.attn(lse=lse)
    return lse


@pytest.mark.gpu
def test_strided_q(dev):
    b = Batch([(5, 40), (90, 200)], 2, 4, 64, BF)
    want = b.attn(lse=b.lse).clone()
    w = b.weights(torch.zeros(2, 2, b.mb * PAGE, device="cuda"))
    T, H, D = b.q.shape
    packed = torch.randn(T, H + 6, D, device="cuda").to(BF)
    packed[:, 3:3 + H] = b.q
    for q in (packed[:, 3:3 + H], b.q.transpose(0, 1).contiguous().transpose(0, 1)):
        b.q = q
        assert torch.equal(b.attn(), want)
        assert torch.equal(b.weights(torch.zeros_like(w)), w)
    b.q = b.q[:, :1].expand(T, H, D)   # one head for all
    b.check_attn(b.attn(lse=b.lse), b.lse)


@pytest.mark.gpu
def test_pages_beyond_2_31_elements(dev):
    nkv, D = 8, 128
    pages = (1 << 31) // (nkv * PAGE * 2 * D) + 40
    cache = torch.zeros(pages, nkv, PAGE, 2 * D, dtype=BF, device="cuda")
    b = Batch([(20, 100), (1, 333)], nkv, 2, D, BF)
    want = b.attn(lse=b.lse).clone()
    w = b.weights(torch.zeros(2, nkv, b.mb * PAGE, device="cuda"))
    far = torch.where(b.table >= 0, pages - 1 - b.table, b.table)
    valid = b.table >= 0
    cache[far[valid].long()] = b.cache[b.table[valid].long()]
    b.cache, b.table = cache, far
    assert torch.equal(b.attn(), want)
    assert torch.equal(b.weights(torch.zeros_like(w)), w)


@pytest.mark.gpu
def test_workspace(dev):
    """Nothing behind the workspace is written, too small a one is refused, what it held does not matter."""
    for lens in ([(1, 900)], [(300, 300)], [(1, 5000), (130, 5000)]):
        b = Batch(lens, 2, 4, 64, BF)
        for name, run in (("ws", lambda: b.attn(lse=b.lse)), ("wws", lambda: b.weights(torch.zeros(len(lens), 2, b.mb * PAGE, device="cuda")))):
            n = getattr(b, name).numel()
            assert n > 0
            big = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
            setattr(b, name, big[:n])
            first = run().clone()
            assert (big[n:] == 171).all()
            big[:n] = 0
            assert torch.equal(run(), first)
            setattr(b, name, big[:n - 256])
            with pytest.raises(qf.QkvFrontError, match="workspace"):
                run()
            setattr(b, name, big[:n])


@pytest.mark.gpu
def test_captured_calls_serve_other_lengths(dev):
    """Two graphs on one workspace, replayed in turn with new starts, lengths, tables and contents."""
    a = Batch([(3, 40), (60, 200), (1, 500), (0, 7)], 2, 4, 64, BF, mb=32)
    c = Batch([(20, 20), (1, 300), (30, 100), (13, 490)], 2, 4, 64, BF, seed=3, mb=32)
    assert a.q.shape == c.q.shape
    out, lse = torch.empty_like(a.q), torch.empty_like(a.lse)
    w = torch.zeros(4, 2, 32 * PAGE, device="cuda")
    live = Batch([(3, 40), (60, 200), (1, 500), (0, 7)], 2, 4, 64, BF, mb=32)
    live.cache = torch.zeros(max(len(a.cache), len(c.cache)), 2, PAGE, 128, dtype=BF, device="cuda")
    live.ws = torch.empty(max(a.ws.numel(), c.ws.numel()), dtype=torch.uint8, device="cuda")

    def step():
        live.attn(out=out, lse=lse)
        live.lse = lse
        live.weights(w, decay=0.0)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for b, g in ((a, graphs[0]), (c, graphs[1]), (a, graphs[1]), (c, graphs[0])):
        for name in ("q", "starts", "table", "context"):
            getattr(live, name).copy_(getattr(b, name))
        live.cache[:len(b.cache)] = b.cache
        g.replay()
        torch.cuda.synchronize()
        ref = b.attn(lse=b.lse)
        assert torch.equal(out, ref) and torch.equal(lse, b.lse)
        rw = b.weights(torch.zeros(4, 2, 32 * PAGE, device="cuda"))
        for r, (_, L) in enumerate(b.lens):
            assert torch.equal(w[r, :, :L], rw[r, :, :L])


@pytest.mark.gpu
def test_streams(dev):
    """On another stream, right behind the kernels that write q, the cache, lengths and tables; without
    programmatic launches."""
    b = Batch([(40, 300), (1, 700)], 2, 4, 128, BF)
    want = b.attn(lse=b.lse).clone()
    w = b.weights(torch.zeros(2, 2, b.mb * PAGE, device="cuda"))
    q, cache, table, context, starts = b.q.clone(), b.cache.clone(), b.table.clone(), b.context.clone(), b.starts.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(side):
            for t in (b.q, b.cache, b.table, b.context, b.starts, b.lse):
                t.zero_()
            for t, v in ((b.q, q), (b.cache, cache), (b.table, table), (b.context, context), (b.starts, starts)):
                t.copy_(v)
            out = b.attn(lse=b.lse)
            w2 = b.weights(torch.zeros_like(w))
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(w2, w)
    qf.set_pdl(False)
    try:
        assert torch.equal(b.attn(lse=b.lse), want) and torch.equal(b.weights(torch.zeros_like(w)), w)
    finally:
        qf.set_pdl(True)


# ---- key_weights -------------------------------------------------------------

def check_weights(b, windows=(0, 3), decays=(1.0, 0.0, 0.875)):
    R = len(b.lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    old = torch.rand(R, b.nkv, b.mb * PAGE, generator=g, device="cuda")
    for window in windows:
        for decay in decays[:1] if window else decays:
            w = old.clone()
            assert b.weights(w, window=window, decay=decay) is w
            out = torch.full_like(old, 5.0)
            b.weights(None if decay == 0 else old, window=window, decay=decay, out=out)
            for r, (n, L) in enumerate(b.lens):
                L = max(L, 0)
                assert torch.equal(out[r, :, :L], w[r, :, :L]) and (out[r, :, L:] == 5).all()
                assert torch.equal(w[r, :, L:], old[r, :, L:])
                ref = decay * old[r, :, :L].double()
                tol = 2.0 ** -22 * ref
                if n > 0 and L > 0:
                    s, es = b.scores(r)
                    lse = b.lse[b.rows(r)].double().view(n, b.nkv, b.group).permute(1, 2, 0)[..., None]
                    p = torch.where(lse == -math.inf, 0.0, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)))
                    if window:
                        p[:, :, :max(0, n - window)] = 0.0
                    seen = torch.where(s == -math.inf, 0.0, s.abs())
                    # a weight: its score, the difference to lse in units of ln 2 (three roundings), 2^-21 of exp
                    rel = es + 2.0 ** -22 * (seen + torch.where(lse == -math.inf, 0.0, lse.abs())) + 2.0 ** -20
                    ref = ref + p.sum((1, 2))
                    # and the sum of all rows in FP32
                    tol = tol + (p * rel).sum((1, 2)) + ref * (n * b.group) * 2.0 ** -24
                bad = (w[r, :, :L].double() - ref).abs() > tol + 1e-30
                assert not bad.any(), (r, n, L, window, decay, int(bad.sum()))
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_weights_sum_to_the_rows(dev, D):
    """Every row gives a total of 1 to its keys."""
    b = Batch([(30, 500), (1, 77), (200, 200)], 2, 4, D, BF)
    b.attn(lse=b.lse)
    w = b.weights(torch.zeros(3, 2, b.mb * PAGE, device="cuda"))
    for r, (n, L) in enumerate(b.lens):
        torch.testing.assert_close(w[r].sum(-1), torch.full((2,), n * 4.0, device="cuda"), rtol=1e-5, atol=0)
    again = b.weights(torch.zeros_like(w))
    assert torch.equal(w, again)


@pytest.mark.gpu
def test_weights_of_keys_with_odd_values(dev):
    """A key of NaN spoils its own weight alone; rows that see no key add nothing; decay 0 reads nothing."""
    b = Batch([(40, 100), (5, 2)], 2, 4, 64, BF)
    b.attn(lse=b.lse)
    want = b.weights(torch.zeros(2, 2, b.mb * PAGE, device="cuda"))
    assert torch.isinf(b.lse[40:43]).all()
    b.cache[int(b.table[0, 80 // PAGE]), :, 80 % PAGE, :64] = math.nan
    got = b.weights(torch.full_like(want, math.nan), decay=0.0)
    keep = torch.arange(100, device="cuda") != 80
    assert torch.equal(got[0, :, :100][:, keep], want[0, :, :100][:, keep]) and got[0, :, 80].isnan().all()
    assert torch.equal(got[1, :, :2], want[1, :, :2])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("D,group", [(64, 4), (128, 8), (64, 64)])
def test_rows_of_lse_minus_infinity(dev, D, group, value):
    """A row of lse -infinity adds nothing, whatever its q holds."""
    b = Batch([(70, 400), (1, 50), (2, 300)], 2, group, D, BF)
    b.attn(lse=b.lse)
    b.lse[3] = b.lse[30:36] = b.lse[70] = -math.inf
    b.lse[71, 1] = -math.inf
    for window in (0, 64):
        want = b.weights(torch.zeros(3, 2, b.mb * PAGE, device="cuda"), window=window)
        assert want[0, :, :300].isfinite().all() and (want[1, :, :50] == 0).all()
        q = b.q
        b.q = b.q.clone()
        b.q[3], b.q[30:36], b.q[70], b.q[71, 1] = value, value, value, value
        assert torch.equal(b.weights(torch.zeros_like(want), window=window), want)
        b.q = q


# ---- together ----------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_serving_chain(dev, in_place):
    """Prompts written, attended and scored in chunks, cut down to a budget, then decoded step by step: against
    plain attention over the kept keys."""
    torch.manual_seed(0)
    nkv, group, D, keep, recent = 2, 4, 64, 96, 16
    H, prompts, blocks = nkv * group, [150, 61, 230], 20
    R = len(prompts)
    cs = qf.rope_table(1024, D)
    qw, kw = (1 + 0.2 * torch.randn(2, D, device="cuda")).to(BF)
    cache = torch.zeros(R * blocks * 2, nkv, PAGE, 2 * D, dtype=BF, device="cuda")
    order = torch.randperm(R * blocks * 2, device="cuda").to(torch.int32)
    table = order[:R * blocks].view(R, blocks).contiguous()
    weights = torch.zeros(R, nkv, blocks * PAGE, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    seen = [0] * R      # tokens so far, of each request

    def step(counts):
        T = sum(counts)
        row = torch.randn(T, (H + 2 * nkv) * D, device="cuda").to(BF)
        q, k, v = (row[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, H), (H, H + nkv), (H + nkv, H + 2 * nkv)))
        starts = [0]
        pos, slots = [], []
        for r, n in enumerate(counts):
            starts.append(starts[-1] + n)
            j = torch.arange(n, device="cuda") + int(lens[r])
            pos.append(torch.arange(n, device="cuda") + seen[r])
            slots.append(table[r].long()[j // PAGE] * PAGE + j % PAGE)
            seen[r] += n
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        lens.add_(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        qr = qf.norm_rope_kv_append(q, k, v, qw, kw, torch.cat(pos), torch.cat(slots), cs, cache, layout="half")
        lse = torch.empty(T, H, device="cuda")
        size = (T, R, H, nkv, D, blocks)
        ws = torch.empty(max(qf.chunk_attn_workspace_bytes(*size), qf.key_weights_workspace_bytes(*size)),
                         dtype=torch.uint8, device="cuda")
        out = qf.chunk_attn(qr, cache, starts, table, lens, ws, lse=lse)
        before = weights.clone()
        qf.key_weights(qr, cache, lse, starts, table, lens, weights, ws)
        for r, n in enumerate(counts):
            L = int(lens[r])
            j = torch.arange(L, device="cuda")
            kv = cache[table[r].long()[j // PAGE], :, j % PAGE].double().permute(1, 0, 2)
            rows = slice(int(starts[r]), int(starts[r + 1]))
            s = torch.einsum("nghd,gld->ghnl", qr[rows].double().view(n, nkv, group, D), kv[..., :D]) * D ** -0.5
            s = s.masked_fill(j > (L - n + torch.arange(n, device="cuda"))[:, None], -math.inf)
            p = torch.softmax(s, -1)
            ref = torch.einsum("ghnl,gld->nghd", p, kv[..., D:]).reshape(n, H, D)
            assert (out[rows].double() - ref).abs().max() < 2.0 ** -7 * float(kv[..., D:].abs().max())
            torch.testing.assert_close(weights[r, :, :L].double() - before[r, :, :L].double(), p.sum((1, 2)), rtol=1e-3,
                                       atol=1e-4)
        if counts == [1] * R:   # the decode kernel of a shared prefix sees the same keys
            pws = torch.empty(qf.prefix_attn_workspace_bytes(R, 1, H, nkv, D, 0, blocks), dtype=torch.uint8, device="cuda")
            other = qf.prefix_attn(qr, cache, None, None, table, lens, pws)
            assert (other.float() - out.float()).abs().max() < 2.0 ** -6 * float(kv[..., D:].abs().max())
    for part in range(3):
        step([n * (part + 1) // 3 - n * part // 3 for n in prompts])
    old_cache, old_table, old_lens = cache.clone(), table.clone(), lens.clone()
    if in_place:
        kept = qf.kv_evict(cache, weights, table, lens, keep, recent)
    else:
        new = order[R * blocks:].view(R, blocks).contiguous()
        w2, l2 = torch.zeros_like(weights), torch.zeros_like(lens)
        kept = qf.kv_evict(cache, weights, table, lens, keep, recent, out_table=new, out_weights=w2, out_lens=l2)
        table, weights, lens = new, w2, l2
    for r in range(R):
        n = min(int(old_lens[r]), keep)
        assert int(lens[r]) == n
        i = torch.arange(n, device="cuda")
        for g in range(nkv):
            k = kept[r, g, :n].long()
            assert torch.equal(cache[table[r].long()[i // PAGE], g, i % PAGE],
                               old_cache[old_table[r].long()[k // PAGE], g, k % PAGE])
    for _ in range(3):
        step([1] * R)
    assert qf.status() == 0
