"""kv_evict: refusals on the host (no GPU needed), then the kept keys, their
weights, lengths and slots against a plain selection, exactly."""
import math
import random

import pytest
import torch

from kv_insert_gb300 import _build
from kv_insert_gb300 import qkv_front as qf

BF, HF = torch.bfloat16, torch.float16
PAGE = 16

C, W, BT, CL, OT, OW, OL, KP = ((i + 1) << 42 for i in range(8))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qf.load()


@pytest.fixture(scope="module")
def dev(lib):
    qf.status()
    return torch.device("cuda:0")


def call(lib, **kw):
    a = dict(c=C, pages=64, w=W, bt=BT, mb=8, cl=CL, R=3, nkv=2, D=64, keep=40, rec=8, ot=OT, ob=4, ow=OW, ol=OL, kp=KP)
    a.update(kw)
    code = lib.kv_evict(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.kv_evict_unsupported(*a.values())) > 5
    return code


def test_refusals(lib):
    here = dict(ot=BT, ob=8, ow=W, ol=CL)   # in place
    assert call(lib, R=-1) == 1 and call(lib, R=65536) == 1
    for kw in (dict(D=0), dict(D=12), dict(D=520), dict(nkv=0), dict(nkv=1025)):
        assert call(lib, **kw) == 10, kw
    for kw in (dict(pages=0), dict(mb=0), dict(ob=0), dict(mb=(1 << 20) + 1), dict(keep=0), dict(keep=(1 << 24) + 1),
               dict(rec=-1), dict(rec=41), dict(ob=2)):
        assert call(lib, **kw) == 7, kw
    for name in ("c", "w", "bt", "cl", "ot", "ow", "ol", "kp"):
        assert call(lib, **{name: 0}) == 3, name
    assert call(lib, c=C + 8) == 4 and call(lib, kp=KP + 2) == 4 and call(lib, w=W + 2) == 4
    for kw in (dict(ot=BT, ob=8), dict(ow=W), dict(ol=CL), dict(here, ob=4), dict(here, ow=OW), dict(ot=BT + 4),
               dict(ow=W + 64), dict(ow=C), dict(kp=W), dict(kp=OW + 4), dict(ol=BT), dict(w=C + 64),
               dict(here, kp=BT)):
        assert call(lib, **kw) == 9, kw
    assert call(lib, R=0, c=0) == 0
    if not torch.cuda.is_available():
        assert call(lib) in (5, 6) and call(lib, **here) in (5, 6) and call(lib, **dict(here, keep=4000)) in (5, 6)


def test_binding_refusals():
    cache, w = torch.zeros(4, 1, 16, 128, dtype=BF), torch.zeros(1, 1, 32)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    kept = torch.zeros(1, 1, 8, dtype=torch.int32)
    assert "CUDA" in qf.kv_evict_unsupported(cache, w, table, lens, 8, kept)
    assert "all be given" in qf.kv_evict_unsupported(cache, w, table, lens, 8, kept, out_lens=lens)


class Case:
    """Requests of `lens` keys in random pages (negative: padding)."""

    def __init__(self, lens, nkv, D, dtype, keep, seed=0, weights="heavy"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nkv, self.D, self.keep = lens, nkv, D, keep
        R = len(lens)
        self.mb, self.ob = max(1, max(-(-max(L, 0) // PAGE) for L in lens)) + 1, -(-keep // PAGE) + 1
        pages = torch.randperm(R * (self.mb + self.ob) + 2, generator=g, device="cuda").to(torch.int32)
        self.table = pages[:R * self.mb].view(R, self.mb).contiguous()
        self.out_table = pages[R * self.mb:R * (self.mb + self.ob)].view(R, self.ob).contiguous()
        self.cache = torch.randn(len(pages), nkv, PAGE, 2 * D, generator=g, device="cuda").to(dtype)
        self.context = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (R, nkv, self.mb * PAGE)
        if weights == "heavy":
            w = torch.exp(3 * torch.randn(shape, generator=g, device="cuda") - 5)
        elif weights == "ties":
            w = torch.randint(0, 4, shape, generator=g, device="cuda").float()
        elif weights == "equal":
            w = torch.full(shape, 0.25, device="cuda")
        elif weights == "near":   # differ in the last bits alone
            w = 1.0 + torch.randint(0, 1000, shape, generator=g, device="cuda") * 2.0 ** -23
        else:
            special = torch.tensor([0.0, -0.0, 1e-45, -1e-45, math.inf, -math.inf, math.nan, 1.0, -1.0, 3e38, -3e38],
                                   device="cuda")
            w = special[torch.randint(0, len(special), shape, generator=g, device="cuda")]
        self.w = w

    def expected(self, r, h, recent):
        L = max(self.lens[r], 0)
        old = L - min(L, recent)
        w = self.w[r, h, :L].tolist()
        order = sorted(range(old), key=lambda j: (-(math.inf if math.isnan(w[j]) else w[j]),
                                                  not math.isnan(w[j]), j))
        return sorted(order[:max(0, min(L, self.keep) - (L - old))]) + list(range(old, L))

    def check(self, recent, in_place, skipped=()):
        before = {n: getattr(self, n).clone() for n in ("cache", "w", "context")}
        R, kw = len(self.lens), {}
        expected = [[self.expected(r, h, recent) for h in range(self.nkv)] for r in range(R)]
        cache, w, context, table = self.cache, self.w, self.context, self.table
        if not in_place:
            table = self.out_table
            w = torch.full((R, self.nkv, self.ob * PAGE), 9.0, device="cuda")
            context = torch.full((R,), -5, dtype=torch.int32, device="cuda")
            kw = {"out_table": table, "out_weights": w, "out_lens": context}
        kept = qf.kv_evict(self.cache, self.w, self.table, self.context, self.keep, recent, **kw)
        want_cache = before["cache"].clone()
        for r, L in enumerate(self.lens):
            if L < 0 or r in skipped:
                assert (kept[r] == -1).all()
                assert int(context[r]) == (int(before["context"][r]) if in_place else -5)
                assert torch.equal(w[r].nan_to_num(7.0), before["w"][r].nan_to_num(7.0)) if in_place else (w[r] == 9).all()
                continue
            n = min(L, self.keep)
            assert int(context[r]) == n
            for h in range(self.nkv):
                k = expected[r][h]
                assert kept[r, h].tolist() == k + [-1] * (self.keep - n)
                k = torch.tensor(k, dtype=torch.int64, device="cuda")
                i = torch.arange(n, device="cuda")
                want_cache[table[r].long()[i // PAGE], h, i % PAGE] = before["cache"][self.table[r].long()[k // PAGE], h, k % PAGE]
                assert torch.equal(w[r, h, :n].view(torch.int32), before["w"][r, h, k].view(torch.int32))
                end = L if in_place else w.shape[2]
                assert (w[r, h, n:end] == 0).all()
                if in_place:
                    assert torch.equal(w[r, h, end:].view(torch.int32), before["w"][r, h, end:].view(torch.int32))
        assert torch.equal(cache.view(torch.int16), want_cache.view(torch.int16))
        if not in_place:
            assert torch.equal(self.w.view(torch.int32), before["w"].view(torch.int32))
            assert torch.equal(self.context, before["context"])


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("weights", ["heavy", "ties", "equal", "near", "special"])
@pytest.mark.parametrize("lens,nkv,D,keep,recent", [
    ([1], 1, 64, 1, 0), ([2, 1, 0, 3], 2, 64, 1, 1), ([100, 17, 40, -1, 41, 39], 2, 64, 40, 8), ([300], 3, 128, 299, 0),
    ([700, 64], 1, 80, 64, 64), ([1025, 4097, 1024], 2, 8, 1000, 1), ([33, 90], 2, 256, 32, 5), ([20, 10], 1, 512, 100, 50)])
def test_small(dev, lens, nkv, D, keep, recent, weights, in_place):
    Case(lens, nkv, D, BF, keep, seed=keep, weights=weights).check(recent, in_place)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("weights", ["heavy", "near"])
def test_long(dev, weights, in_place):
    Case([40000, 9000, 12345], 2, 64, HF, 5000, seed=1, weights=weights).check(100, in_place)
    Case([70001], 1, 128, BF, 60000, seed=2, weights=weights).check(0, in_place)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens", [[37, 130, 2], [20001, 18432, 18433]])
def test_weights_off_the_16_byte_grid(dev, lens, in_place):
    c = Case(lens, 2, 64, BF, 30, seed=3)
    room = torch.empty(c.w.numel() + 1, device="cuda")
    w = room[1:].view(c.w.shape).copy_(c.w)
    c.w = w
    c.check(7, in_place)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(8))
def test_drawn(dev, seed):
    rng = random.Random(seed)
    for _ in range(4):
        top = rng.choice([5, 50, 500, 5000])
        keep = rng.randint(1, top)
        c = Case([rng.randint(-1, top) for _ in range(rng.randint(1, 7))], rng.randint(1, 4), rng.choice([16, 64, 128]),
                 rng.choice([BF, HF]), keep, seed=seed, weights=rng.choice(["heavy", "ties", "special"]))
        c.check(rng.randint(0, keep), rng.random() < 0.5)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_bad_requests(dev, in_place):
    """A length beyond the table, a page outside the cache that is needed: that request is left alone and flagged;
    one that is not needed does not matter."""
    c = Case([100, 90, 80], 2, 64, BF, 40)
    c.table[1, 3] = len(c.cache)
    c.table[0, 100 // PAGE + 1] = -1
    if not in_place:
        c.out_table[0, 3] = 1 << 30     # behind the 40 kept keys
    c.check(4, in_place, skipped={1})
    assert qf.status() == 8
    c = Case([100, 90, 80], 2, 64, BF, 40)
    c.context[2] = c.mb * PAGE + 1
    c.check(4, in_place, skipped={2})
    assert qf.status() == 8
    if not in_place:
        c = Case([100, 90, 80], 2, 64, BF, 40)
        c.out_table[1, 2] = -3
        c.check(4, in_place, skipped={1})
        assert qf.status() == 8


@pytest.mark.gpu
def test_repeated_captured_and_on_another_stream(dev):
    """In place a second call finds nothing to do; a captured call serves other lengths and weights; a side stream."""
    c = Case([100, 33, 70], 2, 64, BF, 40)
    c.check(8, True)
    state = [t.clone() for t in (c.cache, c.w, c.context)]
    qf.kv_evict(c.cache, c.w, c.table, c.context, 40, 8)
    for a, b in zip(state, (c.cache, c.w, c.context)):
        assert torch.equal(a, b)
    a, b = Case([100, 33, 70], 2, 64, BF, 40), Case([56, 100, 12], 2, 64, BF, 40, seed=9)
    live = Case([100, 33, 70], 2, 64, BF, 40)
    kept = torch.zeros(3, 2, 40, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qf.kv_evict(live.cache, live.w, live.table, live.context, 40, 8, kept=kept)
    side = torch.cuda.Stream()
    for x in (b, a):
        for n in ("cache", "w", "table", "context"):
            getattr(live, n).copy_(getattr(x, n))
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = Case(x.lens, 2, 64, BF, 40)
            for n in ("cache", "w", "table", "context"):
                getattr(other, n).copy_(getattr(x, n))
        k2 = qf.kv_evict(other.cache, other.w, other.table, other.context, 40, 8, stream=side)
        side.synchronize()
        ref = qf.kv_evict(x.cache, x.w, x.table, x.context, 40, 8)
        for n in ("cache", "w", "context"):
            assert torch.equal(getattr(live, n), getattr(x, n)) and torch.equal(getattr(other, n), getattr(x, n))
        assert torch.equal(kept, ref) and torch.equal(k2, ref)


@pytest.mark.gpu
def test_reasons(dev):
    c = Case([100], 2, 64, BF, 40)
    kept = torch.zeros(1, 2, 40, dtype=torch.int32, device="cuda")
    assert qf.kv_evict_unsupported(c.cache, c.w, c.table, c.context, 40, kept, 8) is None
    assert "recent" in qf.kv_evict_unsupported(c.cache, c.w, c.table, c.context, 40, kept, 41)
    assert "kept" in qf.kv_evict_unsupported(c.cache, c.w, c.table, c.context, 39, kept, 8)
    with pytest.raises(qf.QkvFrontError, match="keep"):
        qf.kv_evict(c.cache, c.w, c.table, c.context, 0)
    assert qf.kv_evict(c.cache, c.w[:0], c.table[:0], c.context[:0], 40).shape == (0, 2, 40)


@pytest.mark.parametrize("in_place", [True, False])
def test_host_tensors_are_refused_before_any_launch(in_place):
    """All of them on the host: the binding refuses the call itself, on a machine with a GPU too."""
    cache, w = torch.zeros(4, 1, 16, 128, dtype=BF), torch.zeros(1, 1, 32)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    kept = torch.zeros(1, 1, 8, dtype=torch.int32)
    other = {} if in_place else {"out_table": table.clone(), "out_weights": w.clone(), "out_lens": lens.clone()}
    with pytest.raises(ValueError, match="CUDA"):
        qf._evict_args(cache, w, table, lens, 8, 0, *(other.get(n) for n in ("out_table", "out_weights", "out_lens")), kept)
    for k in (kept, None):
        with pytest.raises(ValueError, match="CUDA"):
            qf.kv_evict(cache, w, table, lens, 8, kept=k, **other)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_more_rows_than_a_grid_row(dev, in_place):
    """33,002 rows (request, KV head): the launches take them in two grid planes, the second partly filled."""
    R, nkv, D, L, keep = 16501, 2, 8, 11, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    pages = torch.randperm(2 * R, generator=g, device="cuda").to(torch.int32)
    table, other = pages[:R].view(R, 1).contiguous(), pages[R:].view(R, 1).contiguous()
    cache = torch.randn(2 * R, nkv, PAGE, 2 * D, generator=g, device="cuda").to(BF)
    old, w = cache.clone(), torch.rand(R, nkv, PAGE, generator=g, device="cuda")
    old_w, lens = w.clone(), torch.full((R,), L, dtype=torch.int32, device="cuda")
    kw, out_w, out_lens, to = {}, w, lens, table
    if not in_place:
        out_w, out_lens, to = torch.full_like(w, 9.0), torch.zeros_like(lens), other
        kw = {"out_table": to, "out_weights": out_w, "out_lens": out_lens}
    kept = qf.kv_evict(cache, w, table, lens, keep, 1, **kw)
    order = torch.sort(old_w[:, :, :L - 1], dim=-1, descending=True, stable=True).indices[..., :keep - 1]
    want = torch.cat([order.sort(-1).values, torch.full((R, nkv, 1), L - 1, device="cuda")], -1)
    assert torch.equal(kept.long(), want) and (out_lens == keep).all()
    assert torch.equal(out_w[..., :keep], old_w.gather(2, want))
    end = L if in_place else PAGE
    assert (out_w[..., keep:end] == 0).all() and (not in_place or torch.equal(w[..., L:], old_w[..., L:]))
    moved = old[table[:, 0].long()].gather(2, want[..., None].expand(R, nkv, keep, 2 * D))
    expect = old.clone()
    expect[to[:, 0].long(), :, :keep] = moved
    assert torch.equal(cache, expect) and qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_pages_beyond_2_31_elements(dev, in_place):
    nkv, D, keep = 8, 128, 70
    count = (1 << 31) // (nkv * PAGE * 2 * D) + 90
    near = Case([300, 40, 150], nkv, D, BF, keep)
    cache = torch.zeros(count, nkv, PAGE, 2 * D, dtype=BF, device="cuda")
    cache[count - len(near.cache):] = near.cache.flip(0)
    far = Case([300, 40, 150], nkv, D, BF, keep)
    far.cache, far.table, far.out_table = cache, count - 1 - near.table, count - 1 - near.out_table

    def run(c):
        kw = {}
        if not in_place:
            kw = {"out_table": c.out_table, "out_weights": torch.zeros(3, nkv, c.ob * PAGE, device="cuda"),
                  "out_lens": torch.zeros(3, dtype=torch.int32, device="cuda")}
        return qf.kv_evict(c.cache, c.w, c.table, c.context, keep, 9, **kw)
    near.check(9, in_place)
    near = Case([300, 40, 150], nkv, D, BF, keep)
    assert torch.equal(run(near), run(far)) and torch.equal(near.w, far.w) and torch.equal(near.context, far.context)
    assert torch.equal(cache[count - len(near.cache):].flip(0), near.cache)
    assert not cache[:count - len(near.cache)].any() and qf.status() == 0
