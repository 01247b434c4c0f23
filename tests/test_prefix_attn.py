"""prefix_attn: refusals on the host (no GPU needed), values against a plain
64-bit softmax at the lengths, head layouts and contents where it can go
wrong, and the serving chain it ends: rope_table, rope_kv_append, prefix_attn."""
import math

import pytest
import torch

from kv_insert_gb300 import _build
from kv_insert_gb300 import qkv_front as qf

BF, HF = torch.bfloat16, torch.float16

Q, C, PP, PL, BT, CL, O, LSE, WS = ((i + 1) << 42 for i in range(9))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qf.load()


@pytest.fixture(scope="module")
def dev(lib):
    qf.status()
    return torch.device("cuda:0")


# ---- host refusals -----------------------------------------------------------

def call(lib, **kw):
    a = dict(q=Q, qt=512, qh=64, c=C, pages=64, pp=PP, nb=8, pl=PL, bt=BT, mb=4, cl=CL, R=3, ql=1, H=8,
             nkv=2, D=64, sc=0.125, dt=0, o=O, lse=LSE, ws=WS, n=1 << 40)
    a.update(kw)
    code = lib.prefix_attn(*a.values(), None)
    if code not in (0, 5, 6):
        assert len(lib.prefix_attn_unsupported(*a.values())) > 5
    return code


def test_refusals(lib):
    assert call(lib, R=-1) == 1 and call(lib, R=65536) == 1 and call(lib, ql=0) == 1 and call(lib, ql=1025) == 1
    for kw in (dict(D=32), dict(D=96), dict(nkv=0), dict(nkv=65, H=65), dict(H=0), dict(H=9), dict(H=130),
               dict(dt=2), dict(qt=-8), dict(qt=516), dict(qh=60)):
        assert call(lib, **kw) == 10, kw
    assert call(lib, nb=-1) == 7 and call(lib, mb=-1) == 7 and call(lib, mb=(1 << 24) + 1) == 7
    assert call(lib, pages=0) == 7 and call(lib, pages=1 << 31) == 7
    assert call(lib, R=65535, ql=1024, H=64) == 7
    for sc in (0.0, -1.0, math.nan, math.inf):
        assert call(lib, sc=sc) == 9
    for name in ("q", "c", "pp", "pl", "bt", "cl", "o", "ws"):
        assert call(lib, **{name: 0}) == 3, name
    assert call(lib, q=Q + 8) == 4 and call(lib, o=O + 8) == 4 and call(lib, bt=BT + 2) == 4
    assert call(lib, ws=WS + 128) == 4 and call(lib, lse=LSE + 2) == 4
    assert call(lib, o=Q) == 9 and call(lib, o=C + 4096) == 9 and call(lib, lse=O + 64) == 9
    assert call(lib, ws=Q) == 9 and call(lib, ws=BT) == 9 and call(lib, o=CL) == 9
    assert call(lib, R=0, q=0) == 0
    if not torch.cuda.is_available():
        assert call(lib) in (5, 6) and call(lib, lse=0) in (5, 6)
        assert call(lib, nb=0, pp=0, pl=0) in (5, 6) and call(lib, mb=0, bt=0) in (5, 6)


def test_page_counts_past_64_bits(lib):
    """num_pages * num_kv_heads is bounded without forming a product that wraps."""
    assert call(lib, pages=1 << 62, nkv=4) == 7 and call(lib, pages=(1 << 63) - 1, nkv=8) == 7


def test_packed_calls(lib):
    """The packed calls refuse as the plain ones do, and an integer that would
    not fit its parameter instead of cutting it."""
    a = dict(q=Q, qt=512, qh=64, c=C, pages=64, pp=PP, nb=8, pl=PL, bt=BT, mb=4, cl=CL, R=3, ql=1, H=8,
             nkv=2, D=64, sc=0.125, dt=0, o=O, lse=LSE, ws=WS, n=1 << 40)

    def packed(**kw):
        return lib.prefix_attn_packed(qf._PACK["prefix_attn"](*{**a, **kw}.values()), None)
    for kw in (dict(R=-1), dict(D=96), dict(H=9), dict(dt=2), dict(nb=-1), dict(sc=-1.0), dict(q=0), dict(ws=WS + 128),
               dict(o=Q), dict(R=0)):
        assert packed(**kw) == call(lib, **kw), kw
    for name in ("nb", "mb", "R", "ql", "H", "nkv", "D", "dt"):
        assert packed(**{name: a[name] + (1 << 32)}) == 7, name
    assert lib.rope_packed(qf._PACK["rope"](*[1 << 42, 64, 64, 2 << 42, 3 << 42, 8, 4 << 42, 64, 64, 4 + (1 << 32), 1, 64,
                                              64, 0, 0, 0]), None) == 7
    assert lib.rope_table_packed(qf._PACK["rope_table"](1 << 42, 0, 8, 63, 1e4, 0, 1.0, 0, 1.0, 32.0, 1.0), None) == 10
    for name in qf._PACK:
        assert getattr(lib, name + "_packed")(None, None) == 3, name


def test_binding_refusals():
    q = torch.zeros(4, 8, 64, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        qf.prefix_attn(q, None, None, None, None, None, None, out=q)
    assert qf.prefix_attn_workspace_bytes(1, 0, 8, 1, 64, 1, 1) == 0
    assert qf.prefix_attn_workspace_bytes(1, 1, 8, 1, 96, 1, 1) == 0


# ---- values ------------------------------------------------------------------

def make(R, q_len, nkv, G, D, P, lens, dtype, seed=0, spare=3, fill=math.nan):
    """Inputs on the GPU.  Every slot that no length reaches holds `fill`, and
    every table entry past a length names no page of the cache."""
    g = torch.Generator().manual_seed(seed + 131 * R + 17 * P + G)
    nb = (P + 15) // 16
    own = [(max(0, n) + 15) // 16 for n in lens]
    mb = max(own) if own else 0
    pages = torch.randperm(nb + sum(own) + spare, generator=g)
    cache = torch.full((len(pages), nkv, 16, 2 * D), fill, dtype=dtype)
    prefix = torch.full((nb + 1,), -7, dtype=torch.int32)
    prefix[:nb] = pages[:nb]
    table = torch.full((R, mb + 1), 1 << 30, dtype=torch.int32)
    k = nb
    for r in range(R):
        table[r, :own[r]] = pages[k:k + own[r]]
        k += own[r]
    for entries, n in [(prefix, P)] + [(table[r], lens[r]) for r in range(R)]:
        for b in range((max(n, 0) + 15) // 16):
            m = min(16, n - 16 * b)
            cache[entries[b], :, :m] = torch.randn(nkv, m, 2 * D, generator=g).to(dtype)
    d = dict(q=torch.randn(R * q_len, nkv * G, D, generator=g).to(dtype), kv_cache=cache, prefix_pages=prefix,
             prefix_len=torch.tensor([P], dtype=torch.int32), block_table=table,
             context_lens=torch.tensor(lens, dtype=torch.int32))
    return {n: t.to("cuda:0") for n, t in d.items()}


def workspace(q, kv_cache, prefix_pages, block_table, q_len):
    n = qf.prefix_attn_workspace_bytes(block_table.shape[0], q_len, q.shape[1], kv_cache.shape[1], q.shape[2],
                                       0 if prefix_pages is None else prefix_pages.shape[0], block_table.shape[1])
    return torch.full((n,), 0xA5, dtype=torch.uint8, device=q.device)


def attend(d, q_len, scale=None, ws=None, **kw):
    ws = workspace(d["q"], d["kv_cache"], d["prefix_pages"], d["block_table"], q_len) if ws is None else ws
    T, H, _ = d["q"].shape
    lse = torch.full((T, H), 5.0, device=d["q"].device)
    out = torch.full((T, H, d["q"].shape[2]), 3.0, dtype=d["q"].dtype, device=d["q"].device)
    qf.prefix_attn(d["q"], d["kv_cache"], d["prefix_pages"], d["prefix_len"], d["block_table"],
                   d["context_lens"], ws, q_len=q_len, scale=scale, out=out, lse=lse, **kw)
    return out, lse


def check(d, q_len, out, lse, scale=None):
    """Against the 64-bit softmax.  A weight is rounded to the cache's type
    (half a step, relative), so out may be off by half a step of sum p |v| and
    by its own rounding.  Scores: D products summed in FP32, each step off by
    2^-24 of sum |q k|, which an exponent turns into as much relative error of
    a weight, in the numerator and the sum; the exponential, the sums and the
    division add less than 2^-18 together (exponents up to 2^7 in size are
    rounded to 2^-17 at most; longer sums are split over partials)."""
    q, cache = d["q"].double(), d["kv_cache"].double()
    D = q.shape[2]
    nkv = cache.shape[1]
    G = q.shape[1] // nkv
    scale = D ** -0.5 if scale is None else scale
    half_step = torch.finfo(d["q"].dtype).eps / 2
    rows = cache.permute(0, 2, 1, 3)
    P = int(d["prefix_len"]) if d["prefix_pages"] is not None else 0

    def keys(entries, n):
        return rows[entries[:(n + 15) // 16].long()].reshape(-1, nkv, 2 * D)[:n]
    pre = keys(d["prefix_pages"], P) if P else rows.new_zeros(0, nkv, 2 * D)
    for r, L in enumerate(d["context_lens"].tolist()):
        if L < 0:
            assert torch.all(out[r * q_len:(r + 1) * q_len] == 3.0) and torch.all(lse[r * q_len:(r + 1) * q_len] == 5.0)
            continue
        own = keys(d["block_table"][r], L)
        for i in range(q_len):
            t = r * q_len + i
            kv = torch.cat([pre, own[:max(0, L - q_len + i + 1)]])
            if kv.shape[0] == 0:
                assert torch.all(out[t] == 0) and torch.all(lse[t] == -math.inf)
                continue
            k, v = kv[..., :D].repeat_interleave(G, 1), kv[..., D:].repeat_interleave(G, 1)
            s = torch.einsum("hd,khd->hk", q[t], k) * scale
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            ref, mass = torch.einsum("hk,khd->hd", p, v), torch.einsum("hk,khd->hd", p, v.abs())
            size = (torch.einsum("hd,khd->hk", q[t].abs(), k.abs()) * scale).amax(1)
            d_score = D * 2.0 ** -24 * size + 2.0 ** -18
            tol = half_step * (mass + ref.abs()) * (1 + half_step) + 2 * d_score[:, None] * mass
            bad = ~((out[t].double() - ref).abs() <= tol + (2.0 ** -24 if out.dtype == HF else 0))
            assert not bad.any(), (r, i, int(bad.sum()), float((out[t].double() - ref).abs().max()))
            assert ((lse[t].double() - z).abs() <= 2 * d_score + 2.0 ** -22 * z.abs()).all(), (r, i, lse[t], z)


CASES = [  # R, q_len, nkv, G, D, prefix, own lengths
    (1, 1, 1, 1, 64, 1, [0]), (1, 1, 1, 1, 64, 0, [1]), (1, 1, 1, 8, 128, 0, [0]), (2, 1, 1, 8, 64, 16, [1, 17]),
    (3, 1, 2, 8, 64, 127, [5, 0, 33]), (3, 1, 2, 4, 128, 129, [128, 129, 1]), (4, 1, 1, 7, 64, 500, [1, 40, 16, 15]),
    (2, 8, 2, 8, 64, 300, [8, 70]), (3, 5, 1, 3, 128, 77, [2, 5, 130]), (2, 3, 1, 5, 64, 0, [1, 300]),
    (40, 1, 1, 8, 64, 260, list(range(40))), (17, 1, 2, 16, 64, 1000, [7 * k for k in range(17)]),
    (5, 40, 1, 8, 64, 200, [40, 10, 41, 256, 500]), (2, 130, 1, 2, 128, 0, [130, 260]), (1, 1, 4, 64, 64, 2000, [3]),
    (70, 2, 1, 5, 128, 4099, [2 + k % 3 for k in range(70)]), (1, 1, 1, 2, 64, 20011, [9000]),
    (2, 1, 64, 1, 64, 33, [2, 3]), (1, 7, 3, 33, 64, 640, [7]), (300, 1, 1, 1, 64, 31, [k % 50 for k in range(300)]),
    (9, 1, 1, 8, 64, 128, [-1, 5, -3, 0, 128, 384, -1, 16, 1]), (3, 1, 1, 4, 64, 0, [-1, 0, 700]),
    (75, 1, 50, 4, 64, 3000, [k % 9 for k in range(75)]), (700, 1, 8, 8, 128, 600, [k % 3 for k in range(700)]),
    (1, 1, 2, 8, 128, 70000, [1]), (6, 1, 8, 8, 128, 3000, [100, 2000, 1, 0, 513, 1024]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_values(dev, case, dtype):
    R, q_len, nkv, G, D, P, lens = case
    d = make(R, q_len, nkv, G, D, P, lens, dtype)
    out, lse = attend(d, q_len)
    assert qf.status() == 0
    check(d, q_len, out, lse)
    again, lse2 = attend(d, q_len)                        # the same bits every time
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    (1, 1, 1, 8, 64, 20000, [9]), (5, 1, 1, 8, 128, 20001, [17, 0, 3, -1, 40]), (21, 1, 1, 8, 64, 30007, [5] * 21),
    (70, 1, 1, 8, 128, 20000, [1, 20] * 35), (1, 1, 1, 1, 64, 0, [9003]), (2, 3, 2, 1, 128, 33, [9000, 2]),
], ids=lambda c: "-".join(map(str, c[:6])))
def test_many_partials(dev, case):
    """Long keys of few heads: up to 128 splits of either kind, joined by
    several warps a row."""
    d = make(*case, BF)
    out, lse = attend(d, case[1])
    check(d, case[1], out, lse)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("scale,size", [(0.5, 1.0), (1e-3, 1.0), (0.125, 12.0), (4.0, 3.0)])
def test_scales_and_large_scores(dev, scale, size):
    """Nearly uniform weights, and scores whose maximum grows key after key."""
    d = make(3, 2, 1, 8, 64, 777, [2, 90, 300], BF, seed=4)
    cache = d["kv_cache"]
    cache[..., :64] *= size
    ramp = torch.linspace(0.1, 1.0, d["prefix_pages"].shape[0] - 1, device=dev).to(BF)
    cache[d["prefix_pages"][:-1].long(), ..., :64] *= ramp[:, None, None, None]
    out, lse = attend(d, 2, scale=scale)
    assert qf.status() == 0
    check(d, 2, out, lse, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [14.3, 18.4, 21.5, 22.0, 26.0])
@pytest.mark.parametrize("case", [   # prefix: tiles of 128, 16 and 64 rows; own keys: of 16, 64 and 128
    (70, 1, 16, 2, 64, 6000, [0] * 70), (140, 1, 8, 1, 128, 9000, [1] * 140), (2, 1, 2, 8, 64, 9000, [3, 0]),
    (8, 1, 4, 8, 64, 8000, [0] * 8), (40, 1, 4, 4, 128, 0, [900] * 40), (12, 2, 8, 16, 64, 0, [1500] * 12),
    (4, 70, 8, 1, 64, 0, [4000] * 4), (3, 70, 8, 1, 128, 0, [3000] * 3),
], ids=lambda c: "-".join(map(str, c[:6])))
def test_a_dominant_key_leaves_the_others_their_bits(dev, case, bits):
    """fp16 weights far below a row's largest: one early key with V = 0 takes
    almost all of the weight, thousands of keys `bits` bits below it make the
    output.  With the largest weight at 2^8 at least, weights down to 2^-22 of
    it (2^-14) are rounded to half a step, and no weight by more than half a
    step of a subnormal, 2^-25, or 2^-33 of the largest."""
    R, q_len, nkv, G, D, P, lens = case
    d = make(R, q_len, nkv, G, D, P, lens, HF)
    low = 1.0 - bits * math.log(2.0) / 16.0
    cache = d["kv_cache"]
    used = torch.isfinite(cache[..., :1].float())
    k, v = torch.zeros_like(cache[..., :D]), cache[..., D:].abs() + 0.5
    k[..., 0] = low
    firsts = [d["prefix_pages"][0]] if P else [d["block_table"][r, 0] for r in range(R)]
    for page in firsts:
        k[page.long(), :, 0, 0], v[page.long(), :, 0] = 1.0, 0.0
    d["kv_cache"] = torch.where(used, torch.cat([k, v], -1), cache)
    d["q"] = torch.zeros_like(d["q"])
    d["q"][..., 0] = 16.0
    out, lse = attend(d, q_len, scale=1.0)
    assert qf.status() == 0
    half_step = torch.finfo(HF).eps / 2
    rows = d["kv_cache"].double().permute(0, 2, 1, 3)                     # [pages, 16, nkv, 2 D]

    def keys(entries, n):
        return rows[entries[:(n + 15) // 16].long()].reshape(-1, nkv, 2 * D)[:n]
    for r in range(R):
        for i in range(q_len):
            kv = torch.cat([keys(d["prefix_pages"], P), keys(d["block_table"][r], max(0, lens[r] - q_len + i + 1))])
            p = torch.softmax(16.0 * kv[..., 0], 0)[..., None]            # one row of scores a KV head
            ref, mass = (p * kv[..., D:]).sum(0), (p * kv[..., D:].abs()).sum(0)
            # scores are exact products (16 k), so exponents are off by their own
            # rounding alone: 2^-18 with the exponential, the sums and the division
            tol = half_step * (mass + ref.abs()) * (1 + half_step) + 2 * 2.0 ** -18 * mass + 2.0 ** -24
            if bits > 22:
                tol += 2.0 ** -33 * kv[..., D:].abs().sum(0)
            got = out[r * q_len + i].double().view(nkv, G, D)
            worst = ((got - ref[:, None]).abs() / tol[:, None]).max()
            assert worst <= 1, (r, i, float(worst), float(ref.max()))
    z = torch.logsumexp(16.0 * kv[..., 0], 0)
    assert (lse[-1].double().view(nkv, G) - z[:, None]).abs().max() <= 2.0 ** -17


@pytest.mark.gpu
def test_rows_do_not_disturb_one_another(dev):
    """A NaN or infinite q row, and keys of +-inf score, stay in their rows."""
    d = make(5, 1, 1, 4, 64, 300, [20, 0, 5, 1, 200], BF, seed=9)
    clean, lse = attend(d, 1)
    d["q"][1, 2] = math.nan
    d["q"][3, 0] = math.inf
    out, lse2 = attend(d, 1)
    keep = torch.ones(5, 4, dtype=torch.bool, device=dev)
    keep[1, 2] = keep[3, 0] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], lse2[keep])
    assert torch.isnan(out[~keep].float()).all()
    page = int(d["block_table"][4, 0])
    d["kv_cache"][page, 0, 3, :64] = math.nan             # one key of request 4
    out, lse2 = attend(d, 1)
    keep[4] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[4].float()).all()
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", [   # rows of a request against its keys in tiles of 16, 64 and 128
    (3, 4, 1, 4, 64, 0, [4, 90, 33]), (3, 5, 2, 3, 128, 70, [5, 17, 300]), (2, 8, 1, 8, 64, 300, [200, 9]),
    (3, 8, 2, 5, 128, 0, [64, 8, 129]), (2, 33, 2, 4, 64, 200, [700, 40]), (2, 130, 1, 2, 128, 0, [600, 530]),
    (1, 300, 1, 1, 64, 900, [1000]), (2, 20, 1, 64, 64, 3000, [520, 19]),
], ids=lambda c: "-".join(map(str, c[:6])))
def test_a_key_reaches_only_the_rows_that_see_it(dev, case, dtype):
    """Infinities and NaN in V, and a NaN in K, of keys that a request's later
    tokens see and its earlier ones do not: the earlier rows keep their bits,
    and so do the other columns of V everywhere."""
    R, q_len, nkv, G, D, P, lens = case
    d = make(R, q_len, nkv, G, D, P, lens, dtype)
    clean, lse = attend(d, q_len)
    check(d, q_len, clean, lse)
    e = {n: t.clone() for n, t in d.items()}
    touched = {}                                                      # (row, KV head) -> {column: value}
    for r, L in enumerate(lens):
        for n, back in enumerate({0, 1, q_len // 2, q_len - 1}):      # keys from the last on
            key, g = L - 1 - back, n % nkv
            if key < 0:
                continue
            value = (math.inf, math.nan, -math.inf)[(r + n) % 3]
            e["kv_cache"][int(e["block_table"][r, key // 16]), g, key % 16, D + 7 + 5 * n] = value
            for i in range(q_len):
                if key <= L - q_len + i:
                    touched.setdefault((r * q_len + i, g), {})[7 + 5 * n] = value
    out, lse2 = attend(e, q_len)
    assert qf.status() == 0 and torch.equal(lse, lse2)
    same = torch.ones_like(out, dtype=torch.bool)
    for (t, g), columns in touched.items():
        for c, value in columns.items():
            got = out[t, g * G:(g + 1) * G, c].float()
            assert torch.all(torch.isnan(got) if math.isnan(value) else got == value), (t, g, c, value)
            same[t, g * G:(g + 1) * G, c] = False
    assert torch.equal(out[same], clean[same])
    e = {n: t.clone() for n, t in d.items()}
    e["kv_cache"][int(e["block_table"][0, (lens[0] - 1) // 16]), :, (lens[0] - 1) % 16, 3] = math.nan
    out, lse2 = attend(e, q_len)
    same = torch.ones_like(out, dtype=torch.bool)
    same[q_len - 1] = False                                           # request 0's last token
    assert torch.equal(out[same], clean[same]) and torch.isnan(out[q_len - 1].float()).all()
    assert torch.equal(lse2[same[..., 0]], lse[same[..., 0]]) and qf.status() == 0


@pytest.mark.gpu
def test_no_prefix_and_no_tables(dev):
    d = make(3, 1, 2, 4, 64, 0, [5, 0, 300], HF, seed=2)
    d["prefix_pages"] = d["prefix_len"] = None
    check(d, 1, *attend(d, 1))
    e = make(3, 2, 2, 4, 128, 333, [0, 0, 0], HF, seed=2)
    out, lse = attend(e, 2)
    check(e, 2, out, lse)
    ws = workspace(e["q"], e["kv_cache"], e["prefix_pages"], e["block_table"], 2)
    got = qf.prefix_attn(e["q"], e["kv_cache"], e["prefix_pages"], e["prefix_len"], None, e["context_lens"], ws, q_len=2)
    check(e, 2, got, lse)
    assert qf.status() == 0


@pytest.mark.gpu
def test_a_batch_without_requests(dev):
    """Nothing to do, and nothing written."""
    assert 0 < qf.prefix_attn_workspace_bytes(0, 1, 8, 2, 64, 8, 4) <= qf.prefix_attn_workspace_bytes(1, 1, 8, 2, 64, 8, 4)
    d = make(1, 1, 2, 4, 64, 40, [9], BF)
    ws = workspace(d["q"], d["kv_cache"], d["prefix_pages"], d["block_table"], 1)
    out = qf.prefix_attn(d["q"][:0], d["kv_cache"], d["prefix_pages"], d["prefix_len"], d["block_table"][:0],
                         d["context_lens"][:0], ws)
    assert out.shape == (0, 8, 64) and torch.all(ws == 0xA5) and qf.status() == 0


@pytest.mark.gpu
def test_strided_q(dev):
    """The q columns of packed rows, and heads-major q, as they lie."""
    d = make(4, 1, 2, 4, 64, 200, [3, 40, 0, 17], BF, seed=3)
    ref, lse = attend(d, 1)
    packed = torch.full((4, 24 * 64), math.nan, dtype=BF, device=dev)
    packed[:, 128:128 + 512] = d["q"].reshape(4, -1)
    for q in (packed[:, 128:128 + 512].view(4, 8, 64), d["q"].transpose(0, 1).contiguous().transpose(0, 1)):
        out, lse2 = attend(dict(d, q=q), 1)
        assert torch.equal(out, ref) and torch.equal(lse, lse2)
    with pytest.raises(qf.QkvFrontError, match="multiples of 8"):
        attend(dict(d, q=torch.zeros(4, 8 * 64 + 4, dtype=BF, device=dev)[:, :512].view(4, 8, 64)), 1)


@pytest.mark.gpu
def test_bad_requests_are_skipped(dev):
    """A length beyond its table, a page outside the cache: that request's rows
    stay, the others' bits do not change; a bad prefix stops every row."""
    d = make(6, 2, 2, 4, 64, 150, [30, 10, 64, 20, 2, 300], BF, seed=5)
    good, lse = attend(d, 2)
    assert qf.status() == 0
    e = {k: v.clone() for k, v in d.items()}
    e["context_lens"][1] = 16 * e["block_table"].shape[1] + 1
    e["block_table"][3, 1] = -1
    e["block_table"][5, 11] = e["kv_cache"].shape[0]
    out, lse2 = attend(e, 2)
    assert qf.status() == qf.STATUS_BAD_REQUEST
    for r in range(6):
        rows = slice(2 * r, 2 * r + 2)
        if r in (1, 3, 5):
            assert torch.all(out[rows] == 3.0) and torch.all(lse2[rows] == 5.0)
        else:
            assert torch.equal(out[rows], good[rows]) and torch.equal(lse2[rows], lse[rows])
    for change in (dict(prefix_len=-1), dict(prefix_len=16 * d["prefix_pages"].shape[0] + 1), dict(page=-2),
                   dict(page=d["kv_cache"].shape[0])):
        e = {k: v.clone() for k, v in d.items()}
        if "page" in change:
            e["prefix_pages"][9] = change["page"]
        else:
            e["prefix_len"][0] = change["prefix_len"]
        out, lse2 = attend(e, 2)
        assert qf.status() == qf.STATUS_BAD_REQUEST
        assert torch.all(out == 3.0) and torch.all(lse2 == 5.0), change


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(6, 2, 2, 4, 64, 150, [30, 10, 64, 20, 2, 300]), (4, 20, 2, 5, 128, 0, [700, 640, 530, 20]),
                                  (6, 1, 1, 1, 64, 20000, [5, 1, 9, 70, 2, 40])], ids=lambda c: "-".join(map(str, c[:6])))
def test_skipped_rows_of_a_new_output_are_zero(dev, case):
    """An output that the call makes holds nothing before: rows of padding, of a
    length beyond its table and of a bad page must not show what lay there;
    nor any row behind a bad prefix."""
    R, q_len, nkv, G, D, P, lens = case
    d = make(*case, BF)
    good, _ = attend(d, q_len)
    ws = workspace(d["q"], d["kv_cache"], d["prefix_pages"], d["block_table"], q_len)

    def new():
        torch.full_like(d["q"], 3.0)                                  # its memory is the next output's
        return qf.prefix_attn(d["q"], d["kv_cache"], d["prefix_pages"], d["prefix_len"], d["block_table"],
                              d["context_lens"], ws, q_len=q_len)
    assert torch.equal(new(), good) and qf.status() == 0
    d["context_lens"][0] = -4
    d["context_lens"][1] = 16 * d["block_table"].shape[1] + 1
    d["block_table"][2, 0] = d["kv_cache"].shape[0]
    out = new()
    assert qf.status() == qf.STATUS_BAD_REQUEST
    assert torch.all(out[:3 * q_len] == 0) and torch.equal(out[3 * q_len:], good[3 * q_len:])
    d["prefix_len"][0] = -1
    assert torch.all(new() == 0) and qf.status() == qf.STATUS_BAD_REQUEST


@pytest.mark.gpu
@pytest.mark.parametrize("L", [-1, -9, -(2 ** 31) + 3, -(2 ** 31)])
def test_any_negative_length_is_padding(dev, L):
    """Also where a request's rows are two tiles, whose first ends before the
    request's last token: no sum with such a length may wrap."""
    d = make(3, 10, 2, 8, 64, 100, [40, -1, 7], BF)
    d["context_lens"][1] = L
    out, lse = attend(d, 10)
    check(d, 10, out, lse)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", [
    (3, 20, 2, 5, 64, 130, [700, -1, 12]), (2, 9, 1, 16, 128, 0, [1030, 600]), (5, 33, 2, 4, 128, 70, [520, 0, 33, 32, 1]),
    (1, 300, 1, 3, 64, 2000, [5000]), (2, 130, 4, 2, 64, 16, [131, 2000]), (3, 17, 1, 64, 64, 0, [513, 17, 1024]),
], ids=lambda c: "-".join(map(str, c[:6])))
def test_many_own_rows(dev, case, dtype):
    """Long own keys of many rows a request: tiles of 128 rows whose tokens see
    one key more each, with and without a prefix."""
    d = make(*case, dtype)
    out, lse = attend(d, case[1])
    check(d, case[1], out, lse)
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("P", [0, 200])
def test_a_bad_page_voids_its_request_alone(dev, P):
    """Neighbouring requests share a block of threads there."""
    d = make(4, 20, 2, 5, 64, P, [700, 640, 530, 20], BF)
    good, good_lse = attend(d, 20)
    check(d, 20, good, good_lse)
    assert qf.status() == 0
    d["block_table"][2, 3] = -5
    out, lse = attend(d, 20)
    assert qf.status() == 8
    keep = torch.ones(80, dtype=torch.bool, device=out.device)
    keep[40:60] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])
    assert torch.all(out[40:60] == 3.0) and torch.all(lse[40:60] == 5.0)


@pytest.mark.gpu
@pytest.mark.parametrize("R,q_len,nkv,G,D,blocks,dtype", [
    (70, 1, 2, 2, 64, 1200, BF), (70, 1, 1, 4, 128, 600, HF), (300, 1, 1, 1, 64, 2048, HF),   # pairs of tiles
    (100, 1, 2, 1, 64, 512, BF), (40, 1, 3, 1, 64, 1100, HF), (5, 4, 1, 2, 128, 700, BF),     # one tile
    (9, 8, 1, 1, 64, 1500, BF), (4, 40, 1, 2, 64, 900, BF),                                   # own keys of 16 and 128 rows
])
def test_short_prefix_in_a_wide_table(dev, R, q_len, nkv, G, D, blocks, dtype):
    """A captured call with room for a long prefix serves every shorter one:
    splits, groups and blocks of threads without keys, a first page that is not
    the one fetched ahead, partials that nothing wrote.  The entries behind the
    length name no page, the workspace holds NaN."""
    own = [q_len + r % 20 for r in range(R)] if q_len < 40 else [600 + r for r in range(R)]
    lengths = [0, 1, 127, 129, 1000, 16 * blocks - 5]
    calls = [make(R, q_len, nkv, G, D, P, own, dtype, seed=3) for P in lengths]
    pages = max(c["kv_cache"].shape[0] for c in calls)
    buf = {n: torch.zeros_like(t) for n, t in calls[0].items()}
    buf["kv_cache"] = torch.zeros(pages, nkv, 16, 2 * D, dtype=dtype, device=dev)
    buf["prefix_pages"] = torch.full((blocks,), 1 << 30, dtype=torch.int32, device=dev)
    buf["block_table"] = torch.full((R, max(c["block_table"].shape[1] for c in calls)), -9, dtype=torch.int32, device=dev)
    ws = workspace(buf["q"], buf["kv_cache"], buf["prefix_pages"], buf["block_table"], q_len)
    out = torch.zeros_like(buf["q"])
    lse = torch.zeros(out.shape[:2], device=dev)

    def fill(c):
        for n in ("q", "context_lens", "prefix_len"):
            buf[n].copy_(c[n])
        buf["kv_cache"].fill_(math.nan)
        buf["kv_cache"][:c["kv_cache"].shape[0]] = c["kv_cache"]
        buf["prefix_pages"].fill_(1 << 30)
        n = min(blocks, c["prefix_pages"].shape[0] - 1)
        buf["prefix_pages"][:n] = c["prefix_pages"][:n]
        buf["block_table"].fill_(-9)
        buf["block_table"][:, :c["block_table"].shape[1]] = c["block_table"]
        ws.fill_(0xFF)

    def call():
        qf.prefix_attn(buf["q"], buf["kv_cache"], buf["prefix_pages"], buf["prefix_len"], buf["block_table"],
                       buf["context_lens"], ws, q_len=q_len, out=out, lse=lse)
    fill(calls[0])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, (P, c) in enumerate(zip(lengths + lengths[::-1], calls + calls[::-1])):
        fill(c)
        out.fill_(3.0)
        lse.fill_(5.0)
        call() if i % 2 else graph.replay()
        torch.cuda.synchronize()
        check(buf, q_len, out, lse)
    assert qf.status() == 0


@pytest.mark.gpu
def test_workspace_bounds(dev):
    d = make(3, 1, 1, 8, 64, 1500, [3, 40, 100], BF, seed=6)
    n = qf.prefix_attn_workspace_bytes(3, 1, 8, 1, 64, d["prefix_pages"].shape[0], d["block_table"].shape[1])
    parent = torch.full((n + 1024,), 0x5A, dtype=torch.uint8, device=dev)
    ref, _ = attend(d, 1)
    out, _ = attend(d, 1, ws=parent[512:512 + n])
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert torch.all(parent[:512] == 0x5A) and torch.all(parent[512 + n:] == 0x5A)
    with pytest.raises(qf.QkvFrontError, match="workspace"):
        attend(d, 1, ws=parent[512:512 + n - 1])
    # tables narrower than those the workspace was sized for
    small = dict(d, prefix_pages=d["prefix_pages"][:20].contiguous(),
                 block_table=d["block_table"][:, :1].contiguous(),
                 prefix_len=torch.tensor([317], dtype=torch.int32, device=dev),
                 context_lens=torch.tensor([3, 16, 9], dtype=torch.int32, device=dev))
    check(small, 1, *attend(small, 1, ws=parent[512:512 + n]))


@pytest.mark.gpu
def test_far_pages(dev):
    """Pages whose element offset passes 2^32."""
    nkv, D = 4, 128
    pages = (1 << 32) // (nkv * 16 * 2 * D) + 40
    cache = torch.empty(pages, nkv, 16, 2 * D, dtype=BF, device=dev)
    g = torch.Generator().manual_seed(1)
    far = pages - 1 - torch.randperm(30, generator=g)
    cache[far.to(dev)] = torch.randn(30, nkv, 16, 2 * D, generator=g).to(BF).to(dev)
    d = dict(q=torch.randn(2, 8, D, generator=g).to(BF).to(dev), kv_cache=cache[pages - 40:],
             prefix_pages=far[:20].to(torch.int32).to(dev) - (pages - 40),
             prefix_len=torch.tensor([309], dtype=torch.int32, device=dev),
             block_table=far[20:].view(2, 5).to(torch.int32).to(dev) - (pages - 40),
             context_lens=torch.tensor([80, 33], dtype=torch.int32, device=dev))
    near, lse = attend(d, 1)
    check(d, 1, near, lse)
    e = dict(d, kv_cache=cache, prefix_pages=d["prefix_pages"] + (pages - 40), block_table=d["block_table"] + (pages - 40))
    out, lse2 = attend(e, 1)
    assert qf.status() == 0
    assert torch.equal(out, near) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_the_most_rows(dev):
    """65535 requests and nearly 2^24 rows: offsets of out, q and the partials
    pass 2^31 bytes, and the last of them are right."""
    R, nkv, G, D, P = 65535, 4, 64, 64, 200
    d = make(4, 1, nkv, G, D, P, [0, 5, 33, 1], BF, seed=12)
    want, want_lse = attend(d, 1)
    check(d, 1, want, want_lse)
    rows = torch.arange(R, device=dev) % 4
    big = dict(d, q=d["q"][rows], block_table=d["block_table"][rows].contiguous(),
               context_lens=d["context_lens"][rows].contiguous())
    out, lse = attend(big, 1)
    assert qf.status() == 0
    half_step = torch.finfo(BF).eps / 2
    for r in range(4):   # the split may differ from the small call's: each within its own bound of the formula
        tol = 2 * half_step * (1 + half_step) * (2 * want[r].abs().amax().float() + 4)
        assert ((out[r::4].float() - want[r].float()).abs() <= tol).all()
        assert torch.equal(out[r::4], out[r].expand_as(out[r::4])) and torch.equal(lse[r::4], lse[r].expand_as(lse[r::4]))
    last = {n: big[n][-4:].contiguous() for n in ("q", "block_table", "context_lens")}
    check(dict(d, **last), 1, out[-4:], lse[-4:])


@pytest.mark.gpu
def test_without_programmatic_launches(dev):
    """Every kernel behind the whole of the one before it: the same bits."""
    calls = [(make(70, 1, 2, 4, 64, 900, [20 + r % 9 for r in range(70)], BF), 1),
             (make(3, 20, 2, 5, 128, 130, [700, -1, 12], HF), 20), (make(2, 3, 2, 8, 64, 500, [3, 90], BF), 3)]
    want = [attend(d, q_len) for d, q_len in calls]
    qf.set_pdl(False)
    try:
        got = [attend(d, q_len) for d, q_len in calls]
        torch.cuda.synchronize()
    finally:
        qf.set_pdl(True)
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert qf.status() == 0


@pytest.mark.gpu
def test_streams_graphs_and_a_shared_workspace(dev):
    """Side streams with a workspace each give the direct call's bits; a
    captured call follows the lengths; two captured graphs may share one
    workspace when they run one after the other."""
    a = make(6, 1, 2, 8, 64, 900, [4, 0, 33, 100, 64, 1], BF, seed=7)
    b = make(3, 8, 2, 8, 64, 2000, [8, 100, 500], BF, seed=8)
    ref_a, ref_b = attend(a, 1), attend(b, 8)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            got_a = attend(a, 1)
        with torch.cuda.stream(s2):
            got_b = attend(b, 8)
    torch.cuda.synchronize()
    for got, ref in ((got_a, ref_a), (got_b, ref_b)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    sizes = [qf.prefix_attn_workspace_bytes(6, 1, 16, 2, 64, a["prefix_pages"].shape[0], a["block_table"].shape[1]),
             qf.prefix_attn_workspace_bytes(3, 8, 16, 2, 64, b["prefix_pages"].shape[0], b["block_table"].shape[1])]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=dev)
    graphs = []
    for d, q_len in ((a, 1), (b, 8)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = attend(d, q_len, ws=ws)
        graphs.append((g, res))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_, got), ref in zip(graphs, (ref_a, ref_b)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    a["context_lens"].copy_(torch.tensor([1, 16, 20, 3, 0, 0], dtype=torch.int32))
    a["block_table"][1] = a["block_table"][3]
    a["prefix_len"].fill_(555)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check(a, 1, *graphs[0][1])
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,q_len,nkv,G,D,P,own", [
    (4, 20, 2, 5, 64, 130, 600), (70, 1, 2, 4, 128, 900, 200), (2, 1, 2, 8, 64, 500, 300), (3, 40, 1, 4, 128, 0, 700),
])
def test_calls_follow_the_kernels_before_them(dev, R, q_len, nkv, G, D, P, own):
    """Launched right behind the append that writes their keys, on one stream
    and on two at once, calls give the bits of calls with a device
    synchronization in between: no kernel starts on keys not yet written."""
    g = torch.Generator().manual_seed(17)
    d = make(R, q_len, nkv, G, D, P, [own + r % 3 for r in range(R)], BF, fill=0.0)
    steps, T = 6, R * q_len
    table = qf.rope_table(4096, D)
    new = [torch.randn(2, T, nkv, D, generator=g).to(BF).to(dev) for _ in range(steps)]
    qs = [torch.randn(T, nkv * G, D, generator=g).to(BF).to(dev) for _ in range(steps)]
    pos = torch.tensor([own + r % 3 - q_len + i for r in range(R) for i in range(q_len)], device=dev)
    req = torch.arange(R, device=dev).repeat_interleave(q_len)
    slots = d["block_table"][req, pos // 16].long() * 16 + pos % 16

    def run(sync, e):
        ws = workspace(d["q"], d["kv_cache"], d["prefix_pages"], d["block_table"], q_len)
        outs = [(torch.zeros_like(q), torch.zeros(T, nkv * G, device=dev)) for q in qs]
        turned = [torch.zeros_like(q) for q in qs]
        for (k, v), q, t, (out, lse) in zip(new, qs, turned, outs):   # nothing else is launched in between
            qf.rope_kv_append(q, k, v, pos, slots, table, e["kv_cache"], q_out=t)
            if sync:
                torch.cuda.synchronize()
            qf.prefix_attn(t, e["kv_cache"], e["prefix_pages"], e["prefix_len"], e["block_table"], e["context_lens"],
                           ws, q_len=q_len, out=out, lse=lse)
            if sync:
                torch.cuda.synchronize()
        return outs
    want = run(True, {n: t.clone() for n, t in d.items()})
    torch.cuda.synchronize()
    copies = [{n: t.clone() for n, t in d.items()} for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, e in zip((torch.cuda.Stream(), torch.cuda.Stream()), copies):
        with torch.cuda.stream(s):
            got.append(run(False, e))
    torch.cuda.synchronize()
    for outs in got + [run(False, {n: t.clone() for n, t in d.items()})]:
        for a, b in zip(outs, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,q_len,nkv,G,D,P,own", [
    (4, 20, 2, 5, 64, 900, 640), (70, 1, 2, 4, 128, 900, 200), (16, 8, 2, 8, 64, 1500, 300), (3, 40, 1, 4, 128, 0, 700),
    (2, 1, 2, 8, 64, 500, 300),
])
def test_calls_follow_inputs_rewritten_in_place(dev, R, q_len, nkv, G, D, P, own):
    """A decode loop's buffers: q, the lengths, the tables and the prefix's
    length get new contents at the same addresses right before every call, by
    the kernels just ahead of it.  The bits are those of calls with a device
    synchronization in between: no CTA works on what an earlier call found
    there."""
    g = torch.Generator().manual_seed(23)
    steps, T, H = 24, R * q_len, nkv * G
    nb, mb = (P + 15) // 16, (own + 15) // 16
    pages = nb + R * mb
    cache = torch.randn(pages, nkv, 16, 2 * D, generator=g).to(BF).to(dev)
    table = qf.rope_table(4096, D)
    pos = torch.randint(0, 4096, (T,), generator=g).to(dev)
    none = torch.full((T,), -1, dtype=torch.int64, device=dev)       # no slot is written
    kv = torch.zeros(T, nkv, D, dtype=BF, device=dev)
    per_step = [dict(q=torch.randn(T, H, D, generator=g).to(BF).to(dev),
                     prefix_pages=torch.randperm(pages, generator=g)[:nb].to(torch.int32).to(dev),
                     prefix_len=torch.tensor([P - (i * 37) % (P // 2 + 1)], dtype=torch.int32, device=dev),
                     block_table=torch.randint(0, pages, (R, mb), generator=g).to(torch.int32).to(dev),
                     context_lens=torch.randint(0, own + 1, (R,), generator=g).to(torch.int32).to(dev))
                for i in range(steps)]

    def run(sync):
        b = {n: t.clone() for n, t in per_step[0].items()}
        turned = torch.zeros_like(b["q"])
        ws = workspace(turned, cache, b["prefix_pages"], b["block_table"], q_len)
        outs = [(torch.zeros_like(turned), torch.zeros(T, H, device=dev)) for _ in range(steps)]
        torch.cuda.synchronize()
        for i, (step, (out, lse)) in enumerate(zip(per_step, outs)):
            names = ["prefix_pages", "prefix_len", "block_table", "context_lens"]
            for n in names[i % 4:] + names[:i % 4]:
                b[n].copy_(step[n])
                if i % 2 == 0 and n == names[i % 4]:
                    qf.rope_kv_append(step["q"], kv, kv, pos, none, table, cache, q_out=turned)
            if i % 2:
                qf.rope_kv_append(step["q"], kv, kv, pos, none, table, cache, q_out=turned)
            if sync:
                torch.cuda.synchronize()
            qf.prefix_attn(turned, cache, b["prefix_pages"] if nb else None, b["prefix_len"], b["block_table"],
                           b["context_lens"], ws, q_len=q_len, out=out, lse=lse)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs
    want = run(True)
    for _ in range(5):
        for i, (a, b) in enumerate(zip(run(False), want)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i
    first = dict(per_step[-1], q=qf.rope(per_step[-1]["q"], pos, table), kv_cache=cache)
    if not nb:
        first["prefix_pages"] = first["prefix_len"] = None
    check(first, q_len, *want[-1])
    assert qf.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout,D,rot,dtype", [("interleaved", 64, 64, BF), ("half", 128, 96, HF)])
def test_serving_chain(dev, layout, D, rot, dtype):
    """As a serving program runs them: a scaled table; the prefix's tokens
    appended once; then decode steps of every request appended and attended,
    each against the 64-bit attention over what the cache holds."""
    nkv, G, P, R, steps = 2, 4, 205, 3, 18
    g = torch.Generator().manual_seed(11)
    table = qf.rope_table(4096, rot, scaling="ramp", factor=4.0, original_len=1024, device=dev)
    nb, mb = (P + 15) // 16, (steps + 15) // 16
    pages = torch.randperm(nb + R * mb, generator=g).to(torch.int32).to(dev)
    cache = torch.full((nb + R * mb, nkv, 16, 2 * D), math.nan, dtype=dtype, device=dev)
    prefix, own = pages[:nb].contiguous(), pages[nb:].view(R, mb).contiguous()

    def project(T):
        x = torch.randn(T, (G + 2) * nkv, D, generator=g).to(dtype).to(dev)
        return x[:, :G * nkv], x[:, G * nkv:(G + 1) * nkv], x[:, (G + 1) * nkv:]
    _, k, v = project(P)
    pos = torch.arange(P, device=dev)
    qf.rope_kv_append(None, k, v, pos, prefix[pos // 16].long() * 16 + pos % 16, table, cache, layout=layout)
    plen = torch.tensor([P], dtype=torch.int32, device=dev)
    ws = torch.empty(qf.prefix_attn_workspace_bytes(R, 1, G * nkv, nkv, D, nb, mb), dtype=torch.uint8, device=dev)
    for step in range(steps):
        q, k, v = project(R)
        pos = torch.full((R,), P + step, device=dev)
        slots = own[:, step // 16].long() * 16 + step % 16
        q = qf.rope_kv_append(q, k, v, pos, slots, table, cache, layout=layout)
        d = dict(q=q, kv_cache=cache, prefix_pages=prefix, prefix_len=plen, block_table=own,
                 context_lens=torch.full((R,), step + 1, dtype=torch.int32, device=dev))
        check(d, 1, *attend(d, 1, ws=ws))
    assert qf.status() == 0
