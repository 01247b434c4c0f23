"""Cases of the rotary, cache-append and shared-prefix attention operators, for
measuring them: their inputs, their plain form in elementary torch operations,
the calls a user makes of the library, and their definition in 64 bits.

The operators are the steps of a serving layer around a paged cache
[pages, kv_heads, 16, 2 head_dim] (K | V per slot):

  rope_table      cos | sin rows of positions, scaled for long contexts
  rope            rotate heads by their position (and the gradient of that)
  rope_kv_append  rotate q and k, write k and v into the tokens' cache slots
  prefix_attn     decode attention of requests that share a prefix
"""
import math

import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def _table(name, rows, rot, scaling, factor):
    return {"name": name, "op": "rope_table", "rows": rows, "rot": rot, "base": 10000.0,
            "scaling": scaling, "factor": factor, "original": 8192, "first": 0}


def _rope(name, T, heads, dim, rot, layout, dtype, back, rows=32768):
    return {"name": name, "op": "rope", "T": T, "heads": heads, "dim": dim, "rot": rot,
            "layout": layout, "dtype": dtype, "back": back, "rows": rows}


def _append(name, T, nkv, group, dim, rot, layout, dtype, rows=32768):
    return {"name": name, "op": "rope_kv_append", "T": T, "nkv": nkv, "group": group, "dim": dim,
            "rot": rot, "layout": layout, "dtype": dtype, "rows": rows}


def _attn(name, R, q_len, nkv, group, dim, prefix, own_min, own_max, dtype):
    return {"name": name, "op": "prefix_attn", "R": R, "q_len": q_len, "nkv": nkv, "group": group,
            "dim": dim, "prefix": prefix, "own_min": own_min, "own_max": own_max, "dtype": dtype}


def listed():
    return [
        # the table of a short-context model, made when it is loaded
        _table("table_4k", 4096, 64, "none", 1.0),
        # 128K positions of a model stretched 16 times beyond what it was trained on
        _table("table_128k_ramp", 131072, 128, "ramp", 16.0),
        # q and k heads of one 8-token verify step (64 + 8 heads of 64)
        _rope("rope_decode_8", 8, 72, 64, 64, "interleaved", "bf16", False),
        # a training batch's q heads, half layout
        _rope("rope_train_16k", 16384, 32, 128, 128, "half", "bf16", False),
        # the gradient of a partly rotated projection of odd shape
        _rope("rope_back_odd", 4099, 25, 80, 32, "interleaved", "fp16", True),
        # one decode step's tokens into the cache, 8 KV heads of 64
        _append("append_decode_8", 8, 8, 8, 64, 64, "interleaved", "bf16"),
        # a prefill chunk of the same layer
        _append("append_prefill_4k", 4096, 8, 8, 64, 64, "interleaved", "bf16"),
        # an odd prefill chunk with 128-wide heads, half of each rotated
        _append("append_half_8191", 8191, 8, 4, 128, 64, "half", "fp16"),
        # a few samples of one short prompt: latency
        _attn("prefix_short_r4", 4, 1, 1, 8, 64, 500, 1, 40, "bf16"),
        # one system prompt, 16 requests in the 8-token verify step
        _attn("prefix_verify_r16", 16, 8, 8, 8, 64, 8192, 8, 1024, "bf16"),
        # single-token decode of 33 samples of a document, 128-wide heads, 5 q heads per KV head
        _attn("prefix_odd_r33", 33, 1, 4, 5, 128, 16001, 0, 700, "fp16"),
        # single-token decode of 64 requests over a 32K prefix
        _attn("prefix_decode_r64", 64, 1, 8, 8, 64, 32768, 16, 1024, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope_table", "rope", "rope", "rope_kv_append", "rope_kv_append",
                     "prefix_attn", "prefix_attn", "prefix_attn"])
    if op == "rope_table":
        rot = 2 * rng.randint(8, 64)
        c = _table("", _log(rng, 1024, 131072), rot, rng.choice(["none", "linear", "base", "ramp"]),
                   rng.choice([2.0, 4.0, 8.0, 16.0, 32.0]))
        if c["scaling"] == "none":
            c["factor"] = 1.0
        c["first"] = rng.choice([0, 0, rng.randrange(1 << 20)])
        c["base"] = rng.choice([10000.0, 500000.0])
    elif op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        heads = _log(rng, 1, 96)
        T = _log(rng, 1, min(16384, (16384 * 32 * 128) // (heads * dim)))
        dtype = rng.choice(["bf16", "fp16", "fp32"]) if T * heads * dim <= 8192 * 32 * 128 else "bf16"
        c = _rope("", T, heads, dim, rot, rng.choice(["interleaved", "half"]), dtype,
                  rng.random() < 0.5, rng.choice([4096, 32768, 131072]))
    elif op == "rope_kv_append":
        dim = rng.choice([64, 64, 96, 128, 128])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        nkv, group = _log(rng, 1, 16), rng.choice([1, 2, 4, 5, 8, 8])
        T = _log(rng, 1, min(8192, (8191 * 8 * 6 * 128) // (nkv * (group + 2) * dim)))
        c = _append("", T, nkv, group, dim, rot, rng.choice(["interleaved", "half"]),
                    rng.choice(["bf16", "fp16"]), rng.choice([4096, 32768, 131072]))
    else:
        dim = rng.choice([64, 64, 128])
        nkv, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 8])
        q_len = rng.choice([1, 1, 1, 2, 5, 8])
        R = _log(rng, 1, max(1, min(96, 512 // (q_len * max(1, group // 2)))))
        own_max = _log(rng, 1, 1024)
        most = min(131072, (64 * 64 * 64 * 32768) // (R * q_len * nkv * group * dim), (8 * 64 * 49152) // (nkv * dim))
        c = _attn("", R, q_len, nkv, group, dim, _log(rng, 64, most), rng.randint(0, own_max // 2),
                  own_max, rng.choice(["bf16", "fp16"]))
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------

def _frequencies(rot, base, scaling="none", factor=1.0, original=8192, slow=1.0, fast=32.0):
    """Radians per position of each pair, 64 bits."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2.0))
    f = torch.exp(-(i / rot) * math.log(base))
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        g = ((f * original / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * g + (f / factor) * (1.0 - g)
    return f


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def _make_table(rows, rot, base=10000.0):
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * _frequencies(rot, base)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _pages(need, spare, g):
    """Distinct pages in random order out of need + spare."""
    return torch.randperm(need + spare, generator=g, device="cuda")[:need]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}

    def normal(*shape, dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if op == "rope_table":
        # the position of the first row moves with the seed: a chunk of a long context
        s["first"] = case["first"] + seed % 4096
        s["out"] = torch.empty(case["rows"], case["rot"], dtype=torch.float32, device="cuda")
        return s
    dtype = DTYPES[case["dtype"]]
    if op in ("rope", "rope_kv_append"):
        T, rows = case["T"], case["rows"]
        s["cos_sin"] = _make_table(rows, case["rot"])
        first = int(torch.randint(0, max(1, rows - T), (1,), generator=g, device="cuda"))
        s["positions"] = (first + torch.arange(T, device="cuda", dtype=torch.int64)) % rows
        if T <= 64:   # decode: every token at its own request's position
            s["positions"] = torch.randint(0, rows, (T,), generator=g, device="cuda")
    if op == "rope":
        s["x"] = normal(T, case["heads"], case["dim"], dtype=dtype)
        s["out"] = torch.empty_like(s["x"])
    elif op == "rope_kv_append":
        nkv, hq, D = case["nkv"], case["nkv"] * case["group"], case["dim"]
        # the projection's output rows [q | k | v], viewed head by head
        row = normal(T, (hq + 2 * nkv) * D, dtype=dtype)
        s["q"] = row[:, :hq * D].view(T, hq, D)
        s["k"] = row[:, hq * D:(hq + nkv) * D].view(T, nkv, D)
        s["v"] = row[:, (hq + nkv) * D:].view(T, nkv, D)
        s["q_out"] = torch.empty(T, hq, D, dtype=dtype, device="cuda")
        n = -(-T // PAGE)
        if T <= 64:
            s["slots"] = torch.randperm(64 * PAGE, generator=g, device="cuda")[:T]
            n = 64
        else:
            pages = _pages(n, 64, g)
            t = torch.arange(T, device="cuda")
            s["slots"] = pages[t // PAGE] * PAGE + t % PAGE
        s["kv_cache"] = normal(n + 64, nkv, PAGE, 2 * D, dtype=dtype)
    else:
        R, nkv, hq, D = case["R"], case["nkv"], case["nkv"] * case["group"], case["dim"]
        T, P = R * case["q_len"], case["prefix"]
        s["q"] = normal(T, hq, D, dtype=dtype)
        lens = torch.randint(case["own_min"], case["own_max"] + 1, (R,), generator=g, device="cuda")
        lens[0] = case["own_max"]
        npre, nown = -(-P // PAGE), -(-case["own_max"] // PAGE)
        pages = _pages(npre + R * nown, 16, g).to(torch.int32)
        s["kv_cache"] = normal(npre + R * nown + 16, nkv, PAGE, 2 * D, dtype=dtype)
        s["prefix_pages"] = pages[:npre].contiguous()
        s["prefix_len"] = torch.full((1,), P, dtype=torch.int32, device="cuda")
        s["block_table"] = pages[npre:].view(R, nown).contiguous()
        s["context_lens"] = lens.to(torch.int32)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, hq, dtype=torch.float32, device="cuda")
        if own:
            from kv_insert_gb300 import qkv_front as qf
            n = qf.prefix_attn_workspace_bytes(R, case["q_len"], hq, nkv, D, npre, nown)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def _rotate(x, positions, cos_sin, layout, back):
    """x [T, heads, dim] rotated over its first cos_sin.shape[1] columns, fp32."""
    rot = cos_sin.shape[1]
    row = cos_sin[positions][:, None, :]
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    if back:
        s = -s
    x = x.float()
    xr = x[..., :rot]
    if layout == "interleaved":
        a, b = xr[..., 0::2], xr[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = xr[..., : rot // 2], xr[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_table(s, case):
    f = _frequencies(case["rot"], case["base"], case["scaling"], case["factor"], case["original"])
    p = torch.arange(s["first"], s["first"] + case["rows"], dtype=torch.float64, device="cuda")
    ang = p[:, None] * f
    s["out"].copy_(torch.cat([ang.cos(), ang.sin()], 1) * _magnitude(case))
    return s["out"]


def _plain_append(s, case):
    D, cache, slots = case["dim"], s["kv_cache"], s["slots"]
    s["q_out"].copy_(_rotate(s["q"], s["positions"], s["cos_sin"], case["layout"], False))
    k = _rotate(s["k"], s["positions"], s["cos_sin"], case["layout"], False).to(cache.dtype)
    cache[slots // PAGE, :, slots % PAGE, :D] = k
    cache[slots // PAGE, :, slots % PAGE, D:] = s["v"]
    return s["q_out"], cache


def _plain_attn(s, case):
    R, q_len, nkv, D = case["R"], case["q_len"], case["nkv"], case["dim"]
    G, cache, P = case["group"], s["kv_cache"], case["prefix"]
    T = R * q_len
    q = s["q"].float().view(R, q_len, nkv, G, D).permute(2, 0, 1, 3, 4) * s["scale"]
    # the prefix: [nkv, keys, 2 D], one product for every row of a KV head
    pre = cache[s["prefix_pages"].long()].permute(1, 0, 2, 3).reshape(nkv, -1, 2 * D)[:, :P].float()
    sp = torch.matmul(q.reshape(nkv, T * G, D), pre[..., :D].transpose(1, 2))
    sp = sp.view(nkv, R, q_len * G, P)
    # each request's own keys: [nkv, R, keys, 2 D]
    mine = cache[s["block_table"].long()].permute(2, 0, 1, 3, 4).reshape(nkv, R, -1, 2 * D).float()
    so = torch.matmul(q.reshape(nkv, R, q_len * G, D), mine[..., :D].transpose(2, 3))
    last = s["context_lens"][:, None].long() - q_len + torch.arange(q_len, device="cuda")
    hidden = torch.arange(mine.shape[2], device="cuda") > last[..., None]            # [R, q_len, keys]
    so = so.masked_fill(hidden[:, :, None, :].expand(-1, -1, G, -1).reshape(R, q_len * G, -1), -math.inf)
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    ep, eo = torch.exp(sp - m), torch.exp(so - m)
    total = ep.sum(-1) + eo.sum(-1)
    o = torch.matmul(ep.view(nkv, T * G, P), pre[..., D:]).view(nkv, R, q_len * G, D)
    o = (o + torch.matmul(eo, mine[..., D:])) / total[..., None]
    lse = m[..., 0] + torch.log(total)
    s["out"].copy_(o.view(nkv, T, G, D).permute(1, 0, 2, 3).reshape(T, nkv * G, D))
    s["lse"].copy_(lse.view(nkv, T, G).permute(1, 0, 2).reshape(T, nkv * G))
    return s["out"], s["lse"]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from kv_insert_gb300 import qkv_front as qf
        if op == "rope_table":
            return qf.rope_table(case["rows"], case["rot"], base=case["base"], scaling=case["scaling"],
                                 factor=case["factor"], original_len=case["original"],
                                 first_position=s["first"], out=s["out"])
        if op == "rope":
            f = qf.rope_backward if case["back"] else qf.rope
            return f(s["x"], s["positions"], s["cos_sin"], out=s["out"], layout=case["layout"])
        if op == "rope_kv_append":
            q = qf.rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"],
                                  s["kv_cache"], q_out=s["q_out"], layout=case["layout"])
            return q, s["kv_cache"]
        out = qf.prefix_attn(s["q"], s["kv_cache"], s["prefix_pages"], s["prefix_len"],
                             s["block_table"], s["context_lens"], s["workspace"],
                             q_len=case["q_len"], scale=s["scale"], out=s["out"], lse=s["lse"])
        return out, s["lse"]
    if op == "rope_table":
        return _plain_table(s, case)
    if op == "rope":
        s["out"].copy_(_rotate(s["x"], s["positions"], s["cos_sin"], case["layout"], case["back"]))
        return s["out"]
    return _plain_append(s, case) if op == "rope_kv_append" else _plain_attn(s, case)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope_table":
        n = case["rows"] * case["rot"]
        return {"bytes": 4 * n, "flops": 10 * n}
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("rope", "rope_kv_append"):
        table = min(case["T"], case["rows"]) * case["rot"] * 4
    if op == "rope":
        n = case["T"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * size + table + 8 * case["T"], "flops": 3 * case["T"] * case["heads"] * case["rot"]}
    D, nkv, hq = case["dim"], case["nkv"], case["nkv"] * case["group"]
    if op == "rope_kv_append":
        n = case["T"] * (hq + 2 * nkv) * D
        return {"bytes": 2 * n * size + table + 16 * case["T"], "flops": 3 * case["T"] * (hq + nkv) * case["rot"]}
    R, q_len, mean = case["R"], case["q_len"], (case["own_min"] + case["own_max"]) / 2
    keys = case["prefix"] + R * mean
    rows = R * q_len * hq
    return {"bytes": keys * nkv * 2 * D * size + 2 * rows * D * size + 4 * rows + 4 * keys / PAGE,
            "flops": 4 * D * rows * (case["prefix"] + max(0.0, mean - (q_len - 1) / 2))}


# ---- the definition, in 64 bits ----------------------------------------------

def _turn(x, angles_cos, angles_sin, pairs):
    """x (64 bits) with each pair of columns (first, second) turned by its angle."""
    first, second = pairs
    y = x.clone()
    y[..., first] = x[..., first] * angles_cos - x[..., second] * angles_sin
    y[..., second] = x[..., first] * angles_sin + x[..., second] * angles_cos
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope_table":
        rot, base, factor = case["rot"], case["base"], case["factor"]
        cols = []
        p = torch.arange(case["rows"], dtype=torch.float64, device="cuda") + s["first"]
        for i in range(rot // 2):
            b = base * factor ** (rot / (rot - 2)) if case["scaling"] == "base" else base
            f = b ** (-2.0 * i / rot)
            if case["scaling"] == "linear":
                f /= factor
            elif case["scaling"] == "ramp":
                g = min(1.0, max(0.0, (case["original"] * f / (2 * math.pi) - 1.0) / 31.0))
                f = (1 - g) * f / factor + g * f
            cols.append(p * f)
        ang = torch.stack(cols, 1)
        mag = 1.0 + 0.1 * math.log(factor) if case["scaling"] == "ramp" else 1.0
        return torch.cat([torch.cos(ang), torch.sin(ang)], 1) * mag
    if op in ("rope", "rope_kv_append"):
        rot = case["rot"]
        i = torch.arange(rot // 2, device="cuda")
        pairs = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + rot // 2)
        rows = s["cos_sin"].double()[s["positions"]]
        cos, sin = rows[:, None, : rot // 2], rows[:, None, rot // 2:]
    if op == "rope":
        return _turn(s["x"].double(), cos, -sin if case["back"] else sin, pairs)
    D = case["dim"]
    cache = s["kv_cache"].double()
    if op == "rope_kv_append":
        k = _turn(s["k"].double(), cos, sin, pairs)
        flat = cache.permute(0, 2, 1, 3).reshape(-1, case["nkv"], 2 * D)
        flat[s["slots"]] = torch.cat([k, s["v"].double()], -1)
        cache = flat.view(-1, PAGE, case["nkv"], 2 * D).permute(0, 2, 1, 3).contiguous()
        return _turn(s["q"].double(), cos, sin, pairs), cache
    G, q_len, P = case["group"], case["q_len"], case["prefix"]
    rows = cache.permute(0, 2, 1, 3)                                     # [pages, 16, nkv, 2 D]
    pre = rows[s["prefix_pages"].long()].reshape(-1, case["nkv"], 2 * D)[:P]
    q = s["q"].double()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    lens = s["context_lens"].tolist()
    for g in range(case["nkv"]):
        heads = slice(g * G, (g + 1) * G)
        sp = (q[:, heads].reshape(-1, D) @ pre[:, g, :D].T * s["scale"]).view(case["R"], q_len, G, P)
        for r in range(case["R"]):
            mine = rows[s["block_table"][r].long()].reshape(-1, case["nkv"], 2 * D)[: lens[r], g]
            for i in range(q_len):
                t, n = r * q_len + i, max(0, lens[r] - q_len + i + 1)
                w = torch.cat([sp[r, i], q[t, heads] @ mine[:n, :D].T * s["scale"]], 1)
                z = torch.logsumexp(w, 1)
                w = torch.exp(w - z[:, None])
                out[t, heads] = w[:, :P] @ pre[:, g, D:] + w[:, P:] @ mine[:n, D:]
                lse[t, heads] = z
    return out, lse
