"""Cases of the normed rotation, chunk attention and cache eviction operators,
for measuring them: their inputs, their plain form in elementary torch
operations, the calls a user makes of the library, and their definition in 64
bits.

The operators are the steps of a serving or training layer around a paged
cache [pages, kv_heads, 16, 2 head_dim] (K | V per slot):

  norm_rope            RMS norm of every head, times a weight, and its rotation
  norm_rope_backward   the gradients of that with respect to x and the weight
  norm_rope_kv_append  norm and rotate q and k, write k and v into the cache
  chunk_attn           attention of each request's new tokens over its paged keys
  key_weights          the attention weight that each cached key received
  kv_evict             the keys of least weight dropped, the others moved together
"""
import math
import random

import torch

own = False

PAGE = 16
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def _norm(name, step, T, heads, dim, rot, layout, dtype, rows=32768):
    return {"name": name, "op": "norm_rope", "step": step, "T": T, "heads": heads, "dim": dim,
            "rot": rot, "layout": layout, "dtype": dtype, "rows": rows}


def _append(name, T, nkv, group, dim, rot, layout, dtype, rows=32768):
    return {"name": name, "op": "norm_rope_kv_append", "T": T, "nkv": nkv, "group": group, "dim": dim,
            "rot": rot, "layout": layout, "dtype": dtype, "rows": rows}


def _chunk(name, R, chunks, n_max, ctx_max, nkv, group, dim, dtype, lens=1):
    return {"name": name, "op": "chunk_attn", "R": R, "chunks": chunks, "n_max": n_max, "ctx_max": ctx_max,
            "nkv": nkv, "group": group, "dim": dim, "dtype": dtype, "lens": lens}


def _weights(name, R, chunks, n_max, ctx_max, nkv, group, dim, window, decay, dtype, lens=1):
    return {"name": name, "op": "key_weights", "R": R, "chunks": chunks, "n_max": n_max, "ctx_max": ctx_max,
            "nkv": nkv, "group": group, "dim": dim, "window": window, "decay": decay, "dtype": dtype,
            "lens": lens}


def _evict(name, R, len_min, len_max, keep, recent, nkv, dim, dtype, lens=1):
    return {"name": name, "op": "kv_evict", "R": R, "len_min": len_min, "len_max": len_max, "keep": keep,
            "recent": recent, "nkv": nkv, "dim": dim, "dtype": dtype, "lens": lens}


def listed():
    return [
        # q heads of one 8-token step: latency
        _norm("norm_decode_8", "forward", 8, 64, 64, 64, "interleaved", "bf16"),
        # a training batch's q heads, half layout: the call and its gradients
        _norm("norm_train_8k", "train", 8192, 32, 128, 128, "half", "bf16"),
        # the gradients of a partly rotated projection of odd shape
        _norm("norm_back_odd", "backward", 4099, 25, 80, 32, "interleaved", "fp16"),
        # a decode step of 33 requests into the cache, 8 KV heads of 128
        _append("append_decode_33", 33, 8, 4, 128, 128, "half", "bf16"),
        # an odd prefill chunk, 5 q heads per KV head, half of each head rotated
        _append("append_prefill_8191", 8191, 8, 5, 128, 64, "half", "fp16"),
        # single tokens of 64 requests at contexts of up to 4K keys
        _chunk("chunk_decode_r64", 64, 0, 1, 4096, 8, 4, 128, "bf16"),
        # a mixed step: four prefill chunks over long contexts beside 20 decoding requests
        _chunk("chunk_mixed_r24", 24, 4, 1021, 16384, 8, 8, 64, "fp16"),
        # prompts prefilled whole, the longest of 8192 tokens
        _chunk("chunk_prefill_8k", 3, 3, 8192, 0, 8, 4, 128, "bf16"),
        # a decode step's weights added to the sums kept so far
        _weights("weights_decode_r16", 16, 0, 1, 8192, 8, 8, 64, 0, 1.0, "bf16"),
        # two prompts' keys scored by the last 64 tokens of their last chunk, before most of them go
        _weights("weights_window_32k", 2, 2, 1021, 32768, 8, 4, 128, 64, 0.0, "bf16"),
        # four short contexts a little over their budget
        _evict("evict_step_r4", 4, 900, 1100, 1000, 100, 2, 64, "fp16"),
        # prompts of up to 16K keys cut down to 2K into new pages
        _evict("evict_prompt_r8", 8, 8000, 16384, 2048, 64, 8, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw(rng):
    op = rng.choice(["norm", "norm", "append", "append", "chunk", "chunk", "chunk", "weights", "weights",
                     "evict", "evict"])
    lens = rng.randrange(1 << 30)
    if op in ("norm", "append"):
        dim = rng.choice([64, 64, 80, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        layout, rows = rng.choice(["interleaved", "half"]), rng.choice([8192, 32768, 131072])
    if op == "norm":
        return _norm("", rng.choice(["forward", "backward", "train"]), _log(rng, 1, 16384), _log(rng, 1, 96),
                     dim, rot, layout, rng.choice(["bf16", "fp16", "fp32"]), rows)
    if op == "append":
        return _append("", _log(rng, 1, 8192), _log(rng, 1, 16), rng.choice([1, 2, 4, 5, 8]), dim, rot, layout,
                       rng.choice(["bf16", "fp16"]), rows)
    dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    nkv, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 8])
    if op == "chunk":
        R = _log(rng, 1, 96)
        chunks = rng.choice([0, 1, R, rng.randint(0, R)])
        return _chunk("", R, chunks, _log(rng, 2, 8192) if chunks else 1, rng.choice([0, _log(rng, 1, 32768)]),
                      nkv, group, dim, dtype, lens)
    if op == "weights":
        R = _log(rng, 1, 48)
        chunks = rng.choice([0, 1, R])
        n_max = _log(rng, 2, 2048) if chunks else 1
        return _weights("", R, chunks, n_max, _log(rng, 1, 32768), nkv, group, dim,
                        rng.choice([0, 0, rng.randint(1, n_max)]), rng.choice([0.0, 1.0, 0.875]), dtype, lens)
    len_max = _log(rng, 40, 32768)
    keep = _log(rng, 17, len_max)
    return _evict("", _log(rng, 1, 32), rng.randint(0, len_max), len_max, keep, rng.randint(0, keep), nkv, dim,
                  dtype, lens)


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], [0, 0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])
    while True:
        c = _draw(rng)
        w, m = work(c), most[c["op"]]
        if w["bytes"] <= m[0] and w["flops"] <= m[1]:
            del c["name"]
            return c


def _lengths(case):
    """(new tokens, keys) of each request, from the case alone."""
    rng = random.Random(case["lens"])
    if case["op"] == "kv_evict":
        lens = [rng.randint(case["len_min"], case["len_max"]) for _ in range(case["R"])]
        lens[0] = case["len_max"]
        return lens
    out = []
    for r in range(case["R"]):
        n = 1
        if r < case["chunks"]:
            n = case["n_max"] if r == 0 else _log(rng, 1, case["n_max"])
        out.append((n, n + (case["ctx_max"] if r == case["R"] - 1 else rng.randint(0, case["ctx_max"]))))
    rng.shuffle(out)   # the long ones anywhere in the batch
    return out


# ---- inputs ------------------------------------------------------------------

def _make_table(rows, rot):
    f = torch.exp(-(torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) * math.log(10000.0))
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _pages(need, spare, g):
    """Distinct pages in random order out of need + spare."""
    return torch.randperm(need + spare, generator=g, device="cuda")[:need].to(torch.int32)


def _cache(shape, g, dtype):
    """A cache of normal values, filled some pages at a time."""
    cache = torch.empty(shape, dtype=dtype, device="cuda")
    for part in cache.split(max(1, (1 << 27) // cache[0].numel())):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return cache


def _keys_of(cache, row, L, dim):
    """K and V [nkv, L, dim] of one request's table row."""
    kv = cache[row[: -(-L // PAGE)].long()].permute(1, 0, 2, 3).reshape(cache.shape[1], -1, 2 * dim)[:, :L]
    return kv[..., :dim], kv[..., dim:]


def _seen(n, L):
    """Which of L keys each of the last n tokens sees."""
    return torch.arange(L, device="cuda") <= torch.arange(L - n, L, device="cuda")[:, None]


def _lse(s, case, lens):
    """ln sum exp of every row's scores, as the attention before the call gives it."""
    nkv, G, D = case["nkv"], case["group"], case["dim"]
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    t = 0
    for r, (n, L) in enumerate(lens):
        k, _ = _keys_of(s["kv_cache"], s["block_table"][r], L, D)
        q = s["q"][t:t + n].float().view(n, nkv, G, D).permute(1, 2, 0, 3) * s["scale"]
        sc = torch.matmul(q.reshape(nkv, G * n, D), k.float().transpose(1, 2)).view(nkv, G, n, L)
        sc = sc.masked_fill(~_seen(n, L), -math.inf)
        lse[t:t + n] = torch.logsumexp(sc, -1).permute(2, 0, 1).reshape(n, nkv * G)
        t += n
    return lse


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s, dtype = case["op"], {"case": case}, DTYPES[case["dtype"]]
    D = case["dim"]

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if op in ("norm_rope", "norm_rope_kv_append"):
        T, rows = case["T"], case["rows"]
        s["cos_sin"] = _make_table(rows, case["rot"])
        if T <= 64:   # decode: every token at its own request's position
            s["positions"] = torch.randint(0, rows, (T,), generator=g, device="cuda")
        else:
            first = int(torch.randint(0, max(1, rows - T), (1,), generator=g, device="cuda"))
            s["positions"] = (first + torch.arange(T, device="cuda", dtype=torch.int64)) % rows
    if op == "norm_rope":
        # activations of tokens and heads of different sizes, a weight around 1
        size = torch.exp(0.5 * torch.randn(T, case["heads"], 1, generator=g, device="cuda"))
        s["x"] = (normal(T, case["heads"], D, dtype=torch.float32) * size).to(dtype)
        s["weight"] = (1.0 + 0.2 * normal(D, dtype=torch.float32)).to(dtype)
        if case["step"] == "train":
            s["x"].requires_grad_()
            s["weight"].requires_grad_()
        if case["step"] != "forward":
            s["grad"] = normal(T, case["heads"], D)
        if case["step"] == "forward":
            s["out"] = torch.empty_like(s["x"])
        if case["step"] == "backward":
            s["grad_x"] = torch.empty_like(s["x"])
            s["grad_weight"] = torch.empty(D, dtype=torch.float32, device="cuda")
            if own:
                from kv_insert_gb300 import qkv_front as qf
                n = qf.norm_rope_backward_workspace_bytes(T, case["heads"], D)
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    elif op == "norm_rope_kv_append":
        nkv, hq = case["nkv"], case["nkv"] * case["group"]
        # the projection's output rows [q | k | v], viewed head by head
        row = normal(T, (hq + 2 * nkv) * D)
        s["q"] = row[:, :hq * D].view(T, hq, D)
        s["k"] = row[:, hq * D:(hq + nkv) * D].view(T, nkv, D)
        s["v"] = row[:, (hq + nkv) * D:].view(T, nkv, D)
        s["q_weight"] = (1.0 + 0.2 * normal(D, dtype=torch.float32)).to(dtype)
        s["k_weight"] = (1.0 + 0.2 * normal(D, dtype=torch.float32)).to(dtype)
        s["q_out"] = torch.empty(T, hq, D, dtype=dtype, device="cuda")
        n = -(-T // PAGE)
        if T <= 64:
            s["slots"] = torch.randperm(64 * PAGE, generator=g, device="cuda")[:T]
            n = 64
        else:
            t = torch.arange(T, device="cuda")
            s["slots"] = _pages(n, 64, g).long()[t // PAGE] * PAGE + t % PAGE
        s["kv_cache"] = _cache((n + 64, nkv, PAGE, 2 * D), g, dtype)
    elif op in ("chunk_attn", "key_weights"):
        lens, R, nkv, hq = _lengths(case), case["R"], case["nkv"], case["nkv"] * case["group"]
        T, blocks = sum(n for n, _ in lens), -(-max(L for _, L in lens) // PAGE)
        s["q"] = normal(T, hq, D)
        counts = [-(-L // PAGE) for _, L in lens]
        pages = _pages(sum(counts), 16, g)
        s["kv_cache"] = _cache((sum(counts) + 16, nkv, PAGE, 2 * D), g, dtype)
        s["block_table"] = torch.zeros(R, blocks, dtype=torch.int32, device="cuda")
        for row, part in zip(s["block_table"], pages.split(counts)):
            row[: len(part)] = part
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["context_lens"] = torch.tensor([L for _, L in lens], dtype=torch.int32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(D)
        if op == "chunk_attn":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(T, hq, dtype=torch.float32, device="cuda")
        else:
            s["lse"] = _lse(s, case, lens)
            # sums of earlier steps; the buffers of two steps take turns
            s["weights"] = torch.rand(R, nkv, blocks * PAGE, generator=g, device="cuda").square()
            s["new_weights"] = torch.zeros_like(s["weights"])
        if own:
            from kv_insert_gb300 import qkv_front as qf
            f = qf.chunk_attn_workspace_bytes if op == "chunk_attn" else qf.key_weights_workspace_bytes
            s["workspace"] = torch.empty(f(T, R, hq, nkv, D, blocks), dtype=torch.uint8, device="cuda")
    else:
        lens, R, nkv, keep = _lengths(case), case["R"], case["nkv"], case["keep"]
        blocks, out_blocks = -(-max(lens) // PAGE), -(-keep // PAGE)
        pages = _pages(R * (blocks + out_blocks), 16, g)
        s["kv_cache"] = _cache((len(pages) + 16, nkv, PAGE, 2 * D), g, dtype)
        s["block_table"] = pages[: R * blocks].view(R, blocks).contiguous()
        s["out_table"] = pages[R * blocks:].view(R, out_blocks).contiguous()
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # few keys have most of the weight, some have none at all
        w = torch.exp(2.5 * torch.randn(R, nkv, blocks * PAGE, generator=g, device="cuda") - 6.0)
        none = torch.rand(w.shape, generator=g, device="cuda") < 0.05
        past = torch.arange(blocks * PAGE, device="cuda") >= s["context_lens"][:, None, None]
        s["weights"] = w.masked_fill(none | past, 0.0)
        s["out_weights"] = torch.empty(R, nkv, out_blocks * PAGE, dtype=torch.float32, device="cuda")
        s["out_lens"] = torch.empty_like(s["context_lens"])
        s["kept"] = torch.empty(R, nkv, keep, dtype=torch.int32, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def _rotate(x, row, layout):
    """x [T, heads, dim] (fp32) rotated over its first row.shape[-1] columns."""
    rot = row.shape[1]
    c, s = row[:, None, : rot // 2], row[:, None, rot // 2:]
    xr = x[..., :rot]
    if layout == "interleaved":
        a, b = xr[..., 0::2], xr[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = xr[..., : rot // 2], xr[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(x, weight, positions, cos_sin, layout):
    x = x.float()
    return _rotate(x * _rms(x) * weight.float(), cos_sin[positions], layout)


def _plain_norm_back(grad, x, weight, positions, cos_sin, layout):
    rot, row = cos_sin.shape[1], cos_sin[positions]
    back = torch.cat([row[:, : rot // 2], -row[:, rot // 2:]], 1)
    g = _rotate(grad.float(), back, layout)
    x = x.float()
    r = _rms(x)
    xh = x * r
    u = g * weight.float()
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    # a long sum, in 64 bits
    dw = (g * xh).sum(1).double().sum(0)
    return dx, dw


def _plain_append(s, case):
    D, cache, slots = case["dim"], s["kv_cache"], s["slots"]
    args = s["positions"], s["cos_sin"], case["layout"]
    s["q_out"].copy_(_plain_norm(s["q"], s["q_weight"], *args))
    cache[slots // PAGE, :, slots % PAGE, :D] = _plain_norm(s["k"], s["k_weight"], *args).to(cache.dtype)
    cache[slots // PAGE, :, slots % PAGE, D:] = s["v"]
    return s["q_out"], cache


def _scores(s, case, r, t, n, L):
    nkv, G, D = case["nkv"], case["group"], case["dim"]
    k, v = _keys_of(s["kv_cache"], s["block_table"][r], L, D)
    q = s["q"][t:t + n].float().view(n, nkv, G, D).permute(1, 2, 0, 3) * s["scale"]
    sc = torch.matmul(q.reshape(nkv, G * n, D), k.float().transpose(1, 2)).view(nkv, G, n, L)
    return sc, v


def _plain_chunk(s, case):
    nkv, G, D = case["nkv"], case["group"], case["dim"]
    t = 0
    for r, (n, L) in enumerate(_lengths(case)):
        sc, v = _scores(s, case, r, t, n, L)
        sc = sc.masked_fill(~_seen(n, L), -math.inf)
        m = sc.amax(-1, keepdim=True)
        e = torch.exp(sc - m)
        total = e.sum(-1, keepdim=True)
        o = torch.matmul(e.view(nkv, G * n, L), v.float()).view(nkv, G, n, D) / total
        s["out"][t:t + n] = o.permute(2, 0, 1, 3).reshape(n, nkv * G, D).to(s["out"].dtype)
        s["lse"][t:t + n] = (m + torch.log(total))[..., 0].permute(2, 0, 1).reshape(n, nkv * G)
        t += n
    return s["out"], s["lse"]


def _plain_weights(s, case):
    nkv, G = case["nkv"], case["group"]
    t = 0
    for r, (n, L) in enumerate(_lengths(case)):
        w = min(n, case["window"] or n)
        sc, _ = _scores(s, case, r, t + n - w, w, L)
        lse = s["lse"][t + n - w:t + n].view(w, nkv, G).permute(1, 2, 0)
        e = torch.exp(sc - lse[..., None]).masked_fill(~_seen(w, L), 0.0)
        total = e.sum((1, 2))
        if case["decay"]:
            total = total + case["decay"] * s["weights"][r, :, :L]
        s["new_weights"][r, :, :L] = total
        t += n
    return s["new_weights"]


def _plain_evict(s, case):
    R, nkv, keep, cache = case["R"], case["nkv"], case["keep"], s["kv_cache"]
    L = s["context_lens"].long()[:, None, None]
    j = torch.arange(s["weights"].shape[2], device="cuda")
    w = s["weights"].masked_fill(j >= L - case["recent"], math.inf).masked_fill(j >= L, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(torch.where(order < L, order, 1 << 30), dim=-1).values
    if kept.shape[2] < keep:
        kept = torch.cat([kept, kept.new_full((R, nkv, keep - kept.shape[2]), 1 << 30)], -1)
    valid = kept < L
    src = torch.where(valid, kept, 0)
    r, h, i = valid.nonzero(as_tuple=True)
    k = src[r, h, i]
    cache[s["out_table"][r, i // PAGE].long(), h, i % PAGE] = cache[s["block_table"][r, k // PAGE].long(), h, k % PAGE]
    s["out_weights"].zero_()
    s["out_weights"][..., :keep] = torch.where(valid, torch.gather(s["weights"], 2, src), 0.0)
    s["out_lens"].copy_(s["context_lens"].clamp(max=keep))
    s["kept"].copy_(torch.where(valid, kept, -1))
    return s["kept"], s["out_lens"], s["out_weights"], cache


def _own_norm(s, case, qf):
    where = s["positions"], s["cos_sin"]
    how = {"eps": EPS, "layout": case["layout"]}
    if case["step"] == "forward":
        return qf.norm_rope(s["x"], s["weight"], *where, out=s["out"], **how)
    if case["step"] == "backward":
        return qf.norm_rope_backward(s["grad"], s["x"], s["weight"], *where, grad_x=s["grad_x"],
                                     grad_weight=s["grad_weight"], workspace=s["workspace"], **how)
    y = qf.norm_rope(s["x"], s["weight"], *where, **how)
    dx, dw = torch.autograd.grad(y, (s["x"], s["weight"]), s["grad"])
    return y.detach(), dx, dw


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from kv_insert_gb300 import qkv_front as qf
        if op == "norm_rope":
            return _own_norm(s, case, qf)
        if op == "norm_rope_kv_append":
            q = qf.norm_rope_kv_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"],
                                       s["slots"], s["cos_sin"], s["kv_cache"], q_out=s["q_out"], eps=EPS,
                                       layout=case["layout"])
            return q, s["kv_cache"]
        if op == "chunk_attn":
            out = qf.chunk_attn(s["q"], s["kv_cache"], s["starts"], s["block_table"], s["context_lens"],
                                s["workspace"], scale=s["scale"], out=s["out"], lse=s["lse"])
            return out, s["lse"]
        if op == "key_weights":
            return qf.key_weights(s["q"], s["kv_cache"], s["lse"], s["starts"], s["block_table"],
                                  s["context_lens"], s["weights"], s["workspace"], window=case["window"],
                                  decay=case["decay"], scale=s["scale"], out=s["new_weights"])
        kept = qf.kv_evict(s["kv_cache"], s["weights"], s["block_table"], s["context_lens"], case["keep"],
                           recent=case["recent"], out_table=s["out_table"], out_weights=s["out_weights"],
                           out_lens=s["out_lens"], kept=s["kept"])
        return kept, s["out_lens"], s["out_weights"], s["kv_cache"]
    if op == "norm_rope":
        where = s["positions"], s["cos_sin"], case["layout"]
        x, weight = s["x"].detach(), s["weight"].detach()
        if case["step"] == "forward":
            s["out"].copy_(_plain_norm(x, weight, *where))
            return s["out"]
        dx, dw = _plain_norm_back(s["grad"], x, weight, *where)
        if case["step"] == "backward":
            s["grad_x"].copy_(dx)
            s["grad_weight"].copy_(dw)
            return s["grad_x"], s["grad_weight"]
        return _plain_norm(x, weight, *where).to(x.dtype), dx.to(x.dtype), dw.to(weight.dtype)
    plain = {"norm_rope_kv_append": _plain_append, "chunk_attn": _plain_chunk, "key_weights": _plain_weights,
             "kv_evict": _plain_evict}
    return plain[op](s, case)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op, size, D = case["op"], 4 if case["dtype"] == "fp32" else 2, case["dim"]
    if op in ("norm_rope", "norm_rope_kv_append"):
        table = min(case["T"], case["rows"]) * case["rot"] * 4
    if op == "norm_rope":
        n = case["T"] * case["heads"] * D
        passes, flops = {"forward": (2, 7), "backward": (3, 16), "train": (5, 23)}[case["step"]]
        return {"bytes": passes * n * size + table + 8 * case["T"] + 2 * D * size, "flops": flops * n}
    if op == "norm_rope_kv_append":
        nkv, hq = case["nkv"], case["nkv"] * case["group"]
        n = case["T"] * (hq + 2 * nkv) * D
        return {"bytes": 2 * n * size + table + 16 * case["T"] + 2 * D * size,
                "flops": 7 * case["T"] * (hq + nkv) * D}
    if op == "kv_evict":
        lens, nkv = _lengths(case), case["nkv"]
        moved = sum(min(L, case["keep"]) for L in lens) * nkv
        return {"bytes": 4 * nkv * sum(lens) + moved * (2 * 2 * D * size + 8) + 4 * nkv * case["R"] * case["keep"],
                "flops": 2 * nkv * sum(lens)}
    nkv, hq, lens = case["nkv"], case["nkv"] * case["group"], _lengths(case)
    keys = sum(L for _, L in lens)
    if op == "chunk_attn":
        rows = sum(n for n, _ in lens) * hq
        seen = hq * sum(n * L - n * (n - 1) // 2 for n, L in lens)
        return {"bytes": keys * nkv * 2 * D * size + 2 * rows * D * size + 4 * rows + 4 * keys // PAGE,
                "flops": 4 * D * seen}
    lens = [(min(n, case["window"] or n), L) for n, L in lens]
    rows = sum(n for n, _ in lens) * hq
    seen = hq * sum(n * L - n * (n - 1) // 2 for n, L in lens)
    return {"bytes": keys * nkv * (D * size + (8 if case["decay"] else 4)) + rows * (D * size + 4) + 4 * keys // PAGE,
            "flops": 2 * D * seen}


# ---- the definition, in 64 bits ----------------------------------------------

def _pairs(case):
    i = torch.arange(case["rot"] // 2, device="cuda")
    return (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + case["rot"] // 2)


def _turn(x, cos, sin, pairs):
    """x (64 bits) with each pair of columns (first, second) turned by its angle."""
    first, second = pairs
    y = x.clone()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., first] * sin + x[..., second] * cos
    return y


def _exact_norm(s, case):
    rows = s["cos_sin"].double()[s["positions"]]
    half, pairs = case["rot"] // 2, _pairs(case)
    cos, sin = rows[:, None, :half], rows[:, None, half:]

    def normed(x, weight):
        x = x.detach().double()
        return _turn(x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.detach().double(), cos, sin, pairs)

    return normed, lambda g: _turn(g.double(), cos, -sin, pairs)


def _exact_evict(s, case):
    keep, nkv, cache = case["keep"], case["nkv"], s["kv_cache"].clone()
    kept = torch.full((case["R"], nkv, keep), -1, dtype=torch.int64, device="cuda")
    weights = torch.zeros(s["out_weights"].shape, dtype=torch.float64, device="cuda")
    lens = _lengths(case)
    for r, L in enumerate(lens):
        for h in range(nkv):
            old = min(L, case["recent"])
            w = s["weights"][r, h, :L - old].double()
            # by weight, the lower index first among equals
            best = sorted(range(L - old), key=list(zip((-w).tolist(), range(L - old))).__getitem__)
            at = sorted(best[: max(0, min(L, keep) - old)]) + list(range(L - old, L))
            at = torch.tensor(at[-keep:], dtype=torch.int64, device="cuda")
            i = torch.arange(len(at), device="cuda")
            kept[r, h, : len(at)] = at
            weights[r, h, : len(at)] = s["weights"][r, h, at].double()
            new, old_page = s["out_table"][r].long()[i // PAGE], s["block_table"][r].long()[at // PAGE]
            cache[new, h, i % PAGE] = s["kv_cache"][old_page, h, at % PAGE]
    return kept, torch.tensor([min(L, keep) for L in lens], device="cuda"), weights, cache


def exact(case, seed):
    s, op, D = prepare(case, seed), case["op"], case["dim"]
    if op == "norm_rope":
        normed, unturned = _exact_norm(s, case)
        y = normed(s["x"], s["weight"])
        if case["step"] == "forward":
            return y
        x, w, g = s["x"].detach().double(), s["weight"].detach().double(), unturned(s["grad"])
        ms = x.square().mean(-1, keepdim=True) + EPS
        dw = (g * x / ms.sqrt()).sum((0, 1))
        dx = g * w / ms.sqrt() - x * ((g * w * x).sum(-1, keepdim=True) / D) * ms.pow(-1.5)
        return (dx, dw) if case["step"] == "backward" else (y, dx, dw)
    if op == "norm_rope_kv_append":
        normed, _ = _exact_norm(s, case)
        cache = s["kv_cache"].double()
        flat = cache.permute(0, 2, 1, 3).reshape(-1, case["nkv"], 2 * D)
        flat[s["slots"]] = torch.cat([normed(s["k"], s["k_weight"]), s["v"].double()], -1)
        cache = flat.view(-1, PAGE, case["nkv"], 2 * D).permute(0, 2, 1, 3).contiguous()
        return normed(s["q"], s["q_weight"]), cache
    if op == "kv_evict":
        return _exact_evict(s, case)
    G, t = case["group"], 0
    rows = s["kv_cache"].permute(0, 2, 1, 3)   # [pages, 16, nkv, 2 D]
    q = s["q"].double()
    if op == "chunk_attn":
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    else:
        out = s["new_weights"].double()
    for r, (n, L) in enumerate(_lengths(case)):
        mine = rows[s["block_table"][r, : -(-L // PAGE)].long()].reshape(-1, case["nkv"], 2 * D)[:L].double()
        first = t if op == "chunk_attn" else t + n - min(n, case["window"] or n)
        for g in range(case["nkv"]):
            heads = slice(g * G, (g + 1) * G)
            total = 0.0
            for a in range(first, t + n, 1024):   # some tokens at a time
                b = min(t + n, a + 1024)
                end = L - (t + n - b)   # keys that the last of them sees
                w = torch.matmul(q[a:b, heads].transpose(0, 1), mine[:end, g, :D].T) * s["scale"]
                hidden = torch.arange(end, device="cuda") > torch.arange(end - (b - a), end, device="cuda")[:, None]
                w = w.masked_fill(hidden, -math.inf)
                if op == "chunk_attn":
                    z = torch.logsumexp(w, -1, keepdim=True)
                    out[a:b, heads] = torch.matmul(torch.exp(w - z), mine[:end, g, D:]).transpose(0, 1)
                    lse[a:b, heads] = z[..., 0].T
                else:
                    part = torch.exp(w - s["lse"][a:b, heads].double().T[..., None]).sum((0, 1))
                    total = total + torch.cat([part, part.new_zeros(L - end)])
            if op == "key_weights":
                if case["decay"]:
                    total = total + case["decay"] * s["weights"][r, g, :L].double()
                out[r, g, :L] = total
        t += n
    return (out, lse) if op == "chunk_attn" else out
