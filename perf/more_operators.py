"""Cases and plain forms of the operators that score, thin out and position a paged cache:

  weights  the attention weights that each cached token gets from a decode batch's
           queries or from a chunk of new tokens (all of them, or the last few of
           each request), added to the scores that the token has gathered
  evict    the tokens with the lowest scores leave a request's row of the slot
           table, which closes up; single tokens or whole pages
  rope     rotary positions with several axes (time, height, width)
  append   new keys and values into the paged cache, keys and queries rotated on
           the way at positions that are given (several axes, or rows whose
           positions no longer count the cached tokens)

With `own` false, `run` computes an operator in elementary torch operations;
with `own` true it makes the library's calls.
"""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA = 500000.0
K_SCALE, V_SCALE = 0.75, 1.25


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _weights(name, pool, requests, plo, phi, lo, hi, window, heads, kv_heads, dim, page, decay, empty, lens):
    """hi 0: a decode batch of contexts plo .. phi; else chunks of lo .. hi tokens behind plo .. phi cached ones, of
    which the last `window` ask (0: all)."""
    return {"name": name, "op": "weights", "pool": pool, "requests": requests, "plo": plo, "phi": phi, "lo": lo,
            "hi": hi, "window": window, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "decay": decay,
            "empty": empty, "lens": lens}


def _evict(name, requests, lo, hi, page, drop, keep, sinks, recent, positions, lens):
    """Budgets: `drop` tokens less than a request has, or (drop 0) the share `keep` of them."""
    return {"name": name, "op": "evict", "requests": requests, "lo": lo, "hi": hi, "page": page, "drop": drop,
            "keep": keep, "sinks": sinks, "recent": recent, "positions": positions, "lens": lens}


def _rope(name, dtype, rows, heads, kv_heads, dim, rot, layout, axes, arrange, ladder):
    return {"name": name, "op": "rope", "dtype": dtype, "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "axes": axes, "arrange": arrange, "ladder": ladder}


def _append(name, pool, requests, plo, phi, lo, hi, heads, kv_heads, dim, rot, layout, axes, arrange, ladder, pad, lens):
    return {"name": name, "op": "append", "pool": pool, "requests": requests, "plo": plo, "phi": phi, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "layout": layout, "axes": axes,
            "arrange": arrange, "ladder": ladder, "pad": pad, "lens": lens}


def listed():
    return [
        # one user's decode step: nothing but latency
        _weights("weights one request", "bf16", 1, 180, 180, 0, 0, 0, 32, 8, 128, 1, 1.0, False, 1),
        # a decode batch over long contexts of very different lengths in pages of 16, one request without context yet
        _weights("weights long ragged", "bf16", 64, 1, 8192, 0, 0, 0, 32, 8, 128, 16, 1.0, True, 2),
        # two KV heads of width 64 with eight query heads each over an E4M3 cache, an odd batch, fading scores
        _weights("weights narrow heads in 8 bits", "fp8", 33, 17, 1500, 0, 0, 0, 16, 2, 64, 1, 0.875, False, 3),
        # prompts scored once, by their last 32 tokens, before they are thinned out: a 4-bit cache
        _weights("weights of prompts' ends in 4 bits", "fp4", 16, 1500, 4000, 512, 512, 32, 32, 8, 128, 1, 0.0, False, 4),
        # short chunks behind short prefixes, one to two hundred tokens each, over an E4M3 cache
        _weights("weights short chunks in 8 bits", "fp8", 3, 0, 300, 1, 200, 0, 64, 8, 128, 1, 1.0, False, 5),
        # chunked prefill: 512 new tokens behind 4096 cached ones for each request, every new token asks
        _weights("weights cached prefixes", "bf16", 8, 4096, 4096, 512, 512, 0, 64, 8, 128, 1, 1.0, False, 6),
        # a serving loop at its budget: each request gives a token back per step
        _evict("evict a token each", 48, 100, 2000, 1, 1, 0.0, 4, 32, True, 7),
        # prompts thinned out to a quarter before decoding
        _evict("evict prompts", 64, 1024, 8192, 1, 0, 0.25, 4, 64, False, 8),
        # very long contexts halved in pages of 16
        _evict("evict long rows in pages", 4, 100000, 131072, 16, 0, 0.5, 16, 1024, False, 9),
        # the queries and keys of a prefill of images or video, out of one fused projection
        _rope("rope a video's tokens", "bf16", 16384, 64, 8, 128, 128, "half", "16+24+24", "blocks", "shared"),
        # a decode batch's, the axes taking turns over the pairs
        _rope("rope a decode batch", "bf16", 64, 32, 8, 128, 128, "half", "24+20+20", "turns", "shared"),
        # ragged chunks of image tokens into an E4M3 cache, rows and columns with frequencies of their own, in a batch
        # padded to its bucket
        _append("append an image's tokens in 8 bits", "fp8", 7, 100, 3000, 1, 600, 16, 4, 128, 64, "half", "16+16",
                "blocks", "own", 23, 10),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, pairs):
    n = rng.choice([1, 2, 3, 3, 4])
    cut = sorted(rng.sample(range(1, pairs), n - 1))
    return "+".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))


def draw(rng):
    op = rng.choice(["weights", "weights", "weights", "evict", "evict", "rope", "append"])
    kv_heads, group = rng.choice([(8, 4), (8, 8), (4, 4), (2, 8), (8, 1), (5, 2), (1, 8)])
    dim = rng.choice([64, 128])
    heads = kv_heads * group
    lens = rng.randrange(1, 1 << 20)
    pool = rng.choice(["f32", "bf16", "fp8", "fp4"])
    if op == "weights":
        decay, page = rng.choice([1.0, 1.0, 0.0, 0.9]), rng.choice([1, 1, 16])
        if rng.random() < 0.5:
            n = _between(rng, 1, 64)
            hi = min(_between(rng, 32, 8192), 250000 // n)
            c = _weights("", pool, n, rng.randrange(1, hi + 1), hi, 0, 0, 0, heads, kv_heads, dim, page, decay,
                         rng.random() < 0.3 and n > 1, lens)
        else:
            most = 96 if pool == "f32" else 512
            n, hi, phi = _between(rng, 1, 8), _between(rng, 1, most), _between(rng, 1, 4096)
            c = _weights("", pool, n, rng.choice([0, phi]), phi, rng.randrange(1, hi + 1), hi,
                         rng.choice([0, 0, _between(rng, 1, 64)]), heads, kv_heads, dim, page, decay, False, lens)
    elif op == "evict":
        n = _between(rng, 1, 64)
        hi = min(_between(rng, 32, 131072), 500000 // n)
        recent = rng.choice([0, _between(rng, 1, 256)])
        c = _evict("", n, rng.randrange(1, hi + 1), hi, rng.choice([1, 1, 16, 5]), rng.choice([0, 0, 1]),
                   rng.choice([0.1, 0.5, 0.9, 1.0]), rng.choice([0, 4]), recent, rng.random() < 0.3, lens)
    else:
        rot = rng.choice([dim, dim // 2, 32])
        layout, arrange, ladder = (rng.choice(x) for x in (["half", "pairs"], ["blocks", "turns"], ["shared", "own"]))
        axes = _sections(rng, rot // 2)
        if op == "rope":
            c = _rope("", rng.choice(["bf16", "f32"]), _between(rng, 1, 8192), heads, kv_heads, dim, rot, layout, axes,
                      arrange, ladder)
        else:
            n, hi = _between(rng, 1, 64), _between(rng, 1, 120)
            c = _append("", pool, n, 0, rng.choice([0, 1000, 120000]), rng.randrange(1, hi + 1), hi, heads, kv_heads,
                        dim, rot, layout, axes, arrange, ladder, rng.randrange(0, 40), lens)
    del c["name"]
    return c


def _lengths(c):
    """(cached, new) tokens of each request; a decode batch's whole context counts as cached, an eviction's too."""
    rng = np.random.default_rng(c["lens"])
    n = c["requests"]
    if c["op"] == "evict":
        old = rng.integers(c["lo"], c["hi"] + 1, size=n)
        return old, np.zeros(n, dtype=np.int64)
    old = rng.integers(c["plo"], c["phi"] + 1, size=n)
    new = rng.integers(c["lo"], c["hi"] + 1, size=n) if c["hi"] else np.zeros(n, dtype=np.int64)
    if c.get("empty"):
        old[n // 2] = 0
    return old, new


def _asking(c, new):
    """How many of a request's new tokens ask."""
    return np.minimum(new, c["window"]) if c["window"] else new


def _budgets(c, old):
    return np.maximum(old - c["drop"], 0) if c["drop"] else (old * c["keep"]).astype(np.int64)


def _row_bytes(c):
    hkv, d = c["kv_heads"], c["dim"]
    if c["pool"] == "fp4":
        return (hkv * (d // 2 + d // 16) + 15) // 16 * 16
    return hkv * d * {"f32": 4, "bf16": 2, "fp8": 1}[c["pool"]]


def _kept(c, old):
    """The tokens that each request keeps."""
    p, budget = c["page"], _budgets(c, old)
    first = np.maximum(old - c["recent"], 0) // p          # the first recent page
    head = np.minimum(-(-c["sinks"] // p), first)
    fixed = head * p + old - first * p
    more = np.clip((budget - fixed) // p, 0, first - head)
    return np.where(old <= budget, old, fixed + more * p)


def work(c):
    if c["op"] == "rope":
        es = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * (c["heads"] + c["kv_heads"])
        return {"bytes": n * c["dim"] * es * 2 + 4 * c["rows"] * len(_axes(c)), "flops": n * c["rot"] * 3}
    old, new = _lengths(c)
    if c["op"] == "evict":
        cells = 12 if c["positions"] else 8
        gone = int((old - _kept(c, old)).sum())
        return {"bytes": 2 * cells * int(old.sum()) + 4 * gone + 16 * len(old), "flops": int(old.sum())}
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        es = 4 if c["pool"] == "f32" else 2
        n = int(new.sum())
        return {"bytes": n * (2 * hq * d * es + 2 * hkv * d * es + 2 * _row_bytes(c) + 4 + 4 * len(_axes(c))),
                "flops": n * (hq + hkv) * c["rot"] * 3}
    total = old + new
    ask = _asking(c, new) if c["hi"] else (old > 0).astype(np.int64)
    # (asking token i of n sees all but the n - 1 - i last positions)
    pairs = int((ask * total - ask * (ask - 1) // 2).sum())
    es = 4 if c["pool"] == "f32" else 2
    had = int((total if c["decay"] else total * 0).sum())
    return {"bytes": int(total.sum()) * (_row_bytes(c) + 4 + 4) + 4 * had + int(ask.sum()) * hq * (d * es + 4),
            "flops": 2 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _columns(kv_heads, dim, device):
    """Columns of a 4-bit row: each head's code bytes and scale bytes. Heads are kept in blocks of four, a block's
    codes before its scales."""
    start = [(h // 4) * 4 * (dim // 2 + dim // 16) for h in range(kv_heads)]
    heads = [min(4, kv_heads - h // 4 * 4) for h in range(kv_heads)]
    codes = [[s + (h % 4) * (dim // 2) + i for i in range(dim // 2)] for h, s in enumerate(start)]
    scales = [[s + n * (dim // 2) + (h % 4) * (dim // 16) + i for i in range(dim // 16)]
              for h, (s, n) in enumerate(zip(start, heads))]
    return torch.tensor(codes, device=device), torch.tensor(scales, device=device)


def _fp4_put(pool, slots, x, scale, cols):
    """x [n, kv_heads, d] (fp32) into the rows `slots` of a 4-bit pool: per 16 values the E4M3 scale nearest to their
    largest magnitude over 6, then the nearest E2M1 values, ties to even. (The divisors are tensors: a division by a
    number multiplies by its rounded reciprocal.)"""
    b = x.reshape(*x.shape[:-1], -1, 16)
    sf = (b.abs().amax(-1) / torch.full((), 6.0 * scale, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = (sf.float() * scale)[..., None]
    y = torch.where(f > 0, b / f, b * 0.0)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(y).int()).to(torch.uint8).reshape(x.shape)
    rows = torch.zeros(x.shape[0], pool.shape[1], dtype=torch.uint8, device=pool.device)
    rows[:, cols[0]] = code[..., 0::2] | (code[..., 1::2] << 4)
    rows[:, cols[1]] = sf.view(torch.uint8)
    pool[slots] = rows


def _fp4_values(rows, cols):
    """Values of 4-bit rows [..., row bytes] as [..., kv_heads, d] fp32 (without the tensor's scale)."""
    code = rows[..., cols[0]]
    both = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    mag = torch.tensor(E2M1, device=rows.device)[(both & 7).long()]
    val = torch.where(both > 7, -mag, mag)
    sf = rows[..., cols[1]].view(torch.float8_e4m3fn).float()
    return (val.reshape(*sf.shape, 16) * sf[..., None]).flatten(-2)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _table(lens, page, seed):
    """A slot table [requests, ld] (-1 past a row's end) for contexts `lens`, in pages in a random order, and the
    pool's slots."""
    pages = -(-lens // page)
    need = int(pages.sum())
    slots = max(64, need + need // 4) * page
    order = np.random.default_rng([seed, 1]).permutation(slots // page)
    table = np.full((len(lens), max(1, int(lens.max()))), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(lens):
        mine = (order[at:at + pages[r], None] * page + np.arange(page)).reshape(-1)
        table[r, :n] = mine[:n]
        at += pages[r]
    return table, slots


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "rope":
        _prepare_rope(s, g)
    elif c["op"] == "append":
        _prepare_append(s, g, seed)
    elif c["op"] == "evict":
        _prepare_evict(s, g, seed)
    else:
        _prepare_weights(s, g, seed)
    if own:
        _own_prepare(s)
    return s


def _prepare_weights(s, g, seed):
    c = s["c"]
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    old, new = _lengths(c)
    total = old + new
    table, slots = _table(total, c["page"], seed)
    es = torch.float32 if c["pool"] == "f32" else torch.bfloat16
    kp = torch.zeros(slots, *((_row_bytes(c),) if c["pool"] == "fp4" else (hkv, d)), device="cuda",
                     dtype={"f32": torch.float32, "bf16": torch.bfloat16}.get(c["pool"], torch.uint8))
    s["cols"] = _columns(hkv, d, "cuda")
    for a in range(0, slots, 1 << 16):
        b = min(slots, a + (1 << 16))
        x = _normal(g, b - a, hkv, d, dtype=es)
        if c["pool"] == "fp4":
            _fp4_put(kp, torch.arange(a, b, device="cuda"), x.float(), K_SCALE, s["cols"])
        elif c["pool"] == "fp8":
            kp[a:b] = (x.float() / K_SCALE).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            kp[a:b] = x
    n = int(new.sum()) if c["hi"] else c["requests"]
    s.update(kp=kp, slots=slots, table=_i32(table), pre=_i32(old), ext=_i32(new), old=old, new=new,
             most=int(_asking(c, new).max()) if c["hi"] else 1, q=_normal(g, n, hq, d, dtype=es))
    s["scores"] = torch.rand(table.shape, generator=g, device="cuda") * 4.0
    s["out"] = torch.zeros_like(s["scores"])
    # the log-sum-exp of each query row, as the attention call before left it
    s["lse"] = torch.full((n, hq), -math.inf, device="cuda")
    first = np.cumsum(new) - new
    for r in range(c["requests"]):
        if total[r] == 0:
            continue
        k = _keys(s, s["table"][r, :int(total[r])])
        rows = slice(int(first[r]), int(first[r] + new[r])) if c["hi"] else slice(r, r + 1)
        q = s["q"][rows].float()
        w = torch.einsum("nhgd,lhd->nhgl", q.reshape(q.shape[0], hkv, hq // hkv, d), k).flatten(1, 2) / math.sqrt(d)
        if c["hi"]:
            i = torch.arange(int(total[r]), device="cuda")
            w.masked_fill_(i[None, :] > int(old[r]) + torch.arange(int(new[r]), device="cuda")[:, None, None], -math.inf)
        s["lse"][rows] = torch.logsumexp(w, -1)


def _prepare_evict(s, g, seed):
    c = s["c"]
    old, _ = _lengths(c)
    table, slots = _table(old, c["page"], seed)
    ld = table.shape[1]
    # what tokens gather: a few get most of it, many the same little, some nothing
    w = torch.randn(c["requests"], ld, generator=g, device="cuda").mul_(2.0).exp_()
    few = torch.rand(c["requests"], ld, generator=g, device="cuda")
    w = torch.where(few < 0.1, torch.zeros_like(w), torch.where(few < 0.3, (w * 8.0).round() / 8.0, w))
    s.update(table=_i32(table), scores=w, pre=_i32(old), budgets=_i32(_budgets(c, old)), old=old)
    s["table_out"] = torch.full_like(s["table"], -1)
    s["scores_out"] = torch.zeros_like(w)
    s["lens_out"] = torch.zeros_like(s["pre"])
    s["evicted"] = torch.full_like(s["table"], -1)
    s["count"] = torch.zeros_like(s["pre"])
    if c["positions"]:
        # rows that have given tokens back before: positions rise by more than one
        step = torch.randint(1, 4, s["table"].shape, generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = step.cumsum(1).to(torch.int32)
        s["positions_out"] = torch.full_like(s["positions"], -1)


def _axes(c):
    return [int(x) for x in c["axes"].split("+")]


def _places(c, n, g):
    """Positions [axes, n] of tokens in images or video: far in time, near in space."""
    far = [100000, 256, 256, 64]
    return torch.stack([torch.randint(0, far[a], (n,), generator=g, device="cuda", dtype=torch.int32)
                        for a in range(len(_axes(c)))])


def _prepare_rope(s, g):
    c = s["c"]
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    # q and k as a fused projection leaves them: columns of one matrix
    qkv = _normal(g, c["rows"], (hq + 2 * hkv) * d, dtype=torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["pos"] = _places(c, c["rows"], g)
    s["q_out"] = torch.empty(c["rows"], hq, d, dtype=qkv.dtype, device="cuda")
    s["k_out"] = torch.empty(c["rows"], hkv, d, dtype=qkv.dtype, device="cuda")
    s["freq"], s["axis"] = _frequencies(c)


def _prepare_append(s, g, seed):
    c = s["c"]
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    old, new = _lengths(c)
    n = int(new.sum())
    slots = n + n // 4 + 64
    order = np.random.default_rng([seed, 1]).permutation(slots).astype(np.int32)
    table = np.full((c["requests"], int((old + new).max())), -1, dtype=np.int32)
    ends = np.cumsum(new)
    for r in range(c["requests"]):
        table[r, old[r]:old[r] + new[r]] = order[ends[r] - new[r]:ends[r]]
    es = torch.float32 if c["pool"] == "f32" else torch.bfloat16
    if c["pool"] == "fp4":
        s["kp"], s["vp"] = (torch.zeros(slots, _row_bytes(c), dtype=torch.uint8, device="cuda") for _ in "kv")
    elif c["pool"] == "fp8":
        s["kp"], s["vp"] = (_normal(g, slots, hkv, d).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
    else:
        s["kp"], s["vp"] = (_normal(g, slots, hkv, d, dtype=es) for _ in "kv")
    all_rows = n + c["pad"]
    s["q"], s["k"], s["v"] = (_normal(g, all_rows, h, d, dtype=es) for h in (hq, hkv, hkv))
    s["q_out"] = torch.zeros_like(s["q"])
    s["pos"] = _places(c, all_rows, g)
    s.update(table=_i32(table), pre=_i32(old), ext=_i32(new), slots=slots, rows=n, cols=_columns(hkv, d, "cuda"),
             new_slots=torch.from_numpy(order[:n].astype(np.int64)).cuda())
    s["freq"], s["axis"] = _frequencies(c)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_prepare(s):
    import radixattention_prefix_shared_radix_gb300 as sgl
    c = s["c"]
    if "axes" in c:
        s["rope"] = sgl.sgl_rope_create(
            c["dim"], rot_dim=c["rot"], theta=THETA, axes=_axes(c), own_ladder=c["ladder"] == "own",
            layout=sgl.SGL_ROPE_HALF if c["layout"] == "half" else sgl.SGL_ROPE_PAIRS,
            arrange=sgl.SGL_ROPE_AXES_BLOCKS if c["arrange"] == "blocks" else sgl.SGL_ROPE_AXES_TURNS)
    size = 256
    if c["op"] in ("weights", "append"):
        kind = {"f32": sgl.SGL_DTYPE_F32, "bf16": sgl.SGL_DTYPE_BF16, "fp8": sgl.SGL_DTYPE_BF16_FP8KV,
                "fp4": sgl.SGL_DTYPE_BF16_FP4KV}[c["pool"]]
        host = {"host_prefix_lens": s["old"], "host_extend_lens": s["new"]} if c["op"] == "weights" and c["hi"] else {}
        s["params"] = sgl.make_params(kind, c["requests"], c["heads"], c["kv_heads"], c["dim"], s["slots"],
                                      c.get("page", 1), k_scale=K_SCALE, v_scale=V_SCALE, **host)
        if c["op"] == "weights":
            size = sgl.sgl_attn_weights_workspace_bytes(s["params"], c["window"])
    s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")


def _own_run(s):
    import radixattention_prefix_shared_radix_gb300 as sgl
    c = s["c"]
    if c["op"] == "weights":
        sgl.sgl_attn_weights(s["q"], s["lse"], s["kp"], s["table"], s["pre"], s["ext"] if c["hi"] else None, s["params"],
                             s["scores"] if c["decay"] else None, s["out"], s["ws"], decay=c["decay"],
                             window=c["window"])
    elif c["op"] == "evict":
        sgl.sgl_kv_evict(s["scores"], s["table"], s["pre"], s["budgets"], s["scores_out"], s["table_out"], s["lens_out"],
                         s["ws"], evicted=s["evicted"], evicted_count=s["count"], positions=s.get("positions"),
                         positions_out=s.get("positions_out"), page_size=c["page"], sinks=c["sinks"],
                         recent=c["recent"])
    elif c["op"] == "rope":
        sgl.sgl_rope(s["rope"], s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
    else:
        sgl.sgl_kv_append_at(s["rope"], s["params"], s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["pre"],
                             s["ext"], s["pos"], s["q_out"], s["ws"])


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _keys(s, at):
    """The keys of the pool's rows `at` in fp32."""
    rows = s["kp"][at.clamp(min=0).long()]
    if s["c"]["pool"] == "fp4":
        return _fp4_values(rows, s["cols"]) * K_SCALE
    if s["c"]["pool"] == "fp8":
        return rows.view(torch.float8_e4m3fn).float() * K_SCALE
    return rows.float()


def _plain_weights(s):
    c = s["c"]
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    where = torch.arange(s["table"].shape[1], device="cuda")
    k = _keys(s, s["table"]).permute(0, 2, 3, 1)                       # [b, hkv, d, L]
    total = (s["pre"] + s["ext"])[:, None]
    if c["hi"]:
        # the asking rows in a rectangle of the longest request's
        ask = s["ext"].clamp(max=c["window"]) if c["window"] else s["ext"]
        i = torch.arange(s["most"], device="cuda")
        there = i[None] < ask[:, None]
        row = torch.where(there, (s["ext"].cumsum(0) - ask)[:, None] + i, 0).long()
        q, lse = s["q"][row], s["lse"][row]                            # [b, n, hq, ..]
        seen = (where <= (total - ask[:, None] + i)[..., None]) & there[..., None]
        fresh = where >= s["pre"][:, None]
    else:
        q, lse = s["q"][:, None], s["lse"][:, None]
        seen = (where < total)[:, None]
        fresh = where >= total - 1
    b, n = q.shape[:2]
    w = q.float().reshape(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d) @ k
    w = w.reshape(b, hkv, n, hq // hkv, -1) * (1.0 / math.sqrt(d))
    w = w - lse.reshape(b, n, hkv, hq // hkv).permute(0, 2, 1, 3)[..., None]
    w = w.exp().masked_fill(~seen[:, None, :, None], 0.0).sum((1, 2, 3))
    if c["decay"]:
        w = torch.where(fresh, w, s["scores"] * c["decay"] + w)
    s["out"].copy_(torch.where(where < total, w, s["out"]))


def _plain_evict(s):
    c = s["c"]
    p, n, budget = c["page"], s["pre"][:, None], s["budgets"][:, None]
    b, ld = s["table"].shape
    where = torch.arange(ld, device="cuda", dtype=torch.int32)[None]
    pages = -(-ld // p)
    page = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    first = torch.div((n - c["recent"]).clamp(min=0), p, rounding_mode="floor")
    head = first.clamp(max=-(-c["sinks"] // p))
    fixed = head * p + n - first * p
    more = torch.div(budget - fixed, p, rounding_mode="floor").clamp(min=0).minimum(first - head)
    # a page is worth its best token
    w = torch.full((b, pages * p), -math.inf, device="cuda")
    w[:, :ld] = s["scores"]
    w = w.reshape(b, pages, p).amax(-1)
    middle = (page >= head) & (page < first)
    order = w.masked_fill(~middle, -math.inf).sort(dim=1, descending=True, stable=True).indices
    # (pages outside the middle, worth nothing, may stand between those inside: count these alone)
    counted = middle.gather(1, order).cumsum(1)
    rank = torch.empty_like(counted).scatter_(1, order, counted)
    keep = (~middle | (rank <= more)).repeat_interleave(p, 1)[:, :ld]
    keep = (keep | (n <= budget)) & (where < n)
    to = keep.cumsum(1) - 1
    left = keep.sum(1, keepdim=True)
    gone = (where < n) & ~keep
    for name, fill in (("table", -1), ("scores", 0.0)) + ((("positions", -1),) if c["positions"] else ()):
        moved = torch.full((b, ld + 1), fill, dtype=s[name].dtype, device="cuda")
        moved.scatter_(1, torch.where(keep, to, ld), s[name])
        out = s[name + "_out"]
        out.copy_(torch.where(where < left, moved[:, :ld], torch.where(where < n, fill, out)))
    lost = torch.full((b, ld + 1), -1, dtype=torch.int32, device="cuda")
    lost.scatter_(1, torch.where(gone, gone.cumsum(1) - 1, ld), s["table"])
    s["evicted"].copy_(torch.where(where < n - left, lost[:, :ld], s["evicted"]))
    s["lens_out"].copy_(left[:, 0])
    s["count"].copy_((n - left)[:, 0])


def _frequencies(c):
    """Radians per position of each pair, and its axis."""
    axes, pairs = _axes(c), c["rot"] // 2
    if c["arrange"] == "blocks":
        axis = [a for a, n in enumerate(axes) for _ in range(n)]
    else:
        axis, left = [], list(axes)
        while len(axis) < pairs:
            for a in range(len(axes)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    if c["ladder"] == "own":
        f = [THETA ** (-axis[:j].count(a) / axes[a]) for j, a in enumerate(axis)]
    else:
        f = [THETA ** (-j / pairs) for j in range(pairs)]
    return torch.tensor(f, dtype=torch.float64, device="cuda"), torch.tensor(axis, device="cuda")


def _rotated(x, pos, s):
    """x [n, heads, d] with the first `rot` values of each head turned by its row's positions [axes, n], in fp32."""
    c = s["c"]
    turn = pos.double()[s["axis"]].T * s["freq"]
    cos, sin = (t.float()[:, None] for t in (turn.cos(), turn.sin()))
    x = x.float()
    y, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["layout"] == "half":
        a, b = y.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)


def _plain_append(s):
    c, rows = s["c"], s["rows"]
    req = torch.repeat_interleave(torch.arange(c["requests"], device="cuda"), s["ext"].long(), output_size=rows)
    first = s["ext"].cumsum(0) - s["ext"]
    at = s["pre"][req] + torch.arange(rows, device="cuda") - first[req]
    slots, pos = s["table"][req, at].long(), s["pos"][:, :rows]
    s["q_out"][:rows] = _rotated(s["q"][:rows], pos, s).to(s["q_out"].dtype)
    k = _rotated(s["k"][:rows], pos, s).to(s["k"].dtype)
    for pool, x, scale in ((s["kp"], k, K_SCALE), (s["vp"], s["v"][:rows], V_SCALE)):
        if c["pool"] == "fp4":
            _fp4_put(pool, slots, x.float(), scale, s["cols"])
        elif c["pool"] == "fp8":
            by = torch.full((), scale, device=pool.device)
            pool[slots] = (x.float() / by).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool[slots] = x


def _plain_run(s):
    op = s["c"]["op"]
    if op == "weights":
        _plain_weights(s)
    elif op == "evict":
        _plain_evict(s)
    elif op == "append":
        _plain_append(s)
    else:
        s["q_out"].copy_(_rotated(s["q"], s["pos"], s))
        s["k_out"].copy_(_rotated(s["k"], s["pos"], s))


def _pool_values(s):
    """The appended pools as values. A 4-bit pool's codes and scales: the rows of the new tokens (the others are as
    prepare made them), unpacked by a table of the 256 code pairs."""
    c = s["c"]
    if c["pool"] == "fp8":
        return [s[p].view(torch.float8_e4m3fn) for p in ("kp", "vp")]
    if c["pool"] != "fp4":
        return [s["kp"], s["vp"]]
    if "pair_values" not in s:
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        b = torch.arange(256, device="cuda")
        s["pair_values"] = (v[b & 15].to(torch.int16) | (v[b >> 4].to(torch.int16) << 8))
    rows = torch.stack((s["kp"], s["vp"]))[:, s["new_slots"]]
    codes = s["pair_values"][rows[:, :, s["cols"][0]].int()].view(torch.float8_e4m3fn)
    return [codes, rows[:, :, s["cols"][1]].view(torch.float8_e4m3fn)]


def run(state):
    if own:
        _own_run(state)
    else:
        _plain_run(state)
    op = state["c"]["op"]
    if op == "weights":
        return [state["out"]]
    if op == "evict":
        names = ["table_out", "scores_out", "lens_out", "evicted", "count", "positions_out"]
        return [state[x] for x in names if x in state]
    if op == "rope":
        return [state["q_out"], state["k_out"]]
    return [state["q_out"]] + _pool_values(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in 64 bits, for whole e: the exponent field itself (a power function need not be exact)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(x, bits, low, top):
    """x to the nearest value with `bits` bits after the leading one, exponents from `low` up, ties to even."""
    _, e = torch.frexp(x)
    step = _power((e - 1).clamp(min=low) - bits)
    return ((x / step).round() * step).clamp(-top, top)


def _exact_fp4(x, scale):
    """(E2M1 values, E4M3 scales) of x [..., d] in 64 bits."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    most = b.abs().amax(-1)
    sf = _nearest(most / torch.full_like(most, 6 * scale), 3, -6, 448.0)
    y = torch.where(sf[..., None] > 0, b / (sf * scale).clamp(min=1e-300)[..., None], torch.zeros_like(b))
    return _nearest(y, 1, 0, 6.0).reshape(x.shape), sf


def _e4m3(code):
    """Values of E4M3 codes (whole numbers) in 64 bits, from their bits."""
    e, m = code // 8 % 16, (code % 8).double()
    return torch.where(e > 0, _power(e - 7) * (1 + m / 8), m * 2.0 ** -9) * (1 - 2 * (code // 128)).double()


def _exact_keys(c, rows):
    """Keys of pool rows in 64 bits."""
    hkv, d = c["kv_heads"], c["dim"]
    if c["pool"] in ("f32", "bf16"):
        return rows.double()
    if c["pool"] == "fp8":
        return _e4m3(rows.int()) * K_SCALE
    out, at = [], 0
    for h0 in range(0, hkv, 4):
        n = min(4, hkv - h0)
        code = rows[:, at:at + n * d // 2].int()
        at += n * d // 2
        sf = rows[:, at:at + n * d // 16].int()
        at += n * d // 16
        nib = torch.stack((code % 16, code // 16), -1).reshape(-1, n, d)
        e, m = nib % 8 // 2, (nib % 2).double()
        val = torch.where(e > 0, _power(e - 1) * (1 + m / 2), m / 2) * (1 - 2 * (nib // 8)).double()
        out.append(val * _e4m3(sf).reshape(-1, n, d // 16).repeat_interleave(16, -1))
    return torch.cat(out, 1) * K_SCALE


def _exact_weights(c, s):
    old, new = _lengths(c)
    out = s["out"].double()
    at = 0
    for r in range(c["requests"]):
        length = int(old[r] + new[r])
        n = int(new[r]) if c["hi"] else 1
        q, lse = s["q"][at:at + n].double(), s["lse"][at:at + n].double()
        at += n
        if not length:
            continue
        ask = min(n, c["window"]) if c["window"] else n
        q, lse = q[n - ask:], lse[n - ask:]
        k = _exact_keys(c, s["kp"][s["table"][r, :length].long()])
        k = k.repeat_interleave(c["heads"] // c["kv_heads"], 1)
        got = torch.zeros(length, dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            w = torch.exp(q[:, h] @ k[:, h].T / math.sqrt(c["dim"]) - lse[:, h, None])
            # the i-th from the end sees all but the i last positions
            got += torch.tril(w, length - ask).sum(0)
        before = int(old[r]) if c["hi"] else length - 1
        got[:before] += s["scores"][r, :before].double() * c["decay"]
        out[r, :length] = got
    return [out]


def _exact_evict(c, s):
    table, scores = s["table"].cpu().numpy(), s["scores"].cpu().numpy()
    old, _ = _lengths(c)
    budget, p = _budgets(c, old), c["page"]
    places = s["positions"].cpu().numpy() if c["positions"] else None
    names = ["table_out", "scores_out", "lens_out", "evicted", "count", "positions_out"]
    out = {x: s[x].cpu().numpy().astype(np.float64) for x in names if x in s}
    for r, n in enumerate(int(x) for x in old):
        keep = np.ones(n, dtype=bool)
        if n > budget[r]:
            pages = [range(a, min(a + p, n)) for a in range(0, n, p)]
            # positions from n - recent on, and the first `sinks` ones, keep their pages
            held = [pg.start < c["sinks"] or pg.stop > n - c["recent"] or len(pg) < p for pg in pages]
            room = (int(budget[r]) - sum(len(pg) for pg, h in zip(pages, held) if h)) // p
            rest = [i for i, h in enumerate(held) if not h]
            best = sorted(rest, key=lambda i: (-scores[r, pages[i].start:pages[i].stop].max(), i))
            for i in best[max(room, 0):]:
                keep[pages[i].start:pages[i].stop] = False
        m = int(keep.sum())
        out["table_out"][r, :m], out["table_out"][r, m:n] = table[r, :n][keep], -1
        out["scores_out"][r, :m], out["scores_out"][r, m:n] = scores[r, :n][keep], 0
        if places is not None:
            out["positions_out"][r, :m], out["positions_out"][r, m:n] = places[r, :n][keep], -1
        out["evicted"][r, :n - m] = table[r, :n][~keep]
        out["lens_out"][r], out["count"][r] = m, n - m
    return [torch.from_numpy(out[x]).cuda() for x in names if x in out]


def _exact_rotate(c, x, pos):
    """x [n, heads, d], pos [axes, n]."""
    axes, pairs = np.array(_axes(c)), c["rot"] // 2
    j = np.arange(pairs)
    if c["arrange"] == "blocks":
        axis = np.repeat(np.arange(len(axes)), axes)
        index = j - (np.cumsum(axes) - axes)[axis]
    else:
        # pair i of axis a stands behind the pairs of rounds before and those of its own round's earlier axes
        place = [(i, a) for i in range(int(axes.max())) for a in range(len(axes)) if i < axes[a]]
        index, axis = (np.array(v) for v in zip(*place))
    power = index / axes[axis] if c["ladder"] == "own" else j / pairs
    t = pos.cpu().numpy().astype(np.float64)[axis].T * np.power(THETA, -power)
    cos, sin = (torch.from_numpy(f(t)).cuda()[:, None, :] for f in (np.cos, np.sin))
    y = x.double().clone()
    one = slice(0, pairs) if c["layout"] == "half" else slice(0, 2 * pairs, 2)
    two = slice(pairs, 2 * pairs) if c["layout"] == "half" else slice(1, 2 * pairs, 2)
    a, b = x.double()[..., one], x.double()[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = a * sin + b * cos
    return y


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "weights":
        return _exact_weights(c, s)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    if c["op"] == "rope":
        return [_exact_rotate(c, s["q"], s["pos"]), _exact_rotate(c, s["k"], s["pos"])]
    n, to = s["rows"], s["new_slots"]
    q = s["q_out"].double()
    q[:n] = _exact_rotate(c, s["q"][:n], s["pos"][:, :n])
    k, v = _exact_rotate(c, s["k"][:n], s["pos"][:, :n]), s["v"][:n].double()
    if c["pool"] in ("f32", "bf16"):
        kp, vp = s["kp"].double(), s["vp"].double()
        kp[to], vp[to] = k, v
        return [q, kp, vp]
    # a quantised pool holds codes of the key as a bf16 tensor would hold it
    k = _nearest(k, 7, -126, 3.4e38)
    if c["pool"] == "fp8":
        pools = [s[p].view(torch.float8_e4m3fn).double() for p in ("kp", "vp")]
        pools[0][to] = _nearest(k / torch.full_like(k, K_SCALE), 3, -6, 448.0)
        pools[1][to] = _nearest(v / torch.full_like(v, V_SCALE), 3, -6, 448.0)
        return [q] + pools
    pairs = [_exact_fp4(k, K_SCALE), _exact_fp4(v, V_SCALE)]
    return [q, torch.stack([x[0] for x in pairs]), torch.stack([x[1] for x in pairs])]
