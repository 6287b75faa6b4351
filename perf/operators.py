"""Cases and plain forms of the operators that fill and read a 4-bit KV cache:

  decode   one query token per request over a paged cache held in 4 bits
           (E2M1 codes, one E4M3 scale for 16 values, one scale per tensor)
  extend   new tokens over such a cache (chunked prefill), causal in the new block
  append   new keys and values into the paged cache (fp32, bf16, E4M3 or 4-bit
           pools), the keys and queries rotated on the way
  step     a decode step: append, then decode
  rope     rotary positions of queries and keys

With `own` false, `run` computes an operator in elementary torch operations;
with `own` true it makes the library's calls.
"""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _decode(name, requests, prefix, lo, hi, heads, kv_heads, dim, page, empty, lens):
    return {"name": name, "op": "decode", "requests": requests, "prefix": prefix, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "empty": empty, "lens": lens}


def _extend(name, requests, plo, phi, lo, hi, heads, kv_heads, dim, lens):
    return {"name": name, "op": "extend", "requests": requests, "plo": plo, "phi": phi, "lo": lo, "hi": hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "lens": lens}


def _append(name, pool, requests, plo, phi, lo, hi, heads, kv_heads, dim, rot, layout, scaling, pad, lens):
    return {"name": name, "op": "append", "pool": pool, "requests": requests, "plo": plo, "phi": phi, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "layout": layout,
            "scaling": scaling, "pad": pad, "lens": lens}


def _step(name, requests, lo, hi, heads, kv_heads, dim, lens):
    return {"name": name, "op": "step", "requests": requests, "prefix": 0, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": 16, "empty": False, "lens": lens, "pool": "fp4", "rot": dim,
            "layout": "half", "scaling": "none"}


def _rope(name, rows, heads, kv_heads, dim, rot, layout, scaling, far):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "layout": layout, "scaling": scaling, "far": far}


def listed():
    return [
        # one user at the start of a conversation: nothing but latency
        _decode("decode one request", 1, 0, 180, 180, 32, 8, 128, 1, False, 1),
        # a batch that shares a system prompt, each request with its own suffix
        _decode("decode shared prompt", 64, 2048, 64, 512, 32, 8, 128, 1, False, 2),
        # long contexts of very different lengths in pages of 16, one request without context yet
        _decode("decode long ragged", 64, 0, 1, 8192, 32, 8, 128, 16, True, 3),
        # two KV heads of width 64 with eight query heads each, an odd batch
        _decode("decode narrow heads", 33, 0, 17, 1500, 16, 2, 64, 1, False, 4),
        # a decode step of a serving loop: rotate, quantise into the pages, attend
        _step("decode step", 48, 100, 2000, 32, 8, 128, 5),
        # short chunks behind short prefixes, one to two hundred tokens each
        _extend("extend short chunks", 3, 0, 300, 1, 200, 64, 8, 128, 6),
        # chunked prefill: 512 new tokens behind 4096 cached ones for each request
        _extend("extend cached prefixes", 8, 4096, 4096, 512, 512, 64, 8, 128, 7),
        # the append of a decode step into a bf16 cache
        _append("append a token each", "bf16", 64, 64, 4000, 1, 1, 32, 8, 128, 128, "half", "none", 0, 8),
        # a prefill of long prompts quantised into a 4-bit cache
        _append("append prompts in 4 bits", "fp4", 4, 0, 0, 2048, 2048, 32, 8, 128, 128, "half", "banded", 0, 9),
        # ragged chunks at far positions into an E4M3 cache, half of each head rotated in
        # neighbouring pairs, in a batch padded to its bucket
        _append("append far chunks in 8 bits", "fp8", 7, 100000, 130000, 1, 300, 16, 4, 128, 64, "pairs", "ramp", 23, 10),
        # a decode batch's queries and keys out of one fused projection
        _rope("rope a decode batch", 64, 32, 8, 128, 128, "half", "none", 4000),
        # a prefill's queries and keys at far positions
        _rope("rope a long prefill", 16384, 64, 8, 128, 128, "half", "banded", 131072),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "extend", "append", "append", "step", "rope"])
    kv_heads, group = rng.choice([(8, 4), (8, 8), (4, 4), (2, 8), (8, 1), (5, 2), (1, 8)])
    dim = rng.choice([64, 128])
    heads = kv_heads * group
    lens = rng.randrange(1, 1 << 20)
    if op == "decode":
        n = _between(rng, 1, 64)
        hi = min(_between(rng, 32, 8192), 250000 // n)
        prefix = rng.choice([0, 0, _between(rng, 16, 2048)])
        c = _decode("", n, prefix, rng.randrange(1, hi + 1), hi, heads, kv_heads, dim, rng.choice([1, 1, 16]),
                    rng.random() < 0.3 and n > 1, lens)
    elif op == "step":
        hi = _between(rng, 32, 4000)
        c = _step("", _between(rng, 1, 64), rng.randrange(1, hi + 1), hi, heads, kv_heads, dim, lens)
    elif op == "extend":
        n, hi, phi = _between(rng, 1, 8), _between(rng, 1, 512), _between(rng, 1, 4096)
        c = _extend("", n, rng.choice([0, phi]), phi, rng.randrange(1, hi + 1), hi, heads, kv_heads, dim, lens)
    elif op == "append":
        n, hi = _between(rng, 1, 64), _between(rng, 1, 120)
        far = rng.choice([0, 1000, 120000])
        c = _append("", rng.choice(["f32", "bf16", "fp8", "fp4"]), n, 0, far, rng.randrange(1, hi + 1), hi, heads,
                    kv_heads, dim, rng.choice([dim, dim // 2, 16]), rng.choice(["half", "pairs"]),
                    rng.choice(["none", "linear", "base", "ramp", "banded"]), rng.randrange(0, 40), lens)
    else:
        c = _rope("", _between(rng, 1, 8192), heads, kv_heads, dim, rng.choice([dim, dim // 2, 16]),
                  rng.choice(["half", "pairs"]), rng.choice(["none", "linear", "base", "ramp", "banded"]),
                  rng.choice([100, 131072, 1000000]))
    del c["name"]
    return c


def _lengths(c):
    """(cached, new) tokens of each request: decode's whole context counts as cached."""
    rng = np.random.default_rng(c["lens"])
    n = c["requests"]
    new = rng.integers(c["lo"], c["hi"] + 1, size=n)
    if c["op"] in ("decode", "step"):
        if c["empty"]:
            new[n // 2] = 0
        return np.where(new > 0, new + c["prefix"], 0) if c["op"] == "decode" else new, new
    return rng.integers(c["plo"], c["phi"] + 1, size=n), new


def _row_bytes(kv_heads, dim):
    return (kv_heads * (dim // 2 + dim // 16) + 15) // 16 * 16


def work(c):
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "rope":
        return {"bytes": c["rows"] * ((hq + hkv) * d * 2 * 2 + 4), "flops": c["rows"] * (hq + hkv) * c["rot"] * 3}
    old, new = _lengths(c)
    row = 2 * _row_bytes(hkv, d)
    if c["op"] == "decode":
        read = int((old - np.where(old > 0, c["prefix"], 0)).sum()) + (c["prefix"] if old.max() > 0 else 0)
        return {"bytes": read * (row + 4) + c["requests"] * hq * (4 * d + 4), "flops": 4 * d * hq * int(old.sum())}
    if c["op"] == "step":
        n = c["requests"]
        return {"bytes": int(old.sum()) * (row + 4) + n * (hq * (4 * d + 4) + hq * d * 2 + hkv * d * 4),
                "flops": 4 * d * hq * int(old.sum())}
    if c["op"] == "extend":
        pairs = int((new * old + new * (new + 1) // 2).sum())
        return {"bytes": int((old + new).sum()) * (row + 4) + int(new.sum()) * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    es = 4 if c["pool"] == "f32" else 2
    n = int(new.sum())
    put = {"f32": 8 * hkv * d, "bf16": 4 * hkv * d, "fp8": 2 * hkv * d, "fp4": row}[c["pool"]]
    return {"bytes": n * (2 * hq * d * es + 2 * hkv * d * es + put + 4), "flops": n * (hq + hkv) * c["rot"] * 3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
SCALINGS = {"none": {}, "linear": {"factor": 4.0}, "base": {"factor": 8.0},
            "ramp": {"factor": 16.0, "original": 8192, "low": 1.0, "high": 32.0},
            "banded": {"factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0}}
THETA = 500000.0


def _columns(kv_heads, dim, device):
    """Columns of a 4-bit row: each head's code bytes and scale bytes. Heads are kept in blocks of four, a block's
    codes before its scales."""
    start = [(h // 4) * 4 * (dim // 2 + dim // 16) for h in range(kv_heads)]
    heads = [min(4, kv_heads - h // 4 * 4) for h in range(kv_heads)]
    codes = [[s + (h % 4) * (dim // 2) + i for i in range(dim // 2)] for h, s in enumerate(start)]
    scales = [[s + n * (dim // 2) + (h % 4) * (dim // 16) + i for i in range(dim // 16)]
              for h, (s, n) in enumerate(zip(start, heads))]
    return torch.tensor(codes, device=device), torch.tensor(scales, device=device)


def _fp4_codes(x, scale):
    """(codes, E4M3 scales) of x [..., d] (fp32 values): per 16 values the scale nearest to their largest
    magnitude over 6, then the nearest E2M1 values, ties to even. (Keys are bf16 values, so that exact ties are
    common: the divisors are tensors, because a division by a number multiplies by its rounded reciprocal.)"""
    b = x.reshape(*x.shape[:-1], -1, 16)
    sf = (b.abs().amax(-1) / torch.full((), 6.0 * scale, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = (sf.float() * scale)[..., None]
    y = torch.where(f > 0, b / f, b * 0.0)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * torch.signbit(y).int()
    return code.to(torch.uint8).reshape(x.shape), sf


def _fp4_put(pool, slots, x, scale, cols):
    """x [n, kv_heads, d] quantised into the rows `slots` of a 4-bit pool."""
    code, sf = _fp4_codes(x, scale)
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


def _table(c, total, seed):
    """req_to_token [requests, ld] (-1 past a row's end) for lengths `total`, and the pool's slots: pages in a random
    order, the shared prefix (if any) once."""
    page = c.get("page", 1)
    prefix = c.get("prefix", 0)
    own_len = np.where(total > 0, total - prefix, 0)
    pages = [-(-int(n) // page) for n in own_len]
    shared = -(-prefix // page) if prefix and total.max() > 0 else 0
    need = sum(pages) + shared
    slots = -(-max(64, need + need // 4) // page) * page if page > 1 else max(64, need + need // 4)
    if page > 1:
        slots = max(64, need + need // 4) * page
    order = np.random.default_rng([seed, 1]).permutation(slots // page)
    spread = (order[:, None] * page + np.arange(page)[None, :]).reshape(-1).astype(np.int32)
    table = np.full((c["requests"], max(1, int(total.max()))), -1, dtype=np.int32)
    at = shared * page
    for r, n in enumerate(total):
        if n:
            table[r, :prefix] = spread[:prefix]
            table[r, prefix:n] = spread[at:at + int(n) - prefix]
            at += pages[r] * page
    return table, slots


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    s = {"c": c, "sm": 1.0 / math.sqrt(d)}
    if "rot" in c:
        s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
        s["att"] = 0.1 * math.log(SCALINGS["ramp"]["factor"]) + 1.0 if c["scaling"] == "ramp" else 1.0
    if c["op"] == "rope":
        # q and k as a fused projection leaves them: columns of one matrix
        qkv = _normal(g, c["rows"], (hq + 2 * hkv) * d, dtype=torch.bfloat16)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["pos"] = torch.randint(0, c["far"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty(c["rows"], hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(c["rows"], hkv, d, dtype=torch.bfloat16, device="cuda")
        if own:
            s["rope"] = _own_rope(c)
        return s
    old, new = _lengths(c)
    if c["op"] in ("decode", "step"):
        total = old
    elif c["op"] == "extend":
        total = old + new
    else:
        # an append touches only the new tokens' slots: the prefix is a position, not rows of a pool
        total = old + new
    s["cols"] = _columns(hkv, d, "cuda")
    s["k_scale"], s["v_scale"] = 0.75, 1.25
    es = torch.float32 if c.get("pool") == "f32" else torch.bfloat16
    if c["op"] == "append":
        ld = int(total.max())
        n = int(new.sum())
        slots = n + n // 4 + 64
        order = np.random.default_rng([seed, 1]).permutation(slots).astype(np.int32)
        table = np.full((c["requests"], ld), -1, dtype=np.int32)
        ends = np.cumsum(new)
        for r in range(c["requests"]):
            table[r, old[r]:total[r]] = order[ends[r] - new[r]:ends[r]]
        s["new_slots"] = torch.from_numpy(order[:n].astype(np.int64)).cuda()
    else:
        table, slots = _table(c, total, seed)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy(total.astype(np.int32)).cuda()
    s["pre"] = torch.from_numpy(old.astype(np.int32)).cuda()
    s["ext"] = torch.from_numpy(new.astype(np.int32)).cuda()
    if c["op"] == "append":
        n = int(new.sum()) + c["pad"]
        if c["pool"] == "fp4":
            s["kp"], s["vp"] = (torch.zeros(slots, _row_bytes(hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv")
        elif c["pool"] == "fp8":
            s["kp"], s["vp"] = (_normal(g, slots, hkv, d).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
        else:
            s["kp"], s["vp"] = (_normal(g, slots, hkv, d, dtype=es) for _ in "kv")
    else:
        s["kp"], s["vp"] = (torch.zeros(slots, _row_bytes(hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv")
        for pool, scale in ((s["kp"], s["k_scale"]), (s["vp"], s["v_scale"])):
            for a in range(0, slots, 1 << 16):
                b = min(slots, a + (1 << 16))
                _fp4_put(pool, torch.arange(a, b, device="cuda"), _normal(g, b - a, hkv, d, dtype=torch.bfloat16).float(),
                         scale, s["cols"])
        n = c["requests"] if c["op"] in ("decode", "step") else int(new.sum())
    s["q"] = _normal(g, n, hq, d, dtype=es)
    if c["op"] in ("append", "step"):
        s["k"], s["v"] = _normal(g, n, hkv, d, dtype=es), _normal(g, n, hkv, d, dtype=es)
        s["q_out"] = torch.zeros_like(s["q"])
    if c["op"] != "append":
        s["o"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(n, hq, dtype=torch.float32, device="cuda")
    s["rows"] = int(new.sum())
    s["most"] = int(new.max())
    if own:
        _own_prepare(s, table, total, old, new, slots)
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_rope(c):
    import radixattention_prefix_shared_radix_gb300 as sgl
    kind = {"none": sgl.SGL_ROPE_SCALE_NONE, "linear": sgl.SGL_ROPE_SCALE_LINEAR, "base": sgl.SGL_ROPE_SCALE_NTK,
            "ramp": sgl.SGL_ROPE_SCALE_YARN, "banded": sgl.SGL_ROPE_SCALE_BANDED}[c["scaling"]]
    p = SCALINGS[c["scaling"]]
    return sgl.sgl_rope_create(c["dim"], rot_dim=c["rot"], theta=THETA,
                               layout=sgl.SGL_ROPE_HALF if c["layout"] == "half" else sgl.SGL_ROPE_PAIRS, scaling=kind,
                               factor=p.get("factor", 1.0), original_positions=p.get("original", 0),
                               low=p.get("low", 0.0), high=p.get("high", 0.0))


def _own_prepare(s, table, total, old, new, slots):
    import radixattention_prefix_shared_radix_gb300 as sgl
    c = s["c"]
    kind = {"f32": sgl.SGL_DTYPE_F32, "bf16": sgl.SGL_DTYPE_BF16, "fp8": sgl.SGL_DTYPE_BF16_FP8KV,
            "fp4": sgl.SGL_DTYPE_BF16_FP4KV}[c.get("pool", "fp4")]
    s["params"] = sgl.make_params(kind, c["requests"], c["heads"], c["kv_heads"], c["dim"], slots, c.get("page", 1),
                                  host_prefix_lens=old, host_extend_lens=new, k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
    if "rot" in c:
        s["rope"] = _own_rope(c)
    if c["op"] in ("decode", "step"):
        groups = sgl.sgl_groups_create()
        sgl.sgl_groups_from_table(table, total, groups)
        s["plan"] = sgl.sgl_decode_plan(s["params"], total, sgl.sgl_groups_view(groups))
        sgl.sgl_groups_destroy(groups)
        s["ws"] = torch.zeros(max(256, s["plan"].workspace_bytes), dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(s["plan"], s["ws"])
    else:
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


def _own_run(s):
    import radixattention_prefix_shared_radix_gb300 as sgl
    c = s["c"]
    if c["op"] == "rope":
        sgl.sgl_rope(s["rope"], s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
    elif c["op"] == "append":
        sgl.sgl_kv_append(s["rope"], s["params"], s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["pre"],
                          s["ext"], s["q_out"], s["ws"])
    elif c["op"] == "extend":
        sgl.sgl_extend_attn(s["q"], s["kp"], s["vp"], s["table"], s["pre"], s["ext"], s["params"], s["o"], s["lse"],
                            s["ws"])
    else:
        q = s["q"]
        if c["op"] == "step":
            q = s["q_out"]
            sgl.sgl_kv_append(s["rope"], s["params"], s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"],
                              None, q, s["ws"])
        sgl.sgl_decode_attn(q, s["kp"], s["vp"], s["table"], s["lens"], s["plan"], s["o"], s["lse"], s["ws"])


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _frequencies(c):
    """Radians per position of each pair."""
    n, p = c["rot"], SCALINGS[c["scaling"]]
    theta, by = THETA, p.get("factor", 1.0)
    if c["scaling"] == "base":
        theta = theta * by ** (n / (n - 2)) if n > 2 else theta
    f = [theta ** (-2.0 * j / n) for j in range(n // 2)]
    if c["scaling"] == "linear":
        return [x / by for x in f]
    if c["scaling"] == "ramp":
        at = [n * math.log(p["original"] / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (p["high"], p["low"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        hi = hi if hi > lo else lo + 0.001
        w = [min(max((j - lo) / (hi - lo), 0.0), 1.0) for j in range(n // 2)]
        return [x / by * a + x * (1 - a) for x, a in zip(f, w)]
    if c["scaling"] == "banded":
        turns = [p["original"] * x / (2 * math.pi) for x in f]
        w = [min(max((t - p["low"]) / (p["high"] - p["low"]), 0.0), 1.0) for t in turns]
        return [x / by * (1 - a) + x * a for x, a in zip(f, w)]
    return f


def _rotated(x, pos, s):
    """x [n, heads, d] with the first `rot` values of each head turned by its row's position, in fp32."""
    c = s["c"]
    turn = pos.double()[:, None] * s["freq"]
    cos, sin = ((t * s["att"]).float()[:, None] for t in (turn.cos(), turn.sin()))
    x = x.float()
    y, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["layout"] == "half":
        a, b = y.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)


def _put(s, slots, pos, rows):
    """Rotates the first `rows` rows of q and k, stores k and v into the pools' rows `slots`."""
    c = s["c"]
    s["q_out"][:rows] = _rotated(s["q"][:rows], pos, s).to(s["q_out"].dtype)
    k = _rotated(s["k"][:rows], pos, s).to(s["k"].dtype)
    for pool, x, scale in ((s["kp"], k, s["k_scale"]), (s["vp"], s["v"][:rows], s["v_scale"])):
        if c["pool"] == "fp4":
            _fp4_put(pool, slots, x.float(), scale, s["cols"])
        elif c["pool"] == "fp8":
            by = torch.full((), scale, device=pool.device)
            pool[slots] = (x.float() / by).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool[slots] = x


def _attend(q, k, v, seen, sm):
    """q [b, hq, n, d], k and v [b, L, hkv, d], seen [b, n, L]: (o [b, n, hq, d] bf16, lse [b, n, hq])."""
    b, hq, n, d = q.shape
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    hkv = k.shape[1]
    w = (q.float().reshape(b, hkv, hq // hkv * n, d) @ k.transpose(-1, -2)).reshape(b, hq, n, -1) * sm
    w = w.masked_fill(~seen[:, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = (w - top.clamp(min=-3e38)).exp()
    total = w.sum(-1, keepdim=True)
    o = (w.reshape(b, hkv, -1, w.shape[-1]) @ v).reshape(b, hq, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.transpose(1, 2).to(torch.bfloat16), (top + total.log())[..., 0].transpose(1, 2)


def _plain_run(s):
    c = s["c"]
    if c["op"] == "rope":
        s["q_out"].copy_(_rotated(s["q"], s["pos"], s))
        s["k_out"].copy_(_rotated(s["k"], s["pos"], s))
        return
    if c["op"] == "append":
        req = torch.repeat_interleave(torch.arange(c["requests"], device="cuda"), s["ext"].long(), output_size=s["rows"])
        first = s["ext"].cumsum(0) - s["ext"]
        pos = s["pre"][req] + torch.arange(s["rows"], device="cuda") - first[req]
        _put(s, s["table"][req, pos].long(), pos, s["rows"])
        return
    if c["op"] == "step":
        pos = (s["lens"] - 1).long()
        _put(s, s["table"].gather(1, pos[:, None])[:, 0].long(), pos, c["requests"])
    at = s["table"].clamp(min=0).long()
    k = _fp4_values(s["kp"][at], s["cols"]) * s["k_scale"]
    v = _fp4_values(s["vp"][at], s["cols"]) * s["v_scale"]
    where = torch.arange(at.shape[1], device="cuda")
    if c["op"] == "extend":
        # the ragged rows in a rectangle of the longest request's
        i = torch.arange(s["most"], device="cuda")
        first = s["ext"].cumsum(0) - s["ext"]
        there = i[None] < s["ext"][:, None]
        q = s["q"][torch.where(there, first[:, None] + i, 0).long()]
        seen = where <= (s["pre"][:, None] + i)[..., None]
        o, lse = _attend(q.transpose(1, 2), k, v, seen, s["sm"])
        s["o"].copy_(o[there])
        s["lse"].copy_(lse[there])
        return
    q = s["q_out"] if c["op"] == "step" else s["q"]
    o, lse = _attend(q[:, :, None], k, v, (where < s["lens"][:, None])[:, None], s["sm"])
    s["o"].copy_(o[:, 0])
    s["lse"].copy_(lse[:, 0])


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
    c = state["c"]
    if c["op"] == "rope":
        return [state["q_out"], state["k_out"]]
    if c["op"] == "append":
        return [state["q_out"]] + _pool_values(state)
    if c["op"] == "step":
        # the new rows of the 4-bit pools are read by the attention that follows
        return [state["q_out"], state["o"], state["lse"]]
    return [state["o"], state["lse"]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_angles(c, pos):
    """cos and sin [n, rot / 2] in 64 bits (numpy), times the amplitude of the scaling."""
    n, p = c["rot"], SCALINGS[c["scaling"]]
    j = np.arange(n // 2, dtype=np.float64)
    theta = THETA
    if c["scaling"] == "base" and n > 2:
        theta = THETA * np.power(p["factor"], n / (n - 2.0))
    f = np.power(theta, -2.0 * j / n)
    amp = 1.0
    if c["scaling"] == "linear":
        f = f / p["factor"]
    elif c["scaling"] == "ramp":
        lo = max(np.floor(n * np.log(p["original"] / (p["high"] * 2 * np.pi)) / (2 * np.log(theta))), 0.0)
        hi = min(np.ceil(n * np.log(p["original"] / (p["low"] * 2 * np.pi)) / (2 * np.log(theta))), n - 1.0)
        if hi <= lo:
            hi = lo + 0.001
        r = np.clip((j - lo) / (hi - lo), 0, 1)
        f = f * (r / p["factor"] + 1 - r)
        amp = 0.1 * np.log(p["factor"]) + 1.0
    elif c["scaling"] == "banded":
        wave = 2 * np.pi / f
        keep = np.clip((p["original"] / wave - p["low"]) / (p["high"] - p["low"]), 0, 1)
        f = f * (keep + (1 - keep) / p["factor"])
    a = pos.astype(np.float64)[:, None] * f
    return np.cos(a) * amp, np.sin(a) * amp


def _exact_rotate(c, x, pos):
    cos, sin = (torch.from_numpy(t).cuda()[:, None, :] for t in _exact_angles(c, pos))
    y = x.double().clone()
    h = c["rot"] // 2
    one = slice(0, h) if c["layout"] == "half" else slice(0, 2 * h, 2)
    two = slice(h, 2 * h) if c["layout"] == "half" else slice(1, 2 * h, 2)
    a, b = x.double()[..., one], x.double()[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = a * sin + b * cos
    return y


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


def _exact_row(row, kv_heads, dim):
    """Values of 4-bit rows [n, row bytes] as [n, kv_heads, dim] in 64 bits, from the bits of codes and scales."""
    out = []
    at = 0
    for h0 in range(0, kv_heads, 4):
        n = min(4, kv_heads - h0)
        code = row[:, at:at + n * dim // 2].int()
        at += n * dim // 2
        sf = row[:, at:at + n * dim // 16].int()
        at += n * dim // 16
        nib = torch.stack((code % 16, code // 16), -1).reshape(-1, n, dim).double()
        sign, mag = 1 - 2 * (nib >= 8).double(), nib % 8
        e, m = torch.div(mag, 2, rounding_mode="floor"), mag % 2
        val = sign * torch.where(e > 0, _power(e - 1) * (1 + m / 2), m / 2)
        e, m = (sf // 8 % 16).double(), (sf % 8).double()
        scale = torch.where(e > 0, _power(e - 7) * (1 + m / 8), m * 2.0 ** -9) * (1 - 2 * (sf // 128)).double()
        out.append(val * scale.reshape(-1, n, dim // 16).repeat_interleave(16, -1))
    return torch.cat(out, 1)


def _exact_softmax(q, k, v, last, sm):
    """q [n, hq, d], k and v [L, hkv, d] in 64 bits, row i sees positions 0 .. last[i]: (o, lse)."""
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    w = torch.einsum("nhd,lhd->hnl", q, k) * sm
    w[:, torch.arange(k.shape[0], device=w.device)[None, :] > last[:, None]] = -math.inf
    lse = torch.logsumexp(w, -1)
    return torch.einsum("hnl,lhd->nhd", torch.exp(w - lse[..., None]), v), lse.T


def exact(c, seed):
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    if c["op"] == "rope":
        pos = s["pos"].cpu().numpy()
        return [_exact_rotate(c, s["q"], pos), _exact_rotate(c, s["k"], pos)]
    old, new = _lengths(c)
    if c["op"] == "append":
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(old, new)])
        n = len(pos)
        q = s["q_out"].double()
        q[:n] = _exact_rotate(c, s["q"][:n], pos)
        k = _exact_rotate(c, s["k"][:n], pos)
        v = s["v"][:n].double()
        to = s["new_slots"]
        if c["pool"] in ("f32", "bf16"):
            kp, vp = s["kp"].double(), s["vp"].double()
            kp[to], vp[to] = k, v
            return [q, kp, vp]
        # a quantised pool holds codes of the key as a bf16 tensor would hold it
        k = _nearest(k, 7, -126, 3.4e38)
        if c["pool"] == "fp8":
            pools = [s[p].view(torch.float8_e4m3fn).double() for p in ("kp", "vp")]
            pools[0][to] = _nearest(k / torch.full_like(k, s["k_scale"]), 3, -6, 448.0)
            pools[1][to] = _nearest(v / torch.full_like(v, s["v_scale"]), 3, -6, 448.0)
            return [q] + pools
        pairs = [_exact_fp4(k, s["k_scale"]), _exact_fp4(v, s["v_scale"])]
        return [q, torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])]
    q = s["q"].double()
    k_new = v_new = None
    out = []
    if c["op"] == "step":
        pos = old - 1
        q = _exact_rotate(c, s["q"], pos)
        out.append(q)
        q = _nearest(q, 7, -126, 3.4e38)
        k = _nearest(_exact_rotate(c, s["k"], pos), 7, -126, 3.4e38)
        k_new, v_new = ((a * b.repeat_interleave(16, -1)) for a, b in
                        (_exact_fp4(k, s["k_scale"]), _exact_fp4(s["v"].double(), s["v_scale"])))
    o, lse, at = [], [], 0
    for r in range(c["requests"]):
        n = int(new[r]) if c["op"] == "extend" else 1
        length = int(old[r] + new[r]) if c["op"] == "extend" else int(old[r])
        rows = s["table"][r, :length].long()
        if not length:
            o.append(torch.zeros(1, c["heads"], c["dim"], dtype=torch.float64, device="cuda"))
            lse.append(torch.full((1, c["heads"]), -math.inf, dtype=torch.float64, device="cuda"))
            at += n
            continue
        k, v = (_exact_row(p[rows], c["kv_heads"], c["dim"]) for p in (s["kp"], s["vp"]))
        if k_new is not None:
            k[-1], v[-1] = k_new[r], v_new[r]
        last = torch.arange(length - n, length, device="cuda")
        x, y = _exact_softmax(q[at:at + n], k * s["k_scale"], v * s["v_scale"], last, s["sm"])
        o.append(x)
        lse.append(y)
        at += n
    return out + [torch.cat(o), torch.cat(lse)]
