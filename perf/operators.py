"""Measured cases of the paged 8-bit KV cache operators: block tables and slot maps (plan), rotary
positions with several axes (rope), writing new keys and values into the cache (append) and
attention that reads it (attend).

listed() names fixed cases, draw() more of the same ranges; prepare() makes a case's inputs from a
seed, run() is one pass (the plain form where `own` is false, the library's kernels where it is
true), exact() the same outputs in 64 bits from the definition, work() the bytes and operations
that a pass cannot do without.

The cache, as both sides hold it: pages of 64 tokens; per (page, KV head) a K tile and a V tile of
64 x D bytes one after the other, then a section of fp32 scales [page][head][2] (K, V). An int8
code q in -127..127 is stored as the byte q + 128, an e4m3 code as its bits. The V tile is
transposed (byte d * 64 + token). In the K tile the byte of (token, d) is at
((((token % 16) / 2) * (D / 64) + d / 64) * 8 + (token / 16) * 2 + token % 2) * 64 + d % 64.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
TWO_PI = 2.0 * math.pi
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------- cases

def listed():
    heads = {"q_heads": 40, "kv_heads": 8, "dim": 128}   # the INT4 layer set's attention: 40 query, 8 KV heads of 128
    plain = {"kv": "int8", "type": "bf16", "softcap": 0.0, "slopes": False, "window": 0, "prefix": 0}
    return [
        # one decode step of a small server: 64 requests, one token each, some leaving
        {"name": "plan_step", "op": "plan", "requests": 64, "ctx": 16384, "new": 1, "tight": False},
        # admission of many prompts at once with a pool that does not hold them all
        {"name": "plan_prompts", "op": "plan", "requests": 512, "ctx": 2048, "new": 128, "tight": True},
        # one decode token's query and key heads, straight from the fp32 matvec output
        {"name": "rope_token", "op": "rope", "tokens": 1, "heads": 48, "dim": 128, "rot": 128, "axes": 1,
         "interleaved": False, "inverse": False, "type": "f32", "out": "bf16", "span": 32768},
        # a video prompt: time, height and width axes
        {"name": "rope_video", "op": "rope", "tokens": 8192, "heads": 48, "dim": 128, "rot": 128, "axes": 3,
         "interleaved": False, "inverse": False, "type": "bf16", "out": "bf16", "span": 8192},
        # the gradient through an image encoder's two-axis rotation, partial and interleaved, in fp32
        {"name": "rope_image_grad", "op": "rope", "tokens": 4095, "heads": 16, "dim": 64, "rot": 48, "axes": 2,
         "interleaved": True, "inverse": True, "type": "f32", "out": "f32", "span": 64},
        # one decode step of 64 requests: rotate q and k, write k and v
        {"name": "append_step", "op": "append", "requests": 64, "ctx": 4096, "new": 1, "kv": "int8", "type": "f32",
         "axes": 1, **heads},
        # two prompts of 8190 tokens in all, the first of them continuing a cached context
        {"name": "append_prompt", "op": "append", "requests": 2, "ctx": 1000, "new": 4095, "kv": "e4m3", "type": "bf16",
         "axes": 3, **heads},
        # the smallest attention call: one token of one short conversation
        {"name": "attend_one", "op": "attend", "requests": 1, "ctx": 1000, "new": 1, **heads, **plain},
        # verification of four draft tokens over one long document
        {"name": "attend_verify", "op": "attend", "requests": 1, "ctx": 32771, "new": 5, **heads, **plain},
        # a decode step of 64 requests with contexts up to 16384
        {"name": "attend_batch", "op": "attend", "requests": 64, "ctx": 16384, "new": 1, **heads, **plain},
        # a decode step with capped scores, a distance bias and a window, heads of 64, e4m3 codes
        {"name": "attend_capped", "op": "attend", "requests": 24, "ctx": 12000, "new": 2, "q_heads": 32, "kv_heads": 8,
         "dim": 64, "kv": "e4m3", "type": "f16", "softcap": 30.0, "slopes": True, "window": 4096, "prefix": 0},
        # prompt chunks, each over its cached context, with a bidirectional prefix
        {"name": "attend_prompt", "op": "attend", "requests": 3, "ctx": 4096, "new": 1500, **heads, **plain,
         "prefix": 300},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "append", "attend", "attend", "attend", "attend"])
    q_heads, kv_heads = rng.choice([(40, 8), (32, 8), (16, 16), (8, 1), (24, 4), (5, 1), (12, 4), (64, 4)])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice(["int8", "int8", "e4m3"])
    if op == "plan":
        new = rng.choice([1, 1, _logint(rng, 2, 200)])
        return {"op": op, "requests": _logint(rng, 1, min(1500, 65536 // new)), "ctx": _logint(rng, 1, 16384), "new": new,
                "tight": rng.random() < 0.4}
    if op == "rope":
        heads = _logint(rng, 1, 48)
        kind, out = rng.choice([("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f16")])
        axes = rng.randint(1, 4)
        return {"op": op, "tokens": _logint(rng, 1, 8192), "heads": heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, dim - 16]), "axes": axes, "interleaved": rng.random() < 0.4,
                "inverse": rng.random() < 0.3, "type": kind, "out": out, "span": _logint(rng, 16, 131072)}
    if op == "append":
        new = rng.choice([1, rng.randint(2, 16), _logint(rng, 17, 4096)])
        return {"op": op, "requests": _logint(rng, 1, max(1, min(128, 8190 // new))), "ctx": _logint(rng, 1, 4096), "new": new,
                "kv": kv, "type": rng.choice(["f32", "bf16", "f16"]), "axes": rng.randint(1, 3), "q_heads": q_heads,
                "kv_heads": kv_heads, "dim": dim}
    shape = rng.choice(["step", "step", "verify", "prompt"])
    if shape == "prompt":
        new = _logint(rng, 17, 1500)
        ctx = new + _logint(rng, 1, 2500)
        requests = rng.randint(1, 3)
        while requests > 1 and requests * new * ctx * q_heads > 7.0e8:
            requests -= 1
    else:
        new = 1 if shape == "step" else rng.randint(2, 16)
        ctx = max(new, _logint(rng, 1, 16384))
        requests = _logint(rng, 1, max(1, min(64, 500000 // ctx)))
        while requests > 1 and requests * ctx * max(kv_heads, q_heads * new / 64.0) > 4.5e6:
            requests = (requests + 1) // 2
    return {"op": op, "requests": requests, "ctx": ctx, "new": new, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "kv": kv, "type": rng.choice(["bf16", "bf16", "f16"]), "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "slopes": rng.random() < 0.3, "window": rng.choice([0, 0, _logint(rng, 16, 8192)]),
            "prefix": rng.choice([0, 0, _logint(rng, 1, max(1, ctx))])}


# ----------------------------------------------------------------------------- sizes that follow from a case

def _spread(n, lo, hi):
    """n whole numbers spread over lo..hi in no order (golden-ratio steps), the last of them hi."""
    v = [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(c):
    """Per request: cached tokens before the call and new tokens."""
    n = c["requests"]
    if c["op"] == "plan":
        lens = _spread(n, 0 if c["new"] > 1 else 1, c["ctx"])
        add = [c["new"] if c["new"] == 1 else 1 + (i * 7919) % (2 * c["new"] - 1) for i in range(n)]
        if n > 8:
            for i in range(5, n, 16):
                add[i] = -1      # the request has ended: its pages go back
            for i in range(7, n, 16):
                add[i] = 0       # the request waits this step
        return lens, add
    if c["op"] == "append":
        lens = _spread(n, 0, c["ctx"])
        return lens, [c["new"]] * n
    total = _spread(n, max(c["new"], c["ctx"] // 16), c["ctx"])   # context lengths with the new tokens in them
    return [t - c["new"] for t in total], [c["new"]] * n


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _positions(c, g, count):
    """int32 [axes][tokens] positions: a clip of frames, rows and columns, or text positions, from an offset."""
    axes, span = c["axes"], c["span"]
    base = int(torch.randint(0, max(1, span), (1,), generator=g))
    t = torch.arange(count)
    side = max(1, int(round(math.sqrt(min(count, 1024)))))
    rows = [t // (side * side) if axes > 1 else t, (t // side) % side, t % side, t][:axes]
    return torch.stack([(r + base) % max(span, 2) for r in rows]).to(torch.int32)


def _frequencies(c):
    """Inverse frequencies of the rotated pairs, and the axis of each pair (contiguous sections)."""
    pairs = c["rot"] // 2
    inv = [10000.0 ** (-i / pairs) for i in range(pairs)]
    axis = [i * c["axes"] // pairs for i in range(pairs)]
    return inv, axis


def _turns(inv):
    """Turns per position as 64-bit fixed point (2^64 = one turn), in two's complement."""
    out = []
    for f in inv:
        x = f * (1.0 / TWO_PI)
        x -= math.floor(x)
        v = int(x * 18446744073709551616.0) & 0xFFFFFFFFFFFFFFFF
        out.append(v - (1 << 64) if v >> 63 else v)
    return out


# ----------------------------------------------------------------------------- inputs

def _code_bytes(g, n, kv):
    """n bytes of cache codes as normal keys and values leave them."""
    out = torch.empty(n, dtype=torch.uint8, device=DEV)
    for i in range(0, n, 1 << 26):
        m = min(1 << 26, n - i)
        x = torch.randn(m, generator=g, device=DEV)
        if kv == "int8":
            out[i:i + m] = (x * 32).round().clamp(-127, 127).add(128).to(torch.uint8)
        else:
            out[i:i + m] = (x * 110).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _cache(c, seed, g, gc):
    """A paged cache whose requests' pages lie anywhere in the pool, and its block table."""
    lens, add = _lengths(c)
    need = [_pages(a + b) for a, b in zip(lens, add)]
    most = max(need)
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gc, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(need), most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    H, D = c["kv_heads"], c["dim"]
    code_bytes = n_pages * H * 2 * PAGE * D
    scale_off = -(-code_bytes // 256) * 256
    total = -(-(scale_off + n_pages * H * 8) // 256) * 256
    cache = torch.zeros(total, dtype=torch.uint8, device=DEV)
    cache[:code_bytes] = _code_bytes(g, code_bytes, c["kv"])
    step = 0.035 if c["kv"] == "int8" else 0.01
    scales = torch.randn((n_pages, H, 2), generator=g, device=DEV).mul(0.3).exp().mul(step)
    cache[scale_off:scale_off + n_pages * H * 8] = scales.view(torch.uint8).reshape(-1)
    return {"lens": lens, "add": add, "n_pages": n_pages, "table_host": table, "table": table.to(DEV), "cache": cache,
            "code_bytes": code_bytes, "scale_off": scale_off}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed * 2 + 1)
    gc = torch.Generator().manual_seed(seed * 2 + 2)
    s = {"case": c}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if c["op"] == "plan":
        lens, add = _lengths(c)
        n = len(lens)
        cap = _pages(max(a + max(b, 0) for a, b in zip(lens, add))) + 1
        held = [_pages(v) for v in lens]
        want = sum(_pages(a + max(b, 0)) - h for a, b, h in zip(lens, add, held))
        n_pages = sum(held) + want + 7
        free = n_pages - sum(held) if not c["tight"] else max(0, want * 2 // 3)
        order = torch.randperm(n_pages, generator=gc, dtype=torch.int64).to(torch.int32)
        table = torch.full((n, cap), -1, dtype=torch.int32)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        head = int(torch.randint(0, n_pages, (1,), generator=gc))
        ring = torch.full((n_pages,), -1, dtype=torch.int32)
        ring[(torch.arange(free) + head) % n_pages] = order[at:at + free]
        T = sum(max(a, 0) for a in add)
        s |= {"lens": i32(lens), "add": i32(add), "table": table.to(DEV), "ring": ring.to(DEV),
              "ring_state": i32([head, free]), "n_tokens": T, "n_pages": n_pages}
        if own:
            import quantized_gemv_unpack_gb300 as q
            s["call"] = q.KvPlan(s["lens"], s["add"], s["table"], s["ring"], s["ring_state"], T)
        return s
    if c["op"] == "rope":
        inv, axis = _frequencies(c)
        s["x"] = torch.randn((c["tokens"], c["heads"], c["dim"]), generator=g, device=DEV).to(TYPES[c["type"]])
        s["positions"] = _positions(c, gc, c["tokens"]).to(DEV)
        s |= {"inv": inv, "axis": torch.tensor(axis, device=DEV), "turns": torch.tensor(_turns(inv), dtype=torch.int64, device=DEV)}
        if own:
            import quantized_gemv_unpack_gb300 as q
            s["out"] = torch.empty_like(s["x"], dtype=TYPES[c["out"]])
            s["call"] = q.Rope(q.rope_desc(c["dim"], inv, axis=axis, interleaved=c["interleaved"]), s["x"], s["positions"],
                               s["out"], inverse=c["inverse"])
        return s

    s |= _cache(c, seed, g, gc)
    H, Hq, D = c["kv_heads"], c["q_heads"], c["dim"]
    lens, add = s["lens"], s["add"]
    T = sum(add)
    start = [0]
    for a in add:
        start.append(start[-1] + a)
    s["q_start"] = i32(start)
    s["ctx"] = i32([a + b for a, b in zip(lens, add)])
    kind = TYPES[c["type"]]
    if c["op"] == "append":
        # slots of the new tokens, the runs of tokens that share a page, and every filled slot of the pages touched
        slots, runs, read, pos = [], [], [], []
        for b, (l, a) in enumerate(zip(lens, add)):
            pos += list(range(l, l + a))
            row = s["table_host"][b].tolist()
            slots += [row[p // PAGE] * PAGE + p % PAGE for p in range(l, l + a)]
            p = l
            while p < l + a:
                n = min(PAGE - p % PAGE, l + a - p)
                runs.append((start[b] + p - l, n))
                read += [row[p // PAGE] * PAGE + o for o in range(p % PAGE + n)]
                p += n
        c2 = dict(c, rot=D, span=max(pos) + 1)
        inv, axis = _frequencies(c2)
        # a qkv row as the projections leave it: query heads, key heads, value heads; a few key channels larger
        qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device=DEV)
        qkv[:, Hq:Hq + H, ::37] *= 6.0
        s["qkv"] = qkv.to(kind)
        if c["axes"] == 1:
            s["positions"] = i32(pos).reshape(1, -1)
        else:
            s["positions"] = _positions(c2, gc, T).to(DEV)
        s |= {"slots": i32(slots), "runs": i32(runs), "read": i32(read), "inv": inv, "axis": torch.tensor(axis, device=DEV),
              "turns": torch.tensor(_turns(inv), dtype=torch.int64, device=DEV)}
        if own:
            import quantized_gemv_unpack_gb300 as q
            desc = q.kv8_desc(q.QMV_KV_INT8 if c["kv"] == "int8" else q.QMV_KV_E4M3, s["n_pages"], H, D)
            s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
            s["k_out"], s["v_out"] = (torch.empty((len(read), H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            x = s["qkv"]
            s["call"] = q.KvAppend(desc, s["cache"], x[:, Hq:Hq + H], x[:, Hq + H:], s["slots"], s["runs"],
                                   rope=q.rope_desc(D, inv, axis=axis), positions=s["positions"], q=x[:, :Hq], q_out=s["q_out"])
            s["read_call"] = q.KvRead(desc, s["cache"], s["read"], s["k_out"], s["v_out"])
        return s

    s["q"] = (torch.randn((T, Hq, D), generator=g, device=DEV) * 1.5).to(kind)
    s["scale"] = 1.0 / math.sqrt(D)
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=DEV) if c["slopes"] else None
    s["prefix"] = i32([min(c["prefix"], a + b) for a, b in zip(lens, add)]) if c["prefix"] else None
    if own:
        import quantized_gemv_unpack_gb300 as q
        desc = q.kv8_desc(q.QMV_KV_INT8 if c["kv"] == "int8" else q.QMV_KV_E4M3, s["n_pages"], H, D)
        s["out"] = torch.empty_like(s["q"])
        s["call"] = q.KvAttend(desc, s["cache"], s["q"], s["out"], s["q_start"], s["ctx"], s["table"], s["scale"],
                               max_new=c["new"], softcap=c["softcap"], slopes=s["slopes"], window=c["window"], prefix=s["prefix"])
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plan_plain, "rope": _rope_plain, "append": _append_plain, "attend": _attend_plain}[op](s)
    s["call"].run()
    if op == "plan":
        p = s["call"]
        return {"lens": p.lens_out, "ctx": p.ctx, "status": p.status, "q_start": p.q_start, "slots": p.slots,
                "positions": p.positions, "runs": p.runs, "ring_state": p.ring_state_out, "table": s["table"], "ring": s["ring"]}
    if op == "append":
        s["read_call"].run()
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    return {"out": s["out"]}


def _plan_plain(s):
    lens, add, table, ring = s["lens"].long(), s["add"].long(), s["table"], s["ring"]
    n, cap, N, T = len(lens), table.shape[1], s["n_pages"], s["n_tokens"]
    head, count = s["ring_state"].long()
    dev = lens.device
    tok = add.clamp(min=0)
    ends = tok.cumsum(0)
    starts = ends - tok
    held = (lens + 63) // 64
    after = (lens + tok + 63) // 64
    bad = (lens < 0) | (held > cap) | (after > cap) | (ends > T)
    need = torch.where(bad | (add < 0), 0, after - held)
    upto = need.cumsum(0)
    first = upto - need
    short = ~bad & (need > 0) & (upto > count)
    leaves = ~bad & (add < 0)
    given = ~bad & ~short & ~leaves
    status = torch.where(bad, 2, torch.where(short, 1, torch.where(leaves, 3, 0)))
    popped = torch.where(given, need, 0).sum()
    # pages that come back: in the order of requests, then of the table
    back = torch.where(leaves, held, 0)
    col = torch.arange(cap, device=dev)
    gone = table.long()[col[None, :] < back[:, None]]
    ring_out = ring.clone()
    ring_out[(head + count + torch.arange(len(gone), device=dev)) % N] = gone.int()
    # new table entries
    fresh = given[:, None] & (col[None, :] >= held[:, None]) & (col[None, :] < after[:, None])
    at = (head + first[:, None] + col[None, :] - held[:, None]) % N
    table_out = torch.where(fresh, ring[at], table)
    # tokens
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(ends, t, right=True)
    inside = b < n
    b = b.clamp(max=n - 1)
    inside &= given[b]
    pos = lens[b] + t - starts[b]
    page = table_out[b, (pos // 64).clamp(0, cap - 1)].long()
    slots = torch.where(inside, page * 64 + pos % 64, -1)
    positions = torch.where(inside, pos, -1)
    # runs of tokens that share a page
    first_of = inside & ((pos % 64 == 0) | (t == starts[b]))
    count_of = torch.minimum(64 - pos % 64, ends[b] - t)
    most = min(T, T // 64 + 2 * min(n, T))
    rank = first_of.long().cumsum(0) - 1
    runs = torch.zeros((most + 1, 2), dtype=torch.int64, device=dev)
    where = torch.where(first_of, rank, most)
    runs[where] = torch.stack([t, count_of], 1)
    runs = runs[:most]
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), ends]).clamp(max=T)
    state = torch.stack([(head + popped) % N, count - popped + len(gone)])
    lens_out = torch.where(given, lens + tok, torch.where(leaves, 0, lens))
    ctx = torch.where(given, lens + tok, 0)
    out = {"lens": lens_out, "ctx": ctx, "status": status, "q_start": q_start, "slots": slots, "positions": positions,
           "runs": runs, "ring_state": state, "table": table_out, "ring": ring_out}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _angles(positions, axis, turns):
    """fp32 cosine and sine [tokens][pairs] of the pairs' angles: the fraction of a turn is exact."""
    pos = positions.long()[axis].T                       # [tokens][pairs]
    half_turns = ((pos * turns) >> 32).float() * (2.0 ** -31)
    angle = half_turns * math.pi
    return torch.cos(angle), torch.sin(angle)


def _rotate(x, cos, sin, interleaved):
    """x: fp32 [tokens][heads][D]; the first 2 * pairs values rotated."""
    pairs = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * pairs:]], -1)


def _rope_plain(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], s["axis"], s["turns"])
    if c["inverse"]:
        sin = -sin
    return {"out": _rotate(s["x"].float(), cos, sin, c["interleaved"]).to(TYPES[c["out"]])}


def _tiles(s, pages):
    """Codes (fp32, K and V each [.., head, token, d]) and scales [.., head, 2] of cache pages."""
    c = s["case"]
    H, D = c["kv_heads"], c["dim"]
    codes = s["cache"][:s["code_bytes"]].view(s["n_pages"], H, 2, PAGE * D)
    scales = s["cache"][s["scale_off"]:s["scale_off"] + s["n_pages"] * H * 8].view(torch.float32).view(s["n_pages"], H, 2)
    got = codes[pages]
    lead = got.shape[:-2]
    n = len(lead)
    k = got[..., 0, :].reshape(*lead, 8, D // 64, 4, 2, 64)     # j, half of d, token / 16, token % 2, d % 64
    k = k.permute(*range(n), n + 2, n, n + 3, n + 1, n + 4).reshape(*lead, PAGE, D)
    v = got[..., 1, :].reshape(*lead, D, PAGE).transpose(-1, -2)
    if c["kv"] == "int8":
        return k.float() - 128, v.float() - 128, scales[pages]
    return (k.contiguous().view(torch.float8_e4m3fn).float(), v.contiguous().view(torch.float8_e4m3fn).float(), scales[pages])


def _round_codes(x, kv):
    if kv == "int8":
        return x.clamp(-127, 127).round()
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _append_plain(s):
    c = s["case"]
    H, Hq, D, kv = c["kv_heads"], c["q_heads"], c["dim"], c["kv"]
    top = 127.0 if kv == "int8" else 448.0
    x = s["qkv"].float()
    cos, sin = _angles(s["positions"], s["axis"], s["turns"])
    turned = _rotate(x[:, :Hq + H], cos, sin, False)
    new = torch.stack([turned[:, Hq:], x[:, Hq + H:]], 2)        # [T][H][2][D]
    first, count = s["runs"].long().T
    slot = s["slots"].long()[first]
    page, off = slot // PAGE, slot % PAGE
    k, v, scales = _tiles(s, page)
    old = torch.stack([k, v], 2)                                  # [R][H][2][64][D]
    old_scale = torch.where((off > 0)[:, None, None], scales, 0.0)
    at = torch.arange(PAGE, device=x.device)
    is_new = (at >= off[:, None]) & (at < (off + count)[:, None])
    token = (first[:, None] + at - off[:, None]).clamp(0, len(x) - 1)
    fresh = torch.where(is_new[..., None, None, None], new[token], 0.0).permute(0, 2, 3, 1, 4)
    scale = torch.maximum(old_scale, fresh.abs().amax((-1, -2)) / top)
    inv = torch.where(scale > 0, 1.0 / scale, 0.0)
    kept = _round_codes(old * (old_scale * inv)[..., None, None], kv)
    codes = torch.where(is_new[:, None, None, :, None], _round_codes(fresh * inv[..., None, None], kv), kept)
    # the updated pages go back into the cache
    bytes_ = (codes + 128).to(torch.uint8) if kv == "int8" else codes.to(torch.float8_e4m3fn).view(torch.uint8)
    R = len(page)
    kb = bytes_[:, :, 0].reshape(R, H, 4, 8, 2, D // 64, 64).permute(0, 1, 3, 5, 2, 4, 6).reshape(R, H, PAGE * D)
    vb = bytes_[:, :, 1].transpose(-1, -2).reshape(R, H, PAGE * D)
    n = s["n_pages"]
    s["cache"][:s["code_bytes"]].view(n, H, 2, PAGE * D)[page] = torch.stack([kb, vb], 2)
    s["cache"][s["scale_off"]:s["scale_off"] + n * H * 8].view(torch.float32).view(n, H, 2)[page] = scale
    # every filled slot of the pages touched, as the values the codes stand for
    values = (codes * scale[..., None, None]).permute(2, 0, 3, 1, 4)   # [2][R][64][H][D]
    filled = at < (off + count)[:, None]
    return {"q": turned[:, :Hq].to(torch.bfloat16), "k": values[0][filled].to(torch.bfloat16), "v": values[1][filled].to(torch.bfloat16)}


def _attend_plain(s):
    c = s["case"]
    H, Hq, D, Q = c["kv_heads"], c["q_heads"], c["dim"], c["new"]
    G = Hq // H
    table = s["table"].long().clamp(min=0)
    B, P = table.shape
    k, v, scales = _tiles(s, table)                               # [B][P][H][64][D], [B][P][H][2]
    k = (k * scales[..., 0, None, None]).transpose(1, 2).reshape(B, H, P * PAGE, D)
    v = (v * scales[..., 1, None, None]).transpose(1, 2).reshape(B, H, P * PAGE, D)
    qs = s["q_start"].long()
    at = (qs[:-1, None] + torch.arange(Q, device=qs.device)).clamp(max=len(s["q"]) - 1)
    q = s["q"].float()[at].view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    score = (q @ k.transpose(-1, -2)) * s["scale"]
    del k
    score = score.view(B, H, Q, G, P * PAGE)
    if c["softcap"]:
        score = torch.tanh(score / c["softcap"]) * c["softcap"]
    ctx = s["ctx"].long()
    pos = (ctx - (qs[1:] - qs[:-1]))[:, None] + torch.arange(Q, device=qs.device)   # [B][Q]
    key = torch.arange(P * PAGE, device=qs.device)
    gap = pos[:, :, None] - key                                                      # [B][Q][L]
    if s["slopes"] is not None:
        score = score - s["slopes"].view(1, H, 1, G, 1) * gap.abs()[:, None, :, None].float()
    seen = gap >= 0
    if s["prefix"] is not None:
        seen |= key < s["prefix"].long()[:, None, None]
    if c["window"]:
        seen &= gap < c["window"]
    seen &= key < ctx[:, None, None]
    score = torch.where(seen[:, None, :, None], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    del score
    total = p.sum(-1)
    o = p.view(B, H, Q * G, P * PAGE) @ v
    total = total.view(B, H, Q * G, 1)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(B, H, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, D)
    return {"out": o.reshape(B * Q, Hq, D).to(TYPES[c["type"]])}


# ----------------------------------------------------------------------------- the outputs in 64 bits

def _exact_angles(positions, axis, inv, sign=1.0):
    a = positions.double()[axis].T * torch.tensor(inv, dtype=torch.float64, device=positions.device)
    return torch.cos(a), torch.sin(a) * sign


def _exact_rotate(x, cos, sin, interleaved):
    """Complex multiplication pair by pair, in float64."""
    pairs = cos.shape[1]
    i = torch.arange(pairs, device=x.device)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    z = torch.complex(x[..., one], x[..., two]) * torch.complex(cos, sin)[:, None]
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_value(byte, kv):
    """Float64 value of each code byte."""
    b = torch.arange(256, device=byte.device, dtype=torch.float64)
    if kv == "int8":
        return (b - 128)[byte.long()]
    e, m = (torch.arange(256, device=byte.device) >> 3) & 15, b % 8
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    return torch.where(b >= 128, -mag, mag)[byte.long()]


def _exact_kv(s, row, count):
    """Float64 K and V [count][H][D] of the first `count` tokens of a block-table row, byte by byte."""
    c = s["case"]
    H, D = c["kv_heads"], c["dim"]
    dev = s["cache"].device
    tok = torch.arange(count, device=dev)
    page = row.to(dev).long()[tok // PAGE][:, None, None]
    o = (tok % PAGE)[:, None, None]
    h = torch.arange(H, device=dev)[None, :, None]
    d = torch.arange(D, device=dev)[None, None, :]
    tile = (page * H + h) * (2 * PAGE * D)
    kb = tile + ((((o % 16) // 2) * (D // 64) + d // 64) * 8 + (o // 16) * 2 + o % 2) * 64 + d % 64
    vb = tile + PAGE * D + d * 64 + o
    sc = s["cache"][s["scale_off"]:s["scale_off"] + s["n_pages"] * H * 8].view(torch.float32).double().view(-1)
    at = (page * H + h) * 2
    return (_exact_value(s["cache"][kb], c["kv"]) * sc[at], _exact_value(s["cache"][vb], c["kv"]) * sc[at + 1])


def exact(case, seed):
    c = dict(case)
    if c["op"] == "plan":
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        cos, sin = _exact_angles(s["positions"], s["axis"], s["inv"], -1.0 if c["inverse"] else 1.0)
        return {"out": _exact_rotate(s["x"].double(), cos, sin, c["interleaved"])}
    H, Hq, D = c["kv_heads"], c["q_heads"], c["dim"]
    if c["op"] == "append":
        cos, sin = _exact_angles(s["positions"], s["axis"], s["inv"])
        x = s["qkv"].double()
        turned = _exact_rotate(x[:, :Hq + H], cos, sin, False)
        new = {0: turned[:, Hq:], 1: x[:, Hq + H:]}
        top = 127.0 if c["kv"] == "int8" else 448.0

        def code(v):
            v = v.clamp(-top, top)
            if c["kv"] == "int8":
                return v.round()
            e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
            return torch.round(v / 2.0 ** (e - 3)) * 2.0 ** (e - 3)

        got = {0: [], 1: []}
        for t, n in s["runs"].tolist():
            slot = int(s["slots"][t])
            page, off = slot // PAGE, slot % PAGE
            row = torch.tensor([page])
            held = _exact_kv(s, row, off) if off else None
            at = s["scale_off"] + page * H * 8
            sc = s["cache"][at:at + H * 8].view(torch.float32).double().view(H, 2)
            for w in (0, 1):
                v = new[w][t:t + n]
                was = sc[:, w] if off else torch.zeros(H, dtype=torch.float64, device=v.device)
                now = torch.maximum(was, v.abs().amax((0, 2)) / top)[None, :, None]
                part = [code(held[w] / now) * now] if off else []
                got[w].append(torch.cat(part + [code(v / now) * now]))
        return {"q": turned[:, :Hq], "k": torch.cat(got[0]), "v": torch.cat(got[1])}
    out = torch.zeros((len(s["q"]), Hq, D), dtype=torch.float64, device=DEV)
    G = Hq // H
    starts, ctx = s["q_start"].tolist(), s["ctx"].tolist()
    for b in range(c["requests"]):
        t0, t1, L = starts[b], starts[b + 1], ctx[b]
        k, v = _exact_kv(s, s["table_host"][b].clamp(min=0), L)
        key = torch.arange(L, device=DEV)
        pos = torch.arange(L - (t1 - t0), L, device=DEV)[:, None]
        ok = key <= pos
        if c["prefix"]:
            ok = ok | (key < min(c["prefix"], L))
        if c["window"]:
            ok = ok & (pos - key < c["window"])
        for h in range(Hq):
            sc = s["q"][t0:t1, h].double() @ k[:, h // G].T / math.sqrt(D)
            if c["softcap"]:
                sc = c["softcap"] * torch.tanh(sc / c["softcap"])
            if c["slopes"]:
                sc = sc - float(s["slopes"][h].double()) * (pos - key).abs()
            out[t0:t1, h] = torch.softmax(sc.masked_fill(~ok, float("-inf")), -1) @ v[:, h // G]
    return {"out": out}


# ----------------------------------------------------------------------------- work

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": n * (size[c["type"]] + size[c["out"]]) + 4 * c["axes"] * c["tokens"],
                "flops": c["tokens"] * c["heads"] * c["rot"] * 3}
    lens, add = _lengths(c)
    T = sum(max(a, 0) for a in add)
    n = len(lens)
    if c["op"] == "plan":
        held = [_pages(v) for v in lens]
        fresh = sum(_pages(a + max(b, 0)) - h for a, b, h in zip(lens, add, held))
        back = sum(h for h, a in zip(held, add) if a < 0)
        runs = min(T, T // 64 + 2 * min(n, T))
        # lens, add, each request's current page; lens, context, status and start out; pages taken and given back; slots, positions, runs
        return {"bytes": 4 * (3 * n + 4 * n + 2 * fresh + 2 * back + 2 * T + 2 * runs), "flops": 0}
    H, Hq, D = c["kv_heads"], c["q_heads"], c["dim"]
    if c["op"] == "append":
        filled = sum(l % PAGE + a for l, a in zip(lens, add))
        fresh = T * H * 2 * D
        # qkv in, rotated q out, new codes and scales out; every filled slot of the touched pages read back as 16 bits
        return {"bytes": T * (Hq + 2 * H) * D * size[c["type"]] + T * Hq * D * 2 + fresh + filled * H * 2 * D * (1 + 2) + T * 4 * c["axes"],
                "flops": T * (Hq + H) * D * 3 + fresh * 3}
    keys = pairs = 0
    for l, a in zip(lens, add):
        L = l + a
        lo = L
        for i in range(a):
            top = max(l + i + 1, min(c["prefix"], L))
            low = max(0, l + i + 1 - c["window"]) if c["window"] else 0
            pairs += top - low
            lo = min(lo, low)
        keys += L - lo
    return {"bytes": keys * H * D * 2 + sum(_pages(a + b) for a, b in zip(lens, add)) * (8 * H + 4) + 2 * T * Hq * D * 2,
            "flops": 4 * pairs * Hq * D}
