"""Measured cases of the operators that a serving step has around its packed projections: embedding rows
out of a packed matrix (embed), low-rank adapters of many requests beside a shared projection (plan,
lora) and log probabilities of given tokens with entropy, rank and top alternatives (logprob).

listed() names fixed cases, draw() more of the same ranges; prepare() makes a case's inputs from a
seed, run() is one pass (the plain form where `own` is false, the library's kernels where it is
true), exact() the same outputs in 64 bits from the definition, work() the bytes and operations
that a pass cannot do without.

Adapters lie in pools of rank rows: adapter a of a projection K -> N takes rows first..first + rank
of A [rows][K] and of B [rows][N], with table[a] = (first, rank), and adds scale[a] * (x A^T) B to the
projection's y. A plan groups a step's tokens by adapter, in their order, into tiles of up to 16
tokens (64 from 1024 tokens on): (adapter, first place in order, count, 0).

A packed matrix, as both sides hold it: section 0 codes, section 1 fp16 scales (one per row and
block of 128 columns), each starting at a multiple of 256 bytes, in one of four layouts (ternary or
INT4, row-group records or byte lookup); _pack() writes them from their specification.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # which adapter serves which token of a decode step: once per step, before all layers
        {"name": "plan_step", "op": "plan", "tokens": 64, "adapters": 48, "runs": False, "bare": 0.1},
        # the same for a step of long prompt chunks, with all of a large pool's adapters resident
        {"name": "plan_prompts", "op": "plan", "tokens": 16384, "adapters": 512, "runs": True, "bare": 0.1},
        # one token of one request beside one square projection
        {"name": "lora_one", "op": "lora", "tokens": 1, "adapters": 1, "runs": False, "bare": 0.0, "rank": 16, "mixed": False,
         "k": 4096, "n": "4096", "type": "f32"},
        # a decode step of 64 requests with adapters of different ranks, the q|k|v projections that share one x
        {"name": "lora_step", "op": "lora", "tokens": 64, "adapters": 48, "runs": False, "bare": 0.1, "rank": 64, "mixed": True,
         "k": 5120, "n": "5120,1024,1024", "type": "f32"},
        # 16 requests with four draft tokens each, the gate|up projections
        {"name": "lora_verify", "op": "lora", "tokens": 80, "adapters": 12, "runs": True, "bare": 0.0, "rank": 16, "mixed": False,
         "k": 5120, "n": "13824,13824", "type": "f32"},
        # prompts of four customers and of the bare model, gate|up, activations in 16 bits
        {"name": "lora_prompt", "op": "lora", "tokens": 8190, "adapters": 5, "runs": True, "bare": 0.2, "rank": 64, "mixed": False,
         "k": 5120, "n": "13824,13824", "type": "bf16"},
        # short prompts, the down projection, high and odd ranks
        {"name": "lora_down", "op": "lora", "tokens": 1023, "adapters": 24, "runs": True, "bare": 0.1, "rank": 128, "mixed": True,
         "k": 13824, "n": "5120", "type": "f32"},
        # one answer token with 20 alternatives
        {"name": "logprob_one", "op": "logprob", "rows": 1, "vocab": 131072, "type": "f32", "top": 20, "scale": 1.0, "masked": 0.0},
        # a decode step of 64 requests whose answers follow a grammar: most of the vocabulary at -inf, an odd vocabulary
        {"name": "logprob_step", "op": "logprob", "rows": 64, "vocab": 128257, "type": "f32", "top": 5, "scale": 1.25, "masked": 0.9},
        # scoring a prompt: every token's log probability and the entropy
        {"name": "logprob_prompt", "op": "logprob", "rows": 4095, "vocab": 131072, "type": "bf16", "top": 0, "scale": 1.0, "masked": 0.0},
        # the tokens of a decode step, out of the packed LM head that is tied to the embedding
        {"name": "embed_step", "op": "embed", "tokens": 64, "vocab": 65536, "k": 5120, "format": "ternary_lut", "type": "bf16",
         "scale": 1.0},
        # a prompt's tokens, scaled as some models want it
        {"name": "embed_prompt", "op": "embed", "tokens": 8190, "vocab": 65536, "k": 5120, "format": "int4", "type": "bf16",
         "scale": 71.5},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "lora", "lora", "lora", "logprob", "logprob", "logprob", "embed"])
    if op == "plan":
        tokens = _logint(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "adapters": _logint(rng, 1, 1024), "runs": rng.random() < 0.5,
                "bare": rng.choice([0.0, 0.1, 0.5])}
    if op == "lora":
        tokens = rng.choice([_logint(rng, 1, 16), _logint(rng, 17, 256), _logint(rng, 257, 8190)])
        k, n = rng.choice([(5120, "5120,1024,1024"), (5120, "13824,13824"), (13824, "5120"), (4096, "4096"), (4096, "2048,2048"),
                           (2048, "4096"), (8 * rng.randint(16, 700), str(rng.randint(33, 9000)))])
        kind = rng.choice(["f32", "f32", "bf16", "f16"])
        tokens = min(tokens, int(8.0e8) // (2 * SIZE[kind] * sum(int(v) for v in n.split(","))))
        return {"op": op, "tokens": tokens, "adapters": _logint(rng, 1, 64) if tokens <= 1024 else _logint(rng, 2, 16),
                "runs": tokens > 1024 or rng.random() < 0.5, "bare": rng.choice([0.0, 0.0, 0.2]),
                "rank": rng.choice([8, 16, 16, 32, 64]) if tokens > 1024 else rng.choice([4, 8, 16, 16, 32, 64, 128, rng.randint(1, 128)]),
                "mixed": rng.random() < 0.5, "k": k, "n": n, "type": kind}
    if op == "logprob":
        kind = rng.choice(["f32", "f32", "bf16", "f16"])
        top = rng.choice([0, 0, 1, 5, 20, rng.randint(1, 32)])
        vocab = rng.choice([131072, rng.randint(32000, 160000), _logint(rng, 100, 32000)])
        rows = rng.choice([_logint(rng, 1, 16), _logint(rng, 17, 256), _logint(rng, 257, 4095)])
        rows = max(1, min(rows, (6 * 10 ** 7 if top else 2.6 * 10 ** 8) // vocab))
        return {"op": op, "rows": int(rows), "vocab": vocab, "type": kind, "top": top, "scale": rng.choice([1.0, 1.0, 0.7, 2.0]),
                "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    return {"op": op, "tokens": _logint(rng, 1, 8190), "vocab": _logint(rng, 1000, 65536), "k": 128 * rng.randint(4, 40),
            "format": rng.choice(["ternary", "ternary_lut", "int4", "int4_lut"]), "type": rng.choice(["bf16", "bf16", "f32", "f16"]),
            "scale": rng.choice([1.0, 45.25])}


# ----------------------------------------------------------------------------- adapters: sizes and inputs

def _tile(tokens):
    return 16 if tokens < 1024 else 64


def _max_tiles(c):
    return c["tokens"] // _tile(c["tokens"]) + min(c["tokens"], c["adapters"])


def _ids(c, g):
    """The adapter of each token on the host, -1 for the bare model: requests' runs of tokens, or a token each."""
    T, A = c["tokens"], c["adapters"]
    if c["runs"]:
        n = max(1, min(T, 2 * A))
        cuts = torch.sort(torch.randint(0, T, (n - 1,), generator=g)).values
        run = torch.searchsorted(cuts, torch.arange(T), right=True)
    else:
        n, run = T, torch.arange(T)
    who = torch.randperm(max(n, A), generator=g)[:n] % A
    if c["bare"]:
        who[torch.rand(n, generator=g) < c["bare"]] = -1
    return who[run]


def _ranks(c, g):
    A, r = c["adapters"], c["rank"]
    if not c["mixed"]:
        return torch.full((A,), r, dtype=torch.int64)
    low = max(1, r // 8)
    ranks = low + torch.randint(0, r - low + 1, (A,), generator=g)
    ranks[0] = r
    return ranks


def _outs(c):
    return [int(v) for v in c["n"].split(",")]


# ----------------------------------------------------------------------------- packed matrices

def _codes(c, seed):
    """int8 codes [vocab][k] and fp16 scales [vocab][k / 128]."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    N, K = c["vocab"], c["k"]
    q = torch.randint(-1, 2, (N, K), generator=g, device=DEV, dtype=torch.int8) if c["format"].startswith("ternary") else \
        torch.randint(-7, 8, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sc = (0.02 * (0.5 + torch.rand((N, K // 128), generator=g, device=DEV))).to(torch.float16)
    return q, sc


def _aligned(n):
    return (n + 255) // 256 * 256


def _pack(c, q, sc):
    """The packed buffer (uint8) of codes q and scales sc, and the byte at which the scales start."""
    N, K = q.shape
    KB = K // 128
    lut, tern = c["format"].endswith("_lut"), c["format"].startswith("ternary")
    rows = 32 if lut else 16
    G = -(-N // rows)
    q = torch.nn.functional.pad(q, (0, 0, 0, G * rows - N))
    sc = torch.nn.functional.pad(sc, (0, 0, 0, G * rows - N))
    if tern:
        u = torch.where(q < 0, torch.full_like(q, 2), q)
    else:
        u = q & 15
    if not lut:
        per = 16 if tern else 8
        r = torch.arange(per, device=DEV)
        at = torch.where(r % 2 == 0, r, 15 + r) if tern else torch.where(r % 2 == 0, 2 * r, 14 + 2 * r)
        w = torch.zeros((G * rows, K // per), dtype=torch.int32, device=DEV)
        for i in range(per):
            w |= u[:, i::per].to(torch.int32) << int(at[i])
        w = w.view(G, 16, KB, -1)
        full = KB // 8 * 8
        a = w[:, :, :full].reshape(G, 16, full // 8, 8 * w.shape[3]).transpose(1, 2).reshape(G, -1)
        codes = torch.cat([a, w[:, :, full:].reshape(G, -1)], 1).reshape(-1).view(torch.uint8)
        S = -(-KB // 8)
        scales = torch.nn.functional.pad(sc, (0, S * 8 - KB)).view(G, 16, S, 8).transpose(1, 2).contiguous()
    else:
        per = 4 if tern else 2
        b = torch.zeros((G * 32, K // per), dtype=torch.uint8, device=DEV)
        for i in range(per):
            b |= (u[:, i::per].to(torch.int32) << (i * (8 // per))).to(torch.uint8)
        b = b.view(G, 32, KB, -1, 32)                                     # group, row, block, half, byte
        turn = (torch.arange(32, device=DEV)[:, None] + torch.arange(32, device=DEV)) % 32   # row, position -> byte
        b = torch.gather(b, 4, turn.view(1, 32, 1, 1, 32).expand(b.shape))
        codes = b.reshape(G, 32, KB, -1, 16).permute(2, 0, 3, 1, 4).reshape(-1)
        scales = sc.T.contiguous()
    at = _aligned(codes.numel())
    out = torch.zeros(_aligned(at + scales.numel() * 2), dtype=torch.uint8, device=DEV)
    out[:codes.numel()] = codes
    out[at:at + scales.numel() * 2] = scales.reshape(-1).view(torch.uint8)
    return out, at


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if own:
        import quantized_gemv_unpack_gb300 as lib
    if c["op"] == "plan":
        s["ids"] = _ids(c, gc).to(torch.int32).to(DEV)
        if own:
            s["call"] = lib.LoraPlan(s["ids"], c["adapters"])
        return s
    if c["op"] == "lora":
        T, K, Ns = c["tokens"], c["k"], _outs(c)
        ids, ranks = _ids(c, gc), _ranks(c, gc)
        # the adapters' rows in the pool: in no order, with rows of others between them
        order = torch.randperm(c["adapters"], generator=gc)
        first = torch.zeros_like(ranks)
        first[order] = torch.cumsum(ranks[order] + 1, 0) - ranks[order]
        rows = int((first + ranks).max()) + 3
        s["ids"] = ids.to(torch.int32).to(DEV)
        s["table"] = torch.stack([first, ranks], 1).to(torch.int32).to(DEV)
        s["scale"] = (0.5 + 2.0 * torch.rand(c["adapters"], generator=gc)).to(DEV)
        s["most"], s["rank"] = int(torch.bincount(ids[ids >= 0], minlength=1).max()), int(ranks.max())
        s["x"] = torch.randn((T, K), generator=g, device=DEV).to(torch.bfloat16)
        s["a"] = [(torch.randn((rows, K), generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16) for _ in Ns]
        s["b"] = [(torch.randn((rows, (n + 7) // 8 * 8), generator=g, device=DEV) * (0.2 / math.sqrt(c["rank"]))).to(torch.bfloat16)[:, :n]
                  for n in Ns]
        s["y"] = [torch.randn((T, n), generator=g, device=DEV).to(TYPES[c["type"]]) for n in Ns]
        if own:
            s["plan"] = lib.LoraPlan(s["ids"], c["adapters"])
            s["plan"].run()
            s["call"] = lib.Lora(s["plan"], s["table"], s["scale"], s["x"], list(zip(s["a"], s["b"], s["y"])),
                                 max_rank=c["rank"])
        return s
    if c["op"] == "logprob":
        T, V = c["rows"], c["vocab"]
        # an LM head's logits: a bulk and a few likely tokens, among them mostly the given one
        x = torch.empty((T, (V + 7) // 8 * 8), dtype=TYPES[c["type"]], device=DEV)[:, :V]
        at = 0
        while at < T:
            n = min(256, T - at)
            z = torch.randn((n, V), generator=g, device=DEV) * 2.0
            likely = torch.randint(0, V, (n, 12), generator=g, device=DEV)
            z.scatter_add_(1, likely, 12.0 * torch.rand((n, 12), generator=g, device=DEV))
            if c["masked"]:
                z.masked_fill_(torch.rand((n, V), generator=g, device=DEV) < c["masked"], float("-inf"))
                z.scatter_(1, likely[:, :4], 5.0 + torch.rand((n, 4), generator=g, device=DEV))
            x[at:at + n] = z.to(x.dtype)
            tok = torch.where(torch.rand(n, generator=g, device=DEV) < 0.8, likely[:, 0],
                              torch.randint(0, V, (n,), generator=g, device=DEV))
            s["tokens"] = torch.cat([s["tokens"], tok]) if at else tok
            at += n
        s["x"], s["tokens"] = x, s["tokens"].to(torch.int32)
        if own:
            s["call"] = lib.LogProb(x, s["tokens"], top=c["top"], scale=c["scale"])
        return s
    s["tokens"] = torch.randint(0, c["vocab"], (c["tokens"],), generator=g, device=DEV).to(torch.int32)
    s["packed"], s["scales_at"] = _pack(c, *_codes(c, seed))
    if own:
        kind = {"ternary": lib.QMV_TERNARY2, "ternary_lut": lib.QMV_TERNARY2_LUT, "int4": lib.QMV_INT4, "int4_lut": lib.QMV_INT4_LUT}
        s["out"] = torch.empty((c["tokens"], c["k"]), dtype=TYPES[c["type"]], device=DEV)
        s["call"] = lib.Embed(lib.qmv_pack_desc(kind[c["format"]], c["vocab"], c["k"]), s["packed"], s["tokens"], s["out"], scale=c["scale"])
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plan_plain, "lora": _lora_plain, "logprob": _logprob_plain, "embed": _embed_plain}[op](s)
    call = s["call"]
    call.run()
    if op == "plan":
        return {"order": call.order, "tiles": call.tiles}
    if op == "lora":
        return {"y": s["y"]}
    if op == "embed":
        return {"out": s["out"]}
    out = {"logprob": call.logprob, "rank": call.rank, "lse": call.lse, "entropy": call.entropy}
    if s["case"]["top"]:
        out |= {"top_index": call.top_index, "top_logprob": call.top_logprob}
    return out


def _plan_plain(s):
    c, ids = s["case"], s["ids"].long()
    T, A, tile = c["tokens"], c["adapters"], _tile(c["tokens"])
    key = torch.where(ids < 0, A, ids)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(A + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    order = torch.where(torch.arange(T, device=DEV) < T - count[A], order, -1)
    count = count[:A]
    first = torch.cumsum(count, 0) - count
    ends = torch.cumsum((count + tile - 1) // tile, 0)
    i = torch.arange(_max_tiles(c), device=DEV)
    a = torch.searchsorted(ends, i, right=True)
    there = a < A
    a = a.clamp(max=A - 1)
    j = i - (ends[a] - (count[a] + tile - 1) // tile)
    tiles = torch.stack([a, first[a] + j * tile, torch.clamp(count[a] - j * tile, max=tile), torch.zeros_like(a)], 1)
    return {"order": order.to(torch.int32), "tiles": torch.where(there[:, None], tiles, 0).to(torch.int32)}


def _lora_plain(s):
    c, ids = s["case"], s["ids"].long()
    T, A, most, R = c["tokens"], c["adapters"], s["most"], s["rank"]
    # the tokens of each adapter side by side, padded to the longest: [A][most]
    key = torch.where(ids < 0, A, ids)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(A + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))[:A]
    i = torch.arange(most, device=DEV)
    there = i < count[:, None]
    token = order[((torch.cumsum(count, 0) - count)[:, None] + i).clamp(max=T - 1)]
    j = torch.arange(R, device=DEV)
    held = j < s["table"][:, 1:]
    row = torch.where(held, s["table"][:, :1] + j, 0).long()
    x = s["x"].float()[token]
    place = torch.where(there, token, T)
    return {"y": [_lora_add(x, torch.where(held[:, :, None], a[row].float(), 0.0), torch.where(held[:, :, None], b[row].float(), 0.0),
                            s["scale"], y, place) for a, b, y in zip(s["a"], s["b"], s["y"])]}


def _lora_add(x, a, b, scale, y, place):
    d = torch.matmul(torch.matmul(x, a.transpose(1, 2)), b) * scale[:, None, None]
    sum = torch.zeros((y.shape[0] + 1, y.shape[1]), device=DEV)
    sum[place.reshape(-1)] = d.reshape(-1, y.shape[1])
    y.copy_(y.float() + sum[:-1])
    return y


def _logprob_plain(s):
    c, x = s["case"], s["x"]
    T, V = x.shape
    at = s["tokens"].long()[:, None]
    z = x.float() * c["scale"]
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = torch.log(total) - (e * torch.where(e > 0, d, 0.0)).sum(1, keepdim=True) / total
    given = x.gather(1, at)
    ahead = (x > given).sum(1) + ((x == given) & (torch.arange(V, device=DEV) < at)).sum(1)
    out = {"logprob": ((z.gather(1, at) - m) - torch.log(total))[:, 0], "rank": ahead.to(torch.int32), "lse": lse[:, 0], "entropy": entropy[:, 0]}
    if c["top"]:
        best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out |= {"top_index": best.to(torch.int32), "top_logprob": (z.gather(1, best) - m) - torch.log(total)}
    return out


def _embed_plain(s):
    c, n = s["case"], s["tokens"].long()[:, None]
    K = c["k"]
    KB, NG = K // 128, -(-c["vocab"] // 32)
    k = torch.arange(K, device=DEV)
    b, i = k // 128, k % 128
    tern = c["format"].startswith("ternary")
    if c["format"].endswith("_lut"):
        per = 4 if tern else 2
        byte = i // per
        t = byte // 32 * 32 + (byte % 32 - n) % 32
        at = (b * NG + n // 32) * (1024 if tern else 2048) + t // 16 * 512 + n % 32 * 16 + t % 16
        u = s["packed"][at].to(torch.int32) >> (i % per * (8 // per))
        scale_at = b * NG * 32 + n
    else:
        per = 16 if tern else 8
        nbk = torch.clamp(KB - b // 8 * 8, max=8)
        at = (n // 16 * 16 * KB + b // 8 * 128 + n % 16 * nbk + b % 8) * (128 // per) + i // per
        r = i % per
        r = torch.where(r % 2 == 0, r, 15 + r) if tern else torch.where(r % 2 == 0, 2 * r, 14 + 2 * r)
        u = s["packed"].view(torch.int32)[at] >> r.to(torch.int32)
        scale_at = (n // 16 * (-(-KB // 8)) + b // 8) * 128 + n % 16 * 8 + b % 8
    if tern:
        q = (u & 1) - ((u >> 1) & 1)
    else:
        q = ((u & 15) ^ 8) - 8
    sc = s["packed"][s["scales_at"]:].view(torch.float16)[scale_at].float()
    return {"out": (q.float() * sc * c["scale"]).to(TYPES[c["type"]])}


# ----------------------------------------------------------------------------- the same in 64 bits, from the definition

def exact(case, seed):
    c = dict(case)
    if c["op"] == "plan":
        return None
    s = prepare(c, seed)
    if c["op"] == "lora":
        got = [y.double() for y in s["y"]]
        ids, table = s["ids"].cpu().numpy(), s["table"].cpu().numpy()
        for a in np.unique(ids[ids >= 0]):
            t = torch.from_numpy(np.flatnonzero(ids == a)).to(DEV)
            lo, hi = int(table[a, 0]), int(table[a, 0] + table[a, 1])
            for p, y in enumerate(got):
                h = s["x"][t].double() @ s["a"][p][lo:hi].double().T
                y[t] += s["scale"][a].double() * (h @ s["b"][p][lo:hi].double())
        return {"y": got}
    if c["op"] == "embed":
        q, sc = _codes(c, seed)
        t = s["tokens"].long()
        return {"out": (q[t].double().view(len(t), -1, 128) * sc[t].double()[:, :, None] * c["scale"]).view(len(t), -1)}
    lse, entropy, logprob, top = [], [], [], []
    for at in range(0, c["rows"], 256):
        x = s["x"][at:at + 256].double()
        z = x * c["scale"]
        n = torch.logsumexp(z, 1)
        p = torch.exp(z - n[:, None])
        lse.append(n)
        entropy.append(-torch.special.xlogy(p, p).sum(1))
        logprob.append(z.gather(1, s["tokens"][at:at + 256].long()[:, None])[:, 0] - n)
        if c["top"]:
            top.append(torch.topk(z, c["top"], 1).values - n[:, None])
    out = {"logprob": torch.cat(logprob), "rank": None, "lse": torch.cat(lse), "entropy": torch.cat(entropy)}
    if c["top"]:
        out |= {"top_index": None, "top_logprob": torch.cat(top)}
    return out


# ----------------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "plan":
        return {"bytes": 8 * c["tokens"] + 16 * _max_tiles(c), "flops": 0}
    if c["op"] == "logprob":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * SIZE[c["type"]] + c["rows"] * (4 + 16 + 8 * c["top"]), "flops": 5 * n}
    if c["op"] == "embed":
        rows = c["vocab"] * (1.0 - (1.0 - 1.0 / c["vocab"]) ** c["tokens"])     # tokens that differ, on average
        bits = 2 if c["format"].startswith("ternary") else 4
        return {"bytes": 4 * c["tokens"] + rows * (c["k"] * bits / 8 + c["k"] / 64) + c["tokens"] * c["k"] * SIZE[c["type"]],
                "flops": 2 * c["tokens"] * c["k"]}
    g = torch.Generator().manual_seed(1)
    ids, ranks = _ids(c, g), _ranks(c, g)
    used = torch.unique(ids[ids >= 0])
    T, N = int((ids >= 0).sum()), sum(_outs(c))
    rows = int(ranks[used].sum())
    # x and the used adapters' rows in, y in and out
    return {"bytes": 2 * T * c["k"] + 2 * rows * (c["k"] * len(_outs(c)) + N) + 2 * T * N * SIZE[c["type"]] + 4 * c["tokens"],
            "flops": 2 * int(ranks[ids[ids >= 0]].sum()) * (c["k"] * len(_outs(c)) + N)}
