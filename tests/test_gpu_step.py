"""GPU parity of qmv_embed, lora_plan, lora_run and logprob_run with the float64 oracle, their edges, and a run of them together
around the packed matvecs as a serving step makes it."""
import math

import numpy as np
import pytest

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # half a step, relative
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half of the smallest step, or more


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import quantized_gemv_unpack_gb300 as q
    assert torch.cuda.is_available()
    q.qmv_check_status()
    return q, torch, torch.device("cuda:0")


def _type(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _f64(t):
    return t.double().cpu().numpy()


def _guarded(torch, dev, rows, cols, kind, ld=None, fill=7.0):
    """A [rows][cols] view with rows of stride ld inside a buffer of `fill`, and the buffer."""
    ld = ld or cols
    buf = torch.full((rows * ld + 64,), fill, dtype=_type(torch, kind), device=dev)
    return buf[:rows * ld].view(rows, ld)[:, :cols], buf


# ----------------------------------------------------------------------------- embedding rows

def _packed(env, fmt, N, K, seed):
    from oracle import int4, ternary
    q, torch, dev = env
    g = np.random.default_rng(seed)
    top = 1 if "ternary" in fmt else 7
    codes = g.integers(-top, top + 1, (N, K)).astype(np.int8)
    s16 = (0.02 * (0.5 + g.random((N, K // 128)))).astype(np.float16)
    s16[0, 0] = 6e-8                                    # a subnormal scale
    mod = ternary if "ternary" in fmt else int4
    buf = (mod.pack_lut if fmt.endswith("_lut") else mod.pack)(codes, s16.view(np.uint16))
    d = q.qmv_pack_desc({"ternary": q.QMV_TERNARY2, "ternary_lut": q.QMV_TERNARY2_LUT, "int4": q.QMV_INT4, "int4_lut": q.QMV_INT4_LUT}[fmt], N, K)
    t = torch.from_numpy(np.frombuffer(buf, np.uint8).copy()).to(dev)
    return d, t, codes, s16


@pytest.mark.parametrize("fmt", ["ternary", "ternary_lut", "int4", "int4_lut"])
@pytest.mark.parametrize("kind", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("N,K,T", [(1, 128, 1), (33, 384, 70), (100, 1024, 5), (47, 1152, 300), (130, 2304, 4000)])
def test_embed(env, fmt, kind, N, K, T):
    """Exact: q * s is exact in fp32, and so are one rounding of its product with scale and one to the output's type."""
    q, torch, dev = env
    d, packed, codes, s16 = _packed(env, fmt, N, K, N + K)
    g = np.random.default_rng(T)
    tok = g.integers(0, N, T)
    if T > 4:
        tok[[1, 4]] = -1, -2 ** 31                      # padding
    for scale in (1.0, 0.37, -45.25):
        out, buf = _guarded(torch, dev, T, K, kind, ld=K + 16)
        q.qmv_embed(d, packed, torch.tensor(tok, dtype=torch.int32, device=dev), out, scale)
        w = codes.astype(np.float32) * np.repeat(s16.astype(np.float32), 128, axis=1)
        want = np.where((tok >= 0)[:, None], w[np.clip(tok, 0, N - 1)] * np.float32(scale), np.float32(0))
        want = torch.from_numpy(want).to(_type(torch, kind)).to(dev)
        assert torch.equal(out, want)
        assert bool((buf[:T * (K + 16)].view(T, K + 16)[:, K:] == 7).all()) and bool((buf[T * (K + 16):] == 7).all())
    assert q.qmv_check_status() == 0


def test_embed_follows_the_oracle(env):
    from oracle import int4, step
    q, torch, dev = env
    d, packed, codes, s16 = _packed(env, "int4", 40, 256, 3)
    tok = [5, 39, 5, -1, 0]
    out = torch.empty((5, 256), device=dev)
    q.qmv_embed(d, packed, torch.tensor(tok, dtype=torch.int32, device=dev), out, 3.0)
    want = step.embed(int4.dequant(codes, s16.view(np.uint16)), tok, 3.0)
    assert np.all(np.abs(_f64(out) - want) <= HALF["f32"] * np.abs(want))


@pytest.mark.parametrize("fmt", ["ternary", "ternary_lut"])
def test_embed_reports_what_is_no_row(env, fmt):
    q, torch, dev = env
    d, packed, codes, s16 = _packed(env, fmt, 20, 256, 5)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    out = torch.full((3, 256), 7.0, device=dev)
    for bad in (20, 2 ** 31 - 1):
        q.qmv_embed(d, packed, i32([1, bad, 2]), out, 1.0)
        assert q.qmv_check_status() == q.QMV_ERR_CORRUPT and q.qmv_check_status() == 0
        w = codes.astype(np.float32) * np.repeat(s16.astype(np.float32), 128, axis=1)
        assert np.array_equal(out.cpu().numpy(), np.stack([w[1], 0 * w[1], w[2]]))
    packed[:d.bytes[0]] = 0xFF                          # every code is 11
    q.qmv_embed(d, packed, i32([3]), out[:1], 1.0)
    assert q.qmv_check_status() == q.QMV_ERR_CORRUPT and not bool(out[0].any())


# ----------------------------------------------------------------------------- grouping by adapter

def _plan(env, ids, A):
    q, torch, dev = env
    p = q.LoraPlan(torch.as_tensor(np.asarray(ids, dtype=np.int32), device=dev), A)
    p.order.fill_(-9)
    p.tiles.fill_(-9)
    p.run()
    return p


@pytest.mark.parametrize("T", [1, 15, 16, 17, 300, 511, 512, 1023, 1024, 1500, 4096, 9000])
@pytest.mark.parametrize("A", [1, 2, 31, 300, 1024])
def test_plan(env, T, A):
    from oracle import step
    q = env[0]
    g = np.random.default_rng(T * 7 + A)
    for kind in range(4):
        if kind == 0:
            ids = g.integers(0, A, T)
        elif kind == 1:                                 # runs, some of them bare
            ids = np.repeat(g.integers(-1, A, T), g.integers(1, 60, T))[:T]
        elif kind == 2:
            ids = np.full(T, A - 1)
        else:
            ids = g.integers(-3, min(A, 2), T)
        p = _plan(env, ids, A)
        order, tiles = step.plan(ids, A, q.lora_tile(T), q.lora_max_tiles(T, A))
        assert np.array_equal(p.order.cpu().numpy(), order) and np.array_equal(p.tiles.cpu().numpy(), tiles)
    assert q.qmv_check_status() == 0


def test_plan_reports_ids_past_the_adapters(env):
    from oracle import step
    q = env[0]
    ids = [0, 3, 2 ** 31 - 1, 1, -2 ** 31, 0]
    p = _plan(env, ids, 3)
    assert q.qmv_check_status() == q.QMV_ERR_CORRUPT
    order, tiles = step.plan([0, -1, -1, 1, -1, 0], 3, 16, 3)
    assert np.array_equal(p.order.cpu().numpy(), order) and np.array_equal(p.tiles.cpu().numpy(), tiles)


# ----------------------------------------------------------------------------- adapters

def _adapters(g, A, ranks):
    """table [A][2] of rows in no order, with rows of none between them; the pool's rows."""
    first, at = np.zeros(A, dtype=np.int64), 2
    for i in g.permutation(A):
        first[i] = at
        at += ranks[i] + int(g.integers(0, 3))
    return np.stack([first, ranks], 1), at + 1


def _lora_case(env, ids, ranks, K, Ns, kind, seed, max_rank=None, ldx=None, ldy=0, magnitude=1.0, x=None):
    """One call over tasks of Ns columns: each output within the rounding errors of its own terms."""
    from oracle import step
    q, torch, dev = env
    g = np.random.default_rng(seed)
    T, A = len(ids), len(ranks)
    ranks = np.asarray(ranks)
    table, rows = _adapters(g, A, ranks)
    scale = (g.random(A) * 3 - 1).astype(np.float32)
    xt, _ = _guarded(torch, dev, T, K, "bf16", ld=ldx, fill=math.nan)
    xt.copy_(torch.from_numpy((g.standard_normal((T, K)) * magnitude).astype(np.float32) if x is None else x))
    tasks, bufs, before = [], [], []
    used = np.zeros(rows, dtype=bool)
    for f, r in table:
        used[f:f + r] = True
    for n in Ns:
        a = torch.from_numpy(g.standard_normal((rows, K)).astype(np.float32)).to(torch.bfloat16).to(dev)
        b = torch.full((rows, (n + 7) // 8 * 8 + 8), math.nan, dtype=torch.bfloat16, device=dev)[:, :n]
        b.copy_(torch.from_numpy(g.standard_normal((rows, n)).astype(np.float32)))
        free = torch.from_numpy(~used).to(dev)
        a[free], b[free] = math.nan, math.nan           # rows of no adapter are not looked at
        y, buf = _guarded(torch, dev, T, n, kind, ld=n + ldy)
        y.copy_(torch.from_numpy((g.standard_normal((T, n)) * 30).astype(np.float32)))
        tasks.append((a, b, y))
        bufs.append(buf)
        before.append(_f64(y))
    plan = _plan(env, ids, A)
    call = q.Lora(plan, torch.as_tensor(table.astype(np.int32), device=dev), torch.as_tensor(scale, device=dev), xt, tasks,
                  max_rank=max_rank or int(max(ranks.max(), 1)))
    call.run()
    assert q.qmv_check_status() == 0
    for (a, b, y), buf, was, n in zip(tasks, bufs, before, Ns):
        av, bv = np.nan_to_num(_f64(a)), np.nan_to_num(_f64(b))
        want, s1, s2 = step.lora(was, _f64(xt), ids, table, scale.astype(np.float64), av, bv)
        # fp32 sums, each addition within a step (2^-23): K / 16 matrix products with 16 additions inside and 16 joins; then rank /
        # 16 times three of them. The values between are rounded to 2^-26 (three parts), y once more and to its type.
        bound = (K / 16 + 32) * 2.0 ** -23 * s1 + (3 * 8 + 16 + 2) * 2.0 ** -23 * s2
        bound += (HALF["f32"] + (0 if kind == "f32" else HALF[kind])) * (np.abs(want) + bound) + LEAST[kind]
        got = _f64(y)
        bad = np.asarray(ids) < 0
        assert np.array_equal(got[bad], was[bad])
        assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / bound))
        room = buf[:T * (n + ldy)].view(T, n + ldy)[:, n:]
        assert bool((room == 7).all()) and bool((buf[T * (n + ldy):] == 7).all())
    return call, tasks, before, plan


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,A", [(1, 1), (5, 3), (16, 1), (17, 1), (64, 40), (200, 5), (1024, 3), (1100, 60), (1300, 3), (4000, 61)])
@pytest.mark.parametrize("K,N,rank", [(8, 1, 1), (72, 33, 16), (512, 640, 8), (1000, 257, 64), (200, 96, 128), (2048, 72, 17)])
def test_lora(env, kind, T, A, K, N, rank):
    g = np.random.default_rng(T + K)
    ids = g.integers(-1 if T > 1 else 0, A, T)
    ranks = g.integers(0, rank + 1, A)
    ranks[0] = rank
    _lora_case(env, ids, ranks, K, [N], kind, T + N, magnitude=0.1 if kind == "f16" else 1.0)


@pytest.mark.parametrize("T", [3, 40, 1300])
def test_lora_several_projections_and_strides(env, T):
    g = np.random.default_rng(T)
    ids = np.repeat(g.integers(-1, 6, T), 7)[:T]
    for ldy in (0, 1, 4, 8):
        _lora_case(env, ids, [4, 16, 0, 33, 64, 9], 640, [320, 64, 61, 128, 2, 1000, 8, 31], "f32", T + ldy, max_rank=128, ldx=656, ldy=ldy)
        _lora_case(env, ids, [4, 16, 0, 33, 64, 9], 640, [320, 64, 61], "bf16", T + ldy, ldy=ldy)


@pytest.mark.parametrize("T", [1, 16, 33, 1025, 2049])
@pytest.mark.parametrize("max_rank", [16, 32, 64, 128])
def test_lora_same_result_whatever_the_neighbours(env, T, max_rank):
    """A token's result has the same bits in another order and, where K is cut alike (few tiles), in a call of its own."""
    q, torch, dev = env
    g = np.random.default_rng(T)
    ids = g.integers(0, 4, T)
    call, tasks, before, plan = _lora_case(env, ids, [16, 3, 9, 16], 768, [200], "f32", 5, max_rank=max_rank)
    a, b, y = tasks[0]
    xt, table, scale = call.keep[3], call.keep[1], call.keep[2]
    for t in sorted({0, T // 2, T - 1}) if T < 1024 else []:
        one = torch.from_numpy(before[0][t:t + 1]).to(dev).float()
        p = _plan(env, ids[t:t + 1], 4)
        q.Lora(p, table, scale, xt[t:t + 1], [(a, b, one)], max_rank=max_rank).run()
        assert torch.equal(one[0], y[t])
    flip = torch.from_numpy(before[0]).to(dev).float().flip(0).contiguous()
    q.Lora(_plan(env, ids[::-1].copy(), 4), table, scale, xt.flip(0).contiguous(), [(a, b, flip)], max_rank=max_rank).run()
    assert torch.equal(flip.flip(0), y)


def test_lora_infinite_and_nan_tokens_stay_by_themselves(env):
    q, torch, dev = env
    g = np.random.default_rng(1)
    for T in (16, 1040, 2080):
        x = torch.randn((T, 256), device=dev).to(torch.bfloat16)
        x[3, 7], x[5, 9], x[7] = math.nan, math.inf, 3e38
        A = torch.randn((16, 256), device=dev).to(torch.bfloat16)
        B = torch.randn((16, 64), device=dev).to(torch.bfloat16)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        p = _plan(env, np.zeros(T), 1)
        clean = x.clone()
        clean[[3, 5, 7]] = 0
        ys = []
        for v in (x, clean):
            y = torch.ones((T, 64), device=dev)
            q.Lora(p, i32([[0, 16]]), torch.ones(1, device=dev), v, [(A, B, y)], max_rank=16).run()
            ys.append(y)
        keep = [t for t in range(T) if t not in (3, 5, 7)]
        assert torch.equal(ys[0][keep], ys[1][keep]) and bool(torch.isfinite(ys[0][keep]).all())
        assert bool(torch.isnan(ys[0][3]).all()) and not bool(torch.isfinite(ys[0][5]).any())
    # an infinite value between the products stays infinite: one rank row, so h = +-inf and y = +-inf
    x = torch.full((1, 64), 3e38, device=dev).to(torch.bfloat16)
    A = torch.ones((1, 64), device=dev).to(torch.bfloat16)
    B = torch.tensor([[1.0, -2.0, 0.5, 4.0]], device=dev).to(torch.bfloat16)
    B = torch.nn.functional.pad(B, (0, 4))[:, :4]
    y = torch.zeros((1, 4), device=dev)
    q.Lora(_plan(env, [0], 1), torch.tensor([[0, 1]], dtype=torch.int32, device=dev), torch.ones(1, device=dev), x, [(A, B, y)], max_rank=1).run()
    assert y[0].tolist() == [math.inf, -math.inf, math.inf, math.inf]


@pytest.mark.parametrize("T", [20, 1100, 2100])
@pytest.mark.parametrize("what", ["rows", "negative", "rank", "below", "tile", "count", "place", "adapter"])
def test_lora_leaves_out_what_is_corrupt(env, T, what):
    """A table, tile or place outside its array is reported, nothing of it is read or written, and the others are served."""
    from oracle import step
    q, torch, dev = env
    ids = [t % 2 for t in range(T)]
    g = np.random.default_rng(3)
    A = torch.randn((40, 128), device=dev).to(torch.bfloat16)
    B = torch.randn((40, 96), device=dev).to(torch.bfloat16)
    x = torch.randn((T, 128), device=dev).to(torch.bfloat16)
    table = torch.tensor([[3, 8], [20, 16]], dtype=torch.int32, device=dev)
    scale = torch.ones(2, device=dev)
    good, y = torch.ones((T, 96), device=dev), torch.ones((T, 96), device=dev)
    p = _plan(env, ids, 2)
    q.Lora(p, table, scale, x, [(A, B, good)], max_rank=16).run()
    assert q.qmv_check_status() == 0
    gone = [t for t in range(T) if ids[t] == 0]
    table, n0 = table.clone(), int((p.tiles[:, 0] == 0).logical_and(p.tiles[:, 2] > 0).sum())
    if what == "rows":
        table[0, 0] = 33
    elif what == "negative":
        table[0, 0] = -1
    elif what == "rank":
        table[0, 1] = 17
    elif what == "below":
        table[0, 1] = -3
    elif what == "tile":
        p.tiles[:n0, 1] = T - p.tiles[:n0, 2] + 1
    elif what == "count":
        p.tiles[:n0, 2] = 65
    elif what == "place":
        p.order[torch.tensor([i for i in range(len(gone))], device=dev)] = torch.tensor([T, -7], dtype=torch.int32, device=dev).repeat(T)[:len(gone)]
    else:
        p.tiles[:n0, 0] = 2
    q.Lora(p, table, scale, x, [(A, B, y)], max_rank=16).run()
    assert q.qmv_check_status() == q.QMV_ERR_CORRUPT
    rest = [t for t in range(T) if t not in set(gone)]
    assert torch.equal(y[rest], good[rest]) and bool((y[gone] == 1).all())


def test_lora_more_tiles_than_blocks(env):
    """Clusters take several tiles each: many adapters with a token each, and empty entries of the list between the tasks."""
    g = np.random.default_rng(9)
    for T, A in [(1024, 1024), (1000, 600), (2000, 1000)]:
        ids = g.permutation(A)[np.arange(T) % A]
        _lora_case(env, ids, g.integers(1, 9, A), 64, [40, 24, 8], "f32", T)
    _lora_case(env, np.zeros(1024, dtype=int), np.full(1024, 3), 64, [40, 24], "f32", 4)


# ----------------------------------------------------------------------------- log probabilities

def _logprob_check(env, rows, kind, scale, tokens, top, ld=None, pad=math.nan):
    from oracle import step
    q, torch, dev = env
    rows = np.asarray(rows, dtype=np.float64)
    T, V = rows.shape
    x, _ = _guarded(torch, dev, T, V, kind, ld=ld, fill=pad)
    x.copy_(torch.from_numpy(rows))
    tok = torch.tensor(tokens, dtype=torch.int32, device=dev)
    call = q.LogProb(x, tok, top=top, scale=scale)
    for t in (call.lse, call.entropy, call.logprob, call.rank, call.top_index, call.top_logprob):
        if t is not None:
            t.fill_(77)
    call.run()
    xv = _f64(x)
    scale = float(np.float32(scale))
    for i in range(T):
        lp, rank, lse, h, idx, vals = step.logprob(xv[i], scale, tokens[i], top)
        assert int(call.rank[i]) == rank, i
        if top:
            assert call.top_index[i].tolist() == idx, i
        # fp32: a power 2^d, d = (x - m) scale log2 e, is off by 3 steps of 2^-24 |d| (difference, product, constant) and 2^-22 (exp2); a sum of
        # n = V / 256 + 64 terms in a row by n 2^-24. Weighted by p, |d| is at most the entropy's and the maximum's share: log2 V + 1.
        n, bits = V / 256 + 64, math.log2(V) + 1
        rel = 2.0 ** -22 + n * 2.0 ** -24 + 3 * 2.0 ** -24 * bits
        pairs = [(float(call.lse[i]), lse, rel), (float(call.logprob[i]), lp, rel), (float(call.entropy[i]), h, 3 * rel * bits)]
        if top:
            pairs += [(float(call.top_logprob[i, j]), vals[j], rel) for j in range(top)]
        biggest = max([abs(v) * scale for v in xv[i] if math.isfinite(v)], default=0.0)
        for got, want, off in pairs:
            if math.isfinite(want):
                # the differences of large logits are rounded to their own step
                assert abs(got - want) <= off + 3 * 2.0 ** -24 * (abs(want) + 1) + (0 if off > rel else 2.0 ** -24 * biggest), (i, got, want)
            else:
                assert got == want or (math.isnan(got) and math.isnan(want)), (i, got, want)
    assert q.qmv_check_status() == 0
    return call


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 255, 1000, 4099, 20001])
@pytest.mark.parametrize("T,top", [(1, 0), (1, 1), (3, 20), (40, 5), (320, 32)])
def test_logprob(env, kind, V, T, top):
    if V * T > 10 ** 6:
        T = 40
    g = np.random.default_rng(V * 31 + T)
    rows = g.standard_normal((T, V)) * 3
    rows[:, g.integers(0, V, 3)] += 8
    tokens = g.integers(0, V, T)
    tokens[::2] = rows[::2].argmax(1)
    _logprob_check(env, rows, kind, 0.8, tokens, min(top, V), ld=V + (T % 3))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 320])
def test_logprob_of_a_large_vocabulary(env, kind, T):
    """Rows cut over a cluster, and whole: sampled against each other and one row against the oracle."""
    q, torch, dev = env
    V = 131073
    g = torch.Generator(device=dev).manual_seed(V)
    x = (torch.randn((T, V), generator=g, device=dev) * 2.5).to(_type(torch, kind))
    tokens = torch.randint(0, V, (T,), generator=g, device=dev).to(torch.int32)
    whole = q.LogProb(x, tokens, top=32)
    whole.run()
    rows = [0, T // 2, T - 1]
    for r in sorted(set(rows)):
        one = _logprob_check(env, _f64(x[r:r + 1]), kind, 1.0, [int(tokens[r])], 32)
        assert torch.equal(one.top_index[0], whole.top_index[r]) and int(one.rank[0]) == int(whole.rank[r])
        for a, b in ((one.lse, whole.lse), (one.entropy, whole.entropy), (one.logprob, whole.logprob)):
            assert abs(float(a[0]) - float(b[r])) <= 1e-4


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [5, 700, 9000])
def test_logprob_special_values(env, kind, V):
    g = np.random.default_rng(V)
    inf, nan = math.inf, math.nan
    low = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38, "f16": -65504.0}[kind]
    base = np.round(g.standard_normal((16, V)) * 4)      # whole numbers: ties in plenty
    rows = base.copy()
    rows[0] = -inf                                       # nothing left
    rows[1] = low                                        # masked by the lowest value, all of it: an even row
    rows[2, 1:] = -inf                                   # one left
    rows[3, 2:] = low
    rows[4, 1::2] = -inf
    rows[5] = 0.0
    rows[5, ::2] = -0.0                                  # zeros of both signs are equal
    rows[6, 3] = nan
    rows[7, 2] = inf
    rows[8] = nan
    rows[9, :] = -inf
    rows[9, V - 1] = nan
    rows[10] = np.sort(base[10])                         # every value passes the ones before it
    rows[11] = np.sort(base[11])[::-1]
    rows[12] = 3.0
    rows[13, 0], rows[13, V - 1] = inf, inf
    rows[14] = 60000.0 if kind == "f16" else 1e30
    rows[15] = -low
    for tok in (0, 3, V - 1):
        for top in (1, 5):
            _logprob_check(env, rows, kind, 1.0, [tok] * 16, top, ld=V + 3)
    if kind != "f16":
        _logprob_check(env, rows[:14], kind, 0.25, [2] * 14, 4, ld=V + 1)


def test_logprob_sorted_rows_and_thresholds(env):
    """Long rows in which candidates keep coming, from one lane, from one warp, or equal ones."""
    V = 12000
    g = np.random.default_rng(2)
    up = np.arange(V) / 1000.0
    rows = np.stack([up, -up, np.where(np.arange(V) % 32 == 5, up, -1.0), np.where(np.arange(V) // 128 % 8 == 3, up, 0.0),
                     np.repeat(np.arange(V // 100), 100) * 0.5, g.permutation(up), np.full(V, 2.0), np.where(np.arange(V) > V - 20, up, -math.inf)])
    for top in (1, 31, 32):
        _logprob_check(env, rows, "f32", 1.0, g.integers(0, V, len(rows)), top)
    _logprob_check(env, np.repeat(rows, 50, 0)[:320], "bf16", 1.0, g.integers(0, V, 320), 32)


def test_logprob_padding_and_tokens_outside(env):
    q, torch, dev = env
    x = torch.randn((4, 100), device=dev)
    call = q.LogProb(x, torch.tensor([5, -1, 100, -2 ** 31], dtype=torch.int32, device=dev), top=2)
    call.run()
    assert q.qmv_check_status() == q.QMV_ERR_CORRUPT
    assert call.rank[1:].tolist() == [-1] * 3 and call.logprob[1:].tolist() == [0.0] * 3
    want = torch.log_softmax(x.double(), 1)
    assert abs(float(call.logprob[0]) - float(want[0, 5])) < 1e-5 and int(call.rank[0]) == int((x[0] > x[0, 5]).sum())
    bare = q.LogProb(x)
    bare.run()
    assert bare.logprob is None and torch.equal(bare.lse, call.lse) and torch.equal(bare.entropy, call.entropy)
    assert q.qmv_check_status() == 0


# ----------------------------------------------------------------------------- together

class _Step:
    """tokens -> packed embedding -> INT4 projection with adapters -> packed LM head with its adapter -> log probabilities."""

    def __init__(self, env, T, seed=0):
        q, torch, dev = env
        from quantized_gemv_unpack_gb300 import synth
        self.q, self.torch, self.T = q, torch, T
        gen = synth.torch_generator(seed, dev)
        H, V, A = 512, 900, 5
        self.H, self.V, self.A = H, V, A
        self.w = {}
        for name, n in (("head", V), ("proj", H)):
            d = q.qmv_pack_desc(q.QMV_INT4, n, H)
            buf = torch.empty(d.total_bytes, dtype=torch.uint8, device=dev)
            q.qmv_pack_int4(d, synth.student_t4_torch(gen, (n, H), device=dev), buf)
            self.w[name] = (d, buf)
        self.tokens = torch.zeros(T, dtype=torch.int32, device=dev)
        self.ids = torch.zeros(T, dtype=torch.int32, device=dev)
        self.table = torch.tensor([[0, 8], [8, 16], [24, 4], [28, 0], [30, 16]], dtype=torch.int32, device=dev)
        self.scale = torch.tensor([1.0, -0.5, 2.0, 1.0, 0.25], device=dev)
        new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.x, self.y, self.x2, self.logits = new(T, H, dt=torch.bfloat16), new(T, H), new(T, H, dt=torch.bfloat16), new(T, V)
        pool = lambda n: (torch.randn((48, n), generator=gen, device=dev) * 0.1).to(torch.bfloat16)  # noqa: E731
        self.pa, self.pb, self.ha, self.hb = pool(H), pool(H), pool(H), pool(904)[:, :V]
        self.plan = q.LoraPlan(self.ids, A)
        self.calls = [
            q.Embed(self.w["head"][0], self.w["head"][1], self.tokens, self.x, 20.0),
            self.plan,
            q.Batch(q.QMV_INT4, [(*self.w["proj"], self.x, self.y)], T),
            q.Lora(self.plan, self.table, self.scale, self.x, [(self.pa, self.pb, self.y)], max_rank=16)]
        self.head = [
            q.Batch(q.QMV_INT4, [(*self.w["head"], self.x2, self.logits)], T),
            q.Lora(self.plan, self.table, self.scale, self.x2, [(self.ha, self.hb, self.logits)], max_rank=16)]
        self.out = q.LogProb(self.logits, self.tokens, top=4)

    def run(self):
        for c in self.calls:
            c.run()
        self.x2.copy_(self.y)
        for c in self.head:
            c.run()
        self.out.run()

    def check(self):
        from oracle import int4, matvec, step
        x = _f64(self.x)
        w = {}
        for name, (d, buf) in self.w.items():
            codes, s16 = int4.unpack(buf.cpu().numpy().tobytes(), d.N, d.K)
            w[name] = int4.dequant(codes, s16)
        tok, ids = self.tokens.tolist(), self.ids.tolist()
        table, scale = self.table.tolist(), self.scale.double().tolist()
        e = step.embed(w["head"], tok, 20.0)
        assert np.all(np.abs(x - e) <= (HALF["bf16"] + 2.0 ** -23) * np.abs(e))
        for name, xin, y, a, b in (("proj", x, self.y, self.pa, self.pb), ("head", _f64(self.x2), self.logits, self.ha, self.hb)):
            base, B = matvec.matvec(w[name], xin)
            want, s1, s2 = step.lora(base, xin, ids, table, scale, _f64(a), _f64(b))
            assert np.all(np.abs(_f64(y) - want) <= 2e-3 * B + 1e-5 * (s1 + s2) + 2.0 ** -23 * np.abs(want))
        z = _f64(self.logits)
        for t in range(self.T):
            lp, rank, lse, h, idx, vals = step.logprob(z[t], 1.0, tok[t], 4)
            assert int(self.out.rank[t]) == rank and self.out.top_index[t].tolist() == idx
            assert abs(float(self.out.logprob[t]) - lp) <= 1e-4 and abs(float(self.out.entropy[t]) - h) <= 1e-4

    def fill(self, seed):
        g = self.torch.Generator().manual_seed(seed)
        r = self.torch.randint
        self.tokens.copy_(r(0, self.V, (self.T,), generator=g))
        self.ids.copy_(r(-1, self.A, (self.T,), generator=g))


@pytest.mark.parametrize("T", [1, 5, 16])
def test_step_together_and_in_a_graph(env, T):
    q, torch, dev = env
    s = _Step(env, T)
    s.fill(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (1, 2):
        s.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        s.check()
        got = [t.clone() for t in (s.logits, s.out.lse, s.out.entropy, s.out.logprob, s.out.top_logprob)]
        s.run()
        assert all(torch.equal(a, b) for a, b in zip(got, (s.logits, s.out.lse, s.out.entropy, s.out.logprob, s.out.top_logprob)))
    assert q.qmv_check_status() == 0


def test_two_streams_at_once(env):
    """Calls of the same kind on two streams share nothing: no workspace, no counters."""
    q, torch, dev = env
    a, b = _Step(env, 16, seed=1), _Step(env, 16, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.fill(5)
    b.fill(6)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert q.qmv_check_status() == 0


def test_streams_by_argument(env):
    q, torch, dev = env
    s = torch.cuda.Stream()
    d, packed, codes, s16 = _packed(env, "int4_lut", 40, 256, 3)
    tok = torch.tensor([1, 2], dtype=torch.int32, device=dev)
    out = torch.empty((2, 256), device=dev)
    torch.cuda.synchronize()
    q.qmv_embed(d, packed, tok, out, 1.0, stream=s)
    call = q.LogProb(out, tok)
    call.run(s)
    call.run(s.cuda_stream)
    s.synchronize()
    assert abs(float(call.lse[0]) - float(torch.logsumexp(out[0].double(), 0))) < 1e-5


# ----------------------------------------------------------------------------- sizes, workspaces and graphs

def test_rows_past_32_bits(env):
    """Rows whose offsets, in values and in bytes, are past 2^32."""
    from oracle import int4, step
    q, torch, dev = env
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    far = lambda rows, cols, ld, dt: torch.empty((rows - 1) * ld + cols, dtype=dt, device=dev).as_strided((rows, cols), (ld, 1))  # noqa: E731
    g = np.random.default_rng(4)
    # an embedding table of 4.5 GB whose last 16 rows, one group of the layout, are those of a small one; far rows of the result
    n, K = 2 ** 21 + 16, 4096
    small, packed, codes, s16 = _packed(env, "int4", 16, K, 3)
    d = q.qmv_pack_desc(q.QMV_INT4, n, K)
    big = torch.zeros(d.total_bytes, dtype=torch.uint8, device=dev)
    for i in (0, 1):
        of = lambda e: slice(e.off[i] + e.bytes[i] - small.bytes[i], e.off[i] + e.bytes[i])  # noqa: E731
        big[of(d)] = packed[of(small)]
    out = far(5, K, 2 ** 30 + 8, torch.float32)
    q.qmv_embed(d, big, i32([n - 1, 0, n - 16, n - 7, n - 2]), out, 1.0)
    w = torch.from_numpy(int4.dequant(codes, s16.view(np.uint16))).float().to(dev)
    assert torch.equal(out[[0, 2, 3, 4]], w[[15, 0, 9, 14]]) and not bool(out[1].any())
    del big, out
    # adapters of one tile and of many: rows of x, A, B and y
    for T, ld in ((3, 2 ** 31 + 8), (1300, 2 ** 23)):
        x, y = far(T, 64, ld, torch.bfloat16), far(T, 72, ld, torch.bfloat16)
        a, b = far(3, 64, 2 ** 31 + 8, torch.bfloat16), far(3, 72, 2 ** 31 + 8, torch.bfloat16)
        for t in (x, y, a, b):
            t.copy_(torch.from_numpy(g.standard_normal(tuple(t.shape))))
        was, ids = _f64(y), np.zeros(T, dtype=int)
        q.Lora(_plan(env, ids, 1), i32([[0, 3]]), torch.ones(1, device=dev), x, [(a, b, y)], max_rank=3).run()
        want, s1, s2 = step.lora(was, _f64(x), ids, [(0, 3)], [1.0], _f64(a), _f64(b))
        assert np.all(np.abs(_f64(y) - want) <= 2.0 ** -16 * (s1 + s2) + (HALF["bf16"] + 2.0 ** -20) * np.abs(want))
        del x, y, a, b
    torch.cuda.empty_cache()
    # logits: an odd stride
    x = far(3, 1000, 2 ** 31 + 5, torch.bfloat16)
    x.copy_(torch.from_numpy(g.standard_normal((3, 1000)) * 3))
    call = q.LogProb(x, i32([5, 999, 0]), top=3)
    call.run()
    for t in range(3):
        lp, rank, lse, h, idx, vals = step.logprob(_f64(x[t]), 1.0, (5, 999, 0)[t], 3)
        assert int(call.rank[t]) == rank and call.top_index[t].tolist() == idx
        assert abs(float(call.lse[t]) - lse) <= 1e-5 and abs(float(call.logprob[t]) - lp) <= 1e-5 and abs(float(call.entropy[t]) - h) <= 1e-4
    assert q.qmv_check_status() == 0
    del x
    torch.cuda.empty_cache()


def test_no_tokens(env):
    q, torch, dev = env
    empty = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
    d, packed, codes, s16 = _packed(env, "int4", 16, 128, 3)
    ids = empty(0, dt=torch.int32)
    q.qmv_embed(d, packed, ids, empty(0, 128), 1.0)
    plan = q.LoraPlan(ids, 4)
    plan.run()
    a, b = empty(4, 64, dt=torch.bfloat16), empty(4, 8, dt=torch.bfloat16)
    q.Lora(plan, torch.zeros((4, 2), dtype=torch.int32, device=dev), empty(4), empty(0, 64, dt=torch.bfloat16), [(a, b, empty(0, 8))]).run()
    q.LogProb(empty(0, 50), ids, top=3).run()
    torch.cuda.synchronize()
    assert q.qmv_check_status() == 0


def test_lora_long_runs_of_an_adapter(env):
    """Many tokens: runs and windows that end inside the list, adapters that end inside a run, and rows without an adapter."""
    g = np.random.default_rng(11)
    for T, A, K, Ns, kind, rank in [(9000, 1, 40, [40], "f32", 5), (5000, 3, 104, [264, 16], "bf16", 33), (2500, 7, 72, [33], "f16", 100), (1537, 2, 2048, [300], "f32", 64)]:
        ids = np.sort(g.integers(-1, A, T))
        ids[g.integers(0, T, 9)] = -1
        _lora_case(env, ids, np.maximum(g.integers(0, rank + 1, A), np.arange(A) == 0), K, Ns, kind, T, max_rank=rank, magnitude=0.1)


class _Prompt:
    """Two layers' adapters of a prompt chunk, on one workspace, with the step's plan."""

    def __init__(self, env, T=1500, seed=0):
        q, torch, dev = env
        self.env, self.T, self.A = env, T, 6
        g = torch.Generator(device=dev).manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
        self.ids = torch.zeros(T, dtype=torch.int32, device=dev)
        self.table = torch.tensor([[0, 16], [16, 7], [23, 1], [24, 0], [30, 12], [4, 16]], dtype=torch.int32, device=dev)
        self.scale = torch.tensor([1.0, -0.5, 2.0, 1.0, 0.25, 1.5], device=dev)
        self.x, self.a, self.b = new(T, 256), [new(48, 256), new(48, 200)], [new(48, 200), new(48, 264)]
        self.y0 = [torch.randn((T, n), generator=g, device=dev) for n in (200, 264)]
        self.y = [torch.empty_like(y) for y in self.y0]
        self.mid = torch.empty((T, 200), dtype=torch.bfloat16, device=dev)
        self.plan = q.LoraPlan(self.ids, self.A)
        first = q.Lora(self.plan, self.table, self.scale, self.x, [(self.a[0], self.b[0], self.y[0])], max_rank=16)
        assert first.workspace.numel() > 0
        self.calls = [first, q.Lora(self.plan, self.table, self.scale, self.mid, [(self.a[1], self.b[1], self.y[1])], max_rank=16, workspace=first.workspace)]

    def run(self):
        for y, y0 in zip(self.y, self.y0):
            y.copy_(y0)
        self.plan.run()
        self.calls[0].run()
        self.mid.copy_(self.y[0])
        self.calls[1].run()

    def check(self):
        from oracle import step
        for x, a, b, y, y0 in zip((self.x, self.mid), self.a, self.b, self.y, self.y0):
            want, s1, s2 = step.lora(_f64(y0), _f64(x), self.ids.tolist(), self.table.tolist(), self.scale.double().tolist(), _f64(a), _f64(b))
            # K / 16 matrix products with 16 additions inside and 16 joins, then 26, each within 2^-23; y's rounding
            assert np.all(np.abs(_f64(y) - want) <= (x.shape[1] / 16 + 32) * 2.0 ** -23 * s1 + 42 * 2.0 ** -23 * s2 + 2.0 ** -22 * np.abs(want) + 1e-30)

    def fill(self, seed):
        torch = self.env[1]
        self.ids.copy_(torch.randint(-1, self.A, (self.T,), generator=torch.Generator().manual_seed(seed)))


def test_lora_many_tokens_in_graphs_and_on_streams(env):
    """A chunk's calls captured twice over one workspace, replayed on other ids, and run eagerly on streams of their own."""
    q, torch, dev = env
    s = _Prompt(env)
    s.fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    s.check()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gr in graphs:
        with torch.cuda.graph(gr):
            s.run()
    for seed in (1, 2):
        s.fill(seed)
        graphs[seed % 2].replay()
        graphs[(seed + 1) % 2].replay()
        torch.cuda.synchronize()
        s.check()
        got = [y.clone() for y in s.y]
        s.run()
        assert all(torch.equal(a, b) for a, b in zip(got, s.y))
    other = _Prompt(env, seed=7)
    other.fill(3)
    two = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            s.run()
        with torch.cuda.stream(two):
            other.run()
    torch.cuda.synchronize()
    s.check()
    other.check()
    assert q.qmv_check_status() == 0


@pytest.mark.parametrize("T", [40, 1100, 1500])
def test_lora_of_a_longer_list_of_tiles(env, T):
    """max_tiles past what the split can need: the plan empties the rest, and the workspace does not have to grow with it."""
    q, torch, dev = env
    g = torch.Generator(device=dev).manual_seed(T)
    new = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    x, a, b = new(T, 128), new(20, 128), new(20, 72)
    ids = torch.randint(-1, 3, (T,), generator=g, device=dev).to(torch.int32)
    table, scale = torch.tensor([[0, 8], [8, 5], [13, 7]], dtype=torch.int32, device=dev), torch.ones(3, device=dev)
    want, y = torch.ones((T, 72), device=dev), torch.ones((T, 72), device=dev)
    plan = q.LoraPlan(ids, 3)
    plan.run()
    q.Lora(plan, table, scale, x, [(a, b, want)], max_rank=8).run()
    few = plan.tiles
    plan.tiles = torch.full((few.shape[0] + 500, 4), -9, dtype=torch.int32, device=dev)
    plan.args.tiles, plan.args.max_tiles = plan.tiles.data_ptr(), plan.tiles.shape[0]
    plan.run()
    assert torch.equal(plan.tiles[:few.shape[0]], few) and not bool(plan.tiles[few.shape[0]:].any())
    call = q.Lora(plan, table, scale, x, [(a, b, y)], max_rank=8)
    assert call.args.max_tiles == few.shape[0] + 500 and call.workspace.numel() == q.lora_workspace_size(T, 3, 8, 1)
    room = torch.full((call.workspace.numel() + 4096,), 7, dtype=torch.uint8, device=dev)
    call.workspace = room
    if call.args.workspace:
        call.args.workspace = room.data_ptr()
    call.run()
    assert torch.equal(y, want) and bool((room[-4096:] == 7).all())
    assert q.qmv_check_status() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V", [(1, 131073), (70, 70001), (400, 40000)])
def test_logprob_alternatives_among_equal_values(env, kind, T, V):
    """More values at the threshold than are sorted at once, fewer that are not masked than alternatives, and exactly as many."""
    q, torch, dev = env
    g = torch.Generator(device=dev).manual_seed(V)
    rows = [torch.round(torch.randn((T, V), generator=g, device=dev) * 2), torch.full((T, V), -math.inf, device=dev), torch.full((T, V), 1.5, device=dev),
            torch.randn((T, V), generator=g, device=dev)]
    rows[1][:, [5, V // 2, V - 1]] = torch.tensor([1.0, 3.0, 1.0], device=dev)
    for n in (63, 64, 65, 300):                         # that many values share the first place
        x = torch.randn((T, V), generator=g, device=dev).clamp(max=3)
        x.scatter_(1, torch.rand((T, V), generator=g, device=dev).topk(n, dim=1).indices, 4.0)
        rows.append(x)
    for x in rows:
        x = x.to(_type(torch, kind))
        want = torch.sort(x, dim=1, descending=True, stable=True).indices
        for top in (1, 5, 32):
            call = q.LogProb(x, top=top)
            call.run()
            assert torch.equal(call.top_index.long(), want[:, :top])
            assert torch.equal(call.top_logprob.isinf(), torch.gather(x, 1, want[:, :top]).isinf())
    assert q.qmv_check_status() == 0
