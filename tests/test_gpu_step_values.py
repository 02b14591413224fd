"""GPU values of logprob_run and lora_run outside the ordinary: finite masks and logits of any magnitude, infinite factors, what
the fp32 values between the products keep, large sizes and pools, empty entries in a list of tiles. Against the definitions in 64 bits."""
import math

import numpy as np
import pytest

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


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


# ----------------------------------------------------------------------------- log probabilities

def _logprob(x, scale, token, top):
    """(lse, entropy, log probability, top's log probabilities, top's indices, rank) of a row without NaN and +inf."""
    z = x * scale
    m = z.max()
    if m == -math.inf:
        return -math.inf, 0.0, -math.inf, np.full(top, -math.inf), np.arange(top), token
    e = np.exp(z - m)
    ln_s = math.log(math.fsum(e))
    lp = (z - m) - ln_s
    seq = np.lexsort((np.arange(len(x)), -x))
    return m + ln_s, math.fsum(-np.exp(v) * v for v in lp[lp > -800]), lp[token], lp[seq[:top]], seq[:top], int(np.flatnonzero(seq == token)[0])


def _logprob_rows(env, rows, kind, scale, tokens, top, copies):
    """Rows, each `copies` times, against the definition. Copies lie alike in memory and have the same bits."""
    q, torch, dev = env
    n, V = rows.shape
    ld = (V + 15) // 8 * 8
    x = torch.full((n * copies, ld), math.nan, dtype=_type(torch, kind), device=dev)[:, :V]
    x.copy_(torch.from_numpy(np.tile(rows, (copies, 1))))
    call = q.LogProb(x, torch.tensor(list(tokens) * copies, dtype=torch.int32, device=dev), top=top, scale=scale)
    call.run()
    assert q.qmv_check_status() == 0
    outs = [call.lse, call.entropy, call.logprob, call.rank] + ([call.top_logprob, call.top_index] if top else [])
    for o in outs:
        assert torch.equal(o.view(torch.int32)[n:], o.view(torch.int32)[:n].repeat((copies - 1,) + (1,) * (o.dim() - 1)))
    xv, scale = _f64(x[:n]), float(np.float32(scale))
    for i in range(n):
        lse, h, lp, best, at, rank = _logprob(xv[i], scale, tokens[i], top)
        # fp32: a power 2^d, d = (x - m) scale log2 e, is off by 3 steps of 2^-24 |d| (difference, product, constant) and by 2^-22 (exp2). Where d is
        # taken from the rounded product P of the maximum it has what the rounding took, r <= P 2^-24, in it: another step of 2^-24 |d|, since
        # values that differ from the maximum are at least as far from it. A sum of n = V / 256 + 64 terms in a row is off by n 2^-24, the
        # entropy's by that of r too, which is at most 2^6. Weighted by p, |d| is at most log2 V + 1. Then the last sums and products, each
        # within 2^-24 of the result or of ln S.
        n_sum, bits = V / 256 + 64, math.log2(V) + 1
        rel = 2.0 ** -22 + n_sum * 2.0 ** -24 + 4 * 2.0 ** -24 * bits
        rest = min(2.0 ** 6, abs(float(xv[i].max())) * scale * math.log2(math.e) * 2.0 ** -24)
        pairs = [(float(call.lse[i]), lse, rel), (float(call.logprob[i]), lp, rel), (float(call.entropy[i]), h, 3 * rel * bits + n_sum * 2.0 ** -24 * rest)]
        pairs += [(float(call.top_logprob[i, j]), best[j], rel) for j in range(top)]
        for k, (got, want, off) in enumerate(pairs):
            if abs(want) < 3.4e38:
                assert abs(got - want) <= off + 3 * 2.0 ** -24 * (abs(want) + bits), (i, k, got, want)
            else:
                assert got == math.copysign(math.inf, want), (i, k, got, want)
        assert int(call.rank[i]) == rank, i
        if top:
            assert call.top_index[i].tolist() == at.tolist(), i


MASKS = {"f32": [-1e9, -1e10, -3e10, -1e12, -1e15, -1e20, -1e27, 1e10], "bf16": [-1e9, -1e10, -3e10, -1e12, -1e15, -1e20, -1e27, 1e10],
         "f16": [-65504.0, -60000.0, -49000.0, -2048.0, 60000.0]}


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [0.8, 1.0, 1.25, 1e5, 5e5])
@pytest.mark.parametrize("V,copies", [(9001, 1), (9001, 40), (70001, 1)])
def test_logprob_of_large_finite_values(env, kind, scale, V, copies):
    """Rows masked by a finite value: all of them, a thread's first values, a tail, nine tenths, all but a few; and likely values so large."""
    g = np.random.default_rng(V)
    for mask in MASKS[kind] if V < 10000 else MASKS[kind][1:4:2]:
        some = g.standard_normal((9, V)) * 3
        rows = some.copy()
        rows[0] = mask
        rows[1] = mask
        rows[1, V // 2] = some[1, 0]
        rows[2, :V * 2 // 3] = mask
        rows[3, V // 2:] = mask
        rows[4, g.random(V) < 0.9] = mask
        rows[5, g.random(V) < 0.999] = mask
        rows[6] = mask * (1 + np.round(some[6]) / 64) if kind != "f16" else mask + 32 * np.abs(np.round(some[6]))   # near one another, and large
        rows[7, g.random(V) < 0.5] = mask
        rows[7, g.random(V) < 0.5] = -math.inf
        rows[8, g.random(V) < 0.5] = -abs(mask) * 0.75
        if kind == "f16":
            rows = np.clip(rows, np.where(np.isinf(rows), -math.inf, -65504.0), 65504.0)
        tokens = [int(t) for t in g.integers(0, V, 9)]
        tokens[1], tokens[4] = V // 2, int(rows[4].argmax())
        for top in (0, 5):
            _logprob_rows(env, rows, kind, scale, tokens, top, copies)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [1.0, 0.4, 1e5])
@pytest.mark.parametrize("copies", [1, 40])
@pytest.mark.parametrize("bound,reach", [(20, 30.0), (24, 60.0), (27, 300.0), (31, 3000.0)])
def test_logprob_across_the_plain_bound(env, kind, scale, copies, bound, reach):
    """Values on both sides of where the maximum's product is 2^bound (and of half and twice it), in orders that cross it inside a thread, a warp and a block."""
    V = 9001
    g = np.random.default_rng(3)
    at = 2.0 ** bound / (scale * math.log2(math.e))
    rows = []
    for centre in (at, -at, 2 * at, -2 * at, at / 2):
        up = centre + np.linspace(-reach, reach, V) / scale
        rows += [up, up[::-1], g.permutation(up), np.where(g.random(V) < 0.5, up, -math.inf)]
    rows = np.stack(rows)
    if kind == "f16":
        rows = np.clip(rows, np.where(np.isinf(rows), -math.inf, -65504.0), 65504.0)
    for top in (0, 3):
        _logprob_rows(env, rows, kind, scale, [int(t) for t in g.integers(0, V, len(rows))], top, copies)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("copies", [1, 40])
def test_logprob_of_the_largest_values_under_a_small_scale(env, kind, copies):
    """The distance of two values is past what fp32 holds, their logits' is not."""
    V = 3001
    g = np.random.default_rng(5)
    for most, scale in [(3.3e38, 2e-38), (3.3e38, 1e-36), (1e38, 0.04)]:
        rows = np.stack([g.uniform(-most, most, V), np.where(g.random(V) < 0.5, most, -most), np.linspace(-most, most, V), np.linspace(most, -most, V)])
        for top in (0, 4):
            _logprob_rows(env, rows, kind, scale, [0, 5, V - 1, V - 1], top, copies)


def test_logprob_last_step(env):
    """n equal values in a row that is otherwise -inf: S = n exactly, so that of ln n only the logarithm is rounded."""
    q, torch, dev = env
    V, T = 5000, 600
    x = torch.full((T, V), -math.inf, device=dev)
    n = torch.arange(2, T + 2, device=dev)
    x[torch.arange(V, device=dev) * 7919 % V < n[:, None]] = 0.0
    call = q.LogProb(x, torch.zeros(T, dtype=torch.int32, device=dev), top=1)
    call.run()
    assert bool((call.rank == 0).all())
    want = torch.log(n.double())
    step = torch.exp2(torch.floor(torch.log2(want)) - 23)
    for got in (call.lse, call.entropy, -call.logprob, -call.top_logprob[:, 0]):
        assert bool(((got.double() - want).abs() <= step).all())                      # a logarithm is within a step


# ----------------------------------------------------------------------------- adapters

def _call(env, ids, table, scale, x, a, b, y, max_rank):
    q, torch, dev = env
    plan = q.LoraPlan(torch.as_tensor(np.asarray(ids, dtype=np.int32), device=dev), len(table))
    plan.run()
    call = q.Lora(plan, torch.as_tensor(np.asarray(table, dtype=np.int32), device=dev), torch.as_tensor(np.asarray(scale, dtype=np.float32), device=dev),
                  x, [(a, b, y)], max_rank=max_rank)
    call.run()
    assert q.qmv_check_status() == 0
    return call, plan


def _follows(got, want, bound):
    """got has want's NaN and infinities, and is within the bound elsewhere."""
    there = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.all(np.abs(got - want)[there] <= bound[there])


def _infinite_case(env, T, rank, max_rank, kind, seed, spoil):
    """Small whole factors of which spoil(x, a, b) makes some infinite: y as the definition has it."""
    q, torch, dev = env
    g = np.random.default_rng(seed)
    K, N, A = 64, 72, 3
    rows = A * rank + 2
    draw = lambda *s: g.integers(1, 4, s) * g.choice([-1.0, 1.0], s)  # noqa: E731
    x, a, b, y = draw(T, K), draw(rows, K), draw(rows, N), draw(T, N)
    spoil(x, a, b)
    x, a, b = (torch.from_numpy(v).to(torch.bfloat16).double().numpy() for v in (x, a, b))
    ids = np.arange(T) % A
    table = [(1 + i * rank, rank) for i in range(A)]
    scale = [1.0, -2.0, 0.5]
    t = lambda v, k="bf16": torch.from_numpy(v).to(_type(torch, k)).to(dev)  # noqa: E731
    yt = t(y, kind)
    _call(env, ids, table, scale, t(x), t(a), t(b), yt, max_rank)
    h = np.stack([a[f:f + r] @ x[i] for i in range(T) for f, r in [table[ids[i]]]])
    # value by value: a product of matrices may leave out what is 0
    own = [(f, f + r) for f, r in (table[i] for i in ids)]
    by = np.array(scale)[ids][:, None]
    want = y + by * np.stack([(h[i][:, None] * b[f:e]).sum(0) for i, (f, e) in enumerate(own)])
    s2 = np.abs(by) * np.stack([np.abs(h[i][:, None] * b[f:e]).sum(0) for i, (f, e) in enumerate(own)])
    # h is exact (64 products of 16 bits, of up to 9.3); then rank / 16 times three products with 16 additions inside, each within 2^-23 of what
    # is summed up; two parts leave 2^-17; y and its type
    bound = (3 * 8 + 16 + 2) * 2.0 ** -23 * s2 + (0 if kind == "f32" else 2.0 ** -17) * s2
    bound += (2.0 ** -23 if kind == "f32" else 2.0 ** -8 + 2.0 ** -24) * (np.abs(want) + bound)
    _follows(_f64(yt), want, bound)


SIZES = [(5, 16), (5, 32), (40, 64), (40, 128), (1300, 16), (1300, 32), (1300, 64), (1300, 128)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,max_rank", SIZES)
@pytest.mark.parametrize("rank", [1, 2, 8, 9, 12, 16, 17, 40, 100])
def test_lora_of_infinite_activations(env, kind, T, max_rank, rank):
    """An infinite x (or value of A) makes the values between infinite, of the ranks that there are and no others."""
    if rank > max_rank:
        rank = max_rank - 1

    def spoil(x, a, b):
        x[1, 5] = math.inf
        x[3, 63] = -math.inf
        a[1 + 2 * rank, 9] = math.inf                   # the first rank row of the third adapter
        b[:, ::2] = np.abs(b[:, ::2])                   # columns in which infinities may agree
        a[:, 5] = np.abs(a[:, 5])

    _infinite_case(env, T, rank, max_rank, kind, T + rank, spoil)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,max_rank", SIZES)
@pytest.mark.parametrize("rank", [1, 5, 16, 17, 64, 100])
def test_lora_of_infinite_columns(env, kind, T, max_rank, rank):
    """An infinite value of B makes its column infinite by the sign of the value that it is multiplied by, whatever parts that is held in."""
    if rank > max_rank:
        rank = max_rank - 1

    def spoil(x, a, b):
        b[0] = b[-1] = math.inf                         # rows of no adapter
        b[1, [0, 9, 31, 71]] = math.inf                 # of the first
        b[2 * rank, 8] = -math.inf                      # the second's last
        b[1 + 2 * rank, 40] = math.nan
        x[2, 7] = math.inf                              # meets it
        x *= 1 + 2.0 ** -7                              # values between of more bits than one part holds, rests of either sign
        a *= 1 + 2.0 ** -6 * (np.arange(64) % 2)

    _infinite_case(env, T, rank, max_rank, kind, T + rank, spoil)


@pytest.mark.parametrize("T", [20, 1300])
def test_lora_infinite_columns_leave_the_others(env, T):
    """Columns and tokens that an infinite value does not reach keep their bits."""
    q, torch, dev = env
    x, a, b = (torch.randn(s, device=dev).to(torch.bfloat16) for s in ((T, 200), (30, 200), (30, 104)))
    ids = np.arange(T) % 2
    ys = []
    for bad in (False, True):
        if bad:
            b[3, 17], x[4, 0] = math.inf, math.nan
        y = torch.ones((T, 104), device=dev)
        _call(env, ids, [(0, 12), (12, 18)], [1.0, 0.5], x, a, b, y, 32)
        ys.append(y)
    keep = torch.ones((T, 104), dtype=torch.bool, device=dev)
    keep[::2, 17] = False
    keep[4] = False
    assert torch.equal(ys[0][keep], ys[1][keep]) and not bool(torch.isfinite(ys[1][::2, 17]).any()) and bool(torch.isnan(ys[1][4]).all())
    assert not bool(torch.isnan(ys[1][::2, 17]).sum() > 1)


@pytest.mark.parametrize("T,N", [(40, 300), (1100, 300), (2100, 300), (40000, 1100)])
def test_lora_empty_entries_inside_a_list(env, T, N):
    """An entry of no tokens is passed over, wherever it stands, by every kernel alike."""
    q, torch, dev = env
    x, a, b = (torch.randn(s, device=dev).to(torch.bfloat16) for s in ((T, 128), (20, 128), (20, 1104)))
    b = b[:, :N]
    ids = np.minimum(np.arange(T) // 16, 2)
    want, y = torch.ones((T, N), device=dev), torch.ones((T, N), device=dev)
    call, plan = _call(env, ids, [(0, 8), (8, 5), (13, 7)], [1.0, 0.5, 2.0], x, a, b, want, 16)
    call.tasks[0].y = y.data_ptr()
    used = int((plan.tiles[:, 2] > 0).sum())
    assert used > 2
    if used == plan.tiles.shape[0]:                     # no room for an empty one: the list's last is left out, and its tokens
        used -= 1
    t, n, o = plan.tiles[used - 1:used, 1:3].sum(), used, plan.order.long()
    gone = o[int(t):]
    gone = gone[gone >= 0]
    for at in (0, 1, 2):
        y.fill_(1)
        moved = torch.cat([plan.tiles[:at], torch.zeros_like(plan.tiles[:1]), plan.tiles[at:n], torch.zeros_like(plan.tiles[n + 1:])])
        keep = plan.tiles.clone()
        plan.tiles.copy_(moved)
        call.run()
        torch.cuda.synchronize()
        plan.tiles.copy_(keep)
        left = want.clone()
        left[gone] = 1
        assert torch.equal(y, left), at
    assert q.qmv_check_status() == 0


@pytest.mark.parametrize("T", [1, 20, 1300])
@pytest.mark.parametrize("rank", [1, 16, 30, 64, 128])
def test_lora_values_between_keep_their_bits(env, T, rank):
    """fp32 y: the values between the products have 24 bits, of which three bf16 parts keep all. One rank row of each adapter is at work, B is +-1 there:
    y is the value itself."""
    q, torch, dev = env
    g = np.random.default_rng(T + rank)
    K, N = 256, 96
    at = g.integers(0, rank, 2)                         # the rank rows at work
    a, b = np.zeros((2 * rank, K)), g.standard_normal((2 * rank, N))
    for i in range(2):
        # bytes with their upper bit set at three places of x: sums of whole numbers below 2^24, exact in any order
        a[i * rank + at[i], [3, 100, 250]] = g.integers(128, 256, 3)
        b[i * rank + at[i]] = g.choice([-1.0, 1.0], N)
    x = np.zeros((T, K))
    x[:, [3, 100, 250]] = [65536.0, 256.0, 1.0]
    x *= g.choice([0.25, 1.0, 2.0], (T, 1))
    ids = np.arange(T) % 2
    t = lambda v: torch.from_numpy(v).to(torch.bfloat16).to(dev)  # noqa: E731
    y = torch.zeros((T, N), device=dev)
    _call(env, ids, [(0, rank), (rank, rank)], [1.0, 1.0], t(x), t(a), t(b), y, rank)
    h = np.array([a[i * rank + at[i]] @ x[k] for k, i in enumerate(ids)])
    two = torch.from_numpy(h).to(torch.bfloat16).double()
    two += (torch.from_numpy(h) - two).to(torch.bfloat16).double()
    # a matrix product may cut what it adds at two bits below an fp32 sum's last: 2^-22. Two parts would be off by more.
    assert np.all(np.abs(_f64(y) - h[:, None] * b[ids * rank + at[ids]]) <= 2.0 ** -22 * h[:, None])
    assert T == 1 or np.max(np.abs(two.numpy() - h) / h) > 2.0 ** -22


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,A,pool,K,N,rank", [(70, 6, 6, 13824, 5120, 128), (1300, 4, 4, 5120, 13824, 64), (3, 2, 2, 5120, 13824, 16),
                                               (2000, 5, 512, 512, 1499, 16), (4100, 5, 1024, 256, 520, 24), (50, 5, 1024, 4096, 4096, 16)])
def test_lora_of_large_sizes_and_pools(env, kind, T, A, pool, K, N, rank):
    """Projections of a large model, and pools of many more adapters than a step uses, on which the kernels' choice goes."""
    q, torch, dev = env
    g = torch.Generator(device=dev).manual_seed(T)
    new = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    x, a, b = new(T, K), new(pool * rank, K), new(pool * rank, (N + 7) // 8 * 8)[:, :N]
    y0 = (torch.randn((T, N), generator=g, device=dev) * 30).to(_type(torch, kind))
    used = torch.randperm(pool, generator=g, device=dev)[:A].cpu().numpy()
    ids = used[np.sort(np.arange(T) * 7919 % A)]
    ranks = np.where(np.arange(pool) % 3 == 1, max(1, rank - 5), rank)
    table, scale = np.stack([np.arange(pool) * rank, ranks], 1), 0.5 + np.arange(pool) % 4
    y = y0.clone()
    _call(env, ids, table, scale, x, a, b, y, rank)
    for i in used:
        t = torch.from_numpy(np.flatnonzero(ids == i)).to(dev)
        f, r = table[i]
        A64, B64, X = a[f:f + r].double(), b[f:f + r].double(), x[t].double()
        h = X @ A64.T
        want = y0[t].double() + float(scale[i]) * (h @ B64)
        s1, s2 = float(scale[i]) * ((X.abs() @ A64.abs().T) @ B64.abs()), float(scale[i]) * (h.abs() @ B64.abs())
        # fp32 sums, each addition within a step (2^-23) of what is summed up: K / 16 matrix products with 16 additions inside and 16 joins, then
        # rank / 16 times three of them; two parts leave 2^-17 of the values between, three nothing; y once more and to its type
        bound = (K / 16 + 32) * 2.0 ** -23 * s1 + (3 * 8 + 16 + 2) * 2.0 ** -23 * s2 + (0 if kind == "f32" else 2.0 ** -17) * s2
        bound += (2.0 ** -24 + (0 if kind == "f32" else 2.0 ** -8)) * (want.abs() + bound)
        assert bool(((y[t].double() - want).abs() <= bound).all())
    assert q.qmv_check_status() == 0
