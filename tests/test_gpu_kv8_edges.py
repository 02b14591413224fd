"""GPU parity of the paged 8-bit KV cache calls at the ends of their ranges, with the float64 oracle.

The bounds are those of test_gpu_kv8.py unless a test derives its own.
"""
import math

import numpy as np
import pytest

from test_gpu_kv8 import ULP, _Case, _check_plan, _f64, _fresh_cache, _host, _plan_state, _q, _run_plan, _tt, env  # noqa: F401 (env is a fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


# ----------------------------------------------------------------------------- plan

@pytest.mark.parametrize("add", [[2 ** 29] * 4 + [1, 1], [2 ** 30, 2 ** 30, 1], [3, 2 ** 30 - 3, 2 ** 30, 1, 0, -1], [2 ** 31 - 1] * 70 + [1, 0, -1, 2],
                                 [1, 2 ** 31 - 1, -2 ** 31, 1], [2, 2 ** 30 + 1] * 150 + [1], [2 ** 24] * 200 + [0, 1], [5] + [2 ** 31 - 65] * 2000 + [1]])
@pytest.mark.parametrize("T", [0, 4, 700])
def test_plan_sums_past_31_bits(env, add, T):
    """Requests that ask for more than any call has are refused, and so is whoever comes after them, whatever the sum."""
    from oracle import kv8
    g = np.random.default_rng(len(add))
    B = len(add)
    lens, table, ring, head = _plan_state(g, B, 20, 3 * B + 40, B + 30, 128)
    add = np.array(add, dtype=np.int32)
    want = kv8.plan(lens, add, table, ring, head, B + 30, T, _q(env).kv_max_runs(B, T))
    _check_plan(_run_plan(env, lens, add, table, ring, head, B + 30, T), want)
    _check_plan(_run_plan(env, lens, add, table, ring, head, B + 30, T, in_place=True), want)


# ----------------------------------------------------------------------------- read

@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128)])
def test_read_of_negative_slots_gives_zeros(env, kind, H, D):
    """Any negative slot, alone or between others, as the slot map of a plan holds them."""
    q, torch, dev = env
    d, cache = _fresh_cache(env, kind, 4, H, D, fill=0x41)
    ref = _host(cache, d)
    g = np.random.default_rng(kind)
    ref.scales[:] = np.exp(g.standard_normal(ref.scales.shape))
    ref.codes[:] = g.integers(0, 126, ref.codes.shape)
    cache.copy_(torch.from_numpy(ref.buf))
    slots = [-1, 70, -2, -63, -64, -65, 71, 72, 255, -2 ** 31, 0, -2 ** 31 + 1, -1000, -1] + [-1 - 5 * i for i in range(60)] + [64, 3, -3]
    for out in ("f32", "bf16"):
        ko, vo = (torch.full((len(slots), H, D), 9.0, device=dev, dtype=_tt(torch, out)) for _ in range(2))
        q.KvRead(d, cache, torch.tensor(slots, dtype=torch.int32, device=dev), ko, vo).run()
        for w, o in ((0, ko), (1, vo)):
            want = np.stack([ref.page_values(s // 64, w)[:, s % 64] if s >= 0 else np.zeros((H, D)) for s in slots])
            assert np.all(np.abs(_f64(o) - want) <= ULP[out] * np.abs(want))
    assert q.qmv_check_status() == 0


# ----------------------------------------------------------------------------- append with rotation

def _check_rotated_append(env, kind, H, Hq, D, before, new, inter, rot, axes, x="f32", seed=0, pad=0):
    """A call that puts new[i] tokens behind before[i] in page i (a run each): the values that come back against the rotation
    in float64, as in test_gpu_kv8.py, and the tokens that were there."""
    q, torch, dev = env
    from oracle import kv8
    g = np.random.default_rng(seed)
    P = len(new)
    order = g.permutation(P + 2)[:P]
    d, cache = _fresh_cache(env, kind, P + 2, H, D)
    i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=dev)  # noqa: E731
    had = [int(order[p]) * 64 + i for p, n in enumerate(before) for i in range(n)]
    if had:
        first = torch.from_numpy((g.standard_normal((len(had), H, D)) * 0.1).astype(np.float32)).to(dev)
        at = np.concatenate([[0], np.cumsum([n for n in before if n])])
        q.KvAppend(d, cache, first, first, i32(had), i32([[at[i], at[i + 1] - at[i]] for i in range(len(at) - 1)])).run()
        old = _host(cache, d)
    slots, runs, t = [], [], 0
    for p, n in enumerate(new):
        slots += [int(order[p]) * 64 + before[p] + i for i in range(n)]
        runs.append([t, n])
        t += n
    T = len(slots)
    qkv = torch.from_numpy(g.standard_normal((T, Hq + 2 * H, D)).astype(np.float32)).to(dev).to(_tt(torch, x))
    pos = g.integers(0, 100000, (axes, T)).astype(np.int32)
    inv, axis = [500.0 ** (-i / (rot // 2)) for i in range(rot // 2)], [i * axes // (rot // 2) for i in range(rot // 2)]
    qo = torch.full((T, Hq, D), 9.0, device=dev)
    q.KvAppend(d, cache, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], i32(slots), i32(runs + [[0, 0]] * pad), rope=q.rope_desc(D, inv, axis=axis, interleaved=inter),
               positions=torch.from_numpy(pos).to(dev), q=qkv[:, :Hq], q_out=qo).run()
    v = _f64(qkv)
    y = kv8.rotate(v[:, :Hq + H], pos, inv, axis, inter)
    size = np.abs(v).max() * 2
    assert np.all(np.abs(_f64(qo) - y[:, :Hq]) <= 1e-6 * size)
    after = _host(cache, d)
    page, off = np.array(slots) // 64, np.array(slots) % 64
    for which, want in ((0, y[:, Hq:]), (1, v[:, Hq + H:])):
        sc = after.scales[page, :, which].astype(np.float64)[:, :, None]
        codes = np.stack([after.codes[page, h, which][np.arange(T)[:, None], after.at[which][off]] for h in range(H)], 1)
        got = kv8.decode(codes, kind) * sc
        step = 0.5 * sc if kind == 1 else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * sc)
        bad = np.abs(got - want) > step * (1 + 1e-5) + 2e-6 * size
        assert not bad.any(), (which, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
        # the scale is the run's largest magnitude over the code's, or what it was
        for p in range(P):
            rows = slice(runs[p][0], runs[p][0] + runs[p][1])
            top = np.abs(want[rows]).max((0, 2)) / (127 if kind == 1 else 448)
            was = old.scales[order[p], :, which] if before[p] else 0
            assert np.all(np.abs(after.scales[order[p], :, which] - np.maximum(top, was)) <= 2e-6 * size)
            if before[p]:
                a, b = old.page_values(order[p], which)[:, :before[p]], after.page_values(order[p], which)[:, :before[p]]
                s = after.scales[order[p], :, which].astype(np.float64)[:, None, None]
                assert np.all(np.abs(a - b) <= (0.5 * s if kind == 1 else np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * s)) * (1 + 1e-5))
    assert q.qmv_check_status() == 0


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("H,D,P", [(10, 128, 41), (10, 128, 83), (6, 128, 300), (10, 64, 90), (6, 64, 230), (10, 64, 300)])
def test_append_of_prompts_whose_heads_share_angles(env, kind, H, D, P):
    """Runs enough for blocks of 2, 4 and 8 heads (152 SMs), the last of them not full; full pages, pages that go on, short ones."""
    new = [[64, 64, 34, 1, 59, 20][p % 6] for p in range(P)]
    before = [[0, 0, 30, 63, 5, 17][p % 6] for p in range(P)]
    _check_rotated_append(env, kind, H, 3, D, before, new, P % 2 == 1, D if P % 3 else D - 32, 1 + P % 3, "bf16" if D == 128 else "f32", seed=P)


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("inter,rot,axes", [(False, 128, 1), (True, 64, 2), (False, 96, 3), (True, 128, 4), (True, 16, 1), (False, 16, 1)])
@pytest.mark.parametrize("H,D,Hq,x", [(2, 128, 10, "f32"), (3, 64, 33, "bf16"), (1, 128, 1, "f16")])
def test_append_of_single_tokens_rotates(env, kind, inter, rot, axes, H, D, Hq, x):
    """The kernel of a decode step with partial, interleaved and many-axis rotation; runs of one to five tokens."""
    rot = min(rot, D)
    new = [1, 1, 3, 1, 5, 2, 1, 1, 1]
    before = [0, 40, 61, 63, 10, 0, 1, 16, 33]
    _check_rotated_append(env, kind, H, Hq, D, before, new, inter, rot, axes, x, seed=rot + axes)
    _check_rotated_append(env, kind, H, Hq, D, before, new, inter, rot, axes, x, seed=rot, pad=9)


@pytest.mark.parametrize("inplace", [False, True])
def test_append_of_a_prompt_in_a_graph(env, inplace):
    """The rotation and the cache write of a prompt follow what made their inputs and precede what reads their outputs: steps
    of plan, append and read captured together and replayed, against the same calls with a wait after each."""
    q, torch, dev = env
    H, Hq, D, T = 4, 24, 128, 500
    rope = q.rope_desc(D, [50.0 ** (-i / 64) for i in range(64)])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731

    def make():
        d, cache = _fresh_cache(env, 1, 40, H, D, fill=0)
        lens, state = i32([0, 0]), i32([0, 40])
        p = q.KvPlan(lens, i32([T - 37, 37]), torch.full((2, 20), -1, dtype=torch.int32, device=dev), i32(list(range(40))), state, T,
                     lens_out=lens, ring_state_out=state)
        g = torch.Generator(device=dev).manual_seed(3)
        src = torch.randn((T, Hq + 2 * H, D), generator=g, device=dev)
        x = torch.zeros_like(src)
        qo = x[:, :Hq] if inplace else torch.zeros((T, Hq, D), device=dev)
        ko, vo = (torch.zeros((T, H, D), device=dev) for _ in range(2))
        calls = [p, q.KvAppend(d, cache, x[:, Hq:Hq + H], x[:, Hq + H:], p.slots, p.runs, rope=rope, positions=p.positions, q=x[:, :Hq], q_out=qo),
                 q.KvRead(d, cache, p.slots, ko, vo), q.Rope(rope, ko, p.positions, ko, inverse=True)]
        return src, x, qo, ko, vo, calls

    src, x, qo, ko, vo, calls = make()
    x.copy_(src)
    for c in calls:
        c.run()
        torch.cuda.synchronize()
    want = [t.clone() for t in (qo, ko, vo)]
    assert float((want[1] - src[:, Hq:Hq + H]).abs().max()) <= 0.02 * float(src.abs().max())
    src, x, qo, ko, vo, calls = make()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.copy_(src)
        for c in calls:
            c.run()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, (qo, ko, vo)))
    for _ in range(3):                         # and issued one behind the other
        src, x, qo, ko, vo, calls = make()
        x.copy_(src)
        for c in calls:
            c.run()
        assert all(torch.equal(a, b) for a, b in zip(want, (qo, ko, vo)))
    assert q.qmv_check_status() == 0


# ----------------------------------------------------------------------------- attention: items of the prompt kernel

@pytest.mark.parametrize("D,kind", [(64, 1), (128, 2)])
@pytest.mark.parametrize("B,H", [(700, 1), (400, 3), (60, 1)])
def test_prompts_of_two_row_tiles_among_many_of_one(env, D, kind, B, H):
    """One group of rows sits out item after item, while the other takes them as fast as it can."""
    g = np.random.default_rng(B)
    new = np.where(np.arange(B) % 11 == 0, 200, g.integers(33, 60, B))
    ctx = new + np.where(np.arange(B) % 11 == 0, 300, g.integers(0, 9, B))
    c = _Case(env, [int(v) for v in ctx], [int(v) for v in new], H, H, D, kind, seed=B)
    first = c.check()
    for _ in range(3):
        assert (c.run(workspace=c.call.workspace)[0] == first).all()


# ----------------------------------------------------------------------------- append: the smallest scales

@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("D", [64, 128])
def test_tiny_scales_grow_without_losing_what_is_there(env, kind, n, D):
    """Values whose scale is below the smallest normal number, then larger ones in the same page: a code of zero stays zero,
    no code is a NaN, and every value is off by half a step per rounding, with steps of 2^-126 at least."""
    q, torch, dev = env
    H, top = 2, (127 if kind == 1 else 448)
    d, cache = _fresh_cache(env, kind, 3, H, D)
    g = np.random.default_rng(kind * 7 + n)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    amps = [1e-40, 1e-38, 1e-37, 4e-37, 1.2e-36, 1e-35]
    if n == 20:
        amps = [1e-38, 3e-37, 1e-36]
    given, steps = [[], []], [[], []]
    for call, amp in enumerate(amps):
        x = (g.uniform(-1, 1, (2, n, H, D)) * amp).astype(np.float32)
        x[:, :, :, ::3] = 0
        x[:, :, :, 1] = np.float32(amp)
        k, v = (torch.from_numpy(a).to(dev) for a in x)
        q.KvAppend(d, cache, k, v, i32([64 + call * n + i for i in range(n)]), i32([[0, n]])).run()
        assert q.qmv_check_status() == 0
        h = _host(cache, d)
        for w in (0, 1):
            given[w].append(x[w].astype(np.float64))
            for s in steps[w]:
                s.append(h.scales[1, :, w].astype(np.float64))
            steps[w].append([h.scales[1, :, w].astype(np.float64)])
            assert np.all(h.scales[1, :, w] <= max(amp / top * (1 + 1e-6), 2.0 ** -126))
        if kind == 2:
            codes = np.stack([h.page_codes(1, w)[:, :(call + 1) * n] for w in (0, 1)])
            assert not ((codes & 127) == 127).any()
    out = [torch.empty((n * len(amps), H, D), device=dev) for _ in (0, 1)]
    q.KvRead(d, cache, i32([64 + i for i in range(n * len(amps))]), *out).run()
    for w in (0, 1):
        got = _f64(out[w]).reshape(len(amps), n, H, D)
        for call, x in enumerate(given[w]):
            assert not got[call][x == 0].any()
            off = 0.0
            for s in dict.fromkeys(tuple(s) for s in steps[w][call]):
                s = np.array(s)[:, None]
                off = off + (0.5 * s if kind == 1 else np.maximum(2.0 ** -4 * (np.abs(x) + off), 2.0 ** -10 * s)) * (1 + 1e-5)
            assert np.all(np.abs(got[call] - x) <= off + 2.0 ** -149 * 2), (call, np.abs(got[call] - x).max(), amps[call])


# ----------------------------------------------------------------------------- attention: the cap

@pytest.mark.parametrize("cap", [0.5, 200.0, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("new,Hq,H", [([5, 2, 1], 6, 2), ([90, 64, 33], 6, 2), ([70, 60, 40], 80, 40)])
def test_cap_is_exact_whatever_its_size(env, cap, new, Hq, H):
    """cap * tanh(s / cap) of scores far below, near and over the cap: the error is that of the score, not of the cap."""
    c = _Case(env, [513, 64, 200], new, Hq, H, 64, 1, "bf16", seed=len(str(cap)))
    cap = float(np.float32(cap))
    c.check(softcap=cap)
    c.check(softcap=cap, scale=8.0)
    c.check(softcap=cap, scale=0.01, slopes=[2.0 ** -(h % 8 + 2) for h in range(Hq)])


@pytest.mark.parametrize("new", [[3], [60]])
def test_smallest_cap(env, new):
    """A cap near the smallest normal number, and queries of zero."""
    c = _Case(env, [150], new, 4, 2, 128, seed=3)
    c.q[0] = 0
    c.q[2, 1] = 0
    c.check(softcap=float(np.float32(1.2e-38)))


# ----------------------------------------------------------------------------- attention: V scales of many sizes

def _check_v_scales(c, slopes=None, window=0, **opt):
    """Against float64 attention with a bound that knows what each key contributes: p s_v is held to 2^-11 of itself or 2^-33
    of the row's largest p s_v, so |do| <= (2^-11 + 2 d + 2^-20) sum p |v| + n 2^-33 max(p s_v) top (see _Case.check for d)."""
    kw = dict(window=window)
    if slopes is not None:
        kw["slopes"] = slopes
    o, lse = c.run(**kw, **opt)
    got = _f64(o)
    from oracle import kv8
    ref, want_lse, pv, _, n, sabs = kv8.attend(c.cache_ref, _f64(c.q), c.q_start, c.ctx, c.table, float(np.float32(c.D ** -0.5)), **kw)
    x = _f64(c.q)
    scale = float(np.float32(c.D ** -0.5))
    G = c.Hq // c.H
    most = np.zeros((len(x), c.Hq))
    for b, L in enumerate(c.ctx):
        t0, t1 = c.q_start[b], c.q_start[b + 1]
        pages = c.table[b, :-(-L // 64)]
        K = np.concatenate([c.cache_ref.page_values(p, 0) for p in pages], 1)[:, :L]
        sv = np.concatenate([np.repeat(c.cache_ref.scales[p, :, 1].astype(np.float64)[:, None], 64, 1) for p in pages], 1)[:, :L]
        key, pos = np.arange(L), (L - (t1 - t0) + np.arange(t1 - t0))[:, None]
        ok = (key <= pos) & ((pos - key < window) if window else True)
        for h in range(c.Hq):
            s = scale * (x[t0:t1, h] @ K[h // G].T)
            if slopes is not None:
                s = s - slopes[h] * np.abs(pos - key)
            p = np.where(ok, np.exp(s - want_lse[t0:t1, h][:, None]), 0.0)
            most[t0:t1, h] = (p * sv[h // G]).max(1)
    top = 127.0 if c.desc.type == 1 else 448.0
    big = sabs + np.where(np.isfinite(want_lse), np.abs(want_lse), 0)
    d = 2.0 ** -20 * big + 2.0 ** -21 + (2.0 ** -20 * np.max(slopes) * float(np.max(c.ctx)) if slopes is not None else 0)
    # the log of a V scale joins the exponent: up to 2^-20 of its magnitude
    ly = np.abs(np.log2(np.maximum(c.cache_ref.scales[c.table[c.table >= 0], :, 1], 1e-45))).max()
    d = d + 2.0 ** -20 * ly
    tol = (2.0 ** -11 + 2 * d + 2.0 ** -20)[..., None] * pv + (n * 2.0 ** -33 * most * top)[..., None]
    bad = np.abs(got - ref) > tol + 1e-37
    assert np.isfinite(got).all()
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
    assert np.all(np.abs(_f64(lse) - want_lse) <= 2 * d + 2.0 ** -20 * (1 + np.abs(want_lse)))


@pytest.mark.parametrize("factor", [1e-8, 1e3, 1e6, 1e8, 1e20, 1e30])
@pytest.mark.parametrize("Hq,H,D,kind,new", [(2, 2, 64, 1, 200), (80, 80, 64, 2, 200), (4, 2, 128, 1, 170), (40, 40, 128, 2, 170), (5, 1, 64, 1, 2)])
def test_a_page_that_a_row_does_not_see_leaves_it_alone(env, factor, Hq, H, D, kind, new):
    """An early page whose V scale is far from the rest, out of most rows' windows or far down their distance bias."""
    q, torch, dev = env
    c = _Case(env, [64 + new], [new], Hq, H, D, kind, "bf16", seed=5, spread=0.0)
    c.cache_ref.scales[c.table[0, 0], :, 1] *= np.float32(factor)
    c.cache.copy_(torch.from_numpy(c.cache_ref.buf))
    _check_v_scales(c, window=64)
    _check_v_scales(c, slopes=[1.0 + h / 64 for h in range(Hq)])
    _check_v_scales(c)


def test_v_scales_from_the_smallest_to_the_largest(env):
    """Every page its own size, rising and falling, with pages of zeros among them."""
    q, torch, dev = env
    for sizes in ([1e-37, 1e-30, 0.0, 1e-10, 1.0, 1e10, 1e30], [1e30, 1e10, 1.0, 0.0, 1e-10, 1e-30, 1e-37], [0.0] * 7, [1e-37] * 7):
        for Hq, H, new in ((2, 2, 200), (80, 80, 100), (2, 2, 3)):
            c = _Case(env, [420], [new], Hq, H, 64, 1, "bf16", seed=6, spread=0.0)
            for i, s in enumerate(sizes):
                c.cache_ref.scales[c.table[0, i], :, 1] = s
            c.cache.copy_(torch.from_numpy(c.cache_ref.buf))
            _check_v_scales(c, window=64)
            _check_v_scales(c)


# ----------------------------------------------------------------------------- attention: probabilities far below the largest

def _one_key_and_many(env, B, pages, new, H, D, kind, gap):
    """Every request reads the same pages: key 0 scores gap * log 2 and has the value 0, all others score 0 and have the
    value 1. Returns the call's arguments and the exact output of a row that sees n keys."""
    q, torch, dev = env
    d, cache = _fresh_cache(env, kind, pages, H, D, fill=128 if kind == 1 else 0)
    ref = _host(cache, d)
    one = 128 + 1 if kind == 1 else 0x38
    ref.scales[:] = 1.0
    for p in range(pages):
        ref.codes[p, :, 1] = one
    from oracle import kv8
    ref.codes[0, :, 0, kv8.k_byte(0, 0, D)] = one
    for at in range(D):
        ref.codes[0, :, 1, kv8.v_byte(0, at)] = 128 if kind == 1 else 0
    cache.copy_(torch.from_numpy(ref.buf))
    x = torch.zeros((B * new, H, D), device=dev)
    x[:, :, 0] = gap                      # an integer: exact in every type
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    ctx = pages * 64
    out = torch.zeros((B * new, H, D), device=dev)
    lse = torch.zeros((B * new, H), device=dev)
    call = q.KvAttend(d, cache, x, out, i32([b * new for b in range(B + 1)]), i32([ctx] * B), i32([list(range(pages))] * B), math.log(2),
                      max_new=new, lse=lse)
    call.run()
    n = np.tile(ctx - new + 1 + np.arange(new), B)
    rest = (n - 1) * 2.0 ** -gap
    return _f64(out), _f64(lse), (rest / (1 + rest))[:, None, None], (np.log1p(rest) + gap * math.log(2))[:, None], n[:, None, None]


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("B,new,H,D", [(1400, 1, 1, 64), (1300, 1, 1, 128), (700, 3, 2, 64), (700, 20, 1, 64), (80, 40, 1, 64), (80, 40, 1, 128),
                                       (3, 200, 1, 64), (1, 40, 1, 128)])
@pytest.mark.parametrize("gap", [20, 26, 28])
def test_many_keys_far_below_the_largest(env, kind, B, new, H, D, gap):
    """Thousands of keys of probability 2^-gap beside one: their sum is the output. A probability is held to 2^-11 of itself
    or 2^-33 of the largest, each value is 1, the scores are exact: |do| <= (2^-11 + 2^-19) o + n 2^-33."""
    out, lse, want, want_lse, n = _one_key_and_many(env, B, 64, new, H, D, kind, gap)
    assert np.all(np.abs(out - want) <= (2.0 ** -11 + 2.0 ** -19) * want + n * 2.0 ** -33), (out.ravel()[:4], want.ravel()[:4])
    assert np.all(np.abs(lse - want_lse) <= 2.0 ** -19 * want_lse)


# ----------------------------------------------------------------------------- attention: the window

@pytest.mark.parametrize("new", [[9, 4], [100, 90]])
def test_largest_window_and_rows_before_the_first_key(env, new):
    """Rows at negative positions see the prefix whatever the window; a window of 2^31 - 1 hides nothing."""
    c = _Case(env, [5, 70], new, 60, 30, 64, seed=7)
    want = c.check(prefix=[3, 20])
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 64):
        assert (c.check(prefix=[3, 20], window=window) == want).all()


# ----------------------------------------------------------------------------- attention: the workspace

@pytest.mark.parametrize("new", [[5], [20], [150]])
def test_workspace_made_on_another_stream(env, new):
    """The object and its workspace are made on a stream with work ahead, the call runs on another: the workspace is ready."""
    q, torch, dev = env
    c = _Case(env, [9000], new, 4, 1, 64, seed=sum(new))
    want, _ = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = torch.full_like(c.call.workspace, 0xFF)     # memory that the allocator gives out next, far from zero
    del junk
    c.call = None
    o = torch.full_like(want, 7.0)
    i32 = lambda v: torch.tensor(np.ascontiguousarray(v, dtype=np.int32), device=dev)  # noqa: E731
    args = [c.desc, c.cache, c.q, o, i32(c.q_start), i32(c.ctx), i32(c.table), 64 ** -0.5]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    call = q.KvAttend(*args, max_new=max(new))
    call.run(side)
    side.synchronize()
    assert torch.equal(o, want)
    torch.cuda._sleep(40_000_000)
    ws = q.kv8_workspace(c.desc, dev)
    o.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    q.KvAttend(*args, max_new=max(new), workspace=ws).run(side)
    side.synchronize()
    assert torch.equal(o, want) and int(ws[:16384].view(torch.int32).abs().sum()) == 0


def test_workspace_outlives_its_object_on_another_stream(env):
    """An object that is dropped while its call still waits on a side stream: its memory is not given to anyone before that."""
    q, torch, dev = env
    c = _Case(env, [9000], [5], 4, 1, 64, seed=2)
    want, _ = c.run()
    keep = c.call.keep
    c.call = None
    o = torch.full_like(want, 7.0)
    i32 = lambda v: torch.tensor(np.ascontiguousarray(v, dtype=np.int32), device=dev)  # noqa: E731
    args = [c.desc, c.cache, c.q, o, i32(c.q_start), i32(c.ctx), i32(c.table), 64 ** -0.5]
    call = q.KvAttend(*args, max_new=5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at, n = call.workspace.data_ptr(), call.workspace.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    call.run(side)
    del call
    other = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(o, want) and keep is not None


def test_workspace_made_aside_used_on_the_default_stream_and_in_a_capture(env):
    q, torch, dev = env
    c = _Case(env, [3000], [5], 4, 1, 64, seed=2)
    want, _ = c.run()
    o = torch.full_like(want, 7.0)
    i32 = lambda v: torch.tensor(np.ascontiguousarray(v, dtype=np.int32), device=dev)  # noqa: E731
    args = [c.desc, c.cache, c.q, o, i32(c.q_start), i32(c.ctx), i32(c.table), 64 ** -0.5]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call = q.KvAttend(*args, max_new=5)
    for _ in range(2):
        call.run()
        assert torch.equal(o, want)
        o.fill_(7.0)
    for inside in (False, True):
        call = q.KvAttend(*args, max_new=5)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if inside:
                call = q.KvAttend(*args, max_new=5)
            call.run()
        for _ in range(3):
            o.fill_(7.0)
            g.replay()
            assert torch.equal(o, want)
        del g


def test_plan_of_every_request_count(env):
    """The number of requests changes from call to call, down and up: each is planned, with the shared memory that it takes."""
    from oracle import kv8
    g = np.random.default_rng(4)
    for B in [8000, 5, 3000, 2457, 2458, 1, 8191] + list(range(250, 260)):
        lens, table, ring, head = _plan_state(g, B, 3, 2 * B + 9, 9, 64)
        add = np.where(g.random(B) < 0.01, 2, 0).astype(np.int32)
        T = int(add.sum())
        want = kv8.plan(lens, add, table, ring, head, 9, T, _q(env).kv_max_runs(B, T))
        _check_plan(_run_plan(env, lens, add, table, ring, head, 9, T), want)


# ----------------------------------------------------------------------------- plan: requests that are shortened

def _run_plan_held(env, lens, add, table, ring, head, count, T, held, in_place=False):
    q, torch, dev = env
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    l, st, h = t(lens), t([head, count]), t(held)
    p = q.KvPlan(l, t(add), t(table), t(ring), st, T, lens_out=l if in_place else None, ring_state_out=st if in_place else None, held=h,
                 held_out=h if in_place else None)
    p.run()
    torch.cuda.synchronize()
    return p


@pytest.mark.parametrize("B,max_len,new,free", [(1, 64, 1, 1), (3, 200, 5, 2), (64, 300, 90, 30), (257, 130, 3, 60), (2048, 500, 7, 300), (6, 300, 3000, 400)])
def test_plan_with_held_pages_matches_oracle(env, B, max_len, new, free):
    """Rows that hold more pages than their lengths fill, and counts that cannot be."""
    from oracle import kv8
    g = np.random.default_rng(B + new)
    cap = (max_len + new + 63) // 64 + 1
    N = B * (max_len // 64 + 1) + free + 5
    lens, table, ring, head = _plan_state(g, B, cap, N, free, max_len)
    held = -(-lens // 64)
    lens = np.maximum(lens - g.integers(0, 150, B), 0).astype(np.int32)
    add = g.integers(0, new + 1, B).astype(np.int32)
    add[g.random(B) < 0.15] = -1
    add[g.random(B) < 0.05] = cap * 64
    held[g.random(B) < 0.03] = cap + 1
    held[g.random(B) < 0.03] = -1
    T = int(np.maximum(add, 0).sum())
    want = kv8.plan(lens, add, table, ring, head, free, T, _q(env).kv_max_runs(B, T), held=held)
    for in_place in (False, True):
        p = _run_plan_held(env, lens, add, table, ring, head, free, T, held, in_place)
        _check_plan(p, want)
        assert p.held_out.tolist() == want["held_out"].tolist()


def test_plan_loses_no_page_of_rejected_drafts(env):
    """200 steps of drafts of which some are taken back, over page ends too: no page is owned twice, none is lost."""
    q, torch, dev = env
    from oracle import kv8
    g = np.random.default_rng(9)
    B, cap, N, T = 12, 8, 50, 300
    lens, held, table = np.zeros(B, dtype=np.int32), np.zeros(B, dtype=np.int32), np.full((B, cap), -1, dtype=np.int32)
    ring, head, count = np.arange(N, dtype=np.int32), 0, N
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    dl, dt, dr, ds, da, dh = t(lens), t(table), t(ring), t([head, count]), t(np.zeros(B)), t(held)
    p = q.KvPlan(dl, da, dt, dr, ds, T, lens_out=dl, ring_state_out=ds, held=dh, held_out=dh)
    for step in range(200):
        add = np.where(g.random(B) < 0.1, -1, g.integers(0, 26, B)).astype(np.int32)
        da.copy_(t(add))
        want = kv8.plan(lens, add, table, ring, head, count, T, q.kv_max_runs(B, T), held=held)
        p.run()
        torch.cuda.synchronize()
        _check_plan(p, want)
        lens, held, table, ring = (want[k].astype(np.int32) for k in ("lens_out", "held_out", "table", "ring"))
        assert p.held_out.tolist() == held.tolist()
        head, count = (int(v) for v in want["ring_state_out"])
        owned = [int(x) for b in range(B) for x in table[b, :held[b]]]
        assert sorted(owned + [int(ring[(head + i) % N]) for i in range(count)]) == list(range(N))
        lens = np.maximum(lens - np.where(g.random(B) < 0.5, g.integers(0, 100, B), 0), 0).astype(np.int32)   # rejected
        dl.copy_(t(lens))


# ----------------------------------------------------------------------------- together

def test_a_mixed_step_in_one_call_and_in_two(env):
    """Single tokens of many requests beside a prompt chunk: the cache write and the attention as one call each, and as one for
    the single tokens and one for the chunk over slices of the plan."""
    q, torch, dev = env
    H, Hq, D, n, chunk = 2, 10, 64, 19, 170
    g = np.random.default_rng(1)
    lens = g.integers(1, 300, n + 1)
    T = n + chunk
    i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=dev)  # noqa: E731
    need = -(-lens // 64)
    order = g.permutation(200)
    table = np.full((n + 1, 9), -1)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    p = q.KvPlan(i32(lens), i32([1] * n + [chunk]), i32(table), i32(np.concatenate([order[at:], np.full(at, -1)])), i32([0, 200 - at]), T)
    p.run()
    assert not p.status.any()
    gen = torch.Generator(device=dev).manual_seed(2)
    x = torch.randn((T, Hq + 2 * H, D), generator=gen, device=dev)
    rope = q.rope_desc(D, [100.0 ** (-i / 32) for i in range(32)])
    d, base = _fresh_cache(env, 1, 200, H, D)
    ref = _host(base, d)
    ref.scales[:] = 0.02
    ref.codes[:] = g.integers(1, 256, ref.codes.shape)
    base.copy_(torch.from_numpy(ref.buf))

    def append(cache, runs, with_q):
        qo = torch.zeros((T, Hq, D), device=dev, dtype=torch.bfloat16)
        kw = dict(q=x[:, :Hq], q_out=qo) if with_q else {}
        q.KvAppend(d, cache, x[:, Hq:Hq + H], x[:, Hq + H:], p.slots, runs, rope=rope, positions=p.positions, **kw).run()
        return qo

    one, two = base.clone(), base.clone()
    qo = append(one, p.runs, True)
    append(two, p.runs[:n], False)
    assert torch.equal(append(two, p.runs[n:], True), qo)
    a, b = _host(one, d), _host(two, d)
    full = np.concatenate([lens[:n] + 1, [lens[n] + chunk]])
    for r in range(n + 1):
        for i in range(-(-int(full[r]) // 64)):
            page, fill = int(p.table[r, i]), min(64, int(full[r]) - 64 * i)
            assert np.array_equal(a.scales[page], b.scales[page])
            for w in (0, 1):
                assert np.array_equal(a.page_codes(page, w)[:, :fill], b.page_codes(page, w)[:, :fill])
    outs = [torch.zeros((T, Hq, D), device=dev) for _ in range(2)]
    q.KvAttend(d, one, qo, outs[0], p.q_start, p.ctx, p.table, D ** -0.5, max_new=chunk).run()
    q.KvAttend(d, one, qo, outs[1], p.q_start[:n + 1], p.ctx[:n], p.table[:n], D ** -0.5, max_new=1).run()
    q.KvAttend(d, one, qo, outs[1], p.q_start[n:], p.ctx[n:], p.table[n:], D ** -0.5, max_new=chunk).run()
    assert torch.equal(outs[0][n:], outs[1][n:])
    # P in fp16 against references of different height: 2^-11 on either side
    assert float((outs[0] - outs[1]).abs().max()) <= 2.0 ** -9 * float(outs[0].abs().max())
    assert q.qmv_check_status() == 0
