"""Host-side checks of the KV cache calls (no GPU): layouts against the oracle, and refusals, which
are found before anything is launched."""
import ctypes
import math

import pytest

import quantized_gemv_unpack_gb300 as q
from oracle import kv8
from quantized_gemv_unpack_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return q.lib()


def _err(rc, want, text=""):
    assert rc == want, (rc, q.qmv_last_error())
    assert text in q.qmv_last_error()


def test_desc_matches_oracle(L):
    for kind in (q.QMV_KV_INT8, q.QMV_KV_E4M3):
        for pages, heads, D in [(1, 1, 64), (3, 8, 128), (1000001, 5, 64), (33554431, 1024, 128)]:
            d = q.kv8_desc(kind, pages, heads, D)
            off, size, total = kv8.sections(pages, heads, D)
            assert list(d.off) == off and list(d.bytes) == size and d.total_bytes == total and d.type == kind


@pytest.mark.parametrize("args,status", [((3, 1, 1, 64), -1), ((1, 0, 1, 64), -1), ((1, 1, 0, 64), -1), ((1, 1, 1025, 64), -1),
                                         ((1, 1, 1, 96), -3), ((1, 1 << 26, 1, 64), -3)])
def test_desc_refusals(L, args, status):
    with pytest.raises(q.QmvError) as e:
        q.kv8_desc(*args)
    assert e.value.status == status


def test_max_runs_bounds_every_split(L):
    for B in (1, 2, 5):
        for T in range(0, 400, 7):
            worst = 0
            # the most runs: every request with tokens starts at offset 63
            share = [T // B + (i < T % B) for i in range(B)]
            for n in share:
                worst += (63 + n - 1) // 64 + 1 if n else 0
            assert worst <= q.kv_max_runs(B, T) <= max(T, 0)
    assert q.kv_max_runs(0, 5) == 0


def test_rope_refusals(L):
    q.rope_desc(256, [1.0] * 128)
    for args in [dict(head_dim=24, inv_freq=[1.0] * 8), dict(head_dim=64, inv_freq=[1.0] * 40),
                 dict(head_dim=64, inv_freq=[1.0] * 9), dict(head_dim=272, inv_freq=[1.0] * 8),
                 dict(head_dim=64, inv_freq=[math.inf] * 8), dict(head_dim=64, inv_freq=[math.nan] * 8),
                 dict(head_dim=64, inv_freq=[1.0] * 8, axis=[5] * 8), dict(head_dim=64, inv_freq=[1.0] * 8, axis=[2] * 8, n_axes=2),
                 dict(head_dim=64, inv_freq=[])]:
        with pytest.raises(q.QmvError) as e:
            q.rope_desc(**args)
        assert e.value.status == q.QMV_ERR_ARG
    with pytest.raises(ValueError):
        q.rope_desc(512, [1.0] * 129)
    r = q.rope_desc(64, [1.0] * 32)
    run = lambda *a: L.rope_run(ctypes.byref(r), *a)  # noqa: E731
    ok = [256, q.QMV_BF16, 4, 2, 128, 256, 4, 512, q.QMV_BF16, 128, 0, None]
    for i, v, status in [(1, 9, -1), (8, 0, -1), (2, -1, -1), (3, 0, -1), (4, 120, -1), (9, 64, -1), (6, 3, -1), (4, 132, -2),
                         (0, 264, -2), (7, 260, -2), (5, 258, -2), (0, None, -1), (5, None, -1), (7, 256, 0)]:
        a = list(ok)
        a[i] = v
        if status == 0:      # in place with another stride
            a[9] = 136
            _err(run(*a), q.QMV_ERR_ARG, "in place")
        else:
            _err(run(*a), status)
    assert run(*(ok[:2] + [0] + ok[3:])) == q.QMV_OK      # no tokens: nothing to do
    assert L.rope_run(None, *ok) == q.QMV_ERR_ARG
    bad = q.qmv_rope.from_buffer_copy(r)
    bad.axis[3] = 1
    assert L.rope_run(ctypes.byref(bad), *ok) == q.QMV_ERR_ARG


def _filled(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


PLAN = dict(n_requests=2, n_tokens=10, n_pages=8, max_pages=4, ld_table=4, max_runs=10, lens=256, add=256, table=256, ring=256,
            ring_state=256, ring_state_out=256, lens_out=256, ctx=256, status=256, q_start=256, slots=256, positions=256, runs=256)


@pytest.mark.parametrize("field,value,status", [
    ("n_requests", 0, -1), ("n_requests", 8193, -1), ("n_tokens", -1, -1), ("n_pages", 0, -1), ("max_pages", 0, -1),
    ("ld_table", 3, -1), ("max_runs", 3, -1), ("lens", None, -1), ("ring_state_out", None, -1), ("slots", None, -1),
    ("runs", 260, -2), ("add", 258, -2), ("positions", 257, -2), ("n_pages", 1 << 26, -3)])
def test_plan_refusals(L, field, value, status):
    a = _filled(q.kv_plan_args, **{**PLAN, field: value})
    assert L.kv_plan(ctypes.byref(a), None) == status, q.qmv_last_error()
    assert L.kv_plan(None, None) == q.QMV_ERR_ARG


APPEND = dict(k=256, v=256, ldk=128, ldv=128, x_type=q.QMV_BF16, n_tokens=4, n_runs=2, slots=256, runs=256)


@pytest.mark.parametrize("change,status", [
    (dict(x_type=0), -1), (dict(ldk=64), -1), (dict(ldv=132), -2), (dict(k=None), -1), (dict(v=264), -2), (dict(slots=257), -2),
    (dict(runs=260), -2), (dict(n_tokens=-1), -1), (dict(n_runs=-1), -1), (dict(q=256, q_out=256, n_q_heads=2, ldq=128, ldqo=128,
     q_out_type=q.QMV_BF16), -1)])
def test_append_refusals(L, change, status):
    d = q.kv8_desc(q.QMV_KV_INT8, 4, 2, 64)
    a = _filled(q.kv8_append_args, **{**APPEND, **change})
    assert L.kv8_append(ctypes.byref(d), 256, None, ctypes.byref(a), None) == status, q.qmv_last_error()


def test_append_rope_refusals(L):
    d = q.kv8_desc(q.QMV_KV_INT8, 4, 2, 64)
    r, other = q.rope_desc(64, [1.0] * 32), q.rope_desc(128, [1.0] * 32)
    base = {**APPEND, "positions": 256, "ldp": 4, "q": 512, "q_out": 1024, "n_q_heads": 4, "ldq": 256, "ldqo": 256,
            "q_out_type": q.QMV_BF16}
    for change, rope, status in [({}, other, -1), (dict(ldp=3), r, -1), (dict(positions=None), r, -1), (dict(q_out=None), r, -1),
                                 (dict(n_q_heads=0), r, -1), (dict(ldq=128), r, -1), (dict(ldqo=260), r, -2),
                                 (dict(q_out_type=7), r, -1), (dict(q_out=512, q_out_type=q.QMV_F16), r, -1)]:
        a = _filled(q.kv8_append_args, **{**base, **change})
        assert L.kv8_append(ctypes.byref(d), 256, ctypes.byref(rope), ctypes.byref(a), None) == status, (change, q.qmv_last_error())
    bad = q.qmv_kv_desc.from_buffer_copy(d)
    bad.off[1] += 256
    a = _filled(q.kv8_append_args, **APPEND)
    assert L.kv8_append(ctypes.byref(bad), 256, None, ctypes.byref(a), None) == q.QMV_ERR_ARG
    assert L.kv8_append(ctypes.byref(d), None, None, ctypes.byref(a), None) == q.QMV_ERR_ARG


def test_read_refusals(L):
    d = q.kv8_desc(q.QMV_KV_E4M3, 4, 2, 64)
    ok = [256, 256, 3, 256, 512, q.QMV_F32, 128, None]
    for i, v, status in [(0, None, -1), (1, 258, -2), (2, -1, -1), (3, 260, -2), (5, 0, -1), (6, 64, -1), (6, 130, -2)]:
        a = list(ok)
        a[i] = v
        assert L.kv8_read(ctypes.byref(d), *a) == status, (i, q.qmv_last_error())
    assert L.kv8_read(ctypes.byref(d), 256, None, 0, None, None, q.QMV_F32, 128, None) == q.QMV_OK


ATTEND = dict(q=256, out=256, ldq=256, ldo=256, x_type=q.QMV_BF16, out_type=q.QMV_BF16, n_requests=2, n_tokens=4, n_q_heads=4,
              max_new=2, q_start=256, ctx=256, table=256, ld_table=4, max_pages=4, scale=0.1, workspace=256, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(n_q_heads=3), -1), (dict(n_q_heads=0), -1), (dict(n_requests=0), -1), (dict(n_requests=9000), -1), (dict(max_new=0), -1),
    (dict(n_tokens=-1), -1), (dict(x_type=9), -1), (dict(out_type=0), -1), (dict(ldq=128), -1), (dict(ldo=260), -2), (dict(q=None), -1),
    (dict(out=264), -2), (dict(ctx=257), -2), (dict(window=-1), -1), (dict(scale=0.0), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(softcap=-1.0), -1), (dict(softcap=math.inf), -1), (dict(ld_table=3), -1), (dict(max_pages=0), -1),
    (dict(workspace=None), -1), (dict(workspace=264), -2), (dict(ws_bytes=100), -1), (dict(slopes=258), -2), (dict(lse=258), -2),
    (dict(n_tokens=1 << 30), -3)])
def test_attend_refusals(L, change, status):
    d = q.kv8_desc(q.QMV_KV_INT8, 4, 2, 64)
    a = _filled(q.kv8_attend_args, **{**ATTEND, **change})
    assert L.kv8_attend(ctypes.byref(d), 256, ctypes.byref(a), None) == status, q.qmv_last_error()
    assert L.kv8_attend(None, 256, ctypes.byref(a), None) == q.QMV_ERR_ARG
    assert L.kv8_attend(ctypes.byref(d), 256, None, None) == q.QMV_ERR_ARG
    assert L.kv8_attend_init(ctypes.byref(d), None, 1 << 40, None) == q.QMV_ERR_ARG


def test_binding_refuses_wrong_tensors(L):
    import torch
    d = q.kv8_desc(q.QMV_KV_INT8, 4, 2, 64)
    cache = torch.zeros(d.total_bytes, dtype=torch.uint8)
    k = torch.zeros((3, 2, 64))
    slots, runs = torch.zeros(3, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    q.KvAppend(d, cache, k, k, slots, runs)
    with pytest.raises(ValueError):
        q.KvAppend(d, cache[:-1], k, k, slots, runs)
    with pytest.raises(ValueError):
        q.KvAppend(d, cache, k[:, :1], k, slots, runs)
    with pytest.raises(ValueError):
        q.KvAppend(d, cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots, runs)
    with pytest.raises(TypeError):
        q.KvAppend(d, cache, k, k.half(), slots, runs)
    with pytest.raises(TypeError):
        q.KvAppend(d, cache, k, k, slots.long(), runs)
    with pytest.raises(ValueError):
        q.KvAppend(d, cache, k, k, slots[:2], runs)
    with pytest.raises(TypeError):
        q.Rope(q.rope_desc(64, [1.0] * 32), k.double(), slots, k)
    with pytest.raises(ValueError):
        q.Rope(q.rope_desc(64, [1.0] * 32), k, slots[:2], k)
    with pytest.raises(ValueError):
        q.Rope(q.rope_desc(64, [1.0] * 32, axis=[1] * 32), k, slots, k)


def test_append_refuses_more_runs_than_it_numbers(L):
    """Runs times heads past 31 bits, before anything is launched (the rotation of q among it)."""
    r = q.rope_desc(64, [1.0] * 32)
    for H, n_runs in ((2, 2 ** 31 - 1), (1024, 2 ** 21), (8, 2 ** 28), (1, 2 ** 30)):
        d = q.kv8_desc(q.QMV_KV_INT8, 4, H, 64)
        for n_tokens in (1, 4):
            a = _filled(q.kv8_append_args, **{**APPEND, "ldk": 64 * H, "ldv": 64 * H, "n_runs": n_runs, "n_tokens": n_tokens, "positions": 256, "ldp": 4,
                                              "q": 512, "q_out": 1024, "n_q_heads": 4, "ldq": 256, "ldqo": 256, "q_out_type": q.QMV_BF16})
            assert L.kv8_append(ctypes.byref(d), 256, ctypes.byref(r), ctypes.byref(a), None) == q.QMV_ERR_UNSUPPORTED, q.qmv_last_error()


def test_plan_held_refusals(L):
    for change, status in [(dict(held=256), -1), (dict(held_out=256), -1), (dict(held=258, held_out=256), -2), (dict(held=256, held_out=257), -2)]:
        a = _filled(q.kv_plan_args, **{**PLAN, **change})
        assert L.kv_plan(ctypes.byref(a), None) == status, q.qmv_last_error()
    import torch
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q.KvPlan(i32(2), i32(2), i32(2, 4), i32(8), i32(2), 5, held=i32(2))
    with pytest.raises(ValueError):
        q.KvPlan(i32(2), i32(2), i32(2, 4), i32(8), i32(2), 5, held_out=i32(2))
    with pytest.raises(ValueError):
        q.KvPlan(i32(2), i32(2), i32(2, 4), i32(8), i32(2), 5, held=i32(3))
