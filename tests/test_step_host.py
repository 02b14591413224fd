"""Host-side checks of qmv_embed, lora_* and logprob_run (no GPU): sizes, and refusals, which are found before anything is
launched and leave every output as it was."""
import ctypes
import math

import pytest

import quantized_gemv_unpack_gb300 as q
from quantized_gemv_unpack_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return q.lib()


def _err(rc, want, text=""):
    assert rc == want, (rc, q.qmv_last_error())
    assert text in q.qmv_last_error()


def test_lora_tiles_bound_every_split(L):
    for T in (1, 2, 15, 16, 17, 100, 1023, 1024, 1025, 1279, 1280, 5000):
        tile = q.lora_tile(T)
        assert tile == (16 if T < 1024 else 64)
        for A in (1, 2, 7, 78, 79, 300, 1024):
            assert (q.lora_workspace_size(T, A, 16, 1) > 0) == (T >= 1280 and T >= 64 * A)
            # the most tiles: as many adapters as can have one token each, the rest in full tiles beside them
            n = min(T, A)
            worst = n + (T - n) // tile
            assert worst <= q.lora_max_tiles(T, A) <= worst + 1 + n // tile
    assert q.lora_max_tiles(0, 5) == 0


def test_embed_refusals(L):
    d = q.qmv_pack_desc(q.QMV_INT4, 100, 256)
    ok = [ctypes.byref(d), 256, 256, 3, 1.0, 256, q.QMV_BF16, 256, None]

    def call(at, v):
        args = list(ok)
        args[at] = v
        return L.qmv_embed(*args)

    for at, v, status in [(0, None, -1), (1, None, -1), (2, None, -1), (5, None, -1), (3, -1, -1), (3, 2 ** 31, -1), (6, 0, -1), (6, 4, -1),
                          (7, 255, -1), (7, 260, -2), (1, 264, -2), (2, 258, -2), (5, 264, -2), (4, math.inf, -1), (4, math.nan, -1)]:
        _err(call(at, v), status)
    for fmt, status in [(q.QMV_CASS_MX, q.QMV_ERR_UNSUPPORTED), (q.QMV_TERNARY2_SPARSE, q.QMV_ERR_UNSUPPORTED), (q.QMV_CASS, q.QMV_ERR_UNSUPPORTED),
                        (0, q.QMV_ERR_ARG), (8, q.QMV_ERR_ARG)]:
        bad = q.qmv_desc.from_buffer_copy(d)
        bad.format = fmt
        _err(call(0, ctypes.byref(bad)), status)
    for fmt in (q.QMV_INT4, q.QMV_INT4_LUT, q.QMV_TERNARY2, q.QMV_TERNARY2_LUT):
        bad = q.qmv_pack_desc(fmt, 100, 256)
        bad.off[1] += 256
        _err(call(0, ctypes.byref(bad)), q.QMV_ERR_ARG, "sections" if fmt in (q.QMV_INT4_LUT, q.QMV_TERNARY2_LUT) else "section")
        bad = q.qmv_pack_desc(fmt, 100, 256)
        bad.abi_version = 7
        _err(call(0, ctypes.byref(bad)), q.QMV_ERR_ARG)
    assert call(3, 0) == q.QMV_OK                     # nothing to do, nothing launched


def test_lora_plan_refusals(L):
    def call(**kw):
        a = dict(n_tokens=100, n_adapters=5, max_tiles=11, ids=256, order=256, tiles=256) | kw
        return L.lora_plan(ctypes.byref(q.lora_plan_args(*(a[n] for n, _ in q.lora_plan_args._fields_))), None)

    _err(L.lora_plan(None, None), -1)
    for kw, status in [(dict(n_tokens=-1), -1), (dict(n_tokens=q.QMV_LORA_MAX_TOKENS + 1, max_tiles=10 ** 6), -1), (dict(n_adapters=0), -1),
                       (dict(n_adapters=1025, max_tiles=2000), -1), (dict(max_tiles=10), -1), (dict(ids=None), -1), (dict(order=None), -1),
                       (dict(tiles=None), -1), (dict(ids=258), -2), (dict(order=257), -2), (dict(tiles=264), -2)]:
        _err(call(**kw), status)
    assert call(n_tokens=0, max_tiles=0) == q.QMV_OK


def test_lora_run_refusals(L):
    def call(n_tasks=2, task=None, at=1, **kw):
        a = dict(x=256, ldx=512, K=512, n_tokens=100, n_adapters=5, max_tiles=11, pool_rows=64, max_rank=16, order=256, tiles=256, table=256,
                 scale=256, workspace=None, ws_bytes=0) | kw
        tasks = (q.lora_task * max(n_tasks, 1))()
        for i in range(n_tasks):
            k = dict(a=256, b=256, y=256, lda=512, ldb=64, ldy=60, N=60, y_type=q.QMV_F32) | ((task or {}) if i == at else {})
            tasks[i] = q.lora_task(*(k[n] for n, _ in q.lora_task._fields_))
        return L.lora_run(ctypes.byref(q.lora_args(*(a[n] for n, _ in q.lora_args._fields_))), tasks, n_tasks, None)

    _err(L.lora_run(None, (q.lora_task * 1)(), 1, None), -1)
    _err(L.lora_run(ctypes.byref(q.lora_args()), None, 1, None), -1)
    for kw, status in [(dict(n_tasks=0), -1), (dict(n_tasks=9), -1), (dict(n_tokens=-1), -1), (dict(n_tokens=2 ** 20 + 1), -1), (dict(n_adapters=0), -1),
                       (dict(n_adapters=1025), -1), (dict(max_rank=0), -1), (dict(max_rank=129), -1), (dict(pool_rows=0), -1), (dict(K=510), -1),
                       (dict(K=0), -1), (dict(ldx=504), -1), (dict(ldx=516), -2), (dict(max_tiles=10), -1), (dict(x=None), -1),
                       (dict(order=None), -1), (dict(tiles=None), -1), (dict(table=None), -1), (dict(scale=None), -1), (dict(x=264), -2),
                       (dict(tiles=264), -2), (dict(order=258), -2), (dict(table=258), -2), (dict(scale=257), -2)]:
        _err(call(**kw), status)
    for task, status in [(dict(a=None), -1), (dict(b=None), -1), (dict(y=None), -1), (dict(a=264), -2), (dict(b=264), -2), (dict(y=264), -2),
                         (dict(lda=504), -1), (dict(lda=516), -2), (dict(ldb=56), -1), (dict(ldb=68), -2), (dict(ldy=59), -1), (dict(N=0), -1),
                         (dict(y_type=0), -1), (dict(y_type=4), -1)]:
        _err(call(task=task), status, "task 1")
    assert call(n_tokens=0, max_tiles=0) == q.QMV_OK
    # many tokens want a workspace; one type for a call's tasks
    many = dict(n_tokens=4000, max_tiles=q.lora_max_tiles(4000, 5))
    need = q.lora_workspace_size(4000, 5, 16, 2)
    assert need > 0 and q.lora_workspace_size(100, 5, 16, 2) == 0 == q.lora_workspace_size(4000, 5, 129, 2)
    assert q.lora_workspace_size(4000, 5, 128, 1) > q.lora_workspace_size(4000, 5, 64, 1)
    for kw, status in [(dict(), -1), (dict(workspace=256, ws_bytes=need - 1), -1), (dict(workspace=264, ws_bytes=need), -2)]:
        _err(call(**many, **kw), status, "workspace")
    _err(call(task=dict(y_type=q.QMV_BF16)), -1, "task 1")


def test_logprob_refusals(L):
    def call(**kw):
        a = dict(x=256, ldx=1000, x_type=q.QMV_F32, n_rows=4, V=1000, top=3, scale=1.0, tokens=256, logprob=256, rank=256, lse=256, entropy=256,
                 top_index=256, top_logprob=256) | kw
        return L.logprob_run(ctypes.byref(q.logprob_args(*(a[n] for n, _ in q.logprob_args._fields_))), None)

    _err(L.logprob_run(None, None), -1)
    for kw, status in [(dict(x=None), -1), (dict(ldx=999), -1), (dict(x_type=0), -1), (dict(x_type=9), -1), (dict(n_rows=-1), -1), (dict(V=0), -1),
                       (dict(V=2 ** 24 + 1, ldx=2 ** 25), -1), (dict(top=33), -1), (dict(top=-1), -1), (dict(V=2, top=3), -1),
                       (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
                       (dict(tokens=None), -1), (dict(tokens=None, logprob=None), -1), (dict(top_index=None), -1), (dict(top_logprob=None), -1),
                       (dict(x=264), -2), (dict(tokens=258), -2), (dict(logprob=257), -2), (dict(rank=258), -2), (dict(lse=257), -2),
                       (dict(entropy=258), -2), (dict(top_index=257), -2), (dict(top_logprob=258), -2)]:
        _err(call(**kw), status)
    assert call(n_rows=0) == q.QMV_OK


def test_classes_check_their_tensors(L):
    import torch
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    i32, bf = torch.int32, torch.bfloat16
    d = q.qmv_pack_desc(q.QMV_INT4, 100, 256)
    packed = z(d.total_bytes, dt=torch.uint8)
    q.Embed(d, packed, z(3, dt=i32), z(3, 256, dt=bf))
    for args, kind in [((packed, z(3, dt=torch.int64), z(3, 256)), TypeError), ((packed, z(3, dt=i32), z(4, 256)), ValueError),
                       ((packed, z(3, dt=i32), z(3, 255)), ValueError), ((packed[:-1], z(3, dt=i32), z(3, 256)), ValueError),
                       ((packed, z(3, dt=i32), z(3, 512)[:, ::2]), ValueError), ((packed, z(3, dt=i32), z(3, 256, dt=torch.float64)), TypeError)]:
        with pytest.raises(kind):
            q.Embed(d, *args)
    plan = q.LoraPlan(z(10, dt=i32), 4)
    assert tuple(plan.tiles.shape) == (4, 4) and tuple(plan.order.shape) == (10,)
    with pytest.raises(TypeError):
        q.LoraPlan(z(10), 4)
    table, scale, x = z(4, 2, dt=i32), z(4), z(10, 64, dt=bf)
    a, b, y = z(20, 64, dt=bf), z(20, 48, dt=bf), z(10, 48)
    q.Lora(plan, table, scale, x, [(a, b, y)])
    for args, kind in [((z(3, 2, dt=i32), scale, x, [(a, b, y)]), ValueError), ((table, z(5), x, [(a, b, y)]), ValueError),
                       ((table, scale, z(10, 64), [(a, b, y)]), TypeError), ((table, scale, z(9, 64, dt=bf), [(a, b, y)]), ValueError),
                       ((table, scale, x, []), ValueError), ((table, scale, x, [(a[:19], b, y), (a, b, y)]), ValueError),
                       ((table, scale, x, [(a, b[:19], y)]), ValueError), ((table, scale, x, [(a[:, :60], b, y)]), ValueError),
                       ((table, scale, x, [(a, b, z(10, 47))]), ValueError), ((table, scale, x, [(a, b, z(9, 48))]), ValueError),
                       ((table, scale, x, [(a.float(), b, y)]), TypeError), ((table, scale, x, [(a, b, y.double())]), TypeError),
                       ((table, scale, x, [(a, b, z(1, 48).expand(10, 48))]), ValueError)]:
        with pytest.raises(kind):
            q.Lora(plan, *args)
    q.LogProb(z(3, 50), z(3, dt=i32), top=2)
    for kw, kind in [(dict(logits=z(3, 50).double()), TypeError), (dict(logits=z(3, 100)[:, ::2]), ValueError),
                     (dict(logits=z(3, 50), tokens=z(3, dt=torch.int64)), TypeError), (dict(logits=z(3, 50), tokens=z(4, dt=i32)), ValueError)]:
        with pytest.raises(kind):
            q.LogProb(**kw)
