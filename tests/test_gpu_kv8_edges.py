"""GPU parity of the paged 8-bit KV cache calls at the ends of their ranges, with the float64 oracle.

The bounds are those of test_gpu_kv8.py unless a test derives its own.
"""
import numpy as np
import pytest

from test_gpu_kv8 import ULP, _check_plan, _f64, _fresh_cache, _host, _plan_state, _q, _run_plan, _tt, env  # noqa: F401 (env is a fixture)

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
