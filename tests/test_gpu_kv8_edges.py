"""GPU parity of the paged 8-bit KV cache calls at the ends of their ranges, with the float64 oracle.

The bounds are those of test_gpu_kv8.py unless a test derives its own.
"""
import numpy as np
import pytest

from test_gpu_kv8 import _check_plan, _plan_state, _q, _run_plan, env  # noqa: F401 (env is a fixture)

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
