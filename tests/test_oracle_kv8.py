"""Pins of the paged 8-bit KV cache oracle: hand-worked codes, layout, plan, rotation and attention."""
import math

import numpy as np
import pytest

from oracle import kv8


def test_e4m3_values_and_rounding():
    v = kv8.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[0x01] == 2.0 ** -9 and v[0xB8] == -1.0 and math.isnan(v[0x7F])
    # every code is its own nearest code; halfway cases go to the even code
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    assert np.array_equal(kv8.encode(v[codes], kv8.E4M3), codes)
    assert kv8.encode([1.0625, 1.1875, 2.0 ** -10, 1e9, -1e9, math.nan], kv8.E4M3).tolist() == [0x38, 0x3A, 0x00, 0x7E, 0xFE, 0]


def test_e4m3_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(4096) * 100, g.standard_normal(4096) * 0.01]).astype(np.float32).clip(-448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = kv8.encode(x, kv8.E4M3)
    assert np.array_equal(np.where(got == 128, 0, got), np.where(want == 128, 0, want))


def test_int8_codes():
    assert kv8.encode([0, 0.5, 1.5, -0.5, 126.6, 200, -200, math.nan], kv8.INT8).tolist() == [128, 128, 130, 128, 255, 255, 1, 128]
    assert kv8.decode([1, 128, 255], kv8.INT8).tolist() == [-127, 0, 127]


@pytest.mark.parametrize("D", [64, 128])
def test_tile_layout_is_a_permutation(D):
    tok, d = np.meshgrid(np.arange(64), np.arange(D), indexing="ij")
    for at in (kv8.k_byte(tok, d, D), kv8.v_byte(tok, d)):
        assert np.array_equal(np.sort(at.ravel()), np.arange(64 * D))
    # token 37 = 16 * 2 + 5: column tile 2, column 2 * 2 + 1; value 70 of 128 is in the second half
    if D == 128:
        assert kv8.k_byte(37, 70, 128) == ((2 * 2 + 1) * 8 + 5) * 64 + 6
    assert kv8.v_byte(37, 10) == 10 * 64 + 37


def test_plan_by_hand():
    lens = np.array([64, 10, 0, 130, 5, 60])
    add = np.array([1, 3, 65, -1, 0, 6])
    table = np.full((6, 4), -1)
    table[0, 0], table[1, 0], table[3, :3], table[4, 0], table[5, 0] = 7, 8, [1, 2, 3], 9, 4
    ring = np.array([20, 21, -1, -1, -1, -1, -1, -1, 30, 31])
    p = kv8.plan(lens, add, table, ring, 8, 4, 75, 20)       # free: 30, 31, 20, 21
    assert p["status"].tolist() == [0, 0, 0, 3, 0, 0]
    assert p["table"][0].tolist() == [7, 30, -1, -1] and p["table"][2].tolist() == [31, 20, -1, -1]
    assert p["table"][5].tolist() == [4, 21, -1, -1]
    assert p["ring_state_out"].tolist() == [2, 3] and p["ring"][2:5].tolist() == [1, 2, 3]
    assert p["slots"][:4].tolist() == [30 * 64, 8 * 64 + 10, 8 * 64 + 11, 8 * 64 + 12]
    assert p["runs"][:6].tolist() == [[0, 1], [1, 3], [4, 64], [68, 1], [69, 4], [73, 2]]
    assert p["ctx"].tolist() == [65, 13, 65, 0, 5, 66] and p["q_start"].tolist() == [0, 1, 4, 69, 69, 69, 75]
    # one page less: the last request that needs one gets none
    p = kv8.plan(lens, add, table, ring, 8, 3, 75, 20)
    assert p["status"].tolist() == [0, 0, 0, 3, 0, 1] and p["ctx"][5] == 0 and p["lens_out"][5] == 60


def test_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    y = kv8.rotate(x, np.array([[1], [2]]), [math.pi / 2, math.pi / 4], [0, 1])
    c = math.sqrt(0.0 + 1.0)    # pair (0, 2) turns by 90 degrees, pair (1, 3) by 2 * 45
    assert np.allclose(y[0, 0], [-3 * c, -4 * c, 1 * c, 2 * c])
    assert np.allclose(kv8.rotate(y, np.array([[1], [2]]), [math.pi / 2, math.pi / 4], [0, 1], inverse=True), x)
    z = kv8.rotate(x, np.array([[1]]), [math.pi / 2, 0.0], [0, 0], interleaved=True)
    assert np.allclose(z[0, 0], [-2, 1, 3, 4])


def _cache(kind, n_pages=3, heads=1, D=64):
    total = kv8.sections(n_pages, heads, D)[2]
    return kv8.Cache(np.zeros(total, dtype=np.uint8), n_pages, heads, D, kind)


def test_append_grows_the_scale_and_rounds_again():
    c = _cache(kv8.INT8)
    k = np.zeros((3, 1, 64), dtype=np.float32)
    k[0, 0, :3] = [127, 63, -5]
    k[1, 0, :2] = [254, 1]
    k[2, 0, 0] = 10
    kv8.append(c, k, k, np.array([64, 65, 66]), [[0, 1]])
    assert c.scales[1, 0].tolist() == [1, 1] and c.page_codes(1, 0)[0, 0, :3].tolist() == [255, 191, 123]
    kv8.append(c, k, k, np.array([64, 65, 66]), [[1, 1]])      # scale 2: 63.5 -> 64, 31.5 -> 32, -2.5 -> -2; 0.5 -> 0
    assert c.scales[1, 0].tolist() == [2, 2] and c.page_codes(1, 0)[0, 0, :3].tolist() == [192, 160, 126]
    assert c.page_codes(1, 1)[0, 1, :2].tolist() == [255, 128]
    kv8.append(c, k, k, np.array([64, 65, 66]), [[2, 1]])      # scale stays
    assert c.scales[1, 0].tolist() == [2, 2] and c.page_codes(1, 0)[0, 2, 0] == 133


def test_attention_by_hand():
    c = _cache(kv8.INT8)
    c.codes[:] = 128
    c.scales[:] = 1
    kb = lambda tok, d: kv8.k_byte(tok, d, 64)  # noqa: E731
    c.codes[2, 0, 0, kb(0, 0)] = 128 + 1            # k_0 = e0, k_1 = 0
    c.codes[2, 0, 1, kv8.v_byte(0, 5)] = 128 + 10   # v_0 = 10 e5, v_1 = 20 e5
    c.codes[2, 0, 1, kv8.v_byte(1, 5)] = 128 + 20
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = math.log(3)                        # scores (log 3, 0): weights 3/4, 1/4
    table = np.array([[2]])
    out, lse, *_ = kv8.attend(c, q, [0, 2], [2], table, 1.0)
    assert np.isclose(out[0, 0, 5], 10) and np.isclose(out[1, 0, 5], 12.5) and np.isclose(lse[1, 0], math.log(4))
    out, *_ = kv8.attend(c, q, [0, 2], [2], table, 1.0, window=1)
    assert np.isclose(out[1, 0, 5], 20)
    out, *_ = kv8.attend(c, q, [0, 2], [2], table, 1.0, prefix=[2])
    assert np.isclose(out[0, 0, 5], 12.5)
    out, *_ = kv8.attend(c, q, [0, 2], [2], table, 1.0, slopes=[math.log(3)])
    assert np.isclose(out[1, 0, 5], 15)             # the distance of 1 takes log 3 from the first key
    out, lse, *_ = kv8.attend(c, q, [0, 2], [1], table, 1.0)
    assert np.isclose(out[1, 0, 5], 10) and not out[0].any() and lse[0, 0] == -np.inf   # position -1 sees nothing
    out, *_ = kv8.attend(c, q * 1e6, [0, 2], [2], table, 1.0, softcap=math.log(3))
    assert np.isclose(out[1, 0, 5], 12.5)           # tanh(large) = 1: the score is the cap


def test_append_keeps_the_least_scale():
    """Scales below 2^-126 are 2^-126, and growing from one leaves zeros zero."""
    for kind, top in ((kv8.INT8, 127), (kv8.E4M3, 448)):
        c = _cache(kind)
        k = np.zeros((2, 1, 64), dtype=np.float32)
        k[0, 0, 1] = 1e-40
        k[1, 0, 1] = np.float32(2.0 ** -125 * top)
        kv8.append(c, k, k, np.array([64, 65]), [[0, 1]])
        assert c.scales[1, 0].tolist() == [2.0 ** -126] * 2 and c.page_values(1, 0)[0, 0, 0] == 0
        kv8.append(c, k, k, np.array([64, 65]), [[1, 1]])
        assert c.scales[1, 0].tolist() == [2.0 ** -125] * 2
        assert c.page_values(1, 1)[0, 1, 1] == 2.0 ** -125 * top and not c.page_values(1, 1)[0, :2, 2:].any()


def test_plan_keeps_the_pages_of_a_shortened_request():
    """Two requests of 130 tokens taken back to 60 and 64: their further pages stay in their rows, serve the next tokens and
    go back with them."""
    table = np.array([[5, 6, 7, -1], [1, 2, 3, -1]])
    ring = np.array([9, 8, -1, -1, -1, -1])
    p = kv8.plan(np.array([60, 64]), np.array([10, -1]), table, ring, 0, 2, 10, 3, held=[3, 3])
    assert p["status"].tolist() == [0, 3] and p["held_out"].tolist() == [3, 0] and p["table"].tolist() == table.tolist()
    assert p["slots"].tolist() == [5 * 64 + i for i in range(60, 64)] + [6 * 64 + i for i in range(6)]
    assert p["ring_state_out"].tolist() == [0, 5] and p["ring"].tolist() == [9, 8, 1, 2, 3, -1]
    p = kv8.plan(np.array([60, 64]), np.array([140, 1]), table, np.array([9, 8, -1, -1]), 0, 2, 141, 9, held=[3, 1])
    assert p["status"].tolist() == [0, 0] and p["table"].tolist() == [[5, 6, 7, 9], [1, 8, 3, -1]] and p["held_out"].tolist() == [4, 2]
    p = kv8.plan(np.array([60, 64]), np.array([1, 1]), table, ring, 0, 2, 2, 2, held=[0, 5])
    assert p["status"].tolist() == [2, 2] and p["held_out"].tolist() == [0, 5]
