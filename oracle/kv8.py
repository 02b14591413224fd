"""Paged 8-bit KV cache, rotary positions and attention, restated in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain loops over requests,
heads and pages; every formula is written from its definition: the plan request by
request in order, the rotation as a complex product, the cache codes value by value,
attention as a softmax over the visible keys.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 64
INT8, E4M3 = 1, 2


# ----------------------------------------------------------------------------- codes and layout

def e4m3_values() -> np.ndarray:
    """Value of each of the 256 e4m3 codes: 1 sign, 4 exponent (bias 7), 3 fraction bits; S.1111.111 is NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = math.nan
        out[b] = -v if b & 128 else v
    return out


def decode(codes, kind):
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.astype(np.float64) - 128 if kind == INT8 else e4m3_values()[codes]


def encode(y, kind):
    """Nearest code of each value (ties to the even code), held to the largest magnitude; NaN gives 0."""
    y = np.asarray(y, dtype=np.float64)
    y = np.where(np.isnan(y), 0.0, y)
    if kind == INT8:
        return (np.rint(np.clip(y, -127, 127)) + 128).astype(np.uint8)
    table = e4m3_values()[:127]                    # +0 .. 448
    mag = np.clip(np.abs(y), 0, 448)
    hi = np.clip(np.searchsorted(table, mag), 1, 126)
    lo = hi - 1
    down, up = mag - table[lo], table[hi] - mag
    pick = np.where(down < up, lo, np.where(down > up, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def k_byte(token, d, D):
    j, g = (token % 16) // 2, (token // 16) * 2 + token % 2     # fragment column tile, column
    return ((j * (D // 64) + d // 64) * 8 + g) * 64 + d % 64


def v_byte(token, d):
    return d * PAGE + token


def sections(n_pages, heads, D):
    codes = n_pages * heads * 2 * PAGE * D
    off = -(-codes // 256) * 256
    scales = n_pages * heads * 2 * 4
    return [0, off], [codes, scales], -(-(off + scales) // 256) * 256


class Cache:
    """Views into a host copy of a cache buffer."""

    def __init__(self, buf, n_pages, heads, D, kind):
        off, size, total = sections(n_pages, heads, D)
        self.buf, self.heads, self.D, self.kind, self.n_pages = buf, heads, D, kind, n_pages
        self.codes = buf[:size[0]].reshape(n_pages, heads, 2, PAGE * D)
        self.scales = buf[off[1]:off[1] + size[1]].view(np.float32).reshape(n_pages, heads, 2)
        tok, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
        self.at = np.stack([k_byte(tok, d, D), v_byte(tok, d)])          # [2][64][D]

    def page_codes(self, page, which):
        """[heads][64][D] code bytes of K (0) or V (1)."""
        return self.codes[page, :, which][:, self.at[which]]

    def page_values(self, page, which):
        return decode(self.page_codes(page, which), self.kind) * self.scales[page, :, which].astype(np.float64)[:, None, None]


# ----------------------------------------------------------------------------- plan

def plan(lens, add, table, ring, head, count, T, max_runs, held=None):
    """One step, request by request. Returns a dict of the outputs; table and ring are copies. held: pages in each row (NULL:
    those that the length fills)."""
    counts = held
    B, cap, N = len(lens), table.shape[1], len(ring)
    table, ring = table.copy(), ring.copy()
    out = {k: np.zeros(B, dtype=np.int64) for k in ("lens_out", "ctx", "status", "held_out")}
    q_start = np.zeros(B + 1, dtype=np.int64)
    slots, positions = np.full(T, -1), np.full(T, -1)
    runs = []
    at = taken = needed = 0
    back = []
    for b in range(B):
        length, new = int(lens[b]), max(int(add[b]), 0)
        q_start[b] = min(at, T)
        full, after = -(-length // PAGE), -(-(length + new) // PAGE)
        held = full if counts is None else int(counts[b])
        out["lens_out"][b] = length
        out["held_out"][b] = held
        if length < 0 or held < full or held > cap or after > cap or at + new > T:
            out["status"][b] = 2
        elif add[b] < 0:
            out["status"][b] = 3
            out["lens_out"][b] = out["held_out"][b] = 0
            back += [int(p) for p in table[b, :held]]
        else:
            needed += max(after - held, 0)
            if after > held and needed > count:
                out["status"][b] = 1
            else:
                for i in range(held, after):
                    table[b, i] = ring[(head + taken) % N]
                    taken += 1
                out["held_out"][b] = max(held, after)
                out["lens_out"][b] = out["ctx"][b] = length + new
                for i in range(new):
                    p = length + i
                    positions[at + i] = p
                    slots[at + i] = table[b, p // PAGE] * PAGE + p % PAGE
                    if i == 0 or p % PAGE == 0:
                        runs.append([at + i, 0])
                    runs[-1][1] += 1
        at += new
    q_start[B] = min(at, T)
    for i, p in enumerate(back):
        ring[(head + count + i) % N] = p
    runs += [[0, 0]] * (max_runs - len(runs))
    return {**out, "q_start": q_start, "slots": slots, "positions": positions, "runs": np.array(runs).reshape(-1, 2),
            "ring_state_out": np.array([(head + taken) % N, count - taken + len(back)]), "table": table, "ring": ring}


# ----------------------------------------------------------------------------- rotation

def rotate(x, positions, inv_freq, axis, interleaved=False, inverse=False):
    """x float64 [T][H][D]; positions [n_axes][T]; pairs (i, i + n) or (2i, 2i + 1)."""
    n = len(inv_freq)
    y = np.array(x, dtype=np.float64)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        z = np.exp((-1j if inverse else 1j) * positions[axis[i]].astype(np.float64) * inv_freq[i])[:, None]
        w = (x[..., a] + 1j * x[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
    return y


# ----------------------------------------------------------------------------- append

def append(cache: Cache, k, v, slots, runs):
    """Write float32 k, v [T][H][D] into the cache in place, with the arithmetic in fp32 as the format defines it."""
    top = np.float32(127 if cache.kind == INT8 else 448)
    f32 = np.float32
    for t, n in runs:
        if n == 0 or slots[t] < 0:
            continue
        page, off = slots[t] // PAGE, slots[t] % PAGE
        for which, x in ((0, k), (1, v)):
            codes = cache.page_codes(page, which)
            for h in range(cache.heads):
                new = x[t:t + n, h].astype(f32)
                fin = np.abs(new[np.isfinite(new)])
                a = fin.max() if fin.size else f32(0)
                was = cache.scales[page, h, which] if off else f32(0)
                now = max(was, f32(a / top))
                if 0 < now < f32(2.0 ** -126):
                    now = f32(2.0 ** -126)
                with np.errstate(all="ignore"):
                    inv = f32(1) / now if now > 0 else f32(0)
                    if off and now > was and was > 0:
                        codes[h, :off] = encode((decode(codes[h, :off], cache.kind).astype(f32) * f32(was * inv)), cache.kind)
                    codes[h, off:off + n] = encode(new * inv, cache.kind)
                cache.scales[page, h, which] = now
            for h in range(cache.heads):
                cache.codes[page, h, which][cache.at[which][:off + n]] = codes[h, :off + n]


# ----------------------------------------------------------------------------- attention

def attend(cache: Cache, q, q_start, ctx, table, scale, softcap=0.0, slopes=None, window=0, prefix=None):
    """Float64 output [T][Hq][D], log-sum-exp [T][Hq], and per row the bound terms: sum p |v|, the largest
    |v| of a seen key, the number of keys seen and the largest scale * sum |q k| of a seen key."""
    T, Hq, D = q.shape
    G = Hq // cache.heads
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    pv, vmax, seen_n, sabs = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(ctx)):
        t0, t1, L = int(q_start[b]), int(q_start[b + 1]), int(ctx[b])
        if t1 <= t0 or L <= 0:
            continue
        pages = [int(p) for p in table[b, :-(-L // PAGE)]]
        there = np.repeat([0 <= p < cache.n_pages for p in pages], PAGE)[:L]
        K = np.concatenate([cache.page_values(p if 0 <= p < cache.n_pages else 0, 0) for p in pages], 1)[:, :L]
        V = np.concatenate([cache.page_values(p if 0 <= p < cache.n_pages else 0, 1) for p in pages], 1)[:, :L]
        key = np.arange(L)
        pos = (L - (t1 - t0) + np.arange(t1 - t0))[:, None]
        ok = (key <= pos) | (key < (0 if prefix is None else prefix[b]))
        if window:
            ok &= pos - key < window
        ok &= there
        some = ok.any(1)
        for hq in range(Hq):
            kk, vv, qq = K[hq // G], V[hq // G], q[t0:t1, hq]
            s = scale * (qq @ kk.T)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[hq] * np.abs(pos - key)
            s = np.where(ok, s, -np.inf)
            m = np.where(some, s.max(1), 0.0)[:, None]
            p = np.exp(s - m)
            l = np.where(some, p.sum(1), 1.0)[:, None]
            out[t0:t1, hq] = (p / l) @ vv
            lse[t0:t1, hq] = np.where(some, m[:, 0] + np.log(l[:, 0]), -np.inf)
            pv[t0:t1, hq] = (p / l) @ np.abs(vv)
            vmax[t0:t1, hq] = np.where(ok, np.abs(vv).max(1), 0.0).max(1)
            sabs[t0:t1, hq] = scale * np.where(ok, np.abs(qq) @ np.abs(kk).T, 0.0).max(1)
        seen_n[t0:t1] = ok.sum(1)[:, None]
    return out, lse, pv, vmax, seen_n, sabs
