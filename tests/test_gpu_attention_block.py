"""The attention half of a decode step through the public calls (examples/attention_block.py): against a plain
computation from the same packed weights, and captured steps against issued ones."""
import os
import sys

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention_block
    return attention_block


def _weight(q, torch, d, buf):
    w = torch.empty((d.N, d.K), dtype=torch.int8, device=buf.device)
    s = torch.empty((d.N, d.K // 128), dtype=torch.float16, device=buf.device)
    q.qmv_unpack(d, buf, w, s)
    return w.double() * s.double().repeat_interleave(128, 1)


def _small(example, seed=0, requests=3):
    return example.AttentionBlock(hidden=256, q_heads=6, kv_heads=2, head_dim=64, requests=requests, max_tokens=300, seed=seed)


def test_block_matches_plain_computation(example):
    """y of every step against float64 attention over the unquantized keys and values: the matvecs' bound (2e-3), a
    bf16 rounding of q and of the output, and the cache's steps (each key and value off by up to 1 / 127 of its page's
    largest) leave an error of a few percent of the output's size."""
    import torch

    import quantized_gemv_unpack_gb300 as q
    blk = _small(example)
    W = {n: _weight(q, torch, *v) for n, v in blk.weights.items()}
    gen = torch.Generator(device=blk.dev).manual_seed(5)
    hist = [[] for _ in range(3)]
    f = np.array([10000.0 ** (-2 * i / 64) for i in range(32)])

    def turn(x, pos):
        x = x.reshape(-1, 64).cpu().numpy()
        z = (x[:, :32] + 1j * x[:, 32:]) * np.exp(1j * pos * f)
        return np.concatenate([z.real, z.imag], 1)

    for add in [[16, 0, 0], [0, 16, 0], [16, 0, 0], [1, 1, 3], [5, -1, 1], [1, 2, 0], [1, 1, 1], [0, 0, 0], [14, 1, 1]]:
        issue, x, y = blk.step(add)
        x.copy_(torch.randn(x.shape, generator=gen, device=blk.dev))
        issue()
        torch.cuda.synchronize()
        assert q.qmv_check_status() == 0
        t = 0
        for b, a in enumerate(add):
            if a < 0:
                hist[b] = []
            for _ in range(max(a, 0)):
                xt = x[t].double()
                pos = len(hist[b])
                qq = turn(W["q"] @ xt, pos)
                hist[b].append((turn(W["k"] @ xt, pos), (W["v"] @ xt).reshape(2, 64).cpu().numpy()))
                K, V = np.stack([k for k, _ in hist[b]]), np.stack([v for _, v in hist[b]])
                o = []
                for h in range(6):
                    s = K[:, h // 3] @ qq[h] / 8.0
                    p = np.exp(s - s.max())
                    o.append((p / p.sum()) @ V[:, h // 3])
                want = W["o"].cpu().numpy() @ np.concatenate(o)
                err = np.abs(y[t].cpu().numpy() - want).max()
                assert err <= 0.06 * np.abs(want).max(), (add, t, err, np.abs(want).max())
                t += 1
    assert blk.lens.tolist() == [len(h) for h in hist]


def test_captured_steps_match_issued_ones(example):
    """Two blocks of the same weights: one issues its decode steps, one replays a captured step."""
    import torch

    import quantized_gemv_unpack_gb300 as q
    one, two = _small(example, seed=3), _small(example, seed=3)
    gen = torch.Generator(device=one.dev).manual_seed(6)
    for blk in (one, two):
        gen.manual_seed(6)
        for b in range(3):
            for _ in range(4):
                issue, x, _ = blk.step([16 if i == b else 0 for i in range(3)])
                x.copy_(torch.randn(x.shape, generator=gen, device=blk.dev))
                issue()
    a, xa, ya = one.step([1, 1, 1])
    b, xb, yb = two.step([1, 1, 1])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b()
    for _ in range(70):     # over a page's end
        x = torch.randn(xa.shape, generator=gen, device=one.dev)
        xa.copy_(x)
        xb.copy_(x)
        a()
        g.replay()
        assert torch.equal(ya, yb) and torch.equal(one.lens, two.lens)
    assert torch.equal(one.table[:, :3], two.table[:, :3])
    assert q.qmv_check_status() == 0
