"""Attention half of a decode step, end to end: requests come, grow and leave, one layer.

Per step: kv_plan (pages, slots and positions of the new tokens), the INT4 q|k|v matvecs, kv8_append
(rotate q and k, write k and v into the paged 8-bit cache), kv8_attend, and the INT4 o matvec. Prompts
go in as chunks of up to 16 tokens per step (the matvecs' limit); then a decode step of one token per
request is captured as a CUDA graph and replayed: lengths, block tables and the free pages advance
on the device, so the host only replays.

    python examples/attention_block.py [--requests 8] [--prompt 200] [--steps 64] [--hidden 5120]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class AttentionBlock:
    """Wq, Wk, Wv, Wo of a grouped-query attention block in INT4 with its paged 8-bit KV cache."""

    def __init__(self, hidden=5120, q_heads=40, kv_heads=8, head_dim=128, requests=8, max_tokens=2048, seed=0, device="cuda:0"):
        import torch

        import quantized_gemv_unpack_gb300 as q
        from quantized_gemv_unpack_gb300 import synth
        self.q, self.torch = q, torch
        dev = self.dev = torch.device(device)
        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.requests = hidden, q_heads, kv_heads, head_dim, requests
        gen = synth.torch_generator(seed, dev)
        self.weights = {}
        for name, n, k in (("q", q_heads * head_dim, hidden), ("k", kv_heads * head_dim, hidden), ("v", kv_heads * head_dim, hidden),
                           ("o", hidden, q_heads * head_dim)):
            d = q.qmv_pack_desc(q.QMV_INT4, n, k)
            buf = torch.empty(d.total_bytes, dtype=torch.uint8, device=dev)
            q.qmv_pack_int4(d, synth.student_t4_torch(gen, (n, k), device=dev), buf)
            self.weights[name] = (d, buf)
        # the cache and the step state: lengths, block table, ring of free pages
        max_pages = -(-max_tokens // q.QMV_KV_PAGE)
        n_pages = requests * max_pages
        self.kv = q.kv8_desc(q.QMV_KV_INT8, n_pages, kv_heads, head_dim)
        self.cache = torch.empty(self.kv.total_bytes, dtype=torch.uint8, device=dev)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.table = torch.zeros((requests, max_pages), dtype=torch.int32, device=dev)
        self.ring = torch.arange(n_pages, dtype=torch.int32, device=dev)
        self.ring_state = torch.tensor([0, n_pages], dtype=torch.int32, device=dev)
        self.rope = q.rope_desc(head_dim, [10000.0 ** (-2 * i / head_dim) for i in range(head_dim // 2)])
        self.workspace = q.kv8_workspace(self.kv, dev)

    def step(self, add):
        """A step in which request b brings add[b] tokens (negative: it leaves): a callable that issues it, its input x
        [tokens][hidden] (bf16) and its output y [tokens][hidden] (fp32). The callable may be issued again, or captured."""
        q, torch, dev = self.q, self.torch, self.dev
        T = sum(max(a, 0) for a in add)
        assert T <= q.QMV_MAX_M, "the matvecs take up to 16 rows"
        Hq, H, D = self.q_heads, self.kv_heads, self.head_dim
        x = torch.empty((T, self.hidden), dtype=torch.bfloat16, device=dev)
        qkv = torch.empty((T, (Hq + 2 * H) * D), device=dev)
        rotated = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        out = torch.empty((T, Hq * D), dtype=torch.bfloat16, device=dev)
        y = torch.empty((T, self.hidden), device=dev)
        plan = q.KvPlan(self.lens, torch.tensor(add, dtype=torch.int32, device=dev), self.table, self.ring, self.ring_state, T,
                        lens_out=self.lens, ring_state_out=self.ring_state)
        cuts = {"q": (0, Hq * D), "k": (Hq * D, (Hq + H) * D), "v": ((Hq + H) * D, (Hq + 2 * H) * D)}
        calls = [plan]
        if T:
            heads = qkv.view(T, Hq + 2 * H, D)
            calls += [
                q.Batch(q.QMV_INT4, [(*self.weights[n], x, qkv[:, a:b]) for n, (a, b) in cuts.items()], T),
                q.KvAppend(self.kv, self.cache, heads[:, Hq:Hq + H], heads[:, Hq + H:], plan.slots, plan.runs, rope=self.rope,
                           positions=plan.positions, q=heads[:, :Hq], q_out=rotated),
                q.KvAttend(self.kv, self.cache, rotated, out.view(T, Hq, D), plan.q_start, plan.ctx, self.table, D ** -0.5,
                           max_new=max(add), workspace=self.workspace),
                q.Batch(q.QMV_INT4, [(*self.weights["o"], out, y)], T)]

        def issue():
            for c in calls:
                c.run()

        issue.plan = plan
        return issue, x, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=5120)
    a = ap.parse_args(argv)
    import torch

    import quantized_gemv_unpack_gb300 as q
    n = a.requests
    block = AttentionBlock(hidden=a.hidden, requests=n, max_tokens=a.prompt + a.steps + 64)
    gen = torch.Generator(device=block.dev).manual_seed(1)

    def fill(x):
        x.copy_(torch.randn(x.shape, generator=gen, device=x.device))

    # prompts, request by request, 16 tokens at a time
    for b in range(n):
        for t in range(0, a.prompt, q.QMV_MAX_M):
            issue, x, _ = block.step([min(q.QMV_MAX_M, a.prompt - t) if i == b else 0 for i in range(n)])
            fill(x)
            issue()
    # decode: one token per request, captured once
    issue, x, y = block.step([1] * n)
    fill(x)
    issue()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        issue()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps - 1):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if q.qmv_check_status() != 0 or issue.plan.status.any():
        raise SystemExit("a step was not served")
    us = start.elapsed_time(end) * 1e3 / max(1, a.steps - 1)
    print(f"{n} requests, {int(block.lens[0])} tokens each: {us:.1f} us per decode step of one attention block "
          f"(cache {block.kv.total_bytes / 2 ** 20:.0f} MiB, |y| {float(y.abs().mean()):.3f})")


if __name__ == "__main__":
    main()
