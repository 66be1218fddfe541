"""A decode step around the quantized projections, on random weights.

Every step appends one token to each request, from the random numbers that it is
given, with this library's calls between the embedding and the next token:

    plan      block tables and slot maps of the step        q4k_kv_plan
    per layer norm (with the residual's addition)           q4k_add_rmsnorm
              q, k, v projection                            q4k_gemv
              new keys and values into the paged cache      q4k_kv_write
              attention over the cache                      q4k_paged_attn
              output projection, norm, gate/up, down        q4k_gemv, q4k_add_rmsnorm, q4k_gemv_glu, q4k_gemv
    the end   norm, vocabulary projection, sampling         q4k_add_rmsnorm, q4k_gemv, q4k_sample

Beside them a layer has two torch casts, because projections give fp32 and
attention and projections take bf16.  The model has no position encoding, and the
library no call that rotates q and k: where one is wanted, rotate them between
the projection and the cache write, by the positions that q4k_kv_plan gives.

Run it on the GPU:  python examples/decode_step.py [--steps N] [--cache e4m3]
It prints the time of a step launched call by call and as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_block_quantized_q4_gb300 as q4k  # noqa: E402
import synth  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class Decoder:
    """A model of `layers` equal layers with a paged cache for `requests` requests."""

    def __init__(self, requests=4, layers=2, hidden=1024, q_heads=8, kv_heads=2, dim=128, ffn=2048,
                 vocab=4096, page=16, max_len=512, cache=BF16, seed=0, device="cuda"):
        self.requests, self.hidden, self.ffn, self.vocab, self.page = requests, hidden, ffn, vocab, page
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.qkv = (q_heads + 2 * kv_heads) * dim
        pages_per_request = -(-max_len // page)
        pages = requests * pages_per_request
        shapes = {"qkv": (self.qkv, hidden), "o": (hidden, q_heads * dim), "gate": (ffn, hidden), "up": (ffn, hidden), "down": (hidden, ffn)}
        # scales that keep the activations near 1 whatever the depth
        weight = lambda n, k, *at: synth.q4k_weight(n, k, seed=synth.derive_seed(seed, *at), quants="normal", d_range=(2e-4, 4e-4)).to(device)  # noqa: E731
        self.layers = []
        g = torch.Generator().manual_seed(seed)
        gamma = lambda: (1 + 0.1 * torch.randn(hidden, generator=g)).to(device)  # noqa: E731
        for i in range(layers):
            layer = {name: weight(n, k, i, name) for name, (n, k) in shapes.items()}
            layer["norm1"], layer["norm2"] = gamma(), gamma()
            size = (pages, kv_heads, page, dim)
            for kv in "kv":
                layer[kv] = torch.zeros(size, dtype=torch.uint8 if cache != BF16 else BF16, device=device)
                layer[kv] = layer[kv].view(cache)
                layer[kv + "_scale"] = torch.zeros(size[:3], device=device) if cache != BF16 else None
            self.layers.append(layer)
        self.embed = (torch.randn((vocab, hidden), generator=g)).to(BF16).to(device)
        self.head, self.norm = weight(vocab, hidden, "head"), gamma()
        # the cache's books: nothing cached, every page free
        self.lens = torch.zeros(requests, dtype=I32, device=device)
        self.table = torch.full((requests, pages_per_request), -1, dtype=I32, device=device)
        self.pool = torch.arange(pages, dtype=I32, device=device)
        self.state = torch.tensor([0, pages], dtype=I32, device=device)
        # what a step reads and leaves
        self.add = torch.ones(requests, dtype=I32, device=device)
        self.tokens = torch.zeros(requests, dtype=I32, device=device)
        self.u = torch.zeros(requests, device=device)
        self.temperature = torch.full((requests,), 0.8, device=device)
        self.top_k = torch.full((requests,), 40, dtype=I32, device=device)
        self.top_p = torch.full((requests,), 0.95, device=device)
        self.status = torch.zeros(requests, dtype=I32, device=device)
        new = lambda n, t: torch.empty(n, dtype=t, device=device)  # noqa: E731
        self.plan_out = (self.lens, new(requests + 1, torch.int64), new(requests, I32), new(requests, I32), self.status, self.state)

    def step(self):
        """One token for every request; self.tokens, self.lens and the cache move on.  Returns (logits, logp)."""
        n, d, hq, hk = self.requests, self.dim, self.q_heads, self.kv_heads
        _, _, slots, _, _, _ = q4k.q4k_kv_plan(self.lens, self.add, self.table, self.pool, self.state, self.page, n, out=self.plan_out)
        residual = self.embed.index_select(0, self.tokens)
        branch = None  # what the last projection adds to the residual stream
        for layer in self.layers:
            x, residual = self._norm(branch, residual, layer["norm1"])
            qkv = q4k.q4k_gemv(layer["qkv"], self.qkv, self.hidden, x).view(n, hq + 2 * hk, d)
            q4k.q4k_kv_write(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, layer["k"], layer["v"], layer["k_scale"], layer["v_scale"])
            attn, _ = q4k.q4k_paged_attn(qkv[:, :hq].to(BF16), layer["k"], layer["v"], self.table, self.lens, d ** -0.5, layer["k_scale"], layer["v_scale"])
            branch = q4k.q4k_gemv(layer["o"], self.hidden, hq * d, attn.view(n, hq * d))
            x, residual = self._norm(branch, residual, layer["norm2"])
            h = q4k.q4k_gemv_glu(layer["gate"], layer["up"], self.ffn, self.hidden, x)
            branch = q4k.q4k_gemv(layer["down"], self.hidden, self.ffn, h.to(BF16))
        x, _ = self._norm(branch, residual, self.norm)
        logits = q4k.q4k_gemv(self.head, self.vocab, self.hidden, x)
        _, logp = q4k.q4k_sample(logits, self.u, self.temperature, self.top_k, self.top_p, out=self.tokens)
        return logits, logp

    def _norm(self, branch, residual, gamma):
        """(normed, residual + branch); before the first layer there is no branch yet."""
        if branch is None:
            return q4k.q4k_add_rmsnorm(residual, None, gamma, 1e-6)[0], residual
        return q4k.q4k_add_rmsnorm(branch, residual, gamma, 1e-6)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    model = Decoder(cache=BF16 if a.cache == "bf16" else torch.float8_e4m3fn, max_len=4 * a.steps + 64)
    g = torch.Generator(device="cuda").manual_seed(1)

    def run(step, steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(steps):
            model.u.uniform_(0.0, 1.0, generator=g)
            step()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / steps * 1e6

    run(model.step, 8)
    eager = run(model.step, a.steps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.step()
    run(graph.replay, 8)
    replay = run(graph.replay, a.steps)
    if q4k.q4k_get_device_error() or bool(model.status.any()):
        raise SystemExit(f"the step failed: request states {model.status.tolist()}")
    print(f"{model.requests} requests, {len(model.layers)} layers, {int(model.lens.max())} tokens cached: "
          f"{eager:.0f} us a step call by call, {replay:.0f} us as a graph; last tokens {model.tokens.tolist()}")


if __name__ == "__main__":
    main()
