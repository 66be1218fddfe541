"""Prompts and decode steps around the quantized projections, on random weights.

Every step appends one token to each request, from the random numbers that it is
given, with this library's calls between the embedding and the next token:

    plan      block tables and slot maps of the step        q4k_kv_plan
    per layer norm (with the residual's addition)           q4k_add_rmsnorm
              q, k, v projection                            q4k_gemv
              new keys and values into the paged cache      q4k_kv_write
              attention over the cache                      q4k_paged_attn
              output projection, norm, gate/up, down        q4k_gemv, q4k_add_rmsnorm, q4k_gemv_glu, q4k_gemv
    the end   norm, vocabulary projection, sampling         q4k_add_rmsnorm, q4k_gemv, q4k_sample

With a base of rotations the model has positions: q and k are rotated on their
way to the cache (q4k_rope_kv_write instead of q4k_kv_write).  Then it also takes
prompts, blocks of ragged numbers of tokens (and continues them, many at a time or
one by one):

    plan                                                    q4k_kv_plan
    per layer norm, q, k, v projection                      q4k_add_rmsnorm, q4k_gemm
              rotation, keys and values into the cache      q4k_rope_kv_write
              attention of each token to those before it    q4k_paged_attn_chunk
              output projection, norm, gate, up, down       q4k_gemm, q4k_add_rmsnorm, q4k_gemm
    the end   norm, vocabulary projection                   q4k_add_rmsnorm, q4k_gemm
              how likely the prompt's own tokens were       q4k_logprobs
              the token after the prompt                    q4k_sample

Beside them a layer has two torch casts in a decode step, because projections give
fp32 and attention and projections take bf16, and torch's silu in a prompt.

Run it on the GPU:  python examples/decode_step.py [--steps N] [--prompt N] [--cache e4m3]
It prints the time of a step launched call by call and as a CUDA graph; with
--prompt, of prompts of N tokens before them.
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
                 vocab=4096, page=16, max_len=512, cache=BF16, seed=0, device="cuda", rotate=0.0):
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
        # the rotation's frequencies; 0: a model without positions
        self.steps, self.amplitude = (t if isinstance(t, float) else t.to(device) for t in q4k.q4k_rope_steps(dim, rotate)) if rotate else (None, 1.0)
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
        _, _, slots, pos, _, _ = q4k.q4k_kv_plan(self.lens, self.add, self.table, self.pool, self.state, self.page, n, out=self.plan_out)
        residual = self.embed.index_select(0, self.tokens)
        branch = None  # what the last projection adds to the residual stream
        for layer in self.layers:
            x, residual = self._norm(branch, residual, layer["norm1"])
            qkv = q4k.q4k_gemv(layer["qkv"], self.qkv, self.hidden, x).view(n, hq + 2 * hk, d)
            q = self._rotate_and_write(qkv, pos, slots, layer) if self.steps is not None else qkv[:, :hq].to(BF16)
            if self.steps is None:
                q4k.q4k_kv_write(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, layer["k"], layer["v"], layer["k_scale"], layer["v_scale"])
            attn, _ = q4k.q4k_paged_attn(q, layer["k"], layer["v"], self.table, self.lens, d ** -0.5, layer["k_scale"], layer["v_scale"])
            branch = q4k.q4k_gemv(layer["o"], self.hidden, hq * d, attn.view(n, hq * d))
            x, residual = self._norm(branch, residual, layer["norm2"])
            h = q4k.q4k_gemv_glu(layer["gate"], layer["up"], self.ffn, self.hidden, x)
            branch = q4k.q4k_gemv(layer["down"], self.hidden, self.ffn, h.to(BF16))
        x, _ = self._norm(branch, residual, self.norm)
        logits = q4k.q4k_gemv(self.head, self.vocab, self.hidden, x)
        _, logp = q4k.q4k_sample(logits, self.u, self.temperature, self.top_k, self.top_p, out=self.tokens)
        return logits, logp

    def prompt(self, tokens, following, add):
        """add [requests] int32 tokens for each request (0: none), one after the other in tokens [n] int32, of which
        the last ones may belong to none; following [n] int32 is what the caller expects after each (-1: nothing).
        self.tokens of a request that got some, self.lens and the cache move on.  Returns (logits [n, vocab] bf16,
        log-probability and rank of the following tokens)."""
        if self.steps is None:
            raise ValueError("the model has no positions: give it a base of rotations")
        n, d, hq = tokens.numel(), self.dim, self.q_heads
        _, cu, slots, pos, _, _ = q4k.q4k_kv_plan(self.lens, add, self.table, self.pool, self.state, self.page, n,
                                                  out=(self.lens, self.plan_out[1], torch.empty_like(tokens), torch.empty_like(tokens), self.status, self.state))
        residual = self.embed.index_select(0, tokens)
        branch = None
        for layer in self.layers:
            x, residual = self._norm(branch, residual, layer["norm1"])
            qkv = q4k.q4k_gemm(layer["qkv"], self.qkv, self.hidden, x).view(n, -1, d)
            q = self._rotate_and_write(qkv, pos, slots, layer)
            attn, _ = q4k.q4k_paged_attn_chunk(q, layer["k"], layer["v"], self.table, self.lens, cu, d ** -0.5, layer["k_scale"], layer["v_scale"], out=torch.zeros_like(q))
            branch = q4k.q4k_gemm(layer["o"], self.hidden, hq * d, attn.view(n, hq * d))
            x, residual = self._norm(branch, residual, layer["norm2"])
            h = torch.nn.functional.silu(q4k.q4k_gemm(layer["gate"], self.ffn, self.hidden, x)) * q4k.q4k_gemm(layer["up"], self.ffn, self.hidden, x)
            branch = q4k.q4k_gemm(layer["down"], self.hidden, self.ffn, h)
        x, _ = self._norm(branch, residual, self.norm)
        logits = q4k.q4k_gemm(self.head, self.vocab, self.hidden, x)
        logp, rank, _, _, _ = q4k.q4k_logprobs(logits, following)
        last = logits.index_select(0, (cu[1:] - 1).clamp(min=0))
        token, _ = q4k.q4k_sample(last, self.u, self.temperature, self.top_k, self.top_p)
        self.tokens.copy_(torch.where(cu[1:] > cu[:-1], token, self.tokens))
        return logits, logp, rank

    def _rotate_and_write(self, qkv, pos, slots, layer):
        """The rotated queries; the rotated keys and the values go into the layer's cache."""
        hq, hk = self.q_heads, self.kv_heads
        return q4k.q4k_rope_kv_write(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], pos, slots, self.steps, layer["k"], layer["v"],
                                     layer["k_scale"], layer["v_scale"], amplitude=self.amplitude)

    def _norm(self, branch, residual, gamma):
        """(normed, residual + branch); before the first layer there is no branch yet."""
        if branch is None:
            return q4k.q4k_add_rmsnorm(residual, None, gamma, 1e-6)[0], residual
        return q4k.q4k_add_rmsnorm(branch, residual, gamma, 1e-6)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--prompt", type=int, default=0)
    a = ap.parse_args()
    model = Decoder(cache=BF16 if a.cache == "bf16" else torch.float8_e4m3fn, max_len=2 * a.prompt + 4 * a.steps + 64,
                    rotate=1e4 if a.prompt else 0.0)
    g = torch.Generator(device="cuda").manual_seed(1)

    def run(step, steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(steps):
            model.u.uniform_(0.0, 1.0, generator=g)
            step()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / steps * 1e6

    if a.prompt:
        tokens = torch.randint(0, model.vocab, (model.requests * a.prompt,), dtype=I32, device="cuda", generator=g)
        following = torch.cat((tokens[1:], tokens.new_full((1,), -1)))
        following[a.prompt - 1::a.prompt] = -1
        add = model.add * a.prompt
        run(lambda: model.prompt(tokens, following, add), 1)
        took = run(lambda: model.prompt(tokens, following, add), 1)
        print(f"{model.requests} prompts of {a.prompt} tokens, behind as many that are cached: {took:.0f} us")
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
