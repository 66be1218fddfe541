"""The decode step of examples/decode_step.py: its logits against the same model in 64 bits, over several steps
with a growing cache, and the whole run as a CUDA graph."""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import pytest
import torch

import oracle

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def example():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import decode_step
    assert decode_step.q4k.q4k_get_device_error() == 0
    return decode_step


def dense(w, n, k):
    return torch.from_numpy(np.asarray(oracle.dequant_f32(w.cpu().numpy(), n, k), dtype=np.float64).reshape(n, k))


class Plain:
    """The model in 64 bits on the CPU, without roundings, fed the tokens that the GPU chose."""

    def __init__(self, m):
        self.m = m
        shapes = {"qkv": (m.qkv, m.hidden), "o": (m.hidden, m.q_heads * m.dim), "gate": (m.ffn, m.hidden), "up": (m.ffn, m.hidden), "down": (m.hidden, m.ffn)}
        self.layers = [{**{k: dense(l[k], *s) for k, s in shapes.items()}, "norm1": l["norm1"].cpu().double(), "norm2": l["norm2"].cpu().double(), "k": [], "v": []} for l in m.layers]
        self.head, self.norm, self.embed = dense(m.head, m.vocab, m.hidden), m.norm.cpu().double(), m.embed.cpu().double()

    def step(self, tokens):
        m = self.m
        rms = lambda h, g: h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * g  # noqa: E731
        h = self.embed[tokens.long()]
        group = m.q_heads // m.kv_heads
        for layer in self.layers:
            y = (rms(h, layer["norm1"]) @ layer["qkv"].T).view(m.requests, -1, m.dim)
            q = y[:, :m.q_heads]
            layer["k"].append(y[:, m.q_heads:m.q_heads + m.kv_heads])
            layer["v"].append(y[:, m.q_heads + m.kv_heads:])
            k, v = (torch.stack(layer[x], 1).repeat_interleave(group, 2) for x in "kv")
            p = torch.softmax(torch.einsum("nhd,nthd->nht", q, k) / math.sqrt(m.dim), -1)
            h = h + torch.einsum("nht,nthd->nhd", p, v).reshape(m.requests, -1) @ layer["o"].T
            x = rms(h, layer["norm2"])
            h = h + (torch.nn.functional.silu(x @ layer["gate"].T) * (x @ layer["up"].T)) @ layer["down"].T
        return rms(h, self.norm) @ self.head.T


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
def test_decode_step_against_the_model_in_64_bits(example, cache):
    m = example.Decoder(requests=3, max_len=64, cache=cache, vocab=1024, hidden=512, q_heads=4, kv_heads=2, ffn=512)
    plain = Plain(m)
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(20):
        before = m.tokens.cpu()
        m.u.uniform_(0.0, 1.0, generator=g)
        logits, logp = m.step()
        want = plain.step(before)
        # A layer rounds its stream twice to bf16 and each projection's input once; a rounding moves a vector by
        # at most 2^-8 of its norm: 2 layers x (2 + 5) + 3 of them, uncorrelated, and as much again for how far a
        # change of the stream is carried on.  An e4m3 cache rounds keys and values by 2^-4 at most.
        part = 2.0 ** -8 * math.sqrt(17) * 2 + (2.0 ** -4 if cache == E4M3 else 0)
        off = (logits.double().cpu() - want).norm() / want.norm()
        assert off <= part, (i, float(off))
        # the token is drawn from these logits: one of the 40 highest, and its probability as told
        x = logits.double().cpu()
        token = m.tokens.cpu().long()
        for r in range(m.requests):
            top = torch.topk(x[r], 40)
            assert int(token[r]) in top.indices.tolist()
            share = torch.softmax(top.values / 0.8, 0)[top.indices == token[r]]
            assert share.log() - 1e-6 <= float(logp[r]) <= share.log() - math.log(0.95) + 0.06
    assert m.lens.tolist() == [20] * 3 and m.status.tolist() == [0] * 3
    assert example.q4k.q4k_get_device_error() == 0


def test_decode_step_as_a_graph_gives_the_same_tokens(example):
    def run(graphed):
        m = example.Decoder(requests=4, max_len=64, vocab=1024)
        g = torch.Generator(device="cuda").manual_seed(5)
        step = m.step
        if graphed:
            keep = [t.clone() for t in (m.lens, m.table, m.pool, m.state, m.tokens)]
            m.step()  # what is set up on a first call is set up outside of the capture
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                m.step()
            for t, k in zip((m.lens, m.table, m.pool, m.state, m.tokens), keep):
                t.copy_(k)
            step = graph.replay
        seen = []
        for _ in range(24):
            m.u.uniform_(0.0, 1.0, generator=g)
            step()
            seen.append(m.tokens.clone())
        torch.cuda.synchronize()
        return torch.stack(seen).tolist()

    assert run(False) == run(True)
