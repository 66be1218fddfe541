"""Prompts and decode steps of the model of examples/decode_step.py with positions: the plan, the rotation on the way to
the cache, attention of many tokens over it, and the log-probabilities of the prompt's tokens, as they are used together,
against the same model in 64 bits; and as a CUDA graph that is replayed on other prompts."""
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
BASE = 1e4


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
    """The model in 64 bits on the CPU, without roundings: one request's tokens, any number at a time."""

    def __init__(self, m):
        self.m = m
        shapes = {"qkv": (m.qkv, m.hidden), "o": (m.hidden, m.q_heads * m.dim), "gate": (m.ffn, m.hidden), "up": (m.ffn, m.hidden), "down": (m.hidden, m.ffn)}
        self.layers = [{**{k: dense(l[k], *s) for k, s in shapes.items()}, "norm1": l["norm1"].cpu().double(), "norm2": l["norm2"].cpu().double()} for l in m.layers]
        self.head, self.norm, self.embed = dense(m.head, m.vocab, m.hidden), m.norm.cpu().double(), m.embed.cpu().double()
        none = torch.zeros(0, m.kv_heads, m.dim, dtype=torch.float64)
        self.cache = [[(none, none) for _ in m.layers] for _ in range(m.requests)]

    def rotated(self, x, pos):
        half = self.m.dim // 2
        angle = pos.double()[:, None, None] * BASE ** (-torch.arange(half, dtype=torch.float64) / half)
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    def tokens(self, r, tokens):
        m, h = self.m, self.embed[tokens.long()]
        rms = lambda h, g: h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * g  # noqa: E731
        group = m.q_heads // m.kv_heads
        for i, layer in enumerate(self.layers):
            k, v = self.cache[r][i]
            pos = len(k) + torch.arange(len(tokens))
            y = (rms(h, layer["norm1"]) @ layer["qkv"].T).view(len(tokens), -1, m.dim)
            q = self.rotated(y[:, :m.q_heads], pos)
            k = torch.cat((k, self.rotated(y[:, m.q_heads:m.q_heads + m.kv_heads], pos)))
            v = torch.cat((v, y[:, m.q_heads + m.kv_heads:]))
            self.cache[r][i] = k, v
            s = torch.einsum("nhd,thd->nht", q, k.repeat_interleave(group, 1)) / math.sqrt(m.dim)
            s = s.masked_fill(torch.arange(len(k))[None, None, :] > pos[:, None, None], -math.inf)
            h = h + torch.einsum("nht,thd->nhd", torch.softmax(s, -1), v.repeat_interleave(group, 1)).reshape(len(tokens), -1) @ layer["o"].T
            x = rms(h, layer["norm2"])
            h = h + (torch.nn.functional.silu(x @ layer["gate"].T) * (x @ layer["up"].T)) @ layer["down"].T
        return rms(h, self.norm) @ self.head.T


def block(m, counts, pad, seed):
    """Random tokens of the requests' lengths with `pad` more behind them, and what follows each: the next one of
    its request."""
    n = sum(counts) + pad
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, m.vocab, (n,), generator=g, dtype=torch.int32)
    following = torch.full((n,), -1, dtype=torch.int32)
    at = 0
    for c in counts:
        if c:
            following[at:at + c - 1] = tokens[at + 1:at + c]
        at += c
    return tokens, following, torch.tensor(counts, dtype=torch.int32)


def size(**more):
    return dict(requests=3, max_len=400, page=16, vocab=1024, hidden=512, q_heads=4, kv_heads=2, ffn=512, rotate=BASE, **more)


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_and_steps_against_the_model_in_64_bits(example, cache, dim):
    m = example.Decoder(**size(cache=cache, dim=dim))
    plain = Plain(m)
    # Roundings to bf16 move a vector by at most 2^-8 of its norm: of a layer, 2 of the stream, 2 of the norms' outputs,
    # and in a prompt those of each projection's output (qkv, o, gate, up, down), of rotated q and k, of the attention's
    # output, of h and of silu: 13 at most; at the end 3 and the logits.  Uncorrelated, and as much again for how far a
    # change of the stream is carried on.  An e4m3 cache rounds keys and values by 2^-4 at most.
    part = 2.0 ** -8 * math.sqrt(2 * 13 + 4) * 2 + (2.0 ** -4 if cache == E4M3 else 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [0, 0, 0]
    for call, (counts, pad) in enumerate((((37, 0, 130), 5), ((1, 0, 70), 0), ((100, 1, 2), 1))):
        tokens, following, add = block(m, counts, pad, call)
        before = m.tokens.tolist()
        m.u.uniform_(0.0, 1.0, generator=g)
        logits, logp, rank = m.prompt(tokens.cuda(), following.cuda(), add.cuda())
        at = 0
        for r, c in enumerate(counts):
            lens[r] += c
            if not c:
                assert int(m.tokens[r]) == before[r]
                continue
            want = plain.tokens(r, tokens[at:at + c])
            mine = logits[at:at + c].double().cpu()
            assert (mine - want).norm() / want.norm() <= part, (call, r, float((mine - want).norm() / want.norm()))
            # the following tokens' probability and rank, of the logits that came out.  fp32 sums of 1024 terms, a
            # logarithm and differences of numbers below 16: 2^-16
            share = torch.log_softmax(mine, -1)
            for i in range(c - 1):
                t = int(following[at + i])
                assert abs(float(logp[at + i]) - float(share[i, t])) <= 2.0 ** -16
                before_it = (mine[i] > mine[i, t]).sum() + (mine[i, :t] == mine[i, t]).sum()
                assert int(rank[at + i]) == int(before_it)
            assert mine[-1, int(m.tokens[r])] >= torch.topk(mine[-1], 40).values[-1]
            at += c
        assert m.lens.tolist() == lens and m.status.tolist() == [0] * 3
    for i in range(4):  # then one token at a time, which the requests chose themselves
        before = m.tokens.cpu()
        m.u.uniform_(0.0, 1.0, generator=g)
        logits, _ = m.step()
        want = torch.cat([plain.tokens(r, before[r:r + 1]) for r in range(3)])
        off = (logits.double().cpu() - want).norm() / want.norm()
        assert off <= part, (i, float(off))
    assert m.lens.tolist() == [n + 4 for n in lens] and m.status.tolist() == [0] * 3
    assert example.q4k.q4k_get_device_error() == 0


def test_prompts_as_a_graph_give_the_same(example):
    def run(graphed):
        m = example.Decoder(**size())
        n = 90
        tokens, following, add = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3))
        add = add[:3]
        call = lambda: m.prompt(tokens, following, add)  # noqa: E731
        m.u.fill_(0.5)
        blocks = [block(m, counts, n - sum(counts), i) for i, counts in enumerate(((40, 3, 47), (0, 0, 0), (1, 60, 0), (9, 9, 9)))]
        if graphed:
            keep = [t.clone() for t in (m.lens, m.table, m.pool, m.state, m.tokens)]
            call()  # what is set up on a first call is set up outside of the capture
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = call()
            for t, k in zip((m.lens, m.table, m.pool, m.state, m.tokens), keep):
                t.copy_(k)
        seen = []
        for b in blocks:
            for to, of in zip((tokens, following, add), b):
                to.copy_(of)
            if graphed:
                graph.replay()
            else:
                out = call()
            used = int(b[2].sum())
            seen.append([t[:used].clone().cpu() for t in out] + [m.tokens.cpu().clone(), m.lens.cpu().clone()])
        return seen

    for a, b in zip(run(False), run(True)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_a_model_without_positions_takes_no_prompt(example):
    m = example.Decoder(requests=1, layers=1, hidden=256, q_heads=2, kv_heads=1, ffn=256, vocab=256, max_len=32)
    with pytest.raises(ValueError):
        m.prompt(m.tokens, m.tokens, m.add)
