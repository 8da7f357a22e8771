#!/usr/bin/env python3
"""Continuous batching on the low-bit library: a small random-weight decoder served step by step.

    python examples/serve_step.py [--steps N]

Every step takes whatever tokens the requests bring -- a prompt, a chunk of one, or the token just
chosen -- and runs
    lb_kv_plan                             pages and slots of the new tokens
    per layer: lb_quantize_q8_0, lb_gemv/gemm_q2_0_g64_grouped (q|k|v), lb_kv4_append, lb_attn_kv4,
               and the output, gate|up and down projections
    lb_gemv_bf16, lb_logits_adjust         head, penalties, biases and a grammar's mask
on fp32 activations.  Norms, rotary positions and the choice of the token are plain torch.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import bit_matvec_lb_gb300 as lb
import synth

HIDDEN, HEADS, KV_HEADS, DIM, FFN, LAYERS, VOCAB = 512, 8, 2, 64, 1024, 2, 1000
PAGE, PAGES = 16, 256


class Matrix:
    """Q2_0_g64 weights [N][K], repacked on the device."""

    def __init__(self, N, K, seed):
        blocks = torch.from_numpy(np.ascontiguousarray(synth.q2_0_blocks(N, K, seed=seed).reshape(-1))).cuda()
        self.N, self.K = N, K
        self.bits = torch.empty(N * K // 4, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(N * lb.scale_stride(K, 64), dtype=torch.int16, device="cuda")
        lb.lb_repack_q2_0_g64(blocks, N, K, self.bits, self.scales)


def project(x, mats):
    """x [T][K] fp32 times each of the matrices: decode GEMV up to eight tokens, GEMM beyond."""
    T, K = x.shape
    q = torch.empty((T, K), dtype=torch.int8, device="cuda")
    d = torch.empty((T, K // 32), dtype=torch.int16, device="cuda")
    lb.lb_quantize_q8_0(x.contiguous(), q, d, T, K)
    y = [torch.empty((T, m.N), dtype=torch.float32, device="cuda") for m in mats]
    if T <= 8:
        lb.lb_gemv_q2_0_g64_grouped([(m.bits, m.scales, o, None, m.N) for m, o in zip(mats, y)], q, d, K, T)
    else:
        ws = torch.empty(lb.lb_gemm_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        lb.lb_gemm_q2_0_g64_grouped([(m.bits, m.scales, o, m.N) for m, o in zip(mats, y)], q, d, T, K, ws)
    return y


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def rotate(x, position):
    """Rotary positions on [T][heads][DIM]."""
    f = 10000.0 ** (-torch.arange(0, DIM, 2, device="cuda") / DIM)
    a = position[:, None, None] * f
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1).flatten(-2)


class Server:
    def __init__(self, requests, grammar=None, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.R = requests
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda")
        self.head = torch.from_numpy(synth.bf16_weights(VOCAB, HIDDEN, seed=seed).view(np.int16)).cuda()
        self.layers = []
        for i in range(LAYERS):
            s = 100 * i + seed
            self.layers.append(dict(qkv=[Matrix(HEADS * DIM, HIDDEN, s), Matrix(KV_HEADS * DIM, HIDDEN, s + 1),
                                         Matrix(KV_HEADS * DIM, HIDDEN, s + 2)],
                                    out=[Matrix(HIDDEN, HEADS * DIM, s + 3)],
                                    up=[Matrix(FFN, HIDDEN, s + 4), Matrix(FFN, HIDDEN, s + 5)],
                                    down=[Matrix(HIDDEN, FFN, s + 6)],
                                    cache=torch.empty(lb.kv4_cache_bytes(PAGES, KV_HEADS, PAGE, DIM),
                                                      dtype=torch.uint8, device="cuda")))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.past = torch.zeros(requests, **i32)
        self.table = torch.full((requests, PAGES), -1, **i32)
        self.free = torch.randperm(PAGES, generator=g, device="cuda").int()
        self.counts = [torch.zeros(2, **i32), torch.zeros(2, **i32)]
        self.grammar = grammar           # allowed tokens as bits, [1][ceil(VOCAB / 32)] int32, or None
        self.prompts = [[] for _ in range(requests)]
        self.answers = [[] for _ in range(requests)]

    def step(self, tokens):
        """tokens: a list per request (empty: idle).  Returns adjusted logits [requests][VOCAB]; rows
        of idle requests mean nothing."""
        R, T = self.R, sum(len(t) for t in tokens)
        ids = torch.tensor(sum(tokens, []), device="cuda")
        fresh = torch.tensor([len(t) for t in tokens], dtype=torch.int32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        q_start, kv_len = torch.empty(R + 1, **i32), torch.empty(R, **i32)
        position, slot = torch.empty(T, **i32), torch.empty(T, dtype=torch.int64, device="cuda")
        before, after = self.counts
        lb.lb_kv_plan(self.past, fresh, R, self.free, PAGES, before[1:], PAGE, self.table, PAGES, T, q_start,
                      kv_len, position, slot, after)
        self.counts = [after, before]
        most = max(len(t) for t in tokens)
        ws = torch.empty(lb.lb_attn_kv4_workspace_bytes(HEADS, KV_HEADS, DIM, most), dtype=torch.uint8, device="cuda")
        x = self.embed[ids]
        for layer in self.layers:
            q, k, v = project(norm(x), layer["qkv"])
            q = rotate(q.unflatten(1, (HEADS, DIM)), position).contiguous()
            k = rotate(k.unflatten(1, (KV_HEADS, DIM)), position).contiguous()
            lb.lb_kv4_append(k, v, lb.OUT_F32, KV_HEADS * DIM, KV_HEADS * DIM, slot, T, layer["cache"], PAGES, PAGE,
                             KV_HEADS, DIM)
            a = torch.empty_like(q)
            lb.lb_attn_kv4(q, lb.OUT_F32, HEADS * DIM, layer["cache"], PAGES, PAGE, HEADS, KV_HEADS, DIM, self.table,
                           PAGES, q_start, kv_len, R, T, most, DIM ** -0.5, True, 0, a, HEADS * DIM, None, ws)
            x = x + project(a.flatten(1), layer["out"])[0]
            gate, up = project(norm(x), layer["up"])
            x = x + project(torch.nn.functional.silu(gate) * up, layer["down"])[0]
        last = norm(x[(q_start[1:] - 1).clamp(min=0).long()])
        logits = torch.empty((R, VOCAB), dtype=torch.float32, device="cuda")
        lb.lb_gemv_bf16(self.head, last, logits, VOCAB, HIDDEN, R)
        self.past = kv_len
        return self.adjust(logits)

    def adjust(self, logits):
        """Penalties for what a request's text holds, one bias, and the grammar, in place."""

        def rows(lists):
            start = np.cumsum([0] + [len(t) for t in lists]).astype(np.int32)
            return (torch.tensor(sum(lists, []) or [0], dtype=torch.int32, device="cuda"),
                    torch.from_numpy(start).cuda())

        (pi, ps), (oi, os_) = rows(self.prompts), rows(self.answers)
        bi, bs = rows([[7]] * self.R)
        f32 = dict(dtype=torch.float32, device="cuda")
        lb.lb_logits_adjust(logits, lb.OUT_F32, VOCAB, logits, VOCAB, self.R, VOCAB, prompt_ids=pi, prompt_start=ps,
                            output_ids=oi, output_start=os_, repetition=torch.full((self.R,), 1.1, **f32),
                            presence=torch.full((self.R,), 0.2, **f32), frequency=torch.full((self.R,), 0.1, **f32),
                            bias_ids=bi, bias_values=torch.full((self.R,), -1.0, **f32), bias_start=bs,
                            mask=self.grammar, mask_stride=(VOCAB + 31) // 32,
                            mask_row=None if self.grammar is None else
                            torch.zeros(self.R, dtype=torch.int32, device="cuda"))
        return logits

    def generate(self, prompts, steps, chunk=None):
        """Greedy answers of `steps` tokens to the prompts, read whole or `chunk` tokens at a time."""
        left = [list(p) for p in prompts]
        self.prompts = [list(p) for p in prompts]
        self.answers = [[] for _ in prompts]
        tokens = [[] for _ in prompts]
        while any(len(a) < steps for a in self.answers):
            for r in range(self.R):
                if left[r]:
                    n = len(left[r]) if chunk is None else min(chunk, len(left[r]))
                    tokens[r], left[r] = left[r][:n], left[r][n:]
                else:
                    tokens[r] = self.answers[r][-1:] if len(self.answers[r]) < steps else []
            best = self.step(tokens).argmax(-1).tolist()
            for r in range(self.R):
                if tokens[r] and not left[r]:
                    self.answers[r].append(best[r])
        return self.answers


def grammar_of(allowed):
    bits = np.zeros((VOCAB + 31) // 32 * 32, bool)
    bits[list(allowed)] = True
    return torch.from_numpy(np.packbits(bits, bitorder="little").view(np.int32)[None].copy()).cuda()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12)
    steps = ap.parse_args().steps
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (70, 3, 33)]
    server = Server(len(prompts), grammar=grammar_of(range(0, VOCAB, 2)))
    for prompt, answer in zip(prompts, server.generate(prompts, steps)):
        print(f"{len(prompt)} prompt tokens -> {answer}")
    assert lb.lb_device_status() == 0


if __name__ == "__main__":
    main()
