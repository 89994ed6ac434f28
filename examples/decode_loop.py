#!/usr/bin/env python3
"""Decoding with drafted tokens and a bounded cache, on the library's operators.

A LLaMA-7B-shaped decoder stack (random k-quant weights, a random embedding;
two layers unless told otherwise) reads a prompt in chunks of 16 tokens and
then generates: every step takes the last token and up to three drafted ones
(the continuation of the last earlier occurrence of the current token), runs
them through the layers together, verifies the drafts against the target's
probabilities, and drops the rejected ones.  Per layer:

    q8_1 quantisation + products (q, k, v, o, gate, up, down)
    rope_append    rotary q and k; k and v into the paged cache
    attn_decode    attention of the new tokens, adding up what each entry got; rows of
                   drafts add nothing until it is known which of them stay
    kv_evict       once the cache is `slack` entries past its budget

Norms, residuals and sampling inputs are plain torch.

    python examples/decode_loop.py [--layers 2] [--prompt 96] [--steps 40] [--budget 64]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_prefill_gemm_mmq_gb300 import ops, synth  # noqa: E402

CHUNK = 16            # tokens per prompt chunk: what the decode products and the attention take at once


class Layer:
    def __init__(self, hidden, heads, kv_heads, dim, ffn, seed, dev):
        shapes = {"q": ("q4_K", heads * dim, hidden), "k": ("q4_K", kv_heads * dim, hidden), "v": ("q6_K", kv_heads * dim, hidden),
                  "o": ("q4_K", hidden, heads * dim), "gate": ("q4_K", ffn, hidden), "up": ("q4_K", ffn, hidden),
                  "down": ("q4_K", hidden, ffn)}
        self.w = {n: (f, O, torch.from_numpy(synth.make_weights(f, O, K, seed + i)).reshape(-1).to(dev))
                  for i, (n, (f, O, K)) in enumerate(shapes.items())}

    def product(self, names, x):
        """The named projections of x [T <= 16][K], quantised once."""
        _, ds, xh, _ = ops.quantize_q8_1(x, want_qs=False, want_xa=False)
        return [ops.gemv(w, xh, ds, O, fmt=f) for f, O, w in (self.w[n] for n in names)]


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Decoder:
    """One sequence through `layers` layers; a cache of `budget` entries per layer plus room for new ones."""

    def __init__(self, layers=2, hidden=4096, heads=32, kv_heads=32, dim=128, ffn=11008, vocab=32000, page=16, room=512,
                 cache_dtype=torch.float16, seed=1, device="cuda"):
        self.dev = torch.device(device)
        g = torch.Generator(device=self.dev)
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.layers = [Layer(hidden, heads, kv_heads, dim, ffn, 100 * (seed + i), self.dev) for i in range(layers)]
        self.embed = torch.randn((vocab, hidden), generator=g, device=self.dev)
        self.rope = ops.rope_table(dim, scaling="by_parts", factor=2.0, context=4096, device=self.dev)
        cols = -(-room // page)
        self.caches = []
        for _ in range(layers):                               # one table and one length for all layers
            self.caches.append(ops.KVCache.allocate(1, cols, kv_heads, dim, page, cache_dtype, self.dev,
                                                    share=self.caches[0] if self.caches else None))
        # bookkeeping after an eviction goes to the other set
        self.spare = [(torch.zeros_like(c.weight), torch.zeros_like(c.pos)) for c in self.caches]
        self.lens = self.caches[0].lens
        self.next_pos = 0
        self.entries = 0                                      # the host's copy of the length
        self.work = {n: ops.attn_workspace(self.caches[0], heads, n, True) for n in range(1, CHUNK + 1)}
        self.evict_work = None
        self.held = None                                      # q rows per layer whose weights are not added yet

    def forward(self, tokens, drafts=0):
        """Logits of the new tokens [n <= 16][vocab]; they become the cache's last entries.

        With drafts among them, what the rows attend to is added to the entries' weights only
        when drop() says which stay: a draft that is turned down must not steer an eviction."""
        self.drop(0)
        self.held = [] if drafts else None
        n = len(tokens)
        self.lens.add_(n)
        self.entries += n
        pos = torch.arange(self.next_pos, self.next_pos + n, dtype=torch.int32, device=self.dev)
        self.next_pos += n
        x = self.embed[torch.tensor(tokens, device=self.dev)]
        for layer, cache in zip(self.layers, self.caches):
            q, k, v = layer.product(("q", "k", "v"), norm(x))
            q = ops.rope_append(cache, self.rope, norm(q.view(n, self.heads, self.dim)), norm(k.view(n, self.kv_heads, self.dim)),
                                v.view(n, self.kv_heads, self.dim), pos)
            a = ops.attn_decode(cache, q, accumulate=not drafts, workspace=self.work[n])
            if drafts:
                self.held.append(q)
            o, = layer.product(("o",), norm(a.view(n, -1)))
            x = x + norm(o)
            gate, up = layer.product(("gate", "up"), norm(x))
            down, = layer.product(("down",), norm(torch.nn.functional.silu(norm(gate)) * up))
            x = x + norm(down)
        return norm(x) @ self.embed.T * x.shape[-1] ** -0.5

    def drop(self, n):
        """Take the last n entries back (rejected drafts), and add the weights of the rows that stay."""
        if n:
            self.lens.sub_(n)
            self.entries -= n
            self.next_pos -= n
        if self.held:
            rows = self.held[0].shape[0]
            stay = torch.full((1,), rows - n, dtype=torch.int32, device=self.dev)
            for cache, q in zip(self.caches, self.held):
                ops.attn_decode(cache, q, new=stay, accumulate=True, workspace=self.work[rows])
            self.held = None

    def evict(self, budget, recent):
        self.drop(0)
        keep_from = torch.full((1,), self.next_pos - recent, dtype=torch.int32, device=self.dev)
        if self.evict_work is None:
            self.evict_work = ops.evict_workspace(self.caches[0], budget)
        for i, cache in enumerate(self.caches):
            old = (cache.weight, cache.pos)
            ops.kv_evict(cache, budget, keep_from, *self.spare[i], workspace=self.evict_work)
            cache.set_bookkeeping(*self.spare[i])
            self.spare[i] = old
        self.lens.clamp_(max=budget)
        self.entries = min(self.entries, budget)


def draft(history, most):
    """The tokens that followed the current one when it came last before."""
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1]:
            return history[i + 1:i + 1 + most]
    return []


def generate(model, prompt, steps, budget, slack=32, drafts=3, temperature=0.05, seed=3):
    """Tokens after the prompt, and (drafted, accepted, evictions)."""
    g = torch.Generator(device=model.dev)
    g.manual_seed(seed)
    history, count = list(prompt), [0, 0, 0]
    for i in range(0, len(prompt) - 1, CHUNK):                 # the last prompt token opens the first step
        model.forward(prompt[i:min(i + CHUNK, len(prompt) - 1)])
        if model.entries > budget + slack:
            model.evict(budget, recent=budget // 4)
            count[2] += 1
    for _ in range(steps):
        guess = draft(history, drafts)
        n = len(guess)
        target = torch.softmax(model.forward([history[-1]] + guess, drafts=n) / temperature, -1)[None]
        uniform = torch.rand((1, n + 1), generator=g, device=model.dev)
        if n:
            tokens, accepted = ops.spec_verify(target.contiguous(), None, torch.tensor([guess], dtype=torch.int32, device=model.dev), uniform)
        else:                                                  # nothing drafted: one token that cannot be accepted
            tokens, accepted = ops.spec_verify(target.expand(1, 2, -1).contiguous(), None,
                                               torch.zeros((1, 1), dtype=torch.int32, device=model.dev), uniform.expand(1, 2).contiguous(),
                                               count=torch.zeros(1, dtype=torch.int32, device=model.dev))
        a = int(accepted[0])
        history += tokens[0, :a + 1].tolist()
        model.drop(n - a)
        count[0] += n
        count[1] += a
        if model.entries > budget + slack:
            model.evict(budget, recent=budget // 4)
            count[2] += 1
    ops.check_status(model.dev)
    return history[len(prompt):], tuple(count)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=96)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--budget", type=int, default=64)
    args = ap.parse_args()
    g = torch.Generator().manual_seed(5)
    prompt = torch.randint(0, 200, (args.prompt,), generator=g).tolist()
    model = Decoder(layers=args.layers, room=args.prompt + args.budget + 4 * args.steps + 64)
    out, (drafted, accepted, evictions) = generate(model, prompt, args.steps, args.budget)
    torch.cuda.synchronize()
    print(f"{len(out)} tokens in {args.steps} steps: {accepted} of {drafted} drafts accepted, {evictions} evictions to {args.budget} entries, "
          f"{model.entries} entries in the cache at position {model.next_pos}")


if __name__ == "__main__":
    main()
