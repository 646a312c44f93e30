"""A small hybrid stack served from two kinds of state: every block is a Gated
DeltaNet layer (recurrent state in a slot) followed by a softmax attention layer
(KV cache in 4 bits). Weights are random; the point is how the calls fit together:

    prompts        gdn prefill per sequence, kv4 append + prefill for all of them
    decode         gdn decode step, kv4 append + decode, one token per sequence
    fork           the KV pages are shared until one side grows, the slot is copied
    compact        the live pages move to the front of every layer

    python examples/hybrid_stack.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_gated_deltanet_gb300 as gdn  # noqa: E402
from nvfp4_gated_deltanet_gb300 import synth  # noqa: E402


def bits(x):
    """BF16 tensor <-> its bits, as the GDN calls take them."""
    return x.contiguous().view(torch.int16)


class HybridStack:
    def __init__(self, n_blocks=2, shape=synth.TINY, n_q_heads=8, n_kv_heads=2, head_dim=64, page_tokens=16,
                 num_pages=256, slots=8, max_prompt=256, seed=0):
        self.shape, self.hq, self.hkv, self.d = shape, n_q_heads, n_kv_heads, head_dim
        self.gdn = [gdn.layer_from_synth(synth.layer_weights(shape, seed + i), max_batch=slots, max_prefill_tokens=max_prompt)
                    for i in range(n_blocks)]
        self.states = [L.new_states(slots) for L in self.gdn]
        self.cache = gdn.KV4Cache(num_pages, page_tokens, n_kv_heads, head_dim, k_scale=2.0 ** -6, v_scale=2.0 ** -6,
                                  n_layers=n_blocks)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        H, rows = shape.hidden, (n_q_heads + 2 * n_kv_heads) * head_dim

        def mat(*dims):
            return (torch.randn(*dims, generator=gen, device="cuda") * dims[0] ** -0.5).bfloat16()

        self.w_qkv = [mat(H, rows) for _ in range(n_blocks)]
        self.w_o = [mat(n_q_heads * head_dim, H) for _ in range(n_blocks)]
        self.free_slots, self.slot_of = list(range(slots)), {}

    @staticmethod
    def _norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def _attention(self, i, x, batch, rows):
        """x [T][H] -> the attention layer's output; the new rows go into the cache first."""
        qkv = (self._norm(x) @ self.w_qkv[i]).view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:]
        self.cache.append(i, k, v, batch)
        if rows is None:
            out = self.cache.prefill(i, q, batch)
        else:
            out = self.cache.decode(i, q.unflatten(0, (-1, rows)), batch)
        return x + out.reshape(x.shape[0], -1) @ self.w_o[i]

    def prompt(self, xs):
        """New sequences from prompts xs (BF16 [T_b][H] each): their ids and the stack's output rows."""
        seqs = [self.cache.new() for _ in xs]
        for s in seqs:
            self.slot_of[s] = self.free_slots.pop(0)
        batch = self.cache.grow(seqs, [x.shape[0] for x in xs])
        x = torch.cat(list(xs))
        for i, L in enumerate(self.gdn):
            conv, ssm = self.states[i]
            parts = self._norm(x).split([t.shape[0] for t in xs])
            y = [L.prefill(bits(t), self.slot_of[s], True, conv, ssm).view(torch.bfloat16) for s, t in zip(seqs, parts)]
            x = self._attention(i, x + torch.cat(y), batch, None)
        return seqs, x

    def decode(self, seqs, x):
        """One token of each sequence: x [B][H] -> [B][H]."""
        batch = self.cache.grow(seqs, 1)
        ids = torch.tensor([self.slot_of[s] for s in seqs], dtype=torch.int32, device="cuda")
        for i, L in enumerate(self.gdn):
            y = L.decode_step(bits(self._norm(x)), ids, *self.states[i]).view(torch.bfloat16)
            x = self._attention(i, x + y, batch, 1)
        return x

    def fork(self, seq):
        child = self.cache.fork(seq)
        self.slot_of[child] = self.free_slots.pop(0)
        for conv, ssm in self.states:
            conv[self.slot_of[child]].copy_(conv[self.slot_of[seq]])
            ssm[self.slot_of[child]].copy_(ssm[self.slot_of[seq]])
        return child

    def free(self, seq):
        self.cache.free(seq)
        self.free_slots.append(self.slot_of.pop(seq))

    def check(self):
        return max([self.cache.check()] + [L.check() for L in self.gdn])


def main():
    torch.manual_seed(0)
    net = HybridStack()
    H = net.shape.hidden
    prompts = [torch.randn(n, H, device="cuda").bfloat16() for n in (70, 33, 5)]
    seqs, y = net.prompt(prompts)
    print("prompts:", [net.cache.book.length(s) for s in seqs], "tokens,", net.cache.book.free_pages, "pages free")
    child = net.fork(seqs[0])
    seqs.append(child)
    x = torch.randn(len(seqs), H, device="cuda").bfloat16()
    x[3] = x[0]                                       # the fork takes the same next token ...
    y = net.decode(seqs, x)
    print("a fork's step equals its parent's:", bool(torch.equal(y[0], y[3])))
    for _ in range(20):                               # ... and then its own
        y = net.decode(seqs, torch.randn(len(seqs), H, device="cuda").bfloat16())
    net.free(seqs.pop(0))
    live = net.cache.compact()
    print("after freeing the parent:", live, "live pages at the front")
    y = net.decode(seqs, torch.randn(len(seqs), H, device="cuda").bfloat16())
    assert np.isfinite(y.float().cpu().numpy()).all() and net.check() == 0
    print("status", net.check())


if __name__ == "__main__":
    main()
