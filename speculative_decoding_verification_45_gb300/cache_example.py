"""Speculative rounds over an 8-bit key/value cache, end to end on one GPU.

    python -m speculative_decoding_verification_45_gb300.cache_example

A small random target (one attention layer between an embedding and its
transpose) decodes a batch of sequences: per round, prompt-lookup drafts
(ngram_propose), one forward over the last token and the drafts (cache_append,
cache_attend), the accept test (verify), the weight that each cached token
received (cache_weigh), and, when a sequence has grown past ``limit``, eviction
to ``keep`` tokens (cache_evict).  Rejected drafts leave the cache by length
alone: the next append writes over them.  Weights are added after the accept
test, from the accepted tokens' queries only: what a rejected draft looked at
must not count, and its own slot must hold no weight when another token takes it.
"""
from __future__ import annotations

import argparse
import math

import torch

import speculative_decoding_verification_45_gb300 as sv


class Decoder:
    """Weights, cache and state of a batch; ``step`` runs one round."""

    def __init__(self, batch=4, vocab=512, heads=8, kv_heads=2, dim=64, block=16, limit=192, keep=96, recent=32, gamma=4,
                 room=1024, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

        width = heads * dim
        self.heads, self.kv_heads, self.dim, self.gamma, self.generator = heads, kv_heads, dim, gamma, g
        self.limit, self.keep, self.recent = limit, keep, recent
        self.embed = rand(vocab, width)
        self.wq = rand(width, width, scale=1 / math.sqrt(width))
        self.wkv = rand(width, 2 * kv_heads * dim, scale=1 / math.sqrt(width))
        self.slopes = torch.exp2(-8 * torch.arange(1, heads + 1, device=device).float() / heads)
        # two sets of pages per sequence: the one in use, and the one that an eviction moves to
        per = -(-(limit + gamma + 1) // block)
        pages = 2 * batch * per
        codes = torch.zeros(2, pages, kv_heads, block, dim, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        scales = torch.ones(2, pages, kv_heads, device=device)
        self.cache = sv.KVCache(codes[0], codes[1], scales[0], scales[1],
                                torch.zeros(pages, kv_heads, block, dtype=torch.int32, device=device))
        self.weights = torch.zeros(pages, kv_heads, block, device=device)
        self.table, self.other = torch.arange(pages, dtype=torch.int32, device=device).reshape(2, batch, per).unbind(0)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)  # cached tokens
        self.text = torch.zeros(batch, room, dtype=torch.int32, device=device)
        self.text[:, :2] = torch.randint(0, vocab, (batch, 2), generator=g, device=device, dtype=torch.int32)
        self.text_len = torch.full((batch,), 2, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.evictions = 0

    def forward(self, tokens, num_new, positions):
        """Logits [batch, n, vocab] of the newest tokens; their keys and values enter the cache.  What `weigh` needs of
        them is kept until the next forward."""
        batch, n = tokens.shape
        x = self.embed[tokens.long()]
        q = (x @ self.wq).view(batch, n, self.heads, self.dim)
        kv = (x @ self.wkv).view(batch, n, 2, self.kv_heads, self.dim)
        sv.cache_append(self.cache, self.table, self.lengths, kv[:, :, 0], kv[:, :, 1], num_new=num_new,
                        positions=positions, status=self.status)
        lengths = self.lengths + num_new
        out, lse = sv.cache_attend(q, self.cache, self.table, lengths, num_new=num_new, slopes=self.slopes,
                                   status=self.status)
        self.asked = q, lse
        return (x + out.view(batch, n, -1)) @ self.embed.t()

    def weigh(self, num_new):
        """Weights from the first num_new queries of the last forward; `lengths` counts their tokens already."""
        q, lse = self.asked
        sv.cache_weigh(q, self.cache, self.table, self.lengths, lse, self.weights, num_new=num_new, slopes=self.slopes,
                       status=self.status)

    def step(self, temperature=0.7):
        """One round; returns (emitted tokens [batch, gamma + 1], accepted drafts [batch])."""
        batch, gamma, dev = len(self.lengths), self.gamma, self.text.device
        drafts, num_draft = sv.ngram_propose(self.text, self.text_len, 1, 3, gamma)
        last = self.text.gather(1, (self.text_len - 1).long()[:, None])
        tokens = torch.cat([last, drafts.clamp(min=0)], 1)
        # positions in the text go on where the last token stands, whatever an eviction has removed
        positions = (self.text_len - 1)[:, None] + torch.arange(gamma + 1, dtype=torch.int32, device=dev)
        # rows come newest last, so a shorter row's tokens are its first num_draft + 1 ones
        logits = self.forward(tokens, num_draft + 1, positions.contiguous())
        uniforms = torch.rand(batch, gamma + 1, generator=self.generator, device=dev)
        emitted, accepted = sv.verify(logits, None, drafts, num_draft, uniforms,
                                      torch.full((batch,), temperature, device=dev), status=self.status)
        at = self.text_len[:, None] + torch.arange(gamma + 1, device=dev)
        keep = torch.arange(gamma + 1, device=dev) <= accepted[:, None]
        self.text.scatter_(1, at.clamp(max=self.text.shape[1] - 1).long(), torch.where(keep, emitted, 0).to(torch.int32))
        self.text_len += accepted + 1
        self.lengths += accepted + 1  # the accepted part of what was appended
        self.weigh(accepted + 1)
        if int(self.lengths.max()) + gamma + 1 > self.limit:
            self.lengths, _ = sv.cache_evict(self.cache, self.table, self.lengths, self.weights, self.keep, self.recent,
                                             self.other, status=self.status)
            self.table, self.other = self.other, self.table
            self.weights[self.other.reshape(-1).long()] = 0
            self.evictions += 1
        return emitted, accepted


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rounds", type=int, default=200)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args(argv)
    d = Decoder(batch=a.batch)
    total = torch.zeros(a.batch, dtype=torch.int64, device="cuda")
    for _ in range(a.rounds):
        total += d.step()[1]
    print(f"{a.rounds} rounds: {d.text_len.float().mean():.1f} tokens a sequence, {total.float().mean() / a.rounds:.2f} "
          f"drafts accepted a round, {int(d.lengths.max())} tokens cached at most, {d.evictions} evictions, status {int(d.status)}")


if __name__ == "__main__":
    main()
