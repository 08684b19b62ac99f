"""Verifying a tree of drafted tokens with compressed layers: one decoder block and a head.

    python examples/verify_drafts.py

The qkv, o and head layers are compressed (4-bit tables with outliers); between and after them run the rotary
positions, the quantised K/V cache, attention of the tree over that cache, and the log probabilities that
accept the drafts.  Weights are random, so the text is not; the steps are those of a serving program:

    prompt   chunks of tokens, each a chain: append to the cache, attend, keep the last row's alternatives
    verify   a tree of drafted tokens at the cache's end, each seeing its ancestors, in one pass
    accept   the longest path whose tokens are the head's first choice, then its entries stay in the cache
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import compressed_linear_amd as cla  # noqa: E402
from synth.layers import make_layer  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 512, 8, 2, 64, 1000
PAGE, PAGES, MAX_NEW = 16, 64, 64


class Block:
    """A decoder block (attention only) and a head, for one sequence."""

    def __init__(self, kind: str = "int8", device: str = "cuda"):
        def layer(i, K, N):
            blob, _ = cla.pack(make_layer(2, i, K=K, N=N))
            return cla.CompressedLinear(blob, max_M=MAX_NEW, device=device)

        g = torch.Generator(device=device).manual_seed(1)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=device)
        self.qkv = layer(0, HIDDEN, (Q_HEADS + 2 * KV_HEADS) * DIM)
        self.o = layer(1, Q_HEADS * DIM, HIDDEN)
        self.head = layer(2, HIDDEN, VOCAB)
        self.rope = cla.rope_table(PAGE * PAGES, DIM, scaling="yarn", factor=2.0, trained=512, device=device)
        self.cache = cla.KVCache(PAGES, PAGE, KV_HEADS, DIM, kind, device=device)
        self.pages = torch.randperm(PAGES, generator=g, device=device).to(torch.int32)[None]  # the sequence's pages
        self.n = 0  # tokens whose entries stay

    def slots(self, at):
        """Cache slots of the sequence's places `at`."""
        return (self.pages[0, at // PAGE] * PAGE + at % PAGE).to(torch.int32)

    def forward(self, tokens, depth, tree_mask=None):
        """Logits of new tokens at the sequence's end; depth: each one's place after the tokens that stay."""
        T, dev = len(tokens), self.embed.device
        room(self.n, T)
        h = self.embed[tokens]
        position = (self.n + depth).to(torch.int32)
        slot = self.slots(torch.arange(self.n, self.n + T, device=dev))
        qkv = self.qkv(norm(h)).view(T, Q_HEADS + 2 * KV_HEADS, DIM)  # fp32
        q = cla.rope(qkv[:, :Q_HEADS], position, self.rope, out_dtype=torch.float16)
        self.cache.append(qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:], slot, position, self.rope)
        o = cla.tree_attention(q, self.cache, self.pages, torch.tensor([self.n], dtype=torch.int32, device=dev),
                               torch.tensor([0, T], dtype=torch.int32, device=dev), max_q=T, max_ctx=self.n,
                               tree_mask=tree_mask)
        h = h + self.o(o.view(T, Q_HEADS * DIM))
        return self.head(norm(h))

    def prompt(self, tokens):
        """Takes the prompt in; returns the next token's first choices."""
        if not len(tokens):
            raise ValueError("an empty prompt")
        for at in range(0, len(tokens), MAX_NEW):
            part = tokens[at:at + MAX_NEW]
            logits = self.forward(part, torch.arange(len(part), device=part.device))
            self.n += len(part)
        last = logits[-1:]
        return cla.token_logprobs(last, torch.zeros(1, 0, dtype=torch.int32, device=last.device), top_k=4)[2][0]

    def verify(self, tokens, parents):
        """One pass over a tree of drafts: token i follows token parents[i], or the sequence where that is -1.
        Returns the accepted tokens' indices, the token that follows them, and each draft's log probability and the
        entropy of what it was drawn from (both after its parent)."""
        dev, T = tokens.device, len(tokens)
        mask, depth = tree_of(parents)
        logits = self.forward(tokens, depth.to(dev), mask.to(dev))
        # what each draft says of its children (up to 4, else padding -1) and its own first choice
        children = [[j for j in range(T) if parents[j] == i][:4] for i in range(T)]
        given = torch.tensor([[int(tokens[j]) for j in c] + [-1] * (4 - len(c)) for c in children], dtype=torch.int32, device=dev)
        logp, entropy, first, _ = cla.token_logprobs(logits, given, top_k=1)
        first = first[:, 0].tolist()
        path, at, following = [], -1, None
        while True:
            want = first[at] if at >= 0 else self.expected
            step = [j for j in range(T) if parents[j] == at and int(tokens[j]) == want]
            if not step:
                following = want
                break
            at = step[0]
            path.append(at)
        self.keep(path)
        return path, following, logp, entropy

    def keep(self, path):
        """Moves the accepted drafts' entries together: they are quantised as they are, so codes and scales are copied."""
        if path:
            dev = self.embed.device
            src = self.slots(self.n + torch.tensor(path, device=dev)).long()
            dst = self.slots(self.n + torch.arange(len(path), device=dev)).long()
            for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
                t[dst // PAGE, :, dst % PAGE] = t[src // PAGE, :, src % PAGE]
        self.n += len(path)


def room(n, new):
    """Refuses new tokens that the layers or the sequence's pages do not hold (an index past the pages is an error on the GPU)."""
    if not 1 <= new <= MAX_NEW:
        raise ValueError("%d new tokens; 1 to %d at a time" % (new, MAX_NEW))
    if n + new > PAGE * PAGES:
        raise ValueError("%d tokens and %d new ones in pages for %d" % (n, new, PAGE * PAGES))


def tree_of(parents):
    """Each token's ancestors and itself as bits [tokens, 1], and its depth; at most 64 tokens."""
    mask, depth = [], []
    for i, p in enumerate(parents):
        mask.append((mask[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    # bit 63 is int64's sign
    return torch.tensor([[m - (1 << 64) if m >> 63 else m] for m in mask]), torch.tensor(depth)


def norm(h):
    return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)).to(torch.float16)


def main():
    block = Block()
    prompt = torch.arange(150, device="cuda") * 37 % VOCAB
    choices = block.prompt(prompt).tolist()
    print("prompt of %d tokens; first choices of the next: %s" % (len(prompt), choices))
    block.expected = choices[0]
    for step in range(4):
        # drafts: the expected token and an alternative, each with two children
        tokens = torch.tensor([block.expected, choices[1], 3, 5, 7, 11], device="cuda")
        path, following, logp, entropy = block.verify(tokens, [-1, -1, 0, 0, 1, 1])
        print("step %d: accepted %s, then token %d (entropy after the first draft %.3f, its children's log p %s)" % (
            step, [int(tokens[i]) for i in path], following, float(entropy[0]), [round(float(v), 3) for v in logp[0, :2]]))
        block.expected, choices = following, [following, (following + 1) % VOCAB]


if __name__ == "__main__":
    main()
