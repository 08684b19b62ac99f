"""Several answers to a prompt with an image: one decoder block and a head in 8-bit integers.

    python examples/image_answers.py

The layers quantise their activations by token (Int8Linear), positions have three axes (time, height, width), and
the answers share the prompt's pages.  Weights are random, so the text is not; the steps are those of a serving program:

    prompt   text, an image's patches and text join the cache as one chain
    fork     each answer starts as a copy of the prompt: its pages are shared, the last one is copied once it is written
    step     every answer's drafts in one pass over its own pages; the accepted ones are moved together, the rest given back
    end      an ended answer's pages are free again, and the pool is compacted
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import compressed_linear_amd as cla  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 512, 8, 2, 64, 1000
PAGE, PAGES, WIDTH, MOST = 16, 96, 24, 256
SECTIONS, ORDER = (12, 10, 10), "turns"


class Answers:
    """A decoder block (attention only) and a head, for a few sequences."""

    def __init__(self, sequences: int = 4, kind: str = "int8", device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(1)

        def layer(K, N):
            return cla.Int8Linear.from_weight(torch.randn(N, K, generator=g, device=device) / K ** 0.5)

        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=device)
        self.qkv = layer(HIDDEN, (Q_HEADS + 2 * KV_HEADS) * DIM)
        self.o = layer(Q_HEADS * DIM, HIDDEN)
        self.head = layer(HIDDEN, VOCAB)
        self.rope = cla.rope_table(PAGE * WIDTH, DIM, device=device)
        self.cache = cla.KVCache(PAGES, PAGE, KV_HEADS, DIM, kind, device=device)
        self.pool = cla.PagePool(PAGES, PAGE, sequences, WIDTH, device=device)
        self.next_position = [0] * sequences  # of text: an image's patches take fewer positions than places
        self.device = device

    def forward(self, hidden, counts, positions, tree_mask=None):
        """Logits of the sequences' new tokens (hidden [tokens, HIDDEN], counts of each sequence, positions [3, tokens]); they join
        the cache.  Where one of them has no room none does, and the sequences stay as they were."""
        T, dev = len(hidden), self.device
        if sum(counts) != T:
            raise ValueError("%d tokens, but %d are counted" % (T, sum(counts)))
        room(counts)
        cu = torch.tensor([0] + counts, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        before = self.pool.lens.clone()
        slots, src, dst = self.pool.extend(cu, T)
        self.cache.copy_pages(src, dst)
        if int(self.pool.left_out):  # the others have their room and their copies already: what they got is given back
            self.pool.truncate(before)
            raise RuntimeError("no pages are left")
        position = positions.to(torch.int32).contiguous()
        qkv = self.qkv(norm(hidden)).view(T, Q_HEADS + 2 * KV_HEADS, DIM)  # fp32
        q = cla.rope(qkv[:, :Q_HEADS], position, self.rope, out_dtype=torch.float16, sections=SECTIONS, order=ORDER)
        self.cache.append(qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:], slots, position, self.rope,
                          sections=SECTIONS, order=ORDER)
        o = cla.tree_attention(q, self.cache, self.pool.block_table, before, cu, max_q=max(counts), tree_mask=tree_mask)
        hidden = hidden + self.o(o.view(T, Q_HEADS * DIM))
        return before, self.head(norm(hidden))

    def prompt(self, text, patches, more):
        """Sequence 0 takes text, an image's patches [height, width, HIDDEN] and more text in; returns the next token's first choices."""
        h, w = patches.shape[:2]
        n, m = len(text), len(more)
        hidden = torch.cat([self.embed[text], patches.reshape(h * w, HIDDEN), self.embed[more]])
        line = torch.arange(max(n, m), device=self.device)
        at = torch.arange(h * w, device=self.device)
        grid = torch.stack([torch.zeros_like(at), at // w, at % w])
        after = n + max(h, w)  # text goes on past the image's largest position
        positions = torch.cat([line[:n].expand(3, n), n + grid, after + line[:m].expand(3, m)], 1)
        counts = [n + h * w + m] + [0] * (self.pool.sequences - 1)
        _, logits = self.forward(hidden, counts, positions)
        self.next_position[0] = after + m
        return self.choices(logits[-1:])[0]

    def choices(self, logits):
        none = torch.zeros(len(logits), 0, dtype=torch.int32, device=self.device)
        return cla.token_logprobs(logits, none, top_k=4)[2].tolist()

    def fork(self, n):
        """The first n sequences become copies of sequence 0."""
        parents = torch.arange(self.pool.sequences, dtype=torch.int32, device=self.device)
        parents[:n] = 0
        self.pool.fork(parents)
        self.next_position = [self.next_position[0] if b < n else p for b, p in enumerate(self.next_position)]

    def step(self, drafts):
        """drafts: for each sequence a list of tokens that follow one another (empty: it waits).  The first one is taken as given; a
        later one is accepted while it is what the model chooses after the one before.  Returns each sequence's accepted tokens
        and the choices after them."""
        counts = [len(d) for d in drafts]
        room(counts)
        tokens = torch.tensor([t for d in drafts for t in d], device=self.device)
        at = torch.tensor([self.next_position[b] + i for b, d in enumerate(drafts) for i in range(len(d))], device=self.device)
        before, logits = self.forward(self.embed[tokens], counts, at.expand(3, len(tokens)))
        chosen, out, first = self.choices(logits), [], 0
        keep = torch.full((len(drafts), max(counts)), -1, dtype=torch.int32)
        for b, d in enumerate(drafts):
            n = min(1, len(d))
            while n < len(d) and d[n] == chosen[first + n - 1][0]:
                n += 1
            keep[b, :n] = torch.arange(n)
            out.append((d[:n], chosen[first + n - 1] if n else None))
            self.next_position[b] += n
            first += len(d)
        self.cache.keep(self.pool.block_table, before, keep.to(self.device))
        self.pool.truncate(before + (keep >= 0).sum(1).to(self.device, torch.int32))
        return out

    def end(self, sequences):
        """The sequences' pages are given back, and those that are left moved to the pool's start."""
        lens = torch.full((self.pool.sequences,), -1, dtype=torch.int32, device=self.device)
        lens[sequences] = 0
        self.pool.truncate(lens)
        self.cache.copy_pages(*self.pool.compact())
        for b in sequences:
            self.next_position[b] = 0


def room(counts):
    """Refuses a pass without new tokens, or with more of a sequence than the attention takes."""
    if not 1 <= max(counts) <= MOST:
        raise ValueError("1 to %d new tokens to a sequence" % MOST)


def norm(h):
    return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)).to(torch.float16)


def main():
    a = Answers()
    g = torch.Generator(device="cuda").manual_seed(2)
    image = torch.randn(6, 9, HIDDEN, generator=g, device="cuda")
    choices = a.prompt(torch.arange(21, device="cuda"), image, torch.arange(40, 50, device="cuda"))
    print("prompt of 21 + 6 x 9 + 10 tokens; first choices of the next: %s" % choices)
    a.fork(4)
    drafts = [[c, 7, 8] for c in choices]
    for step in range(3):
        out = a.step(drafts)
        print("step %d: %s; pages held %d" % (step, ["%s then %d" % (d, c[0]) for d, c in out], int((a.pool.refs > 0).sum())))
        drafts = [[c[0], c[1], c[2]] for _, c in out]
    a.end([1, 2])
    print("two answers ended; pages held %d, the highest is %d" % (int((a.pool.refs > 0).sum()), int(a.pool.refs.nonzero().max())))


if __name__ == "__main__":
    main()
