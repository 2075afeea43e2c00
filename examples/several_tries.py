"""Several tries of each request over one cache: an 8-bit head, drawn tokens, and
caches that are forked and given back.

A one-layer toy model (random weights) stands in for the forward.  Each prompt is
written into the 4-bit cache once and its request forked: the tries share its full
pages and own a copy of the last one.  Every try then denoises its blocks: the
head's product in 8 bits makes the logits of the masked positions, a token is drawn
for each with the try's own random numbers, and the step commits the surest.  When
a block of all tries is done they are reported, the best try of each request is
kept, the others' pages go back, and the next block starts with forks of the best.
At the end the pool's gaps are closed.

    python examples/several_tries.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import denoise_step_token_gb300 as dllm

HEADS, GROUP, D = 2, 4, 64
PAGE = 16


class Toy:
    """Embeddings, one attention layer's projections and an LM head in 8 bits."""

    def __init__(self, V, dev, gen):
        self.q = HEADS * GROUP * D
        rand = lambda *shape: torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
        self.embed = rand(V + 1, 256)                                    # the last row: the mask
        self.qkv = rand(256, self.q + 2 * HEADS * D) / 16
        self.head = dllm.fp8_quantize(rand(V, self.q) / 4, block_rows=128)

    def project(self, ids):
        """Queries [B, L, q_heads, D], keys and values [B, L, HEADS, D]: slices of one projection."""
        x = (self.embed[ids.long()] @ self.qkv).unflatten(-1, (-1, D))
        return x[:, :, :HEADS * GROUP], x[:, :, HEADS * GROUP:-HEADS], x[:, :, -HEADS:]

    def logits(self, att, rows=None):
        """Logits of the attention's output rows (-1: a row of zeros)."""
        x = att["out"].flatten(2).view(-1, self.q)
        return dllm.fp8_matmul(*dllm.fp8_quantize(x, rows=rows), *self.head)


def decode(prompts, *, tries=3, L=8, blocks=3, V=2000, temperature=0.8, top_p=0.95, threshold=0.5, seed=0, say=print):
    """Decode ``blocks`` blocks after each prompt (lists of tokens), the best of ``tries`` each.  Returns (tokens
    [B, blocks * L], the pool's state: refs, table and held)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    model = Toy(V, dev, gen)
    B, mask = len(prompts), V
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    # rows of the batch: the requests, then their tries; pages are handed out as they are needed
    R = B + B * tries
    most = -(-(max(map(len, prompts)) + blocks * L) // PAGE)
    n_pages = 2 * R * most
    pages, weights = dllm.kv4_pages(n_pages, HEADS, PAGE, D, dev)
    pools = [pages, weights]
    refs, held, lens = i32([0] * n_pages), i32([0] * R), i32([0] * R)
    table = torch.zeros(R, most, dtype=torch.int32, device=dev)
    requests, copies = i32(range(B)), i32(range(B, R))

    # the prompts, left-padded as the batch's box is
    W = max(map(len, prompts))
    ids = i32([[0] * (W - len(p)) + list(p) for p in prompts])
    lens[:B] = i32([len(p) for p in prompts])
    dllm.page_grow(refs, table, held, lens, requests, 0, page_size=PAGE)
    _, k, v = model.project(ids)
    dllm.kv4_write(k, v, pages, table[:B], torch.zeros_like(lens[:B]), first=W - lens[:B], count=lens[:B])

    n = B * tries
    thr = torch.full((n,), threshold, device=dev)
    full = lambda x: torch.full((n * L,), x, device=dev)  # noqa: E731
    tokens = []
    for block in range(blocks):
        dllm.page_fork(pools, refs, table, held, lens, requests.repeat_interleave(tries), copies, page_size=PAGE)
        dllm.page_grow(refs, table, held, lens, copies, L, page_size=PAGE)
        mine, start = table[B:], lens[B:]
        ids = torch.full((n, L), mask, dtype=torch.int32, device=dev)
        conf = torch.full((n, L), float("nan"), device=dev)
        for _ in range(L):                                               # a step unmasks at least one position
            q, k, v = model.project(ids)
            dllm.kv4_write(k, v, pages, mine, start)                     # over the block's own slots
            att = dllm.kv4_attend(q, pages, mine, start + L)
            row = torch.arange(n * L, dtype=torch.int32, device=dev)
            row = torch.where(ids.view(-1) == mask, row, torch.full_like(row, -1))
            logits = model.logits(att, row)
            drawn = dllm.sample(logits, torch.rand(n * L, generator=gen, device=dev), V=V, rows=row,
                                temperature=full(temperature), top_p=full(top_p), conf=True)
            out = dllm.step_sampled(drawn["tokens"], drawn["conf"], ids, thr, conf, V=V, mask_id=mask)
            if bool(out["done"].all()):
                break
        q, k, v = model.project(ids)                                     # the block as it was decided
        dllm.kv4_write(k, v, pages, mine, start)
        lens[B:] += L
        att = dllm.kv4_attend(q, pages, mine, lens[B:])
        report = dllm.token_logprobs(model.logits(att), ids.view(-1), V=V)
        score = report["logprob"].view(B, tries, L).sum(-1)
        best = torch.arange(B, device=dev) * tries + score.argmax(1)
        tokens.append(ids[best])
        say(f"block {block}: log probabilities of the tries {score.tolist()}, "
            f"{int((refs > 0).sum())} pages in use")
        # the best try's cache becomes the request's; everything else goes back
        dllm.page_free(refs, table, held, requests)
        dllm.page_fork(pools, refs, table, held, lens, copies[best], requests, page_size=PAGE)
        dllm.page_free(refs, table, held, copies)
    moved = dllm.page_compact(pools, refs, table, held)
    say(f"{int(moved['used'])} pages in use, the first {int(moved['used'])} of the pool")
    return torch.cat(tokens, 1), (refs, table, held, lens)


if __name__ == "__main__":
    done, _ = decode([range(5, 12), range(100, 140), [1]])
    print(done.tolist())
    assert dllm.get_device_error() == 0
