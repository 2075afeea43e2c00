"""Block-wise decoding over the paged 4-bit cache, with reports: every operator
around the step, as a server's loop would call them.

A one-layer toy model (random weights) stands in for the forward.  Prompts are
written into the cache once.  Each block is then denoised: every step writes the
block's keys and values over its own cache slots, attends to prompt, earlier
blocks and itself, and steps on the logits.  A finished block is written for
good, attended once more for the weights that its queries give every cached
token, and reported: log probability, entropy and alternatives of its tokens.
A cache that has outgrown its budget is thinned to its most attended tokens.

    python examples/block_cache.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import denoise_step_token_gb300 as dllm

HEADS, GROUP, D = 2, 4, 64
PAGE = 16


class Toy:
    """Embeddings, one attention layer's projections and an LM head."""

    def __init__(self, V, dev, gen):
        q = HEADS * GROUP * D
        rand = lambda *shape: torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
        self.embed = rand(V + 1, 256)                                    # the last row: the mask
        self.qkv = rand(256, q + 2 * HEADS * D) / 16
        self.head = rand(q, V) / 2
        self.q = q

    def project(self, ids):
        """Queries [B, L, q_heads, D], keys and values [B, L, HEADS, D]: slices of one projection."""
        x = (self.embed[ids.long()] @ self.qkv).unflatten(-1, (-1, D))
        return x[:, :, :HEADS * GROUP], x[:, :, HEADS * GROUP:-HEADS], x[:, :, -HEADS:]


def decode(prompts, *, L=8, blocks=4, V=2000, budget=48, recent=16, threshold=0.6, seed=0, say=print):
    """Decode ``blocks`` blocks after each prompt (lists of tokens).  Returns
    (tokens [B, blocks * L], cached tokens of each request, one dict per block:
    the report's tensors and ``conf``, what the block's last step was sure of)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    model = Toy(V, dev, gen)
    B, mask = len(prompts), V
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    # each request owns two runs of pages: the one in use, and one to be thinned into
    most = -(-(max(map(len, prompts)) + blocks * L) // PAGE)
    pages, weights = dllm.kv4_pages(2 * B * most, HEADS, PAGE, D, dev)
    table, other = torch.randperm(2 * B * most, generator=gen, device=dev).to(torch.int32).view(2, B, most)
    table, other = table.contiguous(), other.contiguous()

    # the prompts, left-padded as the batch's box is
    W = max(map(len, prompts))
    ids = i32([[0] * (W - len(p)) + list(p) for p in prompts])
    lens = i32([len(p) for p in prompts])
    _, k, v = model.project(ids)
    dllm.kv4_write(k, v, pages, table, torch.zeros_like(lens), first=W - lens, count=lens)

    thr = torch.full((B,), threshold, device=dev)
    tokens, reports = [], []
    for block in range(blocks):
        ids = torch.full((B, L), mask, dtype=torch.int32, device=dev)
        conf = torch.full((B, L), float("nan"), device=dev)
        for _ in range(L):                                               # a step unmasks at least one position
            q, k, v = model.project(ids)
            dllm.kv4_write(k, v, pages, table, lens)                     # over the block's own slots
            att = dllm.kv4_attend(q, pages, table, lens + L)
            logits = att["out"].flatten(2).view(B * L, model.q) @ model.head
            out = dllm.step(logits, ids, thr, conf, V=V, mask_id=mask, debug=True)
            if bool(out["done"].all()):
                break
        q, k, v = model.project(ids)                                     # the block as it was decided
        dllm.kv4_write(k, v, pages, table, lens)
        lens = lens + L
        att = dllm.kv4_attend(q, pages, table, lens, prior=weights, weights=weights)
        logits = att["out"].flatten(2).view(B * L, model.q) @ model.head
        report = dllm.token_logprobs(logits, ids.view(-1), V=V, top=3)
        reports.append({**report, "logits": logits, "lse": att["lse"]})
        tokens.append(ids)
        say(f"block {block}: mean log probability {report['logprob'].mean().item():.2f}, "
            f"entropy {report['entropy'].mean().item():.2f}, cached {lens.tolist()}")
        if int(lens.max()) > budget:
            thin = dllm.kv4_evict(pages, weights, table, lens, torch.clamp(lens, max=budget), other, recent=recent)
            weights[table.long()] = 0                                    # the pages go back empty
            lens, table, other = thin["lens"], other, table
            say(f"  thinned to {lens.tolist()}")
    return torch.cat(tokens, 1), lens, reports


if __name__ == "__main__":
    done, cached, _ = decode([range(5, 12), range(100, 140), [1]])
    print(done.tolist())
    assert dllm.get_device_error() == 0
