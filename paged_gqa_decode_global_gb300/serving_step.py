"""A serving loop over one global layer, as its pieces are used together.

A system prompt is written into the cache once; requests that share it get
their own tokens' pages, slots and cache rows step by step, and every decode
step attends [prompt | own tokens] with the prompt read once for all of them:

    append_slots  lengths -> pages, block tables, positions, slots
    write_slots   the new tokens' K / V rows into their slots
    SharedPrefixStep  the attention of the batch

The lengths, tables and free list live on the GPU and are updated in place, so
a step makes no round trip to the host. Random rows stand for a model's, rotated
already: PageTables.positions count a request's own tokens, so a model rotates
its rows by the prompt's length plus those.

    python -m paged_gqa_decode_global_gb300.serving_step [steps]
"""
from __future__ import annotations

import math
import sys
from typing import List, Optional, Sequence

import torch

from . import binding as b


class PageTables:
    """Block tables, lengths and free pages of a batch, on the GPU."""

    def __init__(self, batch: int, page_size: int, num_pages: int, max_pages: int, max_tokens: int, free_pages, free_range,
                 device="cuda"):
        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        self.page_size, self.num_pages = page_size, num_pages
        self.block_tables = torch.full((batch, max_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens, self.token_starts = i32(batch), i32(batch + 1)
        self.slot_map, self.positions = i32(max_tokens), i32(max_tokens)
        self.free_pages, self.free_range = free_pages, free_range
        self.flags = i32(1)
        self.workspace = torch.zeros(b.paged_decode_append_slots_workspace(batch), dtype=torch.uint8, device=device)

    def append(self, new_tokens: torch.Tensor, stream=None) -> None:
        """Pages and slots for new_tokens[r] more tokens of each request."""
        b.paged_decode_append_slots(self.page_size, self.num_pages, self.seq_lens, new_tokens, self.free_pages,
                                    self.free_range, self.block_tables, self.seq_lens, self.token_starts,
                                    self.slot_map, self.positions, self.free_range, self.flags, self.workspace, stream)


class SharedPrefixServer:
    """One global layer's cache and its decode for `batch` requests under one prompt of prompt_tokens (whole pages)."""

    def __init__(self, batch: int, prompt_tokens: int, max_own_tokens: int, *, num_q_heads=16, num_kv_heads=4,
                 head_dim=512, page_size=16, device="cuda", seed=0):
        if prompt_tokens % page_size:
            raise ValueError("the shared prompt is whole pages; its ragged end belongs to the requests")
        own_pages = (max_own_tokens + page_size - 1) // page_size
        pages = prompt_tokens // page_size + batch * own_pages
        gen = torch.Generator().manual_seed(seed)
        free = torch.randperm(pages, generator=gen).to(torch.int32).to(device)
        free_range = torch.tensor([0, pages], dtype=torch.int32, device=device)
        self.desc = b.layer_desc(num_q_heads, num_kv_heads, head_dim, page_size, pages, own_pages)
        pool = (pages, num_kv_heads, page_size, head_dim)
        self.k_pool = torch.zeros(pool, dtype=torch.bfloat16, device=device)
        self.v_pool = torch.zeros_like(self.k_pool)
        self.prompt = PageTables(1, page_size, pages, max(1, prompt_tokens // page_size), prompt_tokens, free, free_range,
                                 device)
        self.requests = PageTables(batch, page_size, pages, own_pages, batch * max_own_tokens, free, free_range, device)
        self.group_starts = torch.tensor([0, batch], dtype=torch.int32, device=device)
        self.scale = 1.0 / math.sqrt(head_dim)
        self.step = b.SharedPrefixStep(num_q_heads, num_kv_heads, head_dim, page_size, pages, own_pages,
                                       [max_own_tokens] * batch, group_starts=[0, batch], prefix_lens=[prompt_tokens],
                                       max_prefix_pages=self.prompt.block_tables.shape[1], device=device)

    def _write(self, tables: PageTables, k: torch.Tensor, v: torch.Tensor) -> None:
        b.paged_decode_write_slots(self.desc, k, v, tables.slot_map[:k.shape[0]], self.k_pool, self.v_pool,
                                   tables.flags)

    def write_prompt(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """The shared prompt's K / V rows [tokens, Hkv, d]."""
        self.prompt.append(torch.tensor([k.shape[0]], dtype=torch.int32, device=k.device))
        self._write(self.prompt, k, v)

    def add(self, new_tokens: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> None:
        """new_tokens[r] more tokens of each request, their rows one request after another."""
        self.requests.append(new_tokens)
        self._write(self.requests, k, v)

    def decode(self, q: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of each request's newest token (its rows added already): q, out bf16 [batch, Hq, d]."""
        out = torch.empty_like(q) if out is None else out
        return self.step(q, self.k_pool, self.v_pool, self.prompt.block_tables, self.prompt.seq_lens,
                         self.group_starts, self.requests.block_tables, self.requests.seq_lens, self.scale, out)

    def check(self) -> None:
        """Raise what the device found wrong (pages, lengths, waits)."""
        self.step.check()
        for t in (self.prompt, self.requests):
            if int(t.flags):
                raise RuntimeError(f"device flags 0x{int(t.flags):x}")


def rows(n: int, heads: int, dim: int, gen, device="cuda") -> torch.Tensor:
    return torch.randn((n, heads, dim), generator=gen, device=device).to(torch.bfloat16)


def run(steps: int = 4, batch: int = 6, prompt_tokens: int = 2048, tails: Optional[Sequence[int]] = None,
        seed: int = 0) -> List[dict]:
    """The loop; returns each decode step's q and out with the rows they attend
    (K and V per request, prompt included), for a comparison."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tails = list(tails) if tails is not None else [1 + 7 * r for r in range(batch)]
    server = SharedPrefixServer(batch, prompt_tokens, max(tails) + steps, seed=seed)
    heads, dim = server.desc.num_kv_heads, server.desc.head_dim
    kp, vp = rows(prompt_tokens, heads, dim, gen), rows(prompt_tokens, heads, dim, gen)
    server.write_prompt(kp, vp)
    # the requests' own prompts, ragged
    k, v = rows(sum(tails), heads, dim, gen), rows(sum(tails), heads, dim, gen)
    server.add(torch.tensor(tails, dtype=torch.int32, device="cuda"), k, v)
    hold = [([kp, a], [vp, c]) for a, c in zip(k.split(tails), v.split(tails))]
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    seen = []
    for _ in range(steps):
        k, v = rows(batch, heads, dim, gen), rows(batch, heads, dim, gen)
        q = rows(batch, server.desc.num_q_heads, dim, gen)
        server.add(one, k, v)
        out = server.decode(q)
        for r in range(batch):
            hold[r][0].append(k[r:r + 1])
            hold[r][1].append(v[r:r + 1])
        seen.append({"q": q, "out": out, "k": [torch.cat(h[0]) for h in hold], "v": [torch.cat(h[1]) for h in hold]})
    server.check()
    return seen


if __name__ == "__main__":
    done = run(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
    for i, s in enumerate(done):
        print(f"step {i}: {len(s['k'])} requests, {len(s['k'][0])}..{max(map(len, s['k']))} tokens, "
              f"|out| {float(s['out'].float().abs().mean()):.4f}")
