"""A small speculative decoding loop: how the operators are used together.

    python -m varlen_top_select_amd.decode_example [steps]

A toy model of two attention layers with random weights serves a batch from paged
KV caches.  Each step drafts a few tokens from a bigram table and runs them
through the model at once:

  layer 0  tree_attention over the whole cache, and attention_weight_add for the
           rows that are accepted;
  layer 1  topk_page_table_transform selects slots from indexer scores, and
           tree_attention reads these and the new tokens;

then verify_draft accepts a prefix of the draft and draws the next token, and
evict_cache cuts layer 0's cache back to its budget when it has grown past it.
"""
from __future__ import annotations

import sys

import torch

import varlen_top_select_amd as vts

HEADS, KV_HEADS, DIM, PAGE, VOCAB = 16, 4, 64, 16, 1000
HIDDEN = HEADS * DIM


class Cache:
    """One layer's pages, and each request's table of them."""

    def __init__(self, batch: int, capacity: int, device):
        self.width = -(-capacity // PAGE)
        pages = 2 * batch * self.width  # room to evict into
        self.k = torch.zeros(pages, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.free = list(range(pages))
        self.table = self.take(batch)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.weights = torch.zeros(batch, KV_HEADS, self.width * PAGE, device=device)

    def take(self, batch: int) -> torch.Tensor:
        n = batch * self.width
        pages, self.free = self.free[:n], self.free[n:]
        return torch.tensor(pages, dtype=torch.int32, device=self.k.device).view(batch, self.width)

    def append(self, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
        """Writes [batch, new, KV_HEADS, DIM] after each request's entries; the lengths with them."""
        pos = self.lens[:, None].long() + torch.arange(k.shape[1], device=k.device)
        page = self.table.long().gather(1, pos // PAGE)
        self.k[page, pos % PAGE] = k
        self.v[page, pos % PAGE] = v
        return self.lens + k.shape[1]

    def evict(self, keep: int, sinks: int, recent: int) -> None:
        """Moves what stays to fresh pages; the old ones are free again."""
        table = self.take(self.table.shape[0])
        kept, self.lens, w = vts.evict_cache(self.weights, self.k, self.v, self.table, self.lens,
                                             keep, self.k, self.v, table, sinks=sinks, recent=recent)
        self.free += self.table.flatten().tolist()
        self.table = table
        self.weights.zero_()
        self.weights[:, :, :keep] = w


class Decoder:
    def __init__(self, batch: int = 4, draft: int = 3, budget: int = 128, top_k: int = 48,
                 capacity: int = 1024, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(*shape, generator=gen, device=device)).bfloat16()

        self.gen, self.draft, self.budget, self.top_k = gen, draft, budget, top_k
        self.embed = normal(VOCAB, HIDDEN)
        wide = HEADS + 2 * KV_HEADS
        self.qkv = [normal(HIDDEN, wide * DIM, scale=HIDDEN ** -0.5) for _ in range(2)]
        self.proj = [normal(HIDDEN, HIDDEN, scale=HIDDEN ** -0.5) for _ in range(2)]
        self.unembed = normal(HIDDEN, VOCAB, scale=3 * HIDDEN ** -0.5)
        # the draft: what the model would say without attention
        self.bigram = torch.softmax((self.embed @ self.unembed).float(), -1)
        self.layers = [Cache(batch, budget + 8 * (draft + 1) + PAGE, device),
                       Cache(batch, capacity, device)]
        self.last = torch.randint(0, VOCAB, (batch,), generator=gen, device=device)
        self.chain = torch.tensor([(2 << t) - 1 for t in range(draft + 1)], dtype=torch.int64,
                                  device=device).expand(batch, -1).contiguous()

    def propose(self):
        """A chain of drafted tokens and the distributions they were drawn from."""
        tokens, probs, x = [], [], self.last
        for _ in range(self.draft):
            probs.append(self.bigram[x])
            x = torch.multinomial(probs[-1], 1, generator=self.gen)[:, 0]
            tokens.append(x)
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    def split(self, x, layer):
        q, k, v = (x @ self.qkv[layer]).unflatten(-1, (-1, DIM)).split((HEADS, KV_HEADS, KV_HEADS), 2)
        return q.contiguous(), k, v

    def slots(self, cache: Cache, q: torch.Tensor) -> torch.Tensor:
        """The top_k cached entries of each new row by a plain indexer score."""
        batch, new = q.shape[:2]
        keys = cache.k[cache.table.long()].flatten(1, 2)[:, :, 0]   # [batch, positions, DIM]
        scores = torch.matmul(q[:, :, 0].float(), keys.float().transpose(1, 2).contiguous())
        rows = cache.table.repeat_interleave(new, 0)
        lens = cache.lens.repeat_interleave(new)
        return vts.topk_page_table_transform(scores.flatten(0, 1), lens, rows, self.top_k,
                                             page_size=PAGE)[0]

    def step(self):
        """One step: [batch] accepted drafted tokens, and the tokens it emitted."""
        tokens, probs = self.propose()
        batch = tokens.shape[0]
        new = torch.cat([self.last[:, None], tokens], 1)   # rows whose entries are not cached yet
        x = self.embed[new]

        dense, sparse = self.layers
        q0, k, v = self.split(x, 0)
        lens0 = dense.append(k, v)
        o, lse = vts.tree_attention(q0, dense.k, dense.v, dense.table, lens0, return_lse=True)
        x = x + o.flatten(2) @ self.proj[0]

        q1, k, v = self.split(x, 1)
        slots = self.slots(sparse, q1)
        lens1 = sparse.append(k, v)
        o, _ = vts.tree_attention(q1, sparse.k, sparse.v, sparse.table, lens1, slots=slots,
                                  tree_mask=self.chain)
        x = x + o.flatten(2) @ self.proj[1]

        target = torch.softmax((x @ self.unembed).float(), -1)
        u = torch.rand(batch, self.draft + 1, generator=self.gen, device=x.device)
        _, count, following = vts.verify_draft(target, tokens.int(), u, draft_probs=probs)

        # the last token and the accepted ones stay, and their rows' weights count
        stay = torch.arange(self.draft + 1, device=x.device) <= count[:, None]
        vts.attention_weight_add(dense.weights, q0, dense.k, dense.table, lens0, lse, row_keep=stay)
        for cache in self.layers:
            cache.lens += 1 + count
        if int(dense.lens.max()) + self.draft + 1 > dense.width * PAGE:
            dense.evict(self.budget, sinks=4, recent=self.budget // 4)
        emitted = torch.where(stay[:, 1:], tokens, -1)
        self.last = following.long()
        return count, torch.cat([emitted, following[:, None].long()], 1)


def main() -> None:
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 150
    decoder = Decoder(capacity=4 * (steps + 1))
    accepted = 0
    for _ in range(steps):
        count, _ = decoder.step()
        accepted += int(count.sum())
    batch = count.shape[0]
    print(f"{steps} steps of {batch} requests: {accepted / steps / batch:.2f} of {decoder.draft} "
          f"drafted tokens accepted a step; cached entries {decoder.layers[0].lens.tolist()} "
          f"(budget {decoder.budget}) and {decoder.layers[1].lens.tolist()}")


if __name__ == "__main__":
    main()
