"""Serving under a KV-cache budget: multi-adapter projections, page writes, attention of prompts, of new tokens and of
drafted trees, eviction.

"S-LoRA, in depth", "Unified paging": adapters and KV cache share one pool, so pages that a long
request does not need are pages for another adapter.  ``BudgetedCache`` keeps every request of a decode
batch under a token budget: each step writes the new token's K and V rows into their pages and attends
over the cache, which adds up the attention weight that every cached token receives; when a request's
cache is full, the lightest older tokens are evicted at every layer and their pages go back to the pool.
Prompts enter an empty cache whole (``prefill``), and drafted tokens are attended as a tree and then kept or
dropped (``draft``, ``accept``): their table entries and slot maps are made on the GPU.  Only decode steps (``grow``,
``attend``) add weight.  Prompts and drafts look at tokens without a trace, so in a loop of drafts alone all weights are
equal, and an eviction keeps the oldest ``budget - recent`` tokens and the newest ``recent``, whatever was looked at; among
decode steps, tokens that none of them saw (those of accepted drafts) are the first to leave.

    python -m adapter_gemm_lora_gb300.kv_budget [--H 4096] [--heads 32] [--requests 64] [--steps 256]
                                                [--layers 2] [--budget 128] [--recent 32] [--slack 32]
                                                [--prompt 0] [--draft 0]

runs such a loop over random weights and prints one JSON line: time per step, evictions, and the KV
pages held against what the same requests would hold without a budget.  With --prompt P every request
starts with a prompt of P/2 to P tokens; with --draft M a step checks a tree of M drafted tokens per
request and keeps one path of it (no step adds weight then).
"""
from __future__ import annotations

import argparse
import json

import numpy as np


class BudgetedCache:
    """The KV cache of a decode batch, one token per request and step.

    A request holds at most ``budget + slack`` tokens; ``make_room`` cuts the batch back to ``budget``
    when one of them is full.  The requests must hold no KV pages yet.  All device state is allocated
    here; ``attend`` only enqueues work.  Each kind of attention belongs to the growth, prompts or drafts that came last
    (``grow`` / ``attend``, ``prefill`` / ``attend_prompt``, ``draft`` / ``attend_drafts``) and is refused after anything else.
    """

    def __init__(self, lib, pool, request_ids, layers: int, n_heads: int, n_kv_heads: int, budget: int, recent: int,
                 slack: int):
        import torch
        if slack < 1:
            raise ValueError("slack must be at least 1")
        self.lib, self.pool, self.ids = lib, pool, list(request_ids)
        if len(set(self.ids)) < len(self.ids):
            raise ValueError("a request is named twice")
        for r in self.ids:                                     # the tables start empty
            if lib.lora_kv_length(pool, r) >= 0:
                raise ValueError(f"request {r} holds KV pages already: free it first")
        self.layers, self.n_heads, self.n_kv_heads = layers, n_heads, n_kv_heads
        self.budget, self.recent, self.cap = budget, recent, budget + slack
        n = len(self.ids)
        dev = "cuda"
        self.table = torch.full((n, self.cap, layers, 2), -1, dtype=torch.int32, device=dev)
        self.weight = torch.zeros((layers, n, self.cap), dtype=torch.float32, device=dev)
        self.seq_len = torch.zeros(n, dtype=torch.int32, device=dev)
        self._next = [torch.empty_like(self.table), torch.empty_like(self.weight), torch.empty_like(self.seq_len)]
        self.keep = torch.empty((layers, n, budget), dtype=torch.int32, device=dev)
        self.row_req = torch.arange(n, dtype=torch.int32, device=dev)
        self.row_pos = torch.zeros(n, dtype=torch.int32, device=dev)
        self.ws_bytes = lib.lora_attention_split_size(pool, n, self.cap, n_heads, n_kv_heads, True)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.lengths = [0] * n
        self.evicted = 0
        self.prompt = self.drafted = None                      # tokens of the last prefill / draft, per request
        self.grown = False                                     # row_pos names the last growth's tokens

    def make_room(self, tokens: int = 1) -> None:
        """Evict down to the budget if a request has no room for `tokens` more (reads the kept positions back)."""
        if self.drafted is not None:
            raise ValueError("make_room: the last drafts are neither kept nor dropped (accept)")
        if not self.lengths or max(self.lengths) + tokens <= self.cap:
            return
        self.prompt, self.grown = None, False                  # tokens move: their rows are no longer where they were
        n = len(self.ids)
        table, weight, seq_len = self._next
        self.lib.lora_kv_evict(self.pool, n, self.table, self.seq_len, self.cap, self.layers, self.weight, self.budget,
                               self.recent, self.keep, seq_len, table, weight, self.cap)
        keep, lengths = self.keep.cpu().numpy(), seq_len.tolist()      # the stream has passed every reader of the pages
        for i, request in enumerate(self.ids):
            self.lib.lora_kv_keep(self.pool, request, np.ascontiguousarray(keep[:, i, :lengths[i]]))
        self.evicted += sum(self.lengths) - sum(lengths)
        self._next = [self.table, self.weight, self.seq_len]
        self.table, self.weight, self.seq_len = table, weight, seq_len
        self.lengths = lengths

    def grow(self) -> None:
        """Pages for one new token per request; LORA_ENOPAGES, and none taken, if the pool has too few for all of them."""
        import torch
        if self.drafted is not None:
            raise ValueError("grow: the last drafts are neither kept nor dropped (accept)")
        self.make_room()
        need, free = 2 * self.layers * len(self.ids), self.lib.lora_pool_stats(self.pool)["free"]
        if need > free:                                        # before any request holds a token the table does not name
            raise self.lib.LoraError(self.lib.LORA_ENOPAGES, f"BudgetedCache.grow: {need} pages asked, {free} free")
        rows = np.array([self.lib.lora_kv_grow(self.pool, r, 1, self.layers) for r in self.ids], dtype=np.int32)
        n = len(self.ids)
        pos = torch.tensor(self.lengths, dtype=torch.int64)
        self.table[torch.arange(n), pos] = torch.from_numpy(rows.reshape(n, self.layers, 2)).cuda()
        self.row_pos.copy_(pos)
        self.seq_len += 1
        self.lengths = [x + 1 for x in self.lengths]
        self.prompt, self.grown = None, True

    def _append(self, counts) -> None:
        """Pages, table entries, lengths and slot maps of counts[i] new tokens per request."""
        import torch
        need, free = 2 * self.layers * sum(counts), self.lib.lora_pool_stats(self.pool)["free"]
        if need > free:                                        # before any request holds a token the table does not name
            raise self.lib.LoraError(self.lib.LORA_ENOPAGES, f"BudgetedCache: {need} pages asked, {free} free")
        n, rows, dev = len(self.ids), sum(counts), self.table.device
        pages = [p for r, c in zip(self.ids, counts) for p in self.lib.lora_kv_grow(self.pool, r, c, self.layers)]
        pages = torch.tensor(pages, dtype=torch.int32, device=dev)
        self.rows, self.start = rows, torch.empty(n + 1, dtype=torch.int32, device=dev)
        self.new_req, self.new_pos = (torch.empty(rows, dtype=torch.int32, device=dev) for _ in range(2))
        self.lib.lora_kv_append(self.pool, n, torch.tensor(counts, dtype=torch.int32, device=dev), self.seq_len, pages, rows,
                                self.table, self.cap, self.layers, self._next[2], self.start, self.new_req, self.new_pos)
        self.seq_len, self._next[2] = self._next[2], self.seq_len
        self.lengths = [x + c for x, c in zip(self.lengths, counts)]

    def _checked(self, counts, most: int, what: str) -> list:
        counts = [int(c) for c in counts]
        if len(counts) != len(self.ids) or any(c < 0 or c > most for c in counts):
            raise ValueError(f"{what}: one count per request, 0 to {most}")
        return counts

    def prefill(self, lengths) -> None:
        """Room for a prompt of lengths[i] tokens per request in an empty cache.  Their rows are packed request by
        request: ``attend_prompt`` then takes every layer's q, k and v of them."""
        import torch
        if any(self.lengths):
            raise ValueError("prefill: the cache is not empty")
        counts = self._checked(lengths, self.cap, "prefill")
        ws_bytes = self.lib.lora_attention_prompt_size(self.pool, len(self.ids), sum(counts), self.n_heads, self.n_kv_heads)
        self._append(counts)                                   # not before the call is known to be small enough
        self.prompt, self.drafted, self.grown, self._rows_ws_bytes = counts, None, False, ws_bytes
        self._rows_ws = torch.empty(max(self._rows_ws_bytes, 256), dtype=torch.uint8, device=self.table.device)

    def attend_prompt(self, layer: int, q, k, v, out) -> None:
        """Write the prompts' K and V rows at `layer`; causal attention of every prompt over itself.  (Prompt tokens
        receive no weight from it: eviction goes by what decode steps look at.)"""
        if self.prompt is None:
            raise ValueError("attend_prompt: no prefill")
        n = len(self.ids)
        self.lib.lora_kv_write(self.pool, self.rows, self.new_req, self.new_pos, k, v, n, self.table, self.cap, self.layers,
                               layer)
        self.lib.lora_attention_prompt(self.pool, n, self.start, self.rows, q, k, v, out, self.n_heads, self.n_kv_heads,
                                       self._rows_ws, self._rows_ws_bytes)

    def draft(self, counts) -> None:
        """Room for a tree of counts[i] drafted tokens per request behind what is cached; evicts first if they do not
        fit (so at most `slack` of them), by the weights that decode steps have left: without any, the tokens between
        the oldest ``budget - recent`` and the newest ``recent``.  ``attend_drafts`` takes their rows, ``accept`` says which stay."""
        import torch
        if self.drafted is not None:
            raise ValueError("draft: the last drafts are neither kept nor dropped (accept)")
        counts = self._checked(counts, min(self.cap - self.budget, self.lib.LORA_MAX_TREE), "draft")
        self.make_room(max(counts, default=0))
        self._append(counts)
        self.prompt, self.drafted, self.grown = None, counts, False
        self._rows_ws_bytes = self.lib.lora_attention_tree_size(self.pool, len(self.ids), self.cap, self.n_heads,
                                                                self.n_kv_heads)
        self._rows_ws = torch.empty(max(self._rows_ws_bytes, 256), dtype=torch.uint8, device=self.table.device)

    def attend_drafts(self, layer: int, q, k, v, mask, out) -> None:
        """Write the drafted tokens' K and V rows at `layer`, then attend: each sees the cache and the drafted tokens
        of its request that its mask (int64 per row, bit j: node j) names.  Cached tokens receive no weight from it."""
        if self.drafted is None:
            raise ValueError("attend_drafts: no drafts")
        n = len(self.ids)
        self.lib.lora_kv_write(self.pool, self.rows, self.new_req, self.new_pos, k, v, n, self.table, self.cap, self.layers,
                               layer)
        self.lib.lora_attention_tree(self.pool, n, self.table, self.seq_len, self.cap, self.layers, layer, self.start, self.rows,
                                     mask, q, out, self.n_heads, self.n_kv_heads, self._rows_ws, self._rows_ws_bytes)

    def accept(self, kept) -> None:
        """Of request i's drafted tokens those in kept[i] (ascending) stay, in that order; the others' pages go back to
        the pool.  No K or V moves: a token is its pages."""
        import torch
        if self.drafted is None:
            raise ValueError("accept: no drafts")
        kept = [[int(j) for j in k] for k in kept]
        if len(kept) != len(self.ids) or any(list(sorted(set(k))) != k or (k and not 0 <= k[0] <= k[-1] < m)
                                             for k, m in zip(kept, self.drafted)):
            raise ValueError("accept: ascending nodes of every request's draft")
        place = []                                             # request, position, its new token's old position or -1
        for i, (k, m) in enumerate(zip(kept, self.drafted)):
            base = self.lengths[i] - m
            place += [(i, base + j, base + k[j] if j < len(k) else -1) for j in range(m)]
            if m > len(k):
                self.lib.lora_kv_keep_last(self.pool, self.ids[i], m, k)
            self.lengths[i] = base + len(k)
        if place:
            r, to, frm = torch.tensor(place, dtype=torch.int64).t().to(self.table.device)
            self.table[r, to] = torch.where(frm[:, None, None] >= 0, self.table[r, frm.clamp(min=0)], -1)
        self.seq_len.copy_(torch.tensor(self.lengths, dtype=torch.int32))
        self.drafted = None

    def attend(self, layer: int, q, k, v, out) -> None:
        """Write the new tokens' K and V rows at `layer`, then attend over the cache, the new token included."""
        if not self.grown:
            raise ValueError("attend: no new tokens (grow)")
        n = len(self.ids)
        self.lib.lora_kv_write(self.pool, n, self.row_req, self.row_pos, k, v, n, self.table, self.cap, self.layers, layer)
        self.lib.lora_attention_split(self.pool, n, self.table, self.seq_len, self.cap, self.layers, layer, q, out,
                                      self.n_heads, self.n_kv_heads, self.ws, self.ws_bytes,
                                      weight_in_dev=self.weight[layer], weight_out_dev=self.weight[layer])

    def free(self) -> None:
        for i, request in enumerate(self.ids):
            if self.lib.lora_kv_length(self.pool, request) >= 0:
                self.lib.lora_kv_free(self.pool, request)
        self.lengths = [0] * len(self.ids)
        self.prompt, self.drafted, self.grown = None, None, False
        self.seq_len.zero_()
        self.weight.zero_()
        self.table.fill_(-1)


def _through_layers(lib, pool, seg, cache: BudgetedCache, x, W, buffers, attend):
    q, k, v, att, y, y_next = buffers
    for layer in range(cache.layers):
        s = 4 * layer
        lib.lora_linear_forward_group(pool, seg, [s, s + 1, s + 2], x, W[s:s + 3], [q, k, v])
        attend(layer, q, k, v, att)
        lib.lora_linear_forward(pool, seg, s + 3, att, W[s + 3], y)
        x, y, y_next = y, y_next, y
    return x


def prompt_step(lib, pool, seg, cache: BudgetedCache, x, W, buffers, lengths):
    """The prompts' rows x (packed, request by request) through every layer, into the empty cache; seg: their
    segments; W and buffers as for decode_step, with a row per prompt token."""
    cache.prefill(lengths)
    return _through_layers(lib, pool, seg, cache, x, W, buffers, cache.attend_prompt)


def draft_step(lib, pool, seg, cache: BudgetedCache, x, W, buffers, counts, mask):
    """The rows x of counts[i] drafted tokens per request through every layer, each seeing the cache and what its mask
    names; ``cache.accept`` has to follow."""
    cache.draft(counts)
    return _through_layers(lib, pool, seg, cache, x, W, buffers,
                           lambda layer, q, k, v, out: cache.attend_drafts(layer, q, k, v, mask, out))


def random_tree(rng, nodes: int):
    """Masks (bit j: node j is the node itself or an ancestor) and parents of a random tree, parents before children."""
    parent = [int(rng.integers(-1, i)) if i else -1 for i in range(nodes)]
    mask = []
    for i, p in enumerate(parent):
        mask.append(1 << i | (mask[p] if p >= 0 else 0))
    return mask, parent


def decode_step(lib, pool, seg, cache: BudgetedCache, x, W, buffers):
    """One decode step through every layer: q, k, v with each token's own adapter, attention over the
    budgeted cache, o.  W[4 l + (0..3)]: the projections of layer l; returns the last layer's output.
    buffers: six bf16 [n][H] (q, k, v, the attention output, and two for the layers' outputs in turn)."""
    cache.grow()
    return _through_layers(lib, pool, seg, cache, x, W, buffers, cache.attend)


def main(argv=None):
    import torch

    import adapter_gemm_lora_gb300 as L
    from adapter_gemm_lora_gb300 import build
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("H", 4096), ("heads", 32), ("requests", 64), ("steps", 256), ("layers", 2), ("budget", 128),
                          ("recent", 32), ("slack", 32), ("adapters", 8), ("rank", 16), ("prompt", 0), ("draft", 0)):
        ap.add_argument(f"--{name}", type=int, default=default)
    args = ap.parse_args(argv)
    build.build()
    H, n, layers, r, slots = args.H, args.requests, args.layers, args.rank, 4 * args.layers
    rng = np.random.default_rng(0)
    num_pages = 2 * r * slots * args.adapters + 2 * layers * n * (args.budget + args.slack) + 16
    pool_t = torch.zeros((num_pages, H), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, num_pages, H, slots, args.adapters)
    try:
        bits = lambda *shape: (torch.randn(shape) / shape[0] ** 0.5).bfloat16().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
        for a in range(args.adapters):
            L.lora_adapter_load(pool, a, r, [bits(H, r) for _ in range(slots)], [bits(r, H) for _ in range(slots)], slots)
        W = [(torch.randn((H, H), device="cuda") / H ** 0.5).bfloat16() for _ in range(slots)]
        adapter = rng.integers(-1, args.adapters, n).astype(np.int32)                      # of each request
        per = max(args.draft, 1)                               # rows of a request in a step
        room = max(n * per, n * args.prompt, 1)
        nbytes = L.lora_segments_size_group(pool, room, 3)
        seg_ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        seg = L.lora_segments_init_group(pool, seg_ws, nbytes, room, 3)
        cache = BudgetedCache(L, pool, range(n), layers, args.heads, args.heads, args.budget, args.recent, args.slack)
        rows = lambda m: [torch.empty((m, H), dtype=torch.bfloat16, device="cuda") for _ in range(6)]  # noqa: E731
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        prompt_tokens, ms_prompt = 0, 0.0
        if args.prompt:
            lengths = rng.integers((args.prompt + 1) // 2, args.prompt + 1, n)
            prompt_tokens = int(lengths.sum())
            token_adapter = torch.from_numpy(np.repeat(adapter, lengths)).cuda()
            x, prompt_rows = torch.randn((prompt_tokens, H), device="cuda").bfloat16(), rows(prompt_tokens)
            start.record()
            L.lora_segments_build(pool, token_adapter, prompt_tokens, seg)
            prompt_step(L, pool, seg, cache, x, W, prompt_rows, lengths)
            stop.record()
            torch.cuda.synchronize()
            ms_prompt = start.elapsed_time(stop)
            del prompt_rows
        L.lora_segments_build(pool, torch.from_numpy(np.repeat(adapter, per)).cuda(), n * per, seg)
        buffers, tokens = rows(n * per), 0
        for step in range(args.steps):
            if step == args.steps // 4:
                start.record()
            x = torch.randn((n * per, H), device="cuda").bfloat16()
            if not args.draft:
                decode_step(L, pool, seg, cache, x, W, buffers)
                tokens += n
                continue
            trees = [random_tree(rng, per) for _ in range(n)]
            mask = torch.from_numpy(np.array([m for tree, _ in trees for m in tree], np.uint64).view(np.int64)).cuda()
            draft_step(L, pool, seg, cache, x, W, buffers, [per] * n, mask)
            kept = []                                          # the path to a node drawn by lot, as a check would find one
            for _, parent in trees:
                path, j = [], int(rng.integers(0, per))
                while j >= 0:
                    path.append(j)
                    j = parent[j]
                kept.append(path[::-1])
            cache.accept(kept)
            tokens += sum(map(len, kept))
        stop.record()
        torch.cuda.synchronize()
        L.lora_status(pool)
        held = sum(L.lora_kv_length(pool, i) for i in range(n)) * 2 * layers
        out = {"tool": "kv_budget", "H": H, "requests": n, "layers": layers, "budget": args.budget, "steps": args.steps,
               "ms_per_step": round(start.elapsed_time(stop) / (args.steps - args.steps // 4), 4),
               "evicted_tokens": cache.evicted, "kv_pages_held": held,
               "kv_pages_without_budget": 2 * layers * (prompt_tokens + tokens),
               "prompt_tokens": prompt_tokens, "ms_prompt": round(ms_prompt, 4), "tokens": tokens, "gpu": torch.cuda.get_device_name(0)}
        cache.free()
    finally:
        L.lora_pool_destroy(pool)
    print(json.dumps(out), flush=True)
    return out


if __name__ == "__main__":
    main()
