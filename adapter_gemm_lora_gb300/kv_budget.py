"""Decode under a KV-cache budget: multi-adapter projections, page writes, split attention, eviction.

"S-LoRA, in depth", "Unified paging": adapters and KV cache share one pool, so pages that a long
request does not need are pages for another adapter.  ``BudgetedCache`` keeps every request of a decode
batch under a token budget: each step writes the new token's K and V rows into their pages and attends
over the cache, which adds up the attention weight that every cached token receives; when a request's
cache is full, the lightest older tokens are evicted at every layer and their pages go back to the pool.

    python -m adapter_gemm_lora_gb300.kv_budget [--H 4096] [--heads 32] [--requests 64] [--steps 256]
                                                [--layers 2] [--budget 128] [--recent 32] [--slack 32]

runs such a loop over random weights and prints one JSON line: time per step, evictions, and the KV
pages held against what the same requests would hold without a budget.
"""
from __future__ import annotations

import argparse
import json

import numpy as np


class BudgetedCache:
    """The KV cache of a decode batch, one token per request and step.

    A request holds at most ``budget + slack`` tokens; ``make_room`` cuts the batch back to ``budget``
    when one of them is full.  The requests must hold no KV pages yet.  All device state is allocated
    here; ``attend`` only enqueues work.
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

    def make_room(self) -> None:
        """Evict down to the budget if a request's cache is full (reads the kept positions back)."""
        if not self.lengths or max(self.lengths) < self.cap:
            return
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

    def attend(self, layer: int, q, k, v, out) -> None:
        """Write the new tokens' K and V rows at `layer`, then attend over the cache, the new token included."""
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
        self.seq_len.zero_()
        self.weight.zero_()
        self.table.fill_(-1)


def decode_step(lib, pool, seg, cache: BudgetedCache, x, W, buffers):
    """One decode step through every layer: q, k, v with each token's own adapter, attention over the
    budgeted cache, o.  W[4 l + (0..3)]: the projections of layer l; returns the last layer's output.
    buffers: six bf16 [n][H] (q, k, v, the attention output, and two for the layers' outputs in turn)."""
    q, k, v, att, y, y_next = buffers
    cache.grow()
    for layer in range(cache.layers):
        s = 4 * layer
        lib.lora_linear_forward_group(pool, seg, [s, s + 1, s + 2], x, W[s:s + 3], [q, k, v])
        cache.attend(layer, q, k, v, att)
        lib.lora_linear_forward(pool, seg, s + 3, att, W[s + 3], y)
        x, y, y_next = y, y_next, y
    return x


def main(argv=None):
    import torch

    import adapter_gemm_lora_gb300 as L
    from adapter_gemm_lora_gb300 import build
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("H", 4096), ("heads", 32), ("requests", 64), ("steps", 256), ("layers", 2), ("budget", 128),
                          ("recent", 32), ("slack", 32), ("adapters", 8), ("rank", 16)):
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
        nbytes = L.lora_segments_size_group(pool, n, 3)
        seg_ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        seg = L.lora_segments_init_group(pool, seg_ws, nbytes, n, 3)
        L.lora_segments_build(pool, torch.from_numpy(rng.integers(-1, args.adapters, n).astype(np.int32)).cuda(), n, seg)
        cache = BudgetedCache(L, pool, range(n), layers, args.heads, args.heads, args.budget, args.recent, args.slack)
        buffers = [torch.empty((n, H), dtype=torch.bfloat16, device="cuda") for _ in range(6)]
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for step in range(args.steps):
            if step == args.steps // 4:
                start.record()
            x = torch.randn((n, H), device="cuda").bfloat16()
            decode_step(L, pool, seg, cache, x, W, buffers)
        stop.record()
        torch.cuda.synchronize()
        L.lora_status(pool)
        held = sum(L.lora_kv_length(pool, i) for i in range(n)) * 2 * layers
        out = {"tool": "kv_budget", "H": H, "requests": n, "layers": layers, "budget": args.budget, "steps": args.steps,
               "ms_per_step": round(start.elapsed_time(stop) / (args.steps - args.steps // 4), 4),
               "evicted_tokens": cache.evicted, "kv_pages_held": held,
               "kv_pages_without_budget": 2 * layers * n * args.steps, "gpu": torch.cuda.get_device_name(0)}
        cache.free()
    finally:
        L.lora_pool_destroy(pool)
    print(json.dumps(out), flush=True)
    return out


if __name__ == "__main__":
    main()
