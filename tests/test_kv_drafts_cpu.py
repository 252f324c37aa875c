"""Prompts and drafted trees in BudgetedCache without a GPU: host bookkeeping and device table stay alike."""
import numpy as np
import pytest

import oracle as O
from test_kv_budget_cpu import HostLib, L, _host_is_device, on_cpu  # noqa: F401

torch = pytest.importorskip("torch")


class AppendLib(HostLib):
    """HostLib with the slot maps of the oracle."""

    def lora_attention_prompt_size(self, *args):
        return 256

    def lora_attention_tree_size(self, *args):
        return 256

    def lora_kv_append(self, pool, n_req, count, old_len, pages, row_cap, table, max_len, layers, new_len, start, req, pos):
        want = O.kv_append(count.tolist(), old_len.tolist(), pages.numpy().reshape(row_cap, layers, 2), table.numpy(), row_cap)
        for out, w in zip((table, new_len, start, req, pos), want):
            out.copy_(torch.from_numpy(np.ascontiguousarray(w)))


def _cache(L, layers=2, budget=6, recent=2, slack=5, pages=400, ids=(7, 8, 9)):
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    pool = L.lora_pool_create(None, pages, 64, 1, 1)
    return pool, BudgetedCache(AppendLib(L), pool, list(ids), layers, 1, 1, budget, recent, slack)


def test_prompts_drafts_and_growth_keep_host_and_device_alike(L, on_cpu):  # noqa: F811
    pool, cache = _cache(L)
    rng = np.random.default_rng(0)
    try:
        cache.prefill([4, 0, 11])
        _host_is_device(L, pool, cache)
        assert cache.new_req.tolist() == [0] * 4 + [2] * 11 and cache.start.tolist() == [0, 4, 4, 15]
        for step in range(40):
            cache.weight += torch.from_numpy(rng.random(cache.weight.shape).astype(np.float32)) * \
                (torch.arange(cache.cap)[None, None, :] < cache.seq_len[None, :, None])
            if step % 3 == 2:
                cache.grow()
            else:
                counts = rng.integers(0, 6, 3)
                cache.draft(counts)
                _host_is_device(L, pool, cache)
                before = [cache.table[i, :cache.lengths[i]].clone() for i in range(3)]
                kept = [sorted(rng.choice(c, rng.integers(0, c + 1), replace=False).tolist()) for c in counts]
                cache.accept(kept)
                for i in range(3):                                # the cached tokens, then those that were kept
                    base = before[i].shape[0] - int(counts[i])
                    order = list(range(base)) + [base + j for j in kept[i]]
                    assert cache.lengths[i] == len(order)
                    assert torch.equal(cache.table[i, :len(order)], before[i][order])
                    assert (cache.table[i, len(order):before[i].shape[0]] == -1).all()
            _host_is_device(L, pool, cache)
            s = L.lora_pool_stats(pool)
            assert s["reserved"] == 2 * cache.layers * sum(cache.lengths)
        assert cache.evicted > 0
        cache.free()
        assert L.lora_pool_stats(pool)["free"] == 400
        cache.prefill([1, 2, 3])
        _host_is_device(L, pool, cache)
    finally:
        L.lora_pool_destroy(pool)


def test_refusals(L, on_cpu):  # noqa: F811
    pool, cache = _cache(L)
    try:
        for fn, arg, message in [(cache.prefill, [1, 2], "one count"), (cache.prefill, [1, -1, 2], "one count"),
                                 (cache.prefill, [1, 2, 12], "one count"), (cache.draft, [1, 2, 6], "one count"),
                                 (cache.accept, [[], [], []], "no drafts")]:
            with pytest.raises(ValueError, match=message):
                fn(arg)
        for fn in (cache.attend_prompt, lambda *a: cache.attend_drafts(*a, None)):
            with pytest.raises(ValueError, match="no "):
                fn(0, None, None, None, None)
        cache.draft([2, 0, 3])
        for fn, arg, message in [(cache.draft, [1, 1, 1], "neither kept nor dropped"), (cache.prefill, [1, 1, 1], "not empty"),
                                 (cache.accept, [[0], []], "ascending"), (cache.accept, [[2], [], []], "ascending"),
                                 (cache.accept, [[1, 0], [], []], "ascending"), (cache.accept, [[0, 0], [], []], "ascending"),
                                 (cache.accept, [[], [0], []], "ascending"), (cache.accept, [[-1], [], []], "ascending")]:
            with pytest.raises(ValueError, match=message):
                fn(arg)
        with pytest.raises(ValueError, match="neither kept nor dropped"):
            cache.grow()
        _host_is_device(L, pool, cache)
        cache.accept([[0], [], [0, 2]])
        assert cache.lengths == [1, 0, 2]
        held = L.lora_pool_reserve(pool, L.lora_pool_stats(pool)["free"] - 7)
        with pytest.raises(L.LoraError) as e:                     # 2 layers x 2 x 2 tokens, 7 pages
            cache.draft([1, 0, 1])
        assert e.value.code == L.LORA_ENOPAGES and cache.drafted is None
        _host_is_device(L, pool, cache)
        L.lora_pool_release(pool, held)
        cache.grow()
        _host_is_device(L, pool, cache)
    finally:
        L.lora_pool_destroy(pool)


class RealSizes(AppendLib):
    def lora_attention_prompt_size(self, *args):
        return self.lib.lora_attention_prompt_size(*args)


def test_more_prompt_tokens_than_a_call_takes_change_nothing(L, on_cpu):  # noqa: F811
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    pool = L.lora_pool_create(None, 300000, 64, 1, 1)
    cache = BudgetedCache(RealSizes(L), pool, [1, 2], 1, 1, 1, 40000, 2, 100)
    try:
        with pytest.raises(L.LoraError) as e:
            cache.prefill([40000, 25537])
        assert e.value.code == L.LORA_EINVAL
        assert L.lora_pool_stats(pool)["free"] == 300000 and cache.lengths == [0, 0] and cache.prompt is None
        cache.prefill([40000, 25536])
        assert cache.lengths == [40000, 25536] and L.lora_pool_stats(pool)["free"] == 300000 - 2 * 65536
    finally:
        L.lora_pool_destroy(pool)


def test_random_tree():
    from adapter_gemm_lora_gb300.kv_budget import random_tree
    mask, parent = random_tree(np.random.default_rng(3), 64)
    for i, p in enumerate(parent):
        assert -1 <= p < i or i == 0
        seen, j = 0, i
        while j >= 0:
            seen |= 1 << j
            j = parent[j]
        assert mask[i] == seen
