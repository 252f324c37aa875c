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


class WriteLib(AppendLib):
    """AppendLib that notes the cache rows a call writes, and attends to nothing."""

    def __init__(self, lib):
        super().__init__(lib)
        self.rows = None

    def lora_kv_write(self, pool, rows, req, pos, k, v, n, table, max_len, layers, layer):
        self.rows = list(zip(req.tolist(), pos.tolist()))

    def lora_attention_split(self, *args, **kw):
        pass

    lora_attention_prompt = lora_attention_tree = lora_attention_split


def test_attention_out_of_turn_is_refused(L, on_cpu):  # noqa: F811
    """A cached token's K and V rows are written with its own attention alone: whatever came between the growth, the
    prompts or the drafts and their attention would have it write over other tokens."""
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    pool = L.lora_pool_create(None, 400, 64, 1, 1)
    lib = WriteLib(L)
    cache = BudgetedCache(lib, pool, [1, 2], 2, 1, 1, 6, 2, 5)
    calls = {"attend": lambda: cache.attend(0, None, None, None, None),
             "attend_prompt": lambda: cache.attend_prompt(0, None, None, None, None),
             "attend_drafts": lambda: cache.attend_drafts(0, None, None, None, None, None)}

    def only(name, rows):
        for other, call in calls.items():
            lib.rows = None
            if other == name:
                call()
                assert lib.rows == rows
            else:
                with pytest.raises(ValueError, match=f"{other}: no "):
                    call()
                assert lib.rows is None

    try:
        only(None, None)
        cache.prefill([3, 11])
        only("attend_prompt", [(0, i) for i in range(3)] + [(1, i) for i in range(11)])
        cache.make_room()                                     # evicts: the prompts' rows lie elsewhere now
        assert cache.lengths == [3, 6]
        only(None, None)
        cache.grow()
        only("attend", [(0, 3), (1, 6)])
        cache.draft([2, 1])
        only("attend_drafts", [(0, 4), (0, 5), (1, 7)])
        with pytest.raises(ValueError, match="make_room: the last drafts"):
            cache.make_room(40)
        cache.accept([[1], []])
        only(None, None)
        cache.grow()
        only("attend", [(0, 5), (1, 7)])
        for _ in range(4):
            cache.grow()
        cache.make_room(5)
        assert cache.lengths == [6, 6]
        only(None, None)
        cache.free()
        only(None, None)
        cache.prefill([1, 0])
        cache.grow()
        only("attend", [(0, 1), (1, 0)])
    finally:
        L.lora_pool_destroy(pool)


def test_what_a_loop_of_drafts_alone_keeps(L, on_cpu):  # noqa: F811
    """No decode step, no weight: the oldest tokens and the most recent ones stay.  Decode steps' weights count, and
    accepted tokens that none of them saw leave first."""
    pool, cache = _cache(L)                                       # budget 6, recent 2, room for 11
    try:
        cache.prefill([9, 3, 0])
        pages = [cache.table[i, :n].clone() for i, n in enumerate([9, 3, 0])]
        for step in range(12):
            counts = [3, 2, 1]
            if any(n + c > cache.cap for n, c in zip(cache.lengths, [max(counts)] * 3)):
                pages = [p if len(p) <= 6 else torch.cat([p[:4], p[-2:]]) for p in pages]
            cache.draft(counts)
            new = [cache.table[i, cache.lengths[i] - c:cache.lengths[i]].clone() for i, c in enumerate(counts)]
            assert (cache.weight == 0).all()
            cache.accept([[0, 2], [1], [0]])
            pages = [torch.cat([p, x[k]]) for p, x, k in zip(pages, new, ([0, 2], [1], [0]))]
            for i, p in enumerate(pages):
                assert torch.equal(cache.table[i, :cache.lengths[i]], p)
        assert cache.evicted > 0
        _host_is_device(L, pool, cache)
        cache.free()
        cache.prefill([5, 5, 5])
        cache.weight[:, :, :5] = torch.tensor([1.0, 5, 2, 4, 3])      # what decode steps have left
        cache.draft([5, 5, 5])
        cache.accept([[0, 1, 2, 3, 4]] * 3)
        was = cache.table[0, :10].clone()
        cache.draft([2, 2, 2])
        assert torch.equal(cache.table[0, :6], was[[1, 2, 3, 4, 8, 9]])
    finally:
        L.lora_pool_destroy(pool)


class CountingLib(AppendLib):
    """AppendLib that counts the positions handed to the pool's bookkeeping."""
    handed = 0

    def lora_kv_keep(self, pool, request, keep):
        self.handed += np.asarray(keep).size
        self.lib.lora_kv_keep(pool, request, keep)

    def lora_kv_keep_last(self, pool, request, n_last, keep):
        self.handed += n_last
        self.lib.lora_kv_keep_last(pool, request, n_last, keep)


def test_accepting_drafts_takes_time_by_the_drafts(L, on_cpu):  # noqa: F811
    """However long the cache, accept hands on no more than the drafted tokens."""
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    pool = L.lora_pool_create(None, 40000, 64, 1, 1)
    lib = CountingLib(L)
    cache = BudgetedCache(lib, pool, [1, 2, 3], 5, 1, 1, 1200, 2, 20)
    try:
        cache.prefill([1000, 1, 700])
        cache.draft([7, 20, 0])
        cache.accept([[0, 3], [19], []])
        assert lib.handed <= 27 and cache.lengths == [1002, 2, 700]
        _host_is_device(L, pool, cache)
        cache.draft([1, 2, 3])
        cache.accept([[0], [0, 1], [0, 1, 2]])                    # nothing is dropped
        assert lib.handed <= 27
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
