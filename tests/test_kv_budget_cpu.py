"""BudgetedCache's host side without a GPU: device buffers on the CPU, planning pools, the device's operators left out."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from adapter_gemm_lora_gb300 import build
    build.build()
    import adapter_gemm_lora_gb300 as lib
    lib.library()
    return lib


class HostLib:
    """The library on a planning pool: bookkeeping is the library's, an eviction the oracle's, nothing runs on a GPU."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def lora_attention_split_size(self, *args):
        return 256

    def lora_kv_evict(self, pool, n_req, table, seq_len, max_len, layers, weight, budget, recent, keep, new_len, table_out,
                      weight_out, max_len_out):
        keep.fill_(-1), table_out.fill_(-1), weight_out.zero_()
        for r, n in enumerate(seq_len.tolist()):
            new_len[r] = min(n, budget)
            for l in range(layers):
                k = O.evict_keep(weight[l, r].numpy(), n, budget, recent)
                keep[l, r, :len(k)] = torch.tensor(k, dtype=torch.int32)
                table_out[r, :len(k), l] = table[r, k, l]
                weight_out[l, r, :len(k)] = weight[l, r, k]


@pytest.fixture()
def on_cpu(monkeypatch):
    for name in ("full", "zeros", "arange", "empty"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, **k: _real(*a, **{**k, "device": "cpu"}))
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **k: self)


def _host_is_device(lib, pool, cache):
    """Every request's pages on the host are those of the device table."""
    for i, r in enumerate(cache.ids):
        n = cache.lengths[i]
        assert max(lib.lora_kv_length(pool, r), 0) == n == int(cache.seq_len[i])
        for l in range(cache.layers if n else 0):
            assert lib.lora_kv_table(pool, r, l).tolist() == cache.table[i, :n, l].tolist()


@pytest.mark.parametrize("spare", [0, 1, 5, 11])
def test_a_refused_growth_leaves_host_and_device_alike(L, on_cpu, spare):
    """The pool runs out in the middle of a batch; pages come free, the growth is tried again, and evictions follow."""
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    n, layers, budget, recent, slack = 3, 2, 6, 2, 3
    need = 2 * layers * n * (budget + slack)
    pool = L.lora_pool_create(None, need, 64, 1, 1)
    try:
        cache = BudgetedCache(HostLib(L), pool, [7, 8, 9], layers, 1, 1, budget, recent, slack)
        rng = np.random.default_rng(spare)
        for step in range(30):
            cache.weight += torch.from_numpy(rng.random(cache.weight.shape).astype(np.float32)) * \
                (torch.arange(cache.cap)[None, None, :] < cache.seq_len[None, :, None])
            if step % 4 == 2:                                     # another user of the pool holds all but `spare` pages
                cache.make_room()
                held = L.lora_pool_reserve(pool, L.lora_pool_stats(pool)["free"] - spare)
                before, free = list(cache.lengths), L.lora_pool_stats(pool)["free"]
                with pytest.raises(L.LoraError) as e:
                    cache.grow()
                assert e.value.code == L.LORA_ENOPAGES
                assert cache.lengths == before and L.lora_pool_stats(pool)["free"] == free
                _host_is_device(L, pool, cache)
                L.lora_pool_release(pool, held)
            cache.grow()
            _host_is_device(L, pool, cache)
        assert cache.evicted > 0
        cache.free()
        assert L.lora_pool_stats(pool)["free"] == need
        cache.grow()
        _host_is_device(L, pool, cache)
    finally:
        L.lora_pool_destroy(pool)


def test_requests_that_hold_tokens_or_come_twice_are_refused(L, on_cpu):
    """The cache starts every request empty, so one with pages of its own, or in two rows, would not match its table."""
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    pool = L.lora_pool_create(None, 64, 64, 1, 1)
    try:
        for layers in (2, 3):                                     # a zero growth fixes the layer count: 2
            L.lora_kv_grow(pool, 5, 0 if layers == 2 else 1, 2)
            with pytest.raises(ValueError, match="holds"):
                BudgetedCache(HostLib(L), pool, [4, 5], layers, 1, 1, 4, 2, 2)
        with pytest.raises(ValueError, match="twice"):
            BudgetedCache(HostLib(L), pool, [1, 2, 1], 2, 1, 1, 4, 2, 2)
        assert L.lora_pool_stats(pool)["reserved"] == 4
        L.lora_kv_free(pool, 5)
        BudgetedCache(HostLib(L), pool, [4, 5], 3, 1, 1, 4, 2, 2).grow()
    finally:
        L.lora_pool_destroy(pool)
