"""A decode loop under a KV budget (GB300 only): the library's projections, page writes, attention and
eviction together, every step checked against the oracle on the rows that the device wrote."""
import numpy as np
import pytest

import oracle as O
import workloads
from helpers import bits_to_torch, torch_to_bits
from kv_bounds import attention_tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adapter_gemm_lora_gb300 import build
    build.build()
    import adapter_gemm_lora_gb300 as lib
    lib.library()
    return lib


def test_decode_loop_under_a_budget(L):
    import torch
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache
    H, heads, n, layers, budget, recent, slack = 256, 2, 3, 2, 12, 4, 5
    order = np.random.default_rng(1).permutation(400)
    pool_t = torch.full((400, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool, model = L.lora_pool_create(pool_t, 400, H, 1, 1, order), O.PoolModel(400, 1, 1, order)
    try:
        cache = BudgetedCache(L, pool, [10, 11, 12], layers, heads, heads, budget, recent, slack)
        rng = np.random.default_rng(2)
        weight = np.zeros((layers, n, budget + slack))
        bound = np.zeros_like(weight)                          # of the weights' accumulated error
        out = torch.empty((n, H), dtype=torch.bfloat16, device="cuda")
        length = 0
        for step in range(40):
            if length == budget + slack:                       # what make_room is about to do
                dev = cache.weight.cpu().numpy()               # near ties are the device's to break
                keep = [[O.evict_keep(dev[l, r], length, budget, recent) for l in range(layers)] for r in range(n)]
                new, new_bound = np.zeros_like(weight), np.zeros_like(weight)
                for r in range(n):
                    assert model.kv_keep(10 + r, keep[r]) == O.OK
                    for l in range(layers):
                        new[l, r, :budget] = weight[l, r, keep[r][l]]
                        new_bound[l, r, :budget] = bound[l, r, keep[r][l]]
                weight, bound, length = new, new_bound, budget
            cache.grow()
            for r in range(n):
                assert model.kv_grow(10 + r, 1, layers)[0] == O.OK
            length += 1
            assert cache.lengths == [length] * n and cache.seq_len.tolist() == [length] * n
            for l in range(layers):
                q, k, v = (workloads.to_bf16_bits(2 * rng.standard_normal((n, H)).astype(np.float32)) for _ in range(3))
                cache.attend(l, bits_to_torch(q), bits_to_torch(k), bits_to_torch(v), out)
                L.lora_status(pool)
                tabs = [model.kv_table(10 + r, l) for r in range(n)]
                assert all(np.array_equal(cache.table[r, :length, l].cpu().numpy(), tabs[r]) for r in range(n))
                rows = torch_to_bits(pool_t)
                assert all(np.array_equal(rows[tabs[r][-1, 0]], k[r]) and np.array_equal(rows[tabs[r][-1, 1]], v[r])
                           for r in range(n))
                ref = O.attention_split(rows, tabs, q, heads, heads)
                got = O.bf16_to_f64(torch_to_bits(out))
                tol_out, _, tol_w = attention_tolerances(ref, [length] * n, H // heads)
                assert np.all(np.abs(got - ref["out"]) <= tol_out)
                for r in range(n):
                    weight[l, r, :length] += ref["weight"][r]
                    # this step's weights, and two roundings of the sum so far
                    bound[l, r, :length] += tol_w[r] + 2.0 ** -24 * (heads + 2) * weight[l, r, :length] + heads * 2.0 ** -126
                assert np.all(np.abs(cache.weight[l].cpu().numpy() - weight[l]) <= bound[l])
        assert cache.evicted == 5 * slack * n                  # full after steps 17, 22, 27, 32 and 37
        s, ms = L.lora_pool_stats(pool), model.stats()
        assert (s["free"], s["reserved"]) == (ms["free"], ms["reserved"])
        cache.free()
        assert L.lora_pool_stats(pool)["free"] == 400
    finally:
        L.lora_pool_destroy(pool)


def test_the_command_runs(L):
    from adapter_gemm_lora_gb300 import kv_budget
    out = kv_budget.main(["--H", "512", "--heads", "4", "--requests", "5", "--steps", "24", "--budget", "8", "--recent", "3",
                          "--slack", "4", "--adapters", "2", "--rank", "8"])
    assert out["evicted_tokens"] > 0 and out["kv_pages_held"] < out["kv_pages_without_budget"]
