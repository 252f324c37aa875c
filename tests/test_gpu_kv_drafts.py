"""Prompts, decode steps and drafted trees over one budgeted cache (GB300 only): slot maps, page writes and the three
attentions together, every layer checked against the oracle on the rows that the device wrote."""
import numpy as np
import pytest

import oracle as O
import workloads
from helpers import bits_to_torch, torch_to_bits
from kv_bounds import attention_tolerances, row_tolerances

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


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 128), (1, 4, 64), (1, 2, 256)])
def test_a_request_from_its_prompt_through_drafts(L, n_kv, G, D):
    import torch
    from adapter_gemm_lora_gb300.kv_budget import BudgetedCache, random_tree
    H, heads, n, layers, pages = n_kv * D, n_kv * G, 3, 2, 4000
    pool_t = torch.full((pages, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, pages, H, 1, 1, np.random.default_rng(1).permutation(pages))
    try:
        cache = BudgetedCache(L, pool, [10, 11, 12], layers, heads, n_kv, 280, 20, 40)
        rng = np.random.default_rng(D)
        bits = lambda rows, width: workloads.to_bf16_bits(rng.standard_normal((rows, width)).astype(np.float32))  # noqa: E731

        def rows_of(m):
            q, k, v = bits(m, heads * D), bits(m, H), bits(m, H)
            return (q, k, v), [bits_to_torch(x) for x in (q, k, v)], torch.empty((m, heads * D), dtype=torch.bfloat16, device="cuda")

        def check(ref, out):
            got = O.bf16_to_f64(torch_to_bits(out))
            tol, _ = row_tolerances(ref, D)
            assert (np.abs(got - ref["out"]) <= tol).all()

        lengths = [300, 0, 41]
        cache.prefill(lengths)
        for l in range(layers):
            (q, k, v), dev, out = rows_of(sum(lengths))
            cache.attend_prompt(l, *dev, out)
            L.lora_status(pool)
            check(O.attention_prompt(q, k, v, [0, 300, 300, 341], heads, n_kv), out)
            written = torch_to_bits(pool_t)                        # the rows are where the tables say
            for r, (a, b) in enumerate([(0, 300), (300, 300), (300, 341)]):
                tab = L.lora_kv_table(pool, 10 + r, l)
                assert np.array_equal(cache.table[r, :b - a, l].cpu().numpy(), tab)
                assert np.array_equal(written[tab[:, 0]], k[a:b]) and np.array_equal(written[tab[:, 1]], v[a:b])
        for step in range(4):
            counts = [[20, 1, 20], [0, 30, 7], [33, 3, 2], [1, 1, 1]][step]
            trees = [random_tree(rng, c) for c in counts]
            masks = [m for tree, _ in trees for m in tree]
            mask = torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()
            cache.draft(counts)
            starts = [0, counts[0], counts[0] + counts[1], sum(counts)]
            for l in range(layers):
                (q, k, v), dev, out = rows_of(sum(counts))
                cache.attend_drafts(l, *dev, mask, out)
                L.lora_status(pool)
                written = torch_to_bits(pool_t)
                tabs = [L.lora_kv_table(pool, 10 + r, l) for r in range(n)]
                assert all(np.array_equal(cache.table[r, :len(tabs[r]), l].cpu().numpy(), tabs[r]) for r in range(n))
                check(O.attention_tree(written, tabs, starts, masks, q, heads, n_kv), out)
            kept = []
            for _, parent in trees:
                path, j = [], len(parent) - 1
                while j >= 0:
                    path.append(j)
                    j = parent[j]
                kept.append(path[::-1])
            cache.accept(kept)
            # a decode step over what is cached now
            cache.grow()
            for l in range(layers):
                (q, k, v), dev, out = rows_of(n)
                cache.attend(l, *dev, out)
                L.lora_status(pool)
                tabs = [L.lora_kv_table(pool, 10 + r, l) for r in range(n)]
                ref = O.attention_split(torch_to_bits(pool_t), tabs, q, heads, n_kv)
                tol, _, _ = attention_tolerances(ref, cache.lengths, D)
                assert (np.abs(O.bf16_to_f64(torch_to_bits(out)) - ref["out"]) <= tol).all()
        assert cache.evicted > 0                                   # the third draft did not fit request 0's cache
        s = L.lora_pool_stats(pool)
        assert s["reserved"] == 2 * layers * sum(cache.lengths)
        cache.free()
        assert L.lora_pool_stats(pool)["free"] == pages
    finally:
        L.lora_pool_destroy(pool)


def test_a_captured_step_of_prompts(L):
    """Slot maps, page writes and prompt attention in one graph, replayed with other lengths."""
    import torch
    n, H, heads, cap, rows = 3, 256, 4, 80, 150
    rng = np.random.default_rng(4)
    pool_t = torch.zeros((800, H), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 800, H, 1, 1)
    try:
        pages = torch.from_numpy(rng.permutation(800)[:2 * rows].astype(np.int32).reshape(rows, 1, 2)).cuda()
        q, k, v = (bits_to_torch(workloads.to_bf16_bits(rng.standard_normal((rows, H)).astype(np.float32))) for _ in range(3))
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        count, table, new_len, start, req, pos = i32(n), i32(n, cap, 1, 2), i32(n), i32(n + 1), i32(rows), i32(rows)
        out = torch.empty_like(q)
        nb = L.lora_attention_prompt_size(pool, n, rows, heads, heads)
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")

        def step():
            L.lora_kv_append(pool, n, count, None, pages, rows, table, cap, 1, new_len, start, req, pos)
            L.lora_kv_write(pool, rows, req, pos, k, v, n, table, cap, 1, 0)
            L.lora_attention_prompt(pool, n, start, rows, q, k, v, out, heads, heads, ws, nb)

        count.copy_(torch.tensor([10, 20, 30], dtype=torch.int32))
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for lengths in ([10, 20, 30], [70, 0, 80], [1, 1, 1], [0, 0, 0], [50, 50, 50]):
            count.copy_(torch.tensor(lengths, dtype=torch.int32))
            out.fill_(-3)
            pool_t.zero_()
            g.replay()
            L.lora_status(pool)
            starts = np.concatenate([[0], np.cumsum(lengths)])
            ref = O.attention_prompt(torch_to_bits(q), torch_to_bits(k), torch_to_bits(v), starts, heads, heads)
            got = O.bf16_to_f64(torch_to_bits(out))
            total = int(starts[-1])
            tol, _ = row_tolerances(ref, H // heads)
            assert (np.abs(got - ref["out"])[:total] <= tol[:total]).all() and (got[total:] == -3).all()
            ids = pages.cpu().numpy()[:, 0]
            written = torch_to_bits(pool_t)
            assert np.array_equal(written[ids[:total, 0]], torch_to_bits(k)[:total])
            assert np.array_equal(written[ids[:total, 1]], torch_to_bits(v)[:total])
            assert (written[ids[total:].reshape(-1)] == 0).all()   # rows of no request are not written
    finally:
        L.lora_pool_destroy(pool)


def test_the_command_runs_with_prompts_and_drafts(L):
    from adapter_gemm_lora_gb300 import kv_budget
    small = ["--H", "512", "--heads", "4", "--requests", "5", "--steps", "16", "--budget", "24", "--recent", "3", "--slack", "8",
             "--adapters", "2", "--rank", "8"]
    out = kv_budget.main(small + ["--prompt", "30", "--draft", "8"])
    assert out["prompt_tokens"] >= 5 * 15 and out["tokens"] >= 5 * 16 and out["ms_prompt"] > 0
    out = kv_budget.main(small + ["--prompt", "20"])
    assert out["tokens"] == 5 * 16 and out["evicted_tokens"] > 0
