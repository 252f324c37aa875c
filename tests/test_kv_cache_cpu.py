"""KV-cache operators without a GPU: what the entry points refuse, the bookkeeping of an eviction,
and the oracle of attention weights and eviction against closed forms."""
import numpy as np
import pytest

import oracle as O
import workloads


@pytest.fixture(scope="module")
def L():
    from adapter_gemm_lora_gb300 import build
    build.build()
    import adapter_gemm_lora_gb300 as lib
    lib.library()
    return lib


@pytest.fixture()
def pool(L):
    p = L.lora_pool_create(None, 400, 256, 1, 1)
    yield p
    L.lora_pool_destroy(p)


# Addresses that are only looked at: every call below is refused before any device work.
A, B, C, D, E, F, G = (0x10000 * (i + 1) for i in range(7))


def _refused(L, fn, message, **over):
    with pytest.raises(L.LoraError) as e:
        fn(**over)
    assert e.value.code == L.LORA_EINVAL
    assert message in e.value.message, e.value.message


def _attend(L, pool):
    base = dict(pool=pool, n_req=3, table_dev=A, seq_len_dev=B, max_len=8, layers=2, layer=1, q_dev=C, out_dev=D,
                n_heads=8, n_kv_heads=4, workspace_dev=E, workspace_bytes=1 << 30, stream=0)
    return lambda **over: L.lora_attention_split(**{**base, **over})


@pytest.mark.parametrize("over,message", [
    (dict(n_req=-1), "bad arguments"), (dict(max_len=0), "bad arguments"), (dict(n_heads=0), "bad arguments"),
    (dict(n_kv_heads=0), "bad arguments"), (dict(n_req=65536), "65535"), (dict(n_req=65535, max_len=1 << 20), "16 x 2^31"),
    (dict(n_heads=6), "1 to 16 times"),
    (dict(n_heads=68), "1 to 16 times"), (dict(n_heads=3, n_kv_heads=3), "multiple of n_kv_heads"),
    (dict(n_heads=8, n_kv_heads=8), "head width"), (dict(layers=0), "layer outside"), (dict(layer=2), "layer outside"),
    (dict(layer=-1), "layer outside"), (dict(weight_in_dev=F), "weight_in without"), (dict(table_dev=None), "null pointer"),
    (dict(seq_len_dev=None), "null pointer"), (dict(q_dev=None), "null pointer"), (dict(out_dev=None), "null pointer"),
    (dict(workspace_dev=None), "null pointer"), (dict(q_stride=504), "strides"), (dict(q_stride=516), "strides"),
    (dict(out_stride=8), "strides"), (dict(q_stride=-8), "strides"), (dict(weight_out_dev=F, weight_stride=7), "weight_stride"),
    (dict(q_dev=C + 8), "16-byte"), (dict(out_dev=D + 2), "16-byte"), (dict(out_dev=C), "alias"),
    (dict(table_dev=A + 4), "8-byte"), (dict(workspace_dev=E + 128), "256-byte"), (dict(lse_dev=F + 2), "4-byte"),
    (dict(weight_out_dev=F + 1), "4-byte"), (dict(seq_len_dev=B + 2), "4-byte"),
    (dict(), "planning pool"), (dict(n_req=0), "planning pool"),
])
def test_attention_split_refuses(L, pool, over, message):
    _refused(L, _attend(L, pool), message, **over)


@pytest.mark.parametrize("max_len", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 1])
def test_attention_split_refuses_positions_near_32_bits(L, pool, max_len):
    """Positions are 32-bit in the kernels, which look a few tiles past a request's end."""
    _refused(L, _attend(L, pool), "2^30", max_len=max_len)
    with pytest.raises(L.LoraError) as e:
        L.lora_attention_split_size(pool, 3, max_len, 8, 4)
    assert e.value.code == L.LORA_EINVAL and "2^30" in e.value.message
    _refused(L, _attend(L, pool), "planning pool", max_len=1 << 30)


def test_attention_split_size_refuses(L, pool):
    for args, message in [((0, 1, 8, 4), "planning"), ((-1, 1, 8, 4), "bad arguments"), ((1, 0, 8, 4), "bad arguments"),
                          ((1, 1, 9, 4), "1 to 16 times"), ((1, 1, 8, 8), "head width")]:
        with pytest.raises(L.LoraError) as e:
            L.lora_attention_split_size(pool, *args)
        assert e.value.code == L.LORA_EINVAL and message in e.value.message
    with pytest.raises(L.LoraError):
        L.lora_attention_split_size(None, 1, 1, 8, 4)


@pytest.mark.parametrize("over,message", [
    (dict(n_rows=-1), "bad arguments"), (dict(n_req=-1), "bad arguments"), (dict(max_len=-1), "bad arguments"),
    (dict(layers=0), "bad arguments"), (dict(layer=2), "bad arguments"), (dict(layer=-1), "bad arguments"),
    (dict(row_req_dev=None), "null pointer"), (dict(row_pos_dev=None), "null pointer"), (dict(k_dev=None), "null pointer"),
    (dict(v_dev=None), "null pointer"), (dict(table_dev=None), "null pointer"), (dict(k_stride=248), "strides"),
    (dict(v_stride=260), "strides"), (dict(k_dev=C + 8), "16-byte"), (dict(v_dev=D + 4), "16-byte"),
    (dict(table_dev=E + 4), "8-byte"), (dict(row_req_dev=A + 2), "4-byte"), (dict(row_pos_dev=B + 1), "4-byte"),
    (dict(), "planning pool"),
])
def test_kv_write_refuses(L, pool, over, message):
    base = dict(pool=pool, n_rows=4, row_req_dev=A, row_pos_dev=B, k_dev=C, v_dev=D, n_req=2, table_dev=E, max_len=8,
                layers=2, layer=1, stream=0)
    _refused(L, lambda **o: L.lora_kv_write(**{**base, **o}), message, **over)


@pytest.mark.parametrize("over,message", [
    (dict(n_req=-1), "bad arguments"), (dict(max_len=0), "bad arguments"), (dict(layers=0), "bad arguments"),
    (dict(budget=0), "budget"), (dict(recent=-1), "budget"), (dict(recent=5), "budget"), (dict(max_len_out=3), "max_len_out"),
    (dict(table_dev=None), "null pointer"), (dict(seq_len_dev=None), "null pointer"), (dict(weight_dev=None), "null pointer"),
    (dict(keep_dev=None), "null pointer"), (dict(new_len_dev=None), "null pointer"), (dict(table_out_dev=None), "null pointer"),
    (dict(weight_out_dev=None), "null pointer"), (dict(table_dev=A + 4), "8-byte"), (dict(table_out_dev=F + 4), "8-byte"),
    (dict(seq_len_dev=B + 2), "4-byte"), (dict(weight_dev=C + 1), "4-byte"), (dict(keep_dev=D + 2), "4-byte"),
    (dict(new_len_dev=E + 2), "4-byte"), (dict(weight_out_dev=G + 2), "4-byte"), (dict(table_out_dev=A), "inputs"), (dict(weight_out_dev=C), "inputs"), (dict(new_len_dev=B), "inputs"),
    (dict(n_req=65536, layers=65536), "too many"), (dict(max_len=(1 << 30) + 1), "2^30"),
    (dict(max_len_out=(1 << 30) + 1), "2^30"), (dict(), "planning pool"),
])
def test_kv_evict_refuses(L, pool, over, message):
    base = dict(pool=pool, n_req=3, table_dev=A, seq_len_dev=B, max_len=8, layers=2, weight_dev=C, budget=4, recent=2,
                keep_dev=D, new_len_dev=E, table_out_dev=F, weight_out_dev=G, max_len_out=4, stream=0)
    _refused(L, lambda **o: L.lora_kv_evict(**{**base, **o}), message, **over)


@pytest.mark.parametrize("budget", [(1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1])
def test_kv_evict_refuses_budgets_near_32_bits(L, pool, budget):
    """The kernels step past the end of a row's kept list in 32 bits."""
    base = dict(pool=pool, n_req=1, table_dev=A, seq_len_dev=B, max_len=8, layers=1, weight_dev=C, recent=2, keep_dev=D,
                new_len_dev=E, table_out_dev=F, weight_out_dev=G, max_len_out=8, stream=0)
    _refused(L, lambda **o: L.lora_kv_evict(**{**base, **o}), "2^30", budget=budget)
    _refused(L, lambda **o: L.lora_kv_evict(**{**base, **o}), "planning pool", budget=1 << 30)


# ---- bookkeeping of an eviction ----------------------------------------------------------------
def test_kv_keep_by_hand(L):
    """Three tokens of two layers on 14 pages: layer 0 keeps tokens 0 and 2, layer 1 tokens 1 and 2."""
    p = L.lora_pool_create(None, 14, 64, 1, 1)
    try:
        assert L.lora_kv_grow(p, 5, 3, 2) == [13, 12, 11, 10, 9, 8, 7, 6, 5, 4, 3, 2]
        L.lora_kv_keep(p, 5, [[0, 2], [1, 2]])
        assert L.lora_kv_table(p, 5, 0).tolist() == [[13, 12], [5, 4]]
        assert L.lora_kv_table(p, 5, 1).tolist() == [[7, 6], [3, 2]]
        assert L.lora_pool_stats(p)["free"] == 2 + 4
        # freed in the order they were taken (token 0 layer 1, then token 1 layer 0), taken from the end
        assert L.lora_pool_reserve(p, 4).tolist() == [8, 9, 10, 11]
    finally:
        L.lora_pool_destroy(p)


@pytest.mark.parametrize("keep,message", [
    ([[0, 3]], "ascend"), ([[-1, 2]], "ascend"), ([[1, 1]], "ascend"), ([[2, 1]], "ascend"), ([[0, 1, 2, 2]], "ascend"),
])
def test_kv_keep_refuses_and_changes_nothing(L, pool, keep, message):
    L.lora_kv_grow(pool, 1, 3, 1)
    before = L.lora_kv_table(pool, 1, 0).tolist(), L.lora_pool_stats(pool)
    _refused(L, lambda: L.lora_kv_keep(pool, 1, keep), message)
    assert (L.lora_kv_table(pool, 1, 0).tolist(), L.lora_pool_stats(pool)) == before
    _refused(L, lambda: L.lora_kv_keep(pool, 2, [[0]]), "holds no pages")
    with pytest.raises(ValueError):
        L.lora_kv_keep(pool, 1, [0, 1])


@pytest.mark.parametrize("keep", [[[0]], [[0, 1]], [[0], [0], [0]], np.zeros((0, 1)), np.zeros((0, 0)), np.zeros((3, 0)),
                                  np.zeros((1, 0))])
def test_kv_keep_refuses_rows_that_are_not_the_layers(L, pool, keep):
    """One row per layer of the request, neither fewer (the rest would be read past the array) nor more."""
    L.lora_kv_grow(pool, 1, 3, 2)
    before = [L.lora_kv_table(pool, 1, l).tolist() for l in range(2)], L.lora_pool_stats(pool)
    _refused(L, lambda: L.lora_kv_keep(pool, 1, keep), "2 layers")
    assert ([L.lora_kv_table(pool, 1, l).tolist() for l in range(2)], L.lora_pool_stats(pool)) == before
    L.lora_kv_keep(pool, 1, np.zeros((2, 0)))
    assert L.lora_kv_length(pool, 1) == 0


def test_kv_keep_matches_the_oracle_over_random_sequences(L):
    rng = np.random.default_rng(17)
    order = rng.permutation(600)
    pool, model = L.lora_pool_create(None, 600, 64, 1, 1, order), O.PoolModel(600, 1, 1, order)
    layers = 3
    try:
        for step in range(120):
            r = int(rng.integers(0, 4))
            n = len(model.kv.get(r, [])) // (2 * layers)
            if rng.random() < 0.5 or r not in model.kv:
                grow = int(rng.integers(0, 9))
                st, ids = model.kv_grow(r, grow, layers)
                if st == O.OK:
                    assert L.lora_kv_grow(pool, r, grow, layers) == ids
                else:
                    with pytest.raises(L.LoraError) as e:
                        L.lora_kv_grow(pool, r, grow, layers)
                    assert e.value.code == st
            else:
                k = int(rng.integers(0, n + 1))
                keep = [sorted(rng.choice(n, size=k, replace=False).tolist()) for _ in range(layers)]
                assert model.kv_keep(r, keep) == O.OK
                L.lora_kv_keep(pool, r, np.asarray(keep, np.int32).reshape(layers, k))
            for q in model.kv:
                assert L.lora_kv_length(pool, q) == len(model.kv[q]) // (2 * layers)
                for l in range(layers):
                    assert L.lora_kv_table(pool, q, l).tolist() == model.kv_table(q, l).tolist()
            s, ms = L.lora_pool_stats(pool), model.stats()
            assert (s["free"], s["reserved"]) == (ms["free"], ms["reserved"])
        n_free = L.lora_pool_stats(pool)["free"]
        assert L.lora_pool_reserve(pool, n_free).tolist() == model.free[::-1]
    finally:
        L.lora_pool_destroy(pool)


# ---- the oracle against closed forms ------------------------------------------------------------
def test_oracle_weights_of_two_tokens():
    """One query head, D = 64, K differing in one coordinate: scores 0 and 8 a / 8 = a, so the
    weights are sigmoid(-a) and sigmoid(a), lse = log(1 + e^a)."""
    pool = np.zeros((4, 64), np.uint16)
    pool[1, 5] = workloads.to_bf16_bits(np.float32([2.0]))[0]          # K of token 1
    pool[2, 0], pool[3, 0] = workloads.to_bf16_bits(np.float32([1.0, 3.0]))
    q = np.zeros((1, 64), np.uint16)
    q[0, 5] = workloads.to_bf16_bits(np.float32([4.0]))[0]             # score 8 / sqrt(64) = 1
    res = O.attention_split(pool, [np.array([[0, 2], [1, 3]])], q, 1, 1)
    sig = 1 / (1 + np.exp(-1.0))
    assert np.allclose(res["weight"][0], [1 - sig, sig], rtol=1e-14)
    assert np.allclose(res["lse"], np.log(1 + np.e), rtol=1e-14)
    assert np.allclose(res["out"][0, 0], (1 - sig) * 1 + sig * 3, rtol=1e-14)


def test_oracle_agrees_with_the_unsplit_form_and_shares_heads():
    rng = np.random.default_rng(3)
    pool = workloads.to_bf16_bits(rng.standard_normal((40, 256)).astype(np.float32))
    q = workloads.to_bf16_bits(rng.standard_normal((2, 256)).astype(np.float32))
    tabs = [rng.permutation(40)[:14].reshape(7, 2), np.zeros((0, 2), int)]
    res = O.attention_split(pool, tabs, q, 2, 2)
    assert np.allclose(res["out"], O.attention_decode(pool, tabs, q, 2), rtol=0, atol=1e-12)
    assert np.isclose(res["weight"][0].sum(), 2.0) and np.all(np.isneginf(res["lse"][1]))
    # two query heads on one KV head = each on its own copy of it
    wide = np.concatenate([q[:, :128], q[:, 128:], q[:, :128], q[:, 128:]], axis=1)
    shared = O.attention_split(pool, tabs, wide, 4, 2)["out"]
    assert np.allclose(shared[:, :128], res["out"][:, :128]) and np.allclose(shared[:, 384:], res["out"][:, 128:])


def test_oracle_eviction_by_hand():
    w = np.float32([5, 1, np.nan, 1, 7, 0, 2])
    assert O.evict_keep(w, 7, 4, 2) == [0, 4, 5, 6]
    assert O.evict_keep(w, 7, 5, 2) == [0, 1, 4, 5, 6]               # of the equal weights 1 the earlier one
    assert O.evict_keep(w, 7, 4, 4) == [3, 4, 5, 6]
    assert O.evict_keep(w, 7, 6, 0) == [0, 1, 3, 4, 5, 6]             # NaN goes first
    assert O.evict_keep(w, 7, 7, 3) == list(range(7)) and O.evict_keep(w, 0, 3, 1) == []
    assert O.evict_keep(w, 2, 4, 4) == [0, 1]
