"""Prompt attention, tree attention and slot maps without a GPU: what the entry points refuse, and the oracles
against closed forms and against each other."""
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
A, B, C, D, E, F, G, K = (0x10000 * (i + 1) for i in range(8))


def _refused(L, fn, message, **over):
    with pytest.raises(L.LoraError) as e:
        fn(**over)
    assert e.value.code == L.LORA_EINVAL
    assert message in e.value.message, e.value.message


@pytest.mark.parametrize("over,message", [
    (dict(n_seq=-1), "bad arguments"), (dict(n_heads=0), "bad arguments"), (dict(n_kv_heads=0), "bad arguments"),
    (dict(pool=None), "bad arguments"), (dict(n_seq=65536), "65535"), (dict(n_rows=-1), "n_rows"), (dict(n_rows=65537), "n_rows"),
    (dict(n_heads=6), "1 to 16 times"), (dict(n_heads=68), "1 to 16 times"), (dict(n_heads=3, n_kv_heads=3), "multiple of n_kv_heads"),
    (dict(n_heads=8, n_kv_heads=8), "head width"), (dict(seq_start_dev=None), "null pointer"), (dict(q_dev=None), "null pointer"),
    (dict(k_dev=None), "null pointer"), (dict(v_dev=None), "null pointer"), (dict(out_dev=None), "null pointer"),
    (dict(workspace_dev=None), "null pointer"), (dict(q_stride=504), "strides"), (dict(q_stride=516), "strides"),
    (dict(out_stride=8), "strides"), (dict(k_stride=248), "strides"), (dict(v_stride=260), "strides"), (dict(q_stride=-8), "strides"),
    (dict(v_stride=(1 << 32) + 8), "strides"), (dict(q_dev=B + 8), "16-byte"), (dict(k_dev=C + 2), "16-byte"),
    (dict(v_dev=D + 4), "16-byte"), (dict(out_dev=E + 8), "16-byte"), (dict(out_dev=B), "alias"), (dict(out_dev=C), "alias"),
    (dict(out_dev=D), "alias"), (dict(seq_start_dev=A + 2), "4-byte"), (dict(lse_dev=G + 1), "4-byte"),
    (dict(workspace_dev=F + 128), "256-byte"), (dict(workspace_bytes=8), "workspace has 8 bytes"),
    (dict(), "planning pool"), (dict(n_seq=0), "planning pool"), (dict(n_rows=0), "planning pool"),
])
def test_attention_prompt_refuses(L, pool, over, message):
    base = dict(pool=pool, n_seq=3, seq_start_dev=A, n_rows=40, q_dev=B, k_dev=C, v_dev=D, out_dev=E, n_heads=8, n_kv_heads=4,
                workspace_dev=F, workspace_bytes=1 << 40, stream=0)
    _refused(L, lambda **o: L.lora_attention_prompt(**{**base, **o}), message, **over)


@pytest.mark.parametrize("over,message", [
    (dict(n_req=-1), "bad arguments"), (dict(n_rows=-1), "bad arguments"), (dict(n_heads=0), "bad arguments"),
    (dict(n_kv_heads=0), "bad arguments"), (dict(pool=None), "bad arguments"), (dict(n_req=65536), "65535"),
    (dict(max_len=0), "max_len"), (dict(max_len=(1 << 30) + 1), "max_len"), (dict(layers=0), "layer outside"),
    (dict(layer=2), "layer outside"), (dict(layer=-1), "layer outside"),
    (dict(n_heads=6), "1 to 16 times"), (dict(n_heads=68), "1 to 16 times"), (dict(n_heads=3, n_kv_heads=3), "multiple of n_kv_heads"),
    (dict(n_heads=8, n_kv_heads=8), "head width"), (dict(table_dev=None), "null pointer"), (dict(seq_len_dev=None), "null pointer"),
    (dict(node_start_dev=None), "null pointer"), (dict(mask_dev=None), "null pointer"), (dict(q_dev=None), "null pointer"),
    (dict(out_dev=None), "null pointer"), (dict(workspace_dev=None), "null pointer"), (dict(q_stride=504), "strides"),
    (dict(q_stride=516), "strides"), (dict(out_stride=8), "strides"), (dict(q_dev=E + 8), "16-byte"), (dict(out_dev=F + 8), "16-byte"),
    (dict(out_dev=E), "alias"), (dict(table_dev=A + 4), "8-byte"), (dict(mask_dev=D + 4), "8-byte"), (dict(seq_len_dev=B + 2), "4-byte"),
    (dict(node_start_dev=C + 2), "4-byte"), (dict(lse_dev=K + 1), "4-byte"), (dict(workspace_dev=G + 64), "256-byte"),
    (dict(workspace_bytes=8), "workspace has 8 bytes"), (dict(), "planning pool"), (dict(n_req=0), "planning pool"),
    (dict(n_rows=0), "planning pool"),
])
def test_attention_tree_refuses(L, pool, over, message):
    base = dict(pool=pool, n_req=3, table_dev=A, seq_len_dev=B, max_len=8, layers=2, layer=1, node_start_dev=C, n_rows=9,
                mask_dev=D, q_dev=E, out_dev=F, n_heads=8, n_kv_heads=4, workspace_dev=G, workspace_bytes=1 << 40, stream=0)
    _refused(L, lambda **o: L.lora_attention_tree(**{**base, **o}), message, **over)


@pytest.mark.parametrize("fn,args,message", [
    ("lora_attention_prompt_size", (3, 65537, 8, 4), "n_rows"), ("lora_attention_prompt_size", (3, -1, 8, 4), "n_rows"),
    ("lora_attention_prompt_size", (-1, 4, 8, 4), "bad arguments"), ("lora_attention_prompt_size", (3, 4, 9, 4), "1 to 16 times"),
    ("lora_attention_prompt_size", (3, 4, 8, 8), "head width"), ("lora_attention_tree_size", (3, 0, 8, 4), "max_len"),
    ("lora_attention_tree_size", (3, (1 << 30) + 1, 8, 4), "max_len"), ("lora_attention_tree_size", (65536, 4, 8, 4), "65535"),
    ("lora_attention_tree_size", (3, 4, 9, 4), "1 to 16 times"), ("lora_attention_tree_size", (3, 4, 8, 8), "head width"),
])
def test_size_queries_refuse(L, pool, fn, args, message):
    _refused(L, lambda: getattr(L, fn)(pool, *args), message)
    with pytest.raises(L.LoraError):
        getattr(L, fn)(None, 1, 1, 8, 4)


@pytest.mark.parametrize("over,message", [
    (dict(n_req=-1), "bad arguments"), (dict(row_cap=-1), "bad arguments"), (dict(max_len=0), "bad arguments"),
    (dict(layers=0), "bad arguments"), (dict(pool=None), "bad arguments"), (dict(n_req=65536), "65535"),
    (dict(max_len=(1 << 30) + 1), "2^30"), (dict(layers=(1 << 20) + 1), "2^20"), (dict(count_dev=None), "null pointer"),
    (dict(pages_dev=None), "null pointer"), (dict(table_dev=None), "null pointer"), (dict(new_len_dev=None), "null pointer"),
    (dict(row_start_dev=None), "null pointer"), (dict(row_req_dev=None), "null pointer"), (dict(row_pos_dev=None), "null pointer"),
    (dict(table_dev=D + 4), "8-byte"), (dict(pages_dev=C + 4), "8-byte"), (dict(count_dev=A + 2), "4-byte"),
    (dict(old_len_dev=B + 1), "4-byte"), (dict(new_len_dev=E + 2), "4-byte"), (dict(row_start_dev=F + 2), "4-byte"),
    (dict(row_req_dev=G + 2), "4-byte"), (dict(row_pos_dev=K + 2), "4-byte"), (dict(new_len_dev=B), "inputs"),
    (dict(new_len_dev=A), "inputs"), (dict(row_start_dev=A), "inputs"), (dict(row_start_dev=B), "inputs"),
    (dict(row_start_dev=E), "inputs"), (dict(table_dev=C), "inputs"), (dict(row_pos_dev=G), "inputs"),
    (dict(old_len_dev=None, n_req=65535, max_len=1 << 30, layers=2048), "too large"), (dict(), "planning pool"),
    (dict(n_req=0), "planning pool"), (dict(row_cap=0), "planning pool"),
])
def test_kv_append_refuses(L, pool, over, message):
    base = dict(pool=pool, n_req=3, count_dev=A, old_len_dev=B, pages_dev=C, row_cap=10, table_dev=D, max_len=8, layers=2,
                new_len_dev=E, row_start_dev=F, row_req_dev=G, row_pos_dev=K, stream=0)
    _refused(L, lambda **o: L.lora_kv_append(**{**base, **o}), message, **over)


@pytest.mark.parametrize("out", ["table_dev", "new_len_dev", "row_start_dev", "row_req_dev", "row_pos_dev"])
def test_kv_append_refuses_outputs_over_any_other_array(L, pool, out):
    """By a single element at either end; arrays that touch are taken (and the planning pool refused)."""
    at = dict(count_dev=A, old_len_dev=B, pages_dev=C, table_dev=D, new_len_dev=E, row_start_dev=F, row_req_dev=G, row_pos_dev=K)
    size = dict(count_dev=12, old_len_dev=12, pages_dev=160, table_dev=384, new_len_dev=12, row_start_dev=16, row_req_dev=40,
                row_pos_dev=40)
    unit = 8 if out == "table_dev" else 4
    call = lambda **o: L.lora_kv_append(**{**at, **dict(pool=pool, n_req=3, row_cap=10, max_len=8, layers=2, stream=0), **o})  # noqa: E731
    for other in at:
        if other != out:
            for over in (unit - size[out], 0, (size[other] - 1) // unit * unit):       # first element, start, last element
                _refused(L, call, "inputs", **{out: at[other] + over})
            for beside in (-size[out], -(-size[other] // unit) * unit):
                _refused(L, call, "planning pool", **{out: at[other] + beside})


def test_oracle_tree_of_a_chain_is_the_end_of_a_prompt():
    """The last m tokens of a prompt as a chain of drafted nodes: the same rows."""
    rng = np.random.default_rng(0)
    n, m, n_kv, G, D = 23, 7, 2, 3, 64
    H, width = n_kv * D, n_kv * G * D
    bits = lambda r, c: workloads.to_bf16_bits(rng.standard_normal((r, c)).astype(np.float32))  # noqa: E731
    q, k, v = bits(n, width), bits(n, H), bits(n, H)
    prompt = O.attention_prompt(q, k, v, [0, n], n_kv * G, n_kv)
    table = np.stack([np.arange(n), n + np.arange(n)], 1)
    tree = O.attention_tree(np.concatenate([k, v]), [table], [0, m], [(1 << (i + 1)) - 1 for i in range(m)], q[n - m:],
                            n_kv * G, n_kv)
    for key in ("out", "lse", "mag", "vabs", "n"):
        np.testing.assert_allclose(tree[key], prompt[key][n - m:], rtol=1e-13, atol=1e-13)
    one = O.attention_split(np.concatenate([k, v]), [table], q[-1:], n_kv * G, n_kv)
    np.testing.assert_allclose(one["out"][0], prompt["out"][-1], rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(one["lse"][0], prompt["lse"][-1], rtol=1e-13, atol=1e-13)


def test_oracle_rows_that_see_nothing_and_hidden_nan():
    table = np.array([[0, 1], [2, 3]])
    bits = workloads.to_bf16_bits(np.ones((4, 64), np.float32))
    bits[2] = bits[3] = 0x7FC0                                   # token 1: NaN, seen by node 1 alone
    r = O.attention_tree(bits, [table], [0, 2], [0, 0b10], workloads.to_bf16_bits(np.ones((2, 64), np.float32)), 1, 1)
    assert (r["out"][0] == 0).all() and np.isneginf(r["lse"][0]).all() and r["n"].tolist() == [0, 1]
    assert np.isnan(r["out"][1]).all()
    r = O.attention_prompt(np.ones((2, 64), np.uint16), bits[[0, 2]], bits[[1, 3]], [0, 2], 1, 1)
    assert (r["out"][0] == 1).all() and np.isnan(r["out"][1]).all()


def test_oracle_append_closed_form():
    rng = np.random.default_rng(1)
    pages = rng.integers(0, 99, (7, 2, 2))
    table = np.full((3, 4, 2, 2), -1)
    t, new_len, start, req, pos = O.kv_append([2, 0, 3], [0, 1, 2], pages, table, 7)
    assert new_len.tolist() == [2, 1, 4] and start.tolist() == [0, 2, 2, 5]
    assert req.tolist() == [0, 0, 2, 2, -1, -1, -1] and pos.tolist() == [0, 1, 2, 3, 0, 0, 0]     # a token past max_len
    assert (t[0, :2] == pages[:2]).all() and (t[2, 2:] == pages[2:4]).all() and (t[1] == -1).all()
    t, new_len, start, req, _ = O.kv_append([-1, 9], [0, -5], pages, table[:2], 3)
    assert new_len.tolist() == [0, 3] and start.tolist() == [0, 0, 3] and req.tolist() == [1, 1, 1]
