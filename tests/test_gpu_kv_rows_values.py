"""Values at the ends of the range in prompt and tree attention."""
import numpy as np
import pytest

import oracle as O
import workloads
from helpers import bits_to_torch, torch_to_bits
from kv_bounds import row_tolerances
from test_gpu_kv_rows import L, Prompt, Tree, _bf16  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 2, 128), (1, 3, 128), (1, 2, 256), (1, 16, 64)])
@pytest.mark.parametrize("low", ["first", "last"])
def test_tree_infinities_in_a_part_far_below(L, n_kv, G, D, low):  # noqa: F811
    """One request over many SMs, half of its scores 300 above the others: an infinity of V whose weight is far below
    2^-100 of the row's largest is that infinity or NaN, a NaN is NaN, whichever part they lie in."""
    import torch
    n, m = 4000, 9
    c = Tree(L, n_kv, G, D, [n], [m], seed=21, kinds=("any",))
    try:
        tab, base = c.tables()[0], n - m
        q, k = np.zeros((m, c.heads * D), np.float32), np.zeros((n, n_kv * D), np.float32)
        q[:, ::D] = np.sqrt(D)
        k[(np.arange(n) >= 2000) == (low == "first"), ::D] = 300.0
        c.q, c.bits[tab[:, 0]] = workloads.to_bf16_bits(q), workloads.to_bf16_bits(k)
        c.masks = [(1 << m) - 2 if i % 2 else (1 << m) - 1 for i in range(m)]              # odd rows do not see node 0
        want, z = c.run()
        tokens = (130, 700, 1900) if low == "first" else (2100, 2700, base)
        for d, j, value in zip((3, 5, 9), tokens, (0x7F80, 0x7FC0, 0xFF80)):
            c.bits[tab[j, 1], d] = value
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2) and want.isfinite().all()
        hit = torch.zeros((m, n_kv, G, D), dtype=torch.bool, device="cuda")
        hit[:, 0, :, [3, 5, 9]] = True
        if low == "last":
            hit[1::2, 0, :, 9] = False                                                     # the infinity is node 0's
        hit = hit.view(m, -1)
        assert not got[hit].isfinite().any()
        assert got.view(m, n_kv, G, D)[:, 0, :, 5].isnan().all()
        assert torch.equal(got[~hit], want[~hit])
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(1, 1, 64), (1, 1, 128), (2, 3, 128), (1, 2, 256), (40, 4, 64)])
def test_prompt_rows_without_weight_behind_infinities(L, n_kv, G, D):  # noqa: F811
    """Every score -infinity: out 0 and lse -infinity, whatever V holds in blocks that every row of a tile sees."""
    c = Prompt(L, n_kv, G, D, [700, 3], seed=22)
    try:
        c.q[:], c.k[:] = _bf16(1.0), 0
        c.q[:, ::D], c.k[:, ::D] = _bf16(3e38), _bf16(-3e38)
        c.v[:100] = 0x7F80
        c.v[3:90:5] = 0x7FC0
        c.v[300:310] = 0xFF80
        out, lse = c.run()
        L.lora_status(c.pool)
        assert (out == 0).all() and (lse == float("-inf")).all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(16, 1, 64), (8, 2, 128), (6, 3, 128), (5, 2, 256), (2, 16, 64)])
def test_tree_rows_without_weight_behind_infinities(L, n_kv, G, D):  # noqa: F811
    """Likewise, requests of several blocks that lie in one part or in two."""
    lengths = [400 + 13 * i for i in range(40)]
    c = Tree(L, n_kv, G, D, lengths, [9] * 40, seed=23)
    try:
        c.q[:] = _bf16(1.0)
        c.q[:, ::D] = _bf16(3e38)
        for tab in c.tables():
            k = np.zeros((len(tab), n_kv * D), np.uint16)
            k[:, ::D] = _bf16(-3e38)
            c.bits[tab[:, 0]] = k
            c.bits[tab[:100, 1]] = 0x7F80
            c.bits[tab[140:150, 1]] = 0x7FC0
        out, lse = c.run()
        L.lora_status(c.pool)
        assert (out == 0).all() and (lse == float("-inf")).all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D,n", [(26, 1, 64, 120), (12, 1, 128, 300), (10, 3, 64, 200), (9, 2, 256, 180)])
def test_tree_many_items_of_a_cta_with_infinities_in_most(L, n_kv, G, D, n):  # noqa: F811
    """Ten items and more per SM, the last of them often a request's first blocks without its nodes, infinities and NaN
    in the nodes of most requests, mask bits above the nodes' number: every row has those that it sees and no others."""
    import torch
    rng = np.random.default_rng(27)
    lengths, nodes = [int(x) for x in rng.integers(130, 330, n)], [int(x) for x in rng.integers(1, 20, n)]
    c = Tree(L, n_kv, G, D, lengths, nodes, seed=28, kinds=("any", "tree"))
    try:
        want, z = c.run()
        alive = ~torch.isneginf(z).view(c.rows, n_kv, G, 1)
        expect = want.float().view(c.rows, n_kv, G, D).clone()
        tabs = c.tables()
        for r in rng.permutation(n)[:n * 4 // 5]:
            i, d, kv = int(rng.integers(0, nodes[r])), int(rng.integers(0, D)), int(rng.integers(0, n_kv))
            value = rng.choice(np.array([0x7F80, 0xFF80, 0x7FC0], np.uint16), 1)
            c.bits[tabs[r][lengths[r] - nodes[r] + i, 1], kv * D + d] = value[0]
            for row in range(c.starts[r], c.starts[r + 1]):
                if (c.masks[row] >> i) & 1:
                    expect[row, kv, :, d] += bits_to_torch(value).float()
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2)
        expect = torch.where(alive, expect, torch.zeros_like(expect)).view(c.rows, -1)
        assert torch.equal(got.isnan(), expect.isnan())
        assert torch.equal(got.float().nan_to_num(0), expect.nan_to_num(0))
    finally:
        c.close()


def _far(rng, shape, D, power):
    """Rows whose first feature of each head alone is not zero: 2^power times a bf16 value of 1 to 2, of either sign."""
    x = np.zeros(shape, np.float32)
    x[:, ::D] = 2.0 ** power * (1 + rng.integers(0, 128, x[:, ::D].shape) / 128.0) * rng.choice([-1.0, 1.0], x[:, ::D].shape)
    return workloads.to_bf16_bits(x)


def _check_far(ref, out, lse, D):
    """Scores are one product each, exact in fp32, and far apart or equal: as row_tolerances, without their errors."""
    tol, tol_z = row_tolerances({**ref, "mag": np.zeros_like(ref["mag"])}, D)
    assert (np.abs(O.bf16_to_f64(torch_to_bits(out)) - ref["out"]) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - ref["lse"]) <= tol_z).all()


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 2, 128), (1, 3, 128), (1, 2, 256), (50, 1, 64)])
@pytest.mark.parametrize("power", [13, 16, 18, 30, 62])
def test_prompt_scores_past_the_range_of_the_exponent(L, n_kv, G, D, power):  # noqa: F811
    """Scores whose steps in fp32 are larger than any exponent, V near the end of its range."""
    c = Prompt(L, n_kv, G, D, [300, 45], seed=25)
    try:
        c.q, c.k = (_far(c.rng, x.shape, D, power) for x in (c.q, c.k))
        c.v = workloads.to_bf16_bits((3.0e38 * (0.5 + 0.5 * c.rng.random(c.v.shape))).astype(np.float32))
        out, lse = c.run()
        L.lora_status(c.pool)
        _check_far(c.reference(), out, lse, D)
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 2, 128), (1, 3, 128), (1, 2, 256)])
@pytest.mark.parametrize("power", [13, 16, 18, 30, 62])
def test_tree_scores_past_the_range_of_the_exponent(L, n_kv, G, D, power):  # noqa: F811
    c = Tree(L, n_kv, G, D, [2000, 90, 300], [30, 5, 64], seed=26, kinds=("any", "tree"))
    try:
        tab = np.concatenate(c.tables())
        c.q, c.bits[tab[:, 0]] = _far(c.rng, c.q.shape, D, power), _far(c.rng, (len(tab), n_kv * D), D, power)
        c.bits[tab[:, 1]] = workloads.to_bf16_bits((3.0e38 * (0.5 + 0.5 * c.rng.random((len(tab), n_kv * D)))).astype(np.float32))
        out, lse = c.run()
        L.lora_status(c.pool)
        _check_far(c.reference(), out, lse, D)
    finally:
        c.close()


def test_tree_items_that_take_long(L):  # noqa: F811
    """24 million cached tokens that share 512 pages: an SM's share is one item of 94,000 blocks, which takes longer than
    any wait for a single block may.  Sums of n terms are off by n steps of fp32, 2^-23, at most: 8 products a block."""
    import torch
    heads, D, n, m = 152, 64, 24_000_000, 64
    H, blocks = heads * D, n / 128
    g = torch.Generator(device="cuda").manual_seed(29)
    pool_t = torch.randn((512, H), generator=g, device="cuda").to(torch.bfloat16)
    pool_t[256:] += 1
    pool = L.lora_pool_create(pool_t, 512, H, 1, 1)
    try:
        ids = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.int32)
        table = torch.stack([ids, ids + 256], 1).contiguous().view(1, n, 1, 2)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        q = (0.5 * torch.randn((m, H), generator=g, device="cuda")).to(torch.bfloat16)
        mask = torch.full((m,), -1, dtype=torch.int64, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((m, heads), dtype=torch.float32, device="cuda")
        nb = L.lora_attention_tree_size(pool, 1, n, heads, heads)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        L.lora_attention_tree(pool, 1, table, i32(n), n, 1, 0, i32(0, m), m, mask, q, out, heads, heads, ws, nb, lse_dev=lse)
        L.lora_status(pool)
        k, v = (x.double().view(256, heads, D) for x in (pool_t[:256], pool_t[256:]))
        s = torch.einsum("ihd,jhd->ihj", q.double().view(m, heads, D), k) / D ** 0.5
        times = torch.bincount(ids, minlength=256).double()
        want_lse = torch.logsumexp(s + times.log(), 2)
        p = torch.exp(s + times.log() - want_lse[..., None])
        want, size = torch.einsum("ihj,jhd->ihd", p, v), torch.einsum("ihj,jhd->ihd", p, v.abs())
        tol = (9 * blocks * 2.0 ** -23 + 2.0 ** -7) * size + 2.0 ** -8 * want.abs()
        assert ((out.double().view(m, heads, D) - want).abs() <= tol).all()
        assert ((lse.double() - want_lse).abs() <= 2 * blocks * 2.0 ** -23 + 1e-4).all()
    finally:
        L.lora_pool_destroy(pool)
