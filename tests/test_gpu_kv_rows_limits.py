"""Prompt and tree attention and slot maps at the largest sizes that they take, and several calls together:
one workspace for calls in a row and for two graphs, one tensor as q, k and v, every call under the profiler."""
import numpy as np
import pytest

import oracle as O
from helpers import bits_to_torch, torch_to_bits
from kv_bounds import row_tolerances
from oracle import kv_oracle
from test_gpu_kv_rows import KINDS, L, Prompt, Tree, _bits, _check, _outputs, _workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def _check_some(c, out, lse, rows):
    """The given rows of a single sequence against the oracle's arithmetic."""
    q, k, v = (O.bf16_to_f64(x) for x in (c.q[rows], c.k, c.v))
    ref = kv_oracle._rows_result(len(rows), c.heads, c.D)
    sees = np.arange(c.rows)[None, :] <= np.array(rows)[:, None]
    kv_oracle._attend_rows(q, k, v, sees, ref, slice(0, len(rows)), c.heads, c.n_kv)
    tol_out, tol_lse = row_tolerances(ref, c.D)
    assert (np.abs(O.bf16_to_f64(torch_to_bits(out[rows].contiguous())) - ref["out"]) <= tol_out).all()
    assert (np.abs(lse[rows].cpu().numpy().astype(np.float64) - ref["lse"]) <= tol_lse).all()


@pytest.mark.parametrize("n_kv,G,D", [(2, 2, 64), (1, 1, 128), (1, 16, 256)])
def test_one_prompt_of_the_largest_batch(L, n_kv, G, D):  # noqa: F811
    c = Prompt(L, n_kv, G, D, [65536], seed=31)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        _check_some(c, out, lse, [0, 1, 127, 128, 4095, 32767, 40001, 65408, 65535])
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(1, 1, 64), (3, 2, 128), (1, 3, 256)])
def test_as_many_prompts_as_there_may_be(L, n_kv, G, D):  # noqa: F811
    """Of one token each: the softmax's weight is 1, so every output is its V."""
    import torch
    c = Prompt(L, n_kv, G, D, [1] * 65535, seed=32, behind=1)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        v = bits_to_torch(c.v).view(-1, n_kv, 1, D).expand(-1, n_kv, G, D).reshape(c.rows, -1)
        assert torch.equal(out[:-1], v[:-1]) and (out[-1] == -3).all() and (lse[-1] == -7).all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(3, 1, 64), (1, 4, 128), (1, 1, 256)])
def test_as_many_trees_as_there_may_be(L, n_kv, G, D):  # noqa: F811
    """Of one node each, behind nothing, in pages of no request's bookkeeping."""
    import torch
    n, H = 65535, n_kv * D
    g = torch.Generator(device="cuda").manual_seed(33)
    pool_t = torch.randn((2 * n, H), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    pool = L.lora_pool_create(pool_t, 2 * n, H, 1, 1)
    try:
        ids = torch.randperm(2 * n, generator=g, device="cuda").to(torch.int32)
        q = torch.randn((n, H * G), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        mask = torch.ones(n, dtype=torch.int64, device="cuda")
        seq, starts = torch.ones(n, dtype=torch.int32, device="cuda"), torch.arange(n + 1, dtype=torch.int32, device="cuda")
        nb = L.lora_attention_tree_size(pool, n, 1, n_kv * G, n_kv)
        out, _ = _outputs(n, H * G, n_kv * G)
        L.lora_attention_tree(pool, n, ids.view(n, 1, 1, 2), seq, 1, 1, 0, starts, n, mask, q, out, n_kv * G, n_kv, _workspace(nb), nb)
        L.lora_status(pool)
        want = pool_t[ids.view(n, 2)[:, 1].long()].view(n, n_kv, 1, D).expand(n, n_kv, G, D).reshape(n, -1)
        assert torch.equal(out, want)
    finally:
        L.lora_pool_destroy(pool)


SHARED_OUT = [   # n_kv, G, D, lengths, rows before and behind: enough full items that the CTAs take them in turn
    (20, 4, 128, [700, 1, 0, 300, 77, 64], 0, 0),
    (8, 8, 64, [1300, 33, 32, 31], 3, 700),
    (4, 16, 64, [17, 40, 16, 33] * 50, 1, 2),          # listed by a kernel of their own
    (12, 2, 256, [500, 640, 3, 900], 5, 1),
    (3, 16, 256, [1000], 0, 0),
    (256, 1, 64, [400, 330, 0, 513, 256, 110], 0, 1),  # K and V beyond L2: 85 heads at a time, and the one left
    (64, 1, 256, [900, 128, 700], 0, 0),
    (40, 2, 128, [128, 127, 300, 600, 5], 0, 2000),    # fewer items than tickets
]


@pytest.mark.parametrize("n_kv,G,D,lengths,before,behind", SHARED_OUT)
def test_items_taken_in_turn(L, n_kv, G, D, lengths, before, behind):  # noqa: F811
    import torch
    c = Prompt(L, n_kv, G, D, lengths, seed=46, before=before, behind=behind)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
        for _ in range(3):
            again = c.run()
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    finally:
        c.close()


SHORT = [   # n_kv, G, D, lengths, rows before and behind: short sequences, which share items
    (40, 1, 128, [5, 0, 1, 90, 0, 0, 140, 3, 3, 250, 7, 1], 0, 3),
    (30, 4, 64, [31, 33, 64, 1, 0, 2, 60, 64, 5, 5], 7, 0),
    (25, 2, 256, [1, 63, 64, 65, 30, 34, 0, 128, 1], 63, 40),
    (33, 3, 128, [42, 84, 41, 1, 85, 20, 20], 1, 1),
    (20, 16, 64, [1, 2, 3, 4, 5, 6, 7, 8, 9, 0, 16, 17, 15], 5, 0),
    (20, 5, 256, [25, 1, 24, 26, 0, 13, 12], 2, 9),
    (3, 2, 128, [1, 0, 2, 127, 3, 0, 0, 9] * 20, 120, 0),
    (2, 1, 64, [200, 56, 0, 256, 1, 255, 90, 90, 76] * 9, 0, 1),
]


@pytest.mark.parametrize("n_kv,G,D,lengths,before,behind", SHORT)
def test_short_prompts_that_share_items(L, n_kv, G, D, lengths, before, behind):  # noqa: F811
    """Against the oracle; then NaN in q, k and v of every other sequence leave the rest as it was."""
    import torch
    c = Prompt(L, n_kv, G, D, lengths, seed=49, before=before, behind=behind)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
        for a, b in list(zip(c.starts[:-1], c.starts[1:]))[::2]:
            for x in (c.q, c.k, c.v):
                x[a:b] = 0x7FC0
        got, lse2 = c.run()
        for a, b in list(zip(c.starts[:-1], c.starts[1:]))[1::2]:
            assert torch.equal(got[a:b], out[a:b]) and torch.equal(lse2[a:b], lse[a:b])
    finally:
        c.close()


def test_items_taken_in_turn_on_two_streams_and_in_a_graph(L):  # noqa: F811
    import torch
    c = Prompt(L, 20, 4, 64, [700, 1, 0, 300, 77, 64], seed=47)
    d = Prompt(L, 8, 8, 128, [90, 1200, 8], seed=48)
    try:
        want_c, want_d = c.run(), d.run()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        results = []
        for _ in range(6):
            with torch.cuda.stream(s1):
                results.append((c.run(stream=s1), want_c))
            with torch.cuda.stream(s2):
                results.append((d.run(stream=s2), want_d))
        torch.cuda.synchronize()
        for got, want in results:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        q, k, v = (bits_to_torch(x) for x in (c.q, c.k, c.v))
        starts = torch.tensor(c.starts, dtype=torch.int32, device="cuda")
        out, lse = _outputs(c.rows, c.heads * c.D, c.heads)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lora_attention_prompt(c.pool, 6, starts, c.rows, q, k, v, out, c.heads, c.n_kv, c.ws, c.ws_bytes, lse_dev=lse)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_c[0]) and torch.equal(lse, want_c[1])
        for now in ([0, 100, 200, 300, 400, 500, 600], [1142] * 7, [0] + [1142] * 6):
            starts.copy_(torch.tensor(now, dtype=torch.int32))
            out.fill_(-3)
            lse.fill_(-7)
            g.replay()
            torch.cuda.synchronize()
            _check(O.attention_prompt(c.q, c.k, c.v, now, c.heads, c.n_kv), out, lse, c.D)
        L.lora_status(c.pool)
    finally:
        c.close()
        d.close()


def test_one_tensor_as_q_k_and_v(L):  # noqa: F811
    c = Prompt(L, 2, 1, 128, [300, 40], seed=34)
    try:
        import torch
        x = bits_to_torch(c.q)
        out, lse = _outputs(c.rows, 256, 2)
        L.lora_attention_prompt(c.pool, 2, torch.tensor(c.starts, dtype=torch.int32, device="cuda"), c.rows, x, x, x, out, 2, 2,
                                c.ws, c.ws_bytes, lse_dev=lse)
        L.lora_status(c.pool)
        _check(O.attention_prompt(c.q, c.q, c.q, c.starts, 2, 2), out, lse, 128)
    finally:
        c.close()


@pytest.mark.parametrize("many", [False, True])
def test_calls_in_a_row_and_two_graphs_share_a_workspace(L, many):  # noqa: F811
    """Every call begins where the one before it has ended, whatever it left in the workspace: prompts, trees whose
    requests lie in several parts, and (many) sequences listed by a kernel of their own."""
    import torch
    a = Prompt(L, 2, 2, 128, [500, 33, 200] + [3] * (140 * many), seed=35)
    b = Prompt(L, 1, 4, 64, [90, 600, 9] + [0, 5] * (100 * many), seed=36)
    c = Tree(L, 2, 2, 128, [900, 2033, 200] + [40] * (150 * many), [20, 64, 1] + [3] * (150 * many), seed=37, kinds=KINDS)
    d = Tree(L, 1, 3, 64, [1500, 60] + [7, 9] * (80 * many), [64, 9] + [5, 0] * (80 * many), seed=38, kinds=KINDS)
    try:
        cases = (a, c, b, d)
        want = [x.run() for x in cases]
        for x, w in zip(cases, want):
            _check(x.reference(), *w, x.D)
            L.lora_status(x.pool)
        ws = _workspace(max(x.ws_bytes for x in cases))
        got = [(x.run(ws=ws), w) for _ in range(3) for x, w in zip(cases, want)]
        torch.cuda.synchronize()
        for g, w in got:
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
        graphs = []
        for x in (a, c):
            out, lse = _outputs(x.rows, x.heads * x.D, x.heads)
            st = torch.tensor(x.starts, dtype=torch.int32, device="cuda")
            ts = [bits_to_torch(t) for t in (x.q, x.k, x.v)] if x is a else x.args()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(2):
                    if x is a:
                        L.lora_attention_prompt(x.pool, len(x.lengths), st, x.rows, *ts, out, x.heads, x.n_kv, ws, x.ws_bytes, lse_dev=lse)
                    else:
                        L.lora_attention_tree(x.pool, x.n_req, x.table, x.seq, x.max_len, 1, 0, st, x.rows, ts[1], ts[2], out, x.heads,
                                              x.n_kv, ws, x.ws_bytes, lse_dev=lse)
            graphs.append((g, out, lse, st, ts))
        for _ in range(3):
            for g, out, lse, *_ in graphs:
                out.fill_(-3)
                lse.fill_(-7)
            for g, *_ in graphs:
                g.replay()
            torch.cuda.synchronize()
            for (g, out, lse, *_), w in zip(graphs, (want[0], want[1])):
                assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    finally:
        for x in (a, b, c, d):
            x.close()


def test_profiled_calls(L):  # noqa: F811
    import torch
    a = Prompt(L, 2, 2, 128, [500, 33], seed=39)
    c = Tree(L, 2, 2, 64, [900, 33], [20, 9], seed=40)
    try:
        for x, launches in ((a, 1), (c, 2)):
            want = x.run()
            L.lora_profile_read(x.pool)                      # launches are always counted: from here on
            L.lora_profile_enable(x.pool)
            got = x.run()
            kinds = L.lora_profile_read(x.pool)
            L.lora_profile_enable(x.pool, False)
            assert sum(k["launches"] for k in kinds.values()) == launches
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    finally:
        a.close()
        c.close()


def test_slot_maps_in_a_row(L):  # noqa: F811
    """Each call's new lengths are the next one's old ones, with nothing between: what the last leaves is what the
    oracle makes of them in turn."""
    import torch
    rng = np.random.default_rng(41)
    n, layers, max_len, turns = 40, 2, 90, 6
    table = np.full((n, max_len, layers, 2), -1, np.int32)
    pool_t = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 1, 64, 1, 1)
    try:
        counts = [rng.integers(0, 14, n).astype(np.int32) for _ in range(turns)]
        pages = [rng.integers(0, 1 << 30, (int(x.sum()) + 2, layers, 2)).astype(np.int32) for x in counts]
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        d_counts, d_pages, t = [dev(x) for x in counts], [dev(x) for x in pages], dev(table.copy())
        lens = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(turns + 1)]
        maps = [[torch.full((m,), -99, dtype=torch.int32, device="cuda") for m in (n + 1, len(p), len(p))] for p in pages]
        torch.cuda.synchronize()
        for i in range(turns):
            L.lora_kv_append(pool, n, d_counts[i], lens[i], d_pages[i], len(pages[i]), t, max_len, layers, lens[i + 1], *maps[i])
        L.lora_status(pool)
        old = [0] * n
        for i in range(turns):
            table, new, start, req, pos = O.kv_append(counts[i], old, pages[i], table, len(pages[i]))
            old = new
            assert np.array_equal(lens[i + 1].cpu().numpy(), new)
            for got, want in zip(maps[i], (start, req, pos)):
                assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(t.cpu().numpy(), table)
    finally:
        L.lora_pool_destroy(pool)


VALUES = np.array([0x7F80, 0xFF80, 0x7FC0], np.uint16)


@pytest.mark.parametrize("n_kv,G,D", [(9, 1, 64), (6, 2, 128), (5, 3, 128), (7, 1, 256), (2, 16, 64)])
def test_infinities_all_over_many_prompts(L, n_kv, G, D):  # noqa: F811
    """Many items per CTA, infinities and NaN in any of them and in the rows behind the last sequence."""
    import torch
    rng = np.random.default_rng(42)
    lengths = [int(x) for x in rng.integers(1, 300, 70)]
    c = Prompt(L, n_kv, G, D, lengths, seed=43, behind=60)
    try:
        want, z = c.run()
        expect = want.float().view(c.rows, n_kv, G, D).clone()
        for _ in range(900):
            s, d, kv = int(rng.integers(0, 70)), int(rng.integers(0, D)), int(rng.integers(0, n_kv))
            row, value = c.starts[s] + int(rng.integers(0, lengths[s])), rng.choice(VALUES, 1)
            if c.v[row, kv * D + d] & 0x7F80 != 0x7F80:
                c.v[row, kv * D + d] = value[0]
                expect[row:c.starts[s + 1], kv, :, d] += bits_to_torch(value).float()
        c.v[c.starts[-1]:] = 0x7FC0
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2)
        expect = expect.view(c.rows, -1)
        assert torch.equal(got.isnan(), expect.isnan())
        assert torch.equal(got.float().nan_to_num(0), expect.nan_to_num(0))
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(9, 1, 64), (5, 2, 128), (4, 3, 128), (3, 1, 256), (2, 16, 64)])
def test_infinities_all_over_many_trees(L, n_kv, G, D):  # noqa: F811
    import torch
    rng = np.random.default_rng(44)
    lengths = [int(x) for x in rng.integers(64, 700, 40)]
    nodes = [int(x) for x in rng.integers(1, 65, 40)]
    c = Tree(L, n_kv, G, D, lengths, nodes, seed=45, kinds=KINDS)
    try:
        want, z = c.run()
        alive = ~torch.isneginf(z).view(c.rows, n_kv, G, 1)                                # rows that see a token
        expect = want.float().view(c.rows, n_kv, G, D).clone()
        tabs = c.tables()
        for _ in range(600):
            r, d, kv = int(rng.integers(0, 40)), int(rng.integers(0, D)), int(rng.integers(0, n_kv))
            base = lengths[r] - nodes[r]
            j, value = max(0, lengths[r] - 1 - int(rng.integers(0, 130))), rng.choice(VALUES, 1)
            if c.bits[tabs[r][j, 1], kv * D + d] & 0x7F80 == 0x7F80:
                continue
            c.bits[tabs[r][j, 1], kv * D + d] = value[0]
            for i in range(nodes[r]):
                if j < base or (c.masks[c.starts[r] + i] >> (j - base)) & 1:
                    expect[c.starts[r] + i, kv, :, d] += bits_to_torch(value).float()
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2)
        expect = torch.where(alive, expect, torch.zeros_like(expect)).view(c.rows, -1)
        assert torch.equal(got.isnan(), expect.isnan())
        assert torch.equal(got.float().nan_to_num(0), expect.nan_to_num(0))
    finally:
        c.close()
