"""Attention of packed prompts and of drafted trees, and slot maps, on the GPU.

The attentions are compared with the fp64 oracle under bounds that follow from the arithmetic
(kv_bounds.row_tolerances); page tables, lengths and slot maps have to be exact."""
import numpy as np
import pytest

import oracle as O
import workloads
from helpers import bits_to_torch, torch_to_bits
from kv_bounds import row_tolerances

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


def _bits(rng, *shape, scale=1.0):
    return workloads.to_bf16_bits(scale * rng.standard_normal(shape).astype(np.float32))


def _bf16(x):
    return workloads.to_bf16_bits(np.float32([x]))[0]


def _check(ref, out, lse, D):
    """Every row of a sequence within its bounds; rows of no sequence as they were (_outputs' fill)."""
    tol_out, tol_lse = row_tolerances(ref, D)
    got = O.bf16_to_f64(torch_to_bits(out.contiguous()))
    live = ~np.isnan(ref["lse"]).all(1)
    assert (got[~live] == -3.0).all()
    assert np.isfinite(got[live]).all()
    bad = np.abs(got - ref["out"])[live] > tol_out[live]
    assert not bad.any(), f"{int(bad.sum())} outputs, first at {np.argwhere(bad)[0]}"
    if lse is not None:
        z = lse.cpu().numpy().astype(np.float64)
        assert (z[~live] == -7.0).all()
        empty = np.isneginf(ref["lse"][live])
        assert np.array_equal(np.isneginf(z[live]), empty)
        err = np.abs(np.where(empty, 0, z[live]) - np.where(empty, 0, ref["lse"][live]))
        assert (err <= tol_lse[live]).all(), err.max()


def _outputs(rows, width, heads):
    import torch
    return (torch.full((rows, width), -3.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, heads), -7.0, dtype=torch.float32, device="cuda"))


def _workspace(n):
    import torch
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")               # NaN patterns everywhere


# ---- prompts ---------------------------------------------------------------------------------
class Prompt:
    """Packed prompts of given lengths, `before` and `behind` rows of no sequence around them."""

    def __init__(self, L, n_kv, G, D, lengths, seed, before=0, behind=0, scale=1.0):
        import torch
        self.L, self.n_kv, self.heads, self.D, self.lengths = L, n_kv, n_kv * G, D, list(lengths)
        rng = self.rng = np.random.default_rng(seed)
        self.rows = before + sum(lengths) + behind
        self.starts = [before + sum(lengths[:i]) for i in range(len(lengths) + 1)]
        self.q, self.k, self.v = (_bits(rng, self.rows, w * D, scale=s) for w, s in ((self.heads, 1.0), (n_kv, scale), (n_kv, 1.0)))
        self.pool_t = torch.zeros((1, n_kv * D), dtype=torch.bfloat16, device="cuda")
        self.pool = L.lora_pool_create(self.pool_t, 1, n_kv * D, 1, 1)
        self.ws_bytes = L.lora_attention_prompt_size(self.pool, len(lengths), self.rows, self.heads, n_kv)
        self.ws = _workspace(self.ws_bytes)

    def reference(self):
        return O.attention_prompt(self.q, self.k, self.v, self.starts, self.heads, self.n_kv)

    def run(self, starts=None, with_lse=True, ws=None, stream=None):
        import torch
        out, lse = _outputs(self.rows, self.heads * self.D, self.heads)
        st = torch.tensor(self.starts if starts is None else starts, dtype=torch.int32, device="cuda")
        self.L.lora_attention_prompt(self.pool, len(self.lengths), st, self.rows, bits_to_torch(self.q), bits_to_torch(self.k),
                                     bits_to_torch(self.v), out, self.heads, self.n_kv, self.ws if ws is None else ws,
                                     self.ws_bytes, lse_dev=lse if with_lse else None, stream=stream)
        return out, lse

    def close(self):
        self.L.lora_pool_destroy(self.pool)


PROMPTS = [   # n_kv, G, D, lengths
    (1, 1, 64, [1]),
    (2, 1, 128, [1, 5, 0, 33, 7]),
    (4, 4, 64, [16, 17, 31, 32, 129]),
    (1, 16, 256, [30, 0, 1]),
    (1, 1, 64, [513, 2]),
    (3, 2, 128, [300, 1, 64]),
    (2, 3, 128, [77, 400]),
    (1, 1, 256, [700, 127, 128, 129]),
    (2, 2, 256, [255, 256, 257]),
    (1, 1, 128, [127, 1, 128, 255, 256, 257, 0, 511]),
    (1, 9, 128, [127, 1, 128]),
    (5, 1, 128, [20, 200, 3]),
    (1, 8, 64, [601]),
    (1, 5, 64, [150, 2, 61]),
    (3, 7, 128, [0, 0, 0]),
    (1, 13, 64, [100, 59]),
    (1, 15, 128, [90]),
    (1, 16, 64, [1, 2, 3, 100]),
    (1, 2, 256, [1] * 300),
    (2, 1, 64, [3, 0, 1, 40] * 90),
    (1, 1, 64, [9, 0] * 800),
    (1, 11, 256, [40, 1, 100]),
    (64, 1, 256, [33, 18]),          # H = 16384
    (128, 1, 64, [9, 40]),
    (1, 2, 128, [2049]),
    (1, 1, 64, [1500, 1400]),
    (1, 4, 256, [770]),
]


@pytest.mark.parametrize("n_kv,G,D,lengths", PROMPTS)
def test_prompt_matches_the_oracle(L, n_kv, G, D, lengths):
    import torch
    c = Prompt(L, n_kv, G, D, lengths, seed=n_kv + 7 * G + D, before=3, behind=2)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
        out2, lse2 = c.run(with_lse=False)
        assert torch.equal(out, out2) and (lse2 == -7.0).all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 2, 64), (1, 1, 128), (1, 3, 128), (1, 2, 256)])
def test_prompt_strides(L, n_kv, G, D):
    """q, k, v as columns of one wider matrix, out with room between rows."""
    import torch
    c = Prompt(L, n_kv, G, D, [150, 0, 41], seed=5)
    try:
        wq, wk = c.heads * D, n_kv * D
        wide = torch.full((c.rows, wq + 2 * wk + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 8:8 + wq], wide[:, 8 + wq:8 + wq + wk], wide[:, 16 + wq + wk:16 + wq + 2 * wk] = (
            bits_to_torch(x) for x in (c.q, c.k, c.v))
        out, lse = _outputs(c.rows, wq + 16, c.heads)
        stride = wide.shape[1]
        L.lora_attention_prompt(c.pool, 3, torch.tensor(c.starts, dtype=torch.int32, device="cuda"), c.rows, wide[:, 8:],
                                wide[:, 8 + wq:], wide[:, 16 + wq + wk:], out, c.heads, n_kv, c.ws, c.ws_bytes, lse_dev=lse,
                                q_stride=stride, k_stride=stride, v_stride=stride, out_stride=wq + 16)
        L.lora_status(c.pool)
        _check(c.reference(), out[:, :wq], lse, D)
        assert (out[:, wq:] == -3.0).all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(1, 1, 64), (2, 1, 128), (1, 3, 128), (1, 2, 256), (1, 16, 64)])
@pytest.mark.parametrize("bad", ["nan", "inf", "low"])
def test_prompt_rows_depend_on_what_they_see_alone(L, n_kv, G, D, bad):
    """Anything in later rows, other sequences and rows of no sequence changes no bit."""
    import torch
    lengths, at = [140, 61, 300], [130, 20, 259]
    c = Prompt(L, n_kv, G, D, lengths, seed=6, before=2, behind=5)
    try:
        want, z = c.run()
        value = {"nan": 0x7FC0, "inf": 0x7F80, "low": 0xFF7F}[bad]
        for s, i in enumerate(at):                                 # from position i on, and around the sequences
            c.k[c.starts[s] + i:c.starts[s + 1]] = value
            c.v[c.starts[s] + i:c.starts[s + 1]] = value
        for rows in (slice(0, 2), slice(c.starts[-1], None)):
            c.q[rows], c.k[rows], c.v[rows] = value, value, value
        got, z2 = c.run()
        L.lora_status(c.pool)
        for s, i in enumerate(at):
            rows = slice(c.starts[s], c.starts[s] + i)
            assert torch.equal(got[rows], want[rows]) and torch.equal(z2[rows], z[rows])
        assert (got[:2] == -3).all() and (got[c.starts[-1]:] == -3).all()
        if bad == "nan":
            for s, i in enumerate(at):
                assert got[c.starts[s] + i:c.starts[s + 1]].isnan().all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 2, 128), (1, 1, 256)])
def test_prompt_infinite_values(L, n_kv, G, D):
    """An infinite V is that infinity in every later row of its feature, NaN where both signs meet, and nothing
    before it; NaN likewise."""
    import torch
    c = Prompt(L, n_kv, G, D, [400, 30], seed=7)
    try:
        want, z = c.run()
        put = [(40, 3, 0x7F80), (200, 3, 0xFF80), (130, 5, 0xFF80), (127, 7, 0x7F80), (128, 8, 0x7FC0), (399, 9, 0x7F80),
               (384, D - 1, 0x7F80), (410, 0, 0xFF80)]
        for row, d, value in put:
            c.v[row, d] = value
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2)
        expect = want.float().view(c.rows, n_kv, G, D).clone()
        for row, d, value in put:
            end = 400 if row < 400 else 430
            expect[row:end, 0, :, d] += bits_to_torch(np.array([value], np.uint16)).float()
        expect = expect.view(c.rows, -1)
        assert torch.equal(got.isnan(), expect.isnan())
        assert torch.equal(got.float().nan_to_num(0), expect.nan_to_num(0))
    finally:
        c.close()


@pytest.mark.parametrize("D,scale", [(64, 30.0), (128, 30.0), (256, 30.0), (128, 1e-3)])
def test_prompt_far_scores(L, D, scale):
    c = Prompt(L, 2, 1, D, [300, 45], seed=11, scale=scale)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
    finally:
        c.close()


@pytest.mark.parametrize("D,rise", [(64, 5.4), (128, 5.4), (256, 5.4), (128, 60.0), (256, 300.0)])
def test_prompt_late_maximum_and_values_near_the_end_of_the_range(L, D, rise):
    """Scores that rise block by block, with V near the largest finite value and of one sign: sums of the weights
    times V pass the range unless the weights stay below one."""
    import torch
    n = 700
    c = Prompt(L, 1, 1, D, [n], seed=12)
    try:
        q = np.zeros((n, D), np.float32)
        q[:, 0] = np.sqrt(D)
        k = np.zeros((n, D), np.float32)
        k[:, 0] = rise * (np.arange(n) // 100)
        c.q, c.k = workloads.to_bf16_bits(q), workloads.to_bf16_bits(k)
        c.v = workloads.to_bf16_bits((3.0e38 * (0.5 + 0.5 * c.rng.random((n, D)))).astype(np.float32))
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
        assert out.isfinite().all() and torch.isfinite(lse).all()
    finally:
        c.close()


def test_prompt_overflowing_scores(L):
    """A score of -infinity takes no weight; a row whose every score is -infinity counts as empty."""
    for D in (64, 128, 256):
        c = Prompt(L, 1, 1, D, [200], seed=8)
        try:
            c.q[:] = _bf16(1.0)
            c.q[:, 0] = _bf16(3e38)
            c.k[:] = 0
            c.k[:3, 0] = _bf16(-3e38)                                  # rows 0 to 2 see nothing else
            c.k[150, 0] = _bf16(-3e38)
            ref = c.reference()                                        # in 64 bits: finite, far below
            out, lse = c.run()
            L.lora_status(c.pool)
            got = O.bf16_to_f64(torch_to_bits(out))
            assert (got[:3] == 0).all() and (lse[:3] == float("-inf")).all()
            tol, tol_z = row_tolerances({**ref, "mag": np.zeros_like(ref["mag"])}, D)
            assert (np.abs(got - ref["out"])[3:] <= tol[3:]).all()
            assert (np.abs(lse.cpu().numpy() - ref["lse"])[3:] <= tol_z[3:]).all()
        finally:
            c.close()


def test_prompt_bad_starts(L):
    """Starts that descend or leave the rows: reported, each taken as the largest so far, clamped."""
    c = Prompt(L, 2, 1, 64, [40, 30, 50], seed=13)
    try:
        for given, taken in [([0, 70, 30, 120], [0, 70, 70, 120]), ([-9, 40, 70, 500], [0, 40, 70, 120]),
                             ([200, 0, 5, 120], [120, 120, 120, 120]), ([0, -2 ** 31, 2 ** 31 - 1, 3], [0, 0, 120, 120])]:
            out, lse = c.run(starts=given)
            with pytest.raises(L.LoraError) as e:
                L.lora_status(c.pool)
            assert e.value.code == L.LORA_EDEVICE
            c_ref = O.attention_prompt(c.q, c.k, c.v, taken, c.heads, c.n_kv)
            _check(c_ref, out, lse, c.D)
    finally:
        c.close()


def test_prompt_two_streams_and_a_graph(L):
    """Two calls at once on two streams with a workspace each, and a captured call replayed with other inputs."""
    import torch
    c = Prompt(L, 4, 2, 128, [500, 33, 200], seed=14)
    d = Prompt(L, 4, 2, 128, [90, 600], seed=15)
    try:
        want_c, want_d = c.run(), d.run()
        for x in (c, d):
            _check(x.reference(), *(want_c if x is c else want_d), 128)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        results = []
        for _ in range(5):
            with torch.cuda.stream(s1):
                results.append((c.run(stream=s1), want_c))
            with torch.cuda.stream(s2):
                results.append((d.run(stream=s2), want_d))
        torch.cuda.synchronize()
        for got, want in results:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # captured: starts and rows are read at replay
        q, k, v = (bits_to_torch(x) for x in (c.q, c.k, c.v))
        starts = torch.tensor(c.starts, dtype=torch.int32, device="cuda")
        out, lse = _outputs(c.rows, c.heads * c.D, c.heads)
        args = (c.pool, 3, starts, c.rows, q, k, v, out, c.heads, c.n_kv, c.ws, c.ws_bytes)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lora_attention_prompt(*args, lse_dev=lse)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_c[0]) and torch.equal(lse, want_c[1])
        starts.copy_(torch.tensor([0, 100, 400, 733], dtype=torch.int32))
        k.copy_(bits_to_torch(_bits(c.rng, c.rows, c.n_kv * c.D)))
        out.fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        _check(O.attention_prompt(c.q, torch_to_bits(k), c.v, [0, 100, 400, 733], c.heads, c.n_kv), out, lse, c.D)
        L.lora_status(c.pool)
    finally:
        c.close()
        d.close()


def test_prompt_of_nothing(L):
    c = Prompt(L, 1, 1, 64, [0, 0], seed=1, before=4)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        assert (out == -3).all() and (lse == -7).all()
        L.lora_attention_prompt(c.pool, 0, None, 4, None, None, None, None, 1, 1, None, 0)
        L.lora_attention_prompt(c.pool, 2, None, 0, None, None, None, None, 1, 1, None, 0)
        L.lora_status(c.pool)
    finally:
        c.close()


# ---- trees -----------------------------------------------------------------------------------
def tree_masks(rng, nodes, kind="tree"):
    """Masks of one request's nodes: a random tree, a chain, nothing but itself, or any bits at all."""
    masks = []
    for i in range(nodes):
        parent = int(rng.integers(-1, i)) if i else -1
        masks.append({"tree": (1 << i) | (masks[parent] if parent >= 0 else 0), "chain": (1 << (i + 1)) - 1, "self": 1 << i,
                      "any": int(rng.integers(0, 1 << 63)) * 2 + int(rng.integers(0, 2))}[kind])
    return masks


class Tree:
    """Requests of given lengths with drafted nodes, in a shuffled pool whose other pages hold NaN."""

    def __init__(self, L, n_kv, G, D, lengths, nodes, layers=1, seed=0, kinds=("tree",), before=0, behind=0, max_len=None,
                 scale=1.0):
        import torch
        self.L, self.n_kv, self.heads, self.D, self.layers = L, n_kv, n_kv * G, D, layers
        self.lengths, self.nodes = list(lengths), list(nodes)
        rng = self.rng = np.random.default_rng(seed)
        H = n_kv * D
        self.num_pages = 2 * layers * sum(lengths) + 64
        self.pool_t = torch.full((self.num_pages, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pool = L.lora_pool_create(self.pool_t, self.num_pages, H, 1, 1, rng.permutation(self.num_pages))
        self.bits = np.full((self.num_pages, H), 0x7FC0, np.uint16)
        self.n_req, self.max_len = len(lengths), max_len or max(list(lengths) + [0]) + 3
        for r, n in enumerate(lengths):
            ids = L.lora_kv_grow(self.pool, r, n, layers)
            if ids:
                self.bits[ids] = _bits(rng, len(ids), H, scale=scale)
        self.table = torch.empty((self.n_req, self.max_len, layers, 2), dtype=torch.int32, device="cuda")
        self.seq = torch.empty(self.n_req, dtype=torch.int32, device="cuda")
        L.lora_kv_batch_table(self.pool, list(range(self.n_req)), self.max_len, self.table, self.seq)
        self.starts = [before + sum(nodes[:i]) for i in range(len(nodes) + 1)]
        self.rows = self.starts[-1] + behind
        self.masks = [0] * before
        for r, m in enumerate(nodes):
            self.masks += tree_masks(rng, m, kinds[r % len(kinds)])
        self.masks += [(1 << 64) - 1] * behind
        self.q = _bits(rng, self.rows, self.heads * D)
        self.ws_bytes = L.lora_attention_tree_size(self.pool, self.n_req, self.max_len, self.heads, n_kv)
        self.ws = _workspace(self.ws_bytes)

    def tables(self, layer=0):
        return [self.L.lora_kv_table(self.pool, r, layer).astype(np.int64) for r in range(self.n_req)]

    def reference(self, layer=0, **over):
        a = dict(kv_tables=self.tables(layer), starts=self.starts, masks=self.masks, skip=())
        a.update(over)
        return O.attention_tree(self.bits, a["kv_tables"], a["starts"], a["masks"], self.q, self.heads, self.n_kv, a["skip"])

    def args(self, layer=0, starts=None):
        import torch
        self.pool_t.copy_(bits_to_torch(self.bits))
        st = torch.tensor(self.starts if starts is None else starts, dtype=torch.int32, device="cuda")
        mask = torch.from_numpy(np.array(self.masks, dtype=np.uint64).view(np.int64)).cuda()
        return st, mask, bits_to_torch(self.q)

    def run(self, layer=0, starts=None, with_lse=True, stream=None, ws=None):
        st, mask, q = self.args(layer, starts)
        out, lse = _outputs(self.rows, self.heads * self.D, self.heads)
        self.L.lora_attention_tree(self.pool, self.n_req, self.table, self.seq, self.max_len, self.layers, layer, st, self.rows,
                                   mask, q, out, self.heads, self.n_kv, self.ws if ws is None else ws, self.ws_bytes,
                                   lse_dev=lse if with_lse else None, stream=stream)
        return out, lse

    def close(self):
        self.L.lora_pool_destroy(self.pool)


KINDS = ("tree", "chain", "any", "self")
TREES = [   # n_kv, G, D, layers, lengths, nodes
    (1, 1, 64, 1, [1], [1]),
    (1, 1, 128, 1, [5, 130, 64], [5, 3, 64]),
    (2, 1, 128, 2, [40, 5, 300, 33], [7, 5, 64, 0]),
    (4, 4, 64, 1, [16, 17, 131, 32, 129], [16, 1, 40, 31, 2]),
    (1, 16, 256, 1, [300, 60, 1], [64, 60, 1]),
    (1, 1, 64, 1, [713, 2], [33, 2]),
    (8, 2, 128, 3, [400, 1, 64], [12, 1, 64]),
    (5, 3, 128, 1, [77, 1000], [20, 64]),
    (9, 9, 128, 1, [127, 1, 128], [9, 1, 30]),
    (20, 1, 128, 1, [20, 200, 3], [20, 50, 3]),
    (1, 8, 64, 1, [4001], [64]),
    (2, 5, 256, 2, [700, 699], [13, 64]),
    (6, 1, 256, 1, [47, 90], [47, 10]),
    (64, 1, 256, 1, [33, 18], [5, 18]),          # H = 16384
    (3, 7, 128, 1, [0, 0, 0], [0, 0, 0]),
    (2, 1, 128, 1, [3, 4, 1, 40] * 60, [3, 2, 0, 17] * 60),
    (1, 2, 128, 1, [1] * 700, [1] * 700),
    (1, 13, 64, 1, [200, 64], [64, 64]),
    (1, 16, 64, 1, [900, 33, 64, 1], [64, 33, 1, 1]),
    (1, 16, 128, 1, [257], [64]),
    (3, 11, 256, 1, [70, 1, 100], [64, 1, 40]),
    (1, 1, 64, 1, [128, 256, 384, 129, 255], [1, 64, 63, 2, 1]),
    (1, 3, 64, 1, [9, 64, 90] * 100, [9, 1, 0] * 100),
    (1, 1, 256, 1, [3000], [1]),
    (2, 2, 64, 1, [6000, 64, 1], [64, 64, 1]),
    (16, 1, 64, 1, [1500, 70], [30, 64]),
]


@pytest.mark.parametrize("n_kv,G,D,layers,lengths,nodes", TREES)
def test_tree_matches_the_oracle(L, n_kv, G, D, layers, lengths, nodes):
    import torch
    c = Tree(L, n_kv, G, D, lengths, nodes, layers, seed=n_kv + 7 * G + D, kinds=KINDS, before=2, behind=3)
    try:
        for layer in range(layers):
            out, lse = c.run(layer)
            L.lora_status(c.pool)
            _check(c.reference(layer), out, lse, D)
            out2, lse2 = c.run(layer, with_lse=False)
            assert torch.equal(out, out2) and (lse2 == -7.0).all()
    finally:
        c.close()


def test_tree_one_node_is_decode_attention(L):
    """One node per request with mask 1: the decode attention's outputs, up to their bounds."""
    import torch
    for n_kv, G, D in ((2, 4, 64), (3, 1, 128), (1, 2, 256)):
        lengths = [1, 700, 128, 33]
        c = Tree(L, n_kv, G, D, lengths, [1] * 4, seed=3)
        try:
            out, lse = c.run()
            split, z = torch.empty_like(out), torch.empty_like(lse)
            n = L.lora_attention_split_size(c.pool, 4, c.max_len, c.heads, n_kv, False)
            ws = _workspace(n)
            L.lora_attention_split(c.pool, 4, c.table, c.seq, c.max_len, 1, 0, bits_to_torch(c.q), split, c.heads, n_kv, ws, n,
                                   lse_dev=z)
            L.lora_status(c.pool)
            tol, tol_z = row_tolerances(c.reference(), D)
            assert (np.abs(out.float().cpu().numpy() - split.float().cpu().numpy()) <= 2 * tol).all()
            assert (np.abs(lse.cpu().numpy() - z.cpu().numpy()) <= 2 * tol_z).all()
        finally:
            c.close()


def test_tree_rows_that_see_nothing(L):
    """No cached token but the nodes, and masks without a bit: out 0, lse -infinity."""
    for n_kv, G, D in ((2, 1, 64), (1, 3, 128), (1, 1, 256)):
        c = Tree(L, n_kv, G, D, [5, 200, 64], [5, 3, 64], seed=4, kinds=("any",))
        try:
            c.masks[1] = c.masks[4] = c.masks[20] = c.masks[-1] = 0          # request 1's nodes still see its cache
            c.masks[7] = 0
            ref = c.reference()
            assert np.isneginf(ref["lse"][[1, 4, 20, 71]]).all() and np.isfinite(ref["lse"][7]).all()
            out, lse = c.run()
            L.lora_status(c.pool)
            _check(ref, out, lse, D)
            assert (out[[1, 4, 20, 71]] == 0).all()
        finally:
            c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 3, 128), (1, 2, 256), (1, 16, 64)])
@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF7F])
def test_tree_rows_depend_on_what_they_see_alone(L, n_kv, G, D, value):
    """Nodes that a row does not see, and pages of no token, may hold anything."""
    import torch
    lengths, nodes = [150, 40, 300], [20, 40, 64]
    c = Tree(L, n_kv, G, D, lengths, nodes, seed=6, kinds=("tree", "chain", "any"))
    try:
        for i in range(c.rows):
            c.masks[i] &= ~0b1001                                    # node 0 and node 3: seen by themselves at most
        for r in range(3):
            c.masks[c.starts[r]] |= 1
            c.masks[c.starts[r] + 3] |= 8
        want, z = c.run()
        for r, tab in enumerate(c.tables()):
            base = lengths[r] - nodes[r]
            c.bits[tab[base]], c.bits[tab[base + 3]] = value, value
        got, z2 = c.run()
        L.lora_status(c.pool)
        rows = np.setdiff1d(np.arange(c.rows), [s + i for s in c.starts[:3] for i in (0, 3)])
        assert torch.equal(got[rows], want[rows]) and torch.equal(z2[rows], z[rows])
        if value == 0x7FC0:
            for s in c.starts[:3]:
                assert got[[s, s + 3]].isnan().all()
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 1, 64), (1, 2, 128), (1, 1, 256)])
def test_tree_infinite_values(L, n_kv, G, D):
    """An infinite V is that infinity in every row that sees it, NaN where both signs meet."""
    import torch
    c = Tree(L, n_kv, G, D, [400], [30], seed=7)
    try:
        want, z = c.run()
        tab = c.tables()[0]
        put = [(40, 3, 0x7F80), (200, 3, 0xFF80), (130, 5, 0xFF80), (127, 7, 0x7F80), (383, 8, 0x7FC0), (399, 9, 0x7F80),
               (384, D - 1, 0x7F80), (370, 0, 0xFF80), (371, 0, 0x7F80)]
        for j, d, value in put:
            c.bits[tab[j, 1], d] = value
        got, z2 = c.run()
        L.lora_status(c.pool)
        assert torch.equal(z, z2)
        expect = want.float().view(30, n_kv, G, D).clone()
        for j, d, value in put:
            for i in range(30):
                if j < 370 or (c.masks[i] >> (j - 370)) & 1:
                    expect[i, 0, :, d] += bits_to_torch(np.array([value], np.uint16)).float()
        expect = expect.view(30, -1)
        assert torch.equal(got.isnan(), expect.isnan())
        assert torch.equal(got.float().nan_to_num(0), expect.nan_to_num(0))
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 2, 128), (1, 9, 64), (3, 2, 64), (1, 3, 256)])
def test_tree_skips_bad_pages_and_clamps_lengths(L, n_kv, G, D):
    import torch
    lengths, nodes = [150, 13, 40], [20, 13, 4]
    c = Tree(L, n_kv, G, D, lengths, nodes, seed=4, kinds=("chain",))
    try:
        tabs = c.tables()
        skip = [(0, 0), (0, 17), (0, 149), (0, 128), (1, 0), (1, 1), (1, 2), (2, 39)]
        for i, (r, j) in enumerate(skip):
            c.table[r, j, 0, i % 2] = (1 << 30) if i != 1 else -5
        out, lse = c.run()
        with pytest.raises(L.LoraError) as e:
            L.lora_status(c.pool)
        assert e.value.code == L.LORA_EDEVICE and "page" in e.value.message
        _check(c.reference(skip=skip), out, lse, D)
        # lengths outside [0, max_len]: reported and clamped; nodes past the length have no position
        c.seq.copy_(torch.tensor([-3, 13, 2], dtype=torch.int32))
        out, lse = c.run()
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        assert (out[:20] == 0).all() and torch.isneginf(lse[:20]).all()
        _check(c.reference(skip=skip, kv_tables=[tabs[0][:0], tabs[1], tabs[2][:2]]), out, lse, D)
        c.seq.copy_(torch.tensor([c.max_len + 1, 13, 40], dtype=torch.int32))       # the tail of row 0 holds -1 pages
        out, lse = c.run()
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        long = np.concatenate([tabs[0], np.zeros((c.max_len - 150, 2), np.int64)])
        tail = [(0, j) for j in range(150, c.max_len)]
        _check(c.reference(skip=skip + tail, kv_tables=[long, tabs[1], tabs[2]]), out, lse, D)
    finally:
        c.close()


def test_tree_too_many_nodes_and_bad_starts(L):
    """Nodes past the 64th are left as they were; starts are taken as the largest so far; both are reported."""
    c = Tree(L, 2, 1, 64, [300, 90], [70, 10], seed=5, kinds=("any",))
    try:
        out, lse = c.run()
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        assert (out[64:70] == -3).all() and (lse[64:70] == -7).all()
        # the request's last 64 tokens are its nodes
        ref = c.reference(starts=[0, 64, 64])
        ref2 = c.reference(starts=[70, 70, 80])
        for key in ref:
            ref[key][70:] = ref2[key][70:]
        _check(ref, out, lse, 64)
        out, lse = c.run(starts=[5, 3, 200])
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        ref = c.reference(starts=[5, 5, 5 + 64])
        _check(ref, out, lse, 64)
    finally:
        c.close()


def test_tree_strides(L):
    import torch
    n_kv, G, D = 4, 2, 64
    c = Tree(L, n_kv, G, D, [100, 64, 333, 16], [10, 64, 0, 3], layers=2, seed=2, kinds=KINDS)
    try:
        width = c.heads * D
        st, mask, q = c.args()
        wide = torch.full((c.rows, width + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 8:8 + width] = q
        out, lse = _outputs(c.rows, width + 16, c.heads)
        L.lora_attention_tree(c.pool, 4, c.table, c.seq, c.max_len, 2, 1, st, c.rows, mask, wide[:, 8:], out, c.heads, n_kv, c.ws,
                              c.ws_bytes, lse_dev=lse, q_stride=width + 72, out_stride=width + 16)
        L.lora_status(c.pool)
        _check(c.reference(1), out[:, :width], lse, D)
        assert (out[:, width:] == -3.0).all()
    finally:
        c.close()


@pytest.mark.parametrize("D,rise", [(64, 5.4), (128, 5.4), (256, 5.4), (128, 300.0)])
def test_tree_late_maximum_and_values_near_the_end_of_the_range(L, D, rise):
    import torch
    n = 4000
    c = Tree(L, 1, 1, D, [n], [9], seed=12, kinds=("any",))
    try:
        tab = c.tables()[0]
        q = np.zeros((9, D), np.float32)
        q[:, 0] = np.sqrt(D)
        k = np.zeros((n, D), np.float32)
        k[:, 0] = rise * (np.arange(n) // 500)
        c.q = workloads.to_bf16_bits(q)
        c.bits[tab[:, 0]] = workloads.to_bf16_bits(k)
        c.bits[tab[:, 1]] = workloads.to_bf16_bits((3.0e38 * (0.5 + 0.5 * c.rng.random((n, D)))).astype(np.float32))
        out, lse = c.run()
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, D)
        assert out.isfinite().all() and torch.isfinite(lse).all()
    finally:
        c.close()


def test_tree_a_long_cache_and_a_large_table(L):
    """One request of 30,000 tokens, in a table whose entries pass 32-bit offsets."""
    import torch
    n, layers = 30000, 3
    max_len = (1 << 31) // (8 * layers) + 1000
    c = Tree(L, 1, 2, 64, [n], [64], seed=9)
    try:
        wide = torch.full((2, max_len, layers, 2), -1, dtype=torch.int32, device="cuda")       # 4 GB: request 1's rows lie past 2^31
        wide[1, :n, 2] = c.table[0, :n, 0]
        seq = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        st, mask, q = c.args()
        starts = torch.tensor([0, 0, 64], dtype=torch.int32, device="cuda")
        nb = L.lora_attention_tree_size(c.pool, 2, max_len, 2, 1)
        out, lse = _outputs(64, 128, 2)
        L.lora_attention_tree(c.pool, 2, wide, seq, max_len, layers, 2, starts, 64, mask, q, out, 2, 1, _workspace(nb), nb,
                              lse_dev=lse)
        L.lora_status(c.pool)
        _check(c.reference(), out, lse, 64)
    finally:
        c.close()


def test_tree_two_streams_and_a_graph(L):
    import torch
    c = Tree(L, 4, 2, 128, [500, 1033, 200], [20, 64, 1], seed=14, kinds=KINDS)
    d = Tree(L, 4, 2, 128, [90, 3600], [33, 40], seed=15, kinds=KINDS)
    try:
        want_c, want_d = c.run(), d.run()
        _check(c.reference(), *want_c, 128)
        _check(d.reference(), *want_d, 128)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        results = []
        for _ in range(5):
            with torch.cuda.stream(s1):
                results.append((c.run(stream=s1), want_c))
            with torch.cuda.stream(s2):
                results.append((d.run(stream=s2), want_d))
        torch.cuda.synchronize()
        for got, want in results:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        st, mask, q = c.args()
        out, lse = _outputs(c.rows, c.heads * c.D, c.heads)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lora_attention_tree(c.pool, 3, c.table, c.seq, c.max_len, 1, 0, st, c.rows, mask, q, out, c.heads, c.n_kv, c.ws,
                                  c.ws_bytes, lse_dev=lse)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_c[0]) and torch.equal(lse, want_c[1])
        c.seq.copy_(torch.tensor([400, 100, 150], dtype=torch.int32))          # shorter caches, other node counts
        st.copy_(torch.tensor([0, 5, 60, 85], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        tabs = [t[:n] for t, n in zip(c.tables(), (400, 100, 150))]
        _check(c.reference(kv_tables=tabs, starts=[0, 5, 60, 85]), out, lse, c.D)
        L.lora_status(c.pool)
    finally:
        c.close()
        d.close()


def test_tree_of_nothing(L):
    c = Tree(L, 1, 1, 64, [4, 9], [0, 0], seed=1, before=4)
    try:
        out, lse = c.run()
        L.lora_status(c.pool)
        assert (out == -3).all() and (lse == -7).all()
        L.lora_attention_tree(c.pool, 0, None, None, 8, 1, 0, None, 4, None, None, None, 1, 1, None, 0)
        L.lora_attention_tree(c.pool, 2, None, None, 8, 1, 0, None, 0, None, None, None, 1, 1, None, 0)
        L.lora_status(c.pool)
    finally:
        c.close()


# ---- slot maps -------------------------------------------------------------------------------
@pytest.fixture()
def small_pool(L):
    import torch
    t = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    p = L.lora_pool_create(t, 1, 64, 1, 1)
    yield p
    L.lora_pool_destroy(p)


def _append(L, pool, count, old, layers, max_len, row_cap, seed, fresh=False):
    """Runs the call and the oracle on the same inputs; returns both sides' five arrays."""
    import torch
    rng = np.random.default_rng(seed)
    n = len(count)
    pages = rng.integers(-5, 1 << 30, (row_cap, layers, 2)).astype(np.int32)
    table = rng.integers(0, 1 << 30, (n, max_len, layers, 2)).astype(np.int32)
    want = O.kv_append(count, [0] * n if fresh else old, pages, np.full_like(table, -1) if fresh else table, row_cap)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    t = dev(table)
    outs = [torch.full((m,), -99, dtype=torch.int32, device="cuda") for m in (n, n + 1, row_cap, row_cap)]
    L.lora_kv_append(pool, n, dev(np.array(count, np.int32)), None if fresh else dev(np.array(old, np.int32)), dev(pages), row_cap,
                     t, max_len, layers, *outs)
    return [x.cpu().numpy() for x in (t, *outs)], want


APPENDS = [   # requests, largest count, cached before, layers, room in the row arrays
    (1, 1, 0, 1, 0), (1, 1, 5, 3, 0), (3, 9, 4, 2, 5), (256, 1, 20, 40, 0), (257, 3, 7, 1, 1), (64, 100, 30, 2, 700),
    (5, 700, 0, 5, 3), (1000, 5, 3, 1, 9), (2, 0, 3, 4, 6), (1, 5000, 100, 1, 0), (7, 3, 2, 300, 2), (3, 2, 1, 2500, 1),
    (2600, 2, 1, 1, 4),
]


@pytest.mark.parametrize("n,hi,cached,layers,room", APPENDS)
@pytest.mark.parametrize("fresh", [False, True])
def test_append_matches_the_oracle(L, small_pool, n, hi, cached, layers, room, fresh):
    rng = np.random.default_rng(n + hi)
    count, old = rng.integers(0, hi + 1, n), rng.integers(0, cached + 1, n)
    got, want = _append(L, small_pool, count, old, layers, hi + cached + 2, int(count.sum()) + room, seed=n, fresh=fresh)
    L.lora_status(small_pool)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("count,old,max_len,row_cap", [
    ([3, -2, 4], [0, 1, 2], 9, 10), ([3, 2, 4], [0, -1, 99], 9, 10), ([3, 2, 8], [0, 1, 5], 9, 13), ([3, 2, 4], [0, 1, 2], 9, 4),
    ([3, 2, 4], [9, 9, 9], 9, 0), ([2 ** 31 - 1, 2 ** 31 - 1, 3], [0, 1, 2], 9, 20), ([-2 ** 31, 5, 2], [2 ** 31 - 1, -2 ** 31, 0], 9, 7),
])
@pytest.mark.parametrize("fresh", [False, True])
def test_append_reports_what_does_not_fit(L, small_pool, count, old, max_len, row_cap, fresh):
    got, want = _append(L, small_pool, count, old, 2, max_len, row_cap, seed=1, fresh=fresh)
    clean = fresh and count in ([3, 2, 4], [3, 2, 8]) and row_cap >= sum(count)       # the old lengths are not looked at
    if clean:
        L.lora_status(small_pool)
    else:
        with pytest.raises(L.LoraError) as e:
            L.lora_status(small_pool)
        assert e.value.code == L.LORA_EDEVICE
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_append_of_even_layers_in_unaligned_arrays(L, small_pool):
    """An even number of layers in arrays that start 8 bytes behind a 16-byte boundary."""
    import torch
    rng = np.random.default_rng(7)
    count, old, layers, max_len = [3, 0, 40, 7], [1, 2, 0, 5], 4, 50
    rows = sum(count) + 2
    pages = rng.integers(0, 99, (rows, layers, 2)).astype(np.int32)
    table = rng.integers(0, 99, (4, max_len, layers, 2)).astype(np.int32)
    want = O.kv_append(count, old, pages, table, rows)
    shifted = lambda x: torch.cat([torch.zeros(2, dtype=torch.int32), torch.from_numpy(x).view(-1)]).cuda()[2:]  # noqa: E731
    t, p = shifted(table), shifted(pages)
    assert t.data_ptr() % 16 == 8
    outs = [torch.full((m,), -99, dtype=torch.int32, device="cuda") for m in (4, 5, rows, rows)]
    as_dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    L.lora_kv_append(small_pool, 4, as_dev(count), as_dev(old), p, rows, t, max_len, layers, *outs)
    L.lora_status(small_pool)
    for g, w in zip((t.view(table.shape), *outs), want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_append_many_requests(L, small_pool):
    """65,535 requests, most of them with nothing new."""
    rng = np.random.default_rng(3)
    count = np.where(rng.random(65535) < 0.01, rng.integers(1, 5, 65535), 0)
    old = rng.integers(0, 4, 65535)
    for fresh in (False, True):
        got, want = _append(L, small_pool, count, old, 1, 8, int(count.sum()) + 3, seed=2, fresh=fresh)
        L.lora_status(small_pool)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)


def test_append_of_nothing(L, small_pool):
    import torch
    start = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    L.lora_kv_append(small_pool, 0, None, None, None, 0, None, 4, 2, None, start, None, None)
    assert start.item() == 0
    req, pos = (torch.full((3,), 5, dtype=torch.int32, device="cuda") for _ in range(2))
    L.lora_kv_append(small_pool, 0, None, None, torch.zeros((3, 2, 2), dtype=torch.int32, device="cuda"), 3, None, 4, 2, None,
                     start, req, pos)
    assert (req == -1).all() and (pos == 0).all()
    L.lora_status(small_pool)
