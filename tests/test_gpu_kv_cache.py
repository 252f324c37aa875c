"""KV-cache operators on the GPU: page writes, split decode attention with token weights, eviction.

Attention is compared with the fp64 oracle under bounds that follow from the arithmetic (bf16
inputs, fp32 sums, weights held in two bf16 terms, one bf16 rounding of the output); page writes and
evictions have to be exact."""
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


class Cache:
    """KV pages of some requests in a shuffled pool whose other pages hold NaN, with their table."""

    def __init__(self, L, H, layers, lengths, seed, scale=1.0, room=3, max_len=None):
        import torch
        self.L, self.H, self.layers, self.lengths = L, H, layers, list(lengths)
        rng = self.rng = np.random.default_rng(seed)
        need = 2 * layers * sum(lengths)
        self.num_pages = need + 64
        order = rng.permutation(self.num_pages)
        self.pool_t = torch.full((self.num_pages, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pool = L.lora_pool_create(self.pool_t, self.num_pages, H, 1, 1, order)
        self.bits = np.full((self.num_pages, H), 0x7FC0, np.uint16)
        self.n_req, self.max_len = len(lengths), max_len or max(list(lengths) + [0]) + room
        for r, n in enumerate(lengths):
            ids = L.lora_kv_grow(self.pool, r, n, layers)
            if ids:
                self.bits[ids] = workloads.to_bf16_bits(scale * rng.standard_normal((len(ids), H)).astype(np.float32))
        self.pool_t.copy_(bits_to_torch(self.bits))
        self.table = torch.empty((self.n_req, self.max_len, layers, 2), dtype=torch.int32, device="cuda")
        self.seq = torch.empty(self.n_req, dtype=torch.int32, device="cuda")
        if self.n_req:
            L.lora_kv_batch_table(self.pool, list(range(self.n_req)), self.max_len, self.table, self.seq)

    def tables(self, layer):
        return [self.L.lora_kv_table(self.pool, r, layer).astype(np.int64) for r in range(self.n_req)]

    def workspace(self, n_heads, n_kv, weights):
        import torch
        n = self.L.lora_attention_split_size(self.pool, self.n_req, self.max_len, n_heads, n_kv, weights)
        return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda"), n     # NaN patterns everywhere

    def close(self):
        self.L.lora_pool_destroy(self.pool)


def _check(ref, out, lse, lengths, D, G):
    tol_out, tol_lse, _ = attention_tolerances(ref, lengths, D)
    got = O.bf16_to_f64(torch_to_bits(out.contiguous()))
    assert np.isfinite(got).all()
    bad = np.abs(got - ref["out"]) > tol_out
    assert not bad.any(), f"{int(bad.sum())} outputs, first at {np.argwhere(bad)[0]}"
    if lse is not None:
        got = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(got), empty)
        err = np.abs(np.where(empty, 0, got) - np.where(empty, 0, ref["lse"]))
        assert (err <= tol_lse).all(), err.max()


def _check_weights(ref, got, w_in, lengths, D, G, n_heads):
    _, _, tol_w = attention_tolerances(ref, lengths, D)
    for i, n in enumerate(lengths):
        want = ref["weight"][i] + (0 if w_in is None else w_in[i, :n])
        err = np.abs(got[i, :n] - want)
        assert (err <= tol_w[i] + 2.0 ** -24 * (n_heads + 2) * np.abs(want) + n_heads * 2.0 ** -126).all(), (i, err.max())


SHAPES = [   # n_kv, G, D, layers, lengths
    (2, 1, 128, 2, [1, 5, 0, 33, 7]),
    (4, 4, 64, 1, [16, 17, 31, 32, 129]),
    (1, 16, 256, 1, [300, 0, 1]),
    (1, 1, 64, 1, [513, 2]),
    (8, 2, 128, 3, [1000, 1, 64]),
    (5, 3, 128, 1, [77, 4096]),
    (12, 1, 64, 1, [15, 130]),
    (9, 9, 128, 1, [127, 1, 128]),
    (40, 1, 128, 1, [20, 200, 3]),
    (1, 8, 64, 1, [20001]),
    (2, 5, 256, 2, [700, 699]),
    (6, 1, 256, 1, [47, 90]),
    (64, 1, 256, 1, [33, 18]),          # H = 16384
    (128, 2, 128, 1, [9, 40]),
    (3, 7, 128, 1, [0, 0, 0]),
    (8, 1, 128, 1, [3, 0, 1, 40] * 170),
    (1, 2, 128, 1, [1] * 3000),
    (16, 3, 64, 1, [90, 1, 257]),       # two heads of 64 a warp: 8 of 8, 7 + 6, 8 with 9 query heads each
    (13, 1, 64, 2, [45, 700]),
    (8, 9, 64, 1, [33, 64, 0, 400]),
    (4, 12, 64, 1, [50, 333]),          # 8 + 4 query heads on two warps, each with two heads of 64
    (3, 11, 256, 1, [40, 1, 100]),
    (2, 16, 128, 1, [1000, 17]),
    (8, 1, 128, 1, [61, 0, 16, 1]),     # one CTA per request and head group: D = 128, 64, 256, several warps a head
    (8, 2, 64, 1, [60, 33]),
    (4, 3, 256, 1, [17, 61, 48]),
    (1, 1, 128, 1, [61, 2]),
    (1, 16, 64, 1, [5000, 33, 31]),     # rows of up to 384 bytes: tiles of one head on four warps, two or one
    (1, 9, 64, 2, [129, 0, 127, 16, 17, 128]),
    (2, 3, 64, 1, [1, 0, 700, 64, 63, 65]),
    (2, 12, 64, 1, [300] * 30),
    (3, 1, 64, 1, [31, 33, 6000]),
    (3, 16, 64, 1, [32, 0, 900]),
    (1, 7, 128, 2, [64, 65, 2000, 0, 63]),
    (1, 16, 128, 1, [1, 47, 3000]),
    (1, 10, 64, 1, [61, 1, 32, 33, 0, 17]),   # whole requests of such rows
    (3, 2, 64, 1, [5, 61, 0]),
    (1, 12, 128, 1, [60, 17, 0, 48]),
    (1, 3, 64, 1, [3, 0, 90] * 100),
    (2, 16, 256, 1, [9000]),            # few heads with many partials each
    (1, 2, 128, 1, [7000, 40]),
    (5, 1, 64, 1, [0, 5000, 0]),
    (1, 3, 256, 1, [2600]),
    (1, 8, 256, 2, [700, 63, 0, 65]),   # eight and nine heads: tokens' weights by a warp, by all
    (3, 3, 128, 1, [1, 127, 700]),
    (2, 4, 128, 1, [2 * 64 + 1] * 40),
    (3, 2, 128, 1, [129] * 130),        # more than 128 requests: the range search goes through shared memory
]


@pytest.mark.parametrize("n_kv,G,D,layers,lengths", SHAPES)
def test_attention_split_matches_the_oracle(L, n_kv, G, D, layers, lengths):
    import torch
    n_heads, H = n_kv * G, n_kv * D
    c = Cache(L, H, layers, lengths, seed=H + G)
    try:
        n_req = c.n_req
        for layer in range(layers):
            q_bits = workloads.to_bf16_bits(c.rng.standard_normal((n_req, n_heads * D)).astype(np.float32))
            ref = O.attention_split(c.bits, c.tables(layer), q_bits, n_heads, n_kv)
            q = bits_to_torch(q_bits)
            out = torch.full_like(q, float("nan"))
            lse = torch.full((n_req, n_heads), float("nan"), device="cuda")
            ws, nb = c.workspace(n_heads, n_kv, False)
            L.lora_attention_split(c.pool, n_req, c.table, c.seq, c.max_len, layers, layer, q, out, n_heads, n_kv, ws,
                                   nb, lse_dev=lse)
            L.lora_status(c.pool)
            _check(ref, out, lse, lengths, D, G)
            # with weights: the same output and log-sum-exp, and the weights on top of earlier ones
            w_in = c.rng.random((n_req, c.max_len)).astype(np.float32)
            w_out = torch.full((n_req, c.max_len), -7.0, device="cuda")
            ws, nb = c.workspace(n_heads, n_kv, True)
            out2, lse2 = torch.full_like(q, float("nan")), torch.full_like(lse, float("nan"))
            L.lora_attention_split(c.pool, n_req, c.table, c.seq, c.max_len, layers, layer, q, out2, n_heads, n_kv, ws,
                                   nb, lse_dev=lse2, weight_in_dev=torch.from_numpy(w_in).cuda(), weight_out_dev=w_out)
            L.lora_status(c.pool)
            assert torch.equal(out, out2) and torch.equal(lse, lse2)
            got = w_out.cpu().numpy().astype(np.float64)
            _check_weights(ref, got, w_in.astype(np.float64), lengths, D, G, n_heads)
            for i, n in enumerate(lengths):
                assert (got[i, n:] == -7.0).all()                # past the length: not touched
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,lengths", [
    (2, 1, [300, 0, 1, 33]), (2, 8, [16, 2000, 64, 65]), (2, 9, [100, 31]), (3, 1, [900, 17, 0]), (3, 16, [5, 128]),
])
def test_attention_split_of_a_large_cache_with_short_requests(L, n_kv, G, lengths):
    """max_len says that the cache is large, so that heads of 64 are read together."""
    import torch
    D = 64
    n_heads, H, n_req = n_kv * G, 64 * n_kv, len(lengths)
    max_len = (400 << 20) // (4 * H * n_req) + 1
    c = Cache(L, H, 1, lengths, seed=H + G, max_len=max_len)
    try:
        tabs = c.tables(0)
        c.table[0, 3, 0, 1] = c.num_pages                      # a bad page: its token is skipped
        keep = np.setdiff1d(np.arange(lengths[0]), [3])
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((n_req, n_heads * D)).astype(np.float32))
        ref = O.attention_split(c.bits, [tabs[0][keep]] + tabs[1:], q_bits, n_heads, n_kv)
        q = bits_to_torch(q_bits)
        out = torch.full_like(q, float("nan"))
        lse = torch.full((n_req, n_heads), float("nan"), device="cuda")
        w = torch.zeros((n_req, max_len), device="cuda")
        ws, nb = c.workspace(n_heads, n_kv, True)
        L.lora_attention_split(c.pool, n_req, c.table, c.seq, max_len, 1, 0, q, out, n_heads, n_kv, ws, nb, lse_dev=lse,
                               weight_out_dev=w)
        with pytest.raises(L.LoraError) as e:
            L.lora_status(c.pool)
        assert e.value.code == L.LORA_EDEVICE
        n_tok = [len(keep)] + lengths[1:]
        _check(ref, out, lse, n_tok, D, G)
        got = w[:, :max(lengths)].cpu().numpy().astype(np.float64)
        got[0, :len(keep)] = got[0, keep]
        _check_weights(ref, got, None, n_tok, D, G, n_heads)
    finally:
        c.close()


def test_attention_split_strides_in_place_weights_and_no_lse(L):
    import torch
    n_kv, G, D, lengths = 4, 2, 64, [100, 0, 333, 16]
    n_heads, width = n_kv * G, n_kv * G * D
    c = Cache(L, n_kv * D, 2, lengths, seed=2)
    try:
        wide = torch.full((4, width + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((4, width)).astype(np.float32))
        wide[:, 8:8 + width] = bits_to_torch(q_bits)
        out = torch.full((4, width + 16), -3.0, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros((4, c.max_len + 5), device="cuda")
        ws, nb = c.workspace(n_heads, n_kv, True)
        ref = O.attention_split(c.bits, c.tables(1), q_bits, n_heads, n_kv)
        for _ in range(2):
            L.lora_attention_split(c.pool, 4, c.table, c.seq, c.max_len, 2, 1, wide[:, 8:], out, n_heads, n_kv, ws, nb,
                                   weight_in_dev=w, weight_out_dev=w, weight_stride=c.max_len + 5,
                                   q_stride=width + 72, out_stride=width + 16)
        L.lora_status(c.pool)
        _check(ref, out[:, :width], None, lengths, D, G)
        assert (out[:, width:] == -3.0).all()
        got = w.cpu().numpy().astype(np.float64)
        twice = {**ref, "weight": [2 * x for x in ref["weight"]], "p": [2 * x for x in ref["p"]]}
        _check_weights(twice, got, None, lengths, D, G, 2 * n_heads)
        # without earlier weights the sum starts at zero
        first = torch.full_like(w, 9.0)
        L.lora_attention_split(c.pool, 4, c.table, c.seq, c.max_len, 2, 1, wide[:, 8:], out, n_heads, n_kv, ws, nb,
                               weight_out_dev=first, weight_stride=c.max_len + 5, q_stride=width + 72,
                               out_stride=width + 16)
        _check_weights(ref, first.cpu().numpy().astype(np.float64), None, lengths, D, G, n_heads)
    finally:
        c.close()


@pytest.mark.parametrize("scale,shift", [(30.0, 0.0), (1e-3, 0.0), (1.0, 200.0)])
def test_attention_split_far_scores(L, scale, shift):
    """Scores of hundreds (one token takes everything), of nothing, and with a late maximum."""
    import torch
    n_kv, D, lengths = 2, 128, [700, 45]
    c = Cache(L, 256, 1, lengths, seed=11, scale=scale)
    try:
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((2, 256)).astype(np.float32))
        if shift:                                                # the last token's K along q
            for r in range(2):
                k_page = c.tables(0)[r][-1, 0]
                qf = O.bf16_to_f64(q_bits[r]).reshape(2, 128)
                k = (qf * shift * np.sqrt(128) / (qf ** 2).sum(1, keepdims=True)).reshape(-1)
                c.bits[k_page] = workloads.to_bf16_bits(k.astype(np.float32))
            c.pool_t.copy_(bits_to_torch(c.bits))
        ref = O.attention_split(c.bits, c.tables(0), q_bits, 2, 2)
        q, out = bits_to_torch(q_bits), torch.empty((2, 256), dtype=torch.bfloat16, device="cuda")
        lse, w = torch.empty((2, 2), device="cuda"), torch.zeros((2, c.max_len), device="cuda")
        ws, nb = c.workspace(2, 2, True)
        L.lora_attention_split(c.pool, 2, c.table, c.seq, c.max_len, 1, 0, q, out, 2, 2, ws, nb, lse_dev=lse,
                               weight_out_dev=w)
        L.lora_status(c.pool)
        _check(ref, out, lse, lengths, D, 1)
        _check_weights(ref, w.cpu().numpy().astype(np.float64), None, lengths, D, 1, 2)
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D", [(2, 2, 128), (1, 9, 64), (3, 2, 64), (1, 3, 128)])
def test_attention_split_skips_bad_pages_and_clamps_lengths(L, n_kv, G, D):
    import torch
    lengths, n_heads, width = [50, 3, 20], n_kv * G, n_kv * G * D
    c = Cache(L, n_kv * D, 1, lengths, seed=4)
    try:
        tabs = c.tables(0)
        drop = {0: [0, 17, 49], 1: [0, 1, 2], 2: []}
        for r, js in drop.items():
            for i, j in enumerate(js):
                c.table[r, j, 0, i % 2] = (1 << 30) if i != 1 else -5
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((3, width)).astype(np.float32))
        keep = [np.setdiff1d(np.arange(n), drop[r]) for r, n in enumerate(lengths)]
        ref = O.attention_split(c.bits, [tabs[r][keep[r]] for r in range(3)], q_bits, n_heads, n_kv)
        q, out = bits_to_torch(q_bits), torch.empty((3, width), dtype=torch.bfloat16, device="cuda")
        lse, w = torch.empty((3, n_heads), device="cuda"), torch.full((3, c.max_len), 5.0, device="cuda")
        ws, nb = c.workspace(n_heads, n_kv, True)
        args = (c.pool, 3, c.table, c.seq, c.max_len, 1, 0, q, out, n_heads, n_kv, ws, nb)
        L.lora_attention_split(*args, lse_dev=lse, weight_out_dev=w)
        with pytest.raises(L.LoraError) as e:
            L.lora_status(c.pool)
        assert e.value.code == L.LORA_EDEVICE and "page" in e.value.message
        _check(ref, out, lse, [len(k) for k in keep], D, G)
        got = w.cpu().numpy().astype(np.float64)
        for r, js in drop.items():
            assert (got[r, js] == 0).all()
        _check_weights(ref, np.stack([np.pad(got[r, keep[r]], (0, c.max_len - len(keep[r]))) for r in range(3)]), None,
                       [len(k) for k in keep], D, G, n_heads)
        # lengths outside [0, max_len]: reported and clamped
        c.seq.copy_(torch.tensor([-3, 3, 20], dtype=torch.int32))
        L.lora_attention_split(*args, lse_dev=lse)
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
        c.seq.copy_(torch.tensor([c.max_len + 1, 0, 0], dtype=torch.int32))     # the tail of row 0 holds -1 pages
        L.lora_attention_split(*args, lse_dev=lse)
        with pytest.raises(L.LoraError):
            L.lora_status(c.pool)
        _check({k: v[:1] for k, v in ref.items()}, out[:1], lse[:1], [len(keep[0])], D, G)
    finally:
        c.close()


def test_attention_split_overflowing_scores_and_infinite_values(L):
    """A score of -infinity takes no weight; rows whose every score is -infinity count as empty."""
    import torch
    c = Cache(L, 128, 1, [40, 21], seed=8)
    try:
        big = workloads.to_bf16_bits(np.float32([3e38]))[0]
        neg = workloads.to_bf16_bits(np.float32([-3e38]))[0]
        tabs = c.tables(0)
        q_bits = np.full((2, 128), workloads.to_bf16_bits(np.float32([1.0]))[0], np.uint16)
        q_bits[:, 0] = big
        c.bits[tabs[0][7, 0], 0] = neg                             # request 0, token 7: -infinity
        for j in range(40):
            if j != 7:
                c.bits[tabs[0][j, 0], 0] = 0
        c.bits[tabs[1][:, 0], 0] = neg                             # request 1: every score
        c.pool_t.copy_(bits_to_torch(c.bits))
        keep = np.setdiff1d(np.arange(40), [7])
        ref = O.attention_split(c.bits, [tabs[0][keep], tabs[1][:0]], q_bits, 1, 1)
        q, out = bits_to_torch(q_bits), torch.empty((2, 128), dtype=torch.bfloat16, device="cuda")
        lse, w = torch.empty((2, 1), device="cuda"), torch.full((2, c.max_len), 5.0, device="cuda")
        ws, nb = c.workspace(1, 1, True)
        L.lora_attention_split(c.pool, 2, c.table, c.seq, c.max_len, 1, 0, q, out, 1, 1, ws, nb, lse_dev=lse,
                               weight_out_dev=w)
        L.lora_status(c.pool)
        _check(ref, out, lse, [39, 0], 128, 1)
        got = w.cpu().numpy()
        assert got[0, 7] == 0 and (got[1, :21] == 0).all() and abs(got[0, :40].sum() - 1) < 1e-5
    finally:
        c.close()


def test_attention_split_nan_stays_in_its_own_heads(L):
    """A NaN in one KV head of one token spoils that head's query heads of that request, no others."""
    import torch
    n_kv, G, D = 2, 2, 64
    c = Cache(L, 128, 1, [30, 200], seed=9)
    try:
        tabs = c.tables(0)
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((2, 256)).astype(np.float32))
        ref = O.attention_split(c.bits, tabs, q_bits, 4, 2)
        c.bits[tabs[1][150, 0], 64 + 3] = 0x7FC0                   # K of token 150, KV head 1
        c.pool_t.copy_(bits_to_torch(c.bits))
        q, out = bits_to_torch(q_bits), torch.empty((2, 256), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((2, 4), device="cuda")
        ws, nb = c.workspace(4, 2, False)
        L.lora_attention_split(c.pool, 2, c.table, c.seq, c.max_len, 1, 0, q, out, 4, 2, ws, nb, lse_dev=lse)
        assert torch.isnan(out[1, 128:]).all() and torch.isnan(lse[1, 2:]).all()
        _check({k: v[:1] for k, v in ref.items()}, out[:1], lse[:1], [30], D, G)
        half = {k: ref[k][1:, :n] for k, n in (("out", 128), ("vabs", 128), ("lse", 2), ("mag", 2))}
        half["p"] = [ref["p"][1][:2]]
        _check(half, out[1:, :128], lse[1:, :2], [200], D, G)
    finally:
        c.close()


def test_attention_split_same_bits_again_on_a_side_stream_and_in_a_graph(L):
    import torch
    n_kv, G, D, lengths = 8, 1, 128, [5000, 3, 0, 260, 1]
    c = Cache(L, 1024, 1, lengths, seed=6)
    try:
        q = bits_to_torch(workloads.to_bf16_bits(c.rng.standard_normal((5, 1024)).astype(np.float32)))
        ws, nb = c.workspace(8, 8, True)

        def call(out, lse, w, stream=None):
            L.lora_attention_split(c.pool, 5, c.table, c.seq, c.max_len, 1, 0, q, out, 8, 8, ws, nb, lse_dev=lse,
                                   weight_out_dev=w, stream=stream)

        def bufs():
            return torch.empty_like(q), torch.empty((5, 8), device="cuda"), torch.zeros((5, c.max_len), device="cuda")
        first = bufs()
        call(*first)
        for _ in range(3):
            again = bufs()
            call(*again)
            assert all(torch.equal(a, b) for a, b in zip(first, again))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = bufs()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(*other)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, other))
        held = bufs()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*held)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
        # replayed on other lengths: what an eager call computes
        c.seq.copy_(torch.tensor([77, 2, 0, 0, 1], dtype=torch.int32))
        fresh = bufs()
        call(*fresh)
        for b in held:
            b.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(fresh, held))
        L.lora_status(c.pool)
    finally:
        c.close()


def test_attention_split_of_sixty_thousand_requests(L):
    """One token each (or none): the output is its V, the weight one per query head."""
    import torch
    n, H = 60_000, 64
    pool_t = torch.randn((2 * n, H), device="cuda").bfloat16()
    pool = L.lora_pool_create(pool_t, 2 * n, H, 1, 1)
    try:
        for max_len in (1, 200):
            table = torch.full((n, max_len, 1, 2), -1, dtype=torch.int32, device="cuda")
            pages = torch.randperm(2 * n, device="cuda").to(torch.int32).view(n, 2)
            table[:, 0, 0] = pages
            seq = (torch.arange(n, device="cuda") % 7 != 3).to(torch.int32)
            q = torch.randn((n, 2 * H), device="cuda").bfloat16()
            out, w = torch.full_like(q, float("nan")), torch.full((n, max_len), -1.0, device="cuda")
            nb = L.lora_attention_split_size(pool, n, max_len, 2, 1, True)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            L.lora_attention_split(pool, n, table, seq, max_len, 1, 0, q, out, 2, 1, ws, nb, weight_out_dev=w)
            L.lora_status(pool)
            v = pool_t[pages[:, 1].long()] * seq[:, None].to(torch.bfloat16)
            assert torch.equal(out, torch.cat([v, v], 1))
            assert torch.equal(w[:, 0], torch.where(seq > 0, 2.0, -1.0))
    finally:
        L.lora_pool_destroy(pool)


def test_attention_split_does_not_depend_on_the_other_requests_values(L):
    """A request's result stays the same when another request's rows and query change."""
    import torch
    c = Cache(L, 256, 1, [900, 37, 2500], seed=12)
    try:
        q = bits_to_torch(workloads.to_bf16_bits(c.rng.standard_normal((3, 256)).astype(np.float32)))
        ws, nb = c.workspace(2, 2, False)
        outs = []
        for _ in range(2):
            out = torch.empty_like(q)
            L.lora_attention_split(c.pool, 3, c.table, c.seq, c.max_len, 1, 0, q, out, 2, 2, ws, nb)
            outs.append(out)
            q[1] = -q[1]
            c.pool_t[torch.from_numpy(c.tables(0)[1].reshape(-1)).cuda()] = 3.0
        assert torch.equal(outs[0][[0, 2]], outs[1][[0, 2]]) and not torch.equal(outs[0][1], outs[1][1])
    finally:
        c.close()


def test_attention_split_on_two_streams_at_once(L):
    """Calls with workspaces of their own may overlap: each gives what it gives alone."""
    import torch
    c = Cache(L, 512, 1, [3000, 0, 700, 65], seed=31)
    try:
        qs = [bits_to_torch(workloads.to_bf16_bits(c.rng.standard_normal((4, 1024)).astype(np.float32))) for _ in range(2)]
        spaces = [c.workspace(8, 4, True) for _ in range(2)]

        def call(i, out, w, stream=None):
            L.lora_attention_split(c.pool, 4, c.table, c.seq, c.max_len, 1, 0, qs[i], out, 8, 4, *spaces[i],
                                   weight_out_dev=w, stream=stream)
        alone = [(torch.empty_like(q), torch.zeros((4, c.max_len), device="cuda")) for q in qs]
        for i in range(2):
            call(i, *alone[i])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        both = [(torch.empty_like(q), torch.zeros((4, c.max_len), device="cuda")) for q in qs]
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                call(i, *both[i], stream=streams[i])
        torch.cuda.synchronize()
        L.lora_status(c.pool)
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    finally:
        c.close()


def _attend(L, c, q, n_heads, n_kv, layer=0):
    """One call with log-sum-exp and token weights: (out, lse, weights)."""
    import torch
    out = torch.full_like(q, 7.0)
    lse = torch.full((c.n_req, n_heads), 7.0, device="cuda")
    w = torch.zeros((c.n_req, c.max_len), device="cuda")
    ws, nb = c.workspace(n_heads, n_kv, True)
    L.lora_attention_split(c.pool, c.n_req, c.table, c.seq, c.max_len, c.layers, layer, q, out, n_heads, n_kv, ws, nb,
                           lse_dev=lse, weight_out_dev=w)
    L.lora_status(c.pool)
    return out, lse, w.cpu().numpy().astype(np.float64)


# Shapes of every form: rows read directly (one warp a head, several, two heads a warp in a cache that max_len
# calls large), copied stages of each head width, requests taken whole and split.
FORMS = [
    (1, 1, 64, [1, 2, 33, 700], None), (1, 12, 64, [5, 300], None), (3, 2, 64, [1, 40, 129], None),
    (2, 3, 64, [17, 260], 1 << 20), (3, 1, 64, [90, 2], 1 << 20), (1, 3, 128, [1, 64, 999], None),
    (1, 9, 128, [3, 61], None), (8, 1, 128, [1, 5, 60], None), (8, 2, 128, [900, 1, 64], None),
    (4, 12, 64, [50, 333], None), (13, 1, 64, [45, 700], None), (6, 2, 256, [47, 1, 90], None),
    (1, 16, 256, [300, 2], None), (1, 1, 64, [20001], None), (4, 1, 128, [9000], None),
]


@pytest.mark.parametrize("n_kv,G,D,lengths,max_len", FORMS)
def test_attention_split_infinite_values(L, n_kv, G, D, lengths, max_len):
    """A weight times an infinite V is that infinity, whatever the weight's bits; V of both signs gives NaN; the
    other features, and the weights, stay what they are."""
    n_heads, H = n_kv * G, n_kv * D
    c = Cache(L, H, 1, lengths, seed=H + G, max_len=max_len)
    try:
        n_req, tabs, inf = c.n_req, c.tables(0), 0x7F80
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((n_req, n_heads * D)).astype(np.float32))
        want = np.zeros((n_req, n_heads, D))                       # infinities; the rest from the oracle
        for r, n in enumerate(lengths):
            a, b, third = c.rng.integers(0, n), c.rng.integers(0, n), n - 1
            v = c.bits[tabs[r][:, 1]].reshape(n, n_kv, D)
            v[:, :, :4] = workloads.to_bf16_bits(np.float32([0.0]))[0]
            v[a, :, 0], v[b, :, 1] = inf, inf | 0x8000
            v[third, :, 2], v[:, :, 3] = inf, inf
            if n > 1:
                v[0, :, 2] = inf | 0x8000
            c.bits[tabs[r][:, 1]] = v.reshape(n, H)
            want[r, :, 0], want[r, :, 1], want[r, :, 3] = np.inf, -np.inf, np.inf
            want[r, :, 2] = np.nan if n > 1 else np.inf
        c.pool_t.copy_(bits_to_torch(c.bits))
        finite = c.bits.copy()
        finite[(finite & 0x7FFF) == inf] = 0
        ref = O.attention_split(finite, tabs, q_bits, n_heads, n_kv)
        out, lse, w = _attend(L, c, bits_to_torch(q_bits), n_heads, n_kv)
        got = out.float().cpu().numpy().reshape(n_req, n_heads, D)
        assert np.array_equal(got[:, :, :4], want[:, :, :4], equal_nan=True)
        out.view(n_req, n_heads, D)[:, :, :4] = 0
        _check(ref, out, lse, lengths, D, G)
        _check_weights(ref, w[:, :max(lengths)], None, lengths, D, G, n_heads)
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D,n", [(4, 1, 128, 6), (1, 2, 64, 5), (3, 1, 64, 8), (1, 1, 128, 7), (2, 1, 256, 6),
                                        (8, 3, 64, 4), (1, 12, 64, 6)])
def test_attention_split_weights_reach_the_product_in_full(L, n_kv, G, D, n):
    """V whose last three rows cancel the others, so that what is left of an output is what the weights lost.

    One coordinate of q is not zero, so a score is one exact product q K, times log2(e) / sqrt(D) (itself off by 2 u):
    with |s| <= 0.36 in base 2, s and m are off by 1.1 u each and their difference by another 0.4 u, a weight by
    ln(2) 2.6 u and by exp2's two ulps, 4 u: 6 u in all.  The normaliser adds n sums, 6 u of its own and two
    roundings, the V product one rounding (or cut, 2 u) per term and one of the scaling, 8 u, the last product u:
    (n + 24) u of sum p |V|.  Weights of 16 bits would be off by 2^-17, 128 u, each."""
    n_heads, H, n_req = n_kv * G, n_kv * D, 24
    c = Cache(L, H, 1, [n] * n_req, seed=n + H)
    try:
        tabs, rng = c.tables(0), c.rng
        one = workloads.to_bf16_bits(np.float32([1.0]))[0]
        q_bits = np.zeros((n_req, n_heads, D), np.uint16)
        q_bits[:, :, 5] = one
        for r in range(n_req):
            k = rng.standard_normal((n, n_kv, D)).astype(np.float32)
            k[:, :, 5] = rng.uniform(-0.25, 0.25, (n, n_kv)) * np.sqrt(D)
            k_bits = workloads.to_bf16_bits(k.reshape(n, H))
            p = np.exp(O.bf16_to_f64(k_bits).reshape(n, n_kv, D)[:, :, 5] / np.sqrt(D))
            v = np.zeros((n, n_kv, D))
            for j in range(n):                                     # each of the last three cancels what is there
                x = rng.standard_normal((n_kv, D)) if j < n - 3 else -(p[:j, :, None] * v[:j]).sum(0) / p[j][:, None]
                v[j] = O.bf16_to_f64(workloads.to_bf16_bits(x.astype(np.float32)))
            c.bits[tabs[r][:, 0]], c.bits[tabs[r][:, 1]] = k_bits, workloads.to_bf16_bits(v.reshape(n, H).astype(np.float32))
        c.pool_t.copy_(bits_to_torch(c.bits))
        q_bits = q_bits.reshape(n_req, -1)
        ref = O.attention_split(c.bits, tabs, q_bits, n_heads, n_kv)
        out, _, _ = _attend(L, c, bits_to_torch(q_bits), n_heads, n_kv)
        got = O.bf16_to_f64(torch_to_bits(out))
        tol = 2.0 ** -8 * np.abs(ref["out"]) + (n + 24) * 2.0 ** -24 * ref["vabs"] * 1.01
        bad = np.abs(got - ref["out"]) > tol
        assert not bad.any(), (int(bad.sum()), (np.abs(got - ref["out"]) / tol).max())
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,G,D,lengths", [
    (4, 1, 128, [60] * 8), (16, 2, 64, [60] * 3), (4, 1, 256, [60] * 2), (3, 1, 64, [2000] * 30), (8, 2, 128, [500] * 40),
])
def test_attention_split_large_values_under_late_scores(L, n_kv, G, D, lengths):
    """Scores 5.4 higher in a request's second half, 221 times the weight.  Weights relative to the largest are at
    most 1 and their sum times |V| stays below 2^127, so no sum may overflow."""
    n_heads, H = n_kv * G, n_kv * D
    c = Cache(L, H, 1, lengths, seed=H + G)
    try:
        n_req, tabs = c.n_req, c.tables(0)
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((n_req, n_heads * D)).astype(np.float32))
        q = O.bf16_to_f64(q_bits).reshape(n_req, n_kv, G, D)[:, :, 0]
        high = (5.4 * np.sqrt(D) * q / (q ** 2).sum(-1, keepdims=True)).reshape(n_req, H)
        top = 126 - int(np.ceil(np.log2(2 * max(lengths))))
        for r, n in enumerate(lengths):
            k = np.where(np.arange(n)[:, None] < n // 2, 0.0, high[r])
            v = np.minimum(np.abs(c.rng.standard_normal((n, H))), 4.0) * 2.0 ** top
            c.bits[tabs[r][:, 0]] = workloads.to_bf16_bits(k.astype(np.float32))
            c.bits[tabs[r][:, 1]] = workloads.to_bf16_bits(v.astype(np.float32))
        c.pool_t.copy_(bits_to_torch(c.bits))
        ref = O.attention_split(c.bits, tabs, q_bits, n_heads, n_kv)
        out, lse, w = _attend(L, c, bits_to_torch(q_bits), n_heads, n_kv)
        _check(ref, out, lse, lengths, D, G)
        _check_weights(ref, w, None, lengths, D, G, n_heads)
    finally:
        c.close()


@pytest.mark.parametrize("n_kv,D", [(4, 128), (8, 64), (3, 64)])
def test_attention_split_sums_round_once_a_tile(L, n_kv, D):
    """Sums that climb over most of a long request and fall back to nothing, so that what the roundings on the way
    left is what is left of an output.  The shapes let one warp take a head's 16-token tiles in their order.

    The first token has the largest score, so the sum S_t after tile t is relative to it throughout, and each
    addition of a tile rounds to within u |S_t| (u = 2^-24).  Besides, a weight is off by 7 u (scores as in the
    test of the weights in full, |s| <= 0.72 in base 2), a tile's three terms by a rounding or cut of 2 u each,
    and the join of a request that is cut in two by a few: 20 u of sum p |V| in all."""
    import torch
    H, n, u = n_kv * D, 6400, 2.0 ** -24
    n_req = 2 * torch.cuda.get_device_properties(0).multi_processor_count     # as many as there are ranges
    c = Cache(L, H, 1, [n], seed=H)
    try:
        rng, tab = c.rng, c.tables(0)[0]
        k = rng.standard_normal((n, n_kv, D)).astype(np.float32)
        k[:, :, 5] = rng.uniform(-0.25, 0.25, (n, n_kv)) * np.sqrt(D)
        k[0, :, 5] = 0.5 * np.sqrt(D)
        k_bits = workloads.to_bf16_bits(k.reshape(n, H))
        s = O.bf16_to_f64(k_bits).reshape(n, n_kv, D)[:, :, 5] / np.sqrt(D)
        p = np.exp(s - s[0])[:, :, None]
        v = rng.uniform(1, 2, (n, n_kv, D))
        v[n * 3 // 4:] *= -3
        v *= np.where(rng.random((n_kv, D)) < 0.5, 1, -1)
        v = O.bf16_to_f64(workloads.to_bf16_bits(v.astype(np.float32)))
        for j in range(n - 3, n):
            v[j] = O.bf16_to_f64(workloads.to_bf16_bits((-(p[:j] * v[:j]).sum(0) / p[j]).astype(np.float32)))
        c.bits[tab[:, 0]], c.bits[tab[:, 1]] = k_bits, workloads.to_bf16_bits(v.reshape(n, H).astype(np.float32))
        c.pool_t.copy_(bits_to_torch(c.bits))
        q_bits = np.zeros((1, n_kv, D), np.uint16)
        q_bits[:, :, 5] = workloads.to_bf16_bits(np.float32([1.0]))[0]
        ref = O.attention_split(c.bits, [tab], q_bits.reshape(1, H), n_kv, n_kv)
        climbs = np.abs(np.cumsum(p * v, axis=0)[15::16]).sum(0) / p.sum(0)
        tol = 2.0 ** -8 * np.abs(ref["out"]) + u * climbs.reshape(1, H) + 20 * u * ref["vabs"]
        # every request is the same tokens
        table = c.table.expand(n_req, -1, -1, -1).contiguous()
        seq = c.seq.expand(n_req).contiguous()
        q = bits_to_torch(np.repeat(q_bits.reshape(1, H), n_req, axis=0))
        out = torch.empty_like(q)
        nb = L.lora_attention_split_size(c.pool, n_req, c.max_len, n_kv, n_kv)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        L.lora_attention_split(c.pool, n_req, table, seq, c.max_len, 1, 0, q, out, n_kv, n_kv, ws, nb)
        L.lora_status(c.pool)
        err = np.abs(O.bf16_to_f64(torch_to_bits(out)) - ref["out"])
        assert (err <= tol).all(), (int((err > tol).sum()), (err / tol).max())
    finally:
        c.close()


# ---- page writes ---------------------------------------------------------------------------------
@pytest.mark.parametrize("H,layers,lengths,pad", [
    (64, 1, [1], 0), (256, 2, [5, 0, 9], 8), (5120, 1, [1] * 40, 0), (4096, 3, [130, 1, 17], 64), (16384, 1, [3], 0),
    (320, 1, [2000], 0),
])
def test_kv_write_puts_every_row_in_its_page(L, H, layers, lengths, pad):
    import torch
    c = Cache(L, H, layers, lengths, seed=H)
    try:
        T = sum(lengths)
        req = np.repeat(np.arange(len(lengths)), lengths).astype(np.int32)
        pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
        perm = c.rng.permutation(T)
        req, pos = req[perm], pos[perm]
        skip = c.rng.random(T) < 0.2
        req_s = np.where(skip, -1, req).astype(np.int32)
        rows = [torch.empty((T, H + pad), dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2)]
        want = c.pool_t.clone()
        for layer in range(layers):
            L.lora_kv_write(c.pool, T, torch.from_numpy(req_s).cuda(), torch.from_numpy(pos).cuda(), rows[0], rows[1],
                            c.n_req, c.table, c.max_len, layers, layer, k_stride=H + pad, v_stride=H + pad)
            tabs = c.tables(layer)
            for t in np.flatnonzero(~skip):
                for half in range(2):
                    want[int(tabs[req[t]][pos[t], half])] = rows[half][int(t), :H]
        L.lora_status(c.pool)
        assert torch.equal(want.view(torch.int16), c.pool_t.view(torch.int16))
    finally:
        c.close()


@pytest.mark.parametrize("H,pad", [(64, 0), (128, 8), (192, 0), (256, 64), (320, 8), (512, 0), (576, 0)])
@pytest.mark.parametrize("bad", [False, True])
def test_kv_write_of_many_short_rows(L, H, pad, bad):
    """Enough rows that warps take several; the count ends inside a warp's share."""
    import torch
    lengths = [3000, 0, 1, 2998]
    layers, layer = 2, 1
    c = Cache(L, H, layers, lengths, seed=H)
    try:
        T = sum(lengths)
        rng = np.random.default_rng(H)
        req = np.repeat(np.arange(len(lengths)), lengths).astype(np.int32)
        pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
        perm = rng.permutation(T)
        req, pos = req[perm], pos[perm]
        rows = [torch.empty((T, H + pad), dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2)]
        tabs = c.tables(layer)
        pages = torch.from_numpy(np.stack([tabs[r][p] for r, p in zip(req, pos)])).cuda()
        keep = rng.random(T) < 0.8
        keep[-1] = True
        req = np.where(keep, req, -1).astype(np.int32)
        if bad:                                            # the row after each of these is written
            req[5], pos[6], pos[17], req[T - 3] = len(lengths), -1, c.max_len, -2
            bad_page = int(np.flatnonzero(keep[100:])[0]) + 100
            c.table[int(req[bad_page]), int(pos[bad_page]), layer, 1] = c.num_pages
            req[6] = req[17] = 0
            keep[[5, 6, 17, T - 3, bad_page]] = False
        want = c.pool_t.clone()
        sel = torch.from_numpy(np.flatnonzero(keep)).cuda()
        for half in range(2):
            want[pages[sel, half]] = rows[half][sel, :H]
        L.lora_kv_write(c.pool, T, torch.from_numpy(req).cuda(), torch.from_numpy(pos).cuda(), rows[0], rows[1], c.n_req,
                        c.table, c.max_len, layers, layer, k_stride=H + pad, v_stride=H + pad)
        if bad:
            with pytest.raises(L.LoraError) as e:
                L.lora_status(c.pool)
            assert e.value.code == L.LORA_EDEVICE
        else:
            L.lora_status(c.pool)
        assert torch.equal(want.view(torch.int16), c.pool_t.view(torch.int16))
    finally:
        c.close()


def test_kv_write_reports_bad_rows_and_writes_the_others(L):
    import torch
    c = Cache(L, 128, 1, [4, 4], seed=1)
    try:
        c.table[1, 3, 0, 1] = c.num_pages
        req = torch.tensor([0, 2, 0, -2, 1, 1], dtype=torch.int32, device="cuda")
        pos = torch.tensor([0, 0, c.max_len, 0, 3, 1], dtype=torch.int32, device="cuda")
        k = torch.ones((6, 128), dtype=torch.bfloat16, device="cuda")
        v = 2 * k
        want = c.pool_t.clone()
        tabs = c.tables(0)
        want[int(tabs[0][0, 0])], want[int(tabs[0][0, 1])] = 1.0, 2.0
        want[int(tabs[1][1, 0])], want[int(tabs[1][1, 1])] = 1.0, 2.0
        L.lora_kv_write(c.pool, 6, req, pos, k, v, 2, c.table, c.max_len, 1, 0)
        with pytest.raises(L.LoraError) as e:
            L.lora_status(c.pool)
        assert e.value.code == L.LORA_EDEVICE
        assert torch.equal(want.view(torch.int16), c.pool_t.view(torch.int16))
    finally:
        c.close()


def test_offsets_past_32_bits(L):
    """Pages whose element offset passes 2^31, read and written through a table whose own element
    index passes 2^31 (two requests far apart)."""
    import torch
    H, num_pages = 4096, 600_000
    layers, max_len = 64, (1 << 24) + 9
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    pool_t = torch.empty((num_pages, H), dtype=torch.bfloat16, device="cuda")
    table = torch.empty((3, max_len, layers, 2), dtype=torch.int32, device="cuda")
    pool = L.lora_pool_create(pool_t, num_pages, H, 1, 1)
    try:
        n, layer = 37, 63
        pages = np.arange(num_pages - 2 * n, num_pages).reshape(n, 2)
        table[2, :n, layer] = torch.from_numpy(pages.astype(np.int32)).cuda()
        seq = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
        rng = np.random.default_rng(0)
        kv = workloads.to_bf16_bits(rng.standard_normal((2, n, H)).astype(np.float32))
        L.lora_kv_write(pool, n, torch.full((n,), 2, dtype=torch.int32, device="cuda"),
                        torch.arange(n, dtype=torch.int32, device="cuda"), bits_to_torch(kv[0]), bits_to_torch(kv[1]),
                        3, table, max_len, layers, layer)
        q_bits = workloads.to_bf16_bits(rng.standard_normal((3, H)).astype(np.float32))
        out = torch.empty((3, H), dtype=torch.bfloat16, device="cuda")
        nb = L.lora_attention_split_size(pool, 3, max_len, 32, 32)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        L.lora_attention_split(pool, 3, table, seq, max_len, layers, layer, bits_to_torch(q_bits), out, 32, 32, ws, nb)
        L.lora_status(pool)
        bits = kv.transpose(1, 0, 2).reshape(2 * n, H)
        ref = O.attention_split(bits, [np.zeros((0, 2))] * 2 + [np.arange(2 * n).reshape(n, 2)], q_bits, 32, 32)
        _check(ref, out, None, [0, 0, n], 128, 1)
    finally:
        L.lora_pool_destroy(pool)


# ---- eviction ------------------------------------------------------------------------------------
def _evict(L, pool, table, seq, weight, budget, recent, max_len_out):
    import torch
    layers, n_req, max_len = weight.shape
    keep = torch.full((layers, n_req, budget), -9, dtype=torch.int32, device="cuda")
    new_len = torch.full((n_req,), -9, dtype=torch.int32, device="cuda")
    table_out = torch.full((n_req, max_len_out, layers, 2), -9, dtype=torch.int32, device="cuda")
    weight_out = torch.full((layers, n_req, max_len_out), -9.0, device="cuda")
    L.lora_kv_evict(pool, n_req, table, seq, max_len, layers, weight, budget, recent, keep, new_len, table_out,
                    weight_out, max_len_out)
    return keep.cpu().numpy(), new_len.cpu().numpy(), table_out.cpu().numpy(), weight_out.cpu().numpy()


def _evict_expected(table, lengths, weight, budget, recent, max_len_out):
    layers, n_req, _ = weight.shape
    keep = np.full((layers, n_req, budget), -1, np.int32)
    table_out = np.full((n_req, max_len_out, layers, 2), -1, np.int32)
    weight_out = np.zeros((layers, n_req, max_len_out), np.float32)
    for l in range(layers):
        for r, n in enumerate(lengths):
            k = O.evict_keep(weight[l, r], n, budget, recent)
            keep[l, r, :len(k)] = k
            table_out[r, :len(k), l] = table[r, k, l]
            weight_out[l, r, :len(k)] = weight[l, r, k]
    return keep, np.minimum(lengths, budget).astype(np.int32), table_out, weight_out


def _same(got, want):
    for name, g, w in zip(("keep", "new_len", "table", "weight"), got, want):
        eq = (g == w) | ((g != g) & (w != w)) if g.dtype.kind == "f" else g == w
        assert g.shape == w.shape and eq.all(), (name, np.argwhere(~eq)[:4])


KINDS = ["plain", "ties", "zeros", "special", "ascending"]


def _weights(kind, rng, shape):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, size=shape).astype(np.float32)
    elif kind == "zeros":
        w = np.where(rng.random(shape) < 0.9, np.where(rng.random(shape) < 0.5, 0.0, -0.0), w).astype(np.float32)
    elif kind == "special":
        pick = rng.integers(0, 7, size=shape)
        vals = np.float32([np.nan, np.inf, -np.inf, -1.5, 1e-42, -1e-42, 0.0])
        w = np.where(rng.random(shape) < 0.7, vals[pick], w).astype(np.float32)
    elif kind == "ascending":
        w = np.broadcast_to(np.arange(shape[-1], dtype=np.float32), shape).copy()
    return w


@pytest.mark.parametrize("layers,lengths,budget,recent", [
    (1, [80], 64, 16), (1, [1], 1, 0), (1, [1, 0, 2], 1, 1), (3, [64, 65, 63, 0, 200], 64, 0), (2, [300, 10, 299], 299, 299),
    (5, [1000, 1, 999], 17, 16), (2, [4097, 2049, 2048, 2047], 1024, 100), (1, [40000, 39999, 7], 2000, 1),
    (1, [140001, 3], 5000, 512), (2, [70000], 69999, 3), (40, [128] * 20, 100, 10), (1, [5] * 1000, 3, 1),
    (4, [4090, 0, 33, 4089] * 40, 4000, 3), (32, [2000, 1999, 3] * 7, 1, 1),
    (4, [4096, 0, 1, 31, 33, 127, 4095, 513] * 20, 500, 3), (7, [300, 1, 64, 0, 257] * 23, 64, 0), (1, [700] * 609, 700, 8),
])
@pytest.mark.parametrize("kind", KINDS)
def test_evict_keeps_what_the_definition_keeps(L, layers, lengths, budget, recent, kind):
    import torch
    rng = np.random.default_rng([layers, budget, KINDS.index(kind)])
    max_len = max(lengths) + int(rng.integers(0, 4))
    n_req = len(lengths)
    weight = _weights(kind, rng, (layers, n_req, max_len))
    table = rng.integers(0, 1 << 31, size=(n_req, max_len, layers, 2)).astype(np.int32)
    max_len_out = min(budget, max_len) + int(rng.integers(0, 9))
    pool_t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 4, 64, 1, 1)
    try:
        got = _evict(L, pool, torch.from_numpy(table).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                     torch.from_numpy(weight).cuda(), budget, recent, max_len_out)
        L.lora_status(pool)
        _same(got, _evict_expected(table, lengths, weight, budget, recent, max_len_out))
    finally:
        L.lora_pool_destroy(pool)


@pytest.mark.parametrize("layers,lengths,budget,recent", [
    (2, [100, 0, 37], 6000, 50), (1, [40000, 3], 50001, 49999), (40, [60] * 20, 5000, 0), (3, [17], 18, 18),
])
def test_evict_with_a_budget_above_the_longest_row(L, layers, lengths, budget, recent):
    """Everything stays; the kept list is filled up to the budget, table and weights to max_len_out."""
    import torch
    rng = np.random.default_rng(budget)
    max_len, n_req = max(lengths) + 1, len(lengths)
    weight = _weights("special", rng, (layers, n_req, max_len))
    table = rng.integers(0, 1 << 31, size=(n_req, max_len, layers, 2)).astype(np.int32)
    pool_t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 4, 64, 1, 1)
    try:
        got = _evict(L, pool, torch.from_numpy(table).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                     torch.from_numpy(weight).cuda(), budget, recent, max_len + 3)
        L.lora_status(pool)
        _same(got, _evict_expected(table, lengths, weight, budget, recent, max_len + 3))
    finally:
        L.lora_pool_destroy(pool)


def test_evict_reports_and_clamps_lengths(L):
    import torch
    rng = np.random.default_rng(3)
    weight = _weights("plain", rng, (2, 3, 50))
    table = rng.integers(0, 100, size=(3, 50, 2, 2)).astype(np.int32)
    pool_t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 4, 64, 1, 1)
    try:
        got = _evict(L, pool, torch.from_numpy(table).cuda(), torch.tensor([51, -1, 30], dtype=torch.int32, device="cuda"),
                     torch.from_numpy(weight).cuda(), 20, 5, 20)
        with pytest.raises(L.LoraError) as e:
            L.lora_status(pool)
        assert e.value.code == L.LORA_EDEVICE
        _same(got, _evict_expected(table, [50, 0, 30], weight, 20, 5, 20))
    finally:
        L.lora_pool_destroy(pool)


def test_evict_then_keep_then_attend(L):
    """The device's compacted table is the host bookkeeping's after lora_kv_keep, the freed pages are
    the pool's again, and attention over the kept tokens is attention over those tokens."""
    import torch
    n_kv, D, layers, lengths = 2, 64, 3, [70, 20, 41, 0]
    c = Cache(L, 128, layers, lengths, seed=21)
    try:
        weight = c.rng.random((layers, 4, c.max_len)).astype(np.float32)
        before = [c.tables(l) for l in range(layers)]
        keep, new_len, table_out, _ = _evict(L, c.pool, c.table, c.seq, torch.from_numpy(weight).cuda(), 32, 8, 35)
        free0 = L.lora_pool_stats(c.pool)["free"]
        for r in range(4):
            L.lora_kv_keep(c.pool, r, keep[:, r, :new_len[r]])
        assert L.lora_pool_stats(c.pool)["free"] == free0 + 2 * layers * ((70 - 32) + (41 - 32))
        table = torch.empty((4, 35, layers, 2), dtype=torch.int32, device="cuda")
        seq = torch.empty(4, dtype=torch.int32, device="cuda")
        L.lora_kv_batch_table(c.pool, [0, 1, 2, 3], 35, table, seq)
        assert np.array_equal(table.cpu().numpy(), table_out) and seq.tolist() == new_len.tolist() == [32, 20, 32, 0]
        q_bits = workloads.to_bf16_bits(c.rng.standard_normal((4, 128)).astype(np.float32))
        q = bits_to_torch(q_bits)
        nb = L.lora_attention_split_size(c.pool, 4, 35, 2, 2)
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")
        for l in range(layers):
            out = torch.empty_like(q)
            L.lora_attention_split(c.pool, 4, torch.from_numpy(table_out).cuda(), seq, 35, layers, l, q, out, 2, 2, ws, nb)
            kept = [before[l][r][keep[l, r, :new_len[r]]] for r in range(4)]
            _check(O.attention_split(c.bits, kept, q_bits, 2, 2), out, None, new_len.tolist(), D, 1)
        L.lora_status(c.pool)
    finally:
        c.close()


@pytest.mark.parametrize("long", [900, 20000])                    # a CTA per row, a cluster per row
def test_evict_in_a_graph_and_on_a_side_stream(L, long):
    import torch
    rng = np.random.default_rng(4)
    layers, n_req, max_len = 3, 5, long
    lengths = [long, 10, long // 2, 0, 300]
    weight = torch.from_numpy(_weights("ties", rng, (layers, n_req, max_len))).cuda()
    table = torch.from_numpy(rng.integers(0, 99, size=(n_req, max_len, layers, 2)).astype(np.int32)).cuda()
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pool_t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    pool = L.lora_pool_create(pool_t, 4, 64, 1, 1)
    try:
        keep = torch.zeros((layers, n_req, 256), dtype=torch.int32, device="cuda")
        new_len = torch.zeros(n_req, dtype=torch.int32, device="cuda")
        t_out = torch.zeros((n_req, 256, layers, 2), dtype=torch.int32, device="cuda")
        w_out = torch.zeros((layers, n_req, 256), device="cuda")
        args = (pool, n_req, table, seq, max_len, layers, weight, 256, 32, keep, new_len, t_out, w_out, 256)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            L.lora_kv_evict(*args)
        side.synchronize()
        want = _evict_expected(table.cpu().numpy(), lengths, weight.cpu().numpy(), 256, 32, 256)
        _same([x.cpu().numpy() for x in (keep, new_len, t_out, w_out)], want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lora_kv_evict(*args)
        weight.neg_()
        seq[3] = long - 1
        g.replay()
        torch.cuda.synchronize()
        want = _evict_expected(table.cpu().numpy(), [long, 10, long // 2, long - 1, 300], weight.cpu().numpy(), 256, 32, 256)
        _same([x.cpu().numpy() for x in (keep, new_len, t_out, w_out)], want)
        L.lora_status(pool)
    finally:
        L.lora_pool_destroy(pool)
