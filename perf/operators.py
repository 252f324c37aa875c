"""Timing cases of the KV-cache operators: page writes, split decode attention, eviction by weight.

Three operators over a pool whose pages hold one token's K or V vector of H bf16 values at one layer:
  write   rows of K and V into their pages, by (request, position) through the page table;
  attend  one new token per request over its cached tokens: output, log-sum-exp, and (optionally)
          the attention weight that every cached token received, added to its accumulated weight;
  evict   per request and layer, the tokens that stay under a budget (the newest, and the heaviest
          of the older ones), with page table and weights compacted.
Each case runs either in a plain form (elementary torch operations in 32 bits) or, with `own` set,
through the library's entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_PAD_PAGES = 32          # pages outside every request; they hold NaN
_PLAIN_BYTES = 2 << 30   # the plain attention gathers requests in groups of at most this size


# ---- cases -----------------------------------------------------------------------------------
def listed():
    """The cases with their real uses."""
    return [
        # A first decode step of a small model (the smallest workload's H): latency is all that counts.
        dict(name="attend_first_tokens", op="attend", n_req=4, lo=1, hi=9, H=256, D=64, group=1, layers=2,
             weights=False),
        # The benchmark's decode batch: 256 requests, H = 5120, contexts 128 to 2048.
        dict(name="attend_batch", op="attend", n_req=256, lo=128, hi=2048, H=5120, D=128, group=1, layers=1,
             weights=False),
        # One request with a long document in its cache: nothing but the length to split.
        dict(name="attend_long", op="attend", n_req=1, lo=131072, hi=131072, H=4096, D=128, group=1, layers=1,
             weights=False),
        # A few long chats on shared KV heads (four query heads each), lengths far apart, weights kept.
        dict(name="attend_shared_heads", op="attend", n_req=7, lo=500, hi=33333, H=1024, D=128, group=4, layers=1,
             weights=True),
        # A decode batch whose caches are kept under a budget: weights accumulate at every step.
        dict(name="attend_weights", op="attend", n_req=64, lo=0, hi=2047, H=4096, D=128, group=1, layers=3,
             weights=True),
        # Narrow heads, odd number of requests, short and ragged contexts.
        dict(name="attend_narrow", op="attend", n_req=33, lo=1, hi=515, H=2048, D=64, group=2, layers=1,
             weights=False),
        # A single request a few tokens over its budget, one layer.
        dict(name="evict_one", op="evict", n_req=1, lo=80, hi=80, layers=1, budget=64, recent=16),
        # Every layer of a serving batch cut back to half.
        dict(name="evict_batch", op="evict", n_req=64, lo=500, hi=2048, layers=40, budget=1024, recent=128),
        # One long document cut to a working set, all layers of a 7B-shaped model.
        dict(name="evict_long", op="evict", n_req=1, lo=131071, hi=131071, layers=32, budget=4096, recent=512),
        # The new token of each request of a decode batch.
        dict(name="write_decode", op="write", n_req=256, lo=1, hi=1, H=5120, layers=1),
        # The prompts of a prefill batch (16 requests of 128 to 1024 tokens).
        dict(name="write_prefill", op="write", n_req=16, lo=128, hi=1024, H=4096, layers=2),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n in (3069, 3072) else n


def draw(rng):
    """One more case of the listed ranges (`rng`: random.Random)."""
    op = rng.choice(["attend", "attend", "attend", "evict", "evict", "write"])
    if op == "attend":
        D = rng.choice([64, 128, 256])
        n_kv = rng.choice([n for n in (1, 2, 4, 5, 8, 12, 20, 32, 40) if 64 <= n * D <= 8192 and n * D != 3072])
        group = rng.choice([1, 1, 2, 3, 4, 8, 16]) if n_kv <= 8 else rng.choice([1, 1, 2, 4])
        n_req = _log_int(rng, 1, 256)
        cap = max(4, int(1.5e9 / (n_req * 4 * n_kv * D)))
        hi = _log_int(rng, 2, min(131072, cap))
        lo = rng.choice([0, 1, hi // 3, hi])
        if n_kv * D * group == 3072:
            group += 1
        return dict(op=op, n_req=n_req, lo=lo, hi=hi, H=n_kv * D, D=D, group=group,
                    layers=rng.randint(1, 3), weights=rng.random() < 0.5)
    if op == "evict":
        n_req = _log_int(rng, 1, 128)
        layers = _log_int(rng, 1, 40)
        hi = _log_int(rng, 2, min(131072, max(4, int(3e6 / (n_req * layers)))))
        budget = max(1, int(hi * rng.uniform(0.02, 1.0)))
        budget -= budget == 3072
        return dict(op=op, n_req=n_req, lo=rng.choice([0, hi // 2, hi]), hi=hi, layers=layers, budget=budget,
                    recent=rng.randint(0, budget))
    H = rng.choice([64, 256, 1024, 4096, 5120])
    n_req = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, max(2, int(40e6 / (n_req * H))))
    return dict(op=op, n_req=n_req, lo=rng.choice([0, 1, hi]), hi=hi, H=H, layers=rng.randint(1, 3))


def _lengths(case):
    """Tokens of every request: uniform in [lo, hi], fixed by the case; one request has hi."""
    rng = np.random.default_rng([case["n_req"], case["lo"], case["hi"]])
    n = rng.integers(min(case["lo"], case["hi"]), case["hi"] + 1, size=case["n_req"])
    n[int(rng.integers(0, case["n_req"]))] = case["hi"]
    return n.astype(np.int64)


def _max_len(case):
    return case["hi"] + 3          # a little room, as a program that grows its caches has


def _max_len_out(case):
    return min(case["budget"], case["hi"]) + 3


def work(case):
    """Bytes and operations that one pass cannot do without."""
    tokens = int(_lengths(case).sum())
    if case["op"] == "attend":
        heads = case["H"] // case["D"] * case["group"]
        q = case["n_req"] * heads * case["D"]
        b = tokens * (4 * case["H"] + 8) + 4 * q + 4 * case["n_req"] * heads
        if case["weights"]:
            b += 8 * tokens
        return {"bytes": b, "flops": 4 * tokens * heads * case["D"]}
    if case["op"] == "evict":
        kept = int(np.minimum(_lengths(case), case["budget"]).sum())
        out = case["n_req"] * (_max_len_out(case) * 12 + case["budget"] * 4)
        return {"bytes": case["layers"] * (4 * tokens + 8 * kept + out) + 8 * case["n_req"], "flops": 0}
    return {"bytes": tokens * (8 * case["H"] + 16), "flops": 0}


# ---- inputs ----------------------------------------------------------------------------------
def _table(case, lens, num_pages, first_page, g):
    """int32 [n_req][max_len][layers][2]: pages of the case's last layer are distinct and shuffled;
    entries of other layers name NaN pages; -1 past a request's length."""
    n_req, L, layers = case["n_req"], _max_len(case), case["layers"]
    dev = lens.device
    tab = torch.full((n_req, L, layers, 2), -1, dtype=torch.int32, device=dev)
    valid = torch.arange(L, device=dev)[None, :] < lens[:, None]
    tab[valid] = torch.randint(0, first_page, (int(valid.sum()), layers, 2), generator=g, device=dev,
                               dtype=torch.int32)
    pages = torch.randperm(num_pages - first_page, generator=g, device=dev)[:2 * int(valid.sum())] + first_page
    last = tab[:, :, layers - 1, :]
    last[valid] = pages.to(torch.int32).view(-1, 2)
    return tab


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host_lens = _lengths(case)
    lens = torch.from_numpy(host_lens).to(dev)
    tokens, n_req, L = int(host_lens.sum()), case["n_req"], _max_len(case)
    s = dict(case=case, lens=lens.to(torch.int32), max_len=L)
    if case["op"] == "evict":
        layers, Lo = case["layers"], _max_len_out(case)
        # Accumulated weights: a heavy tail, exact zeros for tokens that nothing looked at.
        w = torch.exp(2.0 * torch.randn((layers, n_req, L), generator=g, device=dev) - 3.0)
        w = torch.where(torch.rand((layers, n_req, L), generator=g, device=dev) < 0.05, 0.0, w)
        valid = torch.arange(L, device=dev)[None, :] < lens[:, None]
        s["weight"] = torch.where(valid[None], w, 0.0).contiguous()
        tab = torch.randint(0, 1 << 30, (n_req, L, layers, 2), generator=g, device=dev, dtype=torch.int32)
        s["table"] = torch.where(valid[:, :, None, None], tab, torch.full_like(tab, -1)).contiguous()
        s["keep"] = torch.empty((layers, n_req, case["budget"]), dtype=torch.int32, device=dev)
        s["new_len"] = torch.empty(n_req, dtype=torch.int32, device=dev)
        s["table_out"] = torch.empty((n_req, Lo, layers, 2), dtype=torch.int32, device=dev)
        s["weight_out"] = torch.empty((layers, n_req, Lo), dtype=torch.float32, device=dev)
        s["max_len_out"] = Lo
        return s
    H, num_pages = case["H"], _PAD_PAGES + 2 * tokens + 2
    s["pool"] = torch.randn((num_pages, H), generator=g, device=dev, dtype=torch.bfloat16)
    if case["op"] == "attend":
        s["pool"][:_PAD_PAGES] = float("nan")
        s["table"] = _table(case, lens, num_pages, _PAD_PAGES, g)
        heads = H // case["D"] * case["group"]
        s["heads"], s["kv_heads"] = heads, H // case["D"]
        s["q"] = torch.randn((n_req, heads * case["D"]), generator=g, device=dev, dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n_req, heads), dtype=torch.float32, device=dev)
        if case["weights"]:
            w = 4.0 * torch.rand((n_req, L), generator=g, device=dev)
            s["weight_in"] = torch.where(torch.arange(L, device=dev)[None, :] < lens[:, None], w, 0.0).contiguous()
            s["weight_out"] = torch.zeros_like(s["weight_in"])
        return s
    # write: every request's tokens in order, as a batch carries them; pages hold older rows
    s["table"] = _table(case, lens, num_pages, _PAD_PAGES, g)
    req = np.repeat(np.arange(n_req), host_lens)
    pos = np.concatenate([np.arange(n) for n in host_lens]) if tokens else np.zeros(0, np.int64)
    s["row_req"] = torch.from_numpy(req.astype(np.int32)).to(dev)
    s["row_pos"] = torch.from_numpy(pos.astype(np.int32)).to(dev)
    s["k"] = torch.randn((tokens, H), generator=g, device=dev, dtype=torch.bfloat16)
    s["v"] = torch.randn((tokens, H), generator=g, device=dev, dtype=torch.bfloat16)
    return s


class _Pool:
    """A pool handle that goes with its state."""

    def __init__(self, storage, num_pages, H):
        import adapter_gemm_lora_gb300 as L
        self.lib = L
        self.handle = L.lora_pool_create(storage, num_pages, H, 1, 1)

    def __del__(self):
        self.lib.lora_pool_destroy(self.handle)


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import adapter_gemm_lora_gb300 as L
    if case["op"] == "evict":
        # The operator reads page ids, not pages: the pool only has to be large enough for them.
        s["pages"] = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
        s["handle"] = _Pool(s["pages"], 1, 64)
        return s
    s["handle"] = _Pool(s["pool"], s["pool"].shape[0], case["H"])
    if case["op"] == "attend":
        s["ws_bytes"] = L.lora_attention_split_size(s["handle"].handle, case["n_req"], s["max_len"], s["heads"],
                                                    s["kv_heads"], case["weights"])
        s["ws"] = torch.empty(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "attend":
        return _attend_own(s) if own else _attend_plain(s)
    if op == "evict":
        return _evict_own(s) if own else _evict_plain(s)
    return _write_own(s) if own else _write_plain(s)


def _attend_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    if c["weights"]:
        L.lora_attention_split(s["handle"].handle, c["n_req"], s["table"], s["lens"], s["max_len"], c["layers"],
                               c["layers"] - 1, s["q"], s["out"], s["heads"], s["kv_heads"], s["ws"], s["ws_bytes"],
                               lse_dev=s["lse"], weight_in_dev=s["weight_in"], weight_out_dev=s["weight_out"])
        return s["out"], s["lse"], s["weight_out"]
    L.lora_attention_split(s["handle"].handle, c["n_req"], s["table"], s["lens"], s["max_len"], c["layers"],
                           c["layers"] - 1, s["q"], s["out"], s["heads"], s["kv_heads"], s["ws"], s["ws_bytes"],
                           lse_dev=s["lse"])
    return s["out"], s["lse"]


def _attend_plain(s):
    c, L = s["case"], s["max_len"]
    n_req, H, D, kv, G = c["n_req"], c["H"], c["D"], s["kv_heads"], c["group"]
    out, lse = s["out"], s["lse"]
    weight_out = s["weight_out"] if c["weights"] else None
    step = max(1, _PLAIN_BYTES // (L * H * 4))
    for a in range(0, n_req, step):
        b = min(n_req, a + step)
        ids = s["table"][a:b, :, c["layers"] - 1, :].long()
        valid = torch.arange(L, device=ids.device)[None, :] < s["lens"][a:b, None]
        ids = torch.where(valid[..., None], ids, 0)
        k = torch.where(valid[..., None], s["pool"][ids[..., 0]].float(), 0.0).view(b - a, L, kv, D)
        q = s["q"][a:b].float().view(b - a, kv, G, D)
        sc = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(D)              # [c, kv, G, L]
        del k
        sc = sc.masked_fill(~valid[:, None, None, :], float("-inf"))
        m = sc.amax(dim=-1, keepdim=True)
        m = torch.where(torch.isinf(m) & (m < 0), 0.0, m)
        p = torch.exp(sc - m)
        l = p.sum(dim=-1, keepdim=True)
        p = torch.where(l > 0, p / l, 0.0)
        v = torch.where(valid[..., None], s["pool"][ids[..., 1]].float(), 0.0).view(b - a, L, kv, D)
        o = torch.matmul(p, v.permute(0, 2, 1, 3))                              # [c, kv, G, D]
        del v
        out[a:b] = o.reshape(b - a, -1).to(torch.bfloat16)
        lse[a:b] = (m + torch.log(l)).reshape(b - a, -1)
        if weight_out is not None:
            weight_out[a:b] = s["weight_in"][a:b] + p.sum(dim=(1, 2))
    return (out, lse, weight_out) if c["weights"] else (out, lse)


def _evict_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    L.lora_kv_evict(s["handle"].handle, c["n_req"], s["table"], s["lens"], s["max_len"], c["layers"], s["weight"],
                    c["budget"], c["recent"], s["keep"], s["new_len"], s["table_out"], s["weight_out"],
                    s["max_len_out"])
    return s["keep"], s["new_len"], s["table_out"], s["weight_out"]


def _evict_plain(s):
    c, L, Lo = s["case"], s["max_len"], s["max_len_out"]
    n_req, layers, budget = c["n_req"], c["layers"], c["budget"]
    lens = s["lens"].long()
    dev = lens.device
    j = torch.arange(L, device=dev)
    w = s["weight"]
    # Ascending integer keys in the order of the values (adding 0 makes -0 into 0; NaN is lowest).
    bits = torch.where(torch.isnan(w), float("-inf"), w + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    key = torch.where((j[None, :] >= lens[:, None] - c["recent"])[None], 1 << 40, key)
    key = torch.where((j[None, :] < lens[:, None])[None], key, -(1 << 40))
    new_len = torch.minimum(lens, torch.full_like(lens, budget))
    n_slots = min(budget, L)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n_slots]
    i = torch.arange(n_slots, device=dev)
    in_row = (i[None, :] < new_len[:, None])[None].expand(layers, -1, -1)
    order = torch.sort(torch.where(in_row, order, L), dim=-1).values               # ascending positions
    keep = torch.full((layers, n_req, budget), -1, dtype=torch.int32, device=dev)
    keep[..., :n_slots] = torch.where(in_row, order, -1).to(torch.int32)
    n = min(n_slots, Lo)
    pick = torch.where(in_row, order, 0)[..., :n]
    weight_out = torch.zeros((layers, n_req, Lo), dtype=torch.float32, device=dev)
    weight_out[..., :n] = torch.where(in_row[..., :n], torch.gather(w, 2, pick), 0.0)
    table_out = torch.full((n_req, Lo, layers, 2), -1, dtype=torch.int32, device=dev)
    r = torch.arange(n_req, device=dev)[:, None, None]
    l = torch.arange(layers, device=dev)[None, None, :]
    pick_t = pick.permute(1, 2, 0)                                                  # [n_req, n, layers]
    table_out[:, :n] = torch.where(in_row[..., :n].permute(1, 2, 0)[..., None], s["table"][r, pick_t, l], -1)
    return keep, new_len.to(torch.int32), table_out, weight_out


def _write_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    L.lora_kv_write(s["handle"].handle, s["row_req"].numel(), s["row_req"], s["row_pos"], s["k"], s["v"], c["n_req"],
                    s["table"], s["max_len"], c["layers"], c["layers"] - 1)
    return s["pool"]


def _write_plain(s):
    ids = s["table"][s["row_req"].long(), s["row_pos"].long(), s["case"]["layers"] - 1].long()
    s["pool"][ids[:, 0]] = s["k"]
    s["pool"][ids[:, 1]] = s["v"]
    return s["pool"]


# ---- the operators' definitions in 64 bits ---------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "attend":
        return _attend_exact(s)
    return _evict_exact(s) if case["op"] == "evict" else _write_exact(s)


def _attend_exact(s):
    c = s["case"]
    D, G, kv = c["D"], c["group"], s["kv_heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device="cuda")
    weight = torch.zeros((c["n_req"], s["max_len"]), dtype=torch.float64, device="cuda")
    for r, n in enumerate(_lengths(c).tolist()):
        if n == 0:
            continue
        pages = s["table"][r, :n, c["layers"] - 1].long()
        for h0 in range(0, kv, 4):                        # four KV heads at a time
            h1 = min(kv, h0 + 4)
            K = s["pool"][pages[:, 0], h0 * D:h1 * D].double().view(n, h1 - h0, D)
            V = s["pool"][pages[:, 1], h0 * D:h1 * D].double().view(n, h1 - h0, D)
            for i in range(G):
                heads = torch.arange(h0, h1, device="cuda") * G + i
                q = s["q"][r].double().view(-1, D)[heads]
                score = (K * q[None]).sum(2) / math.sqrt(D)
                z = torch.logsumexp(score, 0)
                p = torch.exp(score - z)
                lse[r, heads] = z
                out[r].view(-1, D)[heads] = (p[..., None] * V).sum(0)
                weight[r, :n] += p.sum(1)
    if not c["weights"]:
        return out, lse
    for r, n in enumerate(_lengths(c).tolist()):
        weight[r, :n] += s["weight_in"][r, :n].double()
    return out, lse, weight


def _evict_exact(s):
    c, Lo = s["case"], s["max_len_out"]
    w, tab = s["weight"].cpu().double().numpy(), s["table"].cpu().numpy()
    keep = np.full((c["layers"], c["n_req"], c["budget"]), -1, np.int32)
    new_len = np.zeros(c["n_req"], np.int32)
    table_out = np.full((c["n_req"], Lo, c["layers"], 2), -1, np.int32)
    weight_out = np.zeros((c["layers"], c["n_req"], Lo))
    for r, n in enumerate(_lengths(c).tolist()):
        k = min(n, c["budget"])
        old = max(0, n - c["recent"])
        new_len[r] = k
        for layer in range(c["layers"]):
            heavy = np.argsort(-w[layer, r, :old], kind="stable")[:max(0, k - (n - old))]
            kept = np.sort(np.concatenate([heavy, np.arange(old, n)]))[:k]
            keep[layer, r, :k] = kept
            table_out[r, :k, layer] = tab[r, kept, layer]
            weight_out[layer, r, :k] = w[layer, r, kept]
    dev = s["weight"].device
    return tuple(torch.from_numpy(x).to(dev) for x in (keep, new_len, table_out, weight_out))


def _write_exact(s):
    pool = s["pool"].double()
    for half, rows in enumerate((s["k"], s["v"])):
        for a in range(0, rows.shape[0], 4096):
            r, p = s["row_req"][a:a + 4096].long(), s["row_pos"][a:a + 4096].long()
            page = s["table"][r, p, s["case"]["layers"] - 1, half].long()
            pool.index_copy_(0, page, rows[a:a + 4096].double())
    return pool
