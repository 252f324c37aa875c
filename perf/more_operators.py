"""Timing cases of the operators that fill and check a KV cache: prompt attention, tree attention, slot maps.

Three operators beside the page writes, the decode attention and the eviction of the same cache:
  prompt  causal attention over whole prompts, packed one behind another, before any token is decoded:
          output and log-sum-exp, grouped query heads;
  tree    attention of a tree of drafted tokens per request over its cached tokens, the drafted ones
          among them: a node sees every cached token and the nodes that its mask names;
  append  from the requests' token counts, on the GPU: the page table with the new tokens' pages, the
          new lengths, and (request, position) of every new row.
Each case runs either in a plain form (elementary torch operations in 32 bits) or, with `own` set,
through the library's entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_PAD_PAGES = 32          # pages outside every request; they hold NaN
_PLAIN_BYTES = 2 << 30   # the plain attentions work in pieces of at most this size


# ---- cases -----------------------------------------------------------------------------------
def listed():
    """The cases with their real uses."""
    return [
        # First prompts of a small model (the smallest workload's H): latency is all that counts.
        dict(name="prompt_first_tokens", op="prompt", n_req=4, lo=1, hi=9, n_kv=4, D=64, group=1),
        # The benchmark's prefill batch: 16 prompts of 128 to 1024 tokens, H = 4096.
        dict(name="prompt_batch", op="prompt", n_req=16, lo=128, hi=1024, n_kv=32, D=128, group=1),
        # One long document.
        dict(name="prompt_long", op="prompt", n_req=1, lo=16384, hi=16384, n_kv=32, D=128, group=1),
        # A few prompts of very different lengths on shared KV heads.
        dict(name="prompt_shared_heads", op="prompt", n_req=7, lo=100, hi=5000, n_kv=8, D=128, group=4),
        # Many short, ragged prompts, narrow heads.
        dict(name="prompt_narrow", op="prompt", n_req=33, lo=1, hi=515, n_kv=32, D=64, group=2),
        # Wide heads, two prompts.
        dict(name="prompt_wide", op="prompt", n_req=2, lo=2047, hi=4097, n_kv=8, D=256, group=2),
        # One request checks a short draft.
        dict(name="tree_one", op="tree", n_req=1, lo=705, hi=705, n_kv=4, D=64, group=1, nodes=5, layers=2),
        # A serving batch, each request with its own tree.
        dict(name="tree_batch", op="tree", n_req=64, lo=0, hi=2047, n_kv=32, D=128, group=1, nodes=32, layers=2),
        # One long document in the cache, the largest tree.
        dict(name="tree_long", op="tree", n_req=1, lo=131072, hi=131072, n_kv=32, D=128, group=1, nodes=64, layers=1),
        # Long chats on shared KV heads.
        dict(name="tree_shared_heads", op="tree", n_req=7, lo=500, hi=33333, n_kv=8, D=128, group=4, nodes=48, layers=1),
        # One more token for each request of a decode batch, 40 layers.
        dict(name="append_decode", op="append", n_req=256, lo=1, hi=1, layers=40, cached=2047),
        # The prompts of a serving batch enter empty tables.
        dict(name="append_prompts", op="append", n_req=64, lo=500, hi=2048, layers=40, cached=-1),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges (`rng`: random.Random)."""
    op = rng.choice(["prompt", "prompt", "tree", "tree", "append"])
    if op == "append":
        layers = _log_int(rng, 1, 40)
        n_req = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, max(1, min(8192, int(3e6 / (layers * n_req)))))
        return dict(op=op, n_req=n_req, lo=rng.choice([0, 1, hi]), hi=hi, layers=layers,
                    cached=rng.choice([-1, 0, rng.randint(1, max(1, min(4096, int(4e6 / (layers * n_req)))))]))
    D = rng.choice([64, 128, 256])
    n_kv = rng.choice([n for n in (1, 2, 4, 5, 8, 16, 20, 32, 40) if n * D <= 8192])
    group = rng.choice([1, 1, 2, 3, 4, 8, 16]) if n_kv <= 8 else rng.choice([1, 1, 2, 4])
    heads = n_kv * group
    if op == "prompt":
        n_req = _log_int(rng, 1, 256)
        most = math.sqrt(1e12 / (2 * heads * D * n_req))              # tokens per prompt, by operations
        hi = _log_int(rng, 1, max(1, int(min(16384, most, 65536 / n_req, 2.5e8 / (heads * D * n_req)))))
        return dict(op=op, n_req=n_req, lo=rng.choice([0, 1, hi // 3, hi]), hi=hi, n_kv=n_kv, D=D, group=group)
    n_req = _log_int(rng, 1, 128)
    nodes = _log_int(rng, 1, 64)
    cap = max(1, int(min(131072, 1.5e9 / (n_req * 4 * n_kv * D), 1e9 / (n_req * heads * nodes))))
    hi = nodes + _log_int(rng, 1, cap)
    return dict(op=op, n_req=n_req, lo=rng.choice([0, hi // 3, hi]), hi=hi, n_kv=n_kv, D=D, group=group, nodes=nodes,
                layers=rng.randint(1, 3))


def _lengths(case):
    """Tokens of every request: uniform in [lo, hi], fixed by the case; one request has hi."""
    rng = np.random.default_rng([case["n_req"], case["lo"], case["hi"]])
    n = rng.integers(min(case["lo"], case["hi"]), case["hi"] + 1, size=case["n_req"])
    n[int(rng.integers(0, case["n_req"]))] = case["hi"]
    return n.astype(np.int64)


def _nodes(case):
    """Drafted tokens of every request (tree): half of `nodes` to all of them, at most what is cached."""
    rng = np.random.default_rng([case["n_req"], case["nodes"]])
    n = rng.integers((case["nodes"] + 1) // 2, case["nodes"] + 1, size=case["n_req"])
    return np.minimum(n, _lengths(case)).astype(np.int64)


def _old_lengths(case):
    """Tokens that the tables hold before (append): none, or up to `cached`."""
    rng = np.random.default_rng([case["n_req"], case["hi"]])
    return rng.integers(0, max(case["cached"], 0) + 1, size=case["n_req"]).astype(np.int64)


def _max_len(case):
    return case["hi"] + max(case.get("cached", 0), 0) + 3          # a little room, as a program's tables have


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    n = _lengths(case)
    if case["op"] == "append":
        new, entry = int(n.sum()), 8 * case["layers"]
        b = new * (2 * entry + 8) + 16 * case["n_req"]
        if case["cached"] < 0:                                         # the rest of the table is cleared
            b += (case["n_req"] * _max_len(case) - new) * entry
        return {"bytes": b, "flops": 0}
    heads, D, H = case["n_kv"] * case["group"], case["D"], case["n_kv"] * case["D"]
    if case["op"] == "prompt":
        pairs = int((n * (n + 1) // 2).sum())
        return {"bytes": int(n.sum()) * (4 * H + 4 * heads * D + 4 * heads), "flops": 4 * pairs * heads * D}
    nodes = _nodes(case)
    rows, pairs = int(nodes.sum()), int((nodes * n).sum())
    return {"bytes": int(n.sum()) * (4 * H + 8) + rows * (4 * heads * D + 4 * heads + 8), "flops": 4 * pairs * heads * D}


# ---- inputs ----------------------------------------------------------------------------------
def _tree_masks(nodes, rng):
    """One 64-bit mask per node: the node and its ancestors; parents are drawn among the earlier nodes."""
    masks = []
    for n in nodes.tolist():
        own_mask = []
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            own_mask.append((1 << i) | (own_mask[parent] if parent >= 0 else 0))
        masks += own_mask
    return np.array(masks, dtype=np.uint64).view(np.int64)


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, n_req = _lengths(case), case["n_req"]
    tokens, L = int(lens.sum()), _max_len(case)
    s = dict(case=case, max_len=L)
    to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    if case["op"] == "append":
        old, layers = _old_lengths(case), case["layers"]
        s["rows"] = tokens + 5                                          # the row arrays have room, as a padded batch's
        s["count"], s["old"] = to(lens.astype(np.int32)), to(old.astype(np.int32))
        s["pages"] = torch.randint(0, 1 << 30, (s["rows"], layers, 2), generator=g, device=dev, dtype=torch.int32)
        held = torch.arange(L, device=dev)[None, :] < s["old"][:, None]
        tab = torch.randint(0, 1 << 30, (n_req, L, layers, 2), generator=g, device=dev, dtype=torch.int32)
        s["table"] = torch.where(held[:, :, None, None], tab, torch.full_like(tab, -1)).contiguous()
        s["new_len"] = torch.empty(n_req, dtype=torch.int32, device=dev)
        s["row_start"] = torch.empty(n_req + 1, dtype=torch.int32, device=dev)
        s["row_req"] = torch.empty(s["rows"], dtype=torch.int32, device=dev)
        s["row_pos"] = torch.empty(s["rows"], dtype=torch.int32, device=dev)
        return s
    heads, D, kv = case["n_kv"] * case["group"], case["D"], case["n_kv"]
    if case["op"] == "prompt":
        s["start_host"] = _starts(lens)
        s["start"] = to(s["start_host"])
        s["q"], s["k"], s["v"] = normal(tokens, heads * D), normal(tokens, kv * D), normal(tokens, kv * D)
    else:
        nodes, layers = _nodes(case), case["layers"]
        num_pages = _PAD_PAGES + 2 * tokens + 2
        s["lens"], s["start_host"] = to(lens.astype(np.int32)), _starts(nodes)
        s["start"] = to(s["start_host"])
        s["mask"] = to(_tree_masks(nodes, np.random.default_rng(seed)))
        s["pool"] = normal(num_pages, kv * D)
        s["pool"][:_PAD_PAGES] = float("nan")
        # The case's last layer has the requests' pages, distinct and shuffled; other layers name NaN pages.
        tab = torch.full((n_req, L, layers, 2), -1, dtype=torch.int32, device=dev)
        valid = torch.arange(L, device=dev)[None, :] < s["lens"][:, None]
        tab[valid] = torch.randint(0, _PAD_PAGES, (tokens, layers, 2), generator=g, device=dev, dtype=torch.int32)
        pages = torch.randperm(num_pages - _PAD_PAGES, generator=g, device=dev)[:2 * tokens] + _PAD_PAGES
        tab[:, :, layers - 1, :][valid] = pages.to(torch.int32).view(-1, 2)
        s["table"] = tab
        s["q"] = normal(int(nodes.sum()), heads * D)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((s["q"].shape[0], heads), dtype=torch.float32, device=dev)
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
    if case["op"] == "append":
        # The operator moves page ids, not pages: any pool will do.
        s["pages_of_pool"] = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
        s["handle"] = _Pool(s["pages_of_pool"], 1, 64)
        return s
    heads, kv, H = case["n_kv"] * case["group"], case["n_kv"], case["n_kv"] * case["D"]
    if case["op"] == "prompt":
        s["pages_of_pool"] = torch.zeros((1, H), dtype=torch.bfloat16, device="cuda")
        s["handle"] = _Pool(s["pages_of_pool"], 1, H)
        s["ws_bytes"] = L.lora_attention_prompt_size(s["handle"].handle, case["n_req"], s["q"].shape[0], heads, kv)
    else:
        s["handle"] = _Pool(s["pool"], s["pool"].shape[0], H)
        s["ws_bytes"] = L.lora_attention_tree_size(s["handle"].handle, case["n_req"], s["max_len"], heads, kv)
    s["ws"] = torch.empty(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "prompt":
        return _prompt_own(s) if own else _prompt_plain(s)
    if op == "tree":
        return _tree_own(s) if own else _tree_plain(s)
    return _append_own(s) if own else _append_plain(s)


def _prompt_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    L.lora_attention_prompt(s["handle"].handle, c["n_req"], s["start"], s["q"].shape[0], s["q"], s["k"], s["v"], s["out"],
                            c["n_kv"] * c["group"], c["n_kv"], s["ws"], s["ws_bytes"], lse_dev=s["lse"])
    return s["out"], s["lse"]


def _prompt_plain(s):
    c, out, lse = s["case"], s["out"], s["lse"]
    kv, G, D = c["n_kv"], c["group"], c["D"]
    for a, b in zip(s["start_host"][:-1].tolist(), s["start_host"][1:].tolist()):
        step = max(1, _PLAIN_BYTES // (4 * kv * G * max(1, b - a)))
        for r0 in range(a, b, step):                                   # the piece's rows see tokens a .. r1
            r1 = min(b, r0 + step)
            q = s["q"][r0:r1].float().view(r1 - r0, kv, G, D).permute(1, 2, 0, 3).reshape(kv, G * (r1 - r0), D)
            k = s["k"][a:r1].float().view(r1 - a, kv, D).permute(1, 2, 0)
            v = s["v"][a:r1].float().view(r1 - a, kv, D).permute(1, 0, 2)
            sc = (torch.matmul(q, k) / math.sqrt(D)).view(kv, G, r1 - r0, r1 - a)
            future = torch.arange(r1 - a, device=q.device)[None, :] > torch.arange(r0 - a, r1 - a, device=q.device)[:, None]
            sc.masked_fill_(future, float("-inf"))
            m = sc.amax(dim=-1, keepdim=True)
            p = torch.exp(sc - m)
            del sc
            l = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p.view(kv, G * (r1 - r0), r1 - a), v).view(kv, G, r1 - r0, D) / l
            out[r0:r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, -1).to(torch.bfloat16)
            lse[r0:r1] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(r1 - r0, -1)
    return out, lse


def _tree_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    L.lora_attention_tree(s["handle"].handle, c["n_req"], s["table"], s["lens"], s["max_len"], c["layers"], c["layers"] - 1,
                          s["start"], s["q"].shape[0], s["mask"], s["q"], s["out"], c["n_kv"] * c["group"], c["n_kv"],
                          s["ws"], s["ws_bytes"], lse_dev=s["lse"])
    return s["out"], s["lse"]


def _tree_plain(s):
    c, L, out, lse = s["case"], s["max_len"], s["out"], s["lse"]
    n_req, kv, G, D = c["n_req"], c["n_kv"], c["group"], c["D"]
    dev = out.device
    first = s["start_host"][:-1]
    widest = int(np.diff(s["start_host"]).max())
    j = torch.arange(L, device=dev)
    i = torch.arange(widest, device=dev)
    step = max(1, _PLAIN_BYTES // (4 * L * kv * max(D, G * widest, 1)))
    if widest == 0:
        return out, lse
    for a in range(0, n_req, step):
        b = min(n_req, a + step)
        lens = s["lens"][a:b].long()
        start = torch.from_numpy(first[a:b]).to(dev).long()
        nodes = s["start"][a + 1:b + 1].long() - start
        real = i[None, :] < nodes[:, None]                                               # [c, widest]
        row = torch.where(real, start[:, None] + i[None, :], 0)
        valid = j[None, :] < lens[:, None]
        ids = torch.where(valid[..., None], s["table"][a:b, :, c["layers"] - 1, :].long(), 0)
        k = torch.where(valid[..., None], s["pool"][ids[..., 0]].float(), 0.0).view(b - a, L, kv, D)
        q = s["q"][row].float().view(b - a, widest, kv, G, D).permute(0, 2, 3, 1, 4).reshape(b - a, kv, G * widest, D)
        sc = (torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(D)).view(b - a, kv, G, widest, L)
        del k
        node = j[None, :] - (lens - nodes)[:, None]                                      # < 0: cached before the draft
        bit = (s["mask"][row][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1
        sees = ((node < 0)[:, None, :] | (bit == 1)) & valid[:, None, :]                 # [c, widest, L]
        sc.masked_fill_(~sees[:, None, None], float("-inf"))
        m = sc.amax(dim=-1, keepdim=True)
        m = torch.where(torch.isinf(m) & (m < 0), 0.0, m)
        p = torch.exp(sc - m)
        del sc
        l = p.sum(dim=-1, keepdim=True)
        v = torch.where(valid[..., None], s["pool"][ids[..., 1]].float(), 0.0).view(b - a, L, kv, D)
        o = torch.matmul(p.view(b - a, kv, G * widest, L), v.permute(0, 2, 1, 3)).view(b - a, kv, G, widest, D)
        del v, p
        o = torch.where(l > 0, o / l, 0.0).permute(0, 3, 1, 2, 4).reshape(b - a, widest, -1)
        z = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).reshape(b - a, widest, -1)
        out[row[real]] = o[real].to(torch.bfloat16)
        lse[row[real]] = z[real]
    return out, lse


def _append_own(s):
    import adapter_gemm_lora_gb300 as L
    c = s["case"]
    L.lora_kv_append(s["handle"].handle, c["n_req"], s["count"], None if c["cached"] < 0 else s["old"], s["pages"], s["rows"],
                     s["table"], s["max_len"], c["layers"], s["new_len"], s["row_start"], s["row_req"], s["row_pos"])
    return s["table"], s["new_len"], s["row_start"], s["row_req"], s["row_pos"]


def _append_plain(s):
    c, rows, L = s["case"], s["rows"], s["max_len"]
    count = s["count"].long()
    old = s["old"].long() if c["cached"] >= 0 else torch.zeros_like(count)
    end = torch.cumsum(count, 0)
    start = end - count
    t = torch.arange(rows, device=count.device)
    req = torch.searchsorted(end, t, right=True)
    live = req < c["n_req"]
    r = torch.where(live, req, 0)
    pos = old[r] + t - start[r]
    s["row_req"].copy_(torch.where(live, r, -1))
    s["row_pos"].copy_(torch.where(live, pos, 0))
    s["row_start"][0] = 0
    s["row_start"][1:] = end
    s["new_len"].copy_(old + count)
    if c["cached"] < 0:
        s["table"].fill_(-1)
    flat = s["table"].view(c["n_req"] * L, -1)
    flat[(r * L + pos)[live]] = s["pages"].view(rows, -1)[live]
    return s["table"], s["new_len"], s["row_start"], s["row_req"], s["row_pos"]


# ---- the operators' definitions in 64 bits ---------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "prompt":
        return _prompt_exact(s)
    return _tree_exact(s) if case["op"] == "tree" else _append_exact(s)


def _softmax_exact(q, K, V, sees):
    """Rows q over the tokens K, V that each sees: outputs and log-sum-exp, in 64 bits."""
    score = torch.where(sees, torch.einsum("hrd,nd->hrn", q, K) / math.sqrt(q.shape[-1]), float("-inf"))
    z = torch.logsumexp(score, -1)
    weight = torch.where(sees, torch.exp(score - z[..., None]), 0.0)
    return torch.einsum("hrn,nd->hrd", weight, V), z


def _prompt_exact(s):
    c = s["case"]
    kv, G, D = c["n_kv"], c["group"], c["D"]
    rows = s["q"].shape[0]
    out = torch.zeros((rows, kv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, kv * G), dtype=torch.float64, device="cuda")
    for first, n in zip(s["start_host"][:-1].tolist(), _lengths(c).tolist()):
        for h in range(kv):
            K = s["k"][first:first + n, h * D:(h + 1) * D].double()
            V = s["v"][first:first + n, h * D:(h + 1) * D].double()
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                q = s["q"][first + r0:first + r1].double().view(r1 - r0, -1, D)[:, h * G:(h + 1) * G].transpose(0, 1)
                sees = torch.ones((r1 - r0, r1), dtype=torch.bool, device="cuda").tril(r0)
                o, z = _softmax_exact(q, K[:r1], V[:r1], sees)
                out[first + r0:first + r1, h * G:(h + 1) * G] = o.transpose(0, 1)
                lse[first + r0:first + r1, h * G:(h + 1) * G] = z.T
    return out.view(rows, -1), lse


def _tree_exact(s):
    c = s["case"]
    kv, G, D = c["n_kv"], c["group"], c["D"]
    rows = s["q"].shape[0]
    out = torch.zeros((rows, kv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, kv * G), dtype=torch.float64, device="cuda")
    masks = s["mask"].cpu().numpy().view(np.uint64)
    for r, (n, nodes) in enumerate(zip(_lengths(c).tolist(), _nodes(c).tolist())):
        if nodes == 0:
            continue
        first = int(s["start_host"][r])
        sees = np.ones((nodes, n), dtype=bool)
        for i in range(nodes):
            for k in range(nodes):
                sees[i, n - nodes + k] = (int(masks[first + i]) >> k) & 1
        sees = torch.from_numpy(sees).cuda()
        pages = s["table"][r, :n, c["layers"] - 1].long()
        for h in range(kv):
            K = s["pool"][pages[:, 0], h * D:(h + 1) * D].double()
            V = s["pool"][pages[:, 1], h * D:(h + 1) * D].double()
            q = s["q"][first:first + nodes].double().view(nodes, -1, D)[:, h * G:(h + 1) * G].transpose(0, 1)
            o, z = _softmax_exact(q, K, V, sees)
            out[first:first + nodes, h * G:(h + 1) * G] = o.transpose(0, 1)
            lse[first:first + nodes, h * G:(h + 1) * G] = z.T
    return out.view(rows, -1), lse


def _append_exact(s):
    c = s["case"]
    table, pages = s["table"].cpu().numpy(), s["pages"].cpu().numpy()
    if c["cached"] < 0:
        table = np.full_like(table, -1)
    old = _old_lengths(c)
    new_len, start = np.zeros(c["n_req"], np.int32), np.zeros(c["n_req"] + 1, np.int32)
    row_req, row_pos = np.full(s["rows"], -1, np.int32), np.zeros(s["rows"], np.int32)
    t = 0
    for r, n in enumerate(_lengths(c).tolist()):
        o = int(old[r])
        table[r, o:o + n] = pages[t:t + n]
        row_req[t:t + n] = r
        row_pos[t:t + n] = np.arange(o, o + n)
        new_len[r] = o + n
        t += n
        start[r + 1] = t
    return tuple(torch.from_numpy(x).cuda() for x in (table, new_len, start, row_req, row_pos))
