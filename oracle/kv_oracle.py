"""CPU oracle of the KV-cache operators: split decode attention with token weights, eviction, attention of
packed prompts and of drafted trees, and slot maps.

Test infrastructure only; fp64 NumPy from the definitions, sharing no code with the library.
"""
from __future__ import annotations

from typing import Sequence

import numpy as np

from .lora_oracle import bf16_to_f64


def attention_split(pool_bits, kv_tables: Sequence[np.ndarray], q_bits, n_heads: int, n_kv_heads: int):
    """One new token per request over its cached tokens, query head h reading KV head
    h // (n_heads // n_kv_heads).  Returns dict of fp64 arrays: out [n_req, n_heads * D], lse
    [n_req, n_heads] (-inf for an empty request) and lists per request: weight [tokens] (summed
    over query heads), p [n_heads, tokens], and what error bounds need: mag [n_heads], the largest
    sum_d |q_d K_jd| / sqrt(D), and vabs [n_heads * D], sum_j p_j |V_j|."""
    q_all = bf16_to_f64(q_bits)
    n_req = q_all.shape[0]
    H = pool_bits.H if hasattr(pool_bits, "H") else pool_bits.shape[1]
    D, G = H // n_kv_heads, n_heads // n_kv_heads
    res = {"out": np.zeros((n_req, n_heads * D)), "lse": np.full((n_req, n_heads), -np.inf), "weight": [], "p": [],
           "mag": np.zeros((n_req, n_heads)), "vabs": np.zeros((n_req, n_heads * D))}
    for i in range(n_req):
        tab = np.asarray(kv_tables[i], dtype=np.int64).reshape(-1, 2)
        n = tab.shape[0]
        p_all = np.zeros((n_heads, n))
        if n:
            K = bf16_to_f64(pool_bits[tab[:, 0]]).reshape(n, n_kv_heads, D)
            V = bf16_to_f64(pool_bits[tab[:, 1]]).reshape(n, n_kv_heads, D)
            q = q_all[i].reshape(n_heads, D)
            for h in range(n_heads):
                k, v, cols = K[:, h // G], V[:, h // G], slice(h * D, (h + 1) * D)
                s = k @ q[h] / np.sqrt(D)
                e = np.exp(s - s.max())
                p_all[h] = e / e.sum()
                res["lse"][i, h] = s.max() + np.log(e.sum())
                res["out"][i, cols] = p_all[h] @ v
                res["mag"][i, h] = (np.abs(k) @ np.abs(q[h])).max() / np.sqrt(D)
                res["vabs"][i, cols] = p_all[h] @ np.abs(v)
        res["p"].append(p_all)
        res["weight"].append(p_all.sum(0))
    return res


def evict_keep(weight, n: int, budget: int, recent: int) -> list:
    """Positions (ascending) of one request's n tokens that stay at one layer: the newest
    min(n, recent), and the heaviest older ones up to min(n, budget) in all; equal weights keep the
    lowest index, NaN counts as -infinity."""
    new = list(range(n - min(n, recent), n))
    old = sorted(range(n - len(new)), key=lambda j: (-(float(weight[j]) if weight[j] == weight[j] else -np.inf), j))
    return sorted(old[:min(n, budget) - len(new)] + new)


def _attend_rows(q, K, V, sees, res, rows, n_heads: int, n_kv: int):
    """Rows q [R, n_heads * D] over tokens K, V [n, n_kv * D] that each sees (bool [R, n]); what a row does not
    see plays no part, whatever it holds."""
    D, G = K.shape[1] // n_kv, n_heads // n_kv
    finite = np.isfinite(V).all()
    for h in range(n_heads):
        k, v = K[:, h // G * D:(h // G + 1) * D], V[:, h // G * D:(h // G + 1) * D]
        qh, cols = q[:, h * D:(h + 1) * D], slice(h * D, (h + 1) * D)
        with np.errstate(invalid="ignore", over="ignore"):
            s = np.where(sees, qh @ k.T / np.sqrt(D), -np.inf)
            mag = np.where(sees, np.abs(qh) @ np.abs(k).T / np.sqrt(D), 0.0)
            top = s.max(axis=1, initial=-np.inf)
            some = ~np.isneginf(top)
            e = np.where(sees, np.exp(s - np.where(some, top, 0.0)[:, None]), 0.0)
            total = e.sum(1)
            p = e / np.where(some, total, 1.0)[:, None]
            res["lse"][rows, h] = np.where(some, top + np.log(np.where(some, total, 1.0)), -np.inf)
            res["mag"][rows, h] = mag.max(axis=1, initial=0.0)
            if finite:
                res["out"][rows, cols] = p @ v
                res["vabs"][rows, cols] = p @ np.abs(v)
            else:
                for i, row in enumerate(range(*rows.indices(res["out"].shape[0]))):
                    at = np.flatnonzero(sees[i]) if some[i] else []
                    res["out"][row, cols] = (p[i, at, None] * v[at]).sum(0)
                    res["vabs"][row, cols] = (p[i, at, None] * np.abs(v[at])).sum(0)
    res["n"][rows] = sees.sum(1)


def _rows_result(n_rows: int, n_heads: int, D: int) -> dict:
    """out, lse, and what error bounds need: mag [rows, heads], the largest sum_d |q_d K_jd| / sqrt(D) of the
    tokens seen, vabs, sum_j p_j |V_j|, and n, the tokens seen.  Rows of no sequence stay NaN."""
    return {"out": np.full((n_rows, n_heads * D), np.nan), "lse": np.full((n_rows, n_heads), np.nan),
            "mag": np.zeros((n_rows, n_heads)), "vabs": np.zeros((n_rows, n_heads * D)), "n": np.zeros(n_rows, np.int64)}


def attention_prompt(q_bits, k_bits, v_bits, starts: Sequence[int], n_heads: int, n_kv_heads: int) -> dict:
    """Causal attention of packed sequences, rows [starts[s], starts[s + 1]) each."""
    q, k, v = (bf16_to_f64(x) for x in (q_bits, k_bits, v_bits))
    res = _rows_result(q.shape[0], n_heads, k.shape[1] // n_kv_heads)
    for a, b in zip(starts[:-1], starts[1:]):
        if b > a:
            _attend_rows(q[a:b], k[a:b], v[a:b], np.tri(b - a, dtype=bool), res, slice(a, b), n_heads, n_kv_heads)
    return res


def attention_tree(pool_bits, kv_tables: Sequence[np.ndarray], starts: Sequence[int], masks, q_bits, n_heads: int,
                   n_kv_heads: int, skip: Sequence = ()) -> dict:
    """Drafted nodes, the last cached tokens of their request, under their masks (any integers, bit j = node j);
    skip: (request, position) pairs that count as not cached."""
    q = bf16_to_f64(q_bits)
    H = pool_bits.shape[1]
    res = _rows_result(q.shape[0], n_heads, H // n_kv_heads)
    for r, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        if b <= a:
            continue
        tab = np.asarray(kv_tables[r], dtype=np.int64).reshape(-1, 2)
        n, m = tab.shape[0], b - a
        base = max(n - m, 0)
        sees = np.ones((m, n), dtype=bool)
        for i in range(m):
            for j in range(base, n):
                sees[i, j] = (int(masks[a + i]) >> (j - base)) & 1
        for request, j in skip:
            if request == r and j < n:
                sees[:, j] = False
        K, V = bf16_to_f64(pool_bits[tab[:, 0]]).reshape(n, H), bf16_to_f64(pool_bits[tab[:, 1]]).reshape(n, H)
        _attend_rows(q[a:b], K, V, sees, res, slice(a, b), n_heads, n_kv_heads)
    return res


def kv_append(count: Sequence[int], old_len: Sequence[int], pages, table, row_cap: int):
    """New tokens behind the cached ones: (table, new_len, row_start, row_req, row_pos); pages [row_cap, layers, 2]
    in row order, table [n_req, max_len, layers, 2] as it was before.  Tokens past max_len and rows past row_cap
    are dropped, negative counts are 0, old lengths are clamped."""
    table = np.array(table)
    max_len = table.shape[1]
    new_len, start = [], [0]
    row_req, row_pos = np.full(row_cap, -1, np.int32), np.zeros(row_cap, np.int32)
    t = 0
    for r, c in enumerate(count):
        old = min(max(int(old_len[r]), 0), max_len)
        held = 0
        for i in range(max(int(c), 0)):
            if t >= row_cap:
                t += int(c) - i
                break
            held += 1
            if old + i < max_len:
                table[r, old + i] = pages[t]
                row_req[t], row_pos[t] = r, old + i
            t += 1
        new_len.append(min(old + held, max_len))
        start.append(min(t, row_cap))
    return table, np.array(new_len, np.int32), np.array(start, np.int32), row_req, row_pos
