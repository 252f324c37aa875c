"""CPU oracle of the KV-cache operators: split decode attention with token weights, and eviction.

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
