"""Error bounds of the attentions over a KV cache against their fp64 oracles."""
import numpy as np


def attention_tolerances(ref, lengths, D):
    """Error bounds per request from the arithmetic (u = 2^-24, half a step of fp32).

    A score is a sum of D exact products in fp32, scaled once: off by at most
    delta = (D + 4) u mag + 4 u |s| <= (D + 8) u mag.  exp2 adds 2^-22, sums over n tokens n u, and a
    weight held in two bf16 terms 2^-16, so p is off by at most p (2 delta + (n + 8) u + 2^-22 + 2^-16).
    Token weights come out in fp32, which holds nothing between 0 and its smallest numbers: each
    head's term may be off by the smallest normal number, 2^-126, besides."""
    u = 2.0 ** -24
    tol_out, tol_lse, tol_w = [], [], []
    for i, n in enumerate(lengths):
        delta = (D + 8) * u * ref["mag"][i]                                     # per query head
        rel = 2 * delta + (n + 8) * u + 2.0 ** -22 + 2.0 ** -16
        tol_out.append(2.0 ** -8 * np.abs(ref["out"][i]) + np.repeat(rel, D) * ref["vabs"][i] * 1.01 + 1e-30)
        lse = np.where(np.isfinite(ref["lse"][i]), ref["lse"][i], 0.0)
        tol_lse.append(delta + (n + 8) * u + 2.0 ** -22 + 8 * u * np.abs(lse) + 8 * u)
        tol_w.append((ref["p"][i] * (2 * delta + (n + 8) * u + 2.0 ** -20)[:, None]).sum(0) if n else np.zeros(0))
    return np.array(tol_out), np.array(tol_lse), tol_w


def row_tolerances(ref, D):
    """Error bounds of prompt and tree attention (oracle.attention_prompt, attention_tree), per row, from the
    arithmetic.  w = 2^-23 is a step of fp32: the tensor cores cut their sums instead of rounding them.

    A score is a sum of D exact products, scaled once: off by at most delta = (D + 8) w mag.  exp2 adds 2^-22,
    sums over n tokens n w (running rescalings among them), and a weight enters the V product as bf16, off by
    half a step, 2^-8; the sum of the weights takes them unrounded.  So |out| is off by at most
    (2 delta + (n + 8) w + 2^-21 + 2^-8) sum p|V|, and its own rounding 2^-8 |out| (of the value as computed:
    a factor 1.01 covers the product of both).  lse: delta + (n + 8) w + 2^-21, and a few steps of its value."""
    w = 2.0 ** -23
    delta = (D + 8) * w * ref["mag"]
    rel = 2 * delta + (ref["n"][:, None] + 8) * w + 2.0 ** -21
    tol_out = 1.01 * (2.0 ** -8 * np.abs(ref["out"]) + np.repeat(rel + 2.0 ** -8, D, axis=1) * ref["vabs"]) + 1e-30
    lse = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
    return tol_out, delta + (ref["n"][:, None] + 8) * w + 2.0 ** -21 + 8 * w * np.abs(lse)
