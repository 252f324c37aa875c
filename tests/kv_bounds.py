"""Error bounds of split decode attention against the fp64 oracle (oracle.attention_split)."""
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
