"""Attention over a paged cache in float64 with a bound per row from what that row itself sees."""
import numpy as np

import oracle.paged as OP


def attend(q, c, scale, window=0, sink=None, out_eps=0.0, table=None):
    """(out, tol) [T, heads, D] float64 of queries q over the case c (paged_testlib.make's dict).  How far a value may
    be off, all of it relative to the row's own softmax weights w and values:

    per weight 2^-11, its rounding to fp16, and 2^-15 for exp2, its argument's and the sums' rounding (arguments of
    up to 2^7 in log2 units are held to 2^-17; a factor of w each); per score 2^-16 of max|q| * reach (see
    paged_testlib.bound), which moves a weight and the denominator.  What a row's weights are rounded to stays 11 bits
    down to 2^-25 of its largest w * v_scale and is 2^-36 of that off below: times the largest code, 448, per token.
    A scale below 2^-100 counts as 2^-100."""
    val = OP.e4m3_values()
    T, heads, D = q.shape
    H, page = c["k"].shape[1], c["k"].shape[2]
    G = heads // H
    table = c["table"] if table is None else table
    out, tol = np.zeros((T, heads, D)), np.zeros((T, heads, D))
    for b, L in enumerate(c["kv"]):
        r0, r1 = int(c["row_start"][b]), int(c["row_start"][b + 1])
        L = int(L)
        if r0 == r1:
            continue
        ids = table[b, :-(-L // page)]
        for h in range(H):
            k = (val[c["k"][ids, h]] * c["ks"][ids, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            vs = np.repeat(c["vs"][ids, h].astype(np.float64), page)[:L]
            code = val[c["v"][ids, h]].reshape(-1, D)[:L]
            for r in range(r0, r1):
                p = L - (r1 - r0) + r - r0
                lo = max(0, p - window + 1) if window else 0
                if p < lo:
                    continue
                kk, cc, s = k[lo:p + 1], code[lo:p + 1], vs[lo:p + 1]
                heads_of = slice(h * G, (h + 1) * G)
                z = q[r, heads_of].astype(np.float64) @ kk.T * scale
                sk = np.full(G, -np.inf) if sink is None else sink[heads_of].astype(np.float64)
                top = np.maximum(z.max(-1), sk)
                e = np.exp(z - top[:, None])
                w = e / (e.sum(-1) + np.exp(sk - top))[:, None]
                out[r, heads_of] = (w * s) @ cc
                dz = 2.0 ** -16 * np.abs(q[r, heads_of]).max(-1) * abs(scale) * np.abs(kk).sum(-1).max()
                tol[r, heads_of] = ((w * s) @ np.abs(cc) * (2.0 ** -11 + 2.0 ** -15 + 2 * dz[:, None])
                                    + 448 * (len(s) * 2.0 ** -36 * (w * np.maximum(s, 2.0 ** -100)).max(-1)[:, None] + 2.0 ** -100)
                                    + out_eps * np.abs(out[r, heads_of]))
    return out, tol
