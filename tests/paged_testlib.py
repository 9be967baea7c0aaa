"""Inputs of the paged cache's tests: batches of ragged sequences over a fragmented page pool whose
unused slots hold E4M3's NaN codes and whose unused pages have NaN scales."""
import numpy as np
import torch

import oracle.paged as OP

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def values(shape, rng, dtype, spread=1.0):
    """A tensor of the type and its values in float64."""
    t = torch.from_numpy((rng.standard_normal(shape) * spread).astype(np.float32)).to(TYPES[dtype])
    return t, t.double().numpy()


def make(new, kv, page, H, D, seed, exps=(-9, -4)):
    """Sequences with new[b] of kv[b] tokens new (kv may be smaller): plan arrays, table and cache in
    numpy."""
    rng = np.random.default_rng(seed)
    new, kv = np.asarray(new, np.int32), np.asarray(kv, np.int32)
    held = -(-kv // page)
    pages = int(held.sum()) + 2
    ids = rng.permutation(pages).astype(np.int32)
    cols = max(1, int(held.max(initial=0))) + 1
    table = np.full((len(kv), cols), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    k = np.full((pages, H, page, D), 0x7F, np.uint8)
    v = np.full((pages, H, page, D), 0xFF, np.uint8)
    ks, vs = np.full((pages, H), np.nan, np.float32), np.full((pages, H), np.nan, np.float32)
    for b in range(len(kv)):
        for j in range(held[b]):
            g, n = table[b, j], min(page, kv[b] - j * page)
            for c, s in ((k, ks), (v, vs)):
                c[g, :, :n] = OP.e4m3_codes(rng.standard_normal((H, n, D)) * 70)
                s[g] = 2.0 ** rng.integers(*exps, H)
    row_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return {"new": new, "kv": kv, "table": table, "row_start": row_start, "rows": int(new.sum()), "k": k, "v": v,
            "ks": ks, "vs": vs, "page": page, "H": H, "D": D}


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bound(q, case, oracle, out_eps):
    """How far each output may be off.  Per weight: its rounding to fp16 (2^-11) and 2^-15 for exp2, the
    running sums and their joining; per score 2^-16 of max|q| * reach: the query's E4M3 pieces hold it to
    2^-17.8 of its row's maximum (as fp16, with few rows, to 2^-25), its at most 16 fp32 additions and three
    products to 2^-19.  A score's
    error moves a weight and the denominator, twice its size in all.  Weights below fp16's normal range
    are 2^-36 of the largest off at most.  Then the output's own rounding."""
    out, spread, reach = oracle
    amax = np.abs(q).max(-1)
    dz = 2.0 ** -16 * amax * reach
    top = float(np.nanmax(np.abs(case["vs"]), initial=0.0)) * 448
    n = int(case["kv"].max(initial=0))
    return spread * (2.0 ** -11 + 2.0 ** -15 + 2 * dz[..., None]) + 2.0 ** -36 * top * n + out_eps * np.abs(out)
