"""float64 oracle of the paged 8-bit cache: page plan, rotary axes, page writer, paged attention.
Plain loops over sequences, pages and rows; shares no code with the GPU path."""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The values of the 256 OCP E4M3 codes (0x7f and 0xff, the NaNs, included as NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 0x7F == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_GRID = e4m3_values()[:127]  # 0 .. 448 ascending with the code


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code of finite or infinite float64 values, ties to the even code, saturating;
    NaN gives 0."""
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.searchsorted(_GRID, a).clip(1, 126)
    lo = hi - 1
    dlo, dhi = a - _GRID[lo], _GRID[hi] - a
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def page_plan(ctx, new, table, free, page, max_rows):
    """(table, row_start, kv_len, seq_of_row, pos, slot, taken, complete)."""
    table = np.array(table)
    cols = table.shape[1]
    row_start, kv, seq, pos, slot, taken, ok = [0], [], [], [], [], 0, True
    for b, (c, n) in enumerate(zip(np.maximum(ctx, 0).tolist(), np.maximum(new, 0).tolist())):
        entry = {j: int(table[b, j]) for j in range(min(-(-c // page), cols))}
        for j in range(-(-c // page), -(-(c + n) // page)):
            entry[j] = int(free[taken]) if taken < len(free) else -1
            ok &= taken < len(free) and j < cols
            taken += 1
            if j < cols:
                table[b, j] = entry[j]
            else:
                entry[j] = -1
        for t in range(c, c + n):
            g = entry.get(t // page, -1)
            seq.append(b), pos.append(t), slot.append(g * page + t % page if g >= 0 else -1)
            ok &= g >= 0
        row_start.append(row_start[-1] + n), kv.append(c + n)
    ok &= len(seq) <= max_rows
    fill = [-1] * max(0, max_rows - len(seq))
    return (table, np.array(row_start), np.array(kv), np.array((seq + fill)[:max_rows]), np.array((pos + fill)[:max_rows]),
            np.array((slot + fill)[:max_rows]), taken, ok)


def rope_axes(x, pos, axis_of_pair, theta, rot_first=0, half=True, inverse=False):
    """x [T, H, D] float64 turned pair by pair.  The angle is reduced exactly: positions are integers
    and the frequency's turn per position is a float64, so their product is formed in Python integers."""
    out = np.array(x, dtype=np.float64)
    R = 2 * len(axis_of_pair)
    for i, a in enumerate(axis_of_pair):
        turn = float(theta) ** (-2.0 * i / R) / (2 * math.pi)
        num, den = turn.as_integer_ratio()
        frac = np.array([(int(p) * num % den) / den for p in pos[a]])
        ang = 2 * math.pi * frac * (-1 if inverse else 1)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        u, v = (i, i + R // 2) if half else (2 * i, 2 * i + 1)
        u, v = u + rot_first, v + rot_first
        p, q = out[..., u].copy(), out[..., v].copy()
        out[..., u], out[..., v] = p * c - q * s, p * s + q * c
    return out


def write_pages(codes, scale, x, row_start, kv_len, table):
    """One of the two caches after the write: codes [pages, H, page, D] uint8, scale [pages, H] float64."""
    codes, scale, val = np.array(codes), np.array(scale, dtype=np.float64), e4m3_values()
    page = codes.shape[2]
    for b in range(len(kv_len)):
        r, end = int(row_start[b]), int(row_start[b + 1])
        p = int(kv_len[b]) - (end - r)
        while r < end:
            n, o, g = min(page - p % page, end - r), p % page, int(table[b, p // page])
            for h in range(codes.shape[1]):
                part = x[r:r + n, h].astype(np.float64)
                peak = float(np.max(np.abs(part[np.isfinite(part)]), initial=0.0))
                e = -100
                while e < 119 and 448.0 * 2.0 ** e < peak:
                    e += 1
                need = 2.0 ** e
                nan = bool(np.isnan(part).any()) or bool(o and np.isnan(scale[g, h]))
                if o and not nan and scale[g, h] > need:
                    need = scale[g, h]
                if o and not nan and scale[g, h] < need:
                    codes[g, h, :o] = e4m3_codes(val[codes[g, h, :o]] * (scale[g, h] / need))
                codes[g, h, o:o + n] = e4m3_codes(part / need)
                scale[g, h] = np.nan if nan else need
            r, p = r + n, p + n
    return codes, scale


def paged_attn(q, k_codes, v_codes, k_scale, v_scale, row_start, kv_len, table, scale, window=0, sink=None):
    """(out, spread, reach): out [T, heads, D] float64; spread = sum_j weight_j |v_j| per value, reach =
    max_j softmax_scale * sum_d |k_jd| per row, the factors of the error bounds.  Rows of no sequence
    and rows without a key are 0."""
    val = e4m3_values()
    T, heads, D = q.shape
    H, page = k_codes.shape[1], k_codes.shape[2]
    G = heads // H
    out, spread, reach = np.zeros((T, heads, D)), np.zeros((T, heads, D)), np.zeros((T, heads))
    for b in range(len(kv_len)):
        r0, r1, L = int(row_start[b]), int(row_start[b + 1]), int(kv_len[b])
        if r1 <= r0:
            continue
        pages = [int(g) for g in table[b, :-(-L // page)]]
        for h in range(H):
            rows = [(val[k_codes[g, h]] * k_scale[g, h], val[v_codes[g, h]] * v_scale[g, h]) for g in pages]
            k = np.concatenate([a for a, _ in rows])[:L] if rows else np.zeros((0, D))
            v = np.concatenate([a for _, a in rows])[:L] if rows else np.zeros((0, D))
            for r in range(r0, min(r1, T)):
                p = L - (r1 - r0) + r - r0
                lo = max(0, p - window + 1) if window else 0
                if p < lo:
                    continue
                kk, vv = k[lo:p + 1], v[lo:p + 1]
                z = q[r, h * G:(h + 1) * G].astype(np.float64) @ kk.T * scale
                s = np.full(G, -np.inf) if sink is None else sink[h * G:(h + 1) * G].astype(np.float64)
                top = np.maximum(z.max(-1), s)
                e = np.exp(z - top[:, None])
                den = e.sum(-1) + np.exp(s - top)
                w = e / den[:, None]
                out[r, h * G:(h + 1) * G] = w @ vv
                spread[r, h * G:(h + 1) * G] = w @ np.abs(vv)
                reach[r, h * G:(h + 1) * G] = abs(scale) * np.abs(kk).sum(-1).max()
    return out, spread, reach
