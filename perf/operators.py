"""The operators of a paged 8-bit cache: page tables and slot maps from request lengths, rotary positions
with several axes, the cache writer, and attention over the cache - their cases, plain forms and
definitions in 64 bits.

A sequence's tokens live in pages of `page` tokens; its table row lists them.  Keys and values are E4M3
codes [pages, kv heads, page, dim] with one fp32 power-of-two scale per (page, kv head).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E_MIN, E_MAX = -100, 119  # exponents of a page's scale


def listed():
    return [
        # one decode step of 256 running requests: each appends a token, one in sixteen opens a page
        {"name": "plan_decode", "op": "plan", "seqs": 256, "new": 1, "ctx": 8191, "page": 16, "ragged": False},
        # prompts admitted together: some 130 thousand rows of 48 requests, none cached yet
        {"name": "plan_prompts", "op": "plan", "seqs": 48, "new": 5461, "ctx": 0, "page": 64, "ragged": True},
        # queries and keys of a small decode batch, plain text positions on three axes
        {"name": "rope_decode", "op": "rope", "tokens": 32, "heads": 72, "dim": 128, "rot": 128, "axes": 3,
         "pairing": "half", "inverse": False, "type": "bf16"},
        # queries and keys of a long prompt with images, time / height / width
        {"name": "rope_prompt", "op": "rope", "tokens": 16384, "heads": 40, "dim": 128, "rot": 128, "axes": 3,
         "pairing": "half", "inverse": False, "type": "bf16"},
        # the gradient of the same for heads of 192 with 64 rotary dims, adjacent pairs
        {"name": "rope_gradient", "op": "rope", "tokens": 4096, "heads": 33, "dim": 192, "rot": 64, "axes": 2,
         "pairing": "adjacent", "inverse": True, "type": "f32"},
        # 512 requests append one token each, in the middle of their pages
        {"name": "write_decode", "op": "write", "seqs": 512, "new": 1, "ctx": 100, "page": 16, "kv_heads": 8, "dim": 128,
         "ragged": True, "type": "bf16"},
        # a chunk of a long prompt: whole pages
        {"name": "write_prompt", "op": "write", "seqs": 4, "new": 8192, "ctx": 32768, "page": 64, "kv_heads": 8,
         "dim": 128, "ragged": False, "type": "bf16"},
        # the tiny decode's length: one request, where latency counts
        {"name": "attn_one", "op": "attn", "seqs": 1, "new": 1, "ctx": 2047, "page": 64, "heads": 64, "kv_heads": 8,
         "dim": 128, "window": 0, "sink": False, "ragged": False, "type": "bf16"},
        # the batched decode's length: 32 requests of 65,536 tokens
        {"name": "attn_batch", "op": "attn", "seqs": 32, "new": 1, "ctx": 65535, "page": 64, "heads": 64, "kv_heads": 8,
         "dim": 128, "window": 0, "sink": False, "ragged": False, "type": "bf16"},
        # the long-context decode's length, one shared head, small pages, a sink
        {"name": "attn_long", "op": "attn", "seqs": 4, "new": 1, "ctx": 1048575, "page": 16, "heads": 16, "kv_heads": 1,
         "dim": 128, "window": 0, "sink": True, "ragged": False, "type": "bf16"},
        # a few drafted tokens of many ragged requests under a sliding window
        {"name": "attn_drafts", "op": "attn", "seqs": 96, "new": 5, "ctx": 9000, "page": 32, "heads": 24, "kv_heads": 8,
         "dim": 64, "window": 1024, "sink": True, "ragged": True, "type": "f16"},
        # the prefill chunk: 4,096 new tokens behind 32,768 cached ones
        {"name": "attn_chunk", "op": "attn", "seqs": 1, "new": 4096, "ctx": 32768, "page": 64, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0, "sink": False, "ragged": False, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "write", "attn", "attn", "attn"])
    if op == "plan":
        seqs = _log(rng, 1, 2048)
        return {"op": op, "seqs": seqs, "new": _log(rng, 1, max(1, 120000 // seqs)), "ctx": rng.choice([0, _log(rng, 1, 30000)]),
                "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.7}
    if op == "rope":
        dim = rng.choice([64, 128, 192, 256])
        rot = rng.choice([dim, dim // 2])
        return {"op": op, "tokens": _log(rng, 1, 14000), "heads": rng.randint(1, 40), "dim": dim, "rot": rot,
                "axes": rng.randint(1, 4), "pairing": rng.choice(["half", "adjacent"]), "inverse": rng.random() < 0.4,
                "type": rng.choice(["bf16", "f16", "f32"])}
    page, dim = rng.choice([16, 32, 64, 128]), rng.choice([64, 128])
    if op == "write":
        seqs = _log(rng, 1, 600)
        return {"op": op, "seqs": seqs, "new": _log(rng, 1, max(1, 20000 // seqs)), "ctx": rng.choice([0, _log(rng, 1, 4000)]),
                "page": page, "kv_heads": rng.choice([1, 2, 4, 8, 11]), "dim": dim, "ragged": rng.random() < 0.7,
                "type": rng.choice(["bf16", "f16", "f32"])}
    kv_heads = rng.choice([1, 2, 4, 8])
    case = {"op": op, "page": page, "kv_heads": kv_heads, "heads": kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 16]), "dim": dim,
            "window": rng.choice([0, 0, _log(rng, 16, 4000)]), "sink": rng.random() < 0.4, "ragged": rng.random() < 0.7,
            "type": rng.choice(["bf16", "f16"])}
    if rng.random() < 0.6:  # a decode step, some with drafts
        seqs = _log(rng, 1, 256)
        case |= {"seqs": seqs, "new": rng.choice([1, 1, 1, 2, 4]), "ctx": _log(rng, 1, min(200000, 1500000 // seqs))}
    else:  # prompts, some behind a cached part
        seqs = rng.randint(1, 6)
        case["heads"] = min(case["heads"], kv_heads * max(1, 32 // kv_heads))
        new = _log(rng, 17, 2400)
        room = int(2.4e9 / (case["heads"] * seqs * new)) - new  # no more work than the prefill chunk
        case |= {"seqs": seqs, "new": new, "ctx": rng.choice([0, min(room, _log(rng, 1, 12000))])}
    return case


# ---------------------------------------------------------------------------- inputs
def _lengths(case):
    """New and cached lengths: `new` and `ctx`, or spread around them where the batch is ragged.  They are the
    case's own; a seed only changes their order."""
    n = case["seqs"]
    new, ctx = torch.full((n,), case["new"]), torch.full((n,), case["ctx"])
    if case["ragged"]:
        gen = torch.Generator().manual_seed(n)
        new = 1 + (torch.rand(n, generator=gen) * (2 * new - 1)).long()
        ctx = (torch.rand(n, generator=gen) * (2 * ctx + 1)).long()
    return new.int(), ctx.int()


def _layout(case, gen):
    """The pages of a fragmented pool: the table with the cached tokens' pages, and the free list."""
    page = case["page"]
    new, ctx = _lengths(case)
    order = torch.randperm(case["seqs"], generator=gen)
    new, ctx = new[order], ctx[order]
    held, full = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    width, total = int(full.max()), int(full.sum())
    ids = torch.randperm(total + 3, generator=gen).int()
    table = torch.full((case["seqs"], width), -1, dtype=torch.int32)
    table[torch.arange(width) < held[:, None]] = ids[: int(held.sum())]
    return {"new": new.to(DEV), "ctx": ctx.to(DEV), "table": table.to(DEV), "free": ids[int(held.sum()):].to(DEV),
            "rows": int(new.sum()), "pages": total + 3}


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(DEV).manual_seed(seed)

    def codes(shape):
        """E4M3 codes of normal values that fill the range as a writer leaves them."""
        out = torch.empty(shape, dtype=torch.uint8, device=DEV)
        flat = out.view(-1)
        for a in range(0, flat.numel(), 1 << 27):
            part = flat[a:a + (1 << 27)]
            x = torch.empty(part.shape, device=DEV).normal_(0, 70, generator=gen).clamp_(-448, 448)
            part.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
        return out

    s = {"case": case}
    op = case["op"]
    if op == "rope":
        T, A, R = case["tokens"], case["axes"], case["rot"]
        s["x"] = torch.empty((T, case["heads"], case["dim"]), device=DEV).normal_(generator=gen).to(TYPES[case["type"]])
        s["pos"] = torch.randint(0, 200000, (A, T), generator=gen, device=DEV)
        cut = [R // 2 * (i + 1) // A for i in range(A)]
        s["sections"] = [b - a for a, b in zip([0] + cut, cut)]
    else:
        s |= _layout(case, cpu)
    if op in ("write", "attn"):
        page, H, D = case["page"], case["kv_heads"], case["dim"]
        s["k"], s["v"] = (codes((s["pages"], H, page, D)) for _ in range(2))
        s["ks"], s["vs"] = (torch.exp2(torch.randint(-8, -5, (s["pages"], H), generator=gen, device=DEV).float())
                            for _ in range(2))
        s["plan"] = _plain_plan(s["ctx"], s["new"], s["table"], s["free"], page, s["rows"])
        s["table"] = s["plan"][0]
        if op == "write":
            s["xk"], s["xv"] = (torch.empty((s["rows"], H, D), device=DEV).normal_(generator=gen).to(TYPES[case["type"]])
                                for _ in range(2))
        else:
            s["q"] = torch.empty((s["rows"], case["heads"], D), device=DEV).normal_(generator=gen).to(TYPES[case["type"]])
            s["sink"] = torch.empty(case["heads"], device=DEV).normal_(generator=gen) if case["sink"] else None
    return s


def _own(s):
    """The prepared call that a serving loop makes once for its buffers and keeps."""
    import sparse_attention_csa2_gb300 as S
    case = s["case"]
    if case["op"] == "plan":
        return S.PagePlan(s["ctx"], s["new"], s["table"], s["free"], case["page"], s["rows"])
    if case["op"] == "rope":
        return S.RopeAxes(s["x"], s["pos"], sections=s["sections"], theta=10000.0, rot_dim=case["rot"],
                          pairing=case["pairing"], inverse=case["inverse"])
    table, row_start, kv_len, seq_of_row = s["plan"][:4]
    cache = S.PageCache(s["k"], s["v"], s["ks"], s["vs"])
    if case["op"] == "write":
        return S.PageWriter(cache, s["xk"], s["xv"], row_start, kv_len, seq_of_row, table)
    return S.PagedAttn(s["q"], cache, row_start, kv_len, table, softmax_scale=case["dim"] ** -0.5, window=case["window"],
                       sink=s["sink"])


# ---------------------------------------------------------------------------- passes
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        c = s.get("call") or s.setdefault("call", _own(s))
        c()
        if op == "plan":
            return [s["table"], c.row_start, c.kv_len, c.seq_of_row, c.pos, c.slot, c.n_taken]
        if op == "write":
            return [s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn), s["ks"], s["vs"]]
        return [c.out]
    if op == "plan":
        s["table"], *rest = _plain_plan(s["ctx"], s["new"], s["table"], s["free"], case["page"], s["rows"])
        return [s["table"], *rest]
    if op == "rope":
        return [_plain_rope(s["x"], s["pos"], s["sections"], case["rot"], case["pairing"], case["inverse"])]
    if op == "write":
        _plain_write(s["k"], s["ks"], s["xk"], s["plan"], case["page"])
        _plain_write(s["v"], s["vs"], s["xv"], s["plan"], case["page"])
        return [s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn), s["ks"], s["vs"]]
    return [_plain_attn(s)]


def _plain_plan(ctx, new, table, free, page, rows):
    dev = ctx.device
    held, full = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = full - held
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=dev)
    fresh = (col >= held[:, None]) & (col < full[:, None])
    take = (first[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[take], table)
    row_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(new, 0)]).int()
    r = torch.arange(rows, device=dev)
    seq = torch.searchsorted(row_start, r.int(), right=True, out_int32=True) - 1
    pos = ctx[seq].long() + r - row_start[seq]
    slot = table[seq.long(), pos // page].long() * page + pos % page
    return table, row_start, ctx + new, seq, pos, slot, need.sum().int().reshape(1)


def _plain_rope(x, pos, sections, rot, pairing, inverse):
    half = rot // 2
    axis = torch.cat([torch.full((n,), a, device=x.device) for a, n in enumerate(sections)])
    freq = 10000.0 ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / rot)
    angle = pos[axis].T.double() * freq  # [T, half], in 64 bits: 32 lose the angle of a far position
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    y = x.float()
    a, b = (y[..., :half], y[..., half:rot]) if pairing == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    turned = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.cat(turned, -1) if pairing == "half" else torch.stack(turned, -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_write(codes, scales, x, plan, page):
    """One of the two caches: the scale of each touched (page, head), its older tokens, its new ones."""
    table, row_start, kv_len, seq, pos, slot, _ = plan
    x = x.float()
    page_of, off = slot // page, slot % page
    peak = torch.zeros(scales.shape, device=x.device).index_reduce_(0, page_of, x.abs().amax(-1), "amax")
    m, e = torch.frexp(peak / 448)  # peak / 448 = m * 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)
    need = torch.where(peak > 0, torch.exp2(e.float()), 2.0 ** E_MIN)
    # the pages that a sequence's older tokens share with its new ones
    ctx = kv_len - (row_start[1:] - row_start[:-1])
    shared = ctx % page > 0
    old_page = torch.where(shared, table.gather(1, (ctx // page).clamp(max=table.shape[1] - 1)[:, None].long())[:, 0], 0).long()
    old_scale = scales[old_page]
    old = codes[old_page].view(torch.float8_e4m3fn).float()
    scales[page_of] = need[page_of]
    grown = torch.maximum(old_scale, need[old_page])
    again = (old * (old_scale / grown)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = shared[:, None, None, None] & (torch.arange(page, device=x.device) < (ctx % page)[:, None])[:, None, :, None]
    b, h, t, d = torch.nonzero(keep.expand(again.shape), as_tuple=True)
    codes[old_page[b], h, t, d] = again[b, h, t, d]
    scales[old_page[shared]] = grown[shared]
    codes[page_of, :, off] = (x / scales[page_of][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_attn(s):
    case = s["case"]
    table, row_start, kv_len = s["plan"][:3]
    q, H, D, page = s["q"], case["kv_heads"], case["dim"], case["page"]
    n, P = table.shape
    G = q.shape[1] // H
    at = table.clamp(min=0).long()

    def rows(codes, scales):  # [n, H, P * page, D]
        x = codes[at].view(torch.float8_e4m3fn).float() * scales[at][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(n, H, P * page, D)

    new = row_start[1:] - row_start[:-1]
    most = -(-s["rows"] // n) if not case["ragged"] else int(2 * case["new"])  # no sequence has more new rows
    i = torch.arange(most, device=q.device)
    src = (row_start[:-1, None] + i).clamp(max=s["rows"] - 1).long()
    qp = q.float()[src].reshape(n, most, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * most, D)
    z = (qp @ rows(s["k"], s["ks"]).transpose(2, 3) * D ** -0.5).reshape(n, H, G, most, P * page)
    j = torch.arange(P * page, device=q.device)
    p = (kv_len - new)[:, None] + i
    seen = j <= p[..., None]
    if case["window"]:
        seen &= j > p[..., None] - case["window"]
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].reshape(H, G, 1, 1)
        top = torch.maximum(top, sink)
    z = z.sub_(top).exp_()
    den = z.sum(-1, keepdim=True)
    if s["sink"] is not None:
        den = den + (sink - top).exp()
    o = (z.reshape(n, H, G * most, P * page) @ rows(s["v"], s["vs"])).reshape(n, H, G, most, D) / den
    out = o.permute(0, 3, 1, 2, 4).reshape(n * most, H * G, D)
    seq = s["plan"][3].long()
    r = torch.arange(s["rows"], device=q.device)
    return out[seq * most + r - row_start[seq]].to(q.dtype)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}.get(case.get("type"), 0)
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * size * n + 8 * case["axes"] * case["tokens"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    new, ctx = (x.double() for x in _lengths(case))
    rows, page = int(new.sum()), case["page"]
    if op == "plan":
        fresh = int((torch.ceil((ctx + new) / page) - torch.ceil(ctx / page)).sum())
        return {"bytes": 16 * case["seqs"] + 20 * rows + 8 * fresh, "flops": 4 * rows + 8 * case["seqs"]}
    H, D = case["kv_heads"], case["dim"]
    if op == "write":
        pages = int((torch.ceil((ctx + new) / page) - torch.floor(ctx / page)).sum())
        return {"bytes": 2 * rows * H * D * (size + 1) + 8 * pages * H + 16 * rows, "flops": 4 * rows * H * D}
    W = case["window"] or 1 << 40
    first, last = ctx + 1, ctx + new  # keys of the first and of the last new row, before the window
    short = (torch.clamp(last, max=W) - first + 1).clamp(min=0)  # rows with fewer keys than the window has
    keys = float((short * (first + torch.clamp(last, max=W)) / 2 + (new - short) * W).sum())
    span = torch.minimum(last, W + new - 1)
    pages = float((torch.ceil(span / page)).sum())
    return {"bytes": int(2 * float(span.sum()) * H * D + 2 * size * rows * case["heads"] * D + 8 * H * pages),
            "flops": int(4 * keys * case["heads"] * D)}


# ---------------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    def value_table():
        """The 256 values of E4M3 in 64 bits (the two NaN codes aside)."""
        v = []
        for c in range(256):
            e, m = c >> 3 & 15, c & 7
            x = (m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
            v.append(-x if c & 128 else x)
        return torch.tensor(v, dtype=torch.float64, device=DEV)

    def round_e4m3(x):
        """Nearest E4M3 value of 64-bit numbers within the range, ties to the even code."""
        _, e = torch.frexp(x)  # |x| in [2^(e-1), 2^e): steps of 2^(e-1-3), at least 2^-9
        step = torch.exp2((e - 4).clamp(min=-9).double())
        return torch.round(x / step).mul_(step).clamp_(-448, 448)

    def of_plan(s):
        page = s["case"]["page"]
        table, free = s["table"].cpu(), s["free"].cpu().tolist()
        row_start, kv_len, seq, pos, slot, taken = [0], [], [], [], [], 0
        for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
            row = table[b].tolist()
            for i in range(-(-c // page), -(-(c + n) // page)):
                row[i], taken = free[taken], taken + 1
            table[b] = torch.tensor(row, dtype=torch.int32)
            p = torch.arange(c, c + n)
            seq.append(torch.full((n,), b, dtype=torch.int32))
            pos.append(p)
            slot.append(torch.tensor(row)[p // page].long() * page + p % page)
            row_start.append(row_start[-1] + n)
            kv_len.append(c + n)
        i32 = torch.int32
        return [table, torch.tensor(row_start, dtype=i32), torch.tensor(kv_len, dtype=i32), torch.cat(seq), torch.cat(pos),
                torch.cat(slot), torch.tensor([taken], dtype=i32)]

    def of_rope(s):
        case, x = s["case"], s["x"]
        rot = case["rot"]
        out = x.double().clone()
        i = 0
        for a, n in enumerate(s["sections"]):
            for _ in range(n):
                f = math.exp(-2.0 * i / rot * math.log(10000.0))
                t = s["pos"][a].double() * f * (-1 if case["inverse"] else 1)
                c, w = t.cos()[:, None], t.sin()[:, None]
                u, v = (i, i + rot // 2) if case["pairing"] == "half" else (2 * i, 2 * i + 1)
                p, q = x[..., u].double(), x[..., v].double()
                out[..., u], out[..., v] = p * c - q * w, p * w + q * c
                i += 1
        return [out]

    def of_write(s):
        case, value = s["case"], value_table()
        page = case["page"]
        table, row_start, kv_len = s["plan"][:3]
        outs, scales = [], []
        for codes, scale, x in ((s["k"], s["ks"], s["xk"]), (s["v"], s["vs"], s["xv"])):
            c, z, x = value[codes.long()], scale.double().clone(), x.double()
            starts, tab = row_start.tolist(), table.cpu().tolist()
            for b, kv in enumerate(kv_len.tolist()):
                r, end = starts[b], starts[b + 1]
                p = kv - (end - r)
                while r < end:
                    n, o, g = min(page - p % page, end - r), p % page, tab[b][p // page]
                    part = x[r:r + n]
                    peak = part.abs().amax((0, 2)) / 448
                    e = torch.where(peak > 0, torch.ceil(torch.log2(peak)), -math.inf).clamp(E_MIN, E_MAX)
                    new = torch.exp2(e)
                    if o:
                        new = torch.maximum(new, z[g])
                        c[g, :, :o] = round_e4m3(c[g, :, :o] * (z[g] / new)[:, None, None])
                    z[g] = new
                    c[g, :, o:o + n] = round_e4m3(part / new[:, None]).permute(1, 0, 2)
                    r, p = r + n, p + n
            outs.append(c)
            scales.append(z)
        return [*outs, *scales]

    def of_attn(s):
        case, value = s["case"], value_table()
        page, H, W, D = case["page"], case["kv_heads"], case["window"], case["dim"]
        G = case["heads"] // H
        w = work(case)
        if w["flops"] > 6e12 or w["bytes"] > 2e10:
            return None
        table, row_start, kv_len = s["plan"][:3]
        starts, out = row_start.tolist(), torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, L in enumerate(kv_len.tolist()):
            r, n = starts[b], starts[b + 1] - starts[b]
            lo = max(0, L - n - W + 1) if W else 0
            at = table[b, lo // page: -(-L // page)].long()
            lo = lo // page * page
            for h in range(H):
                k, v = ((value[c[at, h].long()] * z[at, h].double()[:, None, None]).reshape(-1, D)[: L - lo]
                        for c, z in ((s["k"], s["ks"]), (s["v"], s["vs"])))
                step = max(1, (1 << 28) // (G * (L - lo)))
                for i in range(0, n, step):
                    q = s["q"][r + i:r + min(n, i + step), h * G:(h + 1) * G].double()
                    m = q.shape[0]
                    z = torch.einsum("mgd,jd->mgj", q, k) / math.sqrt(D)
                    p = torch.arange(L - n + i, L - n + i + m, device=DEV)[:, None]
                    j = torch.arange(lo, L, device=DEV)
                    hide = (j > p) | (j <= p - W) if W else j > p
                    z.masked_fill_(hide[:, None], -math.inf)
                    base = torch.full((G,), -math.inf, dtype=torch.float64, device=DEV) if s["sink"] is None else \
                        s["sink"][h * G:(h + 1) * G].double()
                    top = torch.maximum(z.amax(-1), base)
                    e = torch.exp(z - top[..., None])
                    den = e.sum(-1) + torch.exp(base - top)
                    out[r + i:r + i + m, h * G:(h + 1) * G] = torch.einsum("mgj,jd->mgd", e, v) / den[..., None]
        return [out]

    return {"plan": of_plan, "rope": of_rope, "write": of_write, "attn": of_attn}[case["op"]](prepare(case, seed))
