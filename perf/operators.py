"""The history cache and the attention that reads it: what is timed, and the plain forms.

A generator that makes a video chunk by chunk keeps the keys and values of the
frames it has made in pages, and several continuations of one history share
those pages. Three kinds of cases:

  attend   attention of a batch of continuations over the history they share
           and each one's own rows after it
  grow     one step of the bookkeeping and of the data: the continuations of
           the step before are dropped, the history is forked again, room is
           reserved for the new rows, and they are written
  compact  the pages in use are moved to the front of the pool

The plain forms are elementary torch operations in 32 bits (integers as they
are); `own` switches `run` to the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def _attend(name, B, H, H_kv, d, page, prefix, rows, tail_lo, tail_hi, idle=0):
    return {"name": name, "kind": "attend", "B": B, "H": H, "H_kv": H_kv, "d": d, "page": page,
            "prefix": prefix, "rows": rows, "tail_lo": tail_lo, "tail_hi": tail_hi, "idle": idle}


def _grow(name, H_kv, d, page, parent, kids, rows_lo, rows_hi):
    return {"name": name, "kind": "grow", "H_kv": H_kv, "d": d, "page": page, "parent": parent,
            "kids": kids, "rows_lo": rows_lo, "rows_hi": rows_hi}


def _compact(name, H_kv, d, page, pages, live, moves, seqs):
    return {"name": name, "kind": "compact", "H_kv": H_kv, "d": d, "page": page, "pages": pages,
            "live": live, "moves": moves, "seqs": seqs}


def listed():
    return [
        # one query row each of two continuations of a short history: latency
        _attend("row_short", 2, 8, 8, 64, 16, 500, 1, 1, 40),
        # one row of 16 candidates after 33 frames of 3600 positions, every head its own keys
        _attend("row_frames33", 16, 24, 24, 128, 64, 118800, 1, 256, 512),
        # one row of 64 sequences, four query heads to a key head, ragged tails, an idle slot
        _attend("row_grouped", 64, 32, 8, 128, 32, 20001, 1, 0, 700, 1),
        # one row of 200 sequences, eight query heads to a key head: the shared part is a product
        _attend("row_many", 200, 16, 2, 128, 64, 30000, 1, 16, 300),
        # a few dozen rows at odd sizes: tiles that hold parts of several sequences
        _attend("rows_odd", 5, 6, 3, 64, 16, 12345, 37, 37, 3000),
        # a new frame of 3600 positions for two continuations of a two-frame history
        _attend("frame", 2, 24, 24, 128, 128, 7200, 3600, 3600, 3600),
        # a quarter of a 4080-position frame for three continuations, d = 64, large pages
        _attend("frame_part", 3, 48, 48, 64, 256, 4080, 1020, 1020, 2100),
        # one new row for four continuations: latency of the bookkeeping
        _grow("grow_row", 8, 64, 16, 1000, 4, 1, 1),
        # a few rows for 64 continuations of a long history
        _grow("grow_rows", 8, 128, 128, 118801, 64, 1, 5),
        # about a frame of rows for eight continuations of 11 frames
        _grow("grow_frame", 24, 128, 64, 39610, 8, 3500, 3600),
        # a small pool
        _compact("compact_small", 8, 64, 16, 500, 200, 61, 7),
        # a pool of a few gigabytes, half of the live pages out of place
        _compact("compact_large", 24, 128, 64, 4096, 2000, 1000, 48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["row", "row", "rows", "frame", "grow", "compact"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "row":
        H_kv, G = rng.randint(1, 24), rng.choice([1, 1, 2, 4, 8])
        B = _log(rng, 1, 200)
        prefix = _log(rng, 1, max(1, min(120000, 30_000_000 // (H_kv * max(B * G // 8, 8)))))
        lo = rng.randint(0, 64)
        c = _attend("", B, H_kv * G, H_kv, d, page, prefix, 1, lo, lo + _log(rng, 1, 400),
                    1 if B > 3 and rng.random() < 0.5 else 0)
    elif kind == "rows":
        H_kv, G = rng.randint(1, 8), rng.choice([1, 2, 3])
        rows = _log(rng, 2, 300)
        B = _log(rng, 1, 16)
        prefix = _log(rng, 1, min(20000, 1_000_000_000 // (H_kv * G * B * rows)))
        c = _attend("", B, H_kv * G, H_kv, d, page, prefix, rows, rows, rows + _log(rng, 1, 1000))
    elif kind == "frame":
        rows = _log(rng, 300, 3600)
        B, H = rng.randint(1, 3 if rows < 2000 else 2), rng.randint(4, 24)
        c = _attend("", B, H, H, d, page, _log(rng, 500, 7200), rows, rows, rows)
    elif kind == "grow":
        lo = _log(rng, 1, 1500)
        c = _grow("", rng.randint(1, 24), d, page, _log(rng, 1, 40000), _log(rng, 1, 24), lo,
                  lo + rng.randint(0, 100))
    else:
        live = _log(rng, 20, 1200)
        moves = rng.randint(0, live // 2)
        pages = live + moves + rng.randint(0, live)
        c = _compact("", rng.randint(1, 24), d, min(page, 64), pages, live, moves, rng.randint(1, 16))
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * i // max(n - 1, 1) for i in range(n)]


def _up(a, b):
    return -(-a // b)


def work(c):
    row = c["H_kv"] * c["d"] * 2 * 2  # bytes of one position's keys and values
    if c["kind"] == "attend":
        tails = _spread(c["tail_lo"], c["tail_hi"], c["B"])[c["idle"]:]
        keys = len(tails) * c["prefix"] + sum(tails)
        q = len(tails) * c["H"] * c["rows"]
        entries = _up(c["prefix"], c["page"]) + sum(_up(t, c["page"]) for t in tails)
        return {"bytes": (c["prefix"] + sum(tails)) * row + q * (4 * c["d"] + 4) + 4 * entries,
                "flops": 4 * c["d"] * c["H"] * c["rows"] * keys}
    if c["kind"] == "grow":
        new = sum(_spread(c["rows_lo"], c["rows_hi"], c["kids"]))
        # each continuation but the rows of whole pages copies the history's open page
        new += c["kids"] * (c["parent"] % c["page"])
        return {"bytes": 2 * new * row + 4 * c["kids"] * 2 * _up(c["parent"], c["page"]), "flops": 0}
    entries = c["seqs"] * _up(c["live"], 1)
    return {"bytes": 2 * c["moves"] * c["page"] * row + 2 * 4 * (entries + c["pages"]), "flops": 0}


# --------------------------------------------------------------------------- inputs
def _pool(c, pages, g):
    """Keys with a part that a page's rows share (as the positions of a frame do) and values
    with a part of each channel."""
    shape = (pages, c["H_kv"], c["page"], c["d"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    common = torch.randn((pages, c["H_kv"], 1, c["d"]), generator=g, device=DEV)
    k.mul_(0.8).add_(common.mul_(0.6).to(torch.bfloat16))
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v.mul_(0.9).add_((0.45 * torch.randn((1, c["H_kv"], 1, c["d"]), generator=g, device=DEV)).to(torch.bfloat16))
    return k, v


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    ps = c["page"]
    s = {"case": c, "kept": {}}
    if c["kind"] == "attend":
        B, prefix = c["B"], c["prefix"]
        tails = _spread(c["tail_lo"], c["tail_hi"], B)
        tails = [tails[i] for i in torch.randperm(B, generator=h).tolist()] if not c["idle"] else tails
        shared, full = _up(prefix, ps), prefix // ps
        own_pages = [_up(prefix + t, ps) - full if t else 0 for t in tails]
        pages = shared + sum(own_pages) + 3
        ids = torch.randperm(pages, generator=h).to(torch.int32)
        width = max([shared] + [full + n for n in own_pages])
        table = torch.full((B + 1, width), -1, dtype=torch.int32)
        table[0, :shared] = ids[:shared]
        at, lens = shared, [prefix]
        for b, t in enumerate(tails):
            table[b + 1, :full] = ids[:full]
            if t:
                table[b + 1, full:full + own_pages[b]] = ids[at:at + own_pages[b]]
                at += own_pages[b]
            elif shared > full:
                table[b + 1, full] = ids[full]
            lens.append(prefix + t)
        k, v = _pool(c, pages, g)
        if prefix % ps:  # the open page of the history was copied when a continuation first wrote
            copies = [int(table[b + 1, full]) for b, t in enumerate(tails) if t]
            if copies:
                at = torch.tensor(copies, device=DEV)
                k[at, :, :prefix % ps] = k[int(table[0, full]), :, :prefix % ps]
                v[at, :, :prefix % ps] = v[int(table[0, full]), :, :prefix % ps]
        seqs = [-1 if b < c["idle"] else b + 1 for b in range(B)]
        q = torch.randn((B, c["H"], c["rows"], c["d"]), generator=g, device=DEV)
        near = k[torch.randint(pages, (B,), generator=h).to(DEV)].float().mean(2)  # each looks for something it knows
        q += near.repeat_interleave(c["H"] // c["H_kv"], 1)[:, :, None] * 2.0
        s.update(k=k, v=v, q=q.to(torch.bfloat16), table=table.to(DEV),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 seqs=torch.tensor(seqs, dtype=torch.int32, device=DEV),
                 o=torch.zeros((B, c["H"], c["rows"], c["d"]), dtype=torch.bfloat16, device=DEV),
                 lse=torch.zeros((B, c["H"], c["rows"]), device=DEV), tail_max=max(tails))
        return s
    if c["kind"] == "grow":
        n, parent = c["kids"], c["parent"]
        counts = _spread(c["rows_lo"], c["rows_hi"], n)
        counts = [counts[i] for i in torch.randperm(n, generator=h).tolist()]
        full = _up(parent, ps)
        pages = full + sum(_up(parent + x, ps) - parent // ps for x in counts) + 2
        width = _up(parent + c["rows_hi"], ps)
        ids = torch.randperm(pages, generator=h)[:full].to(torch.int32)
        table = torch.full((n + 1, width), -1, dtype=torch.int32)
        table[0, :full] = ids
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[ids.long()] = 1
        k, v = _pool(c, pages, g)
        shape = (n, c["H_kv"], c["rows_hi"], c["d"])
        s.update(k=k, v=v, table=table.to(DEV), refs=refs.to(DEV),
                 lens=torch.tensor([parent] + [0] * n, dtype=torch.int32, device=DEV),
                 parents=torch.zeros(n, dtype=torch.int32, device=DEV),
                 kids=torch.arange(1, n + 1, dtype=torch.int32, device=DEV),
                 counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                 plan=torch.zeros((n, 4), dtype=torch.int32, device=DEV),
                 k_new=torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16),
                 v_new=torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16))
        return s
    pages, live, moves, S = c["pages"], c["live"], c["moves"], c["seqs"]
    in_use = torch.ones(pages, dtype=torch.bool)
    in_use[live:] = False
    in_use[torch.randperm(live, generator=h)[:moves]] = False
    in_use[live + torch.randperm(pages - live, generator=h)[:moves]] = True
    ids = torch.nonzero(in_use)[:, 0]
    ids = ids[torch.randperm(live, generator=h)].to(torch.int32)
    shared = live // 3  # a history that all sequences have, then each one's own pages
    per = _up(live - shared, S)
    table = torch.full((S, live), -1, dtype=torch.int32)
    table[:, :shared] = ids[:shared]
    for i in range(S):
        mine = ids[shared + i * per:shared + (i + 1) * per]
        table[i, shared:shared + len(mine)] = mine
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    k, v = _pool(c, pages, g)
    s.update(k=k, v=v, table=table.to(DEV), refs=refs.to(DEV),
             table_out=torch.empty_like(table, device=DEV), refs_out=torch.empty_like(refs, device=DEV),
             moves=torch.zeros(2 + 2 * pages, dtype=torch.int32, device=DEV))
    return s


# --------------------------------------------------------------------------- the framework's calls
def _geom(s):
    import video_dit_spatial_b200 as svg
    if "geom" not in s["kept"]:
        c = s["case"]
        s["kept"]["geom"] = svg.CacheGeom(s["k"].shape[0], c["page"], c["H_kv"], c["d"],
                                          s["table"].shape[0], s["table"].shape[1])
    return svg, s["kept"]["geom"]


def _own_attend(s):
    svg, geom = _geom(s)
    c = s["case"]
    if "workspace" not in s["kept"]:
        need = svg.svg_prefix_attention_workspace_bytes(geom, c["B"], c["H"], c["rows"])
        s["kept"]["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    svg.svg_prefix_attention(geom, c["B"], c["H"], c["rows"], 0, c["prefix"], c["d"] ** -0.5, s["q"],
                             s["k"], s["v"], s["table"], s["lens"], s["seqs"], s["o"], s["lse"],
                             s["kept"]["workspace"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_grow(s):
    svg, geom = _geom(s)
    state = (s["table"], s["lens"], s["refs"])
    svg.svg_cache_free(geom, *state, s["kids"])
    svg.svg_cache_fork(geom, *state, s["parents"], s["kids"])
    svg.svg_cache_reserve(geom, *state, s["kids"], s["counts"], s["plan"])
    svg.svg_cache_write(geom, s["table"], s["kids"], s["plan"], s["case"]["rows_hi"], s["k_new"],
                        s["v_new"], s["k"], s["v"])
    return {"k": s["k"], "v": s["v"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}


def _own_compact(s):
    svg, geom = _geom(s)
    svg.svg_cache_compact(geom, s["table"], s["refs"], s["table_out"], s["refs_out"], s["moves"])
    svg.svg_cache_copy_pages(geom, s["moves"], s["case"]["pages"] // 2, s["k"], s["v"], s["k"], s["v"])
    return {"k": s["k"], "v": s["v"], "table": s["table_out"], "refs": s["refs_out"]}


# --------------------------------------------------------------------------- the plain forms
def _rows(pages, entries, at, ps):
    """Rows at positions `at` of the sequences whose table rows are `entries`: [n, len(at), H_kv, d]."""
    page = entries[:, at // ps].long().clamp(min=0)
    return pages[page, :, (at % ps)[None].expand_as(page)].float()


def _plain_attend(s):
    c = s["case"]
    B, H_kv, rows, d, ps, prefix = c["B"], c["H_kv"], c["H"] // c["H_kv"] * c["rows"], c["d"], c["page"], c["prefix"]
    seqs = s["seqs"].long()
    entries, lens = s["table"][seqs.clamp(min=0)], s["lens"][seqs.clamp(min=0)]
    q = s["q"].float().view(B, H_kv, rows, d) * d ** -0.5
    at = torch.arange(prefix, device=DEV)
    kp = _rows(s["k"], s["table"][:1], at, ps)[0].permute(1, 2, 0)                      # H_kv, d, prefix
    x = torch.matmul(q.transpose(0, 1).reshape(H_kv, B * rows, d), kp)                  # H_kv, B rows, prefix
    top = x.amax(-1).view(H_kv, B, rows).transpose(0, 1)
    at2 = prefix + torch.arange(s["tail_max"], device=DEV)
    at2_in = at2.clamp(max=s["table"].shape[1] * ps - 1)
    y = None
    if s["tail_max"]:
        y = torch.matmul(q, _rows(s["k"], entries, at2_in, ps).permute(0, 2, 3, 1))     # B, H_kv, rows, tail
        hidden = (at2[None] >= lens[:, None])[:, None, None]
        y = y.masked_fill_(hidden, -math.inf)
        top = torch.maximum(top, y.amax(-1))
    x = x.sub_(top.transpose(0, 1).reshape(H_kv, B * rows, 1)).exp_()
    total = x.sum(-1).view(H_kv, B, rows).transpose(0, 1)
    vp = _rows(s["v"], s["table"][:1], at, ps)[0].transpose(0, 1)                       # H_kv, prefix, d
    o = torch.matmul(x, vp).view(H_kv, B, rows, d).transpose(0, 1)
    if y is not None:
        y = y.sub_(top[..., None]).exp_()
        total = total + y.sum(-1)
        o = o + torch.matmul(y, _rows(s["v"], entries, at2_in, ps).transpose(1, 2))
    o = (o / total[..., None]).reshape(s["o"].shape).to(torch.bfloat16)
    lse = (top + total.log()).reshape(s["lse"].shape)
    busy = (seqs >= 0)
    s["o"].copy_(torch.where(busy[:, None, None, None], o, s["o"]))
    s["lse"].copy_(torch.where(busy[:, None, None], lse, s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def _plain_grow(s):
    c, table, lens, refs = s["case"], s["table"], s["lens"], s["refs"]
    ps, kids, parents, counts = c["page"], s["kids"].long(), s["parents"].long(), s["counts"]
    slot = torch.arange(table.shape[1], device=DEV)[None]
    # drop the continuations of the step before
    used = slot < ((lens[kids] + ps - 1) // ps)[:, None]
    refs.index_add_(0, table[kids].clamp(min=0).flatten(), -used.flatten().to(torch.int32))
    table[kids] = -1
    lens[kids] = 0
    # fork the history
    used = slot < ((lens[parents] + ps - 1) // ps)[:, None]
    table[kids] = table[parents]
    lens[kids] = lens[parents]
    refs.index_add_(0, table[kids].clamp(min=0).flatten(), used.flatten().to(torch.int32))
    # reserve: the lowest free pages, entry by entry; an open page that others have too is replaced
    first = lens[kids]
    open_slot = (first // ps).long()[:, None]
    last = table[kids].gather(1, open_slot.clamp(max=table.shape[1] - 1))[:, 0]
    replaced = (first % ps != 0) & (refs[last.clamp(min=0)] > 1) & (counts > 0)
    begin = torch.where(replaced, first // ps, (first + ps - 1) // ps)[:, None]
    wanted = (slot >= begin) & (slot < ((first + counts + ps - 1) // ps)[:, None])
    rank = wanted.flatten().cumsum(0).view_as(wanted) - 1
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    new = free[rank.clamp(0, free.numel() - 1)]
    table[kids] = torch.where(wanted, new, table[kids])
    refs.index_add_(0, new.flatten(), wanted.flatten().to(torch.int32))
    refs.index_add_(0, last.clamp(min=0), -replaced.to(torch.int32))
    lens[kids] = first + counts
    # write: the replaced pages' rows, then the new ones
    which = torch.nonzero(replaced)[:, 0]
    old, dst = last[which].long(), table[kids[which], open_slot[which, 0]].long()
    stays = (torch.arange(ps, device=DEV)[None] < (first[which] % ps)[:, None])[:, None, :, None]
    i, j = torch.nonzero(torch.arange(c["rows_hi"], device=DEV)[None] < counts[:, None]).unbind(1)
    at = first[i] + j
    page = table[kids[i], (at // ps).long()].long()
    s["k"][dst] = torch.where(stays, s["k"][old], s["k"][dst])
    s["v"][dst] = torch.where(stays, s["v"][old], s["v"][dst])
    s["k"][page, :, (at % ps).long()] = s["k_new"][i, :, j]
    s["v"][page, :, (at % ps).long()] = s["v_new"][i, :, j]
    return {"k": s["k"], "v": s["v"], "table": table, "lens": lens, "refs": refs}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    page = torch.arange(refs.numel(), device=DEV)
    n = live.sum()
    hole = torch.nonzero(~live & (page < n))[:, 0]
    moved = torch.nonzero(live & (page >= n))[:, 0]
    to = page.clone()
    to[moved] = hole
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table).to(torch.int32))
    s["refs_out"].copy_(refs)
    s["refs_out"][hole] = refs[moved]
    s["refs_out"][moved] = 0
    s["k"][hole] = s["k"][moved]
    s["v"][hole] = s["v"][moved]
    return {"k": s["k"], "v": s["v"], "table": s["table_out"], "refs": s["refs_out"]}


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"attend": _own_attend, "grow": _own_grow, "compact": _own_compact}[kind](s)
    return {"attend": _plain_attend, "grow": _plain_grow, "compact": _plain_compact}[kind](s)


# --------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    if c["kind"] != "attend":  # copies and whole numbers: nothing is computed that rounds
        return None
    s = prepare(c, seed)
    table, lens, seqs, ps = s["table"].tolist(), s["lens"].tolist(), s["seqs"].tolist(), c["page"]
    G, R = c["H"] // c["H_kv"], c["rows"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)

    def rows_of(seq, lo, hi):
        return [table[seq][p // ps] * ps + p % ps for p in range(lo, hi)]

    head = rows_of(0, 0, c["prefix"])
    for kv in range(c["H_kv"]):
        kf, vf = (x[:, kv].reshape(-1, c["d"]) for x in (s["k"], s["v"]))  # page-major rows of this head
        at = torch.tensor(head, device=DEV)
        k0, v0 = kf[at].double(), vf[at].double()
        for b, seq in enumerate(seqs):
            if seq < 0:
                continue
            at = torch.tensor(rows_of(seq, c["prefix"], lens[seq]), dtype=torch.long, device=DEV)
            k = torch.cat([k0, kf[at].double()])
            v = torch.cat([v0, vf[at].double()])
            for h in range(kv * G, kv * G + G):
                z = s["q"][b, h].double() @ k.T / math.sqrt(c["d"])
                top = z.max(-1, keepdim=True).values
                w = torch.exp(z - top)
                t = w.sum(-1, keepdim=True)
                o[b, h] = w @ v / t
                lse[b, h] = (top + torch.log(t))[:, 0]
    return {"o": o, "lse": lse}
