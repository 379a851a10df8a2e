"""The operators of beam search over a paged cache, as cases to measure.

A caller that serves its own target keeps the pages of its cache: it takes pages
for new tokens and gives them back, lets sequences share a prefix, and copies a
shared page before one of them writes to it.  With several beams a request it
also chooses the next beams among all continuations and hands their sequences on.
Each case is one call of one of these operators -- the selection (`select`), the
hand-over of sequences (`fork`), new lengths (`resize`), the copies behind them
(`copy`), moving all pages to the front of the pools (`compact`, with its copies) --
in its plain form (elementary torch operations) or, with `own` set, through
block_diffusion_speculative_hiddens_gb300.ops.

fork, resize and compact change the pool's state in place.  Their passes begin
with that state as it was, written back by one copy on either side, so that every
pass does the same work; the bytes of a pass count the state once read and once
written.

Sizes come from this repository's workloads (vocabularies of 151,936, 128,256,
32,768 and 4,096; 8, 4 and 2 KV heads of 128 and 64; pages of 64; contexts of 512 to
32,768; batches of 1, 4 and 64; 1 to 8 layers) and from the ranges between them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
END = 2  # the token that ends a sequence


def _select(name, batch, beams, n, vocab, dtype, mask="none", first=False, done=0):
    return {"name": name, "op": "select", "batch": batch, "beams": beams, "n": n, "vocab": vocab, "dtype": dtype,
            "mask": mask, "first": first, "done": done}


def _pool_case(name, op, groups, beams, len_lo, len_hi, page, tail, spare, grow=0, leave=0, siblings=False):
    """groups requests of `beams` sequences each, len_lo to len_hi positions long, of which the last `tail` pages
    are a sequence's own (siblings: inherited at the last step); spare: free pages a used one."""
    return {"name": name, "op": op, "groups": groups, "beams": beams, "len_lo": len_lo, "len_hi": len_hi, "page": page,
            "tail": tail, "spare": spare, "grow": grow, "leave": leave, "siblings": siblings}


def _copy(name, moves, layers, page, hkv, d, dtype, full):
    return {"name": name, "op": "copy", "moves": moves, "layers": layers, "page": page, "hkv": hkv, "d": d,
            "dtype": dtype, "full": full}


def _compact(name, layers, hkv, d, dtype, *pool):
    return _pool_case(name, "compact", *pool) | {"layers": layers, "hkv": hkv, "d": d, "dtype": dtype}


def listed():
    return [
        # one request's four beams, twice as many continuations as beams: some of them may end
        _select("select, one request", 1, 4, 8, 151936, "bf16"),
        # a batch of requests in mid-search, some beams at their end
        _select("select, a batch of beams", 64, 8, 16, 151936, "bf16", done=5),
        # a wide search under a grammar: 32-bit logits, most tokens at -inf, one row with nothing left
        _select("select, wide and masked", 3, 32, 64, 128256, "f32", mask="inf"),
        # an odd vocabulary, whose rows begin at every alignment
        _select("select, an odd vocabulary", 11, 5, 5, 100003, "f16", done=1),
        # one request's beams handed on: the smallest call of a search's step
        _pool_case("fork, one request", "fork", 1, 4, 2048, 2048, 64, 2, 0.5),
        # the batch's beams handed on, long contexts
        _pool_case("fork, a batch of beams", "fork", 64, 8, 1000, 32768, 64, 3, 0.3),
        # room for a verify block of each request, before its round
        _pool_case("resize, verify blocks", "resize", 64, 1, 512, 4096, 64, 1, 0.6, grow=16),
        # a token for every beam just handed on: shared last pages are copied, ended requests leave
        _pool_case("resize, a step of beams", "resize", 64, 8, 1000, 32768, 64, 3, 0.3, grow=1, leave=5, siblings=True),
        # last pages of one request's beams in one layer
        _copy("copy, one layer", 4, 1, 64, 8, 128, "bf16", False),
        # last pages of a batch of beams in every layer
        _copy("copy, every layer", 448, 8, 64, 8, 128, "bf16", False),
        # a small pool after a few requests have left
        _compact("compact, a small pool", 2, 2, 64, "f16", 4, 4, 30, 700, 16, 3, 0.8),
        # a large pool after a peak: a third of it in use, all over the place
        _compact("compact, after a peak", 5, 8, 128, "bf16", 32, 1, 512, 4096, 64, 1, 2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "resize", "copy", "compact"])
    if op == "select":
        beams = _log(rng, 1, 32)
        batch = _log(rng, 1, 512 // beams)
        vocab = rng.choice([151936, 128256, 32768, 4096, _log(rng, 100, 150000)])
        n = min(rng.choice([beams, 2 * beams, _log(rng, 1, 64)]), 64)
        dtype = rng.choice(["bf16", "f16", "f32"])
        if dtype == "f32":
            batch = (batch + 1) // 2
        c = _select("", batch, beams, n, vocab, dtype, rng.choice(["none", "none", "inf", "lowest"]),
                    rng.random() < 0.2, rng.choice([0, 0, 1, 4]))
    elif op == "copy":
        hkv, d = rng.choice([(8, 128), (4, 128), (2, 64), (1, 128), (5, 64)])
        page, layers = rng.choice([16, 32, 64, 64, 128]), _log(rng, 1, 36)
        moves = _log(rng, 1, max(2, min(448, 115000000 // (layers * page * hkv * d))))
        c = _copy("", moves, layers, page, hkv, d, rng.choice(["bf16", "f16"]), rng.random() < 0.3)
    else:
        page, beams = rng.choice([16, 32, 64, 64, 128]), rng.choice([1, 1, 2, 4, 8, 13])
        groups = _log(rng, 1, 512 // beams)
        hi = _log(rng, page, max(2 * page, min(32768, 250000 * page // (groups * beams))))
        pool = [groups, beams, rng.randint(1, hi), hi, page, rng.randint(1, 4), rng.uniform(0.3, 2.0)]
        if op == "compact":
            hkv, d = rng.choice([(8, 128), (4, 128), (2, 64), (5, 64)])
            pages = -(-hi // page) * groups * beams  # more than are in use
            pool[0] = max(1, min(groups, groups * 300000000 // (pages * page * hkv * d)))
            c = _compact("", 1, hkv, d, rng.choice(["bf16", "f16"]), *pool)
            c["layers"] = rng.randint(1, max(1, min(8, 300000000 // (pages * page * hkv * d))))
        elif op == "fork":
            c = _pool_case("", op, *pool)
        else:
            c = _pool_case("", op, *pool, grow=rng.choice([1, 1, 16, _log(rng, 1, 300)]),
                           leave=rng.choice([0, 0, 3, 7]), siblings=rng.random() < 0.5)
    del c["name"]
    return c


# ---- the inputs

def _spread(lo, hi, b, stride):
    """b whole numbers over [lo, hi], both ends among them where b > 1, in a mixed order."""
    if b == 1:
        return [hi]
    order = [(i * stride) % b for i in range(b)] if math.gcd(stride, b) == 1 else list(range(b))
    return [lo + (hi - lo) * i // (b - 1) for i in order]


def _shape(case):
    """Lengths of the requests, pages that are in use at most, pages of the pool, columns of the table."""
    page, beams = case["page"], case["beams"]
    lens = _spread(case["len_lo"], case["len_hi"], case["groups"], 11)
    need = [-(-n // page) for n in lens]
    used = sum(max(n - case["tail"], 0) + beams * min(n, case["tail"]) for n in need)
    taken = case["groups"] * beams * (1 + -(-case["grow"] // page))  # by a resize
    width = max(need) + 1 + -(-case["grow"] // page)
    return lens, used, used + max(int(used * case["spare"]), taken), -(-width // 4) * 4


def _prepare_pool(case, st, g):
    lens, _, n_pages, width = _shape(case)
    groups, beams, page, tail = case["groups"], case["beams"], case["page"], case["tail"]
    rows = groups * beams
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda").repeat_interleave(beams)
    need = (lens.long() + page - 1) // page
    col = torch.arange(width, device="cuda")
    live = col < need[:, None]
    me = torch.arange(rows, device="cuda")
    owner = me.clone()
    if case["siblings"]:  # the beam of its request whose pages each beam was given
        owner = me // beams * beams + torch.randint(0, beams, (rows,), generator=g, device="cuda")
    shared = col < (need - tail)[:, None]
    key = torch.where(shared, (me // beams * beams)[:, None], owner[:, None]) * width + col
    # pages handed out in random order, as a pool that has served for a while gives them
    taken = torch.zeros(rows * width, dtype=torch.long, device="cuda")
    taken[key[live]] = 1
    ids = torch.randperm(n_pages, generator=g, device="cuda")[(torch.cumsum(taken, 0) - 1).clamp(min=0)]
    table = torch.where(live, ids[key], -1).to(torch.int32)
    refs = torch.bincount(table[live].long(), minlength=n_pages).to(torch.int32)
    # one allocation for the whole state, its parts at multiples of four values
    parts = [-(-n_pages // 4) * 4, -(-rows // 4) * 4, rows * width]
    st["start"] = torch.cat([torch.nn.functional.pad(x, (0, n - len(x))) for x, n in
                             zip((refs, lens, table.flatten()), parts)])
    st["state"] = st["start"].clone()
    a, b, c = torch.split(st["state"], parts)
    st.update(refs=a[:n_pages], lens=b[:rows], table=c.view(rows, width))
    if case["op"] == "fork":
        st["parents"] = (me // beams * beams + torch.randint(0, beams, (rows,), generator=g, device="cuda")).to(torch.int32)
    elif case["op"] == "resize":
        st["new_lens"] = lens + case["grow"]
        if case["leave"]:
            st["new_lens"] = torch.where(me // beams % case["leave"] == 1, 0, st["new_lens"]).to(torch.int32)
    if own:
        from block_diffusion_speculative_hiddens_gb300 import ops
        st["pool"] = ops.PagePool(st["table"], n_pages, page, refs=st["refs"], lens=st["lens"])
    return n_pages


def _prepare_caches(case, st, g, n_pages):
    shape = (n_pages, case["page"], case["hkv"], case["d"])
    dt = DTYPES[case["dtype"]]
    st["pools"] = [torch.randn(shape, generator=g, device="cuda", dtype=dt) for _ in range(2 * case["layers"])]
    if own:
        from block_diffusion_speculative_hiddens_gb300 import ops
        table = st["table"] if "table" in st else torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        st["caches"] = [ops.PagedCache(k, v, table) for k, v in zip(st["pools"][::2], st["pools"][1::2])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "select":
        batch, beams, vocab, dt = case["batch"], case["beams"], case["vocab"], DTYPES[case["dtype"]]
        rows = batch * beams
        st["logits"] = torch.randn(rows, vocab, generator=g, device="cuda", dtype=dt).mul_(2.5)
        if case["mask"] != "none":  # a grammar: each row allows its own few tokens, the second row none
            allowed = torch.rand(rows, vocab, generator=g, device="cuda") < 0.02
            allowed[1:2] = False
            st["logits"][~allowed] = -math.inf if case["mask"] == "inf" else torch.finfo(dt).min
        st["scores"] = -10 - 4 * torch.rand(batch, beams, generator=g, device="cuda")
        if case["first"]:  # the first step of a search: its beams are still one
            st["scores"][:, 0] = 0
            st["scores"][:, 1:] = -math.inf
        st["done"] = None
        if case["done"]:
            st["done"] = torch.arange(rows, device="cuda").view(batch, beams) % (3 * case["done"]) == case["done"]
        return st
    if case["op"] == "copy":
        m = case["moves"]
        n_pages = 2 * m + 3
        _prepare_caches(case, st, g, n_pages)
        ids = torch.randperm(n_pages, generator=g, device="cuda")[:2 * m].view(2, m)
        st["moves"] = torch.zeros(m + 1, 3, dtype=torch.int32, device="cuda")
        st["moves"][0, 0] = m
        st["moves"][1:, :2] = ids.t()
        st["moves"][1:, 2] = case["page"] if case["full"] else torch.tensor(_copied(case), device="cuda")
        return st
    n_pages = _prepare_pool(case, st, g)
    if case["op"] == "compact":
        _prepare_caches(case, st, g, n_pages)
    return st


def _copied(case):
    """Positions that each move copies."""
    if case["full"]:
        return [case["page"]] * case["moves"]
    return _spread(1, case["page"] - 1, case["moves"], 7)


# ---- the plain forms

def _plain_select(st):
    c = st["case"]
    batch, beams, n, vocab = c["batch"], c["beams"], c["n"], c["vocab"]
    # 64 bits: two beams' continuations may come as close as the rounding of 32
    x = st["logits"].double()
    top = x.amax(-1, keepdim=True)
    x -= torch.where(torch.isfinite(top), top, 0.0)
    s = x - torch.log(torch.exp(x).sum(-1, keepdim=True)).nan_to_num(neginf=0.0)  # a row with nothing left stays -inf
    s = s.view(batch, beams, vocab)
    s += st["scores"].double()[..., None]
    if st["done"] is not None:  # a beam at its end goes on as it is
        only = torch.full((vocab,), -math.inf, dtype=torch.float64, device="cuda")
        only[END] = 0
        s = torch.where(st["done"][..., None], st["scores"].double()[..., None] + only, s)
    s = s.view(batch, -1)
    take = min(n, s.shape[1])
    edge = torch.topk(s, take, dim=-1).values[:, -1:]
    above, level = s > edge, s == edge
    level &= torch.cumsum(level, -1) <= take - above.sum(-1, keepdim=True)  # ties: the lowest of them
    place = torch.arange(s.shape[1], 0, -1, device="cuda")
    at = s.shape[1] - torch.topk(torch.where(above | level, place, 0), take, dim=-1).values  # ascending
    score, order = torch.sort(s.gather(1, at), dim=-1, descending=True, stable=True)
    at = at.gather(1, order)
    row = at // vocab + beams * torch.arange(batch, device="cuda")[:, None]
    none = score == -math.inf
    out = (score.float(), torch.where(none, -1, row).to(torch.int32), torch.where(none, -1, at % vocab).to(torch.int32))
    if take < n:
        fill = (-math.inf, -1, -1)
        out = tuple(torch.nn.functional.pad(x, (0, n - take), value=f) for x, f in zip(out, fill))
    return out


def _hold(refs, ids, where, by):
    """`by` more holders of the pages `ids` where `where`."""
    n = len(refs)
    d = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    at = torch.where(where, ids.long(), n).flatten()
    d.scatter_add_(0, at, torch.full_like(at, by, dtype=torch.int32))
    refs += d[:n]


def _plain_fork(st):
    page, table, lens, refs = st["case"]["page"], st["table"], st["lens"], st["refs"]
    src = st["parents"].long()
    col = torch.arange(table.shape[1], device="cuda")
    new_lens = lens[src]
    had, has = (col < ((x + page - 1) // page)[:, None] for x in (lens, new_lens))
    new = table[src]
    _hold(refs, table, had, -1)
    _hold(refs, new, has, 1)
    table.copy_(torch.where(has, new, torch.where(had, -1, table)))
    lens.copy_(new_lens)


def _plain_resize(st):
    page, table, lens, refs, new = st["case"]["page"], st["table"], st["lens"], st["refs"], st["new_lens"]
    rows, n_pages = len(lens), len(refs)
    me = torch.arange(rows, device="cuda")
    col = torch.arange(table.shape[1], device="cuda")
    old_p, new_p = (lens + page - 1) // page, (new + page - 1) // page
    # a sequence that grows inside a page which others hold too gets a page of its own, but for the last holder
    last = table.gather(1, (old_p - 1).clamp(min=0).long()[:, None])[:, 0]
    grows = (new > lens) & (lens % page != 0)
    at = torch.where(grows, last, 0).long()
    held = refs[at]
    writers = torch.zeros(n_pages, dtype=torch.int32, device="cuda").scatter_add_(0, at, grows.to(torch.int32))
    first = torch.full((n_pages,), rows, dtype=torch.long, device="cuda")
    first.scatter_reduce_(0, at, torch.where(grows, me, rows), "amin")
    copied = grows & ((writers[at] < held) | (first[at] != me))
    taken = (new_p - old_p).clamp(min=0) + copied
    before = torch.cumsum(taken, 0) - taken
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)  # the lowest first
    page_of = free[(before + copied - old_p)[:, None].add(col).clamp(0, len(free) - 1)]
    grown = (col >= old_p[:, None]) & (col < new_p[:, None])
    lost = (col >= new_p[:, None]) & (col < old_p[:, None])
    moves = torch.full((rows + 1, 3), -1, dtype=torch.int32, device="cuda")
    moves[:, 2] = 0
    to = torch.where(copied, torch.cumsum(copied, 0), rows + 1)
    room = torch.cat((moves, moves[:1]))  # its last row takes what is no copy
    own_page = free[before.clamp(max=len(free) - 1)]
    room[to] = torch.stack((last, own_page, lens % page), 1)
    moves[1:] = room[1:rows + 1]
    moves[0] = 0
    moves[0, 0] = copied.sum()
    _hold(refs, last, copied, -1)
    _hold(refs, own_page, copied, 1)
    _hold(refs, table, lost, -1)
    _hold(refs, page_of, grown, 1)
    new_table = torch.where(grown, page_of, torch.where(lost, -1, table))
    table.copy_(torch.where(copied[:, None] & (col == old_p[:, None] - 1), own_page[:, None], new_table))
    lens.copy_(new)
    return moves


def _plain_copy(st, moves):
    m = moves[1:][moves[1:, 2] > 0].long()
    move, pos = torch.nonzero(torch.arange(st["case"]["page"], device="cuda") < m[:, 2:], as_tuple=True)
    src, dst = m[move, 0], m[move, 1]
    for pool in st["pools"]:
        pool[dst, pos] = pool[src, pos]


def _plain_compact(st):
    page, table, lens, refs = st["case"]["page"], st["table"], st["lens"], st["refs"]
    n = len(refs)
    ids = torch.arange(n, device="cuda", dtype=torch.int32)
    used = refs != 0
    total = used.sum()
    src, dst = ids[used & (ids >= total)], ids[~used & (ids < total)]
    moves = torch.full((n // 2 + 1, 3), -1, dtype=torch.int32, device="cuda")
    moves[:, 2] = 0
    moves[0] = 0
    moves[0, 0] = len(src)
    moves[1:len(src) + 1] = torch.stack((src, dst, torch.full_like(src, page)), 1)
    remap = torch.where(used, ids, -1)
    remap[src.long()] = dst
    refs[dst.long()] = refs[src.long()]
    refs[src.long()] = 0
    live = torch.arange(table.shape[1], device="cuda") < ((lens + page - 1) // page)[:, None]
    table.copy_(torch.where(live, remap[table.long().clamp(min=0)], table))
    return moves, remap


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from block_diffusion_speculative_hiddens_gb300 import ops
    if op == "select":
        if own:
            return ops.beam_select(st["logits"], st["scores"], c["n"], done=st["done"], done_token=END)
        return _plain_select(st)
    if op == "copy":
        if own:
            ops.copy_pages(st["caches"], st["moves"])
        else:
            _plain_copy(st, st["moves"])
        return st["pools"]
    st["state"].copy_(st["start"])
    if op == "fork":
        if own:
            ops.fork(st["pool"], st["parents"])
        else:
            _plain_fork(st)
        return st["table"], st["refs"], st["lens"]
    if op == "resize":
        moves = ops.resize(st["pool"], st["new_lens"]) if own else _plain_resize(st)
        return st["table"], st["refs"], st["lens"], moves
    if own:
        moves, remap = ops.compact(st["pool"])
        ops.copy_pages(st["caches"], moves)
    else:
        moves, remap = _plain_compact(st)
        _plain_copy(st, moves)
    return [st["table"], st["refs"], st["lens"], moves, remap] + st["pools"]


def work(case):
    if case["op"] == "select":
        rows, size = case["batch"] * case["beams"], DTYPES[case["dtype"]].itemsize
        values = rows * case["vocab"]
        return {"bytes": values * size + 5 * rows + 12 * case["batch"] * case["n"], "flops": 4 * values}
    if case["op"] == "copy":
        return {"bytes": 8 * sum(_copied(case)) * case["layers"] * case["hkv"] * case["d"] + 12 * case["moves"] + 12,
                "flops": 0}
    lens, used, n_pages, width = _shape(case)
    rows = case["groups"] * case["beams"]
    state = 4 * (n_pages + rows + rows * width)
    if case["op"] == "fork":
        return {"bytes": 2 * state + 4 * rows, "flops": 0}
    if case["op"] == "resize":
        return {"bytes": 2 * state + 4 * rows + 12 * (rows + 1), "flops": 0}
    moved = used * (n_pages - used) // n_pages  # of pages at random places: the used ones behind the first `used`
    data = 8 * moved * case["page"] * case["layers"] * case["hkv"] * case["d"]
    return {"bytes": 2 * state + 12 * (n_pages // 2 + 1) + 4 * n_pages + data, "flops": 0}


# ---- the definitions, in 64 bits

def exact(case, seed):
    global own
    if case["op"] in ("fork", "resize"):  # whole numbers only
        return None
    was, own = own, False  # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "copy":
        out = [pool.double() for pool in st["pools"]]
        for src, dst, n in st["moves"][1:].tolist():
            for pool in out:
                pool[dst, :n] = pool[src, :n]
        return out
    if case["op"] == "compact":
        refs = st["refs"].tolist()
        used = [i for i, r in enumerate(refs) if r]
        behind = [i for i in used if i >= len(used)]
        holes = [i for i, r in enumerate(refs[:len(used)]) if not r]
        out = [pool.double() for pool in st["pools"]]
        for src, dst in zip(behind, holes):
            for pool in out:
                pool[dst] = pool[src]
        return [None] * 5 + out
    scores = torch.full((case["batch"], case["n"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        found = []
        for k in range(case["beams"]):
            score = st["scores"][b, k].double()
            if st["done"] is not None and st["done"][b, k]:
                found.append(score[None])
                continue
            p = torch.log_softmax(st["logits"][b * case["beams"] + k].double(), -1) + score
            found.append(p[~torch.isnan(p)])  # of a row with nothing left, none
        best = torch.cat(found).sort(descending=True).values[:case["n"]]
        scores[b, :len(best)] = best
    return scores, None, None
