"""The page and beam-search operators (new lengths, forks, compaction, page
copies, selection) against their plain definitions, at the sizes and states where
they can go wrong, and a beam search through all of them together."""
import math
import random

import pytest
import torch

from tests import beam_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
PAGE, CAPACITY, ARG, NAN = 0x04, 0x08, 0x10, 0x02


@pytest.fixture(scope="module")
def ops(lib):
    from block_diffusion_speculative_hiddens_gb300 import ops as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# ------------------------------------------------------------------ pools

def make_pool(ops, batch, width, n_pages, page=16, stride=None, offset=0):
    """An empty pool whose table rows are `stride` apart and whose refs begin `offset` values into their memory."""
    stride = stride or width
    table = torch.full((batch, stride), -7, dtype=I32, device="cuda")[:, :width]
    refs = torch.zeros(n_pages + offset, dtype=I32, device="cuda")[offset:]
    lens = torch.zeros(batch, dtype=I32, device="cuda")
    return ops.PagePool(table, n_pages, page, refs=refs, lens=lens)


def same(pool, ref, status=0):
    assert pool.lens.tolist() == ref.lens
    got = pool.page_table.tolist()
    for b, (x, y) in enumerate(zip(got, ref.table)):
        assert x == y, (b, x, y)
    assert pool.refs.tolist() == ref.refs
    assert pool.read_status() == ref.status == status


def moves_of(moves):
    """The copies in a list, which is whole: nothing behind the last."""
    m = moves.tolist()
    n = m[0][0]
    assert m[0][1:] == [0, 0] and 0 <= n < len(m)
    assert all(x == [-1, -1, 0] for x in m[n + 1:])
    return [tuple(x) for x in m[1:n + 1]]


def step(ops, pool, ref, what, arg, status=0):
    if what == "resize":
        assert moves_of(ops.resize(pool, i32(arg))) == ref.resize(arg)
    else:
        ops.fork(pool, i32(arg))
        ref.fork(arg)
    same(pool, ref, status)
    ref.status = 0


@pytest.mark.parametrize("batch,width,n_pages,page,stride,offset", [
    (1, 1, 1, 16, None, 0), (3, 5, 9, 16, 7, 1), (8, 33, 200, 16, 36, 0), (5, 9, 40, 256, None, 3),
    (64, 20, 700, 32, None, 0), (130, 12, 5000, 16, 13, 0), (1500, 6, 40000, 16, None, 2), (33, 70, 1800, 64, None, 0)])
def test_a_pool_through_many_calls(ops, batch, width, n_pages, page, stride, offset):
    """Growing, shrinking, ending, forking in every way, against the lists."""
    rng = random.Random(batch * 1000 + width)
    pool = make_pool(ops, batch, width, n_pages, page, stride, offset)
    ref = beam_ref.Pool.of(pool)
    most = width * page
    for turn in range(8 if batch > 1000 else 14):
        spare = sum(r == 0 for r in ref.refs) // batch * page
        new = []
        for n in ref.lens:
            kind = rng.random()
            new.append(n if kind < 0.15 else 0 if kind < 0.2 else rng.randint(0, n) if kind < 0.35
                       else min(most, n + 1) if kind < 0.6 else min(most, n + rng.randint(0, max(spare - page, 0))))
        before = ref.lens[:]
        want = beam_ref.Pool(ref.refs, ref.table, ref.lens, page)
        want.resize(new)
        step(ops, pool, ref, "resize", new, want.status)
        ref.check()
        if want.status:
            assert want.status == CAPACITY and ref.lens == before
        k = rng.choice([1, 2, 4, batch])
        parents = [rng.choice([b, b, rng.randrange(batch), b // k * k, min(batch - 1, b // k * k + rng.randrange(k)), -1])
                   for b in range(batch)]
        step(ops, pool, ref, "fork", parents)
        ref.check()


def test_new_lengths_at_the_edges_of_pages(ops):
    """0, 1, a page, one more; back; nothing; the last free page; all of the table row."""
    pool = make_pool(ops, 2, 4, 5)
    ref = beam_ref.Pool.of(pool)
    for new in ([0, 0], [1, 0], [16, 1], [17, 1], [16, 16], [16, 17], [16, 16], [0, 64], [0, 0], [64, 16], [33, 0], [33, 31]):
        step(ops, pool, ref, "resize", new)
        ref.check()


def test_shared_last_pages(ops):
    """Who copies, and who keeps a page: all holders grow, some do, one does; full pages and ended growth copy nothing."""
    for page_len in (5, 16):
        for grow in ([1, 1, 1, 1], [0, 1, 1, 0], [0, 0, 0, 1], [1, 0, 0, 0], [0, 0, 0, 0], [17, 40, 1, 2]):
            pool = make_pool(ops, 4, 8, 40)
            ref = beam_ref.Pool.of(pool)
            step(ops, pool, ref, "resize", [32 + page_len, 0, 0, 3])
            step(ops, pool, ref, "fork", [0, 0, 0, 0])
            step(ops, pool, ref, "resize", [n + g for n, g in zip(ref.lens, grow)])
            ref.check()


def test_a_pool_that_is_too_small_changes_nothing(ops):
    pool = make_pool(ops, 3, 8, 6)
    ref = beam_ref.Pool.of(pool)
    step(ops, pool, ref, "resize", [40, 16, 5])  # 3 + 1 + 1 pages
    step(ops, pool, ref, "resize", [0, 48, 5], CAPACITY)  # the pages that the first gives up are not yet free
    assert ref.lens == [40, 16, 5]
    step(ops, pool, ref, "fork", [0, 0, 0])  # 3 pages held, 3 free
    step(ops, pool, ref, "resize", [41, 41, 41])  # two copies
    step(ops, pool, ref, "resize", [2 ** 31 - 1, 50, 41], CAPACITY)  # past its row: alone as it is; the rest: the last free page
    assert ref.lens == [41, 50, 41]
    step(ops, pool, ref, "resize", [0, 65, 41], CAPACITY)  # none left
    assert ref.lens == [41, 50, 41]


def test_bad_lengths_and_parents_leave_a_sequence_alone(ops):
    pool = make_pool(ops, 4, 3, 30)
    ref = beam_ref.Pool.of(pool)
    step(ops, pool, ref, "resize", [20, 30, 40, 48])
    step(ops, pool, ref, "resize", [-1, 31, 49, 0], ARG | CAPACITY)
    assert ref.lens == [20, 31, 40, 0]
    step(ops, pool, ref, "fork", [4, 0, -2, 2 ** 31 - 1], ARG)
    assert ref.lens == [20, 20, 40, 0]
    ref.lens[2] = 1000  # a length of the caller's that its row does not hold
    pool.lens[2] = 1000
    step(ops, pool, ref, "fork", [2, 1, 1, 1], ARG)
    assert ref.lens == [20, 20, 1000, 20]
    step(ops, pool, ref, "resize", [21, 21, 21, 21], ARG)
    assert ref.lens == [21, 21, 1000, 21]
    moves, remap = ops.compact(pool)
    ref.compact()
    same(pool, ref, ARG)


def test_bad_pages_are_left_out(ops):
    """Held entries outside the pool, and pages given up that nobody holds: flagged, nothing else is hurt."""
    pool = make_pool(ops, 4, 3, 12)
    ref = beam_ref.Pool.of(pool)
    step(ops, pool, ref, "resize", [20, 30, 40, 48])
    for b, i, bad in ((0, 1, 12), (1, 0, -1), (2, 1, 2 ** 31 - 1)):
        pool.page_table[b, i] = bad
        ref.table[b][i] = bad
    free = ref.table[3][2]
    pool.refs[free] = 0
    ref.refs[free] = 0
    step(ops, pool, ref, "resize", [21, 30, 40, 48], PAGE)  # grows inside a page that is none
    step(ops, pool, ref, "fork", [2, 1, 0, 3], PAGE)
    moves, remap = ops.compact(pool)
    want, want_remap = ref.compact()
    assert moves_of(moves) == want and remap.tolist() == want_remap
    same(pool, ref, PAGE)
    ref.status = 0
    step(ops, pool, ref, "resize", [0, 0, 0, 0], PAGE)


def test_pinned_pages_stay(ops):
    """Pages with a count below 0: shared without counting, copied before they are written, never moved or handed out."""
    pool = make_pool(ops, 3, 6, 20)
    ref = beam_ref.Pool.of(pool)
    for p in (0, 1, 2, 9, 19):
        pool.refs[p] = -1 - p
        ref.refs[p] = -1 - p
    pool.page_table[0, :3] = i32([9, 1, 2])
    ref.table[0][:3] = [9, 1, 2]
    pool.lens[0] = ref.lens[0] = 40
    step(ops, pool, ref, "fork", [0, 0, 0])
    step(ops, pool, ref, "resize", [41, 48, 49])
    assert [ref.refs[p] for p in (0, 1, 2, 9, 19)] == [-1, -2, -3, -10, -20]
    step(ops, pool, ref, "resize", [41, 0, 80])
    moves, remap = ops.compact(pool)
    want, want_remap = ref.compact()
    assert moves_of(moves) == want and remap.tolist() == want_remap
    same(pool, ref)
    step(ops, pool, ref, "resize", [0, 0, 0])
    assert sum(r != 0 for r in ref.refs) == 5


def test_callers_own_holders_count(ops):
    pool = make_pool(ops, 1, 4, 8)
    ref = beam_ref.Pool.of(pool)
    step(ops, pool, ref, "resize", [20])
    kept = ref.table[0][:2]
    for p in kept:  # a prefix kept for later requests
        pool.refs[p] += 1
        ref.refs[p] += 1
    step(ops, pool, ref, "resize", [21])  # copies the page that is kept
    step(ops, pool, ref, "resize", [0])
    assert [ref.refs[p] for p in kept] == [1, 1] and sum(ref.refs) == 2


@pytest.mark.parametrize("batch,width,n_pages,offset", [(3, 4, 11, 0), (40, 30, 1300, 1), (200, 40, 20000, 0), (7, 9, 70, 2),
                                                        (2, 1100, 2200, 0), (1, 1, 1, 0)])
def test_compact_moves_the_pages_behind_to_the_front(ops, batch, width, n_pages, offset):
    rng = random.Random(n_pages)
    pool = make_pool(ops, batch, width, n_pages, 16, None, offset)
    ref = beam_ref.Pool.of(pool)
    ids = rng.sample(range(n_pages), min(n_pages, batch * width))
    for b in range(batch):
        n = rng.randint(0, width) if batch > 1 else width
        ref.lens[b] = max(0, n * 16 - rng.randint(0, 15)) if n else 0
        for i in range(ref.pages(ref.lens[b])):
            p = ref.table[b][i] = ref.table[b - 1][i] if b and i < 2 and i < ref.pages(ref.lens[b - 1]) else ids.pop()
            ref.refs[p] += 1
    pool.page_table.copy_(i32(ref.table))
    pool.lens.copy_(i32(ref.lens))
    pool.refs.copy_(i32(ref.refs))
    for again in range(2):  # the second finds nothing to move
        moves, remap = ops.compact(pool)
        want, want_remap = ref.compact()
        assert moves_of(moves) == want and remap.tolist() == want_remap
        assert not again or not want
        same(pool, ref)
        ref.check()
        used = sum(r > 0 for r in ref.refs)
        assert all(r > 0 for r in ref.refs[:used])


def test_pools_of_no_use_and_of_full_use(ops):
    pool = make_pool(ops, 2, 3, 6)
    ref = beam_ref.Pool.of(pool)
    for lens in ([0, 0], [48, 48]):
        step(ops, pool, ref, "resize", lens)
        moves, remap = ops.compact(pool)
        want, want_remap = ref.compact()
        assert moves_of(moves) == want == [] and remap.tolist() == want_remap
        same(pool, ref)


def test_the_largest_pool(ops):
    """8,192 sequences, 16 million pages, a table of 64-bit offsets' size in strides."""
    batch, n_pages = 8192, 1 << 24
    pool = make_pool(ops, batch, 3, n_pages, 16, 5)
    pool.refs[:n_pages - 3 * batch - 7] = 1  # all but the last ones
    lens = torch.arange(batch, device="cuda") % 49
    assert ops.resize(pool, lens.to(I32))[0, 0].item() == 0
    need = (lens + 15) // 16
    first = n_pages - 3 * batch - 7 + torch.cumsum(need, 0) - need
    col = torch.arange(3, device="cuda")
    want = torch.where(col < need[:, None], first[:, None] + col, -7)
    assert torch.equal(pool.page_table.long(), want) and pool.read_status() == 0
    parents = torch.randperm(batch, generator=gen(1), device="cuda")
    before = pool.refs.clone()
    ops.fork(pool, parents.to(I32))
    assert torch.equal(pool.lens.long(), lens[parents]) and torch.equal(pool.refs, before)
    has = col < need[parents][:, None]
    assert torch.equal(pool.page_table[has], want[parents][has].to(I32))
    pool.refs[:n_pages - 3 * batch - 7] = 0
    moves, remap = ops.compact(pool)
    used = int(need.sum())
    assert moves[0, 0].item() == used
    assert torch.equal(moves[1:used + 1, 1], torch.arange(used, device="cuda", dtype=I32))
    assert (pool.refs[:used] == 1).all() and (pool.refs[used:] == 0).all()
    assert torch.equal(pool.page_table[has], (want[parents] - (n_pages - 3 * batch - 7))[has].to(I32))
    with pytest.raises(Exception):
        ops.resize(make_pool(ops, 1, 1, 16), i32([1]), moves=torch.zeros(1, 3, dtype=I32, device="cuda"))


def test_tables_past_32_bits(ops):
    """Rows so far apart that the last ones begin past 2^31 entries; odd strides, which take entries one by one."""
    batch, width, page = 8192, 5, 16
    for stride in (270000, 270001):
        table = torch.empty(batch * stride, dtype=I32, device="cuda").as_strided((batch, width), (stride, 1))
        table.fill_(-7)
        pool = ops.PagePool(table, 5 * batch, page)
        lens = torch.arange(batch, device="cuda") * 7 % 81
        ops.resize(pool, lens.to(I32))
        need = (lens + 15) // 16
        col = torch.arange(width, device="cuda")
        want = torch.where(col < need[:, None], (torch.cumsum(need, 0) - need)[:, None] + col, -7)
        assert torch.equal(table.long(), want)
        parents = torch.arange(batch - 1, -1, -1, device="cuda")
        ops.fork(pool, parents.to(I32))
        has = col < need[parents][:, None]
        assert torch.equal(table[has].long(), want[parents][has]) and (table[~has] < 0).all()
        moves, remap = ops.compact(pool)
        assert moves[0, 0].item() == 0 and pool.read_status() == 0
        ops.resize(pool, torch.zeros_like(pool.lens))
        assert not pool.refs.any() and (table < 0).all() and pool.read_status() == 0
        del table, pool


def test_wide_tables_of_few_and_of_many_sequences(ops):
    """Columns shared out to several blocks, a grid of its own for the compaction's table, whole rows given up."""
    for batch, width in ((1, 3000), (9, 2600), (700, 130)):
        n_pages = batch * width + 9
        pool = make_pool(ops, batch, width, n_pages)
        ref = beam_ref.Pool.of(pool)
        rng = random.Random(width)
        step(ops, pool, ref, "resize", [rng.randint(0, width * 16) for _ in range(batch)])
        step(ops, pool, ref, "fork", [rng.randrange(-1, batch) for _ in range(batch)])
        ref.check()
        step(ops, pool, ref, "resize", [n // rng.choice([1, 2, 5, 10 ** 9]) for n in ref.lens])
        moves, remap = ops.compact(pool)
        want, want_remap = ref.compact()
        assert moves_of(moves) == want and remap.tolist() == want_remap
        same(pool, ref)
        ref.check()


def test_entries_behind_a_sequences_end_do_not_matter(ops):
    """Whatever they hold, the pages that come to lie there among it."""
    pool = make_pool(ops, 3, 6, 30)
    ref = beam_ref.Pool.of(pool)
    for fill in (-1, 0, 5, 2 ** 31 - 1, -2 ** 31):
        for b, n in enumerate(ref.lens):
            for i in range(ref.pages(n), 6):
                ref.table[b][i] = fill
        pool.page_table.copy_(i32(ref.table))
        step(ops, pool, ref, "resize", [33, 0, 90])
        for b, n in enumerate(ref.lens):  # the very pages that a fork brings
            for i in range(ref.pages(n), 6):
                ref.table[b][i] = ref.table[(b + 1) % 3][i]
        pool.page_table.copy_(i32(ref.table))
        step(ops, pool, ref, "fork", [1, 2, 0])
        ref.check()
        step(ops, pool, ref, "fork", [0, 0, 0])
        step(ops, pool, ref, "resize", [17, 0, 96])
        ref.check()


# ------------------------------------------------------------------ copies

ORDERS = {"psh": (0, 1, 2, 3), "phs": (0, 2, 1, 3), "hps": (1, 2, 0, 3), "sph": (1, 0, 2, 3)}


def make_caches(ops, n, n_pages, page, hkv, dim, dtype, order="psh", seed=0, at=0, wide=0):
    """n caches with random values, their dimensions in memory in the named order, `at` values into their buffers."""
    dims = {"p": n_pages, "s": page, "h": hkv}
    table = torch.zeros(1, 1, dtype=I32, device="cuda")
    out = []
    for i in range(n):
        pools = []
        for j in range(2):
            shape = [dims[c] for c in order]
            buf = torch.randn(math.prod(shape) * (dim + wide) + at, generator=gen(seed + 2 * i + j), device="cuda").to(dtype)
            t = buf[at:].view(*shape, dim + wide)[..., :dim]
            pools.append(t.permute(*[order.index(c) for c in "psh"], 3))
        out.append(ops.PagedCache(*pools, table))
    return out


def check_copies(ops, caches, moves, capacity=None, status=0):
    want = [p.clone() for c in caches for p in (c.k_pool, c.v_pool)]
    n_pages, page = caches[0].n_pages, caches[0].page_size
    for s, d, n in moves:
        if 0 <= s < n_pages and 0 <= d < n_pages:
            for w in want:
                w[d, :max(0, min(n, page))] = w[s, :max(0, min(n, page))]
    m = i32([[len(moves), 0, 0]] + [list(x) for x in moves] + [[-1, -1, 0]] * 2)
    ops.copy_pages(caches if len(caches) > 1 else caches[0], m)
    for w, p in zip(want, [p for c in caches for p in (c.k_pool, c.v_pool)]):
        assert torch.equal(w, p)
    assert caches[0].read_status() == status


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("order", sorted(ORDERS))
@pytest.mark.parametrize("page,hkv,dim,at,wide", [(64, 8, 128, 0, 0), (16, 1, 64, 0, 0), (256, 2, 128, 0, 0), (16, 5, 80, 0, 0),
                                                  (32, 3, 6, 0, 0), (64, 2, 128, 8, 0), (64, 2, 128, 1, 0), (16, 2, 64, 0, 8),
                                                  (16, 2, 64, 0, 1), (16, 40, 256, 0, 0), (16, 3, 1, 0, 0)])
def test_copies_of_whole_and_partial_pages(ops, dtype, order, page, hkv, dim, at, wide):
    rng = random.Random(page + hkv)
    caches = make_caches(ops, 2, 24, page, hkv, dim, dtype, order, 5, at, wide)
    ids = rng.sample(range(24), 22)
    counts = [page, 1, page - 1, 0, page // 2, 3, page, 2, 7, page // 2 + 1, page + 5]
    check_copies(ops, caches, [(ids[2 * i], ids[2 * i + 1], n) for i, n in enumerate(counts)])


def test_copies_of_pages_outside_the_pool_are_left_out(ops):
    caches = make_caches(ops, 3, 10, 16, 2, 64, BF16)
    check_copies(ops, caches, [(0, 10, 16), (-1, 2, 16), (3, 4, 9), (2 ** 31 - 1, 5, 1), (6, -2 ** 31, 4), (7, 8, -5)],
                 status=PAGE)
    check_copies(ops, caches, [])
    m = torch.zeros(1, 3, dtype=I32, device="cuda")
    m[0, 0] = 5  # more than there is room for
    ops.copy_pages(caches, m)
    m = i32([[9, 0, 0], [1, 2, 16]])
    caches[0].k_pool[2] = 0
    ops.copy_pages(caches, m)
    assert torch.equal(caches[0].k_pool[2], caches[0].k_pool[1])


def test_copies_in_more_caches_than_a_launch_takes(ops):
    caches = make_caches(ops, 130, 6, 16, 1, 64, F16)
    check_copies(ops, caches, [(5, 0, 16), (2, 4, 3)])


def test_copies_past_32_bits(ops):
    """Pools of more than 2^31 values: pages at their far ends."""
    n_pages, page, hkv, dim = 33000, 64, 8, 128  # 2.16e9 values a pool
    k = torch.zeros(n_pages, page, hkv, dim, dtype=BF16, device="cuda")
    v = torch.zeros(n_pages, page, hkv, dim, dtype=BF16, device="cuda")
    cache = ops.PagedCache(k, v, torch.zeros(1, 1, dtype=I32, device="cuda"))
    for p in (k, v):
        p[0].normal_(generator=gen(1))
        p[n_pages - 2].normal_(generator=gen(2))
    ops.copy_pages(cache, i32([[2, 0, 0], [0, n_pages - 1, 64], [n_pages - 2, 1, 31]]))
    for p in (k, v):
        assert torch.equal(p[n_pages - 1], p[0]) and torch.equal(p[1, :31], p[n_pages - 2, :31])
        assert not p[1, 31:].any() and not p[2:n_pages - 2].any()


# ------------------------------------------------------------------ the selection

def check_select(ops, logits, scores, n, done=None, done_token=0, status=0, exact=False):
    word = torch.zeros(1, dtype=I32, device="cuda")
    s, p, t = ops.beam_select(logits, scores, n, done=done, done_token=done_token, status=word)
    assert s.dtype is F32 and p.dtype is I32 and t.dtype is I32 and s.shape == p.shape == t.shape == (scores.shape[0], n)
    flat = beam_ref.continuations(logits, scores, done, done_token)
    want = beam_ref.select(logits, scores, n, done, done_token, flat)
    s, p, t = s.double().tolist(), p.tolist(), t.tolist()
    host = logits.float().cpu()
    beams = scores.shape[1]
    for b, w in enumerate(want):
        k = len(w)
        assert all(x == -math.inf for x in s[b][k:]) and all(x == -1 for x in p[b][k:] + t[b][k:]), b
        got = list(zip(p[b][:k], t[b][:k]))
        assert len(set(got)) == k and all(x >= y for x, y in zip(s[b], s[b][1:]))
        for i, ((x, row, token), at) in enumerate(zip(w, got)):
            tol = beam_ref.select_tolerance(x, 600)
            assert abs(s[b][i] - x) <= tol, (b, i, s[b][i], x)
            if exact:
                assert at == (row, token), (b, i)
            else:  # two rows' scores may be closer than the sums are exact
                assert at == (row, token) or abs(flat[b, at[0] - b * beams, at[1]] - x) <= 2 * tol, (b, i, at, row, token)
        for r in set(p[b][:k]):  # within a row, the logits' own order
            order = [(-host[r, v].item() + 0.0, v) for q, v in got if q == r]
            assert order == sorted(order)
    assert word.item() == status


DTYPES = [BF16, F16, F32]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("batch,beams,vocab,n", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 4), (1, 4, 151936, 8), (3, 5, 100003, 5), (2, 8, 32768, 16), (5, 2, 4097, 33),
    (1, 64, 2500, 64), (2, 33, 1001, 128), (1, 1, 300000, 128), (1, 2, 20, 64), (7, 1, 2048, 1), (300, 2, 515, 3),
    (1, 16, 70001, 24), (1, 3, 8191, 25), (2, 2, 16385, 65)])
def test_selection(ops, dtype, batch, beams, vocab, n):
    g = gen(vocab + n)
    logits = (torch.randn(batch * beams, vocab, generator=g, device="cuda") * 2.5).to(dtype)
    scores = -8 * torch.rand(batch, beams, generator=g, device="cuda")
    check_select(ops, logits, scores, n)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
def test_selection_of_strided_rows_at_every_alignment(ops, dtype):
    g = gen(3)
    for width, at in ((5003, 0), (5008, 0), (5001, 1), (5008, 3), (5004, 2), (5010, 7)):
        buf = torch.randn(6, width + 16, generator=g, device="cuda").to(dtype) * 3
        logits = buf[:, at:at + width - 1]
        scores = -torch.rand(2, 3, generator=g, device="cuda")
        check_select(ops, logits, scores, 6)
    one = torch.randn(1, 5000, generator=g, device="cuda").to(dtype)
    check_select(ops, one.expand(4, 5000), -torch.arange(4., device="cuda").view(2, 2), 5)  # one row for all


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("at,n", [(0, 48), (0, 128), (1, 48), (3, 128)])
def test_selection_from_many_large_cells(ops, dtype, at, n):
    """More vectors to look into again than the join has threads, candidates at the rows' ends, ended beams between."""
    batch, beams, vocab = 2, 24, 90001
    g = gen(n + at)
    logits = (torch.randn(batch * beams, 90008, generator=g, device="cuda") * 2.5).to(dtype)[:, at:at + vocab]
    logits[::5, 0] = 14
    logits[1::7, vocab - 1] = 13
    logits[3, 700:760] = 12.5  # one after another, equal
    scores = -2 * torch.rand(batch, beams, generator=g, device="cuda")
    done = torch.rand(batch, beams, generator=g, device="cuda") < 0.2
    check_select(ops, logits, scores, n)
    check_select(ops, logits, scores, n, done, 5)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
def test_ties_go_to_the_lowest_beam_and_token(ops, dtype):
    vocab = 9001
    flat = torch.zeros(4, vocab, dtype=dtype, device="cuda")
    check_select(ops, flat, torch.zeros(2, 2, device="cuda"), 128, exact=True)
    check_select(ops, flat, -torch.zeros(1, 4, device="cuda"), 64, exact=True)
    some = flat.clone()
    some[:, 5000:] = 1.0  # thousands of equal best ones, late
    check_select(ops, some, torch.zeros(2, 2, device="cuda"), 100, exact=True)
    zeros = flat - 5
    zeros[:, 10::700] = 0.0
    zeros[:, 17::1400] = -0.0  # the same value
    check_select(ops, zeros, torch.zeros(1, 4, device="cuda"), 40, exact=True)
    x = torch.randn(vocab, generator=gen(1), device="cuda").to(dtype)
    for stride in (vocab, vocab + 1, vocab + 7):  # equal rows at other alignments: equal sums
        rows = torch.empty(5 * stride, dtype=dtype, device="cuda")[:5 * stride].view(5, stride)[:, :vocab]
        rows.copy_(x.expand(5, vocab))
        check_select(ops, rows, torch.full((1, 5), -2.5, device="cuda"), 20, exact=True)
    up = torch.arange(vocab, device="cuda", dtype=F32).div(vocab).to(dtype).expand(4, vocab)  # ascending
    check_select(ops, up.contiguous(), torch.zeros(4, 1, device="cuda"), 128, exact=True)
    check_select(ops, up.flip(1).contiguous(), torch.zeros(4, 1, device="cuda"), 128, exact=True)


@pytest.mark.parametrize("batch,beams,vocab,n", [(1, 1, 300000, 128), (2, 16, 151936, 128), (1, 64, 40001, 5), (3, 2, 70000, 64)])
def test_ties_in_every_part_of_many_rows(ops, batch, beams, vocab, n):
    """Every cell reaches the bound, thousands of candidates are equal: taken in turns, the lowest of them kept."""
    g = gen(n)
    flat = torch.zeros(batch * beams, vocab, dtype=BF16, device="cuda")
    check_select(ops, flat, torch.zeros(batch, beams, device="cuda"), n, exact=True)
    few = torch.randint(0, 3, (batch * beams, vocab), generator=g, device="cuda").to(BF16)
    check_select(ops, few, -torch.arange(float(beams), device="cuda").repeat(batch, 1) / 8, n)
    few[:, : vocab // 2] = -math.inf
    few[beams - 1] = -math.inf
    check_select(ops, few, -torch.rand(batch, beams, generator=g, device="cuda"), n)


def test_selection_past_32_bits(ops):
    """More than 2^32 bytes and 2^31 values of logits: the last rows as by themselves."""
    rows, vocab = 14400, 151936
    logits = torch.empty(rows, vocab, dtype=BF16, device="cuda")
    for i in range(0, rows, 1600):
        logits[i:i + 1600].normal_(generator=gen(i))
    scores = -torch.rand(rows // 4, 4, generator=gen(1), device="cuda")
    got = ops.beam_select(logits, scores, 6)
    for b in (0, rows // 8, rows // 4 - 2):
        want = ops.beam_select(logits[4 * b:4 * b + 8], scores[b:b + 2], 6)
        for i in range(2):  # other parts of the rows: sums equal to rounding
            assert torch.equal(got[1][b + i], want[1][i] + 4 * b) and torch.equal(got[2][b + i], want[2][i])
            assert ((got[0][b + i] - want[0][i]).abs() <= 2 * beam_ref.select_tolerance(16.0, 600)).all()
    assert torch.equal(got[2][5], beam_selected(logits[20:24], scores[5:6], 6))


@pytest.mark.parametrize("dtype,beams", [(F32, 1), (BF16, 3), (F16, 40)], ids=["f32", "bf16", "f16"])
def test_the_largest_vocabulary(ops, dtype, beams):
    """Rows of 2^24 tokens, their best ones where cells are widest: at the ends, across parts, next to one another."""
    vocab = 1 << 24
    logits = torch.randn(beams, vocab, generator=gen(beams), device="cuda", dtype=dtype)
    for k in range(beams):
        for i, at in enumerate((0, 1, vocab // 3, vocab // 2 - 1, vocab // 2, vocab - 2, vocab - 1)):
            logits[k, at] = 12 + (i + k) % 7
    scores = -torch.arange(float(beams), device="cuda").view(1, beams) / 64
    s, p, t = ops.beam_select(logits, scores, 9)
    x = logits.double()
    flat = (x - torch.logsumexp(x, -1, keepdim=True) + scores.double().view(-1, 1)).flatten()
    at = p[0].long() * vocab + t[0].long()
    best = torch.topk(flat, 9).values
    assert len(set(at.tolist())) == 9
    # the sums' terms are 2^24 in number: what a thread adds up, 2^24 / (32 * 256), is the longest run of them
    assert ((flat[at] - best).abs() <= 2 * beam_ref.select_tolerance(16.0, 2 ** 24 / 8192)).all()
    assert ((s[0].double() - best).abs() <= beam_ref.select_tolerance(16.0, 2 ** 24 / 8192)).all()


def beam_selected(logits, scores, n):
    return i32([t for _, _, t in beam_ref.select(logits, scores, n)[0]])


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
def test_masked_tokens_and_dead_beams(ops, dtype):
    g = gen(9)
    low = torch.finfo(dtype).min
    for fill in (-math.inf, low):
        logits = (torch.randn(9, 40003, generator=g, device="cuda") * 2).to(dtype)
        logits[0] = fill                     # a row that its mask leaves nothing
        logits[1, 1:] = fill                 # one token
        logits[2, torch.rand(40003, generator=g, device="cuda") < 0.999] = fill
        logits[3, :39000] = fill             # whole parts of a row
        logits[4, 7:] = fill
        logits[5, 100:40002] = fill
        scores = -torch.rand(3, 3, generator=g, device="cuda")
        check_select(ops, logits, scores, 12)
        check_select(ops, logits[:1], scores[:1, :1].contiguous(), 9, exact=True)
        scores[0, 2] = scores[1, 0] = scores[2] = -math.inf
        check_select(ops, logits, scores, 128)
        first = torch.full((3, 3), -math.inf, device="cuda")
        first[:, 0] = 0
        check_select(ops, logits, first, 6)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16", "f32"])
def test_nan_and_infinity_are_not_offered(ops, dtype):
    g = gen(10)
    logits = (torch.randn(8, 30001, generator=g, device="cuda") * 2).to(dtype)
    scores = -torch.rand(2, 4, generator=g, device="cuda")
    check_select(ops, logits, scores, 9)
    logits[1, 5] = math.nan
    logits[1, 29999] = math.inf
    logits[2, 12000:24000] = math.nan
    logits[3] = math.inf
    logits[6, 30000] = math.nan
    check_select(ops, logits, scores, 9, status=NAN)
    logits[:] = math.nan
    check_select(ops, logits, scores, 9, status=NAN)
    logits[:] = 0
    scores[0, 0], scores[1, 1], scores[1, 2] = math.nan, math.inf, -math.inf
    check_select(ops, logits, scores, 9, status=NAN, exact=True)


def test_logits_of_every_size(ops):
    """Large and tiny ones, beyond what exponents hold; f32's whole range."""
    g = gen(11)
    for scale in (1e-30, 1e-3, 50., 1e4, 1e6, 1e20, 1e30, 3e38):
        for at in (0.0, 1.0, -1.0):
            x = (torch.rand(3, 20011, generator=g, device="cuda") * 2 - 1)
            logits = x * scale if at == 0 else at * scale * (1 - 0.1 * x.abs())
            check_select(ops, logits, -torch.rand(1, 3, generator=g, device="cuda"), 10)
    deep = torch.randn(4, 9000, generator=g, device="cuda")
    check_select(ops, deep, torch.tensor([[-3e38, -3.3e38], [-1e30, -2e30]], device="cuda"), 4, exact=False)


@pytest.mark.parametrize("n", [1, 4, 9])
def test_ended_beams_go_on_as_they_are(ops, n):
    g = gen(12)
    for beams in (1, 4):
        logits = torch.randn(6 * beams, 5000, generator=g, device="cuda").to(BF16)
        logits[0] = math.nan  # an ended beam's row is not read
        scores = -4 * torch.rand(6, beams, generator=g, device="cuda") - 3
        done = torch.rand(6, beams, generator=g, device="cuda") < 0.5
        done[0, 0] = True
        done[5] = True
        scores[5, 0] = -math.inf  # ended and dead: nothing
        check_select(ops, logits, scores, n, done, 4999)
        check_select(ops, logits, scores, n, done.to(torch.uint8) * 7, 0)


def test_selection_writes_only_its_outputs(ops):
    """Outputs of the caller's, the scores in place, a workspace of its own, larger than it needs."""
    g = gen(13)
    logits = torch.randn(8, 3001, generator=g, device="cuda").to(F16)
    scores = -torch.rand(2, 4, generator=g, device="cuda")
    want = ops.beam_select(logits, scores)
    keep = [x.clone() for x in (logits, scores)]
    bufs = [torch.full((4, 4), 77, dtype=d, device="cuda") for d in (F32, I32, I32)]
    nbytes = ops.beam_workspace(2, 4, 3001, 4, F16)
    ws = torch.full((nbytes + 256,), 77, dtype=torch.uint8, device="cuda")
    out = ops.beam_select(logits, scores, out=[x[1:3] for x in bufs], workspace=ws)
    for o, w, buf in zip(out, want, bufs):
        assert torch.equal(o, w) and (buf[0] == 77).all() and (buf[3] == 77).all()
    assert (ws[nbytes:] == 77).all() and torch.equal(logits, keep[0]) and torch.equal(scores, keep[1])
    got = ops.beam_select(logits, scores, out=(scores, bufs[1][:2], bufs[2][:2]))
    assert got[0] is scores and all(torch.equal(x, w) for x, w in zip(got, want))


def test_an_empty_batch(ops):
    s, p, t = ops.beam_select(torch.zeros(0, 50, dtype=BF16, device="cuda"), torch.zeros(0, 4, device="cuda"))
    assert s.shape == p.shape == t.shape == (0, 4)


# ------------------------------------------------------------------ streams, graphs, devices

def test_on_a_stream_and_in_a_graph(ops):
    """The step of a search captured and replayed, on the stream given; a replay does what a call does."""
    g = gen(14)
    batch, beams, vocab = 3, 4, 2000
    rows = batch * beams
    logits = torch.randn(rows, vocab, generator=g, device="cuda")
    scores = -torch.rand(batch, beams, generator=g, device="cuda")
    pool, twin = (make_pool(ops, rows, 10, 200) for _ in range(2))
    caches = make_caches(ops, 2, 200, 16, 2, 64, BF16)
    twins = make_caches(ops, 2, 200, 16, 2, 64, BF16)
    lens = i32([30] * rows)
    for p in (pool, twin):
        ops.resize(p, lens)

    def one(pool, caches, scores, stream=None):
        s, parents, tokens = ops.beam_select(logits, scores, stream=stream)
        ops.fork(pool, parents.view(-1), stream=stream)
        new = pool.lens + 1
        moves = ops.resize(pool, new, stream=stream)
        ops.copy_pages(caches, moves, stream=stream)
        m2, remap = ops.compact(pool, stream=stream)
        ops.copy_pages(caches, m2, stream=stream)
        scores.copy_(s)
        return tokens

    a, b = scores.clone(), scores.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tokens = one(pool, caches, a, side)
    for _ in range(5):
        graph.replay()
        want = one(twin, twins, b)
        assert torch.equal(tokens, want) and torch.equal(a, b)
        assert torch.equal(pool.page_table, twin.page_table) and torch.equal(pool.refs, twin.refs)
        for c, d in zip(caches, twins):
            assert torch.equal(c.k_pool, d.k_pool) and torch.equal(c.v_pool, d.v_pool)
    assert pool.read_status() == 0 and twin.read_status() == 0
    ref = beam_ref.Pool.of(pool)
    ref.check()


def test_two_pools_and_two_selections_at_once(ops):
    g = gen(15)
    streams = [torch.cuda.Stream() for _ in range(2)]
    logits = [torch.randn(16, 60000, generator=g, device="cuda").to(BF16) for _ in range(2)]
    scores = [-torch.rand(4, 4, generator=g, device="cuda") for _ in range(2)]
    want = [ops.beam_select(x, y) for x, y in zip(logits, scores)]
    pools = [make_pool(ops, 16, 40, 3000) for _ in range(2)]
    refs = [beam_ref.Pool.of(p) for p in pools]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(10):
        new = i32([(b * 37 + i * 50) % 600 for b in range(16)])
        parents = i32([(b * 5 + i) % 16 for b in range(16)])
        torch.cuda.synchronize()
        for j, s in enumerate(streams):
            got[j].append(ops.beam_select(logits[j], scores[j], stream=s))
            ops.resize(pools[j], new, stream=s)
            ops.fork(pools[j], parents, stream=s)
            refs[j].resize(new.tolist())
            refs[j].fork(parents.tolist())
    torch.cuda.synchronize()
    for j in range(2):
        for o in got[j]:
            assert all(torch.equal(x, y) for x, y in zip(o, want[j]))
        same(pools[j], refs[j])


FIRST_STEP = """
import torch
from block_diffusion_speculative_hiddens_gb300 import ops
i32 = dict(dtype=torch.int32, device="cuda")
B = %d
logits = torch.arange(B * 300., device="cuda").view(B, 300).bfloat16()
scores = torch.zeros(B // 4, 4, device="cuda")
table = torch.full((B, 9), -1, **i32)
refs, lens, status = torch.zeros(20 * B, **i32), torch.zeros(B, **i32), torch.zeros(1, **i32)
pool = ops.PagePool(table, 20 * B, 16, refs=refs, lens=lens)
k, v = (torch.zeros(20 * B, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
cache = ops.PagedCache(k, v, table)
new = torch.full((B,), 40, **i32)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    m0 = ops.resize(pool, new)
    ops.copy_pages(cache, m0)
    s, p, t = ops.beam_select(logits, scores, status=status)
    ops.fork(pool, p.view(-1))
    m1, remap = ops.compact(pool)
    ops.copy_pages(cache, m1)
g.replay()
torch.cuda.synchronize()
assert pool.read_status() == 0 and cache.read_status() == 0 and (lens == 40).all()
assert int(refs.sum()) == 3 * B and m0[0, 0].item() == 0
assert (p >= 0).all() and (t >= 0).all() and torch.isfinite(s).all()
"""


@pytest.mark.parametrize("batch", [4, 2048])
def test_first_step_of_a_process_may_be_captured(batch):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_STEP % batch], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ together

def test_a_beam_search_over_a_paged_cache(ops):
    """A small target of one layer searched with these operators -- selection, fork, resize, copies, append,
    attention -- against a search that keeps each beam's tokens and runs the layer over them in 64 bits."""
    g = gen(16)
    vocab, hq, hkv, dim, beams, batch, page, steps = 211, 4, 2, 64, 3, 2, 16, 22
    emb = torch.randn(vocab, hq * dim, generator=g, device="cuda").div(4).to(BF16)
    wq, wk, wv = (torch.randn(hq * dim, h * dim, generator=g, device="cuda").div(16).to(BF16) for h in (hq, hkv, hkv))
    head = torch.randn(hq * dim, vocab, generator=g, device="cuda").div(8).to(BF16)
    prompts = [torch.randint(0, vocab, (n,), generator=g, device="cuda").tolist() for n in (13, 40)]
    plan = ops.RopePlan(dim, 1e4)
    rows, n_pages = batch * beams, 60
    table = torch.zeros(rows, 8, dtype=I32, device="cuda")
    cache = ops.PagedCache(*(torch.zeros(n_pages, page, hkv, dim, dtype=BF16, device="cuda") for _ in range(2)), table)
    pool = ops.PagePool(table, n_pages, page)

    def layer(tokens, cu, ctx):
        x = emb[tokens]
        q, k, v = ((x.float() @ w.float()).to(BF16).view(len(tokens), -1, dim) for w in (wq, wk, wv))
        q = ops.append(cache, k, v, cu, ctx, plan=plan, q=q)
        o = ops.attention(cache, q, cu, ctx)
        return (x.float() + o.float().flatten(1)) @ head.float() / 4

    # the prompt once a request, then its row handed to every beam
    new = [len(prompts[b // beams]) if b % beams == 0 else 0 for b in range(rows)]
    ops.copy_pages(cache, ops.resize(pool, i32(new)))
    cu = i32([sum(new[:i]) for i in range(rows + 1)])
    flat = torch.tensor(sum(prompts, []), device="cuda")
    logits = layer(flat, cu, i32([0] * rows))[(cu[1:] - 1).long().clamp(min=0)]
    ops.fork(pool, i32([b // beams * beams for b in range(rows)]))
    scores = torch.full((batch, beams), -math.inf, device="cuda")
    scores[:, 0] = 0
    seqs = [list(prompts[b // beams]) for b in range(rows)]
    done = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
    one = i32(list(range(rows + 1)))
    end = 5

    def dense_logits(seq):
        """The layer over a whole sequence, in 64 bits but for the roundings that the cache makes."""
        from tests import ops_ref
        x = emb[torch.tensor(seq, device="cuda")]
        q, k, v = ((x.float() @ w.float()).to(BF16).view(len(seq), -1, dim) for w in (wq, wk, wv))
        freq, amp = ops_ref.frequencies(dim, 1e4)
        pos = torch.arange(len(seq), device="cuda")
        q, k = (ops_ref.rotate(t, pos, dim, freq, amp, False)[0].to(BF16) for t in (q, k))
        o = ops_ref.attention(q[-1:], k, v, len(seq) - 1, len(seq), True, 0, dim ** -0.5)[0]
        return (x[-1:].double() + o.to(BF16).double().flatten(1)) @ head.double() / 4

    for i in range(steps):
        # what each beam's logits should be, from its tokens alone
        for b in range(rows):
            if done.view(-1)[b] or scores.view(-1)[b] == -math.inf:
                continue
            want = dense_logits(seqs[b])[0]
            # bf16 roundings of q, k and o that fall the other way: a step of 2^-8 of |o| <= 4 in a few of 256 values
            # times head / 4 of about 1/32: well below 0.05
            assert (logits[b].double() - want).abs().max() < 0.05, (i, b)
        picked = beam_ref.select(logits, scores, beams, done, end)
        scores, parents, tokens = ops.beam_select(logits, scores, done=done, done_token=end)
        for b in range(batch):
            assert [(r, t) for _, r, t in picked[b]] == list(zip(parents[b].tolist(), tokens[b].tolist()))
        par, tok = parents.view(-1), tokens.view(-1)
        done = done.view(-1)[par.long()].view(batch, beams) | (tokens == end)
        seqs = [seqs[p] + [t] for p, t in zip(par.tolist(), tok.tolist())]
        ctx_now = pool.lens.clone()
        ops.fork(pool, par)
        ctx = pool.lens.clone()
        ops.copy_pages(cache, ops.resize(pool, ctx + 1))
        if i % 5 == 3:
            ops.copy_pages(cache, ops.compact(pool)[0])
        logits = layer(tok.long(), one, ctx)
        beam_ref.Pool.of(pool).check()
        assert (pool.lens == ctx_now[par.long()] + 1).all()
    assert pool.read_status() == 0 and cache.read_status() == 0
    shared = sum(r > 1 for r in pool.refs.tolist())
    assert shared > 0  # the beams still hold their prompts' pages together
    ops.resize(pool, torch.zeros_like(pool.lens))
    assert not pool.refs.any()
