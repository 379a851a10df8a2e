"""Selection and page calls at the limits of what they accept: logits too large for
a shared exponent, the longest sums, counts that are too low, calls that find no
pages, tables wider than any length."""
import pytest
import torch

from tests import beam_ref
from tests.test_gpu_beam import BF16, F16, F32, I32, PAGE, check_select, gen, i32, make_pool, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    from block_diffusion_speculative_hiddens_gb300 import ops as m
    return m


# ------------------------------------------------------------------ large logits

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [3e8, 1e9, 5e9, 1e10, 1e12, 1e20, 2.4e38, None])
def test_one_large_logit_among_ordinary_ones(ops, dtype, value):
    """A token that is forced by a large logit, up to the type's largest, and one that is masked by its negative."""
    value = torch.finfo(dtype).max if value is None else value
    g = gen(21)
    vocab = 20011
    for at in (0, 12345, vocab - 1):
        logits = (torch.randn(3, vocab, generator=g, device="cuda") * 2).to(dtype)
        logits[0, at] = value
        logits[1, at] = -value
        scores = -torch.rand(1, 3, generator=g, device="cuda")
        check_select(ops, logits, scores, 7)
        check_select(ops, logits[:1], scores[:, :1].contiguous(), 5)  # the others far below it


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [1.7e7, 6e7, 1e8, 4e8, 7e8, 1e9, 1.39e9, 1.41e9, 1.8e9, 2.0 ** 31, 2.5e9, 1e10])
def test_rows_of_large_logits(ops, dtype, value):
    """Rows of one large value, of either sign, and of values close to it."""
    g = gen(22)
    for sign in (1, -1):
        flat = torch.full((4, 9001), sign * value, device="cuda").to(dtype)
        check_select(ops, flat, torch.zeros(2, 2, device="cuda"), 40, exact=True)
        near = (sign * value * (1 - 0.1 * torch.rand(3, 20011, generator=g, device="cuda"))).to(dtype)
        check_select(ops, near, -torch.rand(1, 3, generator=g, device="cuda"), 10)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fill", [-1e4, -3e7, -1e9, -1.5e9, -1e10, -1e30, -3e38])
def test_masks_of_every_size(ops, dtype, fill):
    """Rows masked by a large negative value: wholly, but for a token, but for their beginning; more of them wanted
    than are not masked."""
    g = gen(23)
    vocab = 70001
    for at in (0, 1):
        logits = (torch.randn(6, vocab + 7, generator=g, device="cuda") * 2).to(dtype)[:, at:at + vocab]
        logits[0] = fill
        logits[1, :vocab - 1] = fill
        logits[2, 20000:] = fill
        logits[3, torch.rand(vocab, generator=g, device="cuda") < 0.999] = fill
        logits[4, 3:] = fill
        scores = -torch.rand(2, 3, generator=g, device="cuda")
        check_select(ops, logits, scores, 12)
        check_select(ops, logits[4:5], scores[:1, :1].contiguous(), 8)
        check_select(ops, logits[:1], scores[:1, :1].contiguous(), 8, exact=True)


# ------------------------------------------------------------------ long sums

@pytest.mark.parametrize("dtype,most,tops", [
    (F16, -0.59375, (3.0, 3.125, 3.25, 3.375, 3.5)), (BF16, 0.4375, (3.0, 3.125, 3.25, 3.375, 3.5)),
    (F32, -1.46875, (3.0, 3.125, 3.25, 3.375, 3.5)), (F32, 2.0 ** 24 + 2, (2.0 ** 24 + 4,))],
    ids=["f16", "bf16", "f32", "large"])
def test_sums_of_the_longest_rows(ops, dtype, most, tops):
    """320 rows of 2^24 tokens, too many to be split: thousands of equal terms a thread, whose roundings add up in a
    32-bit sum that takes them all."""
    vocab, batch, beams, n = 1 << 24, 5, 64, 8
    row = torch.full((1, vocab), most, dtype=dtype, device="cuda")
    at = (0, vocab // 3, vocab // 2, vocab - 2, vocab - 1)[:len(tops)]
    for token, x in zip(at, tops):
        row[0, token] = x
    scores = -0.0101 * torch.arange(float(beams), device="cuda").repeat(batch, 1)
    s, p, t = ops.beam_select(row.expand(batch * beams, vocab), scores, n)
    lse = torch.logsumexp(row[0].double(), 0).item()
    want = sorted(((b + x - lse, -k, token) for k, b in enumerate(scores[0].tolist()) for token, x in zip(at, tops)), reverse=True)[:n]
    for b in range(batch):
        assert t[b].tolist() == [w[2] for w in want] and p[b].tolist() == [b * beams - w[1] for w in want]
        for got, (x, _, _) in zip(s[b].tolist(), want):
            # a thread's two floats take 256 terms each at most before they are added to a 64-bit sum:
            # units of 2^-34, at most 2^15 roundings of half of one beside a sum above 1/2
            assert abs(got - x) <= beam_ref.select_tolerance(x, 512) + 2.0 ** -19, (b, got, x)


# ------------------------------------------------------------------ counts that are too low

def shared(ops, batch, held):
    """A pool whose first `held` rows hold the same three pages, the others nothing."""
    pool = make_pool(ops, batch, 4, 4 * batch + 8)
    ref = beam_ref.Pool.of(pool)
    step(ops, pool, ref, "resize", [40] + [0] * (batch - 1))
    step(ops, pool, ref, "fork", [0 if b < held else -1 for b in range(batch)])
    return pool, ref


def recount(pool, ref, counts):
    for p, n in zip(ref.table[0], counts):
        ref.refs[p] = n
        pool.refs[p] = n


@pytest.mark.parametrize("batch", [2, 3, 40, 600, 1500])
def test_counts_that_are_too_low_do_not_pin_pages(ops, batch):
    """More entries give up a page than it has holders: flagged, the count ends at 0, and the page is free."""
    for counts in ((1, 1, 1), (0, batch - 1, 1)):
        for what, arg in (("resize", [0] * batch), ("fork", [-1] * batch)):
            pool, ref = shared(ops, batch, batch)
            recount(pool, ref, counts)
            step(ops, pool, ref, what, arg, PAGE)
            assert not any(ref.refs) and min(pool.refs.tolist()) == 0
            step(ops, pool, ref, "resize", [b % 60 for b in range(batch)])  # and serves again
            ref.check()


def status_of(ref, what, arg):
    want = beam_ref.Pool(ref.refs, ref.table, ref.lens, ref.page)
    getattr(want, what)(arg)
    return want.status


@pytest.mark.parametrize("batch", [3, 4, 40, 600])
def test_counts_that_are_too_low_and_copies(ops, batch):
    """All of them grow in a page that has two holders by its count: each but the first gives it up."""
    pool, ref = shared(ops, batch, batch)
    recount(pool, ref, (batch, batch, 2))
    grown = [41] * batch
    assert status_of(ref, "resize", grown) == (PAGE if batch > 3 else 0)
    step(ops, pool, ref, "resize", grown, PAGE if batch > 3 else 0)


@pytest.mark.parametrize("batch", [6, 64, 1500])
def test_counts_that_are_too_low_and_new_holders(ops, batch):
    """In which order a fork counts them is open: the count ends between all that are left and 0."""
    keeps, first = batch // 2 - 1, batch - batch // 3  # the only row of the old ones that stays; the new ones
    pool, ref = shared(ops, batch, keeps + 1)
    recount(pool, ref, (1, 2, keeps))
    pages = ref.table[0][:3]
    parents = [keeps if b == keeps or b >= first else -1 for b in range(batch)]
    ops.fork(pool, i32(parents))
    status = pool.read_status()
    ref.fork(parents)
    assert pool.page_table.tolist() == ref.table and pool.lens.tolist() == ref.lens
    assert all(ref.refs[p] <= pool.refs[p].item() <= batch - first + 1 for p in pages)
    assert status == PAGE or (status == ref.status and pool.refs.tolist() == ref.refs)


@pytest.mark.parametrize("batch", [3, 600, 1500])
def test_pins_of_every_size(ops, batch):
    """Pinned pages that many take and give up in one call keep their counts, the lowest values among them."""
    pins = (-1, -2 ** 31, -2 ** 31 + 5)
    pool, ref = shared(ops, batch, 1)
    recount(pool, ref, pins)
    some = [0 if b % 3 else -1 for b in range(batch)]
    some[0] = 0
    for what, arg in (("fork", [0] * batch), ("fork", some), ("fork", [0] * batch), ("resize", [20 if b % 2 else 40 for b in range(batch)]),
                      ("fork", [0] * batch), ("resize", [41] * batch), ("resize", [0] * batch)):
        step(ops, pool, ref, what, arg)
        assert [ref.refs[p] for p in range(3)] == list(pins)


# ------------------------------------------------------------------ no pages

@pytest.mark.parametrize("n_pages,fail", [(8, 3), (4, 16)])
def test_nothing_is_appended_to_sequences_without_room(ops, n_pages, fail):
    """A captured step of beams on shared pages, replayed where their pool is used up, or too small for the copies
    from the start: its rows have no place, what the cache holds stays as it was, and pages that are given back serve
    again."""
    rows, page, hkv, dim = 4, 16, 2, 64
    g = gen(31)
    table = torch.zeros(rows, 6, dtype=I32, device="cuda")
    cache = ops.PagedCache(*(torch.randn(n_pages, page, hkv, dim, generator=g, device="cuda").to(BF16) for _ in range(2)), table)
    pool = ops.PagePool(table, n_pages, page)
    ops.resize(pool, i32([20, 0, 0, 0]))
    ops.fork(pool, i32([0, 0, 0, 0]))  # two pages, the last of them to be copied
    ref = beam_ref.Pool.of(pool)
    k, v, q = (torch.randn(rows, hkv, dim, generator=g, device="cuda").to(BF16) for _ in range(3))
    cu = i32(range(rows + 1))
    out = torch.empty_like(q)

    def one(step):
        ctx = pool.lens.clone()
        new = ctx + step
        ops.copy_pages(cache, ops.resize(pool, new))
        ctx = torch.where(pool.lens == new, ctx, -2 ** 31)
        ops.append(cache, k, v, cu, ctx)
        ops.attention(cache, q, cu, ctx, out=out)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one(1)

    def kept():  # what each sequence holds
        return [torch.cat([p[t].flatten(0, 1)[:n] for p in (cache.k_pool, cache.v_pool)])
                for t, n in ((table[b].long().clamp(0, n_pages - 1), n) for b, n in enumerate(pool.lens.tolist()))]

    failed = 0
    for turn in range(16):
        before, pools = kept(), [cache.k_pool.clone(), cache.v_pool.clone()]
        new = [n + 1 for n in ref.lens]
        ref.resize(new)
        graph.replay()
        assert pool.lens.tolist() == ref.lens and pool.read_status() == ref.status
        if ref.status:
            failed += 1
            assert torch.equal(cache.k_pool, pools[0]) and torch.equal(cache.v_pool, pools[1])
            assert cache.read_status() == PAGE and not out.any()
        else:
            for b, (x, y, n) in enumerate(zip(before, kept(), ref.lens)):
                x, y = x.view(2, n - 1, hkv, dim), y.view(2, n, hkv, dim)
                assert torch.equal(x, y[:, :-1]) and torch.equal(y[0, -1], k[b]) and torch.equal(y[1, -1], v[b])
            assert cache.read_status() == 0 and out.abs().sum(-1).min() > 0
        ref.status = 0
        if turn == 14:  # one ends
            step(ops, pool, ref, "fork", [-1, 1, 2, 3])
    assert failed == fail


# ------------------------------------------------------------------ wide tables

def test_a_table_wider_than_any_length(ops):
    """One row of 2^31 - 1 entries, most of which no length reaches."""
    width, page = 2 ** 31 - 1, 16
    table = torch.empty(1, width, dtype=I32, device="cuda")
    table[:, :50] = -7
    pool = ops.PagePool(table, 60, page)
    new = i32([0])
    for n in (700, 300, 301, 0, 640):
        assert ops.resize(pool, new.fill_(n))[0, 0].item() == 0
        held = -(-n // page)
        assert pool.lens.item() == n and sorted(table[0, :held].tolist()) == list(range(held))
        assert pool.refs.tolist() == [1] * held + [0] * (60 - held)
    pool.refs[40:45] = pool.refs[:5].clone()
    pool.refs[:5] = 0
    table[0, :5] = i32([44, 43, 42, 41, 40])
    moves, remap = ops.compact(pool)
    assert moves[0, 0].item() == 5 and table[0, :40].tolist() == [4, 3, 2, 1, 0] + list(range(5, 40))
    ops.fork(pool, i32([0]))
    ops.fork(pool, i32([-1]))
    assert not pool.refs.any() and (table[0, :40] == -1).all() and pool.lens.item() == 0 and pool.read_status() == 0
