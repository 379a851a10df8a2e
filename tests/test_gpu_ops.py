"""The caller-target operators (rotary positions, append to a paged cache,
attention over it) against their 64-bit definitions, at the sizes and masks
where they can go wrong, and a run of them together as a target uses them."""
import math

import pytest
import torch

from tests import ops_ref

pytestmark = pytest.mark.gpu

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32


@pytest.fixture(scope="module")
def ops(lib):
    from block_diffusion_speculative_hiddens_gb300 import ops as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def close(got, want, tol, what=""):
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    off = ((got - want).abs() - tol)[torch.isfinite(want)]
    assert off.numel() == 0 or off.max().item() <= 0, (what, off.max().item())


YARN = {"kind": "yarn", "factor": 4.0, "original_len": 32768}
LLAMA3 = {"kind": "llama3", "factor": 8.0, "original_len": 8192}


# ------------------------------------------------------------------ rope

@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("rows,hq,hk,dim,rd,scaling", [
    (1, 1, 1, 64, 64, None), (16, 32, 8, 128, 128, None), (5, 3, 2, 128, 64, YARN), (33, 4, 1, 64, 16, LLAMA3),
    (3, 2, 2, 80, 20, None), (2, 1, 1, 2, 2, None), (7, 5, 1, 256, 256, {"kind": "linear", "factor": 3.0}),
    (9, 2, 1, 96, 96, {"kind": "ntk", "factor": 4.0}), (6000, 3, 1, 128, 96, None)])
def test_rope_matches_its_formula(ops, dtype, inter, rows, hq, hk, dim, rd, scaling):
    g = gen(rows)
    q = torch.randn(rows, hq, dim, generator=g, device="cuda").to(dtype)
    k = torch.randn(rows, hk, dim, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1000000, (rows,), generator=g, device="cuda").to(I32)
    pos[0] = 2 ** 31 - 1
    plan = ops.RopePlan(rd, 5e5, interleaved=inter, scaling=scaling)
    freq, amp = ops_ref.frequencies(rd, 5e5, scaling)
    for backward in (False, True):
        got = ops.rope(plan, q, k, pos, backward=backward)
        for x, y in zip((q, k), got):
            want, mag = ops_ref.rotate(x, pos, rd, freq, amp, inter, backward)
            close(y, want, ops_ref.rotate_tolerance(want, mag, dtype), (backward,))
            assert torch.equal(y[..., rd:], x[..., rd:])


def test_rope_of_strided_views_in_place_and_apart(ops):
    """Views of a fused projection; unaligned heads; one tensor alone; an output of its own strides."""
    plan = ops.RopePlan(64, 1e4)
    freq, amp = ops_ref.frequencies(64, 1e4)
    pos = torch.arange(40, 53, device="cuda").to(I32)
    for width, at in ((128, 0), (128, 8), (131, 1)):  # aligned heads, an offset, odd strides
        buf = torch.randn(13, 7, width, generator=gen(width + at), device="cuda").to(BF16)
        x = buf[:, :, at:at + 96]
        q, k = x[:, :4], x[:, 4:6]
        want = [ops_ref.rotate(t, pos, 64, freq, amp, False) for t in (q, k)]
        out = torch.zeros(4, 13, 100, dtype=BF16, device="cuda")[:, :, 2:98].transpose(0, 1)
        got = ops.rope(plan, q, k, pos, q_out=out)
        assert got[0] is out
        rest = buf.clone()
        here = ops.rope(plan, q, k, pos, q_out=q, k_out=k)  # in place
        for (w, m), y, z in zip(want, got, here):
            close(y, w, ops_ref.rotate_tolerance(w, m, BF16))
            assert torch.equal(y, z)
        rest[:, :6, at:at + 96] = buf[:, :6, at:at + 96]
        assert torch.equal(rest, buf)  # nothing beside the heads was written
    alone, none = ops.rope(plan, q, None, pos)
    assert none is None and alone.shape == q.shape


def test_rope_backward_is_the_gradient(ops):
    """Against the formula's own gradient (autograd of the 64-bit rotation) and against differences of the kernel."""
    for inter, scaling in ((False, None), (True, YARN)):
        plan = ops.RopePlan(32, 1e4, interleaved=inter, scaling=scaling)
        freq, amp = ops_ref.frequencies(32, 1e4, scaling)
        g = gen(3)
        x = torch.randn(5, 2, 48, generator=g, device="cuda").to(F16)
        dy = torch.randn(5, 2, 48, generator=g, device="cuda").to(F16)
        pos = i32([0, 1, 77, 4000, 131071])
        got, _ = ops.rope(plan, dy, None, pos, backward=True)
        leaf = x.double().requires_grad_()
        angle = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
        c, s = (torch.cos(angle) * amp)[:, None], (torch.sin(angle) * amp)[:, None]
        a, b = (leaf[..., 0:32:2], leaf[..., 1:32:2]) if inter else (leaf[..., :16], leaf[..., 16:32])
        y = torch.cat((a * c - b * s, a * s + b * c, leaf[..., 32:]), -1)
        grad = dy.double()
        order = torch.cat((grad[..., 0:32:2], grad[..., 1:32:2], grad[..., 32:]), -1) if inter else grad
        want, = torch.autograd.grad(y, leaf, order)
        _, mag = ops_ref.rotate(dy, pos, 32, freq, amp, inter, True)
        close(got, want, ops_ref.rotate_tolerance(want, mag, F16))
        # differences: the map is linear, so <dy, R(x + e) - R(x)> = <R'dy, e> for a step e of 1 in one value
        for i in (0, 1, 16, 31, 40):
            e = torch.zeros_like(x)
            e[..., i] = 1
            r0, r1 = (ops.rope(plan, t, None, pos)[0].double() for t in (torch.zeros_like(x), e))
            diff = (dy.double() * (r1 - r0)).sum(-1)
            lim = 2.0 ** -11 * (dy.double().abs() * (r1 - r0).abs()).sum(-1) + 2.0 ** -11 * want[..., i].abs() + 1e-5
            assert ((diff - got[..., i].double()).abs() <= lim).all()


def test_rope_of_nothing(ops):
    plan = ops.RopePlan(64, 1e4)
    q, k = ops.rope(plan, torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), None, i32([]))
    assert q.shape == (0, 4, 64) and k is None


# ------------------------------------------------------------------ a paged cache

class Paged:
    """Pools in one of several orders, pages handed out in random order, and the plain keys and values behind them."""

    def __init__(self, ops, lens, hkv, dim, page, dtype, order="phs", seed=0, spare=2, fill=None, extra_cols=0):
        g = gen(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        n_pages = sum(need) + spare
        shape = {"psh": (n_pages, page, hkv, dim), "phs": (n_pages, hkv, page, dim), "hps": (hkv, n_pages, page, dim)}[order]
        perm = {"psh": (0, 1, 2, 3), "phs": (0, 2, 1, 3), "hps": (1, 2, 0, 3)}[order]
        bad = math.nan if fill is None else fill
        self.kp, self.vp = (torch.full(shape, bad, dtype=dtype, device="cuda").permute(perm) for _ in range(2))
        ids = torch.randperm(n_pages, generator=g, device="cuda").to(I32)
        cols = max(need + [1]) + extra_cols
        self.table = torch.full((len(lens), cols), -1, dtype=I32, device="cuda")
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            k, v = (torch.randn(max(n, 0), hkv, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            if n > 0:
                j = torch.arange(n, device="cuda")
                where = self.table[b].long()[j // page], j % page
                self.kp[where] = k
                self.vp[where] = v
        self.cache = ops.PagedCache(self.kp, self.vp, self.table)


def check_attention(ops, heads, rows, ctx, dtype, page=64, causal=True, window=0, kv_len=None, order="psh", scale=None,
                    pad=0, packed=False, seed=0, gain=1.0, **kw):
    hq, hkv, dim = heads
    keys = [c + n if kv_len is None else kv_len[b] for b, (n, c) in enumerate(zip(rows, ctx))]
    pg = Paged(ops, keys, hkv, dim, page, dtype, order, seed)
    cu = [sum(rows[:i]) for i in range(len(rows) + 1)]
    t = cu[-1] + pad
    if packed:
        q = torch.randn(t, hq + 2 * hkv, dim, generator=gen(seed + 1), device="cuda").mul(gain).to(dtype)[:, :hq]
    else:
        q = torch.randn(t, hq, dim, generator=gen(seed + 1), device="cuda").mul(gain).to(dtype)
    lse = torch.full((t, hq), 7.0, device="cuda")
    out = torch.full((t, hq, dim), 5.0, dtype=dtype, device="cuda")
    got = ops.attention(pg.cache, q, i32(cu), i32(ctx), kv_len=None if kv_len is None else i32(kv_len), causal=causal,
                        window=window, scale=scale, out=out, lse=lse, **kw)
    assert got is out
    assert pg.cache.read_status() == 0
    assert (out[cu[-1]:] == 5.0).all() and (lse[cu[-1]:] == 7.0).all()  # padding rows are left as they were
    for b, n in enumerate(rows):
        r = slice(cu[b], cu[b + 1])
        o, l, mag, ds, seen = ops_ref.attention(q[r], pg.k[b], pg.v[b], ctx[b], keys[b], causal, window,
                                                dim ** -0.5 if scale is None else scale)
        vmax = pg.v[b].abs().max().item() if pg.v[b].numel() else 0.0
        to, tl = ops_ref.attention_tolerance(o, l, mag, ds, seen, dtype, dim, vmax)
        close(out[r], o, to, ("out", b))
        close(lse[r], l, tl, ("lse", b))
        assert (out[r][seen == 0] == 0).all() and torch.isneginf(lse[r][seen == 0]).all()
    return pg, q, out


HEADS = [(32, 8, 128), (8, 1, 128), (4, 4, 128), (16, 2, 64), (15, 5, 64), (28, 4, 128), (32, 1, 64), (6, 2, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d_%d_%d" % h)
def test_attention_of_single_tokens(ops, heads, dtype):
    check_attention(ops, heads, [1] * 9, [0, 1, 62, 63, 64, 127, 128, 500, 1300], dtype)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d_%d_%d" % h)
def test_attention_of_ragged_rows(ops, heads, dtype):
    check_attention(ops, heads, [16, 0, 1, 70, 129, 3], [2000, 50, 700, 58, 0, 5], dtype, packed=True, pad=3)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["psh", "phs", "hps"])
def test_attention_of_every_page_size_and_pool_order(ops, page, order):
    check_attention(ops, (8, 2, 128), [5, 1, 40], [77, 300, 10], BF16, page, order=order)
    check_attention(ops, (8, 2, 64), [1, 1], [255, 256], F16, page, order=order)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 17, 128, 200])
@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64)], ids=["d128", "d64"])
def test_attention_masks(ops, heads, causal, window):
    check_attention(ops, heads, [1, 30, 300, 1], [900, 200, 0, 0], BF16, causal=causal, window=window)


def test_attention_of_rows_that_see_nothing(ops):
    """No keys at all; fewer keys than positions (a window that lies beyond them, rows before the first key)."""
    check_attention(ops, (8, 2, 128), [3, 20, 5, 1], [0, 100, 50, 0], BF16, kv_len=[0, 90, 12, 0], window=16)
    check_attention(ops, (8, 2, 128), [3, 20], [0, 100], F16, kv_len=[0, 1])
    check_attention(ops, (8, 2, 64), [40, 4], [-20, -4], F16, kv_len=[20, 9])
    check_attention(ops, (8, 2, 64), [140, 4], [-130, -4], BF16, kv_len=[20, -3], causal=False)


def test_attention_of_fewer_and_more_keys_than_positions(ops):
    check_attention(ops, (8, 2, 128), [16, 16], [300, 0], BF16, kv_len=[200, 500], causal=False)
    check_attention(ops, (8, 2, 128), [16, 16], [300, 0], BF16, kv_len=[200, 500])


def test_attention_of_long_contexts_and_prompts(ops):
    check_attention(ops, (8, 2, 128), [1, 16], [32767, 20011], BF16)
    check_attention(ops, (4, 1, 64), [1], [100000], F16)
    check_attention(ops, (4, 2, 128), [1500, 700], [0, 3333], F16)
    check_attention(ops, (16, 2, 64), [2049], [0], BF16, window=300)


def test_attention_scales_and_sharp_rows(ops):
    """Scores of hundreds (a running maximum that moves a lot), a negative and a zero scale."""
    check_attention(ops, (8, 2, 128), [17, 1], [600, 900], BF16, gain=12.0)
    check_attention(ops, (8, 2, 64), [17, 200], [600, 0], F16, gain=9.0)
    check_attention(ops, (8, 2, 128), [17], [600], F16, scale=-0.05)
    check_attention(ops, (8, 2, 128), [17], [600], BF16, scale=0.0)


def test_attention_into_strided_outputs(ops):
    """Rows of out 32- and 16-byte aligned, heads apart, beside each other and before the rows."""
    pg = Paged(ops, [300, 77], 2, 128, 64, BF16)
    q = torch.randn(60, 6, 128, generator=gen(2), device="cuda").to(BF16)
    cu, ctx = i32([0, 50, 60]), i32([250, 67])
    want = ops.attention(pg.cache, q, cu, ctx)
    for width, at in ((128, 0), (144, 16), (136, 8), (256, 128)):
        buf = torch.full((60, 9, width), 3.0, dtype=BF16, device="cuda")
        out = buf[:, 1:7, at:at + 128]
        ops.attention(pg.cache, q, cu, ctx, out=out)
        assert torch.equal(out, want)
        out.fill_(3.0)
        assert (buf == 3.0).all()
    heads_first = torch.zeros(6, 60, 128, dtype=BF16, device="cuda")
    ops.attention(pg.cache, q.transpose(0, 1).contiguous().transpose(0, 1), cu, ctx, out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), want)


def test_attention_in_place_of_its_queries(ops):
    """out = q: in the middle of a sequence, with rows of the next one in the same tile, split and whole."""
    for rows, ctx in (([16], [2000]), ([1, 1, 5], [5, 900, 70]), ([300, 7, 90], [40, 0, 3000]), ([1] * 70, [500] * 70)):
        pg = Paged(ops, [a + b for a, b in zip(rows, ctx)], 2, 128, 64, BF16)
        cu = i32([sum(rows[:i]) for i in range(len(rows) + 1)])
        qkv = torch.randn(sum(rows), 10, 128, generator=gen(2), device="cuda").to(BF16)
        rest = qkv[:, 6:].clone()
        want = ops.attention(pg.cache, qkv[:, :6], cu, i32(ctx))
        assert ops.attention(pg.cache, qkv[:, :6], cu, i32(ctx), out=qkv[:, :6]).data_ptr() == qkv.data_ptr()
        assert torch.equal(qkv[:, :6], want) and torch.equal(qkv[:, 6:], rest)
        with pytest.raises(ValueError, match="overlaps"):
            ops.attention(pg.cache, qkv[:, :6], cu, i32(ctx), out=qkv[:, 1:7])


def test_attention_of_many_sequences(ops):
    rows = [(i * 7) % 5 for i in range(300)]
    ctx = [(i * 37) % 400 for i in range(300)]
    check_attention(ops, (4, 2, 64), rows, ctx, BF16, page=16)


def test_attention_runs_of_many_small_items_end_alike(ops):
    """Several short items a CTA, most of an M tile's warps without a row: 300
    calls back to back give the first one's output and no wait runs out."""
    rows, ctx = [(i * 7) % 5 for i in range(300)], [(i * 37) % 400 for i in range(300)]
    pg, q, out = check_attention(ops, (4, 2, 64), rows, ctx, BF16, page=16)
    cu = i32([sum(rows[:i]) for i in range(301)])
    for _ in range(300):
        got = ops.attention(pg.cache, q, cu, i32(ctx))
    assert torch.equal(got, out) and pg.cache.read_status() == 0
    pg, q, out = check_attention(ops, (8, 2, 128), [40] * 60, [300] * 60, F16)  # two M tiles an item
    cu = i32([40 * i for i in range(61)])
    for _ in range(100):
        got = ops.attention(pg.cache, q, cu, i32([300] * 60))
    assert torch.equal(got, out) and pg.cache.read_status() == 0


@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 2, 128), (5, 5, 64)], ids=["d64", "d128", "d64_mha"])
def test_attention_of_items_with_one_and_two_m_tiles_in_turn(ops, heads):
    """Runs that mix items of one and of two M tiles, of one key tile and of
    several: the output is right, the same in 100 calls, and no wait runs out."""
    tok = 128 * heads[1] // heads[0]
    lens = [1, 2 * tok, tok, tok + 1, 3 * tok, 0, 5, 2 * tok + 1, 4 * tok]
    rows, ctx = [lens[i % 9] for i in range(90)], [(i * 131) % 1100 for i in range(90)]
    pg, q, out = check_attention(ops, heads, rows, ctx, BF16)
    cu, cx = i32([sum(rows[:i]) for i in range(91)]), i32(ctx)
    for _ in range(100):
        got = ops.attention(pg.cache, q, cu, cx)
    assert torch.equal(got, out) and pg.cache.read_status() == 0


def test_attention_of_many_token_tiles(ops):
    """More token tiles than a CTA has threads: of one sequence, and of more sequences than threads."""
    check_attention(ops, (32, 1, 64), [3000], [5], BF16)
    rows = [33 + i % 18 for i in range(400)]
    check_attention(ops, (8, 2, 64), rows, [(i * 53) % 200 for i in range(400)], F16)


@pytest.mark.parametrize("heads,rows,ctx", [((8, 2, 128), [1, 16, 5], [1000, 700, 64]), ((4, 1, 64), [200, 3], [900, 1500]),
                                            ((8, 2, 128), [1] * 90, [800] * 90)])
def test_attention_needs_no_page_before_its_window(ops, heads, rows, ctx):
    """Pages that every row's window has left are gone from the table and hold NaN."""
    window, page = 150, 64
    hq, hkv, dim = heads
    lens = [a + b for a, b in zip(rows, ctx)]
    pg = Paged(ops, lens, hkv, dim, page, BF16)
    cu = i32([sum(rows[:i]) for i in range(len(rows) + 1)])
    q = torch.randn(sum(rows), hq, dim, generator=gen(4), device="cuda").to(BF16)
    want = ops.attention(pg.cache, q, cu, i32(ctx), window=window)
    for b, c in enumerate(ctx):
        gone = max(c - window + 1, 0) // page  # pages below the first row's first key
        ids = pg.table[b, :gone].long()
        pg.kp[ids] = math.nan
        pg.vp[ids] = math.nan
        pg.table[b, :gone] = -1
    assert torch.equal(ops.attention(pg.cache, q, cu, i32(ctx), window=window), want)
    assert pg.cache.read_status() == 0


def test_attention_of_nothing(ops):
    pg = Paged(ops, [5], 2, 64, 64, BF16)
    out = ops.attention(pg.cache, torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), i32([0, 0]), i32([5]))
    assert out.shape == (0, 4, 64)
    out = torch.ones(3, 4, 64, dtype=BF16, device="cuda")
    ops.attention(pg.cache, out.clone(), i32([0]), i32([]), out=out)  # no sequence: every row is padding
    assert (out == 1).all()


def test_attention_past_the_end_of_a_table_and_bad_pages(ops):
    """Reported, and nothing outside the pool is read: the rest of the batch is right."""
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    pg = Paged(ops, [200, 200, 200], 2, 128, 64, BF16)
    q = torch.randn(3, 4, 128, generator=gen(1), device="cuda").to(BF16)
    cu, ctx = i32([0, 1, 2, 3]), i32([199, 199, 199])
    good = ops.attention(pg.cache, q, cu, ctx)
    assert pg.cache.read_status() == 0
    for value in (-1, pg.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = pg.table.clone()
        table[1, 2] = value
        cache = ops.PagedCache(pg.kp, pg.vp, table)
        out = ops.attention(cache, q, cu, ctx)
        assert torch.equal(out[[0, 2]], good[[0, 2]])
        assert cache.read_status() == DEV_PAGE
    out = ops.attention(pg.cache, q, cu, i32([199, 300, 199]))  # keys 256.. have no table entry
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    assert pg.cache.read_status() == DEV_PAGE


def test_attention_with_pools_beyond_32_bit_offsets(ops):
    """4.4e9 bytes a pool, the sequence's pages at its far end."""
    pages, hkv, dim = 34000, 8, 128
    kp, vp = (torch.zeros(pages, 64, hkv, dim, dtype=BF16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    table = i32([[pages - 1, 3, pages - 2]])
    cache = ops.PagedCache(kp, vp, table)
    n = 150
    k, v = (torch.randn(n, hkv, dim, generator=gen(s), device="cuda").to(BF16) for s in (1, 2))
    assert ops.append(cache, k, v, i32([0, n]), i32([0])) is None
    j = torch.arange(n, device="cuda")
    assert torch.equal(kp[table[0].long()[j // 64], j % 64], k)
    q = torch.randn(2, 16, dim, generator=gen(3), device="cuda").to(BF16)
    out = ops.attention(cache, q, i32([0, 2]), i32([n - 2]))
    o, l, mag, ds, seen = ops_ref.attention(q, k, v, n - 2, n, True, 0, dim ** -0.5)
    close(out, o, ops_ref.attention_tolerance(o, l, mag, ds, seen, BF16, dim, v.abs().max().item())[0])
    assert cache.read_status() == 0


def test_attention_is_the_same_every_time_and_under_other_workspaces(ops):
    pg, q, out = check_attention(ops, (8, 2, 128), [16, 1, 300], [4000, 9000, 0], BF16)
    cu, ctx = i32([0, 16, 17, 317]), i32([4000, 9000, 0])
    need = ops.attention_workspace(pg.cache, 317, 3, 8)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        assert torch.equal(ops.attention(pg.cache, q, cu, ctx), out)
        assert torch.equal(ops.attention(pg.cache, q, cu, ctx, workspace=ws), out)
    from block_diffusion_speculative_hiddens_gb300.binding import DflashError
    with pytest.raises(DflashError) as e:
        ops.attention(pg.cache, q, cu, ctx, workspace=ws[:need - 256] if need > 256 else ws[:0])
    assert e.value.code == 6


def test_attention_refuses_what_it_does_not_take(ops):
    from block_diffusion_speculative_hiddens_gb300.binding import DflashError
    pg = Paged(ops, [70], 2, 128, 64, BF16)
    q = torch.zeros(1, 4, 136, dtype=BF16, device="cuda")
    for bad, code in ((q[:, :3, :128], 2), (q.view(-1)[1:513].view(1, 4, 128), 1),
                      (torch.zeros(1, 4, 129, dtype=BF16, device="cuda")[..., :128], 1)):
        with pytest.raises(DflashError) as e:
            ops.attention(pg.cache, bad, i32([0, 1]), i32([69]))
        assert e.value.code == code


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,dim,rd,inter,page,order", [
    (32, 8, 128, 128, False, 64, "psh"), (4, 1, 64, 32, True, 16, "phs"), (0, 2, 96, 96, False, 128, "hps"),
    (3, 2, 80, 20, True, 32, "psh"), (8, 2, 256, 128, False, 64, "psh"), (4, 2, 128, 0, False, 256, "phs")])
def test_append_rotates_and_writes_its_places_alone(ops, dtype, hq, hkv, dim, rd, inter, page, order):
    rows, ctx = [1, 0, 70, 16, 3], [130, 9, 0, 58, 509]
    lens = [a + b for a, b in zip(rows, ctx)]
    pg = Paged(ops, lens, hkv, dim, page, dtype, order, fill=3.0)
    kp, vp = pg.kp.clone(), pg.vp.clone()
    cu = [sum(rows[:i]) for i in range(6)]
    t = cu[-1] + 2  # and two padding rows
    g = gen(5)
    qkv = torch.randn(t, hq + 2 * hkv, dim, generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    plan = ops.RopePlan(rd, 1e6, interleaved=inter, scaling=LLAMA3) if rd else None
    freq, amp = ops_ref.frequencies(rd, 1e6, LLAMA3) if rd else ([], 1.0)
    q_out = torch.full((t, hq, dim), 9.0, dtype=dtype, device="cuda") if hq else None
    got = ops.append(pg.cache, k, v, i32(cu), i32(ctx), plan=plan, q=q if hq else None, q_out=q_out)
    assert got is q_out and pg.cache.read_status() == 0
    for b, n in enumerate(rows):
        r = slice(cu[b], cu[b + 1])
        pos = ctx[b] + torch.arange(n, device="cuda")
        at = pg.table[b].long()[pos // page], pos % page
        want, mag = ops_ref.rotate(k[r], pos, rd, freq, amp, inter)
        close(pg.kp[at], want, ops_ref.rotate_tolerance(want, mag, dtype), b)
        assert torch.equal(pg.vp[at], v[r])
        if hq:
            want, mag = ops_ref.rotate(q[r], pos, rd, freq, amp, inter)
            close(q_out[r], want, ops_ref.rotate_tolerance(want, mag, dtype), b)
        kp[at], vp[at] = pg.kp[at], pg.vp[at]
    assert torch.equal(kp, pg.kp) and torch.equal(vp, pg.vp)  # nowhere else
    if hq:
        assert (q_out[cu[-1]:] == 9.0).all()


def test_append_without_a_page_writes_nothing_and_says_so(ops):
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    plan = ops.RopePlan(64, 1e4)
    k = torch.randn(4, 2, 64, generator=gen(1), device="cuda").to(F16)
    cu = i32([0, 2, 4])
    for ctx, table in (([10, 255], None), ([10, -1], None), ([10, 64], -1), ([10, 64], 10 ** 6), ([10, 2 ** 31 - 2], None)):
        pg = Paged(ops, [256, 256], 2, 64, 64, F16, fill=3.0)
        if table is not None:
            pg.table[1, 1] = table
        before = pg.kp.clone()
        q = ops.append(pg.cache, k, k, cu, i32(ctx), plan=plan, q=k)
        assert pg.cache.read_status() == DEV_PAGE
        freq, amp = ops_ref.frequencies(64, 1e4)
        pos = i32([ctx[0], ctx[0] + 1]).double().tolist() + [float(ctx[1]), float(ctx[1]) + 1]
        want, mag = ops_ref.rotate(k, torch.tensor(pos, dtype=torch.float64, device="cuda"), 64, freq, amp, False)
        close(q, want, ops_ref.rotate_tolerance(want, mag, F16))  # q is rotated all the same
        changed = (pg.kp != before).any(-1).any(-1)
        ok = [ctx[0], ctx[0] + 1] + [p for p in (ctx[1], ctx[1] + 1) if 0 <= p < 256 and table is None]
        assert changed.sum().item() == sum(1 for p in ok) - (1 if 256 in ok else 0)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_a_targets_steps_equal_attention_over_the_whole_sequence(ops, dtype):
    """Prompt chunks, verify blocks with rejected tails and single tokens of
    three requests through append and attention: every step's output is the
    rows' attention over the whole accepted sequence."""
    hq, hkv, dim, page = 8, 2, 128, 64
    plan = ops.RopePlan(dim, 1e6, scaling=YARN)
    freq, amp = ops_ref.frequencies(dim, 1e6, YARN)
    pg = Paged(ops, [600] * 3, hkv, dim, page, dtype, fill=math.nan)
    pg.kp.fill_(math.nan)
    pg.vp.fill_(math.nan)
    g = gen(11)
    ks, vs = [torch.zeros(0, hkv, dim, dtype=dtype, device="cuda")] * 3, [torch.zeros(0, hkv, dim, dtype=dtype, device="cuda")] * 3
    ctx = [0, 0, 0]
    # rows a step, and how many of them stay
    for rows, keep in (([100, 130, 1], [100, 130, 1]), ([30, 0, 299], [30, 0, 299]), ([16, 16, 16], [3, 16, 1]),
                       ([16, 16, 16], [1, 9, 16]), ([1, 1, 1], [1, 1, 1]), ([16, 0, 16], [16, 0, 5])):
        cu = [sum(rows[:i]) for i in range(4)]
        qkv = torch.randn(cu[-1], hq + 2 * hkv, dim, generator=g, device="cuda").to(dtype)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        qr = ops.append(pg.cache, k, v, i32(cu), i32(ctx), plan=plan, q=q)
        out = ops.attention(pg.cache, qr, i32(cu), i32(ctx))
        for b in range(3):
            r = slice(cu[b], cu[b + 1])
            pos = ctx[b] + torch.arange(rows[b], device="cuda")
            at = pg.table[b].long()[pos // page], pos % page
            kw, mag = ops_ref.rotate(k[r], pos, dim, freq, amp, False)
            close(pg.kp[at], kw, ops_ref.rotate_tolerance(kw, mag, dtype))
            allk, allv = torch.cat((ks[b], pg.kp[at])), torch.cat((vs[b], v[r]))
            o, l, m, ds, seen = ops_ref.attention(qr[r], allk, allv, ctx[b], ctx[b] + rows[b], True, 0, dim ** -0.5)
            vmax = allv.abs().max().item() if allv.numel() else 0.0
            close(out[r], o, ops_ref.attention_tolerance(o, l, m, ds, seen, dtype, dim, vmax)[0], (rows, b))
            ks[b], vs[b] = allk[:ctx[b] + keep[b]], allv[:ctx[b] + keep[b]]
            ctx[b] += keep[b]
    assert pg.cache.read_status() == 0


def test_captured_steps_replay_on_new_values(ops):
    """append and attention in one captured graph, replayed after the rows, lengths and table have changed."""
    hq, hkv, dim = 8, 2, 64
    pg = Paged(ops, [700, 700], hkv, dim, 64, BF16, fill=0.0)
    plan = ops.RopePlan(dim, 1e4)
    q, k, v = (torch.zeros(32, h, dim, dtype=BF16, device="cuda") for h in (hq, hkv, hkv))
    cu, ctx = i32([0, 16, 32]), i32([0, 0])
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.attention(pg.cache, ops.append(pg.cache, k, v, cu, ctx, plan=plan, q=q), cu, ctx, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr = ops.append(pg.cache, k, v, cu, ctx, plan=plan, q=q)
        ops.attention(pg.cache, qr, cu, ctx, out=out)
    for step, (rows, c) in enumerate((([16, 16], [500, 3]), ([1, 31], [640, 0]), ([0, 5], [0, 600]))):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen(step), device="cuda").to(BF16))
        cu.copy_(i32([0, rows[0], sum(rows)]))
        ctx.copy_(i32(c))
        pg.table.copy_(pg.table.flip(0))
        graph.replay()
        got = out.clone()
        n = sum(rows)
        want = ops.attention(pg.cache, ops.append(pg.cache, k, v, cu, ctx, plan=plan, q=q), cu, ctx)
        assert torch.equal(got[:n], want[:n])
        assert n == 0 or want[:n].abs().max() > 0
    assert pg.cache.read_status() == 0


FIRST_CALL = """
import torch
from block_diffusion_speculative_hiddens_gb300 import ops
dev = dict(device="cuda")
kp, vp = (torch.randn(8, 64, 2, 64, **dev).to(torch.bfloat16) for _ in range(2))
rows = %d
q = torch.randn(rows, 4, 64, **dev).to(torch.bfloat16)
k = torch.randn(rows, 2, 64, **dev).to(torch.bfloat16)
cu, ctx = (torch.tensor(x, dtype=torch.int32, **dev) for x in ([0, rows], [30]))
cache = ops.PagedCache(kp, vp, torch.arange(8, dtype=torch.int32, **dev).view(1, 8))
plan = ops.RopePlan(64, 1e4)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = ops.attention(cache, ops.append(cache, k, k, cu, ctx, plan=plan, q=q), cu, ctx)
    r = ops.rope(plan, q, None, cu[1:].expand(rows).contiguous())[0]
g.replay()
torch.cuda.synchronize()
want = ops.attention(cache, ops.append(cache, k, k, cu, ctx, plan=plan, q=q), cu, ctx)
assert torch.equal(out, want) and torch.isfinite(r.float()).all() and cache.read_status() == 0
"""


@pytest.mark.parametrize("rows", [3, 200])
def test_first_call_of_a_process_may_be_captured(ops, rows):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % rows], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_captured_graphs_run_at_once(ops):
    """Each graph holds a workspace and outputs of its own."""
    jobs = []
    for seed, heads, rows, ctx in ((1, (8, 2, 128), [16] * 8, [3000] * 8), (2, (16, 2, 64), [300, 1], [0, 5000])):
        pg = Paged(ops, [a + b for a, b in zip(rows, ctx)], heads[1], heads[2], 64, BF16, seed=seed)
        q = torch.randn(sum(rows), heads[0], heads[2], generator=gen(seed), device="cuda").to(BF16)
        args = (pg.cache, q, i32([sum(rows[:i]) for i in range(len(rows) + 1)]), i32(ctx))
        want = ops.attention(*args)
        torch.cuda.synchronize()
        g, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
        with torch.cuda.graph(g):
            ops.attention(*args, out=out)
        jobs.append((g, out, want, torch.cuda.Stream(), args))  # the inputs live as long as their graph
    for _ in range(10):
        for g, out, _, s, _ in jobs:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in jobs:
            assert torch.equal(out, want)
            out.zero_()


def test_calls_on_two_streams_at_once(ops):
    """Each call has its own workspace and outputs: neither disturbs the other."""
    jobs = []
    for seed, heads, rows, ctx in ((1, (8, 2, 128), [16, 16], [9000, 4000]), (2, (16, 2, 64), [300, 1], [0, 5000])):
        pg = Paged(ops, [a + b for a, b in zip(rows, ctx)], heads[1], heads[2], 64, BF16, seed=seed)
        q = torch.randn(sum(rows), heads[0], heads[2], generator=gen(seed), device="cuda").to(BF16)
        args = (pg.cache, q, i32([0, rows[0], sum(rows)]), i32(ctx))
        jobs.append((args, ops.attention(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (args, _, s) in enumerate(jobs):
            got[i].append(ops.attention(*args, stream=s))
    torch.cuda.synchronize()
    for i, (_, want, _) in enumerate(jobs):
        assert all(torch.equal(x, want) for x in got[i])


# ------------------------------------------------------------------ the status word

@pytest.mark.parametrize("heads,rows,ctx", [((4, 2, 128), [1, 3], [199, 8000]), ((32, 8, 64), [1] * 40, [199] * 39 + [8000]),
                                            ((4, 1, 128), [300, 200], [0, 8000])], ids=["clusters", "runs", "runs of two M tiles"])
def test_attention_whose_window_lies_past_the_table_says_so(ops, heads, rows, ctx):
    """The last sequence sees no position the table can hold: no tile of work, and reported all the same."""
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    hq, hkv, dim = heads
    lens = [a + b for a, b in zip(rows[:-1], ctx[:-1])] + [200]
    pg = Paged(ops, lens, hkv, dim, 64, BF16, extra_cols=8)
    q = torch.randn(sum(rows), hq, dim, generator=gen(1), device="cuda").to(BF16)
    cu = i32([sum(rows[:i]) for i in range(len(rows) + 1)])
    out, lse = torch.ones_like(q), torch.ones(sum(rows), hq, device="cuda")
    ops.attention(pg.cache, q, cu, i32(ctx), window=1024, out=out, lse=lse)
    assert pg.cache.read_status() == DEV_PAGE
    assert (out[-rows[-1]:] == 0).all() and torch.isneginf(lse[-rows[-1]:]).all()
    for b, n in enumerate(rows[:-1]):  # the other sequences are right
        r = slice(sum(rows[:b]), sum(rows[:b + 1]))
        o, l, mag, ds, seen = ops_ref.attention(q[r], pg.k[b], pg.v[b], ctx[b], lens[b], True, 1024, dim ** -0.5)
        to, tl = ops_ref.attention_tolerance(o, l, mag, ds, seen, BF16, dim, pg.v[b].abs().max().item())
        close(out[r], o, to, ("out", b))
        close(lse[r], l, tl, ("lse", b))


def _reports(ops, cache, stream):
    """A token whose only page is outside the pool, on `stream`."""
    q = torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    cu, ctx = i32([0, 1]), i32([5])
    torch.cuda.synchronize()
    return lambda: ops.attention(cache, q, cu, ctx, stream=stream)


def test_status_of_calls_on_another_stream(ops):
    """read_status waits for every stream, also for what is still queued there."""
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    pg = Paged(ops, [6], 2, 64, 64, BF16)
    pg.table.fill_(-1)
    side = torch.cuda.Stream()
    call = _reports(ops, pg.cache, side)
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # about 20 ms
        call()
        assert pg.cache.read_status() == DEV_PAGE
        assert pg.cache.read_status() == 0


def test_status_of_a_first_call_on_another_stream(ops):
    """The status word is clear before the cache can be used anywhere."""
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    pg = Paged(ops, [6], 2, 64, 64, BF16)
    pg.table.fill_(-1)
    side = torch.cuda.Stream()
    call = _reports(ops, pg.cache, side)
    call()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    cache = ops.PagedCache(pg.kp, pg.vp, pg.table)
    q, cu, ctx = torch.empty(1, 4, 64, dtype=BF16, device="cuda"), torch.empty(2, dtype=I32, device="cuda"), \
        torch.empty(1, dtype=I32, device="cuda")
    with torch.cuda.stream(side):
        q.zero_()
        cu[0], cu[1], ctx[0] = 0, 1, 5
    ops.attention(cache, q, cu, ctx, stream=side)
    assert cache.read_status() == DEV_PAGE


def test_status_of_a_cache_built_while_a_graph_is_captured(ops):
    """Its word is cleared by each replay."""
    from block_diffusion_speculative_hiddens_gb300.binding import DEV_PAGE
    pg = Paged(ops, [6], 2, 64, 64, BF16)
    q = torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    cu, ctx = i32([0, 1]), i32([5])
    want = ops.attention(pg.cache, q, cu, ctx)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache = ops.PagedCache(pg.kp, pg.vp, pg.table)
        out = ops.attention(cache, q, cu, ctx)
    g.replay()
    assert cache.read_status() == 0 and torch.equal(out, want)
    pg.table.fill_(-1)
    g.replay()
    assert cache.read_status() == DEV_PAGE


@pytest.mark.parametrize("hq,hkv,dim", [(0, 1, 6), (1, 1, 10), (5, 1, 22), (3, 2, 80), (7, 1, 112), (2, 2, 2)])
def test_append_finds_its_sequence_in_blocks_of_uneven_warps(ops, hq, hkv, dim):
    """Heads whose blocks end in a warp that is not full, rows that share a block, more sequences than lanes."""
    rows = [i % 3 for i in range(150)]
    ctx = [(i * 7) % 50 for i in range(150)]
    pg = Paged(ops, [a + b for a, b in zip(rows, ctx)], hkv, dim, 16, BF16, fill=3.0)
    t = sum(rows)
    k, v = (torch.randn(t, hkv, dim, generator=gen(s), device="cuda").to(BF16) for s in (1, 2))
    q = torch.randn(t, hq, dim, generator=gen(3), device="cuda").to(BF16) if hq else None
    kp, vp = pg.kp.clone(), pg.vp.clone()
    cu = [sum(rows[:i]) for i in range(151)]
    got = ops.append(pg.cache, k, v, i32(cu), i32(ctx), q=q)
    for b, n in enumerate(rows):
        pos = ctx[b] + torch.arange(n, device="cuda")
        at = pg.table[b].long()[pos // 16], pos % 16
        kp[at], vp[at] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
    assert torch.equal(kp, pg.kp) and torch.equal(vp, pg.vp) and pg.cache.read_status() == 0
    assert got is None if q is None else torch.equal(got, q)  # without a plan: copied


def test_outputs_over_other_tensors_of_the_call_are_refused(ops):
    """In the pools, over a workspace, an lse over itself or the output: nothing is queued, nothing changes."""
    from block_diffusion_speculative_hiddens_gb300.binding import DflashError
    pg = Paged(ops, [3000, 3000], 2, 64, 64, BF16, order="psh")
    q = torch.randn(300, 4, 64, generator=gen(1), device="cuda").to(BF16)
    cu, ctx = i32([0, 100, 300]), i32([2900, 2800])
    kv = pg.k[0][:1].expand(300, 2, 64).contiguous()
    inside = pg.kp[:10].view(-1)[:300 * 256].view(300, 4, 64)
    ws = torch.zeros(ops.attention_workspace(pg.cache, 300, 2, 4), dtype=torch.uint8, device="cuda")
    need = 300 * 4 * 64 * 2
    before = pg.kp.clone(), pg.vp.clone(), q.clone()
    for call in (lambda: ops.attention(pg.cache, q, cu, ctx, out=inside),
                 lambda: ops.append(pg.cache, kv, kv, cu, ctx, q=q, q_out=inside),
                 lambda: ops.attention(pg.cache, q, cu, ctx, out=ws[:need].view(BF16).view(300, 4, 64), workspace=ws),
                 lambda: ops.attention(pg.cache, q, cu, ctx, lse=ws[4096:4096 + 4800].view(torch.float32).view(300, 4), workspace=ws),
                 lambda: ops.attention(pg.cache, q, cu, ctx, lse=torch.zeros(300, 1, device="cuda").expand(300, 4)),
                 lambda: ops.attention(pg.cache, q, cu, ctx, lse=q.view(-1)[:2400].view(torch.float32).view(300, 4)),
                 lambda: ops.append(ops.PagedCache(pg.kp, pg.kp, pg.table), kv, kv, cu, ctx)):
        with pytest.raises(DflashError) as e:
            call()
        assert e.value.code == 1
    torch.cuda.synchronize()
    assert all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip((pg.kp, pg.vp, q), before))
    # beside one another they are taken: an lse and an output behind the workspace's bytes, K and V of one pool
    big = torch.zeros(ws.numel() + need + 4800, dtype=torch.uint8, device="cuda")
    out, lse = big[ws.numel():-4800].view(BF16).view(300, 4, 64), big[-4800:].view(torch.float32).view(300, 4)
    ops.attention(pg.cache, q, cu, ctx, out=out, lse=lse, workspace=big[:ws.numel()])
    assert torch.equal(out, ops.attention(pg.cache, q, cu, ctx))
    ops.attention(pg.cache, q, cu, ctx, out=out, lse=lse, workspace=big)  # of a larger one only the needed bytes are used
    assert torch.equal(out, ops.attention(pg.cache, q, cu, ctx))
    same = ops.attention(ops.PagedCache(pg.kp, pg.kp, pg.table), q, cu, ctx)
    assert torch.equal(same, ops.attention(ops.PagedCache(pg.kp, pg.kp.clone(), pg.table), q, cu, ctx))


# ------------------------------------------------------------------ calls at the documentation's edges

@pytest.mark.parametrize("cols", [0, 20, 500])
@pytest.mark.parametrize("heads,rows,ctx", [((32, 8, 128), [16], [2048]), ((16, 2, 64), [16, 1, 3], [700, 2000, 0]),
                                            ((8, 2, 128), [200, 16], [0, 900])])
def test_attention_over_tables_wider_than_their_sequences(ops, heads, rows, ctx, cols):
    """The table's width chooses the launch, never the answer; its unused entries are not read."""
    hq, hkv, dim = heads
    lens = [a + b for a, b in zip(rows, ctx)]
    pg = Paged(ops, lens, hkv, dim, 64, BF16, extra_cols=cols)
    q = torch.randn(sum(rows), hq, dim, generator=gen(1), device="cuda").to(BF16)
    cu = [sum(rows[:i]) for i in range(len(rows) + 1)]
    lse = torch.zeros(hq, sum(rows), device="cuda").t()  # heads first
    out = ops.attention(pg.cache, q, i32(cu), i32(ctx), lse=lse)
    for b in range(len(rows)):
        r = slice(cu[b], cu[b + 1])
        o, l, mag, ds, seen = ops_ref.attention(q[r], pg.k[b], pg.v[b], ctx[b], lens[b], True, 0, dim ** -0.5)
        to, tl = ops_ref.attention_tolerance(o, l, mag, ds, seen, BF16, dim, pg.v[b].abs().max().item())
        close(out[r], o, to, ("out", b))
        close(lse[r], l, tl, ("lse", b))
    assert pg.cache.read_status() == 0


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128)], ids=["d64", "d128"])
def test_largest_batch(ops, heads):
    """8,192 sequences, none to three rows each: append and attention."""
    hq, hkv, dim = heads
    n = 8192
    rows, ctx = [(i * 5) % 4 for i in range(n)], [(i * 3) % 14 for i in range(n)]
    kp, vp = (torch.full((n + 3, 16, hkv, dim), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.randperm(n + 3, generator=gen(1), device="cuda")[:n].to(I32)[:, None].contiguous()  # a page each
    cache = ops.PagedCache(kp, vp, table)
    cu = torch.tensor([0] + rows, device="cuda").cumsum(0).to(I32)
    t = sum(rows)
    # every sequence's positions hold the same keys: rows at one position differ in their queries alone
    k, v = (torch.randn(16, hkv, dim, generator=gen(s), device="cuda").to(BF16) for s in (3, 4))
    kp[:], vp[:] = k, v
    q = torch.randn(t, hq, dim, generator=gen(5), device="cuda").to(BF16)
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(rows, device="cuda"))
    pos = i32(ctx)[seq].long() + torch.arange(t, device="cuda") - cu.long()[seq]
    got = ops.append(cache, k[pos], v[pos], cu, i32(ctx), q=q)
    assert torch.equal(got, q) and cache.read_status() == 0
    out = ops.attention(cache, q, cu, i32(ctx))
    assert cache.read_status() == 0
    for p in range(16):  # rows at position p see the keys 0..p, whoever they belong to
        at = pos == p
        if at.any():
            o, l, mag, ds, seen = ops_ref.attention(q[at], k[:p + 1], v[:p + 1], p, p + 1, False, 0, dim ** -0.5)
            close(out[at], o, ops_ref.attention_tolerance(o, l, mag, ds, seen, BF16, dim, v.abs().max().item())[0], p)


def test_batches_of_empty_sequences(ops):
    """Rows but no sequence that has one: nothing is written, in every form of the launch."""
    for rows, batch, dim, cols in ((3, 2, 64, 0), (200, 2, 128, 0), (500, 300, 128, 0), (40, 300, 64, 600)):
        pg = Paged(ops, [70] * batch, 2, dim, 64, BF16, extra_cols=cols)
        k, v = pg.kp.clone(), pg.vp.clone()
        x = torch.ones(rows, 4, dim, dtype=BF16, device="cuda")
        out, q_out = x * 2, x * 3
        cu, ctx = i32([0] * (batch + 1)), i32([5] * batch)
        ops.append(pg.cache, x[:, :2], x[:, 2:], cu, ctx, q=x, q_out=q_out)
        ops.attention(pg.cache, x, cu, ctx, out=out)
        assert (out == 2).all() and (q_out == 3).all() and pg.cache.read_status() == 0
        assert torch.equal(pg.kp.nan_to_num(9), k.nan_to_num(9)) and torch.equal(pg.vp.nan_to_num(9), v.nan_to_num(9))


def test_inputs_expanded_over_rows_and_heads(ops):
    """Inputs may share memory with themselves: one row for all, one head for all."""
    plan = ops.RopePlan(128, 1e4)
    for rows, ctx in (([16], [300]), ([1, 250], [900, 20])):
        pg = Paged(ops, [a + b for a, b in zip(rows, ctx)], 2, 128, 64, BF16)
        cu, cx, t = i32([0] + [sum(rows[:i + 1]) for i in range(len(rows))]), i32(ctx), sum(rows)
        pos = torch.arange(t, device="cuda").to(I32)
        base = torch.randn(t, 8, 128, generator=gen(1), device="cuda").to(BF16)
        for q in (base[:1].expand(t, 8, 128), base[:, :1].expand(t, 8, 128), base[:1, :1].expand(t, 8, 128)):
            assert torch.equal(ops.attention(pg.cache, q, cu, cx), ops.attention(pg.cache, q.contiguous(), cu, cx))
            assert torch.equal(ops.rope(plan, q, None, pos)[0], ops.rope(plan, q.contiguous(), None, pos)[0])
            k = q[:, :2]
            for x in (k, k.contiguous()):
                ops.append(pg.cache, x, x, cu, cx, plan=plan)
                now = (pg.kp.nan_to_num(9), pg.vp.nan_to_num(9))
                first = now if x is k else first
            assert all(torch.equal(a, b) for a, b in zip(first, now))
    assert pg.cache.read_status() == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=["nan", "inf"])
@pytest.mark.parametrize("heads,n,ctx,window", [((8, 2, 128), 16, 300, 0), ((8, 2, 128), 16, 20000, 0), ((8, 2, 64), 200, 100, 0),
                                                ((16, 2, 128), 300, 0, 0), ((8, 2, 64), 200, 900, 70)])
def test_keys_that_are_not_finite_reach_the_rows_that_see_them_alone(ops, heads, n, ctx, window, bad):
    hq, hkv, dim = heads
    pg = Paged(ops, [ctx + n], hkv, dim, 64, BF16, extra_cols=500)
    q = torch.randn(n, hq, dim, generator=gen(1), device="cuda").to(BF16)
    cu, cx = i32([0, n]), i32([ctx])
    want = ops.attention(pg.cache, q, cu, cx, window=window)
    j = ctx + n // 2
    pg.kp[pg.table[0, j // 64].long(), j % 64] = bad
    got = ops.attention(pg.cache, q, cu, cx, window=window)
    sees = torch.arange(n, device="cuda") >= n // 2
    if window:
        sees &= torch.arange(n, device="cuda") < n // 2 + window
    assert torch.equal(got[~sees], want[~sees])
    if bad != bad:
        assert torch.isnan(got[sees]).all()
    assert pg.cache.read_status() == 0


@pytest.mark.parametrize("device", [17, 1000])
def test_a_device_that_is_not_there_leaves_no_error_behind(ops, lib, device):
    """The call says so, and what runs next does not take the error for its own."""
    import ctypes
    pg = Paged(ops, [6], 2, 64, 64, BF16)
    pg.table.fill_(-1)
    q, cu, ctx = torch.zeros(1, 4, 64, dtype=BF16, device="cuda"), i32([0, 1]), i32([5])
    k, q_out, plan = torch.zeros(1, 2, 64, dtype=BF16, device="cuda"), torch.zeros_like(q), ops.RopePlan(64, 1e4)
    rows = lambda t: (t.data_ptr(), t.stride(0), t.stride(1))
    none = (0, 0, 0)
    there = list(ops._CACHE.unpack(pg.cache._c))
    gone = ops._CACHE.pack(*there[:-1], device)
    word = ctypes.c_uint32(9)
    calls = [lambda: lib.dflash_rope(plan._ref, ops._ROPE.pack(*rows(q), *none, *rows(q_out), *none, ctx.data_ptr(), 1, 4, 0, 64, 1,
                                                               0, device), None),
             lambda: lib.dflash_paged_append(gone, None, ops._APPEND.pack(*rows(k), *rows(k), *none, *none, cu.data_ptr(),
                                                                          ctx.data_ptr(), 1, 1, 0, 0), None),
             lambda: lib.dflash_paged_attention(gone, ops._ATTENTION.pack(*rows(q), *rows(q_out), 0, 0, 0, cu.data_ptr(),
                                                                          ctx.data_ptr(), 0, 0, 0, 1, 1, 4, 1, 0, 0.1), None),
             lambda: lib.dflash_paged_read_status(gone, ctypes.byref(word))]
    for call in calls:
        assert call() == 4
        assert (torch.ones(5, device="cuda") * 2).sum().item() == 10
        call()
        ops.attention(pg.cache, q, cu, ctx)  # its page is not in the pool
        assert pg.cache.read_status() == 4
    assert word.value == 9
