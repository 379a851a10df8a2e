"""The page and beam-search operators on the CPU: the packed argument structs
against the C ones, and the refusals -- a wrong call never reaches the device."""
import ctypes
import math
import os
import random

import pytest
import torch

from block_diffusion_speculative_hiddens_gb300 import _build, binding, ops
from tests import beam_ref
from tests.test_ops_args import NOWHERE, FakeT, Stream, _bytes

I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB):
        _build.build()
    return binding.load()


def test_packed_structs_match_the_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    fields = ["sizeof(dflash_page_pool)", "sizeof(dflash_beam_args)", "offsetof(dflash_page_pool, lens)",
              "offsetof(dflash_page_pool, n_pages)", "offsetof(dflash_beam_args, scores_out)",
              "offsetof(dflash_beam_args, workspace_bytes)", "offsetof(dflash_beam_args, done_token)"]
    src.write_text('#include "%s"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) { printf("%s", %s); return 0; }\n' % (
        binding.HEADER, " ".join(["%zu"] * len(fields)), ", ".join(fields)))
    subprocess.run([cc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ops._POOL.size, ops._BEAM.size, 24, 40, 32, 72, 96]


def _pool(refs=1 << 20, table=1 << 21, stride=4, lens=1 << 22, status=1 << 23, pages=8, page=16, width=4, batch=3,
          device=NOWHERE):
    return ops._POOL.pack(refs, table, stride, lens, status, pages, page, width, batch, device, 0)


GOOD = [{}, dict(stride=9), dict(page=256), dict(pages=1 << 24, refs=1 << 28), dict(batch=8192, lens=1 << 24, status=1 << 26)]
BAD = [(dict(refs=(1 << 20) + 2), 1), (dict(table=(1 << 21) + 1), 1), (dict(lens=(1 << 22) + 3), 1),
       (dict(status=(1 << 23) + 2), 1), (dict(refs=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(status=0), 1), (dict(pages=0), 1), (dict(width=0), 1),
       (dict(batch=0), 1), (dict(stride=3), 1), (dict(device=-1), 1), (dict(page=8), 2), (dict(page=48), 2),
       (dict(page=512), 2), (dict(batch=8193), 3), (dict(pages=(1 << 24) + 1), 3)]


def test_pool_calls_refuse_before_any_cuda_call(lib):
    """4: what passed every check, on a device that no machine has."""
    other = 1 << 32
    calls = {"fork": lambda p, arg=other: lib.dflash_pages_fork(p, arg, None),
             "resize": lambda p, arg=other, moves=2 * other, room=8192: lib.dflash_pages_resize(p, arg, moves, room, None),
             "compact": lambda p, moves=other, room=1 << 24, remap=2 * other: lib.dflash_pages_compact(p, moves, room, remap, None),
             "status": lambda p: lib.dflash_pool_read_status(p, ctypes.byref(ctypes.c_uint32()))}
    for name, call in calls.items():
        for kw in GOOD:
            assert call(_pool(**kw)) == 4, (name, kw)
        for kw, code in BAD:
            assert call(_pool(**kw)) == code, (name, kw)
        assert call(None) == 1
    assert lib.dflash_pool_read_status(_pool(), None) == 1
    p = _pool()
    assert calls["fork"](p, 0) == 1 and calls["resize"](p, 0) == 1 and calls["resize"](p, moves=0) == 1
    assert calls["compact"](p, moves=0) == 1 and calls["compact"](p, remap=0) == 1
    for odd in (other + 1, other + 2):
        assert calls["fork"](p, odd) == 1 and calls["resize"](p, odd) == 1 and calls["resize"](p, moves=odd) == 1
        assert calls["compact"](p, moves=odd) == 1 and calls["compact"](p, remap=odd) == 1
    assert calls["resize"](p, room=3) == 4 and calls["resize"](p, room=2) == 3 and calls["resize"](p, room=-1) == 1
    assert calls["compact"](p, room=4) == 4 and calls["compact"](p, room=3) == 3 and calls["compact"](p, room=-1) == 1
    for call in (calls["resize"], calls["compact"]):  # more room than indexes reach
        assert call(p, moves=1 << 40, room=1 << 30) == 4 and call(p, moves=1 << 40, room=(1 << 30) + 1) == 3
    assert calls["compact"](_pool(pages=9), room=4) == 4 and calls["compact"](_pool(pages=1), room=0) == 4
    for at in ((1 << 20) + 28, (1 << 21) + 4, (1 << 22) + 8, 1 << 23, (1 << 23) + 4, (1 << 20) - 8):  # the pool's own
        assert calls["fork"](p, at) == 1 and calls["resize"](p, at) == 1 and calls["resize"](p, moves=at) == 1
        assert calls["compact"](p, moves=at) == 1 and calls["compact"](p, remap=at) == 1
    assert calls["resize"](p, 2 * other + 4) == 1 and calls["compact"](p, remap=other + 8) == 1
    for kw in (dict(refs=(1 << 21) + 16), dict(lens=(1 << 21) + 12), dict(status=(1 << 20) + 28), dict(lens=(1 << 23) + 4)):
        for name in ("fork", "resize", "compact"):
            assert calls[name](_pool(**kw)) == 1, (name, kw)


def _cache(k=1 << 24, v=1 << 25, ks=(2048, 128, 64), vs=(2048, 128, 64), pages=5, page=16, heads=2, dim=64, dtype=1,
           device=NOWHERE, status=1 << 27):
    return ops._CACHE.pack(k, v, *ks, *vs, 1 << 26, 4, status, 4, pages, page, heads, dim, dtype, device)


def test_page_copies_refuse_before_any_cuda_call(lib):
    def copy(*caches, moves=1 << 30, room=7, n=None):
        return lib.dflash_pages_copy(b"".join(caches) or None, len(caches) if n is None else n, moves, room, None)
    c = _cache()
    far = _cache(k=1 << 28, v=1 << 29, ks=(2048, 64, 1024), status=1 << 31)  # other strides, another status word
    assert copy(c) == 4 and copy(c, far) == 4 and copy(*[c] * 200) == 4
    assert copy(n=0) == 0 and copy(c, room=0) == 0
    assert copy(c, n=-1) == 1 and copy(c, room=-1) == 1 and copy(c, moves=0) == 1 and copy(n=1) == 1
    assert copy(c, moves=(1 << 30) + 2) == 1 and copy(_cache(k=(1 << 24) + 1)) == 1 and copy(_cache(status=(1 << 27) + 2)) == 1
    for kw in (dict(pages=6), dict(page=32), dict(heads=1), dict(dim=32), dict(device=NOWHERE + 1)):
        assert copy(c, _cache(**kw)) == 1, kw
    for kw in (dict(k=0), dict(dtype=7), dict(status=0), dict(pages=0), dict(dim=0)):
        assert copy(_cache(**kw)) == 1, kw
    assert copy(_cache(page=24)) == 2
    assert copy(_cache(v=1 << 24)) == 1 and copy(_cache(ks=(0, 128, 64))) == 1  # K over V, pages over one another
    assert copy(_cache(ks=(2048, 64, 64))) == 1
    assert copy(c, moves=(1 << 24) + 128) == 1 and copy(c, moves=(1 << 25) + 10000) == 1
    assert copy(c, _cache(k=(1 << 27) - 64, v=1 << 29)) == 1  # over the status word


def _select(lib, **kw):
    a = dict(logits=1 << 32, stride=1000, scores=1 << 20, done=0, scores_out=1 << 21, parents=1 << 22, tokens=1 << 23,
             status=0, ws=1 << 40, wsb=1 << 38, batch=2, beams=4, vocab=1000, n=4, done_token=0, dtype=1, device=NOWHERE)
    a.update(kw)
    return lib.dflash_beam_select(ops._BEAM.pack(*a.values(), 0), None)


def test_selection_refuses_before_any_cuda_call(lib):
    assert lib.dflash_beam_select(None, None) == 1
    for kw in ({}, dict(dtype=2), dict(dtype=0), dict(n=128), dict(beams=64), dict(n=1, beams=1, vocab=1), dict(stride=0),
               dict(stride=-1000), dict(done=1 << 24, done_token=999), dict(done_token=-5), dict(status=1 << 24),
               dict(scores_out=1 << 20), dict(vocab=1 << 24, beams=64)):
        assert _select(lib, **kw) == 4, kw
    for kw in (dict(logits=0), dict(scores=0), dict(scores_out=0), dict(parents=0), dict(tokens=0), dict(batch=-1),
               dict(beams=-1), dict(vocab=-1), dict(n=-1), dict(dtype=3), dict(dtype=-1), dict(device=-1),
               dict(done=1 << 24, done_token=1000), dict(done=1 << 24, done_token=-1), dict(logits=(1 << 32) + 1),
               dict(logits=(1 << 32) + 2, dtype=2), dict(scores=(1 << 20) + 2), dict(scores_out=(1 << 21) + 1),
               dict(parents=(1 << 22) + 2), dict(tokens=(1 << 23) + 3), dict(status=(1 << 24) + 2)):
        assert _select(lib, **kw) == 1, kw
    for kw in (dict(beams=0), dict(beams=65), dict(n=0), dict(n=129), dict(vocab=0), dict(vocab=(1 << 24) + 1)):
        assert _select(lib, **kw) == 2, kw
    assert _select(lib, batch=1 << 20, beams=64, vocab=5) == 3
    assert _select(lib, batch=0) == 0
    need = lib.dflash_beam_select_workspace(2, 4, 1000, 4, 1)
    assert need > 0
    assert _select(lib, wsb=need) == 4 and _select(lib, wsb=need - 1) == 6 and _select(lib, ws=0) == 6
    assert _select(lib, ws=(1 << 40) + 128) == 6 and _select(lib, wsb=-1) == 6
    # outputs over inputs, over one another, over the workspace and the status word
    for kw in (dict(scores_out=(1 << 20) + 4), dict(scores_out=1 << 20, n=3), dict(parents=1 << 20), dict(tokens=(1 << 22) + 8),
               dict(scores_out=(1 << 32) + 16000 - 4), dict(parents=1 << 40), dict(status=1 << 21), dict(tokens=1 << 24, status=1 << 24),
               dict(parents=1 << 24, done=(1 << 24) + 31), dict(ws=1 << 32, wsb=1 << 20), dict(scores=(1 << 40) + 64)):
        assert _select(lib, **kw) == 1, kw
    w = lib.dflash_beam_select_workspace
    assert w(0, 4, 1000, 4, 1) == 0 and w(2, 0, 1000, 4, 1) == 0 and w(2, 4, 1000, 4, 9) == 0 and w(-1, 4, 1000, 4, 1) == 0


def test_selection_output_rows_between_input_rows_are_refused_or_apart(lib):
    """Logits with padding between their rows: an output inside the padding is apart, one over a row is not."""
    gap = dict(stride=2000, batch=2, beams=4, vocab=1000, n=4)
    assert _select(lib, **gap, scores_out=(1 << 32) + 2000) == 4
    assert _select(lib, **gap, scores_out=(1 << 32) + 1996) == 1
    assert _select(lib, **gap, parents=(1 << 32) + 4000 - 28) == 1


# ------------------------------------------------------------------ the Python side

@pytest.fixture
def calls(monkeypatch):
    got = []

    class Lib:
        def __getattr__(self, name):
            def fn(*a):
                got.append(name)
                return 0
            return fn
    monkeypatch.setattr(ops, "load", lambda: Lib())
    monkeypatch.setattr(ops, "_clear_word", lambda device, n=1: FakeT([n], I32, ptr=1 << 35))
    return got


def _python_pool(**kw):
    a = dict(page_table=FakeT([3, 4], I32, ptr=1 << 36), n_pages=8, page_size=16)
    a.update(kw)
    return ops.PagePool(a.pop("page_table"), a.pop("n_pages"), a.pop("page_size"), **a)


def test_pools_are_checked(calls):
    p = _python_pool()
    assert ops._POOL.unpack(p._c) == (1 << 35, 1 << 36, 4, 1 << 35, 1 << 35, 8, 16, 4, 3, 0, 0)
    _python_pool(refs=FakeT([8], I32), lens=FakeT([3], I32), page_table=FakeT([3, 4], I32, stride=(9, 1)))
    for kw in (dict(refs=FakeT([7], I32)), dict(refs=FakeT([8], torch.int64)), dict(lens=FakeT([4], I32)),
               dict(lens=FakeT([3], I32, device="cuda:1")), dict(refs=FakeT([8], I32, stride=(2,))),
               dict(page_table=FakeT([3, 4], torch.int64)), dict(page_table=FakeT([3, 4], I32, device="cpu")),
               dict(page_table=FakeT([3, 4], I32, stride=(3, 1))), dict(page_table=FakeT([3, 4], I32, stride=(1, 3))),
               dict(page_table=FakeT([12], I32)), dict(n_pages=0), dict(n_pages=2 ** 31), dict(n_pages=8.5), dict(page_size=24)):
        with pytest.raises(ValueError):
            _python_pool(**kw)


def test_pool_calls_check_their_tensors(calls):
    p, s = _python_pool(), Stream()
    good, moves = FakeT([3], I32), FakeT([4, 3], I32)
    ops.fork(p, good, stream=s)
    assert ops.resize(p, good, moves=moves, stream=s) is moves
    ops.resize(p, good, moves=FakeT([9, 3], I32), stream=s)
    ops.compact(p, moves=FakeT([5, 3], I32), remap=FakeT([8], I32), stream=s)
    assert calls == ["dflash_pages_fork", "dflash_pages_resize", "dflash_pages_resize", "dflash_pages_compact"]
    for bad in (FakeT([4], I32), FakeT([3], torch.int64), FakeT([3], I32, device="cuda:1"), FakeT([3, 1], I32),
                FakeT([3], I32, stride=(2,)), FakeT([3], I32, device="cpu")):
        for call in (lambda: ops.fork(p, bad, stream=s), lambda: ops.resize(p, bad, moves=moves, stream=s)):
            with pytest.raises(ValueError):
                call()
    for bad in (FakeT([3, 3], I32), FakeT([4, 4], I32), FakeT([12], I32), FakeT([4, 3], torch.int64),
                FakeT([4, 3], I32, stride=(6, 1)), FakeT([4, 3], I32, device="cuda:1")):
        with pytest.raises(ValueError, match="moves"):
            ops.resize(p, good, moves=bad, stream=s)
        with pytest.raises(ValueError, match="moves"):
            ops.compact(p, moves=bad, remap=FakeT([8], I32), stream=s)
    with pytest.raises(ValueError, match="remap"):
        ops.compact(p, moves=FakeT([5, 3], I32), remap=FakeT([7], I32), stream=s)
    s.device = torch.device("cuda:1")
    for call in (lambda: ops.fork(p, good, stream=s), lambda: ops.resize(p, good, moves=moves, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call()
    s.device = torch.device("cuda:0")
    assert len(calls) == 4


def test_page_copies_check_their_tensors(calls):
    pools = FakeT([8, 64, 2, 128], ptr=1 << 30), FakeT([8, 64, 2, 128], ptr=1 << 31)
    c, moves = ops.PagedCache(*pools, FakeT([3, 4], I32)), FakeT([4, 3], I32)
    ops.copy_pages(c, moves, stream=Stream())
    ops.copy_pages([c, c], moves, stream=Stream())
    with pytest.raises(ValueError, match="caches"):
        ops.copy_pages([], moves)
    for bad in (FakeT([4, 4], I32), FakeT([0, 3], I32), FakeT([12], I32), FakeT([4, 3], torch.int64),
                FakeT([4, 3], I32, stride=(6, 1)), FakeT([4, 3], I32, device="cuda:1")):
        with pytest.raises(ValueError, match="moves"):
            ops.copy_pages(c, bad, stream=Stream())
    pools[1].requires_grad = True
    graded = ops.PagedCache(*pools, FakeT([3, 4], I32))
    with pytest.raises(ValueError, match="v_pool: requires a gradient"):
        ops.copy_pages([c, graded], moves, stream=Stream())
    with torch.no_grad():
        ops.copy_pages([c, graded], moves, stream=Stream())
    assert calls == ["dflash_pages_copy"] * 3


def _beam(**kw):
    a = dict(logits=FakeT([6, 50]), scores=FakeT([2, 3], F32), n=4, stream=Stream(),
             out=(FakeT([2, 4], F32), FakeT([2, 4], I32), FakeT([2, 4], I32)), workspace=FakeT([256], torch.uint8))
    a.update(kw)
    return ops.beam_select(a.pop("logits"), a.pop("scores"), a.pop("n"), **a)


def test_selection_checks_its_tensors(calls):
    _beam()
    _beam(done=FakeT([2, 3], torch.bool), done_token=3, status=FakeT([2], I32))
    _beam(n=None, out=(FakeT([2, 3], F32), FakeT([2, 3], I32), FakeT([2, 3], I32)), logits=FakeT([6, 50], stride=(64, 1)))
    assert calls == ["dflash_beam_select"] * 3
    for kw in (dict(logits=FakeT([6, 50], torch.float64)), dict(logits=FakeT([6, 50], device="cpu")),
               dict(logits=FakeT([2, 3, 50])), dict(logits=FakeT([6, 50], stride=(1, 6))), dict(logits=FakeT([5, 50])),
               dict(logits=FakeT([6, 50], device="cuda:1")), dict(scores=FakeT([2, 3])), dict(scores=FakeT([6], F32)),
               dict(scores=FakeT([2, 3], F32, stride=(6, 1))), dict(done=FakeT([2, 3], I32)), dict(done=FakeT([6], torch.bool)),
               dict(done=FakeT([2, 3], torch.bool, device="cuda:1")), dict(status=FakeT([1], F32)), dict(status=FakeT([0], I32)),
               dict(status=FakeT([1], I32, device="cuda:1")), dict(workspace=FakeT([256], F32)),
               dict(n=3), dict(n=2 ** 31), dict(n=0, out=None), dict(done_token=0.5), dict(done_token=2 ** 40),
               dict(out=(FakeT([2, 4], F32), FakeT([2, 4], I32), FakeT([2, 4], torch.int64))),
               dict(out=(FakeT([2, 4], F32), FakeT([2, 4], I32, stride=(8, 1)), FakeT([2, 4], I32)))):
        with pytest.raises(ValueError):
            _beam(**kw)
    graded = FakeT([6, 50])
    graded.requires_grad = True
    with pytest.raises(ValueError, match="logits: requires a gradient"):
        _beam(logits=graded)
    assert calls == ["dflash_beam_select"] * 3
    with torch.no_grad():
        _beam(logits=graded)
    with pytest.raises(ValueError, match="dtype"):
        ops.beam_workspace(1, 1, 1, 1, torch.float64)


# ------------------------------------------------------------------ the definitions themselves

def test_the_pools_definition_keeps_its_counts():
    """The lists that the kernels are tested against: no page is lost or held twice through random calls."""
    rng = random.Random(1)
    for trial in range(60):
        batch, width, page = rng.randint(1, 6), rng.randint(1, 5), 16
        n_pages = rng.randint(1, batch * width + 3)
        p = beam_ref.Pool([0] * n_pages, [[-1] * width for _ in range(batch)], [0] * batch, page)
        text = [[] for _ in range(batch)]  # what each sequence should hold, as (writer, position)
        data = {}
        for turn in range(12):
            new = [rng.choice([0, n, n + 1, rng.randint(0, width * page)]) for n in p.lens]
            before = p.lens[:]
            moves = p.resize(new)
            if p.status & beam_ref.CAPACITY:
                p.status = 0
                if p.lens == before:
                    continue
            for s, d, n in moves:
                for i in range(n):
                    data[d, i] = data[s, i]
            for b in range(batch):
                del text[b][p.lens[b]:]
                for pos in range(len(text[b]), p.lens[b]):
                    text[b].append((trial, turn, b, pos))
                    data[p.table[b][pos // page], pos % page] = text[b][-1]
            parents = [rng.choice([b, -1, rng.randrange(batch)]) for b in range(batch)]
            p.fork(parents)
            text = [list(text[q]) if q >= 0 else [] for q in parents]
            p.check()
            moves, _ = p.compact()
            for s, d, n in moves:
                for i in range(n):
                    if (s, i) in data:
                        data[d, i] = data[s, i]
            p.check()
            for b in range(batch):  # every sequence still reads what it wrote, or its forebears
                assert [data[p.table[b][i // page], i % page] for i in range(p.lens[b])] == text[b]


def test_the_selections_definition():
    logits = torch.tensor([[0., 1., 1., -math.inf], [2., math.nan, 0., math.inf]])
    got = beam_ref.select(logits, torch.tensor([[-1., -2.]]), 9)
    lse = [math.log(1 + 2 * math.e), math.log(math.exp(2) + 1)]
    want = [(-1 + 1 - lse[0], 0, 1), (-1 + 1 - lse[0], 0, 2), (-1 - lse[0], 0, 0), (-2 + 2 - lse[1], 1, 0), (-2 - lse[1], 1, 2)]
    want.sort(key=lambda w: -w[0])
    assert [g[1:] for g in got[0]] == [w[1:] for w in want]
    assert all(abs(g[0] - w[0]) < 1e-12 for g, w in zip(got[0], want))


def test_views_of_bytes_are_as_the_checks_see_them():
    assert _bytes((0, ((2, 4), (3, 1))), 4)[1] is False and _bytes((0, ((2, 2), (3, 1))), 4)[1] is True
