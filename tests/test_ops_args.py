"""The caller-target operators on the CPU: the rotation plans against the
scalings' formulas, the packed argument structs against the C ones, and the
refusals -- a wrong tensor never reaches the library."""
import ctypes
import math
import os

import pytest
import torch

from block_diffusion_speculative_hiddens_gb300 import _build, binding, ops
from tests import ops_ref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB):
        _build.build()
    return binding.load()


SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 8.0},
            {"kind": "yarn", "factor": 4.0, "original_len": 32768},
            {"kind": "yarn", "factor": 16.0, "original_len": 4096, "beta_fast": 24.0, "beta_slow": 2.0,
             "attention_factor": 1.25},
            {"kind": "llama3", "factor": 8.0, "original_len": 8192, "low_freq_factor": 1.0, "high_freq_factor": 4.0},
            "factors"]


@pytest.mark.parametrize("rd,theta", [(128, 1e6), (64, 5e5), (32, 1e4), (6, 1e4)])
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: str(s and s["kind"] if isinstance(s, dict) else s))
def test_plan_holds_the_scaled_frequencies(lib, rd, theta, scaling):
    if scaling == "factors":
        scaling = {"kind": "factors", "factors": [1 + 0.5 * i for i in range(rd // 2)], "attention_factor": 1.1}
    p = ops.RopePlan(rd, theta, interleaved=True, scaling=scaling)
    freq, amp = ops_ref.frequencies(rd, theta, scaling)
    assert p.amplitude == pytest.approx(amp, rel=2 ** -24)
    for i, w in enumerate(freq):
        turn = w / (2 * math.pi) % 1.0  # a handful of double roundings, and the last place of 2^-64
        assert abs(p._c.turn[i] / 2.0 ** 64 - turn) <= 16 * 2.0 ** -53 * turn + 2.0 ** -63
    assert all(p._c.turn[i] == 0 for i in range(rd // 2, ops.MAX_PAIRS))


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(rotary_dim=64, theta=1.0),
    dict(rotary_dim=64, theta=math.inf), dict(rotary_dim=64, theta=math.nan),
    dict(rotary_dim=2, scaling={"kind": "ntk", "factor": 2.0}),
    dict(rotary_dim=64, scaling={"kind": "linear", "factor": 0.0}),
    dict(rotary_dim=64, scaling={"kind": "linear", "factor": math.nan}),
    dict(rotary_dim=64, scaling={"kind": "yarn", "factor": 2.0, "original_len": 0}),
    dict(rotary_dim=64, scaling={"kind": "yarn", "factor": 2.0, "original_len": 9, "beta_fast": 1.0, "beta_slow": 2.0}),
    dict(rotary_dim=64, scaling={"kind": "llama3", "factor": 2.0, "original_len": 9, "low_freq_factor": 4.0}),
    dict(rotary_dim=4, scaling={"kind": "factors", "factors": [1.0, -1.0]}),
])
def test_plan_refuses_what_has_no_rotation(lib, kw):
    kw = dict(theta=1e4) | kw
    with pytest.raises(binding.DflashError) as e:
        ops.RopePlan(kw.pop("rotary_dim"), kw.pop("theta"), **kw)
    assert e.value.code == 1


@pytest.mark.parametrize("scaling", [{"kind": "dynamic", "factor": 2.0}, {"factor": 2.0}, {"kind": "linear"},
                                     {"kind": "linear", "factor": 2.0, "original_len": 5},
                                     {"kind": "factors", "factors": [1.0] * 3}])
def test_plan_refuses_scalings_it_does_not_know(lib, scaling):
    with pytest.raises(ValueError):
        ops.RopePlan(64, 1e4, scaling=scaling)


def test_c_entries_refuse_before_any_cuda_call(lib):
    plan = ops.RopePlan(128, 1e4)
    one = ops._ROWS
    rows = (16, 128, 128)

    def rope(rows_n=1, hq=1, hk=1, dim=128, dtype=1, pos=16, plan_=plan, q=rows, out=rows):
        a = ops._ROPE.pack(*q, *rows, *out, *rows, pos, rows_n, hq, hk, dim, dtype, 0, 0)
        return lib.dflash_rope(None if plan_ is None else plan_._ref, a, None)
    assert one == "Pqq"
    assert rope(plan_=None) == 1 and rope(rows_n=-1) == 1 and rope(hq=-1) == 1 and rope(dtype=2) == 1
    assert rope(pos=0) == 1 and rope(out=(0, 0, 0)) == 1
    assert rope(dim=64) == 2 and rope(dim=129) == 2 and rope(dim=258) == 2
    assert rope(rows_n=0) == 0 and rope(hq=0, hk=0) == 0

    def cache(k=256, table=256, status=256, max_pages=4, stride=4, pages=8, page=64, heads=2, dim=128, dtype=1,
              ks=(16384, 256, 128)):
        return ops._CACHE.pack(k, 256, *ks, 16384, 256, 128, table, stride, status, max_pages, pages, page, heads, dim,
                               dtype, 0)

    def append(c=None, rows_n=1, batch=1, k=rows, cu=16, ctx=16, q=(0, 0, 0), hq=0, plan_=plan):
        a = ops._APPEND.pack(*k, *rows, *q, 0, 0, 0, cu, ctx, rows_n, batch, hq, 0)
        return lib.dflash_paged_append(cache() if c is None else c, None if plan_ is None else plan_._ref, a, None)
    assert append(rows_n=-1) == 1 and append(batch=-1) == 1 and append(k=(0, 0, 0)) == 1 and append(cu=0) == 1
    assert append(ctx=0) == 1 and append(q=rows, hq=2) == 1  # q without a place to go
    assert append(rows_n=0) == 0 and append(batch=0) == 0
    assert lib.dflash_paged_append(None, None, None, None) == 1

    def attention(c=None, rows_n=1, batch=1, hq=4, q=rows, out=rows, cu=16, ctx=16, ws=256, wsb=1 << 40, window=0,
                  scale=1.0):
        a = ops._ATTENTION.pack(*q, *out, 0, 0, 0, cu, ctx, 0, ws, wsb, rows_n, batch, hq, 1, window, scale)
        return lib.dflash_paged_attention(cache() if c is None else c, a, None)
    assert attention(rows_n=-1) == 1 and attention(window=-1) == 1 and attention(scale=math.nan) == 1
    assert attention(q=(0, 0, 0)) == 1 and attention(out=(0, 0, 0)) == 1 and attention(cu=0) == 1
    assert attention(ctx=0) == 1
    assert attention(hq=3) == 2 and attention(hq=0) == 2 and attention(hq=66) == 2
    assert attention(q=(24, 128, 128)) == 1 and attention(q=(16, 100, 128)) == 1 and attention(out=(16, 128, 4)) == 1
    assert attention(c=cache(ks=(16384, 260, 128))) == 1 and attention(c=cache(ks=(16380, 256, 128))) == 1
    assert attention(ws=128) == 6 and attention(wsb=-1) == 6
    assert attention(batch=8193) == 3
    assert attention(rows_n=0) == 0 and attention(batch=0) == 0
    for bad, code in ((dict(k=0), 1), (dict(table=0), 1), (dict(status=0), 1), (dict(max_pages=0), 1),
                      (dict(stride=3), 1), (dict(pages=0), 1), (dict(heads=0), 1), (dict(dtype=5), 1),
                      (dict(page=8), 2), (dict(page=48), 2), (dict(page=512), 2)):
        assert append(c=cache(**bad)) == code, bad
        assert attention(c=cache(**bad)) == code, bad
    assert attention(c=cache(dim=96)) == 2
    assert lib.dflash_paged_attention(None, None, None) == 1
    assert lib.dflash_paged_attention_workspace(None, 1, 1, 1) == 0


class FakeT:
    """A tensor that says it is on a CUDA device."""

    def __init__(self, shape, dtype=torch.bfloat16, device="cuda:0", stride=None, ptr=0x100000):
        self.shape, self.dtype, self.device, self.ptr = tuple(shape), dtype, torch.device(device), ptr
        self._s = tuple(stride) if stride else tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def get_device(self):
        return -1 if self.device.type == "cpu" else self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self._s == FakeT(self.shape)._s

    def data_ptr(self):
        return self.ptr


class Stream:
    cuda_stream = 0
    device = torch.device("cuda:0")


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
    return got


def _cache():
    c = ops.PagedCache.__new__(ops.PagedCache)
    c.device, c.dtype, c.head_dim, c.kv_heads, c.batch, c._c = 0, torch.bfloat16, 128, 2, 3, b""
    return c


I32 = torch.int32


def _attention(**kw):
    a = dict(q=FakeT([7, 4, 128]), cu=FakeT([4], I32), ctx=FakeT([3], I32), out=FakeT([7, 4, 128], ptr=1 << 30),
             workspace=FakeT([256], torch.uint8), stream=Stream(), lse=None, kv_len=None)
    a.update(kw)
    return ops.attention(_cache(), a.pop("q"), a.pop("cu"), a.pop("ctx"), **a)


def _append(**kw):
    a = dict(k=FakeT([7, 2, 128], ptr=1 << 28), v=FakeT([7, 2, 128], ptr=1 << 29), cu=FakeT([4], I32), ctx=FakeT([3], I32),
             q=FakeT([7, 4, 128]), q_out=FakeT([7, 4, 128], ptr=1 << 30), stream=Stream())
    a.update(kw)
    return ops.append(_cache(), a.pop("k"), a.pop("v"), a.pop("cu"), a.pop("ctx"), **a)


def _rope(**kw):
    class P:
        _ref = None
    a = dict(q=FakeT([7, 4, 128]), k=FakeT([7, 2, 128], ptr=1 << 28), positions=FakeT([7], I32),
             q_out=FakeT([7, 4, 128], ptr=1 << 30), k_out=FakeT([7, 2, 128], ptr=1 << 31), stream=Stream())
    a.update(kw)
    return ops.rope(P(), a.pop("q"), a.pop("k"), a.pop("positions"), **a)


def test_well_formed_calls_reach_the_library(calls):
    _rope()
    _rope(k=None, k_out=None)
    _rope(q_out=FakeT([7, 4, 128]))  # in place
    _append()
    _append(q=None, q_out=None)
    _attention()
    _attention(lse=FakeT([7, 4], torch.float32), kv_len=FakeT([3], I32))
    assert [c for c in calls if "workspace" not in c] == ["dflash_rope"] * 3 + ["dflash_paged_append"] * 2 + [
        "dflash_paged_attention"] * 2


def test_q_and_k_views_of_one_projection_rotate_in_place_and_apart(calls):
    qkv = dict(stride=(8 * 128, 128, 1))
    q, k = FakeT([7, 4, 128], **qkv), FakeT([7, 2, 128], ptr=0x100000 + 4 * 256, **qkv)
    _rope(q=q, k=k, q_out=q, k_out=k)
    wide = dict(stride=(12 * 128, 128, 1))
    q, k, far = FakeT([7, 4, 128], **wide), *(FakeT([7, n, 128], ptr=0x100000 + h * 256, **wide) for n, h in ((2, 4), (4, 8)))
    _rope(q=q, k=k, q_out=far, k_out=k)  # other heads of the same rows
    for kw in (dict(q_out=FakeT([7, 4, 128], ptr=0x100000 + 2 * 256, **wide)),  # half of q
               dict(q_out=FakeT([7, 4, 128], ptr=0x100000 + 5 * 256, **wide)),  # half of k
               dict(k_out=FakeT([7, 2, 128], ptr=0x100000 + 3 * 256, **wide)),
               dict(q_out=far, k_out=FakeT([7, 2, 128], ptr=0x100000 + 9 * 256, **wide))):
        with pytest.raises(ValueError, match="overlaps"):
            _rope(q=q, k=k, **kw)
    for name in "kv":
        kw = {name: FakeT([7, 2, 128], ptr=(1 << 30) + 512)}
        with pytest.raises(ValueError, match="q_out: overlaps [kv]$"):
            _append(**kw)


def test_outputs_that_overlap_themselves_are_refused(calls):
    for s in ((0, 128, 1), (512, 0, 1), (512, 64, 1), (256, 128, 1), (128, 512, 1)):
        out = FakeT([7, 4, 128], stride=s, ptr=1 << 30)
        for call in (lambda: _rope(q_out=out), lambda: _append(q_out=out), lambda: _attention(out=out)):
            with pytest.raises(ValueError, match="one another"):
                call()
        with pytest.raises(ValueError, match="one another"):
            _attention(q=out, out=out)
    for shape, s in (([7, 4, 128], (128, 7 * 128, 1)), ([1, 4, 128], (0, 128, 1)), ([7, 4, 128], (4096, 136, 1))):
        q = FakeT(shape)
        _attention(q=q, out=FakeT(shape, stride=s, ptr=1 << 30))
        _rope(q=q, k=None, k_out=None, q_out=FakeT(shape, stride=s, ptr=1 << 30), positions=FakeT([shape[0]], I32))


BAD = [FakeT([7, 4, 128], torch.float16), FakeT([7, 4, 128], device="cuda:1"), FakeT([7, 4, 128], device="cpu"),
       FakeT([7, 128]), FakeT([7, 4, 64]), FakeT([7, 4, 128], stride=(1024, 256, 2))]


@pytest.mark.parametrize("bad", BAD, ids=range(len(BAD)))
def test_wrong_row_tensors_are_refused(calls, bad):
    for call in (lambda: _attention(q=bad), lambda: _attention(out=bad), lambda: _append(q=bad), lambda: _append(q_out=bad),
                 lambda: _append(k=bad), lambda: _append(v=bad), lambda: _rope(q_out=bad), lambda: _rope(k=bad)):
        with pytest.raises(ValueError):
            call()
    assert [c for c in calls if "workspace" not in c] == []


@pytest.mark.parametrize("kw", [
    dict(cu=FakeT([3], I32)), dict(cu=FakeT([4], torch.int64)), dict(ctx=FakeT([4], I32), cu=FakeT([5], I32)),
    dict(ctx=FakeT([3], I32, device="cuda:1")), dict(cu=FakeT([4], I32, stride=(2,)))])
def test_wrong_batches_are_refused(calls, kw):
    for call in (_attention, _append):
        with pytest.raises(ValueError):
            call(**kw)
    assert [c for c in calls if "workspace" not in c] == []


def test_other_refusals(calls):
    for kw in (dict(lse=FakeT([7, 4], torch.float16)), dict(lse=FakeT([4, 7], torch.float32)),
               dict(kv_len=FakeT([2], I32)), dict(workspace=FakeT([256], torch.float32)),
               dict(workspace=FakeT([256], torch.uint8, device="cuda:1")), dict(out=FakeT([6, 4, 128]))):
        with pytest.raises(ValueError):
            _attention(**kw)
    for kw in (dict(positions=FakeT([6], I32)), dict(positions=FakeT([7], torch.int64)), dict(q_out=FakeT([7, 5, 128])),
               dict(q_out=FakeT([7, 4, 128], ptr=0x100000 + 256)), dict(k=FakeT([6, 2, 128]))):
        with pytest.raises(ValueError):
            _rope(**kw)
    other = Stream()
    other.device = torch.device("cuda:1")
    for call in (_rope, _append, _attention):
        with pytest.raises(ValueError, match="stream"):
            call(stream=other)
    assert [c for c in calls if "workspace" not in c] == []
    cpu = torch.zeros(4, 64, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.PagedCache(cpu, cpu, torch.zeros(1, 4, dtype=torch.int32))


def test_packed_structs_match_the_header(tmp_path):
    """The sizes a C compiler gives the header's structs."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ["dflash_rope_args", "dflash_paged_cache", "dflash_append_args", "dflash_attention_args",
             "dflash_rope_config", "dflash_rope_plan"]
    src = tmp_path / "s.c"
    src.write_text('#include "%s"\n#include <stdio.h>\nint main(void) { printf("%s", %s); return 0; }\n' % (
        binding.HEADER, " ".join(["%zu"] * 6), ", ".join("sizeof(%s)" % n for n in names)))
    subprocess.run([cc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ops._ROPE.size, ops._CACHE.size, ops._APPEND.size, ops._ATTENTION.size,
                   ctypes.sizeof(ops.RopeConfig), ctypes.sizeof(ops._Plan)]


@pytest.fixture
def no_device(monkeypatch):
    """A cache's own memory, without a device."""
    monkeypatch.setattr(ops, "_clear_word", lambda device: FakeT([1], I32))


def _table(shape, stride):
    pool = FakeT([8, 64, 2, 128])
    cache = ops.PagedCache(pool, FakeT([8, 64, 2, 128], ptr=1 << 30), FakeT(shape, I32, stride=stride, ptr=1 << 34))
    return ops._CACHE.unpack(cache._c)[9:12:2]  # stride and width of a row


@pytest.mark.parametrize("stride", [(0, 1), (1, 1), (3, 1)])
def test_page_tables_whose_rows_overlap_are_refused(no_device, stride):
    """An expanded table (one row for all sequences) has no row stride that the calls could use."""
    for batch in (2, 3, 100):
        with pytest.raises(ValueError, match="page_table: rows overlap"):
            _table([batch, 4], stride)


def test_page_tables_keep_their_row_stride(no_device):
    assert _table([3, 4], (4, 1)) == (4, 4)
    assert _table([3, 4], (16, 1)) == (16, 4)  # a slice of a wider table
    assert _table([1, 4], (0, 1)) == (4, 4)  # the stride of a single row says nothing
    assert _table([1, 4], (16, 1)) == (16, 4)


def test_status_entry_refuses_before_any_cuda_call(lib):
    word = ctypes.c_uint32(7)
    assert lib.dflash_paged_read_status(None, ctypes.byref(word)) == 1
    good = (256, 256, 16384, 256, 128, 16384, 256, 128, 256, 4, 256, 4, 8, 64, 2, 128, 1, 0)
    assert lib.dflash_paged_read_status(ops._CACHE.pack(*good), None) == 1
    bad = list(good)
    bad[10] = 0  # no status word
    assert lib.dflash_paged_read_status(ops._CACHE.pack(*bad), ctypes.byref(word)) == 1
    assert word.value == 7


def test_no_kernel_asks_which_lanes_are_active():
    """A warp's lanes may be apart at any point; masks come from the block's shape."""
    import glob
    for f in glob.glob(os.path.join(_build.CSRC, "*.cu*")) + glob.glob(os.path.join(_build.CSRC, "*.h")):
        with open(f) as src:
            assert "__activemask" not in src.read(), f


@pytest.mark.parametrize("bad", [FakeT([512], ptr=1 << 28), FakeT([7, 512], ptr=1 << 28), FakeT([], ptr=1 << 28),
                                 FakeT([7, 4, 128], torch.float32, ptr=(1 << 28) - 512)], ids=["1d", "2d", "0d", "f32"])
def test_appends_output_is_checked_before_it_is_compared(calls, bad):
    """Its shape and type are refused as such, wherever it lies."""
    with pytest.raises(ValueError, match="q_out: expected"):
        _append(q_out=bad)
    assert calls == []


def test_outputs_without_their_input_are_refused(calls):
    """They would come back unwritten."""
    with pytest.raises(ValueError, match="q_out: given without q"):
        _append(q=None)
    with pytest.raises(ValueError, match="k_out: given without k"):
        _rope(k=None)
    assert calls == []


# A device that no machine has: a call that passes its checks ends there (4), before anything is queued.
NOWHERE = 1000


def _bytes(view, size=2):
    """Every byte of a view (address, count and stride of each dimension in elements), and whether one is there twice."""
    at, dims = view
    where = [at]
    for n, s in dims:
        where = [w + size * s * i for w in where for i in range(n)]
    every = [w + j for w in where for j in range(size)]
    return set(every), len(set(every)) < len(every)


def test_rope_refuses_outputs_that_share_memory(lib):
    """Random strides of rows and heads against the sets of bytes behind them: written bytes are written once, and
    read by nothing but the output's own input (in place)."""
    import random
    rng = random.Random(5)
    plan = ops.RopePlan(2, 1e4)
    seen = {1: 0, 4: 0}
    for trial in range(6000):
        rows, hq, hk, d = rng.randint(1, 5), rng.randint(1, 4), rng.randint(1, 3), rng.choice([2, 4, 6])
        base = 1 << 20

        def rows_of(h):
            kind = rng.random()
            head = d * rng.choice([1, 1, 1, 2, 3])
            row = head * h + d * rng.choice([0, 0, 1, 3, 7, 13])
            if kind < 0.25:  # heads first
                row, head = head, head * rows + d * rng.choice([0, 1, 4])
            elif kind < 0.3:
                row, head = rng.randint(0, 20), rng.randint(0, 20)
            return base + 2 * rng.choice([d * rng.randint(0, 60), rng.randint(0, 300)]), row, head
        q, k = rows_of(hq), rows_of(hk)
        qo = q if rng.random() < 0.4 else rows_of(hq)
        ko = k if rng.random() < 0.4 else rows_of(hk)
        if rng.random() < 0.3:  # heads of one buffer's rows
            wide = d * (hq + hk) * 2
            q, k = (base, wide, d), (base + 2 * d * hq, wide, d)
            qo = rng.choice([q, (base + 2 * d * (hq + hk), wide, d), (base + 2 * d * (hq + hk - 1), wide, d)])
            ko = rng.choice([k, (base + 2 * d * (2 * hq + hk), wide, d)])
        pos = 1 << 24 if rng.random() < 0.9 else base + 4 * rng.randint(0, 300)

        def view(x, h):
            return x[0], ((rows, x[1]), (h, x[2]), (d, 1))

        def same(x, y, h):
            return x[0] == y[0] and (rows == 1 or x[1] == y[1]) and (h == 1 or x[2] == y[2])
        (bq, _), (bk, _) = _bytes(view(q, hq)), _bytes(view(k, hk))
        (bqo, twice), (bko, twice_k) = _bytes(view(qo, hq)), _bytes(view(ko, hk))
        bp, _ = _bytes((pos, ((rows, 1),)), 4)
        wrong = twice or twice_k or bqo & bko or bqo & bk or bko & bq or (bqo | bko) & bp or \
            (bqo & bq and not same(qo, q, hq)) or (bko & bk and not same(ko, k, hk))
        a = ops._ROPE.pack(*q, *k, *qo, *ko, pos, rows, hq, hk, d, 1, 0, NOWHERE)
        got = lib.dflash_rope(plan._ref, a, None)
        seen[got] += 1
        if got == 1 and not wrong:  # strides that are not nested are refused without a closer look
            strides = [sorted((s, n) for n, s in view(x, h)[1] if n > 1) for x, h in ((qo, hq), (ko, hk))]
            assert any(s < 1 + sum((n - 1) * t for t, n in st[:i]) for st in strides for i, (s, _) in enumerate(st))
        else:
            assert got == (1 if wrong else 4), (trial, q, k, qo, ko, rows, hq, hk, d)
    assert min(seen.values()) > 500


def _paged(hq=2, k=1 << 24, v=1 << 25, ks=(2048, 128, 64), vs=(2048, 128, 64), table=1 << 26, pages=5, stride=4):
    return ops._CACHE.pack(k, v, *ks, *vs, table, stride, 1 << 27, 4, pages, 16, 2, 64, 1, NOWHERE)


def test_paged_calls_refuse_outputs_that_share_memory(lib):
    rows, t = lambda at, row=256, head=64: (at, row, head), 7
    none = (0, 0, 0)

    def attention(out=rows(1 << 21), lse=none, q=rows(1 << 20), cache=None, cu=1 << 28, ctx=1 << 29, kv=0):
        a = ops._ATTENTION.pack(*q, *out, *lse, cu, ctx, kv, 0, 0, t, 2, 4, 1, 0, 0.125)
        return lib.dflash_paged_attention(cache or _paged(), a, None)

    def append(q_out=rows(1 << 21), k=rows(1 << 22, 128), v=rows(1 << 23, 128), cache=None):
        a = ops._APPEND.pack(*k, *v, *rows(1 << 20), *q_out, 1 << 28, 1 << 29, t, 2, 4, 0)
        return lib.dflash_paged_append(cache or _paged(), None, a, None)
    good = [attention(), attention(out=rows(1 << 20)), attention(lse=(1 << 22, 4, 1)), append(), append(q_out=rows(1 << 20)),
            attention(out=rows(1 << 21, 64, 64 * t)), attention(lse=(1 << 22, 1, t)),
            # pools that alternate by page, by position and by head; K and V of one pool, which only the append may not have
            append(cache=_paged(ks=(4096, 128, 64), vs=(4096, 128, 64), v=(1 << 24) + 4096)),
            append(cache=_paged(ks=(4096, 256, 64), vs=(4096, 256, 64), v=(1 << 24) + 256)),
            append(cache=_paged(ks=(4096, 256, 128), vs=(4096, 256, 128), v=(1 << 24) + 128)),
            append(cache=_paged(ks=(64, 64 * 5, 64 * 5 * 16), vs=(64, 64 * 5, 64 * 5 * 16))),
            attention(cache=_paged(v=1 << 24)),
            # out behind the heads of the pool's positions
            attention(cache=_paged(ks=(16 * 640, 640, 64)), out=rows((1 << 24) + 256, 640), q=rows(1 << 20))]
    assert good == [4] * len(good), good
    bad = [attention(out=rows((1 << 24) - 512 * t + 2)), attention(out=rows((1 << 25) + 5 * 4096 - 2)),
           attention(out=rows((1 << 26) + 28)), attention(out=rows((1 << 27))), attention(out=rows((1 << 28) + 8)),
           attention(out=rows((1 << 29) - 2 * 1024)), attention(kv=(1 << 21) + 128),
           attention(lse=((1 << 21) + 64, 4, 1)), attention(lse=((1 << 20) + 3580, 4, 1)), attention(lse=((1 << 24), 4, 1)),
           attention(lse=(1 << 22, 0, 1)), attention(lse=(1 << 22, 4, 0)), attention(lse=(1 << 22, 3, 1)),
           attention(lse=((1 << 28) + 8, 4, 1)), attention(out=rows(1 << 21, 192)), attention(out=rows((1 << 20) + 128)),
           attention(out=rows(1 << 20, 256, 128)),
           append(q_out=rows((1 << 24) + 128)), append(q_out=rows((1 << 22) + 512)), append(q_out=rows((1 << 23) + 64)),
           append(q_out=rows((1 << 20) + 128)), append(q_out=rows((1 << 26) + 16)),
           append(cache=_paged(v=1 << 24)), append(cache=_paged(v=(1 << 24) + 4096)), append(cache=_paged(ks=(0, 128, 64))),
           append(cache=_paged(ks=(2048, 64, 64))), append(cache=_paged(ks=(64, 64 * 4, 64 * 4 * 16)))]
    assert bad == [1] * len(bad), bad


def _graded(shape, **kw):
    t = FakeT(shape, **kw)
    t.requires_grad = True
    return t


def test_tensors_that_require_a_gradient_are_refused_while_gradients_are_recorded(calls):
    """The calls are not differentiable by autograd: the graph would be dropped without a word."""
    tries = [(lambda: _rope(q=_graded([7, 4, 128])), "q"), (lambda: _rope(k=_graded([7, 2, 128], ptr=1 << 28)), "k"),
             (lambda: _rope(q_out=_graded([7, 4, 128], ptr=1 << 30)), "q_out"),
             (lambda: _rope(k_out=_graded([7, 2, 128], ptr=1 << 31)), "k_out"),
             (lambda: _append(q=_graded([7, 4, 128])), "q"), (lambda: _append(k=_graded([7, 2, 128], ptr=1 << 28)), "k"),
             (lambda: _append(v=_graded([7, 2, 128], ptr=1 << 29)), "v"),
             (lambda: _append(q_out=_graded([7, 4, 128], ptr=1 << 30)), "q_out"),
             (lambda: _attention(q=_graded([7, 4, 128])), "q"),
             (lambda: _attention(out=_graded([7, 4, 128], ptr=1 << 30)), "out"),
             (lambda: _attention(lse=_graded([7, 4], dtype=torch.float32)), "lse")]
    for call, name in tries:
        with pytest.raises(ValueError, match="^%s: requires a gradient" % name):
            call()
    assert [c for c in calls if "workspace" not in c] == []
    with torch.no_grad():
        for call, _ in tries:
            call()
    with torch.inference_mode():
        tries[0][0]()
    assert len([c for c in calls if "workspace" not in c]) == len(tries) + 1


@pytest.mark.parametrize("which", ["k_pool", "v_pool"])
def test_pools_that_require_a_gradient_are_refused_while_gradients_are_recorded(calls, no_device, which):
    pools = {"k_pool": FakeT([8, 64, 2, 128], ptr=1 << 35), "v_pool": FakeT([8, 64, 2, 128], ptr=1 << 36)}
    pools[which].requires_grad = True
    cache = ops.PagedCache(*pools.values(), FakeT([3, 4], I32, ptr=1 << 37))
    q, cu, ctx = FakeT([7, 4, 128]), FakeT([4], I32), FakeT([3], I32)
    k, v = FakeT([7, 2, 128], ptr=1 << 28), FakeT([7, 2, 128], ptr=1 << 29)
    for call in (lambda: ops.append(cache, k, v, cu, ctx, stream=Stream()),
                 lambda: ops.attention(cache, q, cu, ctx, out=FakeT([7, 4, 128], ptr=1 << 30),
                                       workspace=FakeT([256], torch.uint8), stream=Stream())):
        with pytest.raises(ValueError, match="^%s: requires a gradient" % which):
            call()
        with torch.no_grad():
            call()


@pytest.mark.parametrize("kw", [dict(rotary_dim=2 ** 32 + 64), dict(rotary_dim=-2 ** 32 + 64),
                                dict(scaling={"kind": "yarn", "factor": 4.0, "original_len": 2 ** 32 + 4096}),
                                dict(scaling={"kind": "llama3", "factor": 4.0, "original_len": 2 ** 31}),
                                dict(scaling={"kind": "yarn", "factor": 4.0, "original_len": 4096.5})])
def test_plan_refuses_whole_numbers_that_do_not_fit(lib, kw):
    """They were cut to 32 bits, or to a whole number, and another rotation came back."""
    with pytest.raises(ValueError, match="32-bit whole number"):
        ops.RopePlan(kw.pop("rotary_dim", 64), 1e4, **kw)


def test_plan_takes_whole_numbers_of_other_types(lib):
    want = ops.RopePlan(64, 1e4, scaling={"kind": "yarn", "factor": 4.0, "original_len": 4096})
    got = ops.RopePlan(torch.tensor(64).item(), 1e4, scaling={"kind": "yarn", "factor": 4.0, "original_len": 4096.0})
    assert bytes(got._c) == bytes(want._c)


def test_scales_without_a_softmax_are_refused(lib):
    """Infinite, or infinite once in the logarithm's base: every score would be infinite or NaN."""
    c = _paged()
    for scale, code in ((math.inf, 1), (-math.inf, 1), (3e38, 1), (-3e38, 1), (math.nan, 1), (1e38, 4), (0.0, 4), (-0.1, 4)):
        a = ops._ATTENTION.pack(1 << 20, 256, 64, 1 << 21, 256, 64, 0, 0, 0, 1 << 28, 1 << 29, 0, 0, 0, 1, 1, 4, 1, 0, scale)
        assert lib.dflash_paged_attention(c, a, None) == code, scale
