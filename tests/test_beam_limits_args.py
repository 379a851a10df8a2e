"""Sizes past 32 bits in the page and beam-search calls, on the CPU."""
import pytest
import torch

from block_diffusion_speculative_hiddens_gb300 import ops
from tests.test_ops_args import FakeT, Stream

I32 = torch.int32


@pytest.fixture
def calls(monkeypatch):
    got = []

    class Lib:
        def __getattr__(self, name):
            def fn(*a):
                got.append((name, a))
                return 0
            return fn
    monkeypatch.setattr(ops, "load", lambda: Lib())
    monkeypatch.setattr(ops, "_clear_word", lambda device, n=1: FakeT([n], I32))
    return got


def test_long_lists_of_copies_are_not_cut_by_their_length(calls):
    """2^32 + 1 rows of room are not room for none."""
    moves = FakeT([2 ** 32 + 1, 3], I32)
    cache = ops.PagedCache(FakeT([8, 64, 2, 128], ptr=1 << 30), FakeT([8, 64, 2, 128], ptr=1 << 31), FakeT([3, 4], I32))
    ops.copy_pages(cache, moves, stream=Stream())
    pool = ops.PagePool(FakeT([3, 4], I32), 8, 64)
    ops.resize(pool, FakeT([3], I32), moves=moves, stream=Stream())
    ops.compact(pool, moves=moves, remap=FakeT([8], I32), stream=Stream())
    rooms = {name: a[{"dflash_pages_copy": 3, "dflash_pages_resize": 3, "dflash_pages_compact": 2}[name]] for name, a in calls}
    assert rooms == dict.fromkeys(("dflash_pages_copy", "dflash_pages_resize", "dflash_pages_compact"), 2 ** 31 - 1)
    ops.copy_pages(cache, FakeT([9, 3], I32), stream=Stream())
    assert calls[-1][1][3] == 8


@pytest.mark.parametrize("at", range(4))
def test_sizes_of_a_workspace_are_32_bits(at):
    shape = [2, 4, 1000, 4]
    for bad in (2 ** 31, 2 ** 32 + shape[at], -2 ** 31 - 1):
        shape[at] = bad
        with pytest.raises(ValueError, match=("batch", "beams", "vocab", "n")[at]):
            ops.beam_workspace(*shape, torch.float16)
