"""Selection and page calls at the limits of what they accept: logits too large for
a shared exponent."""
import pytest
import torch

from tests.test_gpu_beam import BF16, F32, check_select, gen

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
@pytest.mark.parametrize("value", [1e8, 1e9, 1.8e9, 2.0 ** 31, 2.5e9, 1e10])
def test_rows_of_large_logits(ops, dtype, value):
    """Rows of one large value, of either sign, and of values close to it."""
    g = gen(22)
    for sign in (1, -1):
        flat = torch.full((4, 9001), sign * value, device="cuda").to(dtype)
        check_select(ops, flat, torch.zeros(2, 2, device="cuda"), 40, exact=True)
        near = (sign * value * (1 - 0.1 * torch.rand(3, 20011, generator=g, device="cuda"))).to(dtype)
        check_select(ops, near, -torch.rand(1, 3, generator=g, device="cuda"), 10)
