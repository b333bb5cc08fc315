"""What token_logprobs_forward and _backward leave as it was, and rows at the kernels' borders (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
from test_logprobs_gpu import TYPES, rows_of, test_forward as check_forward

pytestmark = pytest.mark.gpu


def held_apart(x, dtype, pitch, shift):
    """(x as rows vocab + pitch apart on the GPU, its storage, whose other elements are 99)."""
    rows, vocab = x.shape
    held = torch.full((shift + rows * (vocab + pitch) + 64,), 99.0, dtype=dtype, device="cuda")
    view = held[shift: shift + rows * (vocab + pitch)].view(rows, vocab + pitch)[:, :vocab]
    view.copy_(x.to(dtype))
    return view, held


def only_inside(view, held, what):
    outside = torch.ones_like(held, dtype=torch.bool)
    outside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((held[outside] == 99.0).all()), what
    assert not bool((view == 99.0).any()), what


# (of a CTA a row, several CTAs a row, and a warp each of many; beside chunks of 16 bytes and not)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,pitch,d_pitch,shift,d_shift,top", [
    (1, 1, 3, 3, 1, 1, 1), (3, 2, 1, 5, 1, 0, 2), (40, 333, 7, 7, 3, 3, 5), (40, 333, 7, 2, 3, 1, 5),
    (2, 50257, 7, 7, 5, 5, 32), (5, 50257, 8, 3, 0, 2, 0), (650, 2051, 13, 13, 1, 1, 3),
    (2000, 333, 3, 3, 1, 1, 32), (2000, 1001, 7, 2, 3, 5, 4), (30000, 17, 1, 1, 2, 2, 5)])
def test_the_gradient_writes_its_rows_alone(rows, vocab, pitch, d_pitch, shift, d_shift, top, dtype):
    g = torch.Generator().manual_seed(rows + vocab)
    x, held = held_apart(rows_of("normal", rows, vocab, g), dtype, pitch, shift)
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    tokens[0], tokens[-1] = 0, vocab - 1  # (elements with a weight of their own at the rows' ends)
    if rows > 2:
        tokens[1] = -1
    t = tokens.cuda()
    _, entropy, stats, _, top_token = csa.token_logprobs(x, t, top)
    only_inside(x, held, "forward")
    d, d_top = torch.ones((rows,), device="cuda"), torch.ones((rows, top), device="cuda")
    dx, d_held = held_apart(torch.full((rows, vocab), 99.0), dtype, d_pitch, d_shift)
    csa.token_logprobs_backward(dx, x, t, stats, entropy, d, d, d_top, top_token)
    only_inside(dx, d_held, "apart")
    only_inside(x, held, "apart: logits")
    csa.token_logprobs_backward(x, x, t, stats, entropy, d, d, d_top, top_token)
    only_inside(x, held, "in place")
    assert csa.get_status() == 0


@pytest.mark.parametrize("kind", ["normal", "rising", "equal"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_short_rows_of_31_chunks_and_14_loose_words(dtype, kind):
    """The most words that a lane without a chunk leaves in a row: with 32 alternatives all are candidates."""
    check_forward(kind, 1900, 262, 2, 1, 32, 1.0, dtype)
