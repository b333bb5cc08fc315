"""rotary_forward / rotary_backward on [B, T, heads, size] tensors, single tokens sliced from
longer ones among them, against the formula in 64 bits (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu

H, D = 3, 64


def check(got, want, size, dtype):
    # the bound derived in test_rotary_gpu.py, and one rounding to the type
    bound = size * 2.0 ** -20 + want.abs() * ref.half_step(dtype)
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,T,at", [(4, 9, slice(0, 9)), (4, 9, slice(-1, None)), (4, 9, slice(2, 3)),
                                    (1, 9, slice(3, 7)), (5, 1, slice(0, 1)), (1, 1, slice(0, 1))])
def test_batches(B, T, at, backward):
    """Whole batches, and one token of each, in place and into a tensor of another layout."""
    g = torch.Generator().manual_seed(B + T)
    x = torch.randn((B, T, H, D), generator=g).to(torch.bfloat16)
    part = x[:, at]
    n = part.shape[1]
    table, f = csa.RotaryTable(D), ref.frequencies(D)
    pos = torch.randint(0, 5000, (B, n), generator=g).to(torch.int32)
    want, size = ref.rotary(part.reshape(B * n, H, D), pos.flatten(), f, backward=backward)
    want, size = want.view(B, n, H, D), size.view(B, n, H, D)
    call = csa.rotary_backward if backward else csa.rotary_forward
    xd = x.cuda()
    out = torch.full((B, n, H, D), 7.0, dtype=x.dtype, device="cuda")
    call(out, xd[:, at], table, pos.cuda())
    check(out, want, size, x.dtype)
    assert torch.equal(xd.cpu(), x)
    call(xd[:, at], xd[:, at], table, pos.cuda())
    assert torch.equal(xd[:, at], out)
    rest = torch.ones(T, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(xd.cpu()[:, rest], x[:, rest])


def test_start_and_period_of_single_tokens():
    """One token of each batch, all at the same position: period 1."""
    x = torch.randn((6, 20, H, D), generator=torch.Generator().manual_seed(1))
    out = torch.empty((6, 1, H, D), device="cuda")
    csa.rotary_forward(out, x.cuda()[:, 13:14], csa.RotaryTable(D), start=13, period=1)
    want, size = ref.rotary(x[:, 13], torch.full((6,), 13), ref.frequencies(D))
    check(out[:, 0], want, size, torch.float32)


def test_batches_that_do_not_follow_one_another():
    """Several tokens of each batch of a longer tensor have no one stride: refused."""
    x = torch.zeros((3, 8, H, D), device="cuda")
    with pytest.raises(ValueError):
        csa.rotary_forward(torch.empty((3, 2, H, D), device="cuda"), x[:, 2:4], csa.RotaryTable(D))
    with pytest.raises(ValueError):
        csa.rotary_forward(x[:, 2:4], torch.empty((3, 2, H, D), device="cuda"), csa.RotaryTable(D))
