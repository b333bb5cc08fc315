"""rotary_forward / rotary_backward against the formula in 64 bits (GPU).

Bound per element, from the kernel's arithmetic: the angle's fraction of a turn is rounded
to 32 bits and to fp32 (pi * 2^-25 in all), sincospif is off by at most 2 units of 2^-24 for
values up to 1, the amplitude's product and the two products and one sum round four times:
less than 2^-20 (|x0| + |x1|) a together; then one rounding to the type."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref
from causal_attention_score_gb300 import synth

pytestmark = pytest.mark.gpu

LONG = {"linear": {"factor": 8.0}, "ntk": {"factor": 8.0}, "none": {},
        "by_parts": {"factor": 8.0, "original_length": 4096.0}}


def check(got, want, size, dtype, what):
    bound = size * 2.0 ** -20 + want.abs() * ref.half_step(dtype) + 2.0 ** -25 * (dtype == torch.float16)
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err - bound)[bad].max())}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,size,rd,scaling,backward", [
    (1, 1, 2, 2, "none", False),
    (3, 5, 64, 64, "none", True),
    (37, 9, 80, 48, "linear", False),
    (130, 3, 128, 128, "ntk", True),
    (65, 6, 128, 64, "by_parts", False),
    (17, 2, 34, 10, "none", False),   # rows of no 16-byte multiple
    (5, 33, 96, 24, "by_parts", True),
])
def test_against_formula(tokens, heads, size, rd, scaling, backward, interleaved, dtype):
    g = torch.Generator().manual_seed(tokens + rd)
    x = torch.randn((tokens, heads, size), generator=g).to(dtype)
    pos = torch.randint(0, 2 ** 26, (tokens,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = 0
    pos[-1] = 2 ** 20 - 1
    table = csa.RotaryTable(rd, scaling=scaling, amplitude=1.25, **LONG[scaling])
    want, mag = ref.rotary(x, pos, ref.frequencies(rd, scaling=scaling, **LONG[scaling]),
                           interleaved, backward, 1.25)
    # (a frequency held in 53 bits, a few roundings apart on both sides, moves the angle of
    # position 2^26 by less than 2^-24 radians)
    call = csa.rotary_backward if backward else csa.rotary_forward
    out = torch.full_like(x, 7.0).cuda()
    call(out, x.cuda(), table, pos.cuda(), interleaved=interleaved)
    check(out, want, mag, dtype, "apart")
    y = x.cuda()
    call(y, y, table, pos.cuda(), interleaved=interleaved)
    assert torch.equal(y, out), "in place"
    assert csa.get_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_padding(dtype):
    """Head-major and sliced tensors, out of other strides, odd alignment; rows of negative
    positions stay as they were."""
    T, H, D = 29, 4, 64
    g = torch.Generator().manual_seed(3)
    big = torch.randn((H, T, 2 * D + 1), generator=g).to(dtype)
    pos = torch.randint(0, 1000, (T,), generator=g).to(torch.int32)
    pos[[2, 11, T - 1]] = -1
    table = csa.RotaryTable(32)
    for off in (0, 1, 8):
        x = big.cuda().transpose(0, 1)[:, :, off: off + D]
        assert x.stride(0) < x.stride(1)
        want, mag = ref.rotary(x.cpu(), pos.clamp(min=0), ref.frequencies(32))
        out = torch.full((T, H + 2, D), 5.0, dtype=dtype, device="cuda")
        csa.rotary_forward(out[:, 1: H + 1], x, table, pos.cuda())
        live = pos >= 0
        check(out[:, 1: H + 1][live.cuda()], want[live], mag[live], dtype, f"offset {off}")
        assert bool((out[~live.cuda()] == 5.0).all()) and bool((out[:, 0] == 5.0).all())
        assert bool((out[:, H + 1] == 5.0).all())


def test_start_and_period():
    T, table = 50, csa.RotaryTable(64)
    x = torch.randn((T, 2, 64), generator=torch.Generator().manual_seed(1))
    out = torch.empty_like(x, device="cuda")
    for start, period in ((0, 0), (123456, 0), (7, 20), (2 ** 31 - T, 0)):
        csa.rotary_forward(out, x.cuda(), table, start=start, period=period)
        t = torch.arange(T)
        pos = start + (t % period if period else t)
        want, mag = ref.rotary(x, pos, ref.frequencies(64))
        # near 2^31 the 53 bits of frequencies and angles, a few roundings apart on both
        # sides, are worth 2^31 * 4 * 2^-53 = 2^-20 radians
        check(out, want, mag * 2, torch.float32, f"start {start} period {period}")


def test_packed_qkv_then_scores():
    """rotary_qkv on the packed tensor: V untouched, and the causal scores that trimul then
    computes depend on the distance of two tokens only."""
    B, T, NH, HS = 2, 70, 3, 64
    shape = synth.TrimulShape(B=B, T=T, C=NH * HS, NH=NH)
    qkv = synth.trimul_input(shape, seed=5).reshape(B, T, 3, NH, HS)
    table = csa.RotaryTable(HS)
    f = ref.frequencies(HS)
    here = {}
    for start in (0, 1000):
        d = qkv.cuda()
        csa.rotary_qkv(d, table, start=start)
        assert torch.equal(d[:, :, 2].cpu(), qkv[:, :, 2])
        for part in (0, 1):
            x = qkv[:, :, part].reshape(B * T, NH, HS)
            want, mag = ref.rotary(x, start + torch.arange(B * T) % T, f)
            check(d[:, :, part].reshape(B * T, NH, HS), want, mag, torch.bfloat16, f"part {part}")
        here[start] = csa.trimul(d, mask="-inf").cpu()
        back = d.clone()
        csa.rotary_qkv(back, table, start=start, backward=True)
        # there and back: two bf16 roundings of a pair, 2^-9 of its length each, and the
        # rotation's own error
        pair = torch.hypot(qkv[:, :, :2, :, : HS // 2].double(), qkv[:, :, :2, :, HS // 2:].double())
        err = (back[:, :, :2].cpu().double() - qkv[:, :, :2].double()).abs()
        assert bool((err <= torch.cat([pair, pair], -1) * (2 * 2.0 ** -8 + 2.0 ** -15)).all())
    a, b = here[0], here[1000]
    low = torch.isfinite(a)
    # q and k rounded to bf16 after other rotations: 2^-8 of their lengths each, twice
    q, k = (qkv[:, :, i].double().norm(dim=-1).permute(0, 2, 1) for i in (0, 1))
    room = (q[..., :, None] * k[..., None, :]) * (4 * 2.0 ** -8 * 1.01) / HS ** 0.5
    assert bool(((a - b).abs()[low] <= room[low]).all())


def test_gradient_against_differences():
    """sum(w * forward(x)) in fp32: its gradient by rotary_backward against differences.

    The map is linear, so a central difference of step 1/4 has no truncation error; its
    rounding is a few 2^-24 of the sum's magnitude over the step."""
    g = torch.Generator().manual_seed(9)
    T, H, D, rd = 4, 2, 12, 8
    x, w = (torch.randn((T, H, D), generator=g).cuda() for _ in range(2))
    table = csa.RotaryTable(rd, amplitude=0.75)
    pos = torch.tensor([0, 5, 77, 100003], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        dx = torch.empty_like(w)
        csa.rotary_backward(dx, w, table, pos, interleaved=interleaved)
        y = torch.empty_like(x)

        def f(z):
            csa.rotary_forward(y, z, table, pos, interleaved=interleaved)
            return float((y.double() * w.double()).sum())

        for i in range(0, x.numel(), 5):
            e = torch.zeros(x.numel(), device="cuda")
            e[i] = 0.25
            e = e.view_as(x)
            diff = (f(x + e) - f(x - e)) / 0.5
            assert abs(diff - float(dx.flatten()[i])) <= 2.0 ** -18 * 8


def test_other_stream_limit_and_graph():
    T, H, D = 300, 4, 64
    x = torch.randn((T, H, D), device="cuda").to(torch.float16)
    table = csa.RotaryTable(D)
    want = torch.empty_like(x)
    csa.rotary_forward(want, x, table, start=10)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(x)
    csa.set_stream_sm_limit(st, 3)
    try:
        csa.rotary_forward(out, x, table, start=10, stream=st)
    finally:
        csa.set_stream_sm_limit(st, 0)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.rotary_forward(out, x, table, start=10)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)
