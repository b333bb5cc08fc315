"""Calls on a stream that is not the current one: what the binding allocates and fills for
them is in that stream's order (GPU). Streams are held by a host function
(csa_debug_hold_stream), so nothing waits on the GPU."""
import contextlib
import time

import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref
from causal_attention_score_gb300 import _lib

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def held(handle: int):
    """The stream of this handle stands still inside (10 s at most)."""
    lib = _lib.load()
    assert lib.csa_debug_hold_stream(handle) == 0
    try:
        yield
    finally:
        lib.csa_debug_release_streams()


def attention_case(seed=3):
    """A small call: (q, cache, batch), and its result."""
    b = ref.Batch([2, 1], [90, 40], 2, 64, 32, "int8", seed=seed)
    cache, batch = b.device(csa)
    q = b.rows_of(4, torch.bfloat16).cuda()
    want = csa.cache_attention(q, cache, batch)
    torch.cuda.synchronize()
    return q, cache, batch, want


class Aside:
    """Looks at tensors from a stream of its own, whatever the others still have to do."""

    def __init__(self, *tensors):
        self.stream = torch.cuda.Stream()
        self.host = [torch.empty(t.shape, dtype=t.dtype, pin_memory=True) for t in tensors]

    def look(self, *tensors):
        with torch.cuda.stream(self.stream):
            for h, t in zip(self.host, tensors):
                h.copy_(t, non_blocking=True)
        self.stream.synchronize()
        return self.host


def test_raw_handle_of_the_default_stream():
    """stream=0 is the legacy default stream, also where the binding allocates a workspace."""
    q, cache, batch, want = attention_case()
    X, W = (torch.randn((n, 770), device="cuda").to(torch.bfloat16) for n in (96, 64))
    y = csa.dense(X, W)
    assert csa.dense_workspace_size(X, W, 96, 770, 64) > 0
    out, y2 = torch.full_like(want, 7.0), torch.full_like(y, 7.0)
    csa.cache_attention_forward(torch.empty_like(want), q, cache, batch, stream=0)
    csa.dense_xwt(torch.empty_like(y), X, W, 96, 770, 64, stream=0)
    aside = Aside(out, y2)
    aside.look(out, y2)
    torch.cuda.synchronize()
    with held(0):
        csa.cache_attention_forward(out, q, cache, batch, stream=0)
        csa.dense_xwt(y2, X, W, 96, 770, 64, stream=0)
        time.sleep(0.1)
        early = aside.look(out, y2)
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in early), "ran past the held stream"
    assert torch.equal(out, want) and torch.equal(y2, y)


def test_allocating_attention_while_the_current_stream_is_busy():
    """cache_attention(stream=B) with the current stream held: its zeros and its rows are in
    B's order, so the result is there when B is done and stays."""
    q, cache, batch, want = attention_case()
    host_want = want.cpu()
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(2):  # (once for the allocator's blocks and the modules)
        with torch.cuda.stream(B):
            csa.cache_attention(q, cache, batch)
    aside = Aside(want)
    aside.look(want)
    torch.cuda.synchronize()
    for stream in (B, B.cuda_stream):
        with torch.cuda.stream(A), held(A.cuda_stream):
            out = csa.cache_attention(q, cache, batch, stream=stream)
            B.synchronize()
            early, = aside.look(out)
            assert torch.equal(early, host_want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert csa.get_status() == 0


@pytest.mark.parametrize("which", ["trimul", "causal_softmax", "dense", "cache_attention"])
def test_allocating_forms_leave_the_current_stream_its_memory(which):
    """What the current stream has freed but still has to read is not what a call on another
    stream gets for its output."""
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((1, 200, 3, 2, 64), generator=g).to(torch.bfloat16).cuda()
    X, W = (torch.randn((n, 768), generator=g).to(torch.bfloat16).cuda() for n in (300, 256))
    if which == "cache_attention":
        q, cache, batch, _ = attention_case()
    call = {"trimul": lambda st: csa.trimul(qkv, mask="-inf", stream=st),
            "causal_softmax": lambda st: csa.causal_softmax(qkv, stream=st),
            "dense": lambda st: csa.dense(X, W, stream=st),
            "cache_attention": lambda st: csa.cache_attention(q, cache, batch, stream=st)}[which]
    want = call(None)
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    call(B)
    torch.cuda.synchronize()
    with torch.cuda.stream(A):
        t, keep = torch.full_like(want, 5.0), torch.empty_like(want)
        A.synchronize()
        with held(A.cuda_stream):
            keep.copy_(t)
            del t
            out = call(B)
            B.synchronize()
    torch.cuda.synchronize()
    assert bool((keep == 5.0).all()), "the output took memory that the current stream still read"
    assert torch.equal(out, want)
    assert csa.get_status() == 0


def grouped_case():
    """A batch whose rows no tensor map can describe: (Ys, Xs, W, its workspace's bytes)."""
    g = torch.Generator().manual_seed(3)
    Xs = [torch.randn((m, 770), generator=g).to(torch.bfloat16).cuda() for m in (500, 301)]
    W = torch.randn((256, 770), generator=g).to(torch.bfloat16).cuda()
    Ys = [torch.zeros((len(X), 256), device="cuda") for X in Xs]
    return Ys, Xs, W, csa.DenseGroupedPlan(Ys, Xs, W, 770, 256)._ws.numel()


def test_grouped_workspace_is_in_the_calls_order():
    """dense_xwt_grouped(stream=B): its workspace is not memory that the current stream still
    reads, nor does that stream get it while the call is under way."""
    Ys, Xs, W, nbytes = grouped_case()
    csa.dense_xwt_grouped(Ys, Xs, W, 770, 256)
    want = [Y.clone() for Y in Ys]
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    csa.dense_xwt_grouped(Ys, Xs, W, 770, 256, stream=B)
    torch.cuda.synchronize()
    with torch.cuda.stream(A):
        t = torch.full((nbytes,), 5, dtype=torch.uint8, device="cuda")
        keep = torch.empty_like(t)
        A.synchronize()
        with held(A.cuda_stream):
            keep.copy_(t)
            del t
            csa.dense_xwt_grouped(Ys, Xs, W, 770, 256, stream=B)
            B.synchronize()
        torch.cuda.synchronize()
        assert bool((keep == 5).all()), "took memory that the current stream still read"
        with held(B.cuda_stream):
            csa.dense_xwt_grouped(Ys, Xs, W, 770, 256, stream=B)
            t = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
            A.synchronize()
        torch.cuda.synchronize()
        assert bool((t == 7).all()), "gave memory back before the call was done with it"
    assert all(torch.equal(Y, w) for Y, w in zip(Ys, want))


def test_plan_let_go_while_its_call_is_under_way():
    """A plan made on one stream, called on another and let go of: its workspace stays the call's."""
    Ys, Xs, W, nbytes = grouped_case()
    csa.dense_xwt_grouped(Ys, Xs, W, 770, 256)
    want = [Y.clone() for Y in Ys]
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(A):
        plan = csa.DenseGroupedPlan(Ys, Xs, W, 770, 256)
        A.synchronize()
        with held(B.cuda_stream):
            plan(B)
            del plan
            t = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
            A.synchronize()
        torch.cuda.synchronize()
        assert bool((t == 7).all())
    assert all(torch.equal(Y, w) for Y, w in zip(Ys, want))
