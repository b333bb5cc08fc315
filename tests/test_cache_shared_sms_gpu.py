"""How cache_attention_shared_forward shares the SMs out: between its two parts, and with calls on
other streams (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import shared_ref as ref
from test_cache_shared_gpu import check, run

pytestmark = pytest.mark.gpu


class Large:
    """One group of sequences over random codes, made on the device; every table row is written out,
    so that cache_attention_forward takes the same batch."""

    def __init__(self, new, own, shared, Hq=32, Hkv=8, D=128, P=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        S, lead = len(new), shared // P
        blocks = [-(-(o + n) // P) for o, n in zip(own, new)]
        pages, width = lead + sum(blocks), lead + max(blocks)
        codes = [torch.randint(-127, 128, (pages, Hkv, P, D), generator=g, device="cuda", dtype=torch.int8)
                 for _ in range(2)]
        scales = [torch.rand((pages, Hkv), generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2)]
        self.cache = csa.KvCache(*codes, *scales)
        table = torch.zeros((S, width), dtype=torch.int32)
        at = lead
        for s, n in enumerate(blocks):
            table[s, :lead] = torch.arange(lead, dtype=torch.int32)
            table[s, lead: lead + n] = torch.arange(at, at + n, dtype=torch.int32)
            at += n
        offsets = torch.tensor([sum(new[:s]) for s in range(S + 1)], dtype=torch.int32)
        lengths = torch.tensor([shared + o + n for o, n in zip(own, new)], dtype=torch.int32)
        self.rows = sum(new)
        self.batch = csa.KvBatch(offsets.cuda(), lengths.cuda(), table.cuda(), rows=self.rows, max_new=max(new))
        self.groups = torch.tensor([0, S], dtype=torch.int32, device="cuda")
        self.shared = torch.tensor([shared], dtype=torch.int32, device="cuda")
        self.q = torch.randn((self.rows, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.empty_like(self.q)
        self.ws = torch.empty(csa.cache_attention_shared_workspace_size(self.cache, self.batch, Hq, 1),
                              dtype=torch.uint8, device="cuda")
        self.plain_ws = torch.empty(csa.cache_attention_workspace_size(self.cache, self.batch, Hq),
                                    dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        csa.cache_attention_shared_forward(self.out, self.q, self.cache, self.batch, self.groups, self.shared,
                                           workspace=self.ws, stream=stream)

    def plain(self, stream=None):
        csa.cache_attention_forward(self.out, self.q, self.cache, self.batch, workspace=self.plain_ws,
                                    stream=stream)


def best_us(call, times=10):
    for _ in range(3):
        call()
    took = []
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b) * 1e3)
    return min(took)


# Sequences of more rows a kv head than the kernel of few rows otherwise takes, but too few of them
# for the kernel of prompts: 12 x 9 tokens of 4 query heads a kv head, and a chunk of 64 tokens beside
# 63 single ones.
MIDDLING = [([9] * 12, 3000, 8192), ([1] * 63 + [64], 2000, 8192)]


@pytest.mark.parametrize("new,own,shared", MIDDLING)
def test_rows_left_to_the_kernel_of_few_rows_have_sms(new, own, shared):
    """The own parts of such sequences are work like any other when the SMs are shared out. Not to
    have them counted cost a factor of ten and more; sharing saves work here, so twice the time of
    the call that shares nothing is far off."""
    b = Large(new, [own] * len(new), shared)
    together, plain = best_us(b.call), best_us(b.plain)
    assert csa.get_status() == 0
    assert together < 2 * plain, (together, plain)


@pytest.mark.parametrize("mode", [csa.SHARED_AUTO, csa.SHARED_ALWAYS])
def test_middling_rows_against_definition(mode):
    csa.set_shared_part(mode)
    try:
        b = ref.SharedBatch([9] * 12, [(7 * i) % 60 for i in range(12)], [(0, 12, 192)], 8, 32, 32, "int8", seed=21)
        q, out = run(b, 32, torch.bfloat16)
        check(b, q, out)
    finally:
        csa.set_shared_part(csa.SHARED_AUTO)


def test_a_limited_call_leaves_the_other_sms_to_a_call_beside_it():
    """Two streams limited to half the SMs each: a short call that begins while a long shared one runs
    does not wait for the latter's end."""
    half = torch.cuda.get_device_properties(0).multi_processor_count // 2
    long = Large([1] * 128, [100] * 128, 65536)
    short = Large([1] * 8, [2048] * 8, 64, seed=1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        csa.set_stream_sm_limit(s, half)
    try:
        def timed(beside):
            gate = torch.cuda.Event()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            z = torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            torch.cuda._sleep(1_000_000)  # until everything is launched
            z.record()
            gate.record()
            for s in streams:
                s.wait_event(gate)
            if beside:
                long.call(streams[0])
            end = torch.cuda.Event(enable_timing=True)
            end.record(streams[0])
            with torch.cuda.stream(streams[1]):
                torch.cuda._sleep(200_000)  # the long call's own parts are done
            a.record(streams[1])
            short.plain(streams[1])
            b.record(streams[1])
            torch.cuda.synchronize()
            return a.elapsed_time(b) * 1e3, z.elapsed_time(end) * 1e3

        for _ in range(2):
            timed(True), timed(False)
        want_long, want_short = long.out.clone(), short.out.clone()
        alone = min(timed(False)[0] for _ in range(5))
        runs = [timed(True) for _ in range(5)]
        assert csa.get_status() == 0
        assert torch.equal(long.out, want_long) and torch.equal(short.out, want_short)
        beside, took = min(r[0] for r in runs), min(r[1] for r in runs)
        assert took > 200, took  # (the long call is still under way when the short one begins)
        assert beside < alone + 0.25 * took, (alone, beside, took)
    finally:
        torch.cuda.synchronize()
        for s in streams:
            csa.set_stream_sm_limit(s, 0)
