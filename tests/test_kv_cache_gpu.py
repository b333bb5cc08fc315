"""kv_cache_write / kv_cache_read against their definition in 64 bits: codes and scales are
equal bit for bit, slots that no row names stay as they were (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def raw(t):
    return t.cpu().view(torch.uint8)


def run_write(b: ref.Batch, k, v, what):
    cache, batch = b.device(csa)
    csa.kv_cache_write(cache, batch, k.cuda(), v.cuda())
    assert csa.get_status() == 0, what
    for name, x in (("k", k), ("v", v)):
        codes, scale = b.values(name)
        ref.write(codes, scale, x, b.offsets, b.lengths, b.table, b.fmt)
        got = getattr(cache, name).cpu()
        live = b.live[:, None, :, None].expand(got.shape)
        assert torch.equal(got.float().double()[live], codes[live]), f"{what}: codes of {name}"
        # -0 and 0 are one value; every other slot keeps its bytes
        assert torch.equal(raw(got)[~live], raw(b.codes[name])[~live]), f"{what}: slots of {name}"
        used = b.live.any(1)
        assert torch.equal(getattr(cache, name + "_scale").cpu()[used].double(), scale[used]), \
            f"{what}: scales of {name}"
    return cache


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,old,Hkv,D,P", [
    ([1], [0], 1, 16, 16),
    ([1, 1, 1, 1], [15, 16, 17, 100], 3, 64, 16),
    ([8, 3, 0, 5], [9, 30, 12, 0], 2, 48, 32),
    ([200, 1, 64, 65, 129], [0, 63, 64, 1, 127], 2, 128, 64),
    ([300, 17], [5, 250], 4, 80, 128),
    ([9, 40], [0, 3], 1, 112, 16),
])
def test_write(new, old, Hkv, D, P, dtype, fmt):
    b = ref.Batch(new, old, Hkv, D, P, fmt, seed=sum(new) + D, extra_rows=3)
    # rows of very different size: blocks that grow, and blocks that do not
    k, v = (b.rows_of(Hkv, dtype, seed=s) * torch.exp2(
        torch.randn((b.rows, Hkv, 1), generator=torch.Generator().manual_seed(s)) * 3).to(dtype)
        for s in (1, 2))
    run_write(b, k, v, (new, old))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_write_ties_extremes_and_odd_values(dtype, fmt):
    """Values half-way between codes, the type's largest and smallest, zeros, infinities and
    NaN, in a short (one warp per block) and a long call."""
    top = torch.finfo(dtype).max
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133
    for n in (6, 40):
        b = ref.Batch([n, n], [0, 10], 8, 64, 16, fmt, seed=n)
        k = torch.zeros((b.rows, 8, 64))
        k[:, 0] = (torch.arange(64) - 32) / 2.0          # ties when the scale is 1
        k[:, 0, 0] = 127.0
        k[:, 1] = 0.0
        k[:, 2] = tiny
        k[:, 3] = torch.linspace(-1, 1, 64) * top
        k[:, 4] = torch.randn(64, generator=b.g)
        k[1, 4, 3], k[2, 4, 5], k[3, 4, 9] = float("inf"), float("-inf"), float("nan")
        k[:, 5] = float("nan")
        k[:, 6] = 448.0 * 2.0 ** -3
        k[1, 6] = 449.0
        k[:, 7] = torch.linspace(0, 30, 64) * 2.0 ** -9  # e4m3's subnormal steps beside
        k[0, 7, 0] = 448.0
        k = k.to(dtype)
        run_write(b, k, -k.flip(0), (n, dtype, fmt))


def test_every_quotient_of_a_scale():
    """int8: all 2^15 finite magnitudes of bf16 within 127 s for scales of all 128 leading
    bits: the code is that of the exact quotient (ties included)."""
    x = torch.arange(0, 0x7F80, dtype=torch.int16).view(torch.bfloat16)
    x = x[(x.float() >= 2.0 ** -8) & (x.float() < 2.0 ** 8)]      # 16 binades of 128
    n = 128
    heads = n  # one head per scale: its largest value is m
    m = (2.0 ** 8 * (1 + torch.arange(n) / n)).to(torch.bfloat16)
    per = 64
    rows = -(-x.numel() // per)
    data = torch.zeros((rows * per,), dtype=torch.bfloat16)
    data[: x.numel()] = x
    k = data.view(rows, 1, per).expand(rows, heads, per).clone()
    k = torch.cat([k, m.view(1, heads, 1).expand(1, heads, per)])
    b = ref.Batch([k.shape[0]], [0], heads, per, 128, "int8")
    run_write(b, k.contiguous(), (-k).contiguous(), "quotients")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", DTYPES + [torch.float32])
@pytest.mark.parametrize("new,old,Hkv,D,P", [
    ([1, 1], [0, 31], 3, 16, 16),
    ([5, 0, 7], [20, 9, 0], 2, 96, 32),
    ([300, 64, 1], [0, 64, 191], 2, 128, 64),
])
def test_read(new, old, Hkv, D, P, dtype, fmt):
    b = ref.Batch(new, old, Hkv, D, P, fmt, seed=D, extra_rows=2)
    cache, batch = b.device(csa)
    k, v = (torch.full((b.rows, Hkv, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    csa.kv_cache_read(k, v, cache, batch)
    assert csa.get_status() == 0
    for name, got in (("k", k), ("v", v)):
        codes, scale = b.values(name)
        want = torch.full((b.rows, Hkv, D), 3.0, dtype=torch.float64)
        for s in range(len(new)):
            for j in range(new[s]):
                t = old[s] + j
                p = b.table[s][t // P]
                want[b.offsets[s] + j] = codes[p, :, t % P] * scale[p][:, None]
        assert torch.equal(got.cpu(), want.to(dtype)), name


def test_strided_rows():
    """K and V as slices of one packed row; read into head-major tensors."""
    b = ref.Batch([40, 3], [7, 100], 2, 64, 32, "int8", seed=4)
    packed = torch.randn((b.rows, 6, 64), generator=b.g).to(torch.bfloat16)
    cache, batch = b.device(csa)
    d = packed.cuda()
    csa.kv_cache_write(cache, batch, d[:, 2:4], d[:, 4:6])
    other, _ = b.device(csa)
    csa.kv_cache_write(other, batch, d[:, 2:4].contiguous(), d[:, 4:6].contiguous())
    assert torch.equal(raw(cache.k), raw(other.k)) and torch.equal(raw(cache.v), raw(other.v))
    k, v = (torch.empty((2, b.rows, 64), device="cuda").transpose(0, 1) for _ in range(2))
    csa.kv_cache_read(k, v, cache, batch)
    k2, v2 = (torch.empty((b.rows, 2, 64), device="cuda") for _ in range(2))
    csa.kv_cache_read(k2, v2, cache, batch)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_more_rows_than_tokens():
    """A sequence with more rows than its length: those before its beginning are dropped by
    a write and left alone by a read."""
    b = ref.Batch([5], [0], 1, 16, 16, "int8")
    cache, _ = b.device(csa)
    off, length, table = b.ints()
    length.fill_(3)
    batch = csa.KvBatch(off, length, table, rows=5)
    k = torch.randn((5, 1, 16), device="cuda").to(torch.bfloat16)
    csa.kv_cache_write(cache, batch, k, -k)
    out = torch.full((5, 1, 16), 9.0, device="cuda")
    out2 = out.clone()
    csa.kv_cache_read(out, out2, cache, batch)
    assert bool((out[:2] == 9).all()) and bool((out[2:] != 9).all())
    s = float(cache.k_scale[b.table[0][0], 0])
    assert float((out[2:] - k[2:].float()).abs().max()) <= s / 2
    assert csa.get_status() == 0


def test_bad_indices_are_skipped_and_reported():
    """Page numbers, offsets and lengths out of range (checked by the kernels themselves):
    what they name is skipped, other sequences are served, the status says so once."""
    b = ref.Batch([2, 2, 2, 2], [14, 20, 5, 40], 2, 32, 16, "int8", seed=2)
    k = b.rows_of(2, torch.bfloat16).cuda()

    def run(change):
        cache, _ = b.device(csa)
        off, length, table = b.ints()
        change(off, length, table)
        before = raw(cache.k).clone()
        csa.kv_cache_write(cache, csa.KvBatch(off, length, table, rows=b.rows, max_new=2), k, k)
        assert csa.get_status() == csa.CSA_ERR_INDEX
        assert csa.get_status() == 0
        return before, raw(cache.k)

    page = b.table[1][1]  # the page sequence 1's new tokens go to
    for bad in (-1, b.pages, 2 ** 31 - 1):
        before, after = run(lambda o, n, t: t[1].__setitem__(1, bad))
        assert torch.equal(before[page], after[page])
        assert not torch.equal(before[b.table[3][2]], after[b.table[3][2]])
    for change in (lambda o, n, t: n.__setitem__(1, t.shape[1] * 16 + 1),
                   lambda o, n, t: n.__setitem__(1, -1)):
        before, after = run(change)
        assert torch.equal(before[page], after[page])
        assert not torch.equal(before[b.table[3][2]], after[b.table[3][2]])
    run(lambda o, n, t: o.__setitem__(4, b.rows + 1))   # past the rows
    run(lambda o, n, t: o.__setitem__(1, 7))            # decreasing, and more than max_new


def test_graph_replay_follows_the_batch():
    """Captured once, replayed with the batch's arrays changed in place."""
    P = 16
    b = ref.Batch([1, 1], [3, 16], 2, 32, P, "e4m3", seed=8, width_extra=3)
    cache, batch = b.device(csa)
    x = torch.randn((2, 2, 32), device="cuda").to(torch.bfloat16)
    y = torch.empty((2, 2, 32), device="cuda")
    z = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.kv_cache_write(cache, batch, x, x)
        csa.kv_cache_read(y, z, cache, batch)
    for _ in range(3):
        x.normal_()
        batch.lengths.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        for got, scale in ((y, cache.k_scale), (z, cache.v_scale)):  # (older scales differ)
            sc = torch.stack([scale[b.table[s][(int(batch.lengths[s]) - 1) // P]] for s in range(2)])
            # e4m3: half a step is 2^-4 relatively, or half of the smallest step, 2^-9 scales
            room = torch.maximum(x.float().abs() * 2.0 ** -4, sc[..., None] * 2.0 ** -10)
            assert bool(((got - x.float()).abs() <= room).all())
    assert csa.get_status() == 0
