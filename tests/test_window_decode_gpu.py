"""One-query window attention over 16-bit and block-scaled 8-bit caches
against the 64-bit form: masks, grouped heads, contexts split between blocks
of threads, stale rows and given-back blocks, streams, graphs and
workspaces."""
import pytest
import torch

from paged_kv_cache_481_b200 import binding
from window_helpers import Paged, check_decode, decode

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
STORES = [(F16, None), (BF16, None), (F16, "int8"), (BF16, "e4m3"), (BF16, "int8"), (F16, "e4m3")]


@pytest.mark.parametrize("dtype,codes", STORES)
@pytest.mark.parametrize("lens,heads,kvh,d,bs,window,sinks", [
    ([1], 1, 1, 64, 8, 1, 0),
    ([0, 1, 15, 16, 17, 33], 4, 4, 128, 16, 16, 0),
    ([0, 0, 0], 4, 2, 64, 16, 5, 2),
    ([5, 130, 64, 63, 65, 200], 14, 2, 128, 8, 50, 3),
    ([1000, 31, 0, 999, 257], 32, 2, 64, 32, 100, 70),
    ([300, 1, 2, 700], 17, 1, 128, 64, 1, 4),
    ([513, 40], 128, 1, 128, 128, 300, 130),
    ([3000, 2999], 10, 2, 128, 16, 4000, 0),
    ([77] * 40, 6, 6, 64, 16, 20, 1000),
    ([100, 7, 333, 64], 12, 2, 64, 8, 150, 9),
    ([2500, 100] * 30, 24, 12, 128, 32, 1500, 33),
    ([300] * 9 + [0, 1], 18, 2, 64, 16, 300, 0),
])
def test_against_64_bits(dtype, codes, lens, heads, kvh, d, bs, window, sinks):
    paged = Paged(lens, kvh, d, bs, dtype, seed=len(lens) * 7 + d, codes=codes)
    q = paged.randn((len(lens), heads, d))
    out = decode(paged, q, window, sinks, d ** -0.5)
    assert binding.pa_get_last_device_error() == 0
    check_decode(paged, q, out, window, sinks, d ** -0.5)


@pytest.mark.parametrize("dtype,codes", STORES[:4])
def test_long_contexts_are_split_and_merged(dtype, codes):
    """Few units, so every unit straddles several blocks of threads; the same
    bits on every run."""
    paged = Paged([20011, 9, 4097], 2, 128, 16, dtype, seed=5, codes=codes)
    q = paged.randn((3, 8, 128))
    ws = binding.new_window_workspace(3, 8, 2, 128)
    first = decode(paged, q, 30000, 0, 0.09, workspace=ws)
    check_decode(paged, q, first, 30000, 0, 0.09)
    for _ in range(5):
        assert torch.equal(decode(paged, q, 30000, 0, 0.09, workspace=ws), first)


@pytest.mark.parametrize("dtype,codes", STORES[1:3])
@pytest.mark.parametrize("lens,heads,kvh", [
    ([4100] * 16, 32, 8),                              # a unit to a few CTAs
    ([2100] * 47 + [0], 16, 8),                        # a unit a CTA
    ([1028] * 30 + [700, 1], 40, 40),                  # a unit a warp
    ([500 + 75 * i for i in range(48)], 32, 8),        # unlike lengths: equal ranges
    ([1100] * 60 + [3, 0, 999], 32, 32),               # more units than warps
    ([3000, 2999, 17], 64, 4), ([2000] * 20, 64, 4),   # 16 heads a group, few and many
    ([900] * 7, 40, 2),                                # 20 heads a group
])
def test_large_batches_are_shared_out(dtype, codes, lens, heads, kvh):
    paged = Paged(lens, kvh, 128, 16, dtype, seed=heads + kvh, codes=codes)
    q = paged.randn((len(lens), heads, 128))
    ws = binding.new_window_workspace(len(lens), heads, kvh, 128)
    out = decode(paged, q, 5000, 0, 0.09, workspace=ws)
    assert binding.pa_get_last_device_error() == 0
    check_decode(paged, q, out, 5000, 0, 0.09)
    assert torch.equal(decode(paged, q, 5000, 0, 0.09, workspace=ws), out)


@pytest.mark.parametrize("dtype,codes", STORES[:4])
def test_blocks_that_the_window_left_are_not_looked_at(dtype, codes):
    """Table entries of blocks without a visible position may be anything, and
    rows that are not seen may hold NaN or infinities."""
    lens, bs, window, sinks = [400, 97, 16], 16, 33, 3
    paged = Paged(lens, 2, 128, bs, dtype, seed=9, codes=codes)
    q = paged.randn((3, 4, 128))
    want = decode(paged, q, window, sinks, 0.1)
    check_decode(paged, q, want, window, sinks, 0.1)
    for b, n in enumerate(lens):
        start = n - window
        for t in range(sinks, start):       # hidden rows
            block = int(paged.tables[b, t // bs])
            if codes != "int8":
                for cache, junk in ((paged.k, float("nan")), (paged.v, float("inf"))):
                    if codes == "e4m3":
                        junk = float("nan")
                    rows = cache[block, :, t % bs].float()
                    cache[block, :, t % bs] = torch.full_like(rows, junk).to(cache.dtype)
        for j in range(-(-sinks // bs), max(0, start) // bs):
            paged.tables[b, j] = [-1, 2 ** 30, -7][j % 3]
    assert torch.equal(decode(paged, q, window, sinks, 0.1), want)
    assert binding.pa_get_last_device_error() == 0


@pytest.mark.parametrize("dtype,codes", STORES[:4])
def test_scores_of_large_magnitude(dtype, codes):
    """Scores up to several hundred: one token takes almost all the weight.
    The bound's score term grows with sum |q k| scale."""
    paged = Paged([600], 1, 64, 16, dtype, seed=13, codes=codes)
    q = paged.randn((1, 2, 64)) * 40
    out = decode(paged, q, 600, 0, 0.5)
    k, v = paged.context64(0)
    from window_helpers import attend64, attention_bound
    ref, mass = attend64(q, k, v, [599], 600, 0, 0.5)
    bound = attention_bound(ref, mass, dtype, F16 if codes else dtype, float(v.abs().max()), 600)
    # (64 + 8) 2^-23 sum |q k| scale, in the weight and in the total
    reach = torch.einsum("nhd,td->nht", q.double().abs(), k[:, 0].abs()).max() * 0.5
    bound = bound + 2 * 72 * 2.0 ** -23 * reach * mass
    assert bool(((out.double() - ref).abs() <= bound).all())


def test_zero_and_negative_scale():
    paged = Paged([100, 40], 2, 64, 16, BF16, seed=15)
    q = paged.randn((2, 4, 64))
    for scale in (0.0, -0.2):
        check_decode(paged, q, decode(paged, q, 30, 2, scale), 30, 2, scale)


def test_bad_lengths_and_blocks_are_recorded():
    paged = Paged([50, 20], 1, 64, 8, F16, seed=3, junk=0.0)
    q = paged.randn((2, 2, 64))
    binding.pa_get_last_device_error()
    decode(paged, q, 100, 0, 0.1, max_len=40)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_CONTEXT_LEN
    paged.tables[1, 1] = paged.nb
    out = decode(paged, q, 100, 0, 0.1)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_BLOCK_ID
    check_decode(paged, q, out, 100, 0, 0.1, seqs=[0])


def test_streams_graphs_and_a_shared_workspace():
    """Calls of several sizes and types one after the other on one workspace,
    on a side stream, and replayed from a graph."""
    cases = [(Paged([900, 3, 2500], 2, 128, 16, BF16, seed=1), 8),
             (Paged([5000], 1, 64, 8, F16, seed=2), 3),
             (Paged([700, 70, 7, 0], 4, 64, 32, F16, seed=3, codes="int8"), 4),
             (Paged([2049, 2048], 2, 128, 16, BF16, seed=4, codes="e4m3"), 64)]
    qs = [p.randn((len(p.lens), h, p.d)) for p, h in cases]
    size = max(binding.pa_decode_window_workspace_size(len(p.lens), h, p.kvh, p.d)
               for p, h in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    binding.pa_decode_workspace_init(ws)
    want = [decode(p, q, 2000, 4, 0.1) for (p, _), q in zip(cases, qs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = [decode(p, q, 2000, 4, 0.1, workspace=ws) for (p, _), q in zip(cases, qs)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    tables = [p.dev_tables() for p, _ in cases]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (p, _), q, (t, n), o in zip(cases, qs, tables, outs):
            if p.codes:
                binding.pa_decode_q8(o, q, p.k, p.v, p.scales, t, n, max(p.lens), 2000, 4, 0.1, ws)
            else:
                binding.pa_decode_window(o, q, p.k, p.v, t, n, max(p.lens), 2000, 4, 0.1, ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_whole_context_agrees_with_pa_decode():
    """fp16, one query head per K/V head and a window over everything is
    pa_decode's case; both are within their bounds of the same sum."""
    paged = Paged([1, 40, 700, 2000], 8, 128, 16, F16, seed=8)
    q = paged.randn((4, 8, 128))
    out, old = decode(paged, q, 2000, 0, 0.1), torch.empty_like(q)
    tables, lens = paged.dev_tables()
    binding.pa_decode(old, q, paged.k, paged.v, tables, lens, 2000, 0.1,
                      binding.new_workspace(4, 8, 128, 2000))
    check_decode(paged, q, out, 2000, 0, 0.1)
    check_decode(paged, q, old, 2000, 0, 0.1)


@pytest.mark.parametrize("codes", [None, "int8", "e4m3"])
@pytest.mark.parametrize("lens,heads,kvh,d", [([1, 40, 700, 5000], 8, 2, 128), ([300] * 40, 20, 10, 64),
                                              ([9000], 32, 2, 128), ([77, 0, 900], 5, 5, 64)])
def test_values_as_large_as_the_type_holds(codes, lens, heads, kvh, d):
    """bf16 values of half the type's largest, with one sign or both: their
    weighted mean is representable, and no sum on the way may leave fp32."""
    paged = Paged(lens, kvh, d, 16, BF16, seed=51, codes=codes)
    half = torch.finfo(BF16).max / 2
    for signs in (1, 2):
        if codes is None:
            nan = paged.v.isnan()
            v = torch.rand(paged.v.shape, generator=paged.gen, device="cuda") + 1.0      # [1, 2]
            v = v * (torch.sign(paged.v.float()) if signs == 2 else 1.0) * (half / 2)
            paged.v = v.to(BF16).masked_fill(nan, float("nan"))
        else:
            if signs == 1:
                v = paged.v.float().abs()
                paged.v = v.to(paged.v.dtype)
            top = float(paged.v.float().nan_to_num(0).abs().max())
            s = torch.rand(paged.scales.shape[:2], generator=paged.gen, device="cuda") + 1.0
            paged.scales[..., 1] = s * (half / top / 2)
        q = paged.randn((len(lens), heads, d)) * 2
        out = decode(paged, q, 6000, 3, d ** -0.5)
        assert binding.pa_get_last_device_error() == 0
        check_decode(paged, q, out, 6000, 3, d ** -0.5)


@pytest.mark.parametrize("codes", [None, "int8"])
def test_values_of_very_different_size_in_one_context(codes):
    """The parts of a split context hold values of 2^-90, 1 and 2^100: each
    part's sums are joined at their own size."""
    paged = Paged([12000], 2, 128, 16, BF16, seed=53, codes=codes)
    block = torch.from_numpy(paged.tables[0]).long().cuda()
    for lo, hi, size in ((0, 250, 2.0 ** -90), (250, 500, 1.0), (500, 750, 2.0 ** 100)):
        if codes is None:
            paged.v[block[lo:hi]] *= size
        else:
            paged.scales[block[lo:hi], :, 1] *= size
    q = paged.randn((1, 8, 128))
    check_decode(paged, q, decode(paged, q, 12000, 0, 0.09), 12000, 0, 0.09)
    for window, sinks in ((8000, 0), (4000, 0), (1, 4000)):     # without the smallest, the two smaller, the largest
        check_decode(paged, q, decode(paged, q, window, sinks, 0.09), window, sinks, 0.09)


@pytest.mark.parametrize("dtype,codes", STORES)
@pytest.mark.parametrize("n,heads,kvh,d", [(2, 2, 2, 64), (6, 8, 1, 128), (33, 32, 2, 128), (6, 4, 4, 128),
                                           (20, 9, 3, 64), (9, 6, 1, 128)])
def test_weights_keep_more_than_16_bits(dtype, codes, n, heads, kvh, d):
    """Scores that are exact and V rows that nearly cancel, so that what is
    left shows the weights' rounding and not the result's.
    A score is one fp32 rounding (of at most 5.5: 2^-22) and that of
    log2(e) (as much) off, an exponential 2^-22, the sums of up to 33 terms a
    few 2^-24: under 2^-19 of the mass together.  Of the weights' pair the
    second is rounded: below 2^-7 of the weight by 2^-8 of it in bf16, 2^-15;
    up to 1.5 2^-10 by 2^-11 in fp16, under 2^-20 (8 bits: 2^-22, and two
    roundings of 2^-24 that s_v adds)."""
    from window_helpers import attend64, half_step
    paged = Paged([n], kvh, d, 16, dtype, seed=n + d, codes=codes)
    t, block = torch.arange(n), torch.from_numpy(paged.tables[0]).long()
    at = (block[t // 16].cuda(), slice(None), (t % 16).cuda())
    row = torch.zeros((n, kvh, d), device="cuda")
    row[..., 0] = torch.randint(0, 16, (n, kvh), generator=paged.gen, device="cuda").float()
    unit = 1.0 if codes else 0.25
    paged.k[at] = (row * unit).to(paged.k.dtype)
    # signs that take turns, magnitudes alike
    v = (torch.arange(n, device="cuda") % 2 * 2.0 - 1.0)[:, None, None] * torch.randint(
        60, 65, (n, kvh, d), generator=paged.gen, device="cuda")
    paged.v[at] = (v if codes else v / 64).to(paged.v.dtype)
    if codes:
        paged.scales[..., 0] = 0.25
    q = torch.zeros((1, heads, d), dtype=dtype, device="cuda")
    q[0, :, 0] = (torch.arange(heads) % 8 + 1).cuda() / 8
    out = decode(paged, q, n, 0, 1.0)
    k64, v64 = paged.context64(0)
    ref, mass = attend64(q, k64, v64, [n - 1], n, 0, 1.0)
    pair = 2.0 ** -15 if dtype == BF16 and codes is None else 2.0 ** -20
    inner = (pair + 2.0 ** -19) * mass + n * 2.0 ** -32 * float(v64.abs().max())
    bound = inner + half_step(dtype) * (ref.abs() + inner) + torch.finfo(dtype).smallest_normal
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [0.0, 0.3])
@pytest.mark.parametrize("heads", [2, 6, 16, 64])
def test_infinite_values_that_are_seen_stay_infinite(dtype, size, heads):
    """One dim of V is infinite in one visible row: that dim of the result is
    that infinity (the weight is positive), the others are what they were.
    Equal scores (size 0) have weights of few bits, others of all."""
    paged = Paged([700, 33, 1], 2, 64, 16, dtype, seed=71)
    q = paged.randn((3, heads, 64)) * size
    want = decode(paged, q, 500, 4, 0.125)
    for b, t, dim, value in ((0, 2, 5, "inf"), (0, 650, 40, "-inf"), (1, 30, 0, "inf"), (2, 0, 63, "-inf")):
        paged.v[int(paged.tables[b, t // 16]), :, t % 16, dim] = float(value)
        want[b, :, dim] = float(value)
    assert torch.equal(decode(paged, q, 500, 4, 0.125), want)
