"""Multi-query window attention against the 64-bit form: masks, grouped heads,
ragged batches, stale rows and given-back blocks, refusals on the device,
streams and graphs."""
import pytest
import torch

from paged_kv_cache_481_b200 import binding
from window_helpers import Paged, attend64, attention_bound

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _prefill(paged, q, news, window, sinks, scale, stream=None, out=None, max_len=None, starts=None,
             max_new=None):
    tables, lens = paged.dev_tables()
    if starts is None:
        starts = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
    out = torch.full_like(q, 7.0) if out is None else out
    binding.pa_prefill_window(out, q, paged.k, paged.v, tables, lens,
                              max(paged.lens) if max_len is None else max_len, starts,
                              max(news) if max_new is None else max_new, window, sinks, scale,
                              stream=stream)
    return out


def _check(paged, q, out, news, window, sinks, scale, seqs=None):
    at = 0
    for b, n in enumerate(news):
        if n and (seqs is None or b in seqs):
            k, v = paged.context64(b)
            length = paged.lens[b]
            ref, mass = attend64(q[at:at + n], k, v, list(range(length - n, length)), window, sinks,
                                 scale)
            bound = attention_bound(ref, mass, q.dtype, q.dtype, float(v.abs().max()), length)
            err = (out[at:at + n].double() - ref).abs()
            assert bool((err <= bound).all()), (b, n, length, float((err / bound).max()))
        at += n
    assert bool((out[at:] == 7.0).all())       # rows of no sequence


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,news,heads,kvh,d,bs,window,sinks", [
    ([1], [1], 1, 1, 64, 8, 1, 0),
    ([17, 130, 5], [17, 3, 0], 4, 4, 128, 16, 16, 0),
    ([300, 1, 257], [300, 1, 129], 4, 2, 64, 32, 100, 5),
    ([513, 700, 64, 128], [200, 1, 64, 127], 7, 1, 128, 8, 130, 3),
    ([900, 40], [33, 40], 14, 2, 64, 16, 200, 130),
    ([1500], [700], 32, 8, 128, 16, 384, 4),
    ([1100, 300], [260, 300], 3, 3, 128, 128, 1, 1),
    ([600, 2], [5, 2], 128, 1, 128, 64, 257, 64),
    ([400, 333], [400, 100], 40, 2, 64, 16, 5000, 0),
    ([2048], [2048], 2, 2, 128, 16, 1000, 0),
    ([2048], [1000], 10, 2, 64, 32, 511, 700),
    ([1000, 190, 641], [300, 5, 64], 4, 2, 128, 16, 3, 200),
    ([1000, 640], [33, 200], 8, 1, 64, 32, 40, 400),
    ([900, 321], [260, 130], 1, 1, 64, 8, 65, 10),
    ([9] * 70, [k % 10 for k in range(70)], 2, 1, 128, 8, 4, 2),
])
def test_against_64_bits(dtype, lens, news, heads, kvh, d, bs, window, sinks):
    paged = Paged(lens, kvh, d, bs, dtype, seed=len(lens) * 11 + d)
    q = paged.randn((sum(news) + 3, heads, d))
    out = _prefill(paged, q, news, window, sinks, d ** -0.5)
    torch.cuda.synchronize()
    assert binding.pa_get_last_device_error() == 0
    _check(paged, q, out, news, window, sinks, d ** -0.5)


def test_many_items_of_uneven_length():
    """More items than the GPU holds blocks of threads; the same bits twice."""
    lens = [37 * (b % 13) + 1 + 400 * (b % 3) for b in range(90)]
    news = [min(n, 1 + 29 * (b % 11)) for b, n in enumerate(lens)]
    paged = Paged(lens, 4, 64, 16, BF16, seed=77)
    q = paged.randn((sum(news), 8, 64))
    out = _prefill(paged, q, news, 300, 4, 0.125)
    _check(paged, q, out, news, 300, 4, 0.125)
    assert torch.equal(_prefill(paged, q, news, 300, 4, 0.125), out)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_blocks_that_no_query_sees_are_not_looked_at(dtype):
    lens, news, bs, window, sinks = [700, 300, 500], [20, 150, 1], 16, 90, 3
    paged = Paged(lens, 2, 128, bs, dtype, seed=5)
    q = paged.randn((sum(news), 4, 128))
    want = _prefill(paged, q, news, window, sinks, 0.1)
    _check(paged, q, want, news, window, sinks, 0.1)
    for b, (n, new) in enumerate(zip(lens, news)):
        # K rows may hold anything where the mask hides them; V rows where no
        # query less than 256 positions away sees them
        for t in range(sinks, n - new - window + 1):
            block = int(paged.tables[b, t // bs])
            paged.k[block, :, t % bs] = float("nan")
            paged.v[block, :, t % bs] = float("inf")
        for j in range(-(-sinks // bs), max(0, n - new - window + 1) // bs):
            paged.tables[b, j] = [-1, 2 ** 30, -7][j % 3]
    assert torch.equal(_prefill(paged, q, news, window, sinks, 0.1), want)
    assert binding.pa_get_last_device_error() == 0


def test_scores_that_grow_along_the_context():
    """Each later K row scores far higher than all before: the reference of
    the softmax moves again and again."""
    paged = Paged([1500], 1, 64, 16, F16, seed=31)
    for t in range(1500):
        block = int(paged.tables[0, t // 16])
        paged.k[block, 0, t % 16] = 0
        paged.k[block, 0, t % 16, 0] = t / 8.0
    q = torch.zeros((600, 2, 64), dtype=F16, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    out = _prefill(paged, q, [600], 1000, 7, 1.0)
    k, v = paged.context64(0)
    ref, mass = attend64(q, k, v, list(range(900, 1500)), 1000, 7, 1.0)
    # scores are exact here; c s - m is one rounding of up to 2^9, 2^-15
    bound = attention_bound(ref, mass, F16, F16, float(v.abs().max()), 1500) + 2.0 ** -14 * mass
    assert bool(((out.double() - ref).abs() <= bound).all())


def test_wrong_arguments_are_recorded_and_skipped():
    paged = Paged([50, 20, 30], 1, 64, 8, F16, seed=3, junk=0.0)
    q = paged.randn((60, 2, 64))
    binding.pa_get_last_device_error()
    for starts, skipped in (([0, 10, 40, 45], [1]), ([-5, 10, 20, 25], [0]), ([0, 10, 20, 80], [2])):
        at = torch.tensor(starts, dtype=torch.int32).cuda()
        out = _prefill(paged, q, [1], 100, 0, 0.1, starts=at, max_new=30)
        assert binding.pa_get_last_device_error() == binding.PA_DEVERR_CONTEXT_LEN
        for b in range(3):
            lo, hi = max(0, starts[b]), min(60, starts[b + 1])
            if b in skipped:
                assert bool((out[lo:hi] == 7.0).all())
            else:
                k, v = paged.context64(b)
                n = hi - lo
                ref, mass = attend64(q[lo:hi], k, v, range(paged.lens[b] - n, paged.lens[b]), 100, 0,
                                     0.1)
                bound = attention_bound(ref, mass, F16, F16)
                assert bool(((out[lo:hi].double() - ref).abs() <= bound + 1e-6).all())
    _prefill(paged, q, [4, 4, 4], 100, 0, 0.1, max_len=40)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_CONTEXT_LEN
    paged.tables[1, 1] = paged.nb
    _prefill(paged, q, [4, 4, 4], 100, 0, 0.1)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_BLOCK_ID


def test_streams_and_graphs():
    paged = Paged([900, 40, 333], 2, 128, 16, BF16, seed=41)
    news = [500, 40, 7]
    q = paged.randn((sum(news), 8, 128))
    want = _prefill(paged, q, news, 256, 4, 0.1)
    tables, lens = paged.dev_tables()
    starts = torch.tensor([0, 500, 540, 547], dtype=torch.int32).cuda()
    outs = [torch.zeros_like(q) for _ in range(4)]
    call = lambda o: binding.pa_prefill_window(o, q, paged.k, paged.v, tables, lens, 900, starts, 500,
                                               256, 4, 0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, o in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(4):
                call(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
        call(outs[3])
    graph.replay()
    graph.replay()
    for o in outs:
        assert torch.equal(o, want)


def test_whole_context_agrees_with_pa_prefill():
    paged = Paged([700, 130], 4, 128, 16, F16, seed=8)
    news = [300, 130]
    q = paged.randn((430, 4, 128))
    out, old = _prefill(paged, q, news, 700, 0, 0.1), torch.full_like(q, 7.0)
    tables, lens = paged.dev_tables()
    binding.pa_prefill(old, q, paged.k, paged.v, tables, lens, 700,
                       torch.tensor([0, 300, 430], dtype=torch.int32).cuda(), 300, 0.1)
    _check(paged, q, out, news, 700, 0, 0.1)
    # pa_prefill's weights are fp16 at the softmax's own size
    ref, mass = attend64(q[300:], *paged.context64(1), list(range(130)), 700, 0, 0.1)
    bound = attention_bound(ref, mass, F16, F16) + 130 * 2.0 ** -24 * 8
    assert bool(((old[300:].double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(40, 0), (70, 5)])
def test_hidden_rows_of_the_largest_magnitude_have_no_effect(dtype, window, sinks):
    """Each position is hidden from some query of the same tile that its
    neighbours see; with V = +-max there, any weight but zero would show."""
    length, n, big = 300, 200, torch.finfo(dtype).max
    paged = Paged([length], 1, 64, 16, dtype, seed=17)
    q = paged.randn((n, 2, 64))
    pos = torch.arange(length - n, length)
    for at in (length - 1, 101, 110, 150, 175):   # seen by queries at .. at + window - 1 only
        block, row = int(paged.tables[0, at // 16]), at % 16
        keep = paged.k[block, 0, row].clone(), paged.v[block, 0, row].clone()
        paged.k[block, 0, row], paged.v[block, 0, row] = 0, big
        out = _prefill(paged, q, [n], window, sinks, 0.125)
        hidden = ~((at <= pos) & ((at > pos - window) | (at < sinks)))
        k, v = paged.context64(0)
        v = v.clone()
        v[at] = 0                              # whatever it is, where it is hidden
        ref, mass = attend64(q, k, v, pos.tolist(), window, sinks, 0.125)
        bound = attention_bound(ref, mass, dtype, dtype, float(v.abs().max()), length)
        assert bool(((out.double() - ref).abs() <= bound)[hidden.cuda()].all())
        paged.k[block, 0, row], paged.v[block, 0, row] = keep


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,block_size", [(64, 8), (128, 32)])
def test_scores_that_jump_far_past_the_reference(dtype, d, block_size):
    """Single tokens score hundreds above all before them, first, last and in
    the middle of a step: against the reference as it stood, their weights are
    past the type's range, and those that count are written over them."""
    length, n, group = 700, 300, 4
    paged = Paged([length], 2, d, block_size, dtype, seed=23)
    for t in range(length):
        paged.k[int(paged.tables[0, t // block_size]), :, t % block_size] = 0
    for i, t in enumerate((256, 383, 389, 448, 511, 540, 639, 640, 671, 690, 699)):
        paged.k[int(paged.tables[0, t // block_size]), :, t % block_size, 0] = 200.0 * (i + 1)
    q = torch.zeros((n, 2 * group, d), dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.5, 0.25, 0.0], device="cuda").repeat(2).to(dtype)
    out = _prefill(paged, q, [n], 600, 3, 1.0)
    assert binding.pa_get_last_device_error() == 0
    k, v = paged.context64(0)
    ref, mass = attend64(q, k, v, list(range(length - n, length)), 600, 3, 1.0)
    # scores are exact; tokens of one score share the rounding of c s - m, and
    # those of a lower one are 50 and more below it, so their weights vanish
    bound = attention_bound(ref, mass, dtype, dtype, float(v.abs().max()), length)
    assert bool(((out.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,kvh", [(2, 2), (8, 2), (7, 1)])
@pytest.mark.parametrize("window,sinks,at", [(300, 0, 700), (40, 5, 901), (900, 0, 600),
                                             (90, 901, 900), (500, 3, 1023)])
def test_how_far_a_row_that_is_not_finite_reaches(dtype, heads, kvh, window, sinks, at):
    """V at position `at` is infinite.  Queries that see it get no finite
    value; those 256 positions and more away from all of them get what they
    would without it."""
    length, n = 2000, 1700
    paged = Paged([length], kvh, 64, 16, dtype, seed=37)
    paged.v[int(paged.tables[0, at // 16]), :, at % 16] = float("inf")
    q = paged.randn((n, heads, 64))
    out = _prefill(paged, q, [n], window, sinks, 0.125)
    pos = torch.arange(length - n, length)
    sees = (at <= pos) & ((at > pos - window) | (at < sinks))
    far = ((pos[:, None] - pos[sees][None]).abs() >= 256).all(1)
    assert bool(sees.any()) and bool(far.any())
    assert not bool(out[sees.cuda()].isfinite().any())
    k, v = paged.context64(0)
    v = v.clone()
    v[at] = 0                                  # hidden from all queries looked at
    ref, mass = attend64(q, k, v, pos.tolist(), window, sinks, 0.125)
    bound = attention_bound(ref, mass, dtype, dtype, float(v.abs().max()), length)
    assert bool(((out.double() - ref).abs() <= bound)[far.cuda()].all())


@pytest.mark.parametrize("lens,news,heads,kvh,d", [([1, 700, 300], [1, 260, 300], 8, 2, 128),
                                                   ([3000], [40], 5, 5, 64)])
def test_values_as_large_as_the_type_holds(lens, news, heads, kvh, d):
    """bf16 values of half the type's largest, with one sign or both: their
    weighted mean is representable, and no sum on the way may leave fp32."""
    paged = Paged(lens, kvh, d, 16, BF16, seed=51)
    nan, sign = paged.v.isnan(), torch.sign(paged.v.float())
    for signs in (sign.abs(), sign):
        v = torch.rand(paged.v.shape, generator=paged.gen, device="cuda") + 1.0          # [1, 2]
        paged.v = (v * signs * (torch.finfo(BF16).max / 4)).to(BF16).masked_fill(nan, float("nan"))
        q = paged.randn((sum(news), heads, d)) * 2
        out = _prefill(paged, q, news, 2500, 3, d ** -0.5)
        assert binding.pa_get_last_device_error() == 0
        _check(paged, q, out, news, 2500, 3, d ** -0.5)


def test_starts_that_step_back_are_recorded():
    """query_start_loc that decreases: its sequence has no rows (and others
    may have the same ones twice), which the error word says."""
    paged = Paged([50, 50, 50], 1, 64, 8, F16, seed=3, junk=0.0)
    q = paged.randn((30, 2, 64))
    binding.pa_get_last_device_error()
    at = torch.tensor([0, 20, 15, 30], dtype=torch.int32).cuda()
    out = _prefill(paged, q, [1], 100, 0, 0.1, starts=at, max_new=30)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_CONTEXT_LEN
    k, v = paged.context64(2)
    ref, mass = attend64(q[20:], k, v, range(40, 50), 100, 0, 0.1)
    bound = attention_bound(ref, mass, F16, F16, float(v.abs().max()), 50)
    assert bool(((out[20:].double() - ref).abs() <= bound).all())
