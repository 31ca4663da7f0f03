"""The rotating cache writes against their 64-bit form: both rotations, both
16-bit types, strided and padded rows, neighbours left alone, and the 8-bit
cache's scales as its blocks fill up."""
import math

import pytest
import torch

from paged_kv_cache_481_b200 import binding
from window_helpers import CODES, rope_bound, rope_table, rotate64

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _slots(n, nb, bs, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(nb * bs, generator=gen)[:n].cuda()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,kvh,d,bs,rotary", [
    (1, 1, 1, 64, 8, 64), (5, 4, 4, 128, 16, 128), (37, 7, 1, 128, 32, 16), (300, 10, 2, 64, 64, 32),
    (19, 72, 72, 128, 128, 64), (3, 4, 2, 128, 16, 0), (64, 32, 8, 128, 16, 96),
])
def test_rotates_and_writes(dtype, interleaved, n, heads, kvh, d, bs, rotary):
    nb = -(-n // bs) + 2
    q, k, v = (_rand((n, h, d), dtype, s) for s, h in ((1, heads), (2, kvh), (3, kvh)))
    kc, vc = (_rand((nb, kvh, bs, d), dtype, s) for s in (4, 5))
    kc0, vc0 = kc.clone(), vc.clone()
    slots = _slots(n, nb, bs, 6)
    slots[n // 2] = -1
    table = rope_table(5000, rotary) if rotary else None
    gen = torch.Generator().manual_seed(7)
    pos = torch.randint(0, 5000, (n,), generator=gen).cuda()
    q_out = torch.full_like(q, 3.0)
    binding.pa_rope_and_cache(q_out, q, k, v, kc, vc, table, pos if rotary else None, slots,
                              interleaved=interleaved)
    assert binding.pa_get_last_device_error() == 0
    live = slots >= 0
    assert bool((q_out[~live] == 3.0).all())
    for x, got in ((q, q_out[live]), (k, kc[slots[live] // bs, :, slots[live] % bs])):
        ref, mag = rotate64(x[live], table, pos[live], interleaved)
        bound = rope_bound(ref, mag, dtype)
        assert bool(((got.double() - ref).abs() <= bound).all())
        # dims that are not rotated are copied
        assert torch.equal(got[..., rotary:], x[live][..., rotary:])
    assert torch.equal(vc[slots[live] // bs, :, slots[live] % bs], v[live])
    kc[slots[live] // bs, :, slots[live] % bs] = kc0[slots[live] // bs, :, slots[live] % bs]
    vc[slots[live] // bs, :, slots[live] % bs] = vc0[slots[live] // bs, :, slots[live] % bs]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)   # no other row was touched


def test_slices_of_one_projection_and_q_in_place():
    n, heads, kvh, d, bs = 45, 8, 2, 128, 16
    qkv = _rand((n, heads + 2 * kvh, d), BF16, 11)
    plain = [t.contiguous() for t in qkv.split([heads, kvh, kvh], 1)]
    table, pos, slots = rope_table(100, d), torch.arange(n).cuda(), _slots(n, 5, bs, 12)
    caches = [torch.zeros((5, kvh, bs, d), dtype=BF16, device="cuda") for _ in range(4)]
    q_out = torch.empty_like(plain[0])
    binding.pa_rope_and_cache(q_out, *plain, *caches[:2], table, pos, slots)
    keep = qkv[:, heads:].clone()
    q, k, v = qkv.split([heads, kvh, kvh], 1)
    binding.pa_rope_and_cache(q, q, k, v, *caches[2:], table, pos, slots)
    assert torch.equal(q, q_out) and torch.equal(qkv[:, heads:], keep)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("eight", [False, True])
def test_bad_slots_and_positions_are_recorded_and_skipped(eight):
    n, kvh, d, bs, nb = 6, 2, 64, 8, 2
    q, k, v = (_rand((n, kvh, d), F16, s) for s in (1, 2, 3))
    table = rope_table(10, d)
    pos = torch.tensor([0, 1, 10, 3, -1, 5]).cuda()
    slots = torch.tensor([0, 1, -1, nb * bs, -1, 5]).cuda()
    if eight:
        kc, vc = (torch.zeros((nb, kvh, bs, d), dtype=torch.int8, device="cuda") for _ in "kv")
        scales = torch.zeros((nb, kvh, 2), device="cuda")
        args, call = (kc, vc, scales), binding.pa_rope_and_cache_q8
    else:
        kc, vc = (torch.zeros((nb, kvh, bs, d), dtype=F16, device="cuda") for _ in "kv")
        args, call = (kc, vc), binding.pa_rope_and_cache
    q_out = torch.full_like(q, 3.0)
    binding.pa_get_last_device_error()
    call(q_out, q, k, v, *args, table, pos, slots)   # padding's position is not looked at
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_SLOT
    assert bool((q_out[[2, 3, 4]] == 3.0).all())
    slots = torch.tensor([-1, -1, 9, -1, 8, -1]).cuda()
    call(q_out, q, k, v, *args, table, pos, slots)
    assert binding.pa_get_last_device_error() == binding.PA_DEVERR_POSITION
    assert bool((q_out[[2, 4]] == 3.0).all())


# ------------------------------------------------------------ 8-bit cache
def _check_q8(codes, scales, which, want, mag, top, kind, first_rows=None):
    """Codes of one block's rows [r, KVH, D] against the 64-bit rows they
    stand for.  int8: off by half a scale; e4m3: half a step of 2^-3 relative
    (2^-4), or of the subnormal step 2^-9.  The quotient and the scale add
    fp32 roundings, 2^-22 of the value together."""
    s = scales.double()[None, :, None]
    got = codes.float().double() * s
    if kind == "int8":
        bound = s / 2
    else:
        bound = torch.maximum(2.0 ** -4 * want.abs(), s * 2.0 ** -10)
    bound = bound * (1 + 2.0 ** -20) + 2.0 ** -20 * want.abs() + 4 * 2.0 ** -24 * mag
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,kvh,d,bs,rotary,interleaved", [
    (4, 4, 128, 16, 128, False), (6, 3, 64, 8, 32, True), (8, 1, 128, 32, 64, False),
    (2, 2, 64, 128, 16, False),
])
def test_quantized_blocks_fill_up(kind, dtype, heads, kvh, d, bs, rotary, interleaved):
    """Steps of 1, a few and many tokens of two sequences into the same
    blocks.  A block's scale is max |x| ever held over top; what was written
    before is off by one more half step each time the scale grew."""
    code_type, top = CODES[kind]
    steps = [1, 2, 1, bs // 2, 1, bs + 3, 2 * bs, 1, 5]
    nb = 2 * -(-sum(steps) // bs) + 1
    kc, vc = (torch.full((nb, kvh, bs, d), 9.0, device="cuda").to(code_type) for _ in "kv")
    scales = torch.full((nb, kvh + kvh % 2, 2), 50.0, device="cuda")   # a former owner's
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(3))
    table = rope_table(2000, rotary)
    held = {}            # block -> list of (row64 K, V [KVH, D], mag, times rounded)
    lens = [0, 0]
    for i, n in enumerate(steps):
        rows, pos, slots = 2 * n, [], []
        for b in range(2):
            for t in range(lens[b], lens[b] + n):
                pos.append(t)
                slots.append(int(ids[b * (nb // 2) + t // bs]) * bs + t % bs)
            lens[b] += n
        # magnitudes that grow and shrink from step to step
        x = [_rand((rows, h, d), dtype, 100 + 3 * i + j, 1.7 ** ((i * 5) % 7 - 2))
             for j, h in enumerate((heads, kvh, kvh))]
        pos, slots = torch.tensor(pos).cuda(), torch.tensor(slots).cuda()
        q_out = torch.empty_like(x[0])
        before = scales.clone()
        binding.pa_rope_and_cache_q8(q_out, *x, kc, vc, scales, table, pos, slots,
                                     interleaved=interleaved)
        assert binding.pa_get_last_device_error() == 0
        ref, mag = rotate64(x[0], table, pos, interleaved)
        assert bool(((q_out.double() - ref).abs() <= rope_bound(ref, mag, dtype)).all())
        k64, kmag = rotate64(x[1], table, pos, interleaved)
        v64 = x[2].double()
        blocks = (slots // bs).tolist()
        for block in sorted(set(blocks)):
            mine = [j for j, o in enumerate(blocks) if o == block]
            fresh = int(slots[mine[0]] % bs) == 0
            if fresh:
                held[block] = []
            for which, rows64, m64, codes in ((0, k64, kmag, kc), (1, v64, v64.abs(), vc)):
                m = rows64[mine].abs().amax((0, 2))
                slack = 4 * 2.0 ** -24 * m64[mine].amax((0, 2)) / top
                want = m / top
                if not fresh:
                    want = torch.maximum(want, before[block, :kvh, which].double())
                got = scales[block, :kvh, which].double()
                assert bool(((got - want).abs() <= slack + 2.0 ** -23 * want).all())
                new = codes[block, :, [int(slots[j] % bs) for j in mine]].transpose(0, 1)
                _check_q8(new, scales[block, :kvh, which], which, rows64[mine], m64[mine], top,
                          kind)
                old = [r[which] for r in held[block]] if which < 2 else None
                if old:
                    was = torch.stack(old)                      # [r, KVH, D] values before
                    got_rows = codes[block, :, :len(old)].transpose(0, 1)
                    grew = got > before[block, :kvh, which].double()
                    exact = got_rows.float().double() * got[None, :, None]
                    assert bool((exact == was)[:, ~grew].all())
                    _check_q8(got_rows, scales[block, :kvh, which], which, was,
                              torch.zeros_like(was), top, kind)
            now = [(kc[block, :, r].float().double() * scales[block, :kvh, 0, None].double(),
                    vc[block, :, r].float().double() * scales[block, :kvh, 1, None].double())
                   for r in range(int(slots[mine[-1]] % bs) + 1)]
            held[block] = now


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_zero_rows_and_stale_scales(kind):
    code_type, top = CODES[kind]
    kvh, d, bs = 2, 64, 8
    kc, vc = (torch.full((2, kvh, bs, d), 5.0, device="cuda").to(code_type) for _ in "kv")
    scales = torch.full((2, kvh, 2), 1e6, device="cuda")
    x = torch.zeros((3, kvh, d), dtype=F16, device="cuda")
    call = lambda x, slots: binding.pa_rope_and_cache_q8(
        torch.empty_like(x), x, x, x, kc, vc, scales, None, None,
        torch.tensor(slots, device="cuda"))
    call(x, [8, 9, 10])
    assert bool((scales[1] == 0).all()) and bool((kc[1, :, :3].float() == 0).all())
    assert bool((scales[0] == 1e6).all()) and bool((kc[1, :, 3:].float() == 5).all())
    x1 = torch.full((1, kvh, d), 2.0, dtype=F16, device="cuda")
    call(x1, [11])                                # the first row that is not zero sets the scale
    assert torch.equal(scales[1], torch.full_like(scales[1], 2.0) / top)
    assert bool((kc[1, :, :3].float() == 0).all()) and bool((vc[1, :, 3].float() == top).all())


def test_many_tokens_of_one_call_and_a_replayed_graph():
    """A call over the size at which a CTA looks after several runs, captured
    and replayed: the same codes and scales as token by token of each block."""
    kvh, d, bs, n = 3, 128, 16, 1777
    nb = -(-n // bs)
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(5))
    slots = torch.cat([order[t // bs, None] * bs + t % bs for t in range(n)]).cuda()
    pos = torch.arange(n).cuda()
    x = _rand((n, kvh, d), BF16, 21)
    table = rope_table(n, d)
    made = []
    for captured in (False, True):
        kc, vc = (torch.zeros((nb, kvh, bs, d), dtype=torch.int8, device="cuda") for _ in "kv")
        scales = torch.zeros((nb, kvh + 1, 2), device="cuda")
        q_out = torch.empty_like(x)
        call = lambda: binding.pa_rope_and_cache_q8(q_out, x, x, x, kc, vc, scales, table, pos,
                                                    slots)
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
            graph.replay()
        else:
            call()
        torch.cuda.synchronize()
        made.append((kc, vc, scales, q_out))
    for a, b in zip(*made):
        assert torch.equal(a, b)
    ref, mag = rotate64(x, table, pos, False)
    kc, _, scales, _ = made[0]
    got = kc[slots // bs, :, slots % bs].double() * scales[slots // bs, :kvh, 0, None].double()
    s = scales[slots // bs, :kvh, 0, None].double()
    bound = s / 2 * (1 + 2.0 ** -20) + 2.0 ** -20 * ref.abs() + 4 * 2.0 ** -24 * mag
    assert bool(((got - ref).abs() <= bound).all())
    assert bool((scales[:, kvh] == 0).all())      # the padding head's scales are not written


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_codes_of_extreme_magnitudes(kind):
    """Rows near both ends of bf16's range: the quotient by the scale neither
    overflows nor loses its last bits."""
    code_type, top = CODES[kind]
    kvh, d, bs = 1, 64, 8
    base = _rand((4, kvh, d), torch.float32, 31)
    for factor in (2.0 ** 120, 2.0 ** 100, 1.0, 2.0 ** -100, 2.0 ** -117):
        x = (base * factor).to(BF16)
        kc, vc = (torch.zeros((1, kvh, bs, d), device="cuda").to(code_type) for _ in "kv")
        scales = torch.zeros((1, 2, 2), device="cuda")
        slots = torch.arange(4, device="cuda")
        binding.pa_rope_and_cache_q8(torch.empty_like(x), x, x, x, kc, vc, scales, None, None, slots)
        m = x.double().abs().amax()
        want = x.double() * top / m                 # in codes
        got = kc[0, 0, :4].float().double()
        step = torch.full_like(want, 0.5) if kind == "int8" else torch.maximum(
            2.0 ** -4 * want.abs(), torch.full_like(want, 2.0 ** -10))
        assert bool(((got - want[:, 0]).abs() <= step[:, 0] * (1 + 2.0 ** -20)).all())
        # the scale is m / top rounded once (subnormal ones to 2^-149)
        assert abs(float(scales[0, 0, 0].double() - m / top)) <= max(2.0 ** -24 * float(m / top),
                                                                     2.0 ** -150)


def test_ties_follow_the_exact_quotient():
    """bf16 values whose x top / m lies exactly between two e4m3 numbers go to
    the even one, though the scale itself is rounded."""
    d, top = 64, 448.0
    x = torch.zeros((1, 1, d), dtype=BF16, device="cuda")
    x[0, 0, 0] = 7.0 * 1.375                        # m: s = m / 448 is not a power of two
    m = float(x[0, 0, 0])
    want = []
    for i in range(1, d):
        # v 448 / m = 17/16 * 2^k or 19/16 * 2^k: between neighbours of step 1/8
        v = (17.0 if i % 2 else 19.0) / 16.0 * 2.0 ** (i % 5) * m / 448.0
        x[0, 0, i] = v
        got = float(x[0, 0, i]) * 448.0 / m
        want.append(got)
    kc, vc = (torch.zeros((1, 1, 8, d), device="cuda").to(torch.float8_e4m3fn) for _ in "kv")
    scales = torch.zeros((1, 2, 2), device="cuda")
    binding.pa_rope_and_cache_q8(torch.empty_like(x), x, x, x, kc, vc, scales, None, None,
                                 torch.zeros(1, dtype=torch.int64, device="cuda"))
    exact = torch.tensor(want, dtype=torch.float64).float().to(torch.float8_e4m3fn).float()
    assert torch.equal(vc[0, 0, 0, 1:].float().cpu(), exact)


def test_tensors_of_another_device_or_layout_are_refused():
    x = _rand((2, 1, 64), F16, 1)
    kc, vc = (torch.zeros((1, 1, 8, 64), dtype=F16, device="cuda") for _ in "kv")
    slots = torch.tensor([0, 1], device="cuda")
    call = lambda *a: binding.pa_rope_and_cache(*a, None, None, slots)
    with pytest.raises(ValueError):
        call(x, x.cpu(), x, x, kc, vc)
    with pytest.raises(ValueError):
        call(x, x, x, x, kc.cpu(), vc)
    with pytest.raises(ValueError):      # heads that do not lie side by side
        wide = _rand((2, 2, 64), F16, 1)[:, :, :].transpose(0, 1)
        binding.pa_rope_and_cache(wide.contiguous(), wide, x, x, kc, vc, None, None, slots)
    with pytest.raises(AssertionError):
        call(x, x, x.to(BF16), x, kc, vc)
    with pytest.raises(binding.PAError):  # a token stride that is not a multiple of 8
        odd = torch.zeros((2, 68), dtype=F16, device="cuda")[:, :64].unsqueeze(1)
        call(odd, odd, x, x, kc, vc)


@pytest.mark.parametrize("kind,nb", [("int8", 70001), ("e4m3", 70001), ("int8", 300001)])
def test_blocks_that_a_call_comes_back_to_are_recorded(kind, nb):
    """The 8-bit write takes a block's tokens side by side: interleaved
    sequences and slots given twice set the error bit, wherever in the pool
    they are; runs in any order, split by padding between blocks, do not."""
    kvh, d, bs = 1, 64, 8
    kc, vc = (torch.zeros((nb, kvh, bs, d), device="cuda").to(CODES[kind][0]) for _ in "kv")
    scales = torch.zeros((nb, 2, 2), device="cuda")
    binding.pa_get_last_device_error()

    def recorded(slots):
        x = torch.ones((len(slots), kvh, d), dtype=F16, device="cuda")
        binding.pa_rope_and_cache_q8(torch.empty_like(x), x, x, x, kc, vc, scales, None, None,
                                     torch.tensor(slots, device="cuda"))
        return binding.pa_get_last_device_error()

    for base in (0, 3, 4094, 4095, 4096, 32767, 32768, 65534, 65535, 65536, nb - 3):
        a, b = base * bs, (base + 2) * bs
        assert recorded([a, a + 1, a + 2, b, b + 1]) == 0
        assert recorded([a, b, a + 1, b + 1]) == binding.PA_DEVERR_SLOT    # drafts of two sequences
        assert recorded([b, a, a]) == binding.PA_DEVERR_SLOT               # a slot twice
        assert recorded([a, -1, a + 1]) == binding.PA_DEVERR_SLOT          # padding inside a run
        assert recorded([a + 1, a]) == binding.PA_DEVERR_SLOT              # not in order
        assert recorded([a + 6, a + 7, b, -1, a + 8, a + 9, -1]) == 0      # the next block, padding
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(1))[:3000].tolist()
    runs = [list(range(b * bs + i % 8, b * bs + i % 8 + 1 + i % (8 - i % 8))) for i, b in enumerate(order)]
    assert recorded(sum(runs, [])) == 0
    runs.append([order[7] * bs + 7])            # far from the first run of its block
    assert recorded(sum(runs, [])) == binding.PA_DEVERR_SLOT
    # what was not touched twice holds its values
    codes, scale = kc[order[8:]].float(), scales[order[8:], 0, 0]
    first = torch.tensor([r[0] % bs for r in runs[8:-1]], device="cuda")
    got = codes[torch.arange(len(first), device="cuda"), 0, first, 0] * scale
    assert bool(((got - 1).abs() < 2.0 ** -20).all())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_scales_below_the_normal_numbers(kind):
    """Rotated keys so small that the scale itself is a few times 2^-149: a
    later row that does not raise the rounded scale still has codes of its own
    sign up to the top."""
    code_type, top = CODES[kind]
    d, bs = 64, 8
    kc, vc = (torch.zeros((1, 1, bs, d), device="cuda").to(code_type) for _ in "kv")
    scales = torch.zeros((1, 2, 2), device="cuda")
    # keys of 2^-133 (bf16's smallest) turned by a table whose cosines make them
    # `units` times 2^-149 and whose sines are zero
    units = [int(top * 0.8), int(top * 1.4), -int(top * 1.45), int(top * 0.5), -int(top * 1.49)]
    table = torch.zeros((len(units), d), device="cuda")
    table[:, :d // 2] = torch.tensor(units, device="cuda")[:, None].float() * 2.0 ** -16
    k = torch.full((1, 1, d), 2.0 ** -133, dtype=BF16, device="cuda")
    v = torch.ones((1, 1, d), dtype=BF16, device="cuda")
    for i, u in enumerate(units):
        binding.pa_rope_and_cache_q8(torch.empty_like(k), k, k, v, kc, vc, scales, table,
                                     torch.tensor([i], device="cuda"), torch.tensor([i], device="cuda"))
        assert float(scales[0, 0, 0]) == 2.0 ** -149       # |units| / top rounds to 1
        want = max(-top, min(top, float(u)))
        step = 0.5 if kind == "int8" else 2.0 ** -4 * abs(want)
        got = kc[0, 0, i].float()
        if i > 0 and abs(u) <= top:
            assert bool(((got - want).abs() <= step).all())
        else:                  # x top / m (the scale is new, or would pass the top)
            assert bool((got == math.copysign(top, u)).all())
    assert bool((vc[0, 0, :len(units)].float() == top).all())
