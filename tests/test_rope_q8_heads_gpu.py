"""The 8-bit rotating write over many heads, where several blocks of threads
share a token, and over runs of all lengths: every code and scale of K and V
against the 64-bit rows, whatever the order in which blocks fill up."""
import pytest
import torch

from paged_kv_cache_481_b200 import binding
from window_helpers import CODES, rope_bound, rope_table, rotate64

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


class Cache:
    def __init__(self, nb, kvh, bs, d, kind, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.kvh, self.bs, self.nb, self.d = kind, kvh, bs, nb, d
        code_type, top = CODES[kind]
        x = [torch.randn((nb, kvh, bs, d), generator=self.gen, device="cuda") * (top / 4) for _ in "kv"]
        self.codes = [(t.round() if kind == "int8" else t).clamp(-top, top).to(code_type) for t in x]
        # a former owner's scales, and what a padding head's place holds
        self.scales = torch.rand((nb, kvh + kvh % 2, 2), generator=self.gen, device="cuda")

    def rows(self, n, heads, dtype, size=1.0):
        return (torch.randn((n, heads, self.d), generator=self.gen, device="cuda") * size).to(dtype)

    def write(self, x, table, pos, slots, interleaved=False):
        """One call, held against its definition."""
        before, old_scales = [c.clone() for c in self.codes], self.scales.clone()
        q_out = torch.full_like(x[0], 3.0)
        binding.pa_rope_and_cache_q8(q_out, *x, *self.codes, self.scales, table, pos, slots,
                                     interleaved=interleaved)
        assert binding.pa_get_last_device_error() == 0
        live = slots >= 0
        ref, mag = rotate64(x[0][live], table, pos[live], interleaved)
        assert bool(((q_out[live].double() - ref).abs() <= rope_bound(ref, mag, x[0].dtype)).all())
        assert bool((q_out[~live] == 3.0).all())
        k64, kmag = rotate64(x[1][live], table, pos[live], interleaved)
        v64 = x[2][live].double()
        block, row = slots[live] // self.bs, slots[live] % self.bs
        for which, rows64, m64 in ((0, k64, kmag), (1, v64, torch.zeros_like(v64))):
            self._check(which, before[which], old_scales[:, :, which].double(), rows64, m64, block, row)
        if self.kvh % 2:
            assert torch.equal(self.scales[:, self.kvh], old_scales[:, self.kvh])

    def _check(self, which, before, old, rows64, mag, block, row):
        """A new row is off by half a step: of the scale (int8), or 2^-4 of
        the value, 2^-10 of the scale for subnormal codes (e4m3).  fp32
        rotation adds 4 2^-24 of what it sums, the scale and the quotient 2^-22
        of the value, the scale's rounding 2^-24 of it.  An older row is off by
        half a step from what it was where the scale grew, else the same."""
        kvh, bs, top = self.kvh, self.bs, CODES[self.kind][1]
        old = old[:, :kvh]
        touched = torch.zeros(self.nb, dtype=torch.bool, device="cuda").index_fill_(0, block, True)
        first = torch.full((self.nb,), bs, device="cuda").scatter_reduce_(0, block, row, "amin")
        last = torch.full((self.nb,), -1, device="cuda").scatter_reduce_(0, block, row, "amax")
        index = block[:, None].expand(-1, kvh)
        want = torch.zeros((self.nb, kvh), dtype=torch.float64, device="cuda").scatter_reduce_(
            0, index, rows64.abs().amax(-1), "amax") / top
        slack = torch.zeros_like(want).scatter_reduce_(0, index, 4 * 2.0 ** -24 * mag.amax(-1), "amax") / top
        want = torch.where((first > 0)[:, None], torch.maximum(want, old), want)
        got = self.scales[:, :kvh, which].double()
        assert bool(((got - want).abs() <= slack + 2.0 ** -24 * want * (1 + 2.0 ** -20))[touched].all())
        assert bool((got == old)[~touched].all())

        def close(codes, values, s, extra):
            step = s / 2 if self.kind == "int8" else torch.maximum(2.0 ** -4 * values.abs(), s * 2.0 ** -10)
            bound = step * (1 + 2.0 ** -20) + 2.0 ** -21 * values.abs() + extra
            return bool(((codes.float().double() * s - values).abs() <= bound).all())

        codes = self.codes[which]
        assert close(codes[block, :, row], rows64, got[block][..., None], 4 * 2.0 ** -24 * mag)
        at = torch.arange(bs, device="cuda")[None]
        older = (touched[:, None] & (at < first[:, None]))[:, None, :].expand(-1, kvh, -1)
        grew = (got > old)[:, :, None]
        bits, was = codes.view(torch.uint8), before.view(torch.uint8)
        assert torch.equal(bits[older & ~grew], was[older & ~grew])
        moved = older & grew
        if bool(moved.any()):
            s0, s1 = (s[:, :, None].expand(-1, -1, bs)[moved][:, None] for s in (old, got))
            assert close(codes[moved], before[moved].float().double() * s0, s1, 0.0)
        others = ~touched[:, None] | (at > last[:, None])
        others = others[:, None, :].expand(-1, kvh, -1)
        assert torch.equal(bits[others], was[others])


def _runs(nb, bs, spans, seed):
    """Slots and positions of sequences whose new tokens are positions
    [start, start + n), each over blocks of its own."""
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).tolist()
    slots, pos = [], []
    for start, n in spans:
        blocks = [ids.pop() for _ in range((start + n - 1) // bs - start // bs + 1)]
        for t in range(start, start + n):
            slots.append(blocks[t // bs - start // bs] * bs + t % bs)
            pos.append(t)
    return slots, pos


SHAPES = [(40, 40, 128), (72, 72, 128), (64, 8, 128), (20, 10, 128), (34, 17, 128), (9, 9, 128),
          (33, 1, 128), (20, 20, 64), (72, 72, 64), (128, 1, 64), (17, 17, 64), (66, 33, 64)]


@pytest.mark.parametrize("heads,kvh,d", SHAPES)
@pytest.mark.parametrize("kind,dtype,bs", [("int8", F16, 16), ("e4m3", BF16, 64), ("int8", BF16, 128),
                                           ("e4m3", F16, 8)])
def test_many_heads_and_runs_of_all_lengths(heads, kvh, d, kind, dtype, bs):
    """Single tokens, a few, as many as a span's tokens and one more, and runs
    past the tokens that a block of threads looks ahead at; then single tokens
    behind them with larger and smaller rows."""
    spans = [(0, 1), (bs - 1, 1), (3, 2), (1, 7), (bs // 2, 8), (0, 9), (2, 15), (5, 17), (0, 25), (1, 30),
             (bs - 2, 70), (4, 2 * bs), (2 * bs - 3, 150), (7, 1)]
    nb = sum((s + n - 1) // bs - s // bs + 1 for s, n in spans) + 3
    rotary = d // 2 if kvh % 2 else d
    table = rope_table(4096, rotary)
    cache = Cache(nb, kvh, bs, d, kind, seed=heads + d)
    slots, pos = _runs(nb, bs, spans, seed=kvh)
    for at in (20, 5):                                   # padding between sequences
        cut = [i for i in range(1, len(pos)) if pos[i] != pos[i - 1] + 1][at % 7]
        slots, pos = slots[:cut] + [-1] + slots[cut:], pos[:cut] + [0] + pos[cut:]
    slots, pos = torch.tensor(slots).cuda(), torch.tensor(pos).cuda()
    n = len(pos)
    cache.write([cache.rows(n, h, dtype) for h in (heads, kvh, kvh)], table, pos, slots, interleaved=kvh % 3 == 0)
    # a decode step behind each sequence that has room in its last block
    ends = (pos[1:] != pos[:-1] + 1).nonzero()[:, 0].tolist() + [n - 1]
    ends = [i for i in ends if int(slots[i]) >= 0 and int(slots[i]) % bs != bs - 1]
    for size in (0.5, 3.0):
        at = slots[ends] + 1
        m = len(ends)
        cache.write([cache.rows(m, h, dtype, size) for h in (heads, kvh, kvh)], table, pos[ends] + 1, at,
                    interleaved=kvh % 3 == 0)
        ends = [i for i in ends if int(slots[i]) % bs < bs - 2]
        slots = slots + 1


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("kvh,d,bs", [(3, 128, 16), (12, 64, 32)])
def test_one_call_and_token_by_token(kind, kvh, d, bs):
    """A prompt in one call, in chunks and token by token: each call is held
    against its definition, and all end with the same scales, which the largest
    row of a block alone decides."""
    n, nb = 157, 12
    table = rope_table(n, d)
    slots, pos = (torch.tensor(t).cuda() for t in _runs(nb, bs, [(0, n)], seed=5))
    caches = [Cache(nb, kvh, bs, d, kind, seed=9) for _ in range(3)]
    x = [caches[0].rows(n, kvh, BF16) * (1 + torch.arange(n, device="cuda")[:, None, None] % 7) for _ in "qkv"]
    for cache, step in zip(caches, (n, 23, 1)):
        for i in range(0, n, step):
            part = slice(i, i + step)
            cache.write([t[part].contiguous() for t in x], table, pos[part], slots[part])
    used = slots.unique() // bs
    for cache in caches[1:]:
        assert torch.equal(cache.scales[used], caches[0].scales[used])


def test_a_long_packed_batch_replayed_from_a_graph():
    """7000 tokens of two K/V heads in one call: codes and scales of K and V,
    eager and from a graph."""
    kvh, d, bs = 2, 128, 16
    spans = [(17 * i % 300, 1 + 37 * i % 260) for i in range(54)]
    nb = sum((s + n - 1) // bs - s // bs + 1 for s, n in spans) + 1
    table = rope_table(1000, d)
    slots, pos = (torch.tensor(t).cuda() for t in _runs(nb, bs, spans, seed=1))
    made = []
    for captured in (False, True):
        cache = Cache(nb, kvh, bs, d, "int8", seed=3)
        x = [cache.rows(len(pos), h, BF16) for h in (4, kvh, kvh)]
        if not captured:
            cache.write(x, table, pos, slots)
        else:
            q_out = torch.empty_like(x[0])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                binding.pa_rope_and_cache_q8(q_out, *x, *cache.codes, cache.scales, table, pos, slots)
            graph.replay()
            torch.cuda.synchronize()
        made.append((*cache.codes, cache.scales))
    for a, b in zip(*made):
        assert torch.equal(a, b)
