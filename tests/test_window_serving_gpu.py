"""The window operators together, as a serving program runs them: prompts in
chunks, decode steps, a forked sequence, blocks that the window has left given
back, all addressed through the block manager; and caches beyond 4 GB."""
import numpy as np
import pytest
import torch

from paged_kv_cache_481_b200 import binding
from window_helpers import CODES, attend64, attention_bound, rope_table, rotate64

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


class Layer:
    """One attention layer's caches and the rows that went into them."""

    def __init__(self, nb, kvh, bs, d, dtype, codes):
        self.bs, self.kvh, self.d, self.dtype, self.codes = bs, kvh, d, dtype, codes
        kind = dtype if codes is None else CODES[codes][0]
        fill = float("nan") if kind.is_floating_point else 0.0
        self.k, self.v = (torch.full((nb, kvh, bs, d), fill, device="cuda").to(kind) for _ in "kv")
        self.scales = torch.full((nb, kvh + kvh % 2, 2), float("nan"), device="cuda")

    def write(self, q, k, v, table, pos, slots):
        out = torch.empty_like(q)
        if self.codes is None:
            binding.pa_rope_and_cache(out, q, k, v, self.k, self.v, table, pos, slots)
        else:
            binding.pa_rope_and_cache_q8(out, q, k, v, self.k, self.v, self.scales, table, pos, slots)
        return out

    def copy(self, pairs):
        pairs = torch.from_numpy(pairs).cuda()
        for cache in (self.k, self.v) + (() if self.codes is None else (self.scales,)):
            binding.pa_copy_blocks_raw(cache, pairs)

    def rows(self, table, n):
        """What the cache holds for positions 0 .. n - 1, in 64 bits."""
        t = torch.arange(n)
        block, row = torch.from_numpy(table).long()[t // self.bs].clamp(min=0).cuda(), (t % self.bs).cuda()
        k, v = (c[block, :, row].float().double() if self.codes else c[block, :, row].double()
                for c in (self.k, self.v))
        if self.codes:
            s = self.scales.double()[block, :self.kvh]
            k, v = k * s[..., :1], v * s[..., 1:]
        return k, v


@pytest.mark.parametrize("dtype,codes", [(BF16, None), (F16, None), (F16, "int8"), (BF16, "e4m3")])
def test_prompts_decode_steps_and_a_fork(dtype, codes):
    heads, kvh, d, bs, window, sinks = 8, 2, 128, 16, 150, 4
    scale = d ** -0.5
    nb, width = 200, 40
    manager = binding.BlockManager(nb, bs)
    layer = Layer(nb, kvh, bs, d, dtype, codes)
    table = rope_table(1000, d)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda n, h: torch.randn((n, h, d), generator=gen, device="cuda").to(dtype)
    ws = binding.new_window_workspace(8, heads, kvh, d)
    prompts = [333, 70, 1, 16]
    for s, n in enumerate(prompts):
        manager.add_sequence(s, n)
    history = {s: [] for s in range(len(prompts) + 1)}       # exact rotated K, V rows

    def check(out, q, seqs, tables, lens, news):
        at = 0
        weight = F16 if codes else dtype
        for i, (s, n) in enumerate(zip(seqs, news)):
            length = int(lens[i])
            k, v = layer.rows(tables[i], length)
            # blocks that were given back are not looked at
            gone = torch.arange(length, device="cuda")
            hidden = (gone < length - n - window + 1) & (gone >= sinks)
            k, v = k.masked_fill(hidden[:, None, None], 0), v.masked_fill(hidden[:, None, None], 0)
            ref, mass = attend64(q[at:at + n], k, v, list(range(length - n, length)), window, sinks, scale)
            bound = attention_bound(ref, mass, dtype, weight, float(v.abs().max()), length)
            assert bool(((out[at:at + n].double() - ref).abs() <= bound).all()), (s, length)
            at += n

    # prompts in two chunks each; the second continues the cached context
    for half in range(2):
        news = [(n + 1) // 2 if half == 0 else n // 2 for n in prompts]
        tables, _ = manager.block_tables(list(range(4)), width)
        starts = [0 if half == 0 else (n + 1) // 2 for n in prompts]
        pos = np.concatenate([np.arange(a, a + m) for a, m in zip(starts, news)])
        row = np.repeat(np.arange(4), news)
        slots = torch.from_numpy(tables[row, pos // bs].astype(np.int64) * bs + pos % bs).cuda()
        total = int(sum(news))
        q, k, v = rand(total, heads), rand(total, kvh), rand(total, kvh)
        turned = layer.write(q, k, v, table, torch.from_numpy(pos).cuda(), slots)
        k64, _ = rotate64(k, table, torch.from_numpy(pos).cuda(), False)
        for s in range(4):
            history[s] += list(zip(k64[row == s], v[row == s].double()))
        lens = np.array([a + m for a, m in zip(starts, news)], np.int32)
        if codes is None:
            out = torch.empty_like(turned)
            binding.pa_prefill_window(out, turned, layer.k, layer.v, torch.from_numpy(tables).cuda(),
                                      torch.from_numpy(lens).cuda(), int(lens.max()),
                                      torch.tensor([0, *np.cumsum(news)], dtype=torch.int32).cuda(),
                                      max(news), window, sinks, scale)
            check(out, turned, range(4), tables, lens, news)

    seqs = [0, 1, 2, 3]
    for step in range(40):
        if step == 5:
            manager.fork(1, 4)                 # shares its blocks until it writes
            history[4] = list(history[1])
            seqs.append(4)
        slots, pairs = manager.append_slots(seqs)
        if len(pairs):
            layer.copy(pairs)
        tables, lens = manager.block_tables(seqs, width)
        b = len(seqs)
        pos = torch.from_numpy((lens - 1).astype(np.int64)).cuda()
        q, k, v = rand(b, heads), rand(b, kvh), rand(b, kvh)
        turned = layer.write(q, k, v, table, pos, torch.from_numpy(slots).cuda())
        k64, _ = rotate64(k, table, pos, False)
        for i, s in enumerate(seqs):
            history[s].append((k64[i], v[i].double()))
        for i, n in enumerate(lens):           # entries the window has left
            tables[i, -(-sinks // bs):max(0, int(n) - window) // bs] = -1
        out = torch.empty_like(turned)
        args = (torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), int(lens.max()), window,
                sinks, scale, ws)
        if codes is None:
            binding.pa_decode_window(out, turned, layer.k, layer.v, *args)
        else:
            binding.pa_decode_q8(out, turned, layer.k, layer.v, layer.scales, *args)
        if step % 6 == 5 or step == 39:
            check(out, turned, seqs, tables, lens, [1] * b)
    assert binding.pa_get_last_device_error() == 0
    # the caches hold the rows that went in: 16-bit rows rounded once, 8-bit
    # rows off by at most half a step for the scale they were written with and
    # each one it grew to afterwards (bs - 1 at most)
    tables, lens = manager.block_tables(seqs, width)
    for i, s in enumerate(seqs):
        k, v = layer.rows(tables[i], int(lens[i]))
        for got, j in ((k, 0), (v, 1)):
            want = torch.stack([r[j] for r in history[s]])
            if codes is None:
                tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -20
            else:
                block = torch.from_numpy(tables[i]).long()[torch.arange(int(lens[i])) // bs].cuda()
                step_size = layer.scales.double()[block, :kvh, j][..., None]
                one = step_size / 2 if codes == "int8" else torch.maximum(2.0 ** -4 * want.abs() * 1.2,
                                                                        step_size * 2.0 ** -10)
                tol = one * bs + 2.0 ** -20
            assert bool(((got - want).abs() <= tol).all())


@pytest.mark.slow
@pytest.mark.parametrize("codes", [None, "int8"])
def test_blocks_beyond_four_gigabytes(codes):
    """Blocks whose rows lie past 2^32 bytes (and 2^31 elements) of a cache."""
    kvh, d, bs, heads = 8, 128, 16, 16
    item = 1 if codes else 2
    nb = (1 << 32) // (kvh * bs * d * item) + 200
    layer = Layer.__new__(Layer)
    layer.bs, layer.kvh, layer.d, layer.dtype, layer.codes = bs, kvh, d, BF16, codes
    kind = torch.int8 if codes else BF16
    layer.k, layer.v = (torch.zeros((nb, kvh, bs, d), dtype=kind, device="cuda") for _ in "kv")
    layer.scales = torch.zeros((nb, kvh, 2), device="cuda")
    length, n = 1500, 150
    tables = (nb - 1 - torch.randperm(150, generator=torch.Generator().manual_seed(1))[:94]).to(
        torch.int32)[None]
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda m, h: torch.randn((m, h, d), generator=gen, device="cuda").to(BF16)
    pos = torch.arange(length)
    slots = (tables[0].long()[pos // bs] * bs + pos % bs).cuda()
    table = rope_table(length, d)
    turned = layer.write(rand(length, heads), rand(length, kvh), rand(length, kvh), table, pos.cuda(), slots)
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    k, v = layer.rows(tables[0].numpy(), length)
    assert float(k.abs().max()) > 1
    q, out = turned[-1:].contiguous(), torch.empty_like(turned[-1:])
    ws = binding.new_window_workspace(1, heads, kvh, d)
    if codes:
        binding.pa_decode_q8(out, q, layer.k, layer.v, layer.scales, tables.cuda(), lens, length, length, 0,
                             0.09, ws)
    else:
        binding.pa_decode_window(out, q, layer.k, layer.v, tables.cuda(), lens, length, length, 0, 0.09, ws)
    ref, mass = attend64(q, k, v, [length - 1], length, 0, 0.09)
    bound = attention_bound(ref, mass, BF16, F16 if codes else BF16, float(v.abs().max()), length)
    assert bool(((out.double() - ref).abs() <= bound).all())
    if not codes:
        q, out = turned[-n:].contiguous(), torch.empty_like(turned[-n:])
        binding.pa_prefill_window(out, q, layer.k, layer.v, tables.cuda(), lens, length,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, 400, 4, 0.09)
        ref, mass = attend64(q, k, v, list(range(length - n, length)), 400, 4, 0.09)
        bound = attention_bound(ref, mass, BF16, BF16, float(v.abs().max()), length)
        assert bool(((out.double() - ref).abs() <= bound).all())
    assert binding.pa_get_last_device_error() == 0
