"""Plain 64-bit forms of the window, grouped-head and block-scaled operators,
and the error bounds that their kernels' roundings give."""
from __future__ import annotations

import numpy as np
import torch

from paged_kv_cache_481_b200 import binding

CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Paged:
    """Sequences of given lengths in a pool whose unused rows hold `junk`."""

    def __init__(self, lens, kv_heads, head_dim, block_size, dtype, seed, junk=float("nan"),
                 codes=None, spare=3):
        self.lens = list(lens)
        self.kvh, self.d, self.bs, self.dtype = kv_heads, head_dim, block_size, dtype
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        counts = [-(-n // block_size) for n in self.lens]
        self.nb = sum(counts) + spare
        ids = rng.permutation(self.nb)
        self.tables = np.full((len(self.lens), max(1, max(counts))), -1, np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        shape = (self.nb, kv_heads, block_size, head_dim)
        self.codes = codes
        if codes is None:
            self.k, self.v = self.randn(shape), self.randn(shape)
            self._spoil(self.k, junk)
            self._spoil(self.v, junk)
        else:
            kind, top = CODES[codes]
            x = [torch.randn(shape, generator=self.gen, device="cuda") * (top / 3.5) for _ in "kv"]
            x = [(t.round() if codes == "int8" else t).clamp(-top, top) for t in x]
            if codes == "e4m3":
                for t in x:
                    self._spoil(t, junk)
            self.k, self.v = (t.to(kind) for t in x)
            self.scales = (3.5 / top) * (0.05 + torch.rand((self.nb, kv_heads + kv_heads % 2, 2),
                                                           generator=self.gen, device="cuda"))

    def randn(self, shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(self.dtype)

    def _spoil(self, cache, junk):
        """Rows behind the last token, and blocks of no sequence, hold junk."""
        live = torch.zeros((self.nb, self.bs), dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for j in range(-(-n // self.bs)):
                live[self.tables[b, j], :min(self.bs, n - j * self.bs)] = True
        dead = ~live.cuda()
        cache.masked_fill_(dead[:, None, :, None], junk)

    def dev_tables(self):
        return torch.from_numpy(self.tables).cuda(), torch.tensor(self.lens, dtype=torch.int32,
                                                                  device="cuda")

    def context64(self, b):
        """K, V [L, KVH, D] of sequence b in 64 bits."""
        n = self.lens[b]
        t = torch.arange(n)
        block = torch.from_numpy(self.tables[b]).long()[t // self.bs].cuda()
        row = (t % self.bs).cuda()
        k, v = self.k.double() if self.codes is None else self.k.float().double(), None
        k = k[block, :, row]
        v = (self.v.double() if self.codes is None else self.v.float().double())[block, :, row]
        if self.codes is not None:
            s = self.scales.double()[block, :self.kvh]
            k, v = k * s[..., :1], v * s[..., 1:]
        return k, v


def attend64(q, k, v, positions, window, sinks, scale):
    """q [n, H, D] at `positions` over K, V [L, KVH, D]; (out, the same sum
    over |V|) in 64 bits.  Rows that see nothing are zero."""
    n, h, d = q.shape
    kvh = k.shape[1]
    t = torch.arange(k.shape[0], device=q.device)
    p = torch.as_tensor(positions, device=q.device)[:, None]
    seen = (t <= p) & ((t > p - window) | (t < sinks))
    some = seen.any(0)
    k, v, seen = k[some], v[some], seen[:, some]
    x = q.double().view(n, kvh, h // kvh, d)
    s = torch.einsum("ngrd,tgd->ngrt", x, k) * scale
    s = s.masked_fill(~seen[:, None, None], float("-inf"))
    w = torch.softmax(s, -1)
    w = torch.where(seen[:, None, None], w, torch.zeros_like(w))
    # a row sees its own position at least
    out = torch.einsum("ngrt,tgd->ngrd", w, v)
    mass = torch.einsum("ngrt,tgd->ngrd", w, v.abs())
    return out.reshape(n, h, d), mass.reshape(n, h, d)


def attention_bound(ref, mass, q_dtype, weight_dtype, worst_v=0.0, tokens=0):
    """Bound on |kernel - ref|, elementwise.
    The weights are rounded once to weight_dtype (relative u_w each, so u_w
    times the sum over |V|), the result once to q_dtype.  Scores are fp32 sums
    of D <= 128 products, each off by at most (D + 8) 2^-23 sum |q k| scale,
    under 2^-13 for the unit-variance rows used here (sum |q_d k_d| scale stays
    below 8); an error e of a score changes its weight by e and the total by as
    much, so 2^-12 of the mass, which also covers the 2^-22 of the
    exponential.  Weights are stored 2^7 times the softmax's or more, so those
    below fp16's normal range are off by half its last step, 2^-25, and so by
    2^-32 of the largest weight each (tokens, times the largest |V|)."""
    u_w, u_o = half_step(weight_dtype), half_step(q_dtype)
    inner = (u_w + 2.0 ** -12) * mass + tokens * 2.0 ** -32 * worst_v
    tiny = torch.finfo(q_dtype).smallest_normal * half_step(q_dtype)
    return inner + u_o * (ref.abs() + inner) + tiny


def decode(paged, q, window, sinks, scale, stream=None, workspace=None, max_len=None, out=None):
    tables, lens = paged.dev_tables()
    max_len = max(max(paged.lens), 1) if max_len is None else max_len
    out = torch.full_like(q, 7.0) if out is None else out
    ws = workspace if workspace is not None else binding.new_window_workspace(
        q.shape[0], q.shape[1], paged.kvh, paged.d)
    if paged.codes is None:
        binding.pa_decode_window(out, q, paged.k, paged.v, tables, lens, max_len, window, sinks,
                                 scale, ws, stream=stream)
    else:
        binding.pa_decode_q8(out, q, paged.k, paged.v, paged.scales, tables, lens, max_len, window,
                             sinks, scale, ws, stream=stream)
    return out


def check_decode(paged, q, out, window, sinks, scale, seqs=None):
    weight = torch.float16 if paged.codes is not None else paged.dtype
    for b in range(len(paged.lens)) if seqs is None else seqs:
        n = paged.lens[b]
        if n == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b]))
            continue
        k, v = paged.context64(b)
        ref, mass = attend64(q[b:b + 1], k, v, [n - 1], window, sinks, scale)
        bound = attention_bound(ref, mass, q.dtype, weight, float(v.abs().max()), n)
        err = (out[b:b + 1].double() - ref).abs()
        assert bool((err <= bound).all()), (b, n, float((err / bound).max()))


# ------------------------------------------------------------ rotation
def rope_table(max_position, rotary):
    angle = (torch.arange(max_position, device="cuda", dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64)
                           / max(rotary, 1)))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def rotate64(x, table, positions, interleaved):
    """(rotated rows, sum of the magnitudes that were added) in 64 bits."""
    x = x.double()
    if table is None:
        return x, x.abs()
    rot = table.shape[1]
    c, s = (t[:, None] for t in table.double()[positions].split(rot // 2, -1))
    y, mag = x.clone(), x.abs()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def rope_bound(ref, mag, dtype):
    """Two products and a sum, each rounded to fp32 (2^-24 of at most `mag`
    each, so 3 * 2^-24 mag and a little more), then one rounding to dtype."""
    inner = 4 * 2.0 ** -24 * mag
    tiny = torch.finfo(dtype).smallest_normal * half_step(dtype)
    return inner + half_step(dtype) * (ref.abs() + inner) + tiny
